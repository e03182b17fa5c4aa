"""Decode attention over E4M3 pools with block scales (bsp_decode_attn_fp8_blocks) against the fp64 oracle over the
16-bit values that codes and scales stand for (each product is a number of the q dtype, so these pools are exact).

Bar, with u half a step of the q dtype relative to the value (bf16 2^-8, fp16 2^-11): the output's rounding is u |O|, and
each probability's before the product with V is u p, so u A in all with A = sum p |v|; a score is a sum of D <= 128
products in fp32, off by at most 2 * 128 * 2^-24 * scale * sum |q k| < 2^-11 where scale * sum |q k| < 32 (held by these
inputs: |k| is about 1), which changes p by that much relative, another 2^-11 A; fp16 probabilities below 2^-14 lose
2^-25 each, against a row sum of at least 1: 2^-25 * keys * max |v|. The log-sum-exp is off by at most a score's error.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from beam_search_shared_gb300 import bsp, synth
from oracle import cache

pytestmark = pytest.mark.gpu


class BlockStep:
    """Device buffers of a case with E4M3 pools and block scales, and the plan of an E4M3 geometry."""

    def __init__(self, case, seed, block, lo=119, hi=124):
        wl = case.workload
        g = torch.Generator().manual_seed(seed)
        self.case, self.block = case, block
        pages, heads, ps, D = case.k_pool.shape
        # magnitudes near 50 with scales near 2^-6
        self.k8 = synth.e4m3_codes((pages, heads, ps, D), g, exp_mean=12.0, exp_sd=1.0)
        self.v8 = synth.e4m3_codes((pages, heads, ps, D), g, exp_mean=12.0, exp_sd=1.0)
        table = (pages, heads, ps // block)
        self.ke = torch.randint(lo, hi, table, generator=g, dtype=torch.uint8)
        self.ve = torch.randint(lo, hi, table, generator=g, dtype=torch.uint8)
        self.geo = bsp.geometry(wl.num_q_heads, wl.num_kv_heads, D, ps, case.num_pages, wl.dtype, kv_dtype=bsp.KV_DTYPE_E4M3)
        self.q = case.q.cuda()
        self.kd, self.vd = self.k8.cuda(), self.v8.cuda()
        self.scales = bsp.BlockScales(self.geo, block, k=self.ke.cuda(), v=self.ve.cuda())
        self.beam_pages = torch.from_numpy(case.beam_pages).cuda()
        self.ci = torch.from_numpy(case.cache_indirection).cuda()
        R = wl.batch * wl.beam_width
        self.o = torch.full((R, wl.num_q_heads, D), float("nan"), dtype=self.q.dtype, device="cuda")
        self.lse = torch.full((R, wl.num_q_heads), float("nan"), device="cuda")
        self.scale = 1.0 / math.sqrt(D)
        self.ws = bsp.Workspace(self.geo, max(1, wl.batch), wl.beam_width, case.prefix_pages.shape[1])
        self.plan = self.ws.plan(self.geo, wl.batch, wl.beam_width, case.prefix_len, case.tail_len, case.prefix_pages)

    def attend(self, flags=bsp.FLAG_CHECK):
        bsp.decode_attn_fp8_blocks(self.plan, self.q, self.kd, self.vd, self.scales, self.beam_pages, self.ci, self.scale,
                                   self.o, self.lse, flags=flags)

    def values(self):
        t = synth.TORCH_DTYPES[self.case.workload.dtype]
        out = []
        for codes, exps in ((self.k8, self.ke), (self.v8, self.ve)):
            v = cache.dequantise(codes.numpy(), exps.numpy())
            h = torch.from_numpy(v).to(t)
            assert (h.double().numpy() == v).all()  # exact
            out.append(h)
        return out

    def oracle(self, rows=None, magnitude=False):
        c, wl = self.case, self.case.workload
        k, v = self.values()
        return oracle.decode_attn(
            dtype=wl.dtype, B=wl.batch, W=wl.beam_width, Hq=wl.num_q_heads, Hkv=wl.num_kv_heads, D=wl.head_dim,
            ps=wl.page_size, num_pages=c.num_pages, prefix_len=c.prefix_len, tail_len=c.tail_len,
            prefix_pages=c.prefix_pages, beam_pages=c.beam_pages, cache_indirection=c.cache_indirection,
            q_bits=synth.bits(c.q), k_pool_bits=synth.bits(k), v_pool_bits=synth.bits(v.abs() if magnitude else v),
            scale=self.scale, rows=rows)

    def check(self, rows=None):
        O, L = self.oracle(rows)
        A, _ = self.oracle(rows, magnitude=True)
        sel = slice(None) if rows is None else rows
        o, lse = self.o[sel].double().cpu().numpy(), self.lse[sel].double().cpu().numpy()
        bf16 = self.case.workload.dtype == "bf16"
        u = 2.0 ** -8 if bf16 else 2.0 ** -11
        keys = int(self.case.prefix_len.max() + self.case.tail_len.max())
        tiny = 2.0 ** -24 if bf16 else 2.0 ** -25 * keys * float(np.abs(cache.dequantise(self.v8.numpy(), self.ve.numpy())).max())
        err, bound = np.abs(o - O), u * np.abs(O) + (u + 2.0 ** -11) * A * (1 + u) + tiny
        assert (err <= bound).all(), (err / bound).max()
        np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(L))
        fin = np.isfinite(L)
        assert (np.abs(lse[fin] - L[fin]) <= 2.0 ** -11).all(), np.abs(lse[fin] - L[fin]).max()


@pytest.mark.parametrize("name,batch,block,layout", [
    ("qwen3_0p6b_b64_w30", 6, 32, 1),    # alternating-tile kernel, a scale per page and head
    ("qwen3_0p6b_b64_w30", 3, 1, 1),     # a scale per token and head
    ("wide_beam_b128_w96", 2, 8, 2),     # wide kernel
    ("wide_beam_b128_w96", 1, 32, 2),
    ("qwen3_4b_fp16_d128", 5, 16, 1),    # fp16, tails up to 8
    ("qwen3_4b_fp16_d64", 4, 4, 1),      # head_dim 64: widened by the tail-tile warps
    ("tiny_b1_w4_d64", 1, 2, 1),
])
def test_matches_oracle(name, batch, block, layout):
    wl = synth.WORKLOADS[name].scaled(batch)
    st = BlockStep(synth.make_case(wl, 40 + batch, full_step=False, device="cpu"), 50 + batch, block)
    assert st.plan.layout == layout
    st.attend()
    st.check()


@pytest.mark.parametrize("kw,batch,block", [
    (dict(num_q_heads=24, num_kv_heads=8, beam_width=42), 3, 32),                               # G = 3
    (dict(num_q_heads=64, num_kv_heads=8, beam_width=20), 2, 16),                               # G = 8, wide
    (dict(page_size=8, beam_width=7), 4, 8),
    (dict(page_size=128), 3, 32),
    (dict(head_dim=64, num_q_heads=32, num_kv_heads=8, beam_width=40), 3, 8),                   # head_dim 64, wide
    (dict(head_dim=64, num_q_heads=16, num_kv_heads=8, beam_width=96, dtype="fp16"), 2, 32),
    (dict(head_dim=64, num_q_heads=1, num_kv_heads=1, beam_width=1), 5, 1),
])
def test_shapes(kw, batch, block):
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(batch).with_(**kw)
    st = BlockStep(synth.make_case(wl, 70 + batch, full_step=False, device="cpu"), 80 + batch, block)
    st.attend()
    st.check()


@pytest.mark.parametrize("block", [1, 16])
def test_split_prompts_long_tails_and_empty_requests(block):
    wl = synth.WORKLOADS["qwen3_4b_fp16_d128"].scaled(6)
    case = synth.make_case(wl, 91, full_step=False, device="cpu", prompt_lengths=[3000, 129, 0, 0, 1, 517],
                           tail_lengths=[8, 5, 3, 0, 8, 1])
    st = BlockStep(case, 92, block)
    assert st.plan.tail_requests > 0
    st.attend()
    st.check()


@pytest.mark.parametrize("dtype,lo,hi", [("bf16", 92, 143), ("fp16", 112, 121)])
def test_exponents_over_their_range(dtype, lo, hi):
    """Values from scales far apart (bf16 from 2^-35, fp16 from the smallest): K small enough for finite scores."""
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(2).with_(dtype=dtype)
    st = BlockStep(synth.make_case(wl, 21, full_step=False, device="cpu"), 22, 8, lo, hi)
    st.ke = torch.randint(112, 121, st.ke.shape, generator=torch.Generator().manual_seed(3), dtype=torch.uint8)
    st.scales.k.copy_(st.ke)
    st.attend()
    st.check()


def test_cleared_blocks_read_as_zero_keys():
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(2)
    st = BlockStep(synth.make_case(wl, 31, full_step=False, device="cpu"), 32, 16)
    gone = torch.rand(st.ke.shape, generator=torch.Generator().manual_seed(5)) < 0.3
    st.ke[gone], st.ve[gone] = 0, 0
    st.scales.k.copy_(st.ke)
    st.scales.v.copy_(st.ve)
    st.k8[(gone.repeat_interleave(16, 2))[..., None].expand_as(st.k8)] = 0  # codes of 0 in the oracle's pools
    st.v8[(gone.repeat_interleave(16, 2))[..., None].expand_as(st.v8)] = 0
    st.attend()  # (the device's codes are as they were)
    st.check()


def test_full_size_wide_beam_sampled():
    wl = synth.WORKLOADS["wide_beam_b128_w96"]
    st = BlockStep(synth.make_case(wl, 1100, full_step=False, device="cpu"), 1101, 8)
    st.attend()
    R = wl.batch * wl.beam_width
    rows = np.unique(np.concatenate([np.random.default_rng(9).integers(0, R, 24), [0, R - 1]])).astype(np.int32)
    st.check(rows)
    assert torch.isfinite(st.o).all()
    o, lse = st.o.clone(), st.lse.clone()
    st.attend(flags=0)
    assert torch.equal(o, st.o) and torch.equal(lse, st.lse)


def test_graph_mode_follows_later_plans():
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(4)
    case = synth.make_case(wl, 61, full_step=False, device="cpu", tail_lengths=[4, 2, 0, 3])
    st = BlockStep(case, 62, 32)
    st.attend(flags=bsp.FLAG_GRAPH)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.attend(flags=bsp.FLAG_GRAPH)
    for tails in ([4, 2, 0, 3], [1, 0, 4, 2]):
        case.tail_len[:] = np.minimum(tails, case.tail_len)
        st.plan = st.ws.plan(st.geo, wl.batch, wl.beam_width, case.prefix_len, case.tail_len, case.prefix_pages)
        st.o.fill_(float("nan"))
        g.replay()
        assert bsp.read_device_status(st.plan) == (0, 0)
        st.check()


def test_bad_pages_are_flagged_not_read():
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(2)
    case = synth.make_case(wl, 71, full_step=False, device="cpu", tail_lengths=[3, 3])
    st = BlockStep(case, 72, 32)
    st.ci[0, 5, int(case.prefix_len[0])] = wl.beam_width
    st.beam_pages[wl.beam_width + 1] = case.num_pages + 7
    with pytest.raises(bsp.BspError, match="PAGE_INDEX"):
        st.attend()
    assert torch.isfinite(st.o).all()


def test_refusals():
    wl = synth.WORKLOADS["qwen3_0p6b_b64_w30"].scaled(2)
    st = BlockStep(synth.make_case(wl, 81, full_step=False, device="cpu"), 82, 32)
    call = lambda sc, plan=st.plan, kd=st.kd: bsp.decode_attn_fp8_blocks(  # noqa: E731
        plan, st.q, kd, st.vd, sc, st.beam_pages, st.ci, st.scale, st.o, st.lse)
    host = bsp.BlockScales(st.geo, 32, device="cpu")
    with pytest.raises(bsp.BspError, match="INVALID_ARG"):
        call(host)
    with pytest.raises(ValueError):
        call(st.scales, kd=st.kd[:-1])
    geo2 = bsp.geometry(16, 8, 128, 32, st.case.num_pages + 1, "bf16", kv_dtype=bsp.KV_DTYPE_E4M3)
    with pytest.raises(ValueError):
        call(bsp.BlockScales(geo2, 32))
    geo16 = bsp.geometry(16, 8, 128, 32, st.case.num_pages, "bf16")
    ws = bsp.Workspace(geo16, 2, wl.beam_width, st.case.prefix_pages.shape[1])
    p16 = ws.plan(geo16, 2, wl.beam_width, st.case.prefix_len, st.case.tail_len, st.case.prefix_pages)
    with pytest.raises((ValueError, bsp.BspError)):
        call(st.scales, plan=p16)
    torch.cuda.synchronize()
    assert torch.isnan(st.o).all()


@pytest.mark.parametrize("name,dtype", [("qwen3_0p6b_b64_w30", "bf16"), ("qwen3_0p6b_b64_w30", "fp16"),
                                        ("wide_beam_b128_w96", "fp16"), ("qwen3_4b_fp16_d128", "fp16")])
@pytest.mark.parametrize("tails", [None, 8])
def test_blocks_that_were_never_written_read_as_zero_whatever_they_hold(name, dtype, tails):
    """Cleared exponents over codes of the largest magnitude: values of 0 give rows of exactly 0, keys of 0 scores of 0."""
    wl = synth.WORKLOADS[name].scaled(2).with_(dtype=dtype)
    st = BlockStep(synth.make_case(wl, 41, full_step=False, device="cpu",
                                   tail_lengths=None if tails is None else [tails] * wl.batch), 42, 8)
    st.kd.fill_(0x7e)
    st.vd.fill_(0x7e)
    st.scales.k.zero_()
    st.scales.v.zero_()
    st.attend()
    assert (st.o == 0).all()
    keys = torch.from_numpy(np.repeat(st.case.prefix_len + st.case.tail_len, wl.beam_width)).cuda()
    # a sum of up to 10^4 ones in fp32 parts, and two logarithms of a few units in the last place
    assert (st.lse - keys.double().log()[:, None]).abs().max() <= 2.0 ** -18
