"""NaN codes (0x7f, 0xff) of E4M3 pools, and NaN in 16-bit pools where splits and tails are merged: a NaN in a key that a row attends makes the row's output and log-sum-exp NaN, a
NaN in a value the output's element of that column, whatever kernel reads the tile; every other number stays bit for bit
what it is without the NaN. Blocks with an exponent of 0 keep their NaN codes too.
"""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, synth
from test_gpu_block_attn import BlockStep
from test_gpu_fp8_attn import Fp8Step

pytestmark = pytest.mark.gpu


class Step16:
    """The same with the case's 16-bit pools (their NaN is put by value)."""

    def __init__(self, case):
        self.case, wl = case, case.workload
        self.kd, self.vd, self.q = case.k_pool.cuda(), case.v_pool.cuda(), case.q.cuda()
        self.ci, self.beam_pages = torch.from_numpy(case.cache_indirection).cuda(), torch.from_numpy(case.beam_pages).cuda()
        self.o, self.lse = torch.empty_like(self.q), torch.empty(self.q.shape[:2], device="cuda")
        self.geo = bsp.geometry(wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.page_size, case.num_pages, wl.dtype)
        self.ws = bsp.Workspace(self.geo, wl.batch, wl.beam_width, case.prefix_pages.shape[1])
        self.plan = self.ws.plan(self.geo, wl.batch, wl.beam_width, case.prefix_len, case.tail_len, case.prefix_pages)

    def attend(self, flags=0):
        bsp.decode_attn(self.plan, self.q, self.kd, self.vd, self.beam_pages, self.ci, self.case.workload.head_dim ** -0.5, self.o, self.lse, flags=flags)


def step(scales, name, batch, kw, **lengths):
    """A BlockStep (block of 8 slots), an Fp8Step or a Step16. Beams that are even read beam 1's tail rows, the others beam 0's."""
    wl = synth.WORKLOADS[name].scaled(batch).with_(**kw)
    case = synth.make_case(wl, 900 + batch, full_step=False, device="cpu", **lengths)
    for b in range(batch):
        P, T = int(case.prefix_len[b]), int(case.tail_len[b])
        case.cache_indirection[b, ::2, P:P + T] = min(1, wl.beam_width - 1)
        case.cache_indirection[b, 1::2, P:P + T] = 0
    if scales == "plain":
        return Step16(case)
    return BlockStep(case, 901, 8) if scales == "blocks" else Fp8Step(case, 901, 0.5, 1.5)


def attend(st):
    st.o.fill_(-7.0)
    st.lse.fill_(-7.0)
    st.attend(flags=bsp.FLAG_CHECK)
    return st.o.clone(), st.lse.clone()


def prompt_slot(st, b, i):
    ps = st.case.workload.page_size
    return int(st.case.prefix_pages[b, i // ps]), i % ps


def tail_slot(st, b, src, t):
    ps, W = st.case.workload.page_size, st.case.workload.beam_width
    pos = int(st.case.prefix_len[b]) + t
    return int(st.case.beam_pages[b * W + src, pos // ps]), pos % ps


def put(st, pool, at, head, col, code, cleared):
    pool[at[0], head, at[1], col] = code
    if cleared:
        exps = st.scales.k if pool is st.kd else st.scales.v
        exps[at[0], head, at[1] // 8] = 0


def check(st, clean, got, rows=None, elements=None):
    """NaN where `rows` [R, Hq] (output and log-sum-exp) and `elements` [R, Hq, D] (output) say, else as before."""
    o, lse = got
    rows = torch.zeros_like(lse, dtype=torch.bool) if rows is None else rows.cuda()
    bad = rows[..., None].expand_as(o)
    if elements is not None:
        bad = bad | elements.cuda()
    assert torch.isnan(lse[rows]).all() and torch.equal(lse[~rows], clean[1][~rows])
    assert torch.isnan(o[bad]).all(), int((~torch.isnan(o[bad])).sum())
    assert torch.equal(o[~bad], clean[0][~bad])


# scales, workload, batch, changes to it: what a prompt tile is read by
TILES = [
    ("blocks", "qwen3_0p6b_b64_w30", 2, {}),                                        # one-set kernel
    ("blocks", "qwen3_0p6b_b64_w30", 2, dict(dtype="fp16")),
    ("blocks", "qwen3_0p6b_b64_w30", 2, dict(head_dim=64)),
    ("blocks", "qwen3_0p6b_b64_w30", 2, dict(beam_width=42)),                       # alternating tiles
    ("blocks", "qwen3_0p6b_b64_w30", 2, dict(beam_width=42, dtype="fp16")),
    ("blocks", "qwen3_0p6b_b64_w30", 2, dict(beam_width=42, head_dim=64)),
    ("blocks", "wide_beam_b128_w96", 2, {}),                                        # wide
    ("blocks", "wide_beam_b128_w96", 2, dict(dtype="fp16")),
    ("blocks", "wide_beam_b128_w96", 2, dict(head_dim=64)),
    ("tensor", "qwen3_0p6b_b64_w30", 2, {}),                                        # alternating tiles
    ("tensor", "qwen3_0p6b_b64_w30", 2, dict(dtype="fp16")),
    ("tensor", "qwen3_0p6b_b64_w30", 2, dict(head_dim=64)),
    ("tensor", "wide_beam_b128_w96", 2, {}),
    ("tensor", "wide_beam_b128_w96", 2, dict(head_dim=64)),
]
WHOLE = [  # enough requests that none is split: several tiles of a unit, the output written by the prompt kernel
    ("blocks", "qwen3_0p6b_b64_w30", 40, {}), ("blocks", "qwen3_0p6b_b64_w30", 40, dict(beam_width=42)),
    ("blocks", "wide_beam_b128_w96", 40, {}), ("tensor", "qwen3_0p6b_b64_w30", 40, {}),
]
names = lambda c: "-".join(map(str, (*c[:3], *(f"{k}={v}" for k, v in c[3].items()))))  # noqa: E731


@pytest.mark.parametrize("config", TILES + WHOLE, ids=names)
@pytest.mark.parametrize("cleared", [False, True])
def test_prompt_tiles(config, cleared):
    if cleared and config[0] != "blocks":
        pytest.skip("no block scales")
    batch = config[2]
    st = step(*config, prompt_lengths=[300, 200] * (batch // 2), tail_lengths=[2, 0] * (batch // 2))
    assert (st.plan.tail_requests == 0) == (batch == 40)
    wl = st.case.workload
    W, Hq, Hkv, D = wl.beam_width, wl.num_q_heads, wl.num_kv_heads, wl.head_dim
    G = Hq // Hkv
    # key, column, code; a head of request 0 each
    spots = [(0, 0, 0x7f), (130, 1, 0xff), (299, D - 1, 0x7f), (77, 36, 0xff)]
    for which in ("k", "v"):
        pool = st.kd if which == "k" else st.vd
        if cleared:
            for h, (key, _, _) in enumerate(spots):
                put(st, pool, prompt_slot(st, 0, key), h, 0, 0x31, True)
        clean = attend(st)
        assert torch.isfinite(clean[0]).all()
        kept = pool.clone()
        rows, elements = torch.zeros((batch * W, Hq), dtype=torch.bool), torch.zeros((batch * W, Hq, D), dtype=torch.bool)
        for h, (key, col, code) in enumerate(spots):
            put(st, pool, prompt_slot(st, 0, key), h, col, code, cleared)
            (rows if which == "k" else elements[..., col])[:W, h * G:(h + 1) * G] = True
        check(st, clean, attend(st), rows, elements)
        pool.copy_(kept)


@pytest.mark.parametrize("config", TILES, ids=names)
@pytest.mark.parametrize("cleared", [False, True])
def test_keys_of_gathered_tails(config, cleared):
    """Tail rows that the prompt kernel gathers: the beams that read the row, and no others."""
    if cleared and config[0] != "blocks":
        pytest.skip("no block scales")
    st = step(*config, prompt_lengths=[100, 65], tail_lengths=[3, 1])
    assert st.plan.tail_requests == 0
    wl = st.case.workload
    W, Hq, D = wl.beam_width, wl.num_q_heads, wl.head_dim
    G = Hq // wl.num_kv_heads
    spots = [(0, 0x7f), (1, 0xff), (D - 1, 0x7f)]
    if cleared:
        for h in range(len(spots)):
            put(st, st.kd, tail_slot(st, 0, 1, 1), h, 0, 0x31, True)
    clean = attend(st)
    rows = torch.zeros((2 * W, Hq), dtype=torch.bool)
    for h, (col, code) in enumerate(spots):
        put(st, st.kd, tail_slot(st, 0, 1, 1), h, col, code, cleared)
        rows[0:W:2, h * G:(h + 1) * G] = True
    check(st, clean, attend(st), rows)


MERGED = [(s, "qwen3_4b_fp16_d128", 6, kw) for s in ("blocks", "tensor", "plain") for kw in ({}, dict(dtype="bf16"), dict(head_dim=64))]
MERGED.append(("plain", "qwen3_4b_fp16_d128", 6, dict(head_dim=256)))


@pytest.mark.parametrize("config", MERGED, ids=names)
def test_tails_and_splits_that_are_merged(config):
    """The tail kernel: a NaN in some of a row's tail keys or in all of its keys, tail and splits, and in a value."""
    st = step(*config, prompt_lengths=[3000, 129, 0, 0, 1, 517], tail_lengths=[8, 5, 3, 0, 1, 1])
    assert st.plan.tail_requests >= 4
    wl = st.case.workload
    W, Hq, Hkv, D, ps = wl.beam_width, wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.page_size
    G = Hq // Hkv
    nan = float("nan") if config[0] == "plain" else 0x7f
    clean = attend(st)
    kept = st.kd.clone()
    rows = torch.zeros((6 * W, Hq), dtype=torch.bool)
    for b, h in ((0, 0), (1, 3), (2, 5)):   # a key of a long prompt's, a short prompt's and an empty prompt's tail
        at = tail_slot(st, b, 1, 2)
        st.kd[at[0], h, at[1], (h + D - 1) % D] = nan
        rows[b * W:(b + 1) * W:2, h * G:(h + 1) * G] = True
    for t in range(3):                      # every key that there is, of an empty prompt
        at = tail_slot(st, 2, 0, t)
        st.kd[at[0], 2, at[1], 7] = nan
    rows[2 * W + 1:3 * W:2, 2 * G:3 * G] = True
    for i in range(517):                    # ... of a prompt in splits (its tail's keys stay numbers)
        at = prompt_slot(st, 5, i)
        st.kd[at[0], 1, at[1], 0] = nan
    rows[5 * W:, G:2 * G] = True
    check(st, clean, attend(st), rows)
    st.kd.copy_(kept)
    elements = torch.zeros((6 * W, Hq, D), dtype=torch.bool)
    for b, col in ((0, 1), (1, D - 1), (2, 0)):
        at = tail_slot(st, b, 0, 1)
        st.vd[at[0], 4, at[1], col] = nan
        elements[b * W + 1:(b + 1) * W:2, 4 * G:5 * G, col] = True
    check(st, clean, attend(st), None, elements)


@pytest.mark.parametrize("scales", ["blocks", "tensor", "plain"])
def test_every_key_of_split_prompts_without_tails(scales):
    st = step(scales, "qwen3_4b_fp16_d128", 2, {}, prompt_lengths=[900, 700], tail_lengths=[0, 0])
    assert st.plan.tail_requests == 2
    wl = st.case.workload
    G = wl.num_q_heads // wl.num_kv_heads
    clean = attend(st)
    for i in range(900):
        at = prompt_slot(st, 0, i)
        st.kd[at[0], 2, at[1], 3] = float("nan") if scales == "plain" else 0xff
    rows = torch.zeros((2 * wl.beam_width, wl.num_q_heads), dtype=torch.bool)
    rows[:wl.beam_width, 2 * G:3 * G] = True
    check(st, clean, attend(st), rows)


@pytest.mark.parametrize("config", TILES, ids=names)
def test_values_of_gathered_tails(config):
    """A beam's NaN value stays with the rows that read it, though the tile holds all beams' rows: their elements of its
    column are NaN (the rest of them may be), the other rows are bit for bit what they were."""
    st = step(*config, prompt_lengths=[100, 65], tail_lengths=[3, 1])
    assert st.plan.tail_requests == 0
    wl = st.case.workload
    W, Hq, D = wl.beam_width, wl.num_q_heads, wl.head_dim
    G = Hq // wl.num_kv_heads
    clean = attend(st)
    spots = [(0, 0x7f), (1, 0xff), (D - 1, 0x7f)]
    rows = torch.zeros((2 * W, Hq), dtype=torch.bool)
    for h, (col, code) in enumerate(spots):
        put(st, st.vd, tail_slot(st, 0, 1, 2), h, col, code, False)
        rows[0:W:2, h * G:(h + 1) * G] = True
    o, lse = attend(st)
    for h, (col, _) in enumerate(spots):
        assert torch.isnan(o[0:W:2, h * G:(h + 1) * G, col]).all()
    other = ~rows.cuda()
    assert torch.equal(o[other], clean[0][other]) and torch.equal(lse[other], clean[1][other])


@pytest.mark.parametrize("kw", [{}, dict(dtype="fp16"), dict(head_dim=64)], ids=str)
def test_weights_of_keys(kw):
    """bsp_key_weights_fp8: the weight of a key that holds a NaN, and no other's."""
    st = step("tensor", "qwen3_0p6b_b64_w30", 2, kw, prompt_lengths=[300, 200], tail_lengths=[0, 0])
    wl = st.case.workload
    attend(st)

    def weigh():
        out = torch.full((2, wl.num_kv_heads, 300), -7.0, device="cuda")
        bsp.key_weights_fp8(st.plan, st.q, st.kd, st.lse, st.scale, st.k_scale, out, flags=bsp.FLAG_CHECK)
        return out

    clean = weigh()
    bad = torch.zeros(clean.shape, dtype=torch.bool)
    for h, (key, col, code) in enumerate([(0, 0, 0x7f), (130, 1, 0xff), (299, wl.head_dim - 1, 0x7f)]):
        put(st, st.kd, prompt_slot(st, 0, key), h, col, code, False)
        bad[0, h, key] = True
    got = weigh()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])
