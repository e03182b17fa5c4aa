"""Exponent bytes that no append writes (of scales made elsewhere): the attention reads 0 as 0 and others as the nearest of
its range, 1 .. 142 over bf16 and 112 .. 134 over fp16, and so do the appends and forks that go on with such blocks. Values
are exact here: rows without a norm or rotation, power-of-two scales, codes compared bit for bit.
"""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, synth
from oracle import cache
from test_gpu_norm_append import Tokens
from test_gpu_pages import Forked

pytestmark = pytest.mark.gpu

RANGE = {"bf16": (1, 142), "fp16": (112, 134)}
BYTES = {"bf16": [1, 2, 14, 26, 27, 120, 141, 142, 143, 200, 254, 255], "fp16": [1, 60, 100, 111, 112, 120, 133, 134, 135, 142, 200, 255]}


def as_read(e, dtype):
    e = np.asarray(e, np.int64)
    return np.where(e == 0, 0, np.clip(e, *RANGE[dtype]))


def raised(codes, old, new):
    """Codes of exponent `old` at exponent `new`."""
    return cache.round_e4m3(cache.DECODE[codes] * 2.0 ** (int(old) - int(new)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("run", [1, 3])
def test_appends_go_on_with_foreign_exponents(dtype, prefill, run):
    """Runs of new rows behind 3 rows of a block of 8, small, ordinary and large beside each of the bytes."""
    values = BYTES[dtype]
    sizes = [2.0 ** -12, 1.0, 2.0 ** 12]
    blocks = len(values) * len(sizes)
    Hkv, D, ps, block = 2, 64, 16, 8
    t = Tokens(dtype, 2, Hkv, D, ps=ps, pages=blocks, n=blocks * run, seed=1, prefill=prefill)
    t.slots = (np.arange(blocks)[:, None] * ps + 3 + np.arange(run)).ravel().astype(np.int32)
    size = np.tile(np.repeat(sizes, run), len(values))
    t.x.copy_((torch.randn(t.x.shape, generator=torch.Generator().manual_seed(2)) * torch.from_numpy(size)[:, None]).to(t.x.dtype))
    t.dev.copy_(t.x)
    gen = torch.Generator().manual_seed(3)
    codes = [synth.e4m3_codes((blocks, Hkv, ps, D), gen, exp_mean=9, exp_sd=3) for _ in range(2)]
    old = np.repeat(np.array(values, np.uint8), len(sizes))
    exps = np.full((blocks, Hkv, ps // block), 9, np.uint8)
    exps[:, :, 0] = old[:, None]
    pools = [c.cuda() for c in codes]
    scales = bsp.BlockScales(t.geo, block, k=torch.from_numpy(exps).cuda(), v=torch.from_numpy(exps).cuda())
    bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, t.loc(), *pools, scales)
    assert bsp.read_device_status(t.plan) == (0, 0)
    for which, before, after, got in (("k", codes[0], pools[0], scales.k), ("v", codes[1], pools[1], scales.v)):
        x, after, got = t.rows(which), after.cpu().numpy(), got.cpu().numpy()
        want, we = before.numpy().copy(), exps.copy()
        for b in range(blocks):
            held = int(as_read(old[b], dtype))
            for h in range(Hkv):
                rows = x[b * run:(b + 1) * run, h]
                e = max(cache.exponent(np.abs(rows).max(), dtype), held)
                we[b, h, 0] = e
                if e > held:
                    want[b, h, :3] = raised(want[b, h, :3], held, e)
                want[b, h, 3:3 + run] = cache.round_e4m3(rows * 2.0 ** (127 - e))
        np.testing.assert_array_equal(got, we)
        np.testing.assert_array_equal(cache.DECODE[after], cache.DECODE[want])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forked_rows_of_foreign_exponents(dtype):
    block, Hkv = 8, 3
    f = Forked(prompt=[40, 21, 35, 3], tail=[8, 7, 3, 5], ps=16, forks=4, Hkv=Hkv, dtype=dtype, kv_dtype=bsp.KV_DTYPE_E4M3, seed=6)
    gen = torch.Generator().manual_seed(9)
    for p, d in zip(f.pools, f.dev):
        p.copy_(synth.e4m3_codes(p.shape, gen, exp_mean=9, exp_sd=3))
        d.copy_(p)
    pick = torch.tensor([0, *BYTES[dtype]], dtype=torch.uint8)
    exps = [pick[torch.randint(0, len(pick), (f.pages, Hkv, 16 // block), generator=gen)] for _ in range(2)]
    scales = bsp.BlockScales(f.geo, block, k=exps[0].cuda(), v=exps[1].cuda())
    _, out, served, _ = f.want()
    assert served.all()
    f.tables()
    f.rows(scales)
    assert bsp.read_device_status(f.plan) == (0, 0)
    seen = 0
    for pool, dev, e, ed in zip(f.pools, f.dev, exps, (scales.k, scales.v)):
        old, oe, got, ge = pool.numpy(), as_read(e.numpy(), dtype), dev.cpu().numpy(), ed.cpu().numpy()
        for r, rows in enumerate(f.sources()):
            mine = {}
            for pos, page in rows:
                mine.setdefault((out[r, pos // 16], pos % 16 // block), []).append((pos % 16, page))
            for (page, q), held in mine.items():
                for h in range(Hkv):
                    top = max(int(oe[src, h, q]) for _, src in held)
                    assert int(ge[page, h, q]) == top
                    for s, src in held:
                        a = int(oe[src, h, q])
                        if top:   # (under 0 the codes are read as 0)
                            want = raised(old[src, h, s], a, top) if a else np.zeros(f.D, np.uint8)
                            np.testing.assert_array_equal(cache.DECODE[got[page, h, s]], cache.DECODE[want])
                            seen += a != top
    assert seen > 20
