"""bsp_norm_rope_append_kv_fp8 where rows are skipped or hold zeros, infinities and NaN; bars as test_gpu_norm_append.py."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import cache
from test_gpu_norm_append import CASES, REL, TDT, Tokens, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [CASES[0], CASES[1], CASES[4]], ids=lambda c: f"{c[0]}-D{c[3]}")
@pytest.mark.parametrize("prefill", [False, True])
def test_skipped_tokens_and_extreme_rows(case, prefill):
    dtype, Hq, Hkv, D = case[:4]
    t = Tokens(dtype, Hq, Hkv, D, n=70, seed=4, prefill=prefill)
    norm, rope, want = setup(t, case)
    x = t.x.view(t.n, Hq + 2 * Hkv, D)
    x[0] = 0                                             # (eps alone under the root)
    x[1, Hq:, 3], x[2, Hq:, D - 1] = float("nan"), float("inf")
    x[5, Hq + Hkv:, 0] = -float("inf")
    x[6, Hq + Hkv:] = torch.finfo(TDT[dtype]).max
    t.dev.copy_(t.x)
    bad = [3, 17, 30, 31]
    t.slots[bad[:2]] = [-1, t.pages * t.ps]
    t.positions[bad[2:]] = [-1, 500]
    pools = [torch.full((t.pages, Hkv, t.ps, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q_out = torch.full((t.n, Hq, D), 3.0, dtype=TDT[dtype], device="cuda")
    bsp.norm_rope_append_kv_fp8(t.plan, norm, rope, t.pos(), t.q, t.k, t.v, t.loc(), *pools, k_mul=2.0, v_mul=0.5, q_out=q_out)
    assert bsp.read_device_status(t.plan)[1] == bsp.DEVFLAG_PAGE_INDEX | bsp.DEVFLAG_POSITION
    live = np.setdiff1d(np.arange(t.n), bad)
    t.positions = np.clip(t.positions, 0, 499)
    assert (q_out[bad] == 3.0).all()
    with np.errstate(all="ignore"):
        k, size = want("k")
        v = t.rows("v")
        delta = 2.0 * REL * size
    flat = [cache.DECODE[p.transpose(1, 2).reshape(-1, Hkv, D).cpu().numpy()] for p in pools]
    for got, x, d in ((flat[0], 2.0 * k, delta), (flat[1], 0.5 * v, np.zeros_like(v))):
        got, x, d = got[t.slots[live]], x[live], np.nan_to_num(d[live], nan=0.0, posinf=0.0)
        nan = np.isnan(x)
        assert nan.any() and np.isnan(got[nan]).all() and not np.isnan(got[~nan]).any()
        lo, hi = (cache.DECODE[cache.round_e4m3(np.where(nan, 0, y))] for y in (x - d, x + d))
        assert ((got >= lo) & (got <= hi) | nan).all()
    rest = np.setdiff1d(np.arange(t.pages * t.ps), t.slots[live])
    assert all((f[rest] == cache.DECODE[0x55]).all() for f in flat)
