"""Key weights of padded rows: a row whose log-sum-exp is -inf adds nothing, whatever its q holds."""
import math

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from test_gpu_cache_rows import Cache, check_weights, true_lse

pytestmark = pytest.mark.gpu


def junk(q, rows, heads=slice(None)):
    bad = q.clone()
    for i, r in enumerate(rows):
        bad[r, heads] = [math.nan, math.inf, -math.inf, torch.finfo(q.dtype).max][i % 4]
    return bad


@pytest.mark.parametrize("lens,W,Hq,Hkv,D,ps,dtype,dead", [
    ([300, 129], 3, 6, 2, 128, 16, "bf16", [1, 5]), ([700, 650], 96, 16, 8, 128, 32, "bf16", [0, 40, 95, 96, 130, 191]),
    ([257, 0, 90], 30, 32, 8, 128, 16, "fp16", range(60, 90)), ([200, 333], 17, 8, 1, 256, 64, "bf16", [16, 17, 33]),
    ([1000], 300, 2, 2, 64, 32, "bf16", list(range(250, 300)) + [3]), ([500], 1, 4, 2, 64, 32, "fp16", [0])])
def test_decode_rows_without_log_sum_exp(lens, W, Hq, Hkv, D, ps, dtype, dead):
    c = Cache(sum(lens) + W, lens, Hq, Hkv, D, ps, dtype)
    plan = c.decode_plan(W)
    q = c.rows(len(lens) * W)
    lse = true_lse(c, q, W, None)
    lse[list(dead)] = -math.inf
    bad = junk(q, dead)
    if Hq > Hkv and W > 1:  # one head of a row alone
        r = next(r for r in range(len(lens) * W) if r not in list(dead))
        lse[r, Hq - 1] = -math.inf
        bad[r, Hq - 1] = math.nan
    got = []
    for x in (q, bad):
        out = torch.full((len(lens), Hkv, max(lens)), -7.0, device="cuda")
        bsp.key_weights(plan, x, c.k, lse, 1 / math.sqrt(D), out, flags=bsp.FLAG_CHECK)
        got.append(out)
    check_weights(c, q, lse, W, None, 0, got[0])
    assert torch.equal(*got)


@pytest.mark.parametrize("cached,prompt,window,Hq,Hkv,D,causal", [
    ([0, 37], [200, 1], 0, 8, 2, 64, True), ([10, 130], [129, 260], 0, 16, 2, 128, True), ([9], [333], 40, 6, 2, 256, True),
    ([40, 0], [50, 150], 33, 12, 4, 128, False)])
def test_prefill_rows_without_log_sum_exp(cached, prompt, window, Hq, Hkv, D, causal):
    cached = np.array(cached, np.int32)
    lens = cached + np.array(prompt, np.int32)
    c = Cache(int(lens.sum()), lens, Hq, Hkv, D, 16, "bf16")
    plan = c.prefill_plan(cached, causal)
    n = int(sum(prompt))
    q = c.rows(n)
    lse = true_lse(c, q, None, cached, causal)
    dead = [0, prompt[0] - 1, n - 1, n - 2, n // 2]
    lse[dead] = -math.inf
    got = []
    for x in (q, junk(q, dead)):
        out = torch.full((len(lens), Hkv, int(lens.max())), -7.0, device="cuda")
        bsp.key_weights(plan, x, c.k, lse, 1 / math.sqrt(D), out, window=window, flags=bsp.FLAG_CHECK)
        got.append(out)
    check_weights(c, q, lse, None, cached, window, got[0], causal=causal)
    assert torch.equal(*got)


def test_fp8_rows_without_log_sum_exp():
    c = Cache(5, [300, 77], 16, 8, 128, 32, "bf16", e4m3=True)
    plan = c.decode_plan(40)
    q = c.rows(80, 0.25)
    lse = true_lse(c, q, 40, None, k_scale=0.5)
    dead = [0, 39, 40, 79, 20]
    lse[dead] = -math.inf
    got = []
    for x in (q, junk(q, dead)):
        out = torch.full((2, 8, 300), -7.0, device="cuda")
        bsp.key_weights_fp8(plan, x, c.k, lse, 1 / math.sqrt(128), 0.5, out, flags=bsp.FLAG_CHECK)
        got.append(out)
    check_weights(c, q, lse, 40, None, 0, got[0], k_scale=0.5)
    assert torch.equal(*got)


def test_other_log_sum_exps_keep_their_meaning():
    """+inf gives the row no weight, a NaN shows in every weight of its head, -inf beside them nothing."""
    c = Cache(6, [100], 3, 3, 64, 16, "bf16")
    plan = c.decode_plan(4)
    q = c.rows(4)
    lse = true_lse(c, q, 4, None)
    lse[1, 0], lse[2, 1], lse[3] = math.inf, math.nan, -math.inf
    out = torch.full((1, 3, 100), -7.0, device="cuda")
    bsp.key_weights(plan, junk(q, [3]), c.k, lse, 0.125, out, flags=bsp.FLAG_CHECK)
    assert torch.isnan(out[0, 1]).all()
    s = torch.einsum("rhd,hnd->rhn", q.double(), torch.from_numpy(np.stack(
        [c.k64[c.table[0, :7], h].reshape(-1, 64)[:100] for h in range(3)])).cuda()) * 0.125
    for h, rows in ((0, [0, 2]), (2, [0, 1, 2])):
        want = torch.exp(s[rows, h] - lse[rows, h].double()[:, None]).sum(0)
        # exponent off by 2^-18 at most (64 products below 32, log-sum-exps below 8), as much as the sum
        assert ((out[0, h].double() - want).abs() <= 2.0 ** -16 * want).all()
