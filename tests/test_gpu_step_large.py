"""The operators around a step where offsets pass 31 bits: logits of more than 2^31 elements, pools of more than 2^31
elements whose first and last pages are used."""
import math

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
def test_logits_of_more_than_2_31_elements(masked):
    B, W, V, K = 38, 96, 600_001, 50
    R = B * W
    assert R * V > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(8)
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    plan = ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))
    x = torch.empty((R, V), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rows = [0, 1, R // 2, R - 2, R - 1]
    raw = {r: x[r].double().cpu().numpy() for r in rows}
    tokens = torch.randint(0, V, (R, 6), generator=gen, dtype=torch.int32, device="cuda")
    token_len = torch.full((R,), 6, dtype=torch.int32, device="cuda")
    rep, temp = torch.full((B,), 1.5, device="cuda"), torch.full((B,), 0.5, device="cuda")
    mask = index = allowed = None
    if masked:
        allowed = np.random.default_rng(1).random((3, V)) < 0.02
        mask = torch.from_numpy(steps.pack_mask(allowed)).cuda()
        index = (torch.arange(R, device="cuda") % 3).to(torch.int32)
    lse = torch.empty(R, device="cuda")
    bsp.process_logits(plan, x, bsp.LogitsParams(tokens=tokens, token_len=token_len, repetition_penalty=rep,
                                                 temperature=temp, mask=mask, mask_index=index), lse=lse)
    for r in rows:
        want = steps.process_row(raw[r], (), tokens[r].cpu().numpy(), 1.5, None, None, (), 0.5,
                                 None if allowed is None else allowed[r % 3])
        got = x[r].double().cpu().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(fin, np.isfinite(got))
        # one rounding to bf16, half a step, after fp32 operations
        assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -8 * 1.001 * np.abs(want[fin]) + 1e-30).all()
        # fp32 sums of positive terms in some hundred additions per thread, and the exponentials' few steps
        assert abs(float(lse[r]) - steps.log_sum_exp(got)) <= 5e-5
    cum = torch.randn((B, W), generator=gen, device="cuda")
    scores = torch.empty((B, K), device="cuda")
    parents, chosen = (torch.empty((B, K), dtype=torch.int32, device="cuda") for _ in range(2))
    bsp.beam_select(plan, x, lse, cum, scores, parents, chosen, bsp.beam_select_workspace(B, W, V, K), mask=mask,
                    mask_index=index)
    assert bsp.read_device_status(plan) == (0, 0)
    for b in (0, B - 1):
        sl = slice(b * W, (b + 1) * W)
        s = (x[sl].float() - lse[sl, None]) + cum[b, :, None]
        top, flat = torch.sort(s.view(-1), descending=True, stable=True)  # equal scores: the lower place first
        top, flat = top[:K], flat[:K]
        assert torch.equal(scores[b], top)
        assert torch.equal(parents[b].long(), flat // V) and torch.equal(chosen[b].long(), flat % V)
        del s, top, flat


def test_pools_of_more_than_2_31_elements():
    Hq, Hkv, D, ps, pages, W = 16, 8, 128, 64, 33_000, 3
    assert pages * Hkv * ps * D > 2 ** 31
    lens, keep = np.array([300, 500], np.int32), [130, 77]
    table = np.full((2, 8), -1, np.int32)
    table[0, :5] = [pages - 1, 3, pages - 7, 32_769, 0]
    table[1, :8] = [32_768, pages - 2, 32_767, 5, pages - 9, 1, 32_900, 2]
    gen = torch.Generator(device="cuda").manual_seed(3)
    pools = [torch.zeros((pages, Hkv, ps, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    used = torch.from_numpy(table[table >= 0].astype(np.int64)).cuda()
    for p in pools:
        p[used] = torch.randn((len(used), Hkv, ps, D), generator=gen, device="cuda").bfloat16()
    geo = bsp.geometry(Hq, Hkv, D, ps, pages, "bf16")
    ws = bsp.Workspace(geo, 2, W, 8)
    plan = ws.plan(geo, 2, W, lens, np.zeros(2, np.int32), table)
    q = torch.randn((2 * W, Hq, D), generator=gen, device="cuda").bfloat16()
    scale = 1 / math.sqrt(D)

    def rows(pool, b):  # [Hkv, n, D] fp64
        ids = torch.from_numpy(table[b, :-(-lens[b] // ps)].astype(np.int64)).cuda()
        return pool[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :lens[b]].double().cpu().numpy()

    before = [[rows(p, b) for p in pools] for b in range(2)]
    lse = torch.zeros((2 * W, Hq), device="cuda") + 4.0
    weights = torch.zeros((2, Hkv, 500), device="cuda")
    bsp.key_weights(plan, q, pools[0], lse, scale, weights)
    kept = torch.full((2, Hkv, 500), -1, dtype=torch.int32, device="cuda")
    bsp.evict_prefix(plan, weights, torch.tensor(keep, dtype=torch.int32, device="cuda"), 2, 9, pools[0], pools[1], kept)
    assert bsp.read_device_status(plan) == (0, 0)
    q64, l64, w = q.double().cpu().numpy(), lse.double().cpu().numpy(), weights.cpu().numpy()
    for b, n in enumerate(lens):
        sl, after = slice(b * W, (b + 1) * W), [rows(p, b) for p in pools]
        for h in range(Hkv):
            heads = slice(2 * h, 2 * h + 2)
            want = steps.key_weights(q64[sl, heads], before[b][0][h], l64[sl, heads], scale)
            # the product's fp32 sums are off by 1e-5 of the exponent at most, the exponentials by less
            assert np.allclose(w[b, h, :n], want, rtol=1e-4, atol=0)
            src = steps.evict(w[b, h, :n], keep[b], 2, 9)
            assert np.array_equal(kept[b, h, :keep[b]].cpu().numpy(), src)
            for old, new in zip(before[b], after):
                assert np.array_equal(new[h, :keep[b]], old[h, src]) and np.array_equal(new[h, keep[b]:], old[h, keep[b]:])
