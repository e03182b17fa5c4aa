"""Eviction by logical positions, repeated from restored pools: every call gives the rows that the plain restatement
chooses, bit for bit, for both sizes of the choosing CTAs and for single CTAs and clusters of them."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu


# (request, kv head) pairs: 1 and 4 are clusters of eight large CTAs, 160 single ones, 320 small ones; the last prompt
# is longer than the keys' order that fits in shared memory
@pytest.mark.parametrize("B,Hkv,P,keep,recent,times", [(1, 1, 9000, 2500, 300, 30), (2, 2, 3000, 900, 64, 30),
                                                       (20, 8, 2500, 800, 200, 15), (40, 8, 2000, 700, 100, 15),
                                                       (1, 1, 60000, 20000, 1000, 8)])
def test_repeated_with_positions(B, Hkv, P, keep, recent, times):
    D, ps, sinks = 64, 32, 4
    gen = torch.Generator(device="cuda").manual_seed(P)
    rng = np.random.default_rng(P)
    lens = rng.integers(P - P // 8, P + 1, B).astype(np.int32)
    lens[0] = P
    wide = -(-P // ps)
    table = rng.permutation(B * wide).astype(np.int32).reshape(B, wide)
    geo = bsp.geometry(Hkv, Hkv, D, ps, B * wide, "bf16")
    ws = bsp.Workspace(geo, B, 1, wide)
    plan = ws.plan(geo, B, 1, lens, np.zeros(B, np.int32), table)
    # a row's bytes say which row it is
    shape = (B * wide, Hkv, ps, D)
    k0 = torch.randint(-32768, 32767, shape, generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    v0 = torch.randint(-32768, 32767, shape, generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    weights = torch.exp(2 * torch.randn((B, Hkv, P), generator=gen, device="cuda"))
    # a cache that rows were evicted from before: positions in no order, with gaps
    positions = torch.from_numpy(np.stack([rng.permutation(3 * P)[:P] for _ in range(B * Hkv)]).reshape(B, Hkv, P).astype(np.int32)).cuda()
    keep_d = torch.full((B,), keep, dtype=torch.int32, device="cuda")
    w_h, p_h = weights.cpu().numpy(), positions.cpu().numpy()
    src = np.zeros((B, Hkv, keep), np.int64)
    for b in range(B):
        for h in range(Hkv):
            src[b, h] = steps.evict(w_h[b, h, :lens[b]], keep, sinks, recent, p_h[b, h, :lens[b]])
    want = torch.from_numpy(src).cuda()
    pages = torch.from_numpy(table.astype(np.int64)).cuda()
    b_, h_ = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    i_ = torch.arange(keep, device="cuda").expand(B, Hkv, keep)
    wk, wv = k0.view(torch.int16).clone(), v0.view(torch.int16).clone()
    for new, old in ((wk, k0), (wv, v0)):
        new[pages[b_, i_ // ps], h_, i_ % ps] = old.view(torch.int16)[pages[b_, want // ps], h_, want % ps]
    for _ in range(times):
        k, v = k0.clone(), v0.clone()
        kept = torch.full((B, Hkv, P), -5, dtype=torch.int32, device="cuda")
        wo, po = torch.full_like(weights, -5.0), torch.full_like(kept, -5)
        bsp.evict_prefix(plan, weights, keep_d, sinks, recent, k, v, kept, positions=positions, weights_out=wo, positions_out=po)
        assert torch.equal(kept[:, :, :keep].long(), want) and (kept[:, :, keep:] == -5).all()
        assert torch.equal(wo[:, :, :keep], weights.gather(2, want)) and torch.equal(po[:, :, :keep], positions.gather(2, want))
        assert torch.equal(k.view(torch.int16), wk) and torch.equal(v.view(torch.int16), wv)
    assert bsp.read_device_status(plan) == (0, 0)
