"""Repeated calls of the bookkeeping, the key weights and the eviction agree bit for bit, as those of the processing and the
selection do."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,W,Hq,Hkv,D,most", [(40, 96, 16, 8, 128, 1500), (3, 30, 4, 1, 256, 4000), (1, 4, 2, 2, 64, 9000)])
@pytest.mark.parametrize("positioned", [False, True])
def test_weights_eviction_and_bookkeeping_repeat(B, W, Hq, Hkv, D, most, positioned):
    ps = 32
    gen = torch.Generator(device="cuda").manual_seed(most)
    rng = np.random.default_rng(most)
    lens = rng.integers(most // 2, most + 1, B).astype(np.int32)
    wide = -(-most // ps)
    table = rng.permutation(B * wide).astype(np.int32).reshape(B, wide)
    geo = bsp.geometry(Hq, Hkv, D, ps, B * wide, "bf16")
    ws = bsp.Workspace(geo, B, W, wide)
    plan = ws.plan(geo, B, W, lens, np.zeros(B, np.int32), table)
    k0, v0 = (torch.randn((B * wide, Hkv, ps, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B * W, Hq, D), generator=gen, device="cuda").bfloat16()
    lse = torch.randn((B * W, Hq), generator=gen, device="cuda") + 8
    positions = None
    if positioned:
        positions = torch.stack([torch.randperm(most, generator=gen, device="cuda") for _ in range(B * Hkv)]).view(B, Hkv, most).int()
    keep = torch.from_numpy(rng.integers(1, most // 2, B).astype(np.int32)).cuda()
    parents = torch.randint(0, W, (B, W), generator=gen, dtype=torch.int32, device="cuda")
    ci0 = torch.randint(0, W, (B, W, most + 1), generator=gen, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(15):
        k, v, ci = k0.clone(), v0.clone(), ci0.clone()
        w = torch.zeros((B, Hkv, most), device="cuda")
        kept = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
        bsp.key_weights(plan, q, k, lse, D ** -0.5, w)
        bsp.evict_prefix(plan, w, keep, 4, 50, k, v, kept, positions=positions)
        bsp.beam_advance(plan, parents, parents, ci)
        got = [w.view(torch.int32), kept, k.view(torch.int16), v.view(torch.int16), ci]
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert bsp.read_device_status(plan) == (0, 0)


def test_weights_beside_the_attention_of_another_step():
    """Both hold tensor memory: on two streams at once each gives what it gives alone."""
    def make(seed, B, W, P, Hq, Hkv, D):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        wide = -(-P // 32)
        geo = bsp.geometry(Hq, Hkv, D, 32, B * wide, "bf16")
        ws = bsp.Workspace(geo, B, W, wide)
        plan = ws.plan(geo, B, W, np.full(B, P, np.int32), np.zeros(B, np.int32), np.arange(B * wide, dtype=np.int32).reshape(B, wide))
        k, v = (torch.randn((B * wide, Hkv, 32, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn((B * W, Hq, D), generator=gen, device="cuda").bfloat16()
        out = torch.empty_like(q), torch.empty((B * W, Hq), device="cuda"), torch.zeros((B, Hkv, P), device="cuda")
        attend = lambda s: bsp.decode_attn(plan, q, k, v, None, None, D ** -0.5, out[0], out[1], stream=s)  # noqa: E731
        weigh = lambda s: bsp.key_weights(plan, q, k, out[1], D ** -0.5, out[2], stream=s)  # noqa: E731
        return ws, plan, attend, weigh, out

    steps_ = [make(1, 16, 30, 900, 16, 8, 128), make(2, 8, 96, 1200, 8, 4, 64)]
    want = []
    for _, _, attend, weigh, out in steps_:
        attend(None)
        weigh(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    (_, _, attend_a, weigh_a, _), (_, _, attend_b, weigh_b, _) = steps_
    for _ in range(100):
        attend_a(streams[0])
        weigh_b(streams[1])
        weigh_a(streams[0])
        attend_b(streams[1])
    torch.cuda.synchronize()
    for (_, plan, _, _, out), w in zip(steps_, want):
        assert bsp.read_device_status(plan) == (0, 0)
        assert all(torch.equal(a, b) for a, b in zip(out, w))
