"""Selections whose scanning CTAs fill their buffers all the time: sorted rows, where every vector holds candidates of its
part, with beams that hold none and flagged states among the rows."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,W,V,K", [(2, 12, 40000, 24), (1, 96, 9000, 192), (3, 30, 20001, 512)])
def test_sorted_rows(B, W, V, K, masked):
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    plan = ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))
    rng = np.random.default_rng(V)
    x = torch.arange(V, device="cuda").float().repeat(B * W, 1) / 64 + torch.arange(B * W, device="cuda")[:, None] % 7
    lse = torch.zeros(B * W, device="cuda")
    cum = torch.zeros((B, W), device="cuda")
    cum[:, 1::5] = -np.inf  # beams without candidates between the others
    mask = index = allowed = None
    status = (0, 0)
    if masked:
        states = rng.random((4, V)) < np.array([0.03, 0.3, 0.9, 0.0])[:, None]
        index_h = rng.integers(-1, 4, B * W).astype(np.int32)
        allowed = np.where(index_h[:, None] >= 0, states[np.maximum(index_h, 0)], True)
        index_h[1] = 9  # past the masks: flagged, and the row unmasked
        allowed[1] = True
        allowed = allowed.reshape(B, W, V)
        mask, index = torch.from_numpy(steps.pack_mask(states)).cuda(), torch.from_numpy(index_h).cuda()
        status = (3, bsp.DEVFLAG_PAGE_INDEX)
    want = [steps.select(x[b * W:(b + 1) * W].cpu().numpy(), lse[:W].cpu().numpy(), cum[b].cpu().numpy(), K,
                         None if allowed is None else allowed[b]) for b in range(B)]
    sel = bsp.beam_select_workspace(B, W, V, K)
    for _ in range(20):
        s = torch.empty((B, K), device="cuda")
        p, t = (torch.empty((B, K), dtype=torch.int32, device="cuda") for _ in range(2))
        bsp.beam_select(plan, x, lse, cum, s, p, t, sel, mask=mask, mask_index=index)
        for b in range(B):
            assert all(np.array_equal(g[b].cpu().numpy(), w) for g, w in zip((s, p, t), want[b]))
    assert bsp.read_device_status(plan) == status
