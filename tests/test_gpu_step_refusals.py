"""Calls around a step whose memory is not where the kernels could read it: refused before any launch."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu

INVALID, STALE = 1, 5


def state():
    B, W, V, K = 2, 3, 64, 4
    geo = bsp.geometry(2, 1, 64, 16, 4, "bf16")
    ws = bsp.Workspace(geo, B, W, 2)
    plan = ws.plan(geo, B, W, np.array([5, 20], np.int32), np.zeros(B, np.int32), np.array([[0, -1], [1, 2]], np.int32))
    i32 = torch.int32
    t = dict(x=torch.zeros((B * W, V), device="cuda"), lse=torch.zeros(B * W, device="cuda"), cum=torch.zeros((B, W), device="cuda"),
             scores=torch.zeros((B, K), device="cuda"), parents=torch.zeros((B, K), dtype=i32, device="cuda"),
             tokens=torch.zeros((B, K), dtype=i32, device="cuda"), sel=bsp.beam_select_workspace(B, W, V, K),
             ci=torch.zeros((B, W, 32), dtype=i32, device="cuda"), q=torch.zeros((B * W, 2, 64), dtype=torch.bfloat16, device="cuda"),
             row_lse=torch.zeros((B * W, 2), device="cuda"), k=torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda"),
             v=torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda"), w=torch.zeros((B, 1, 20), device="cuda"),
             keep=torch.tensor([2, 9], dtype=i32, device="cuda"), kept=torch.zeros((B, 1, 20), dtype=i32, device="cuda"))
    return ws, plan, t


CALLS = {
    "process": (lambda p, t: bsp.process_logits(p, t["x"], bsp.LogitsParams(), lse=t["lse"]), ["x", "lse"]),
    "select": (lambda p, t: bsp.beam_select(p, t["x"], t["lse"], t["cum"], t["scores"], t["parents"], t["tokens"], t["sel"]),
               ["x", "lse", "cum", "scores", "parents", "tokens", "sel"]),
    "advance": (lambda p, t: bsp.beam_advance(p, t["parents"], t["tokens"], t["ci"]), ["parents", "tokens", "ci"]),
    "weights": (lambda p, t: bsp.key_weights(p, t["q"], t["k"], t["row_lse"], 0.125, t["w"]), ["q", "k", "row_lse", "w"]),
    "evict": (lambda p, t: bsp.evict_prefix(p, t["w"], t["keep"], 1, 1, t["k"], t["v"], t["kept"]), ["w", "keep", "k", "v", "kept"]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_the_host_is_refused(name):
    """Each tensor in turn in pinned host memory, then the plan's workspace; the call itself is good."""
    ws, plan, t = state()
    call, used = CALLS[name]
    call(plan, t)
    for key in used:
        with pytest.raises(bsp.BspError) as e:
            call(plan, dict(t, **{key: t[key].cpu().pin_memory()}))
        assert e.value.status == INVALID, key
    moved = bsp.Plan.from_buffer_copy(plan)
    host = torch.zeros(4096, dtype=torch.uint8).pin_memory()
    moved.ws_device = host.data_ptr()
    with pytest.raises(bsp.BspError) as e:  # not the workspace that the plan was staged in
        call(moved, t)
    assert e.value.status == STALE
    call(plan, t)
    assert bsp.read_device_status(plan) == (0, 0)
