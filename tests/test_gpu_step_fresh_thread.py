"""Each operator around a step as the first CUDA call of a host thread."""
import threading

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_first_call_of_a_thread(kv):
    B, W, V, K = 2, 3, 640, 4
    i32 = torch.int32
    geo = bsp.geometry(2, 1, 64, 16, 4, "bf16", kv_dtype=bsp.KV_DTYPE_E4M3 if kv == "e4m3" else 0)
    ws = bsp.Workspace(geo, B, W, 2)
    plan = ws.plan(geo, B, W, np.array([5, 20], np.int32), np.zeros(B, np.int32), np.array([[0, -1], [1, 2]], np.int32))
    x = torch.randn((B * W, V), device="cuda")
    lse, cum = torch.zeros(B * W, device="cuda"), torch.zeros((B, W), device="cuda")
    scores = torch.empty((B, K), device="cuda")
    parents, tokens = (torch.zeros((B, K), dtype=i32, device="cuda") for _ in range(2))
    sel, params = bsp.beam_select_workspace(B, W, V, K), bsp.LogitsParams()
    ci = torch.zeros((B, W, 32), dtype=i32, device="cuda")
    q = torch.zeros((B * W, 2, 64), dtype=torch.bfloat16, device="cuda")
    row_lse = torch.zeros((B * W, 2), device="cuda")
    pool = torch.zeros((4, 1, 16, 64), dtype=torch.uint8 if kv == "e4m3" else torch.bfloat16, device="cuda")
    k, v, w = pool, pool.clone(), torch.zeros((B, 1, 20), device="cuda")
    keep, kept = torch.tensor([2, 9], dtype=i32, device="cuda"), torch.zeros((B, 1, 20), dtype=i32, device="cuda")
    stream = torch.cuda.current_stream()

    def weigh():
        if kv == "e4m3":
            bsp.key_weights_fp8(plan, q, k, row_lse, 0.125, 0.5, w, stream=stream)
        else:
            bsp.key_weights(plan, q, k, row_lse, 0.125, w, stream=stream)

    calls = [lambda: bsp.process_logits(plan, x, params, lse=lse, stream=stream),
             lambda: bsp.beam_select(plan, x, lse, cum, scores, parents, tokens, sel, stream=stream),
             lambda: bsp.beam_advance(plan, parents, tokens, ci, stream=stream), weigh,
             lambda: bsp.evict_prefix(plan, w, keep, 1, 1, k, v, kept, stream=stream)]
    failed = []

    def work(call):
        try:
            call()
        except Exception as e:  # noqa: BLE001 - reported below
            failed.append((calls.index(call), repr(e)))

    for call in calls:
        t = threading.Thread(target=work, args=(call,))
        t.start()
        t.join()
    assert not failed, failed
    assert bsp.read_device_status(plan) == (0, 0)
    # every key's score is 0, every log-sum-exp 0: each of the six (row, head) pairs adds one
    assert (w[0, 0, :5] == 6).all() and (w[1, 0, :20] == 6).all()
    assert kept[1, 0, :9].tolist() == list(range(8)) + [19]
