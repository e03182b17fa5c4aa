"""Two host threads with plans, workspaces and streams of their own make calls of one operator that need different amounts of
shared memory: each call is served, whatever the other thread launches meanwhile."""
import threading

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu

CALLS = 20000


def process(big):
    """Tables of 2000 and of 8000 biases."""
    V, n = 20000, 8000 if big else 2000
    plan, ws = decode_plan(1, 2)
    x = torch.randn((2, V), device="cuda")
    out, lse = torch.empty_like(x), torch.empty(2, device="cuda")
    ids = torch.randperm(V, device="cuda")[None, :n].to(torch.int32).contiguous()
    params = bsp.LogitsParams(bias_tokens=ids, bias_values=torch.ones((1, n), device="cuda"))
    want = x.clone()
    want[:, ids[0].long()] += 1.0
    return lambda: bsp.process_logits(plan, x, params, out, lse), lambda: torch.equal(out, want), (ws, params)


def select(big):
    """Merges of 130 and of 35 KB."""
    W, V, K = (96, 32000, 512) if big else (4, 32000, 256)
    plan, ws = decode_plan(1, W)
    x = torch.randn((W, V), device="cuda")
    lse, cum = torch.zeros(W, device="cuda"), torch.zeros((1, W), device="cuda")
    s = torch.empty((1, K), device="cuda")
    p, t = (torch.empty((1, K), dtype=torch.int32, device="cuda") for _ in range(2))
    sel = bsp.beam_select_workspace(1, W, V, K)
    want = torch.topk(x.view(-1), K).values
    return lambda: bsp.beam_select(plan, x, lse, cum, s, p, t, sel), lambda: torch.equal(s[0], want), (ws, sel)


def advance(big):
    """Beams in the thousands."""
    W = 5000 if big else 1200
    plan, ws = decode_plan(1, W, tail=7)
    parents = torch.arange(W - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    tok = torch.randint(0, 99, (W, 8), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(tok)
    return (lambda: bsp.beam_advance(plan, parents, parents, tokens=tok, tokens_out=out),
            lambda: torch.equal(out[:, :7], tok.flip(0)[:, :7]), ws)


def weigh(big):
    """Blocks of 192 and of 8 query rows."""
    W, n, geo = (96 if big else 4), 500, bsp.geometry(2, 1, 64, 32, 16, "bf16")
    ws = bsp.Workspace(geo, 1, W, 16)
    plan = ws.plan(geo, 1, W, np.array([n], np.int32), np.zeros(1, np.int32), np.arange(16, dtype=np.int32)[None])
    k = torch.randn((16, 1, 32, 64), device="cuda").bfloat16()
    q = torch.zeros((W, 2, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((W, 2), device="cuda")
    out = torch.zeros((1, 1, n), device="cuda")
    return lambda: bsp.key_weights(plan, q, k, lse, 0.125, out), lambda: bool((out == 2.0 * W).all()), ws


def evict(big):
    """Orders of 40000 and of 9000 keys in shared memory."""
    n, keep = (40000 if big else 9000), 100
    pages = -(-n // 64)
    geo = bsp.geometry(1, 1, 64, 64, pages, "bf16")
    ws = bsp.Workspace(geo, 1, 1, pages)
    plan = ws.plan(geo, 1, 1, np.array([n], np.int32), np.zeros(1, np.int32), np.arange(pages, dtype=np.int32)[None])
    k, v = (torch.zeros((pages, 1, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.arange(n, device="cuda").float()[None, None].contiguous()
    kept = torch.zeros((1, 1, n), dtype=torch.int32, device="cuda")
    keep_d = torch.full((1,), keep, dtype=torch.int32, device="cuda")
    want = torch.arange(n - keep, n, device="cuda", dtype=torch.int32)
    return lambda: bsp.evict_prefix(plan, w, keep_d, 0, 0, k, v, kept), lambda: torch.equal(kept[0, 0, :keep], want), ws


def decode_plan(B, W, tail=0):
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    return ws.plan(geo, B, W, np.zeros(B, np.int32), np.full(B, tail, np.int32), np.zeros((B, 1), np.int32)), ws


@pytest.mark.parametrize("make", [process, select, advance, weigh, evict])
def test_two_threads(make):
    jobs = [make(False), make(True)]
    for call, check, _ in jobs:
        call()
        torch.cuda.synchronize()
        assert check()
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(call):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            try:
                for i in range(CALLS):
                    call()
                    if i % 100 == 99:
                        torch.cuda.current_stream().synchronize()
            except bsp.BspError as e:
                failed.append(str(e))

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(check() for _, check, _ in jobs)
