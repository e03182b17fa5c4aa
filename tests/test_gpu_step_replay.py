"""Captured calls of the operators around a step, replayed after other plans were staged on their workspace: they follow
decode plans of their shape, and write nothing and say so under any other."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu

REFUSED = (5, bsp.DEVFLAG_GRAPH)


def capture(call):
    """The call in a graph, after one eager run of it on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


class Cache:
    """Pools, weights and tables for B requests of up to `most` prompt rows (tables of `stride` slots) under one
    workspace."""

    def __init__(self, B=2, W=3, Hq=4, Hkv=2, D=64, ps=16, most=2000, stride=None, rows=64, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.W, self.Hkv, self.D, self.ps = B, W, Hkv, D, ps
        wide = -(-most // ps)
        self.pages = B * wide
        self.table = np.random.default_rng(seed).permutation(self.pages).astype(np.int32).reshape(B, wide)
        self.geo = bsp.geometry(Hq, Hkv, D, ps, self.pages, "bf16")
        self.ws = bsp.Workspace(self.geo, B, 1500, wide)
        shape = (self.pages, Hkv, ps, D)
        self.k, self.v = (torch.randn(shape, generator=gen, device="cuda").bfloat16() for _ in range(2))
        stride = most if stride is None else stride
        self.w = torch.rand((B, Hkv, stride), generator=gen, device="cuda")
        self.keep = torch.full((B,), 20, dtype=torch.int32, device="cuda")
        self.kept = torch.full(self.w.shape, -5, dtype=torch.int32, device="cuda")
        self.wo = torch.full_like(self.w, -5.0)
        self.q = torch.randn((max(B * W, rows), Hq, D), generator=gen, device="cuda").bfloat16()
        self.lse = torch.full((max(B * W, rows), Hq), 5.0, device="cuda")
        self.sums = torch.full_like(self.w, -7.0)

    def decode(self, lens, tails=None):
        tails = np.zeros(self.B, np.int32) if tails is None else np.asarray(tails, np.int32)
        return self.ws.plan(self.geo, self.B, self.W, np.asarray(lens, np.int32), tails, self.table)

    def prefill(self, prompt, geo=None):
        return bsp.plan_prefill(geo or self.geo, self.B, np.zeros(self.B, np.int32), np.asarray(prompt, np.int32), self.table,
                                True, self.ws)

    def evict(self, plan):
        bsp.evict_prefix(plan, self.w, self.keep, 2, 5, self.k, self.v, self.kept, weights_out=self.wo)

    def weigh(self, plan):
        rows = plan.total_rows
        bsp.key_weights(plan, self.q[:rows], self.k, self.lse[:rows], 0.125, self.sums)

    def state(self):
        return [t.clone() for t in (self.k, self.v, self.kept, self.wo, self.sums)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def check_evicted(c, lens, before):
    """The pools and tables after an eviction from `before`, against the plain restatement."""
    k0, v0, kept0, wo0, _ = before
    w = c.w.cpu().numpy()
    wk, wv, kept, wo = k0.clone(), v0.clone(), kept0.clone(), wo0.clone()
    pages = torch.from_numpy(c.table.astype(np.int64)).cuda()
    for b, n in enumerate(lens):
        for h in range(c.Hkv):
            src = torch.from_numpy(steps.evict(w[b, h, :n], int(c.keep[b]), 2, 5).astype(np.int64)).cuda()
            i = torch.arange(len(src), device="cuda")
            kept[b, h, :len(src)] = src.int()
            wo[b, h, :len(src)] = c.w[b, h, src]
            for new, old in ((wk, k0), (wv, v0)):
                new[pages[b, i // c.ps], h, i % c.ps] = old[pages[b, src // c.ps], h, src % c.ps]
    assert same((c.k, c.v, c.kept, c.wo), (wk, wv, kept, wo))


@pytest.mark.parametrize("op", ["evict", "weigh"])
def test_prefill_plan_is_followed_by_none_but_itself(op):
    """A captured call on a prefill plan: the plan of the capture is served, any other refused - other lengths, the
    same lengths staged again, more tokens than q and lse hold, a decode plan."""
    c = Cache(rows=200)
    plan = c.prefill([100, 100])
    call = getattr(c, op)
    graph = capture(lambda: call(plan))
    assert bsp.read_device_status(plan) == (0, 0)
    before = c.state()
    graph.replay()
    assert bsp.read_device_status(plan) == (0, 0)
    after = c.state()
    if op == "evict":
        check_evicted(c, [100, 100], before)
    else:  # the eager call wrote the same
        assert same(before, after) and (after[4][:, :, :100] >= 0).all() and (after[4][:, :, 100:] == -7).all()
    for other in ([400, 900], [1500, 64], [3, 5], [60, 140], [100, 100], [0, 100]):
        p = c.prefill(other)
        before = c.state()
        graph.replay()
        assert bsp.read_device_status(p) == REFUSED, other
        assert same(before, c.state()), other
    p = c.decode([100, 100])
    graph.replay()
    assert bsp.read_device_status(p) == REFUSED and same(before, c.state())


@pytest.mark.parametrize("op", ["evict", "weigh"])
def test_decode_capture_refuses_prefill_plans_and_other_geometries(op):
    c = Cache(W=1, rows=200)
    plan = c.decode([100, 300])
    call = getattr(c, op)
    graph = capture(lambda: call(plan))
    p = c.prefill([1, 1])  # as many rows as the decode plan
    before = c.state()
    graph.replay()
    assert bsp.read_device_status(p) == REFUSED and same(before, c.state())
    # batch and beam width agree, the image's layout or the meaning of its page ids does not
    for Hq, Hkv, D, ps in ((4, 1, 64, 16), (8, 2, 64, 16), (4, 2, 128, 16), (4, 2, 64, 8)):
        geo = bsp.geometry(Hq, Hkv, D, ps, c.pages, "bf16")
        lens = np.array([100, 300], np.int32)
        p = c.ws.plan(geo, c.B, c.W, lens, np.zeros(2, np.int32), c.table)
        graph.replay()
        assert bsp.read_device_status(p) == REFUSED and same(before, c.state()), (Hq, Hkv, D, ps)
    p = c.decode([100, 300])
    graph.replay()
    assert bsp.read_device_status(p) == (0, 0)


@pytest.mark.parametrize("most", [3000, 60000])
def test_captured_eviction_follows_shorter_and_longer_prompts(most):
    """The capture holds the orders of its own prompts' keys in shared memory; longer ones are read again."""
    c = Cache(Hkv=1, Hq=1, most=most)
    plan = c.decode([200, 40])
    graph = capture(lambda: c.evict(plan))
    for lens, keep in (([200, 40], 30), ([19, 0], 5), ([700, 201], 150), ([most, most - 999], 1500), ([1, 33], 40)):
        plan = c.decode(lens)
        c.keep.fill_(keep)
        before = c.state()
        graph.replay()
        assert bsp.read_device_status(plan) == (0, 0)
        check_evicted(c, lens, before)


def test_replays_past_the_tables_and_with_tails():
    """Prompts longer than the rows of the captured tables, and tail rows: the request concerned is left, the others are
    served."""
    c = Cache(most=2000, stride=500)
    plan = c.decode([100, 300])
    evict = capture(lambda: c.evict(plan))
    weigh = capture(lambda: c.weigh(plan))
    # request 0 within the tables, request 1 past them
    plan = c.decode([90, 501])
    before = c.state()
    evict.replay()
    assert bsp.read_device_status(plan) == REFUSED
    check_evicted(c, [90, 0], before)
    c.sums.fill_(-7.0)
    weigh.replay()
    assert bsp.read_device_status(plan) == REFUSED
    assert (c.sums[0, :, :90] >= 0).all() and (c.sums[0, :, 90:] == -7).all() and (c.sums[1] == -7).all()
    # at the tables' last slot both are served
    plan = c.decode([90, 500])
    before = c.state()
    evict.replay()
    assert bsp.read_device_status(plan) == (0, 0)
    check_evicted(c, [90, 500], before)
    # a request with tail rows is not cut; its prompt keys are weighed all the same
    plan = c.decode([90, 300], [2, 0])
    before = c.state()
    evict.replay()
    assert bsp.read_device_status(plan) == REFUSED
    check_evicted(c, [0, 300], before)
    weigh.replay()
    assert bsp.read_device_status(plan) == (0, 0)


def test_captured_bookkeeping_past_its_tables():
    """cache_indirection or histories too short for the plan staged at the replay: the request is left as it is."""
    B, W = 2, 4
    geo = bsp.geometry(2, 1, 64, 32, 8, "bf16")
    ws = bsp.Workspace(geo, B, W, 4)
    pages = np.zeros((B, 4), np.int32)

    def make(P, T):
        return ws.plan(geo, B, W, np.asarray(P, np.int32), np.asarray(T, np.int32), pages)

    rng = np.random.default_rng(0)
    parents = rng.integers(0, W, (B, W)).astype(np.int32)
    chosen = rng.integers(0, 99, (B, W)).astype(np.int32)
    pd, cd = torch.from_numpy(parents).cuda(), torch.from_numpy(chosen).cuda()
    ci = torch.from_numpy(rng.integers(0, W, (B, W, 40)).astype(np.int32)).cuda()
    tok = torch.from_numpy(rng.integers(0, 99, (B * W, 6)).astype(np.int32)).cuda()
    n = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    plan = make([10, 20], [1, 2])
    graph = capture(lambda: bsp.beam_advance(plan, pd, cd, ci, None, tok, None, n))
    for P, T, left in (([10, 20], [3, 5], ()), ([10, 35], [3, 4], ()), ([10, 36], [3, 4], (1,)), ([10, 20], [6, 0], (0,)),
                       ([39, 40], [1, 0], (0, 1)), ([0, 39], [0, 0], ())):
        p = make(P, T)
        n.fill_(-1)
        ci0, tok0 = ci.cpu().numpy(), tok.cpu().numpy()
        graph.replay()
        assert bsp.read_device_status(p) == (REFUSED if left else (0, 0))
        for b in range(B):
            rows = slice(b * W, (b + 1) * W)
            wc, wt, wn = ci0[b], tok0[rows], -1
            if b not in left:
                wc, wt = steps.advance(parents[b], chosen[b], P[b], T[b], ci0[b], tok0[rows])
                wn = T[b] + 1
            assert np.array_equal(ci[b].cpu().numpy(), wc) and np.array_equal(tok[rows].cpu().numpy(), wt)
            assert (n[rows] == wn).all()
    p = ws.plan(geo, B, W - 1, np.array([10, 20], np.int32), np.zeros(B, np.int32), pages)
    before = [t.clone() for t in (ci, tok, n)]
    graph.replay()
    assert bsp.read_device_status(p) == REFUSED and same(before, (ci, tok, n))


def test_replays_under_page_ids_past_the_captured_pools():
    """A later plan of larger pools: rows on pages that the captured ones lack are neither read nor written, and flagged.
    (The pools here have twice the pages the capture was told of.)"""
    c = Cache(most=640)
    n = c.pages
    gen = torch.Generator(device="cuda").manual_seed(2)
    shape = (2 * n, c.Hkv, c.ps, c.D)
    c.k, c.v = (torch.randn(shape, generator=gen, device="cuda").bfloat16() for _ in range(2))
    plan = c.decode([300, 500])
    evict = capture(lambda: c.evict(plan))
    weigh = capture(lambda: c.weigh(plan))
    good = c.table.copy()
    c.keep.fill_(200)
    for odd in (1, 2):  # every second page of request 1 out of the capture's range, or all of them
        c.table = good.copy()
        c.table[1, ::3 - odd] += n
        geo = bsp.geometry(4, c.Hkv, c.D, c.ps, 2 * n, "bf16")
        plan = c.ws.plan(geo, c.B, c.W, np.array([300, 500], np.int32), np.zeros(2, np.int32), c.table)
        bsp.key_weights(plan, c.q[:6], c.k, c.lse[:6], 0.125, c.sums)
        want = c.sums.clone()
        c.sums.fill_(-7.0)
        weigh.replay()
        assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
        assert torch.equal(c.sums[0], want[0])
        on_known = torch.from_numpy(c.table[1, np.arange(500) // c.ps] < n).cuda()
        assert torch.equal(c.sums[1][:, :500][:, on_known], want[1][:, :500][:, on_known])
        before = c.state()
        evict.replay()
        assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
        w = c.w.cpu().numpy()
        for b, rows in enumerate((300, 500)):
            for h in range(c.Hkv):
                src = steps.evict(w[b, h, :rows], 200, 2, 5)
                assert np.array_equal(c.kept[b, h, :200].cpu().numpy(), src)
                to, of = c.table[b, np.arange(200) // c.ps], c.table[b, src // c.ps]
                moved = (to < n) & (of < n)
                src = torch.from_numpy(np.where(moved, src, np.arange(200))).cuda()
                pages = torch.from_numpy(c.table[b].astype(np.int64)).cuda()
                i = torch.arange(200, device="cuda")
                for new, old in ((c.k, before[0]), (c.v, before[1])):
                    assert torch.equal(new[pages[i // c.ps], h, i % c.ps], old[pages[src // c.ps], h, src % c.ps])
        assert torch.equal(c.k[n:], before[0][n:]) and torch.equal(c.v[n:], before[1][n:])
