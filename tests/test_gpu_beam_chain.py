"""The operators as a beam search uses them together: a prompt's prefill, its keys weighed by the last tokens and cut
to a budget in place, then decode steps over the shortened prompt whose logits are processed, whose beams are chosen,
and whose tables are advanced for the next step. Every stage is followed by a plain fp64 restatement that is fed the
library's own outputs of the stage before."""
import math

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu


def attend64(q, k, v, scale):
    """q [G, D], k, v [n, D] -> (o [G, D], lse [G])"""
    s = q @ k.T * scale
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    return e @ v / e.sum(-1, keepdims=True), (m[:, 0] + np.log(e.sum(-1)))


@pytest.mark.parametrize("Hq,Hkv,D,ps,dtype", [(8, 4, 128, 32, "bf16"), (6, 2, 64, 16, "fp16"), (4, 2, 256, 8, "bf16")])
def test_prefill_evict_and_beam_steps(Hq, Hkv, D, ps, dtype):
    B, W, V, window, steps_n = 2, 5, 999, 16, 4
    prompt = np.array([150, 90], np.int32)
    keep = np.array([64, 90], np.int32)  # the second request keeps everything
    rng = np.random.default_rng(D)
    gen = torch.Generator(device="cuda").manual_seed(D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    G, scale = Hq // Hkv, 1 / math.sqrt(D)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    # pages: the prompt's, shared by a request's beams, and a few of each beam's own for the tail
    n_prompt = -(-prompt // ps)
    own = -(-(ps - 1 + steps_n + 1) // ps) + 1
    total = int(n_prompt.sum()) + B * W * own
    ids = rng.permutation(total).astype(np.int32)
    table, at = np.full((B, int(n_prompt.max())), -1, np.int32), 0
    for b in range(B):
        table[b, :n_prompt[b]] = ids[at:at + n_prompt[b]]
        at += n_prompt[b]
    geo = bsp.geometry(Hq, Hkv, D, ps, total, dtype)
    ws = bsp.Workspace(geo, B, max(W, int(prompt.max())), table.shape[1])
    k_pool, v_pool = (torch.full((total, Hkv, ps, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))

    # ---- prefill, weights of the last tokens, eviction
    plan = bsp.plan_prefill(geo, B, np.zeros(B, np.int32), prompt, table, True, ws)
    R = int(prompt.sum())
    q, k_new, v_new = rand(R, Hq, D), rand(R, Hkv * D), rand(R, Hkv * D)
    slots = np.concatenate([table[b, np.arange(n) // ps] * ps + np.arange(n) % ps for b, n in enumerate(prompt)]).astype(np.int32)
    bsp.append_kv(plan, k_new, v_new, torch.from_numpy(slots).cuda(), k_pool, v_pool)
    o, lse = torch.empty((R, Hq, D), dtype=dt, device="cuda"), torch.empty((R, Hq), device="cuda")
    bsp.prefill_attn(plan, q, k_pool, v_pool, scale, o, lse)
    weights = torch.zeros((B, Hkv, int(prompt.max())), device="cuda")
    bsp.key_weights(plan, q, k_pool, lse, scale, weights, window=window)
    kept = torch.full(weights.shape, -1, dtype=torch.int32, device="cuda")
    bsp.evict_prefix(plan, weights, torch.from_numpy(keep).cuda(), 2, 8, k_pool, v_pool, kept)
    assert bsp.read_device_status(plan) == (0, 0)
    k64, v64 = (t.double().cpu().numpy().reshape(R, Hkv, D) for t in (k_new, v_new))
    w_h, kept_h, q64, l64 = weights.cpu().numpy(), kept.cpu().numpy(), q.double().cpu().numpy(), lse.double().cpu().numpy()
    keys = [[None] * Hkv for _ in range(B)]  # what the shortened cache holds
    row0 = 0
    for b, n in enumerate(prompt):
        rows = np.arange(row0 + n - window, row0 + n)
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            want = steps.key_weights(q64[rows][:, heads], k64[row0:row0 + n, h], l64[rows][:, heads], scale, np.arange(n - window, n) + 1)
            assert np.allclose(w_h[b, h, :n], want, rtol=1e-4, atol=1e-9)
            src = steps.evict(w_h[b, h, :n], keep[b], 2, 8)
            assert np.array_equal(kept_h[b, h, :keep[b]], src)
            keys[b][h] = (list(k64[row0 + src, h]), list(v64[row0 + src, h]))
        row0 += n

    # ---- decode over the first keep rows; the beams' tails in pages of their own
    beam_pages = np.full((B * W, int(n_prompt.max()) + own), -1, np.int32)
    for r in range(B * W):
        b = r // W
        full = keep[b] // ps
        beam_pages[r, :full] = table[b, :full]
        # the partial page's rows are read through the prompt's table; the tail's through the beam's own pages
        beam_pages[r, full:full + own] = ids[at:at + own]
        at += own
    bp = torch.from_numpy(beam_pages).cuda()
    max_seq = int(keep.max()) + steps_n + 1
    ci = torch.zeros((B, W, max_seq), dtype=torch.int32, device="cuda")
    tokens = torch.full((B * W, steps_n + 1), -1, dtype=torch.int32, device="cuda")
    token_len = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    cum = torch.zeros((B, W), device="cuda")
    cum[:, 1:] = -np.inf  # one live beam before the first choice
    ptok = torch.from_numpy(rng.integers(0, V, (B, 40)).astype(np.int32)).cuda()
    plen = torch.tensor([40, 7], dtype=torch.int32, device="cuda")
    rep, pres, temp = (torch.tensor(v, device="cuda") for v in ([1.3, 0.9], [0.4, 0.0], [0.8, 1.0]))
    states = rng.random((3, V)) < 0.4
    mask_index = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    params = bsp.LogitsParams(prompt_tokens=ptok, prompt_token_len=plen, tokens=tokens, token_len=token_len,
                              repetition_penalty=rep, presence_penalty=pres, temperature=temp,
                              mask=torch.from_numpy(steps.pack_mask(states)).cuda(), mask_index=mask_index)
    sel_ws = bsp.beam_select_workspace(B, W, V, 2 * W)
    scores = torch.empty((B, 2 * W), device="cuda")
    parents, chosen = (torch.empty((B, 2 * W), dtype=torch.int32, device="cuda") for _ in range(2))
    logits, row_lse = torch.empty((B * W, V), dtype=dt, device="cuda"), torch.empty(B * W, device="cuda")
    o, lse = torch.empty((B * W, Hq, D), dtype=dt, device="cuda"), torch.empty((B * W, Hq), device="cuda")
    tails = [[[] for _ in range(W)] for _ in range(B)]  # per beam: (k [Hkv, D], v) of its positions
    hist = [[[] for _ in range(W)] for _ in range(B)]
    head = rand(Hq * D, V).float() / math.sqrt(Hq * D)
    plan = None
    for t in range(steps_n):
        tl = np.full(B, t, np.int32)
        if plan is None:
            plan = ws.plan(geo, B, W, keep, tl, table)
        else:
            bsp.plan_update_tails(plan, tl)
        q = rand(B * W, Hq, D)
        if t:
            # the token chosen last: its K and V at the beam's own slot
            kn, vn = rand(B * W, Hkv * D), rand(B * W, Hkv * D)
            pos = np.repeat(keep + t - 1, W)
            loc = beam_pages[np.arange(B * W), pos // ps] * ps + pos % ps
            bsp.append_kv(plan, kn, vn, torch.from_numpy(loc.astype(np.int32)).cuda(), k_pool, v_pool)
            for r in range(B * W):
                tails[r // W][r % W].append((kn[r].double().cpu().numpy().reshape(Hkv, D), vn[r].double().cpu().numpy().reshape(Hkv, D)))
        bsp.decode_attn(plan, q, k_pool, v_pool, bp, ci, scale, o, lse)
        logits.copy_(o.float().view(B * W, -1) @ head * 4)
        raw = logits.clone()
        mask_index.copy_(torch.from_numpy(rng.integers(-1, 3, B * W).astype(np.int32)))
        cum0 = cum.clone()
        bsp.process_logits(plan, logits, params, lse=row_lse)  # in place
        bsp.beam_select(plan, logits, row_lse, cum, scores, parents, chosen, sel_ws)
        bsp.beam_advance(plan, parents, chosen, ci, None, tokens, None, token_len)
        cum = scores[:, :W].contiguous()
        assert bsp.read_device_status(plan) == (0, 0)

        q64, o64, l64 = (x.double().cpu().numpy() for x in (q, o, lse))
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
        for r in range(B * W):
            b, w = divmod(r, W)
            for h in range(Hkv):
                kk = np.array(keys[b][h][0] + [x[0][h] for x in tails[b][w]])
                vv = np.array(keys[b][h][1] + [x[1][h] for x in tails[b][w]])
                heads = slice(h * G, (h + 1) * G)
                wo, wl = attend64(q64[r, heads], kk, vv, scale)
                assert np.abs(l64[r, heads] - wl).max() <= 1e-4
                # probabilities and output rounded to the 16-bit type: a half step each of values up to max |v|
                assert np.abs(o64[r, heads] - wo).max() <= 2.5 * half * np.abs(vv).max()
        x64, rl = logits.double().cpu().numpy(), row_lse.cpu().numpy()
        raw64, mi = raw.double().cpu().numpy(), mask_index.cpu().numpy()
        sc, pa, ch = scores.cpu().numpy(), parents.cpu().numpy(), chosen.cpu().numpy()
        for r in range(B * W):
            b, w = divmod(r, W)
            want = steps.process_row(raw64[r], ptok[b, :int(plen[b])].cpu().numpy(), hist[b][w], float(rep[b]), None, float(pres[b]),
                                     (), float(temp[b]), states[mi[r]] if mi[r] >= 0 else None)
            fin = np.isfinite(want)
            assert np.array_equal(fin, np.isfinite(x64[r]))
            assert (np.abs(x64[r][fin] - want[fin]) <= half * 1.01 * np.abs(want[fin]) + 1e-6).all()
            assert abs(rl[r] - steps.log_sum_exp(x64[r])) <= 2e-5
        new_tails, new_hist = [], []
        for b in range(B):
            rows = slice(b * W, (b + 1) * W)
            ws_, wp, wt = steps.select(logits[rows].float().cpu().numpy(), rl[rows], cum0[b].cpu().numpy(), 2 * W)
            assert np.array_equal(sc[b], ws_) and np.array_equal(pa[b], wp) and np.array_equal(ch[b], wt)
            p = [wp[w] if wp[w] >= 0 else w for w in range(W)]
            new_tails.append([list(tails[b][p[w]]) for w in range(W)])
            new_hist.append([hist[b][p[w]] + [int(wt[w])] for w in range(W)])
        tails, hist = new_tails, new_hist
        assert tokens[:, :t + 1].cpu().numpy().tolist() == [hist[r // W][r % W] for r in range(B * W)]
        assert (token_len == t + 1).all()


def test_graph_of_a_step_follows_the_plan():
    """Weights, processing, selection and bookkeeping captured once and replayed after the tails grew, equal to the
    eager calls; a replay under a plan of another shape writes nothing and is flagged."""
    B, W, Hq, Hkv, D, ps, V = 2, 4, 4, 2, 64, 16, 500
    gen = torch.Generator(device="cuda").manual_seed(4)
    P = np.array([100, 37], np.int32)
    table = np.arange(14, dtype=np.int32).reshape(2, 7)
    geo = bsp.geometry(Hq, Hkv, D, ps, 20, "bf16")
    ws = bsp.Workspace(geo, B, W, 7)
    plan = ws.plan(geo, B, W, P, np.zeros(B, np.int32), table)
    k = torch.randn((20, Hkv, ps, D), generator=gen, device="cuda").bfloat16()
    q = torch.randn((B * W, Hq, D), generator=gen, device="cuda").bfloat16()
    lse = torch.full((B * W, Hq), 5.0, device="cuda")
    weights = torch.zeros((B, Hkv, 112), device="cuda")
    x = torch.randn((B * W, V), generator=gen, device="cuda")
    y, rl = torch.empty_like(x), torch.empty(B * W, device="cuda")
    cum = torch.zeros((B, W), device="cuda")
    sc = torch.empty((B, W), device="cuda")
    pa, ch = (torch.empty((B, W), dtype=torch.int32, device="cuda") for _ in range(2))
    ci = torch.zeros((B, W, 120), dtype=torch.int32, device="cuda")
    tok = torch.zeros((B * W, 9), dtype=torch.int32, device="cuda")
    sel_ws = bsp.beam_select_workspace(B, W, V, W)
    params = bsp.LogitsParams(temperature=torch.full((B,), 0.9, device="cuda"))

    def step(pl):
        bsp.key_weights(pl, q, k, lse, 0.125, weights)
        bsp.process_logits(pl, x, params, y, rl)
        bsp.beam_select(pl, y, rl, cum, sc, pa, ch, sel_ws)
        bsp.beam_advance(pl, pa, ch, ci, None, tok, None)

    def state():
        return [t.clone() for t in (weights, y, rl, sc, pa, ch, ci, tok)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(plan)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plan)
    for t in range(1, 4):
        P2 = P - t  # other prompt lengths too: a new plan of the same shape
        plan = ws.plan(geo, B, W, P2, np.full(B, t, np.int32), table)
        x.copy_(torch.randn((B * W, V), generator=gen, device="cuda"))
        ci0, tok0 = ci.clone(), tok.clone()
        weights.fill_(-1.0)
        graph.replay()
        assert bsp.read_device_status(plan) == (0, 0)
        got = state()
        ci.copy_(ci0)
        tok.copy_(tok0)
        weights.fill_(-1.0)
        step(plan)
        assert all(torch.equal(a, b) for a, b in zip(got, state()))
    other = ws.plan(geo, B, W - 1, P, np.zeros(B, np.int32), table)
    before = state()
    graph.replay()
    assert bsp.read_device_status(other) == (5, bsp.DEVFLAG_GRAPH)
    after = state()
    assert torch.equal(before[0], after[0]) and torch.equal(before[6], after[6]) and torch.equal(before[7], after[7])


def test_side_stream_and_two_plans():
    """Two steps with workspaces of their own on two streams at once give what each gives alone."""
    def make(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B, W, V, num = 4, 8, 20011, 16
        geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
        ws = bsp.Workspace(geo, B, W, 1)
        plan = ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))
        x = torch.randn((B * W, V), generator=gen, device="cuda").half()
        out = dict(y=torch.empty_like(x), l=torch.empty(B * W, device="cuda"), s=torch.empty((B, num), device="cuda"),
                   p=torch.empty((B, num), dtype=torch.int32, device="cuda"), t=torch.empty((B, num), dtype=torch.int32, device="cuda"))
        cum, sw = -torch.rand((B, W), generator=gen, device="cuda"), bsp.beam_select_workspace(B, W, V, num)
        params = bsp.LogitsParams(temperature=torch.rand(B, generator=gen, device="cuda") + 0.5)
        keep = (ws, params)

        def run(stream=None):
            bsp.process_logits(plan, x, params, out["y"], out["l"], stream=stream)
            bsp.beam_select(plan, out["y"], out["l"], cum, out["s"], out["p"], out["t"], sw, stream=stream)
            return keep
        return run, out

    pairs = [make(1), make(2)]
    want = []
    for run, out in pairs:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
        for v in out.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (run, _), s in zip(pairs, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, out), w in zip(pairs, want):
        assert all(torch.equal(out[k], w[k]) for k in w)
