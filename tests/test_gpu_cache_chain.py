"""The cache's operators as a server uses them together: prompts written with normalised and rotated keys, beam steps that
append and attend, two beams of each request that go on as sequences of their own, the old sequences' pages given back,
the pool compacted, and the forks' next token. Over 16-bit pools and over E4M3 blocks with scales.

What the pools have to hold is restated in fp64 from the tokens alone, along each sequence's path, and the attention from
the values that the pools hold.

Bars. A stored 16-bit key is off by half a step, u |k| (bf16 2^-8, fp16 2^-11; fp16 below its smallest normal number 2^-14
has steps of 2^-24, so half of one is 2^-25 however small k is: 1.1117e-5 is rounded by 2.926e-8, more than 2^-11 of it),
and the 2^-20 (|x| + |y|) of the fp32 computation before it; values are copied. An E4M3 code is off by 2^-4 of its value, or below the smallest normal number
by half a step of 2^-9 times the scale; each time its block's scale grows (a power of two, so only codes that leave the
normal range are rounded again) another half step of the new scale, and half steps of growing scales add up to less than
a whole one of the last, 2^-9 s. Attention: as derived in test_gpu_block_attn.py, u |O| + (u + 2^-11) A with
A = sum p |v|, fp16 probabilities another 2^-25 keys max |v|; |q| and |k| of normalised rows keep scale * sum |q k| below
sqrt(D) * 1.3^2 < 20.
"""
import math

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import cache

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SMALL = {"bf16": 0.0, "fp16": 2.0 ** -25}
PROMPT = (45, 32, 7)   # the second ends with its page
BEAMS, STEPS, FORKS = 4, 4, 2


class Server:
    def __init__(self, dtype, Hq, Hkv, D, ps, block, seed=0):
        self.rs = np.random.RandomState(seed)
        self.dtype, self.Hq, self.Hkv, self.D, self.ps, self.block = dtype, Hq, Hkv, D, ps, block
        self.B, self.pages = len(PROMPT), 96
        self.geo = bsp.geometry(Hq, Hkv, D, ps, self.pages, dtype, bsp.KV_DTYPE_E4M3 if block else 0)
        t = torch.uint8 if block else TDT[dtype]
        fill = 0x7f if block else float("nan")   # whatever is read without having been written shows
        self.k_pool, self.v_pool = (torch.full((self.pages, Hkv, ps, D), fill, dtype=t, device="cuda") for _ in range(2))
        self.scales = bsp.BlockScales(self.geo, block) if block else None
        self.qw, self.kw = (torch.from_numpy(1 + 0.3 * (2 * self.rs.rand(D) - 1)).to(TDT[dtype]) for _ in range(2))
        self.norm = bsp.QkNorm(self.qw.cuda(), self.kw.cuda(), eps=1e-5)
        self.rope = bsp.Rope(128, D // 2, 1e4, scaling=bsp.RopeScaling("linear", 4.0))
        self.theta = cache.frequencies(D // 2, 1e4, "linear", 4.0)
        self.scale = 1 / math.sqrt(D)
        self.refs = torch.zeros(self.pages, dtype=torch.int32, device="cuda")
        self.flags = []

    def cuda(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def rows(self, n):
        """New tokens: one projection's output, its column slices, and the keys and values in fp64."""
        width = (self.Hq + 2 * self.Hkv) * self.D
        x = torch.from_numpy(self.rs.randn(n, width) * np.exp(0.5 * self.rs.randn(n, 1))).to(TDT[self.dtype])
        return x, x.cuda().split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)

    def stored(self, x, positions):
        """fp64 keys (and what a rounding error is relative to) and values of tokens x."""
        y = x.double().numpy()
        k = y[:, self.Hq * self.D:(self.Hq + self.Hkv) * self.D].reshape(-1, self.Hkv, self.D)
        v = y[:, (self.Hq + self.Hkv) * self.D:].reshape(-1, self.Hkv, self.D)
        k, size = cache.norm_rotate(k, self.kw.double().numpy(), float(np.float32(1e-5)), 0.0, positions, self.theta,
                                    self.D // 2, False)
        return k, size, v

    def append(self, plan, dev, positions, slots, q_out):
        q, k, v = dev
        pos, loc = self.cuda(positions.astype(np.int32)), self.cuda(slots.astype(np.int32))
        if self.block:
            bsp.append_kv_fp8_blocks(plan, k, v, loc, self.k_pool, self.v_pool, self.scales, norm=self.norm,
                                     rope=self.rope, positions=pos, q=q, q_out=q_out)
        else:
            bsp.norm_rope_append_kv(plan, self.norm, self.rope, pos, q, k, v, loc, self.k_pool, self.v_pool, q_out=q_out)

    def attend(self, plan, q, beam_pages, ci):
        o = torch.full((plan.total_rows, self.Hq, self.D), float("nan"), dtype=TDT[self.dtype], device="cuda")
        lse = torch.full((plan.total_rows, self.Hq), float("nan"), device="cuda")
        q = q.view(-1, self.Hq, self.D)
        if self.block:
            bsp.decode_attn_fp8_blocks(plan, q, self.k_pool, self.v_pool, self.scales, beam_pages, ci, self.scale, o, lse)
        else:
            bsp.decode_attn(plan, q, self.k_pool, self.v_pool, beam_pages, ci, self.scale, o, lse)
        self.flags.append(bsp.read_device_status(plan))
        return o, lse

    def held(self):
        """Values of the pools in fp64, and the blocks' scales at each slot."""
        if not self.block:
            return [(p.double().cpu().numpy(), None) for p in (self.k_pool, self.v_pool)]
        out = []
        for p, e in ((self.k_pool, self.scales.k), (self.v_pool, self.scales.v)):
            codes, exps = p.cpu().numpy(), e.cpu().numpy()
            out.append((cache.dequantise(codes, exps), np.repeat(cache.scale_of(exps), self.block, 2)))
        return out

    def check_rows(self, where, want):
        """The pools at [(page, slot)] against (keys, size, values) [n, Hkv, D]."""
        page, slot = np.array(where).T
        u = HALF[self.dtype]
        (k, ks), (v, vs) = self.held()
        k, v = k[page, :, slot], v[page, :, slot]
        near = 2.0 ** -20 * want[1]
        if self.block:
            for got, ref, s, d in ((k, want[0], ks, near), (v, want[2], vs, 0.0)):
                s = s[page, :, slot][..., None]
                assert (np.abs(got - ref) <= 2.0 ** -4 * (np.abs(ref) + d) + 2.0 ** -9 * s + d).all()
        else:
            assert (np.abs(k - want[0]) <= u * (np.abs(want[0]) + near) + near + SMALL[self.dtype]).all()
            assert (v == want[2]).all()

    def check_attention(self, o, lse, q, where):
        """Row r of o attends what the pools hold at where[r] = [(page, slot)]."""
        u = HALF[self.dtype]
        q = q.view(-1, self.Hq, self.D).double().cpu().numpy()
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        (kp, _), (vp, _) = self.held()
        G = self.Hq // self.Hkv
        for r, path in enumerate(where):
            page, slot = np.array(path).T
            for h in range(self.Hq):
                k, v = kp[page, h // G, slot], vp[page, h // G, slot]
                s = k @ q[r, h] * self.scale
                assert (np.abs(k) @ np.abs(q[r, h]) * self.scale).max() < 32
                e = np.exp(s - s.max())
                p = e / e.sum()
                A = p @ np.abs(v)
                bar = u * np.abs(p @ v) + (u + 2.0 ** -11) * A + 2.0 ** -25 * len(s) * np.abs(v).max()
                assert (np.abs(o[r, h] - p @ v) <= bar).all(), (r, h)
                assert abs(lse[r, h] - (s.max() + math.log(e.sum()))) <= 2.0 ** -11


def run(s):
    """The whole of it; what every stage left on the device, for comparison of two runs."""
    B, ps, W, P = s.B, s.ps, BEAMS, np.array(PROMPT, np.int32)
    kept = []
    ids = s.rs.permutation(s.pages)[:s.pages * 3 // 4].astype(np.int32)   # the rest is left for the forks
    take = iter(ids)
    cols = -(-int(P.max() + STEPS) // ps)
    prompt = np.full((B, cols), -1, np.int32)
    for b in range(B):
        for c in range(-(-int(P[b]) // ps)):
            prompt[b, c] = next(take)
    ws = bsp.Workspace(s.geo, B * FORKS, W, cols)

    # ---- prompts
    geo = bsp.geometry(s.Hq, s.Hkv, s.D, ps, s.pages, s.dtype)   # a prefill's plan is one of 16-bit pools
    first = bsp.Workspace(geo, B, int(P.sum()), cols)
    plan = bsp.plan_prefill(geo, B, np.zeros(B, np.int32), P, prompt, True, first)
    x, dev = s.rows(int(P.sum()))
    positions = np.concatenate([np.arange(n) for n in P])
    where = [(prompt[b, i // ps], i % ps) for b in range(B) for i in range(P[b])]
    q = torch.empty((len(where), s.Hq * s.D), dtype=TDT[s.dtype], device="cuda")
    s.append(plan, dev, positions, np.array([p * ps + i for p, i in where]), q)
    s.flags.append(bsp.read_device_status(plan))
    keys, size, values = s.stored(x, positions)
    s.check_rows(where, (keys, size, values))
    start = np.concatenate([[0], np.cumsum(P)])
    tokens = {(b, i): tuple(t[start[b] + i] for t in (keys, size, values)) for b in range(B) for i in range(P[b])}

    # ---- beam steps: a beam's own pages from the column of its first token on
    beam_pages = np.full((B * W, cols), -1, np.int32)
    for b in range(B):
        for w in range(W):
            for c in range(int(P[b]) // ps, -(-int(P[b] + STEPS) // ps)):
                beam_pages[b * W + w, c] = next(take)
    max_seq = cols * ps
    ci = np.full((B, W, max_seq), -1, np.int32)
    made = {}   # (request, beam, position): key, size, value
    for t in range(STEPS):
        # a beam goes on from a random one: its history is that one's, its new token its own
        parent = s.rs.randint(0, W, (B, W))
        for b in range(B):
            ci[b] = ci[b][parent[b]]
            ci[b, :, P[b] + t] = np.arange(W)
        plan = ws.plan(s.geo, B, W, P, np.full(B, t + 1, np.int32), prompt)
        x, dev = s.rows(B * W)
        at = np.repeat(P + t, W)
        where = [(beam_pages[r, at[r] // ps], at[r] % ps) for r in range(B * W)]
        q = torch.empty((B * W, s.Hq * s.D), dtype=TDT[s.dtype], device="cuda")
        s.append(plan, dev, at, np.array([p * ps + i for p, i in where]), q)
        new = s.stored(x, at)
        s.check_rows(where, new)
        for r in range(B * W):
            made[r // W, r % W, at[r]] = tuple(y[r] for y in new)
        dci, dpages = s.cuda(ci), s.cuda(beam_pages)
        o, lse = s.attend(plan, q, dpages, dci)
        paths = [[(prompt[b, i // ps], i % ps) for i in range(P[b])] +
                 [(beam_pages[b * W + ci[b, w, i], i // ps], i % ps) for i in range(P[b], P[b] + t + 1)]
                 for b in range(B) for w in range(W)]
        s.check_attention(o, lse, q, paths)
        kept += [o, lse]

    # ---- two beams of each request go on; what was there before is given back
    held = np.concatenate([prompt.ravel(), beam_pages.ravel()])
    refs = np.zeros(s.pages, np.int32)
    np.add.at(refs, held[held >= 0], 1)
    s.refs.copy_(s.cuda(refs))
    beams = s.rs.randint(0, W, (B, FORKS)).astype(np.int32)
    L = P + STEPS
    tables = torch.full((B * FORKS, cols), -1, dtype=torch.int32, device="cuda")
    work = bsp.fork_workspace(B, FORKS)
    bsp.fork_tables(plan, s.cuda(beams), s.refs, s.refs, tables, work)
    bsp.fork_rows(plan, s.cuda(beams), tables, dpages, dci, s.k_pool, s.v_pool, scales=s.scales)
    bsp.free_pages(plan, s.cuda(prompt), s.refs, s.refs)
    bsp.free_pages(plan, dpages, s.refs, s.refs)
    s.flags.append(bsp.read_device_status(plan))
    tab = tables.cpu().numpy()
    want = np.zeros(s.pages, np.int32)
    np.add.at(want, tab[tab >= 0], 1)
    assert np.array_equal(s.refs.cpu().numpy(), want)
    rows = [(b, int(w)) for b in range(B) for w in beams[b]]
    path = [[(tab[r, i // ps], i % ps) for i in range(L[b])] for r, (b, _) in enumerate(rows)]
    for r, (b, w) in enumerate(rows):
        old = [tokens[b, i] if i < P[b] else made[b, ci[b, w, i], i] for i in range(L[b])]
        s.check_rows(path[r], tuple(np.stack(y) for y in zip(*old)))

    # ---- the forks' queries are their beams': attention over the copies, before and after the pool is compacted
    own = torch.tensor([b * W + w for b, w in rows], device="cuda")
    fq = q[own].contiguous()
    FL = np.repeat(L, FORKS).astype(np.int32)
    none = np.zeros(len(rows), np.int32)
    plan = ws.plan(s.geo, len(rows), 1, FL, none, tab)
    fo, flse = s.attend(plan, fq, None, None)
    s.check_attention(fo, flse, fq, path)
    moves = bsp.PageMoves(s.pages)
    bsp.compact_tables(plan, s.refs, s.refs, moves, tables)
    bsp.copy_pages(plan, moves, s.k_pool, s.v_pool, scales=s.scales)
    tab = tables.cpu().numpy()
    live = len(np.unique(tab[tab >= 0]))
    assert moves.count.tolist()[1] == live and tab.max() == live - 1
    assert (s.refs.cpu().numpy()[live:] == 0).all()
    plan = ws.plan(s.geo, len(rows), 1, FL, none, tab)
    again = s.attend(plan, fq, None, None)
    assert torch.equal(again[0], fo) and torch.equal(again[1], flse)   # the same rows in other pages
    kept += [fo, flse, tables.clone(), s.refs.clone()]

    # ---- and their next token, in a page of its own where the last one is full
    nxt = live
    for r in range(len(rows)):
        if FL[r] % ps == 0:
            tab[r, FL[r] // ps] = nxt
            if s.block:
                s.scales.k[nxt].zero_()
                s.scales.v[nxt].zero_()
            nxt += 1
    x, dev = s.rows(len(rows))
    where = [(tab[r, FL[r] // ps], FL[r] % ps) for r in range(len(rows))]
    plan = ws.plan(s.geo, len(rows), 1, FL, none + 1, tab)
    q = torch.empty((len(rows), s.Hq * s.D), dtype=TDT[s.dtype], device="cuda")
    s.append(plan, dev, FL, np.array([p * ps + i for p, i in where]), q)
    s.check_rows(where, s.stored(x, FL))
    fci = np.zeros((len(rows), 1, max_seq), np.int32)
    o, lse = s.attend(plan, q, s.cuda(tab), s.cuda(fci))
    s.check_attention(o, lse, q, [[(tab[r, i // ps], i % ps) for i in range(FL[r] + 1)] for r in range(len(rows))])
    kept += [o, lse, s.k_pool.clone().view(torch.uint8), s.v_pool.clone().view(torch.uint8)]
    assert all(f == (0, 0) for f in s.flags)
    return kept


# dtype, query heads, KV heads, head_dim, page, block (0: 16-bit pools)
SERVERS = [("bf16", 8, 4, 128, 16, 0), ("fp16", 6, 2, 64, 8, 0), ("bf16", 4, 2, 256, 16, 0), ("bf16", 8, 4, 128, 16, 16),
           ("fp16", 8, 2, 64, 32, 8), ("bf16", 4, 1, 128, 32, 32), ("fp16", 3, 3, 128, 8, 1)]


@pytest.mark.parametrize("server", SERVERS, ids=lambda c: "-".join(map(str, c)))
def test_prompts_beams_forks_and_compaction(server):
    run(Server(*server))


@pytest.mark.parametrize("server", [SERVERS[0], SERVERS[4]], ids=lambda c: "-".join(map(str, c)))
def test_runs_on_other_streams_agree(server):
    want = run(Server(*server, seed=3))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        got = run(Server(*server, seed=3))
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
