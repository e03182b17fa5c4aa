"""The keys' attention weights, the eviction of cached rows and the beams' tables (bsp_key_weights,
bsp_evict_prefix, bsp_beam_advance) against plain fp64 restatements."""
import math

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, synth
from oracle import steps

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def page_tables(rng, lens, ps, extra=3):
    need = -(-lens // ps)
    ids = rng.permutation(int(need.sum()) + extra).astype(np.int32)
    table = np.full((len(lens), max(1, int(need.max(initial=0)))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


def rows_of(pool, table, b, h, n, ps):
    """[n, D] fp64 rows of request b, kv head h in order."""
    pages = table[b, :-(-n // ps)].astype(np.int64)
    return pool[pages, h].reshape(-1, pool.shape[-1])[:n]


class Cache:
    def __init__(self, seed, lens, Hq, Hkv, D, ps, dtype, e4m3=False):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.ps, self.Hkv, self.Hq, self.D = rng, np.asarray(lens, np.int32), ps, Hkv, Hq, D
        self.table, total = page_tables(rng, self.lens, ps)
        gen = torch.Generator().manual_seed(seed)
        shape = (total, Hkv, ps, D)
        if e4m3:
            self.k, self.v = (synth.e4m3_codes(shape, gen).cuda() for _ in range(2))
            self.k64 = self.k.cpu().view(torch.float8_e4m3fn).double().numpy()
        else:
            self.k, self.v = (torch.randn(shape, generator=gen).to(TYPES[dtype]).cuda() for _ in range(2))
            self.k64 = self.k.double().cpu().numpy()
        self.geo = bsp.geometry(Hq, Hkv, D, ps, total, dtype, kv_dtype=bsp.KV_DTYPE_E4M3 if e4m3 else 0)
        self.gen, self.dtype = gen, dtype

    def decode_plan(self, W, tails=None):
        B = len(self.lens)
        self.ws = bsp.Workspace(self.geo, max(1, B), W, self.table.shape[1])
        return self.ws.plan(self.geo, B, W, self.lens, np.zeros(B, np.int32) if tails is None else tails, self.table)

    def prefill_plan(self, cached, causal=True):
        B = len(self.lens)
        prompt = self.lens - cached
        self.ws = bsp.Workspace(self.geo, B, max(1, int(prompt.max())), self.table.shape[1])
        return bsp.plan_prefill(self.geo, B, cached, prompt, self.table, causal, self.ws)

    def rows(self, R, scale=1.0):
        return (torch.randn((R, self.Hq, self.D), generator=self.gen) * scale).to(TYPES[self.dtype]).cuda()


def check_weights(c, q, lse, W, cached, window, got, k_scale=1.0, causal=True, before=None):
    q64, l64, scale = q.double().cpu().numpy(), lse.double().cpu().numpy(), 1 / math.sqrt(c.D)
    G, row0 = c.Hq // c.Hkv, 0
    got = got.double().cpu().numpy()
    for b, n in enumerate(c.lens):
        rows = W if cached is None else int(n - cached[b])
        seen = min(window, rows) if window else rows
        sl = slice(row0 + rows - seen, row0 + rows)
        row0 += rows
        sees = None if cached is None or not causal else np.arange(n - seen, n) + 1
        for h in range(c.Hkv):
            if rows == 0:
                assert (got[b, h] == -7.0).all()
                continue
            k = rows_of(c.k64, c.table, b, h, n, c.ps)
            heads = slice(h * G, (h + 1) * G)
            want = steps.key_weights(q64[sl, heads], k, l64[sl, heads], scale * k_scale, sees)
            # relative: exp of a score off by an fp32 sum of D products, D 2^-24 of sum |q||k| (bounded by the
            # norms); exp2's own 2^-22, its argument's rounding 2^-24 of (score + lse) log2(e), lse rounded to
            # fp32 and scaled (2^-23 of it); the sum over the rows, seen G 2^-24
            size = np.linalg.norm(q64[sl, heads], axis=-1).max(initial=0) * np.linalg.norm(k, axis=-1).max(initial=0) * scale * k_scale
            lmax = np.abs(np.where(np.isneginf(l64[sl, heads]), 0, l64[sl, heads])).max(initial=0)
            tol = want * (c.D * 2.0 ** -24 * size + 2.0 ** -22 + 2.0 ** -23 * 2 * (size + lmax) + seen * G * 2.0 ** -24) + 1e-30
            if before is not None:
                want = want + before
                tol = tol + 2.0 ** -24 * np.abs(want) + 2.0 ** -23 * lmax * np.abs(want)
            err = np.abs(got[b, h, :n] - want)
            assert (err <= tol).all(), (b, h, err.max(), want.max())
            assert (got[b, h, n:] == -7.0).all()


def true_lse(c, q, W, cached, causal=True, k_scale=1.0):
    """Natural log-sum-exp of each row over the keys it sees, fp32."""
    q64, scale, G = q.double().cpu().numpy(), 1 / math.sqrt(c.D) * k_scale, c.Hq // c.Hkv
    out = np.full((q.shape[0], c.Hq), -np.inf)
    row0 = 0
    for b, n in enumerate(c.lens):
        rows = W if cached is None else int(n - cached[b])
        for h in range(c.Hkv):
            if n == 0 or rows == 0:
                continue
            k = rows_of(c.k64, c.table, b, h, n, c.ps)
            s = np.einsum("igd,jd->igj", q64[row0:row0 + rows, h * G:(h + 1) * G], k) * scale
            if cached is not None and causal:
                s = np.where(np.arange(n)[None, None] <= (np.arange(rows) + cached[b])[:, None, None], s, -np.inf)
            m = s.max(-1)
            out[row0:row0 + rows, h * G:(h + 1) * G] = m + np.log(np.exp(s - m[..., None]).sum(-1))
        row0 += rows
    return torch.from_numpy(out.astype(np.float32)).cuda()


@pytest.mark.parametrize("lens,W,Hq,Hkv,D,ps,dtype", [
    ([128], 4, 4, 2, 64, 32, "bf16"), ([1], 1, 1, 1, 64, 8, "fp16"), ([0, 5, 300, 129], 3, 6, 2, 128, 16, "bf16"),
    ([700, 650], 96, 16, 8, 128, 32, "bf16"), ([257, 0, 90], 30, 32, 8, 128, 16, "fp16"),
    ([200, 333], 17, 8, 1, 256, 64, "bf16"), ([513], 5, 6, 2, 256, 128, "fp16"), ([1000], 300, 2, 2, 64, 32, "bf16"),
    ([129, 64], 100, 12, 4, 128, 8, "fp16")])
def test_key_weights_decode(lens, W, Hq, Hkv, D, ps, dtype):
    c = Cache(sum(lens) + W, lens, Hq, Hkv, D, ps, dtype)
    plan = c.decode_plan(W)
    q = c.rows(len(lens) * W)
    lse = true_lse(c, q, W, None)
    if W > 2:
        lse[1] = -np.inf  # a row that adds nothing
    got = torch.full((len(lens), Hkv, max(lens) + 5), -7.0, device="cuda")
    bsp.key_weights(plan, q, c.k, lse, 1 / math.sqrt(D), got, flags=bsp.FLAG_CHECK)
    check_weights(c, q, lse, W, None, 0, got)
    # the same call again, in base 2, and added up
    again = torch.full_like(got, -7.0)
    bsp.key_weights(plan, q, c.k, lse, 1 / math.sqrt(D), again)
    assert torch.equal(again, got)
    for b, n in enumerate(lens):
        again[b, :, :n] = 0.5
    bsp.key_weights(plan, q, c.k, lse * 1.4426950408889634, 1 / math.sqrt(D), again,
                    flags=bsp.FLAG_ACCUMULATE | bsp.FLAG_LSE_BASE2 | bsp.FLAG_CHECK)
    check_weights(c, q, lse, W, None, 0, again, before=0.5)


@pytest.mark.parametrize("cached,prompt,window,Hq,Hkv,D,ps,dtype,causal", [
    ([0], [1], 0, 2, 1, 64, 16, "bf16", True), ([0, 37], [200, 1], 0, 8, 2, 64, 16, "fp16", True),
    ([0, 100, 5], [300, 77, 0], 16, 32, 8, 128, 32, "fp16", True), ([10, 130], [129, 260], 0, 16, 2, 128, 32, "bf16", True),
    ([0, 3], [70, 140], 64, 4, 4, 256, 32, "bf16", True), ([9], [333], 0, 6, 2, 256, 8, "fp16", True),
    ([40, 0], [50, 150], 33, 12, 4, 128, 64, "bf16", False)])
def test_key_weights_prefill(cached, prompt, window, Hq, Hkv, D, ps, dtype, causal):
    cached = np.array(cached, np.int32)
    lens = cached + np.array(prompt, np.int32)
    c = Cache(int(lens.sum()), lens, Hq, Hkv, D, ps, dtype)
    plan = c.prefill_plan(cached, causal)
    q = c.rows(int(sum(prompt)))
    lse = true_lse(c, q, None, cached, causal)
    got = torch.full((len(lens), Hkv, int(lens.max())), -7.0, device="cuda")
    bsp.key_weights(plan, q, c.k, lse, 1 / math.sqrt(D), got, window=window, flags=bsp.FLAG_CHECK)
    check_weights(c, q, lse, None, cached, window, got, causal=causal)
    if not window:  # every row's probabilities sum to one
        total = got.clamp(min=0).double().sum((1, 2)).cpu().numpy()
        assert np.allclose(total, np.array(prompt) * Hq, rtol=1e-4)


@pytest.mark.parametrize("lens,W,Hq,Hkv,D,dtype,k_scale", [
    ([300, 0, 128], 30, 16, 8, 128, "bf16", 0.5), ([77], 3, 4, 2, 64, "fp16", 1.0), ([500, 129], 96, 16, 8, 128, "fp16", 0.25),
    ([260], 100, 8, 2, 64, "bf16", 0.25)])
def test_key_weights_fp8(lens, W, Hq, Hkv, D, dtype, k_scale):
    c = Cache(sum(lens), lens, Hq, Hkv, D, 32, dtype, e4m3=True)
    plan = c.decode_plan(W)
    q = c.rows(len(lens) * W, 0.25)
    lse = true_lse(c, q, W, None, k_scale=k_scale)
    got = torch.full((len(lens), Hkv, max(lens)), -7.0, device="cuda")
    bsp.key_weights_fp8(plan, q, c.k, lse, 1 / math.sqrt(D), k_scale, got, flags=bsp.FLAG_CHECK)
    check_weights(c, q, lse, W, None, 0, got, k_scale=k_scale)


def run_evict(c, plan, w, keep, sinks, recent, positions=None, alias=False, lens=None):
    """lens: the rows the plan holds of each request (default: all)."""
    lens = c.lens if lens is None else lens
    k0, v0 = c.k.clone(), c.v.clone()
    kept = torch.full(w.shape, -5, dtype=torch.int32, device="cuda")
    wo = w.clone() if alias else torch.full_like(w, -5.0)
    po = positions.clone() if alias and positions is not None else torch.full_like(kept, -5)
    win, pin = (wo, po if positions is not None else None) if alias else (w, positions)
    keep_d = torch.tensor(keep, dtype=torch.int32, device="cuda")
    bsp.evict_prefix(plan, win, keep_d, sinks, recent, c.k, c.v, kept, positions=pin, weights_out=wo, positions_out=po)
    assert bsp.read_device_status(plan) == (0, 0)
    wh, ph = w.cpu().numpy(), None if positions is None else positions.cpu().numpy()
    for b, n in enumerate(lens):
        pages = c.table[b]
        for h in range(c.Hkv):
            src = steps.evict(wh[b, h, :n], keep[b], sinks, recent, None if ph is None else ph[b, h, :n])
            m = len(src)
            got = kept[b, h].cpu().numpy()
            assert np.array_equal(got[:m], src), (b, h)
            assert (got[m:] == -5).all()
            assert np.array_equal(wo[b, h, :m].cpu().numpy(), wh[b, h, src], equal_nan=True)
            assert np.array_equal(po[b, h, :m].cpu().numpy(), src if ph is None else ph[b, h, src])
            if not alias:
                assert (wo[b, h, m:] == -5).all() and (po[b, h, m:] == -5).all()
            i = np.arange(m)
            for new, old in ((c.k, k0), (c.v, v0)):
                a = new[torch.from_numpy(pages[i // c.ps].astype(np.int64)).cuda(), h, torch.from_numpy(i % c.ps).cuda()]
                want = old[torch.from_numpy(pages[src // c.ps].astype(np.int64)).cuda(), h, torch.from_numpy(src % c.ps).long().cuda()]
                assert torch.equal(a.view(torch.uint8), want.view(torch.uint8))
    # nothing outside the first keep slots of the requests' pages has changed
    for new, old in ((c.k, k0), (c.v, v0)):
        same = (new.view(torch.uint8) == old.view(torch.uint8)).all(-1).cpu().numpy()  # [page, head, slot]
        free = np.ones(same.shape, bool)
        for b, n in enumerate(lens):
            i = np.arange(min(int(n), max(0, keep[b])))
            free[c.table[b][i // c.ps], :, i % c.ps] = False
        assert same[free].all()


@pytest.mark.parametrize("lens,keep,sinks,recent,Hkv,D,ps,dtype", [
    ([100], [40], 4, 8, 2, 64, 16, "bf16"), ([0, 1, 33, 500], [5, 1, 0, 499], 0, 0, 1, 128, 8, "fp16"),
    ([2000, 1500], [700, 5000], 4, 64, 8, 128, 32, "bf16"), ([64, 64], [64, 32], 100, 0, 2, 256, 64, "fp16"),
    ([77, 300], [10, 200], 3, 50, 3, 256, 128, "bf16"), ([5000], [1], 0, 0, 1, 64, 32, "bf16"),
    ([20000], [6000], 4, 300, 1, 64, 32, "bf16"), ([300], [-3], 0, 0, 1, 64, 32, "bf16")])
def test_evict(lens, keep, sinks, recent, Hkv, D, ps, dtype):
    c = Cache(sum(lens), lens, Hkv, Hkv, D, ps, dtype)
    plan = c.decode_plan(2)
    w = torch.exp(2 * torch.randn((len(lens), Hkv, max(lens) + 3), generator=c.gen)).cuda()
    run_evict(c, plan, w, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "inf", "two", "ascending"])
@pytest.mark.parametrize("alias", [False, True])
def test_evict_ties_and_special_weights(kind, alias):
    c = Cache(11, [400, 90], 2, 2, 128, 32, "bf16")
    plan = c.decode_plan(1)
    w = torch.rand((2, 2, 400), generator=c.gen).cuda()
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "zeros":
        w.zero_()
        w[:, :, ::2] = -0.0
    elif kind == "nan":
        w[:, :, 5:380] = np.nan
    elif kind == "inf":
        w[:, :, ::3] = np.inf
        w[:, :, 1::3] = -np.inf
    elif kind == "two":
        w = (w > 0.5).float()
    else:
        w = torch.arange(400, device="cuda").float().expand(2, 2, 400).contiguous()
    positions = torch.stack([torch.randperm(400, generator=c.gen) for _ in range(4)]).view(2, 2, 400).to(torch.int32).cuda()
    run_evict(c, plan, w, [150, 60], 3, 20, positions, alias)


def test_evict_fp8_pools():
    c = Cache(12, [333, 64], 2, 2, 64, 16, "bf16", e4m3=True)
    plan = c.decode_plan(4)
    run_evict(c, plan, torch.rand((2, 2, 333), generator=c.gen).cuda(), [100, 3], 2, 5)


def test_evict_prefill_plan():
    """A prefill plan's cached and prompt rows alike; a request without prompt rows is left as it is."""
    cached = np.array([20, 50, 0], np.int32)
    c = Cache(13, [120, 50, 33], 4, 2, 128, 16, "fp16")
    plan = c.prefill_plan(cached)
    run_evict(c, plan, torch.rand((3, 2, 120), generator=c.gen).cuda(), [60, 10, 5], 1, 4, lens=[120, 0, 33])


@pytest.mark.parametrize("P,stride,keep", [(47000, 47000, 20000), (52001, 52001, 52000), (120000, 120000, 3),
                                           (60000, 1 << 19, 30011)])
def test_evict_long_prompts(P, stride, keep):
    """Prompts whose keys' order does not fit beside the bitmap, and rows of the tables as long as any may be."""
    c = Cache(P, [P], 1, 1, 64, 64, "bf16")
    plan = c.decode_plan(1)
    w = torch.rand((1, 1, stride), generator=c.gen).cuda()
    run_evict(c, plan, w, [keep], 4, 100)


def test_evict_refuses_tails_and_bad_arguments():
    c = Cache(14, [100], 2, 2, 64, 16, "bf16")
    w = torch.rand((1, 2, 100), generator=c.gen).cuda()
    kept = torch.zeros((1, 2, 100), dtype=torch.int32, device="cuda")
    keep = torch.tensor([5], dtype=torch.int32, device="cuda")
    tail = c.decode_plan(2, np.array([1], np.int32))
    with pytest.raises(bsp.BspError) as e:
        bsp.evict_prefix(tail, w, keep, 0, 0, c.k, c.v, kept)
    assert e.value.status == 1
    plan = c.decode_plan(2)
    for bad in (dict(sinks=-1, recent=0), dict(sinks=0, recent=-1)):
        with pytest.raises(bsp.BspError):
            bsp.evict_prefix(plan, w, keep, k_pool=c.k, v_pool=c.v, kept=kept, **bad)
    with pytest.raises(ValueError):
        bsp.evict_prefix(plan, w[:, :, :99].contiguous(), keep, 0, 0, c.k, c.v, kept)
    with pytest.raises(ValueError):
        bsp.evict_prefix(plan, w, keep.long(), 0, 0, c.k, c.v, kept)


@pytest.mark.parametrize("B,W,P,T,inplace", [
    (1, 1, 0, 0, False), (2, 4, 10, 3, True), (3, 30, 5, 7, False), (2, 96, 40, 7, True), (1, 5000, 3, 7, True)])
def test_beam_advance(B, W, P, T, inplace):
    rng = np.random.default_rng(W)
    geo = bsp.geometry(2, 1, 64, 32, 8, "bf16")
    ws = bsp.Workspace(geo, B, W, 2)
    tails = np.maximum(0, T - np.arange(B)).astype(np.int32)
    plan = ws.plan(geo, B, W, np.full(B, P, np.int32), tails, np.tile(np.arange(2, dtype=np.int32), (B, 1)))
    parents = rng.integers(0, W, (B, W + 3)).astype(np.int32)
    parents[0, 0] = -1
    chosen = rng.integers(0, 999, (B, W + 3)).astype(np.int32)
    ci = rng.integers(0, W, (B, W, P + T + 2)).astype(np.int32)
    tok = rng.integers(0, 999, (B * W, T + 3)).astype(np.int32)
    c1, t1 = torch.from_numpy(ci).cuda(), torch.from_numpy(tok).cuda()
    c2, t2 = (c1, t1) if inplace else (c1.clone(), t1.clone())
    n = torch.zeros(B * W, dtype=torch.int32, device="cuda")
    bsp.beam_advance(plan, torch.from_numpy(parents).cuda(), torch.from_numpy(chosen).cuda(), c1, c2, t1, t2, n)
    assert bsp.read_device_status(plan) == (0, 0)
    for b in range(B):
        wc, wt = steps.advance(parents[b, :W], chosen[b, :W], P, tails[b], ci[b], tok[b * W:(b + 1) * W])
        assert np.array_equal(c2[b].cpu().numpy(), wc) and np.array_equal(t2[b * W:(b + 1) * W].cpu().numpy(), wt)
        assert (n[b * W:(b + 1) * W] == int(tails[b]) + 1).all()
    if not inplace:
        assert np.array_equal(c1.cpu().numpy(), ci) and np.array_equal(t1.cpu().numpy(), tok)


def test_beam_advance_flags_bad_parents_and_refuses_short_tables():
    geo = bsp.geometry(2, 1, 64, 32, 8, "bf16")
    ws = bsp.Workspace(geo, 1, 3, 1)
    plan = ws.plan(geo, 1, 3, np.zeros(1, np.int32), np.array([2], np.int32), np.zeros((1, 1), np.int32))
    chosen = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    tok = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    for bad in ([0, 3, 1], [0, -2, 1]):
        t = tok.clone()
        bsp.beam_advance(plan, torch.tensor([bad], dtype=torch.int32, device="cuda"), chosen, tokens=t)
        assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
        assert torch.equal(t[1, :2], tok[1, :2]) and torch.equal(t[2, :2], tok[1, :2])
    with pytest.raises(bsp.BspError):
        bsp.beam_advance(plan, chosen, chosen, tokens=tok[:, :2].contiguous())
    with pytest.raises(bsp.BspError):
        bsp.beam_advance(plan, chosen, chosen, torch.zeros((1, 3, 2), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("W,G,D,dtype,lens", [(96, 2, 128, "bf16", (1200, 1900)), (30, 2, 128, "fp16", (1000, 1600)),
                                              (40, 5, 64, "bf16", (900, 2100)), (64, 4, 256, "bf16", (500, 900))])
def test_key_weights_many_tiles_per_sm(W, G, D, dtype, lens):
    """Dozens of key tiles for every SM, so that rings and accumulators go round many times, against fp64 products."""
    rng = np.random.default_rng(W)
    n = rng.integers(lens[0], lens[1], 40).astype(np.int32)
    Hkv = 8
    c = Cache(W, n, Hkv * G, Hkv, D, 32, dtype)
    plan = c.decode_plan(W)
    q = c.rows(40 * W)
    lse = torch.empty((40 * W, Hkv * G), device="cuda")
    want, size = [], 0.0
    for b in range(40):
        pages = torch.from_numpy(c.table[b, :-(-n[b] // 32)].astype(np.int64)).cuda()
        k = c.k[pages].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n[b]]
        qb = q[b * W:(b + 1) * W].double().view(W, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * W, D)
        s = qb @ k.transpose(1, 2) / math.sqrt(D)
        ls = torch.logsumexp(s, -1).float()
        lse[b * W:(b + 1) * W] = ls.view(Hkv, G, W).permute(2, 0, 1).reshape(W, Hkv * G)
        want.append(torch.exp(s - ls.double()[..., None]).sum(1))
        size = max(size, float(qb.norm(dim=-1).max() * k.norm(dim=-1).max()) / math.sqrt(D))
    for rep in range(3):
        got = torch.full((40, Hkv, int(n.max())), -7.0, device="cuda")
        bsp.key_weights(plan, q, c.k, lse, 1 / math.sqrt(D), got)
        assert bsp.read_device_status(plan) == (0, 0)
        for b in range(40):
            # as check_weights: the product's D 2^-24 of |q||k|, exp2, its argument, lse, the sum
            tol = want[b] * (D * 2.0 ** -24 * size + 2.0 ** -22 + 2.0 ** -22 * (size + 20) + W * G * 2.0 ** -24) + 1e-30
            assert ((got[b, :, :n[b]].double() - want[b]).abs() <= tol).all()
            assert (got[b, :, n[b]:] == -7.0).all()
