"""Page bookkeeping (bsp_fork_tables, bsp_fork_rows, bsp_free_pages, bsp_compact_tables, bsp_copy_pages) against the
restatements of oracle/cache.py: integers and copied rows bit for bit; rows of E4M3 blocks with scales by their values."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, synth
from oracle import cache

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def bytes_of(shape, gen):
    return torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)


class Forked:
    """A beam step over a random paged cache, and forks of its beams."""

    def __init__(self, prompt, tail, W=5, forks=3, ps=16, Hkv=2, D=64, dtype="bf16", kv_dtype=0, spare=40, seed=0, none=0.0):
        rs = np.random.RandomState(seed)
        B = len(prompt)
        wl = synth.Workload("fork", B, W, Hkv * 2, Hkv, D, ps, dtype, (0, 0), (0, 0))
        case = synth.make_case(wl, seed, full_step=False, device="cpu", prompt_lengths=list(prompt), tail_lengths=list(tail))
        self.case, self.B, self.W, self.ps, self.Hkv, self.D = case, B, W, ps, Hkv, D
        self.pages = case.num_pages + spare
        self.geo = bsp.geometry(Hkv * 2, Hkv, D, ps, self.pages, dtype, kv_dtype)
        self.ws = bsp.Workspace(self.geo, B, W, case.prefix_pages.shape[1])
        self.plan = self.ws.plan(self.geo, B, W, case.prefix_len, case.tail_len, case.prefix_pages)
        self.refs = np.zeros(self.pages, np.int32)
        for p in np.unique(case.beam_pages[case.beam_pages >= 0]):
            self.refs[p] = rs.randint(1, 4)
        self.refs[rs.permutation(self.pages)[:spare // 8]] += 1  # (some of the spare ones are held too)
        self.beams = rs.randint(0, W, (B, forks)).astype(np.int32)
        self.beams[rs.rand(B, forks) < none] = -1
        gen = torch.Generator().manual_seed(seed)
        es = 1 if kv_dtype else 2
        self.pools = [bytes_of((self.pages, Hkv, ps, D * es), gen) for _ in range(2)]
        self.dev = [p.cuda() if kv_dtype else p.cuda().view(TDT[dtype]) for p in self.pools]
        self.cols = -(-int((case.prefix_len + case.tail_len).max()) // ps) + 1
        self.out = torch.full((B * forks, self.cols), -7, dtype=torch.int32, device="cuda")
        self.work = bsp.fork_workspace(B, forks)

    def cuda(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def tables(self, refs_out=None):
        refs = self.cuda(self.refs)
        out = torch.full_like(refs, -9) if refs_out is None else refs
        bsp.fork_tables(self.plan, self.cuda(self.beams), refs, out, self.out, self.work)
        return out

    def want(self):
        c = self.case
        return cache.fork_tables(c.prefix_len, c.tail_len, c.prefix_pages, self.beams, self.W, self.ps, self.refs,
                                 np.full(self.out.shape, -7))

    def rows(self, scales=None):
        bsp.fork_rows(self.plan, self.cuda(self.beams), self.out, self.cuda(self.case.beam_pages),
                      self.cuda(self.case.cache_indirection), *self.dev, scales=scales)

    def sources(self):
        c = self.case
        return cache.fork_sources(c.prefix_len, c.tail_len, c.prefix_pages, c.beam_pages, c.cache_indirection, self.beams, self.W, self.ps)


CASES = [
    dict(prompt=[40], tail=[3], W=4, forks=2),
    dict(prompt=[33, 0, 64, 47, 16, 100], tail=[8, 5, 0, 8, 1, 3], ps=16),      # no prompt, no tail, two fresh pages
    dict(prompt=[15, 16, 17], tail=[1, 1, 1], ps=8, Hkv=3, D=128, dtype="fp16"),
    dict(prompt=[130, 255, 128], tail=[8, 2, 0], ps=128, Hkv=1, D=256, forks=9),
    dict(prompt=[50, 60, 70, 80], tail=[2, 3, 4, 5], ps=32, Hkv=8, W=30, forks=30, spare=300, none=0.3),
    dict(prompt=[40, 41], tail=[4, 4], kv_dtype=bsp.KV_DTYPE_E4M3, Hkv=5, D=64),
    dict(prompt=[7] * 70, tail=[6] * 70, ps=8, W=3, forks=64, spare=9000, Hkv=1, none=0.1),  # 4480 rows: several rounds of the scan, the last rows without pages
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(i, in_place):
    f = Forked(**CASES[i], seed=i)
    refs, out, served, short = f.want()
    got = f.tables(refs_out=in_place or None)
    assert bsp.read_device_status(f.plan) == ((4, bsp.DEVFLAG_PAGES) if short else (0, 0))
    np.testing.assert_array_equal(f.out.cpu().numpy(), out)
    np.testing.assert_array_equal(got.cpu().numpy(), refs)
    f.rows()
    assert bsp.read_device_status(f.plan) == (0, 0)
    for pool, dev in zip(f.pools, f.dev):
        want = pool.clone()
        for r, rows in enumerate(f.sources()):
            for pos, page in rows:
                if served[r]:
                    want[out[r, pos // f.ps], :, pos % f.ps] = pool[page, :, pos % f.ps]
        assert torch.equal(dev.view(torch.uint8).cpu(), want)


def test_fork_without_enough_pages():
    f = Forked(prompt=[40, 48, 50], tail=[3, 0, 8], ps=16, forks=7, spare=16, seed=3)
    f.refs[f.refs == 0] = 1
    f.refs[np.random.RandomState(1).permutation(f.pages)[:9]] = 0
    for p in np.unique(f.case.beam_pages[f.case.beam_pages >= 0]):
        f.refs[p] = max(1, f.refs[p])
    refs, out, served, short = f.want()
    assert short and served.any() and not served.all()
    got = f.tables()
    assert bsp.read_device_status(f.plan) == (4, bsp.DEVFLAG_PAGES)
    np.testing.assert_array_equal(f.out.cpu().numpy(), out)
    np.testing.assert_array_equal(got.cpu().numpy(), refs)
    f.rows()  # rows without pages are left out
    assert bsp.read_device_status(f.plan) == (0, 0)


def test_fork_bad_indices_are_flagged():
    f = Forked(prompt=[40, 20], tail=[3, 2], ps=16, forks=3, seed=4)
    f.beams[0] = [0, f.W, 1]
    f.tables()
    assert bsp.read_device_status(f.plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
    f.beams[0, 1] = -1
    _, out, served, _ = f.want()
    np.testing.assert_array_equal(f.out.cpu().numpy(), out)
    before = [d.clone() for d in f.dev]
    ci = f.case.cache_indirection
    ci[0, f.beams[0, 0], 41] = f.W       # one row's source: not copied, and told
    f.rows()
    assert bsp.read_device_status(f.plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
    page, slot = out[0, 41 // 16], 41 % 16
    assert torch.equal(f.dev[0][page, :, slot].view(torch.int16), before[0][page, :, slot].view(torch.int16))
    f.out[0, 40 // 16] = f.pages + 3     # a table from elsewhere
    f.rows()
    assert bsp.read_device_status(f.plan) == (3, bsp.DEVFLAG_PAGE_INDEX)


@pytest.mark.parametrize("block", [1, 4, 16])
@pytest.mark.parametrize("Hkv", [2, 9])
def test_fork_rows_with_block_scales(block, Hkv):
    f = Forked(prompt=[40, 21, 32, 0], tail=[8, 7, 3, 5], ps=16, forks=4, Hkv=Hkv, kv_dtype=bsp.KV_DTYPE_E4M3, seed=5)
    gen = torch.Generator().manual_seed(8)
    for p, d in zip(f.pools, f.dev):
        p.copy_(synth.e4m3_codes(p.shape, gen, exp_mean=7, exp_sd=4))  # (subnormal codes among them)
        d.copy_(p)
    shape = (f.pages, Hkv, 16 // block)
    exps = [torch.randint(120, 126, shape, generator=gen, dtype=torch.uint8) for _ in range(2)]
    scales = bsp.BlockScales(f.geo, block, k=exps[0].cuda(), v=exps[1].cuda())
    _, out, served, _ = f.want()
    f.tables()
    f.rows(scales)
    assert bsp.read_device_status(f.plan) == (0, 0)
    for pool, dev, e, ed in zip(f.pools, f.dev, exps, (scales.k, scales.v)):
        want, we = pool.numpy().copy(), e.numpy().copy()
        old, oe = pool.numpy(), e.numpy()
        for r, rows in enumerate(f.sources()):
            mine = {}
            for pos, page in rows:
                mine.setdefault(out[r, pos // 16], []).append((pos % 16, page))
            for page, held in mine.items():
                we[page] = 0
                for s, src in held:
                    we[page, :, s // block] = np.maximum(we[page, :, s // block], oe[src, :, s // block])
                for s, src in held:
                    for h in range(Hkv):
                        a, b = int(oe[src, h, s // block]), int(we[page, h, s // block])
                        want[page, h, s] = old[src, h, s] if a == b else cache.round_e4m3(cache.DECODE[old[src, h, s]] * 2.0 ** (a - b))
        np.testing.assert_array_equal(ed.cpu().numpy(), we)
        np.testing.assert_array_equal(cache.DECODE[dev.cpu().numpy()], cache.DECODE[want])


def plain_plan(pages, ps=16, Hkv=2, D=64, dtype="bf16", kv_dtype=0):
    geo = bsp.geometry(Hkv, Hkv, D, ps, pages, dtype, kv_dtype)
    ws = bsp.Workspace(geo, 1, 1, 1)
    return geo, ws, ws.plan(geo, 1, 1, [1], [0], np.zeros((1, 1), np.int32))


@pytest.mark.parametrize("rows,cols,pages", [(1, 1, 5), (7, 9, 50), (300, 41, 3000), (3, 0, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_free(rows, cols, pages, in_place):
    rs = np.random.RandomState(rows)
    _, ws, plan = plain_plan(pages)
    wide = rs.randint(-1, pages, (rows, cols + 3)).astype(np.int32)
    refs = rs.randint(0, 3, pages).astype(np.int32) + np.bincount(wide[:, :cols][wide[:, :cols] >= 0].ravel(), minlength=pages).astype(np.int32)
    t, r = torch.from_numpy(wide).cuda()[:, :cols], torch.from_numpy(refs).cuda()
    out = r if in_place else torch.full_like(r, -3)
    bsp.free_pages(plan, t, r, out)
    assert bsp.read_device_status(plan) == (0, 0)
    np.testing.assert_array_equal(out.cpu().numpy(), cache.free_pages(refs, wide[:, :cols]))


def test_free_too_often_and_outside():
    _, ws, plan = plain_plan(10)
    table = torch.tensor([[1, 1, 1, 2], [10, -2, 3, -1]], dtype=torch.int32, device="cuda")
    refs = torch.tensor([5, 2, 1, 0, 0, 0, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    bsp.free_pages(plan, table, refs, refs)
    assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
    assert refs.tolist() == [5, 0, 0, 0, 0, 0, 0, 0, 0, 1]


@pytest.mark.parametrize("pages,share,in_place", [(1, 1.0, False), (2, 0.5, True), (33, 0.4, False), (33, 0.0, False), (33, 1.0, True),
                                                  (5000, 0.5, True), (70001, 0.2, False), (70001, 0.9, False)])
def test_compact(pages, share, in_place):
    rs = np.random.RandomState(pages)
    _, ws, plan = plain_plan(pages)
    refs = np.where(rs.rand(pages) < share, rs.randint(1, 5, pages), 0).astype(np.int32)
    live = np.flatnonzero(refs)
    tables = np.full((13, 11), -1, np.int32)
    if len(live):
        tables[:, :7] = live[rs.randint(0, len(live), (13, 7))]
    r, t = torch.from_numpy(refs).cuda(), torch.from_numpy(tables).cuda()
    ro, to = (r, t) if in_place else (torch.full_like(r, -3), torch.zeros_like(t))
    mv = bsp.PageMoves(pages)
    bsp.compact_tables(plan, r, ro, mv, t, to)
    assert bsp.read_device_status(plan) == (0, 0)
    want, pairs, L, remap, wt = cache.compact(refs, tables)
    assert mv.count.tolist() == [len(pairs), L]
    assert mv.pairs[:len(pairs)].tolist() == [list(map(int, p)) for p in pairs]
    np.testing.assert_array_equal(mv.remap.cpu().numpy(), remap)
    np.testing.assert_array_equal(ro.cpu().numpy(), want)
    np.testing.assert_array_equal(to.cpu().numpy(), wt)
    assert (want[:L] > 0).all() and (want[L:] == 0).all()
    bsp.compact_tables(plan, ro, ro, mv)  # nothing moves any more; no tables
    assert mv.count.tolist() == [0, L]


def test_compact_entries_outside_the_pool():
    _, ws, plan = plain_plan(4)
    refs = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    t = torch.tensor([[3, 4, -2, 1]], dtype=torch.int32, device="cuda")
    bsp.compact_tables(plan, refs, refs, bsp.PageMoves(4), t)
    assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
    assert t.tolist() == [[0, 4, -2, 1]] and refs.tolist() == [1, 1, 0, 0]


@pytest.mark.parametrize("ps,Hkv,D,dtype,kv_dtype,block", [(16, 2, 64, "bf16", 0, None), (8, 1, 64, "fp16", bsp.KV_DTYPE_E4M3, 8),
                                                           (128, 5, 128, "bf16", bsp.KV_DTYPE_E4M3, 1), (32, 8, 256, "bf16", 0, None),
                                                           (64, 3, 128, "fp16", bsp.KV_DTYPE_E4M3, None)])
def test_copy_pages(ps, Hkv, D, dtype, kv_dtype, block):
    pages = 30
    geo, ws, plan = plain_plan(pages, ps, Hkv, D, dtype, kv_dtype)
    gen = torch.Generator().manual_seed(1)
    pools = [bytes_of((pages, Hkv, ps, D * (1 if kv_dtype else 2)), gen) for _ in range(2)]
    dev = [p.cuda() if kv_dtype else p.cuda().view(TDT[dtype]) for p in pools]
    pairs = torch.tensor([[29, 0], [20, 1], [-1, -1], [20, 5], [7, 28], [3, 9]], dtype=torch.int32)
    count = torch.tensor([5], dtype=torch.int32)
    scales = exps = None
    if block:
        exps = [bytes_of((pages, Hkv, ps // block), gen) for _ in range(2)]
        scales = bsp.BlockScales(geo, block, k=exps[0].cuda(), v=exps[1].cuda())
    bsp.copy_pages(plan, bsp.PageMoves(pages, pairs=pairs.cuda(), count=count.cuda()), *dev, scales=scales)
    assert bsp.read_device_status(plan) == (0, 0)

    def moved(x):
        y = x.clone()
        for a, b in pairs[:5].tolist():
            if a >= 0:
                y[b] = x[a]
        return y
    assert all(torch.equal(d.view(torch.uint8).cpu(), moved(p)) for d, p in zip(dev, pools))
    if block:
        assert torch.equal(scales.k.cpu(), moved(exps[0])) and torch.equal(scales.v.cpu(), moved(exps[1]))
    # pairs outside the pool, and a count past the list
    bad = torch.tensor([[0, 30], [-2, 3], [31, 31]], dtype=torch.int32).cuda()
    bsp.copy_pages(plan, bsp.PageMoves(pages, pairs=bad, count=torch.tensor([99], dtype=torch.int32).cuda()), *dev)
    assert bsp.read_device_status(plan) == (3, bsp.DEVFLAG_PAGE_INDEX)
    assert all(torch.equal(d.view(torch.uint8).cpu(), moved(p)) for d, p in zip(dev, pools))


def test_replayed_fork_follows_later_plans_and_refuses_others():
    f = Forked(prompt=[40, 33], tail=[8, 8], ps=16, forks=3, seed=9)
    beams, refs = f.cuda(f.beams), f.cuda(f.refs)
    out = torch.zeros_like(refs)
    bp, ci = f.cuda(f.case.beam_pages), f.cuda(f.case.cache_indirection)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsp.fork_tables(f.plan, beams, refs, out, f.out, f.work)
        bsp.fork_rows(f.plan, beams, f.out, bp, ci, *f.dev)
    for tails in ([8, 8], [3, 0]):
        f.case.tail_len[:] = tails
        for d, p in zip(f.dev, f.pools):
            d.view(torch.uint8).copy_(p)
        f.plan = f.ws.plan(f.geo, f.B, f.W, f.case.prefix_len, f.case.tail_len, f.case.prefix_pages)
        f.out.fill_(-7)
        g.replay()
        assert bsp.read_device_status(f.plan) == (0, 0)
        want, table, _, _ = f.want()
        np.testing.assert_array_equal(f.out.cpu().numpy(), table)
        np.testing.assert_array_equal(out.cpu().numpy(), want)
        whole = f.pools[0].clone()
        for r, rows in enumerate(f.sources()):
            for pos, page in rows:
                whole[table[r, pos // 16], :, pos % 16] = f.pools[0][page, :, pos % 16]
        assert torch.equal(f.dev[0].view(torch.uint8).cpu(), whole)
    one = f.ws.plan(f.geo, 1, f.W, f.case.prefix_len[:1], [0], f.case.prefix_pages[:1])
    f.out.fill_(-7)
    g.replay()
    assert bsp.read_device_status(one) == (5, bsp.DEVFLAG_GRAPH)
    assert (f.out == -7).all()


@pytest.mark.parametrize("pages", [1023, 1024, 1025, 2049])
def test_pools_around_the_size_that_one_cta_scans(pages):
    rs = np.random.RandomState(pages)
    geo = bsp.geometry(2, 1, 64, 8, pages, "bf16")
    ws = bsp.Workspace(geo, 1, 4, 1)
    plan = ws.plan(geo, 1, 4, [3], [6], [[5]])   # nine positions: two fresh pages a fork
    refs = rs.randint(0, 3, pages).astype(np.int32)
    refs[5] = 1
    gone = rs.randint(-1, pages, (9, 60)).astype(np.int32)
    dev = torch.from_numpy(refs).cuda()
    bsp.free_pages(plan, torch.from_numpy(gone).cuda(), dev, freed := torch.empty_like(dev))
    want = cache.free_pages(refs, gone)
    np.testing.assert_array_equal(freed.cpu().numpy(), want)
    bsp.read_device_status(plan)                 # (more were given back than there were)
    want[5] = 1
    freed.copy_(torch.from_numpy(want))
    beams = np.array([[0, 3, -1, 1]], np.int32)
    table = torch.full((4, 3), -7, dtype=torch.int32, device="cuda")
    bsp.fork_tables(plan, torch.from_numpy(beams).cuda(), freed, freed, table, bsp.fork_workspace(1, 4))
    counts, out, _, _ = cache.fork_tables([3], [6], [[5]], beams, 4, 8, want, np.full((4, 3), -7))
    np.testing.assert_array_equal(table.cpu().numpy(), out)
    np.testing.assert_array_equal(freed.cpu().numpy(), counts)
    moves, tables = bsp.PageMoves(pages), rs.randint(-1, pages, (7, 11)).astype(np.int32)
    renamed = torch.from_numpy(tables).cuda()
    bsp.compact_tables(plan, freed, freed, moves, renamed)
    after, pairs, live, remap, named = cache.compact(counts, tables)
    assert moves.count.tolist() == [len(pairs), live]
    np.testing.assert_array_equal(moves.pairs[:len(pairs)].cpu().numpy(), np.array(pairs).reshape(-1, 2))
    np.testing.assert_array_equal(freed.cpu().numpy(), after)
    np.testing.assert_array_equal(moves.remap.cpu().numpy(), remap)
    np.testing.assert_array_equal(renamed.cpu().numpy(), named)
    assert bsp.read_device_status(plan) == (0, 0)
