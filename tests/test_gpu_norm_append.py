"""Appends of normalised and rotated rows (bsp_norm_rope_append_kv, its _fp8 form, bsp_append_kv_fp8_blocks) and the
tables of stretched rotations against the fp64 restatements (oracle/cache.py).

Bar: untouched bytes and copied values bit for bit. A normalised and rotated value is an fp32 result rounded once. Its
relative error: the sum of squares takes 8 fused additions and up to 5 of the shuffles, 13 steps of 2^-24, halved by the
root; the mean's scaling, the addition of eps, root, reciprocal and two products add 6 more: under 13 * 2^-24. The
rotation adds the table's 2^-25, a product and a fused multiply-add: under 2.5 * 2^-24 of |x| + |y|. Together under
2^-20 (|x| + |y|), or 2^-20 |x| where nothing is rotated, so the stored value lies between the roundings of v - delta and
v + delta. A block's exponent is the one that its rows' largest magnitude, off by delta, gives.
"""
import numpy as np
import pytest
import torch

import oracle
from beam_search_shared_gb300 import bsp
from oracle import cache

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}
REL = 2.0 ** -20


def to16(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.float64).to(TDT[dtype])  # one rounding


def between16(got, v, delta, dtype):
    lo, hi = (torch.from_numpy(x).to(TDT[dtype]) for x in (v - delta, v + delta))
    return (got >= lo) & (got <= hi) | (got == lo)


class Tokens:
    """New tokens of a step or a prompt: one projection's output, positions, slots, a plan that bounds them."""

    def __init__(self, dtype="bf16", Hq=8, Hkv=4, D=128, ps=32, pages=40, n=45, seed=0, prefill=False, kv_dtype=0, spread=1.0):
        rs = np.random.RandomState(seed)
        self.dtype, self.Hq, self.Hkv, self.D, self.ps, self.pages, self.n = dtype, Hq, Hkv, D, ps, pages, n
        self.geo = bsp.geometry(Hq, Hkv, D, ps, pages, dtype, kv_dtype)
        self.ws = bsp.Workspace(self.geo, 1, max(n, 1), 1)
        if prefill:
            self.ws = bsp.Workspace(self.geo, 1, n, -(-n // ps))
            self.plan = bsp.plan_prefill(self.geo, 1, [0], [n], np.arange(-(-n // ps))[None], True, self.ws)
        else:
            self.plan = self.ws.plan(self.geo, 1, max(n, 1), [0], [0], np.zeros((1, 1), np.int32))
        width = (Hq + 2 * Hkv) * D
        x = rs.randn(n, width) * np.exp(spread * rs.randn(n, 1))
        self.x = torch.from_numpy(x).to(TDT[dtype])
        self.dev = self.x.cuda()
        self.q, self.k, self.v = self.dev.split([Hq * D, Hkv * D, Hkv * D], 1)
        self.qw, self.kw = (torch.from_numpy(1 + 0.3 * rs.randn(D)) for _ in range(2))
        self.slots = rs.permutation(pages * ps)[:n].astype(np.int32)
        self.positions = rs.randint(0, 500, n).astype(np.int32)

    def rows(self, which):
        a, b = {"q": (0, self.Hq), "k": (self.Hq, self.Hq + self.Hkv), "v": (self.Hq + self.Hkv, self.Hq + 2 * self.Hkv)}[which]
        return self.x[:, a * self.D:b * self.D].double().numpy().reshape(self.n, b - a, self.D)

    def loc(self):
        return torch.from_numpy(self.slots).cuda()

    def pos(self):
        return torch.from_numpy(self.positions).cuda()


CASES = [
    # dtype, Hq, Hkv, D, rot (0: none), interleaved, weights (None, "same", "fp32"), offset, scaling
    ("bf16", 16, 8, 128, 128, False, "same", 0.0, None),
    ("fp16", 32, 8, 128, 64, True, "same", 0.0, "ramp"),
    ("bf16", 6, 2, 64, 32, False, "fp32", 1.0, None),
    ("fp16", 4, 4, 64, 64, True, None, 0.0, "bands"),
    ("bf16", 8, 1, 256, 96, False, "fp32", 0.0, "linear"),   # partners 6 chunks apart
    ("fp16", 8, 2, 256, 256, True, "same", 1.0, "base"),
    ("bf16", 3, 3, 128, 0, False, "same", 0.0, None),        # no rotation
]
SCALED = dict(ramp=dict(factor=8.0, original_positions=64, low=1.0, high=8.0, amplitude=1.25),
              bands=dict(factor=8.0, original_positions=64, low=1.0, high=4.0), linear=dict(factor=4.0), base=dict(factor=3.0))


def setup(t, case):
    dtype, Hq, Hkv, D, rot, inter, weights, offset, kind = case
    wt = {None: None, "same": TDT[dtype], "fp32": torch.float32}[weights]
    qw, kw = (None, None) if wt is None else (t.qw.to(wt), t.kw.to(wt))
    norm = bsp.QkNorm(*(None if w is None else w.cuda() for w in (qw, kw)), eps=1e-5, weight_offset=offset)
    rope = theta = None
    amp = 1.0
    if rot:
        kw_ = SCALED.get(kind, {})
        scaling = None if kind is None else bsp.RopeScaling(kind, **kw_)
        rope = bsp.Rope(500, rot, 1e4, interleaved=inter, scaling=scaling)
        amp = kw_.get("amplitude", 1.0)
        theta = cache.frequencies(rot, 1e4, kind, kw_.get("factor", 1.0), kw_.get("original_positions", 0), kw_.get("low", 0), kw_.get("high", 0))

    def want(which):
        w = {"q": qw, "k": kw}[which]
        return cache.norm_rotate(t.rows(which), None if w is None else w.double().numpy(), float(np.float32(1e-5)), offset, t.positions, theta, rot, inter, amp)
    return norm, rope, want


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-D{c[3]}-rot{c[4]}-{c[6]}-{c[8]}")
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_append(case, in_place):
    dtype, Hq, Hkv, D = case[:4]
    t = Tokens(dtype, Hq, Hkv, D, n=45)
    norm, rope, want = setup(t, case)
    t.slots[[3, 17]] = [-1, t.pages * t.ps]      # skipped tokens
    bad = [3, 17]
    if rope is not None:
        t.positions[[9, 21]] = [-1, 500]
        bad += [9, 21]
    pools = [torch.full((t.pages, Hkv, t.ps, D), 7.0, dtype=TDT[dtype], device="cuda") for _ in range(2)]
    q_out = t.q if in_place else torch.full((t.n, Hq, D), 3.0, dtype=TDT[dtype], device="cuda")
    before = t.dev.clone()
    bsp.norm_rope_append_kv(t.plan, norm, rope, t.pos() if rope else None, t.q, t.k, t.v, t.loc(), *pools, q_out=None if in_place else q_out)
    st, flags = bsp.read_device_status(t.plan)
    assert flags == bsp.DEVFLAG_PAGE_INDEX | (bsp.DEVFLAG_POSITION if rope else 0)
    live = np.setdiff1d(np.arange(t.n), bad)
    safe = t.positions.copy()
    t.positions = np.clip(safe, 0, 499)
    got_q = q_out.reshape(t.n, Hq, D).cpu()
    v, size = want("q")
    assert between16(got_q, v, REL * size, dtype)[live].all()
    left = before[:, :Hq * D].reshape(t.n, Hq, D).cpu() if in_place else torch.full((t.n, Hq, D), 3.0, dtype=TDT[dtype])
    assert torch.equal(got_q[bad], left[bad])
    assert torch.equal(t.dev[:, Hq * D:], before[:, Hq * D:])
    v, size = want("k")
    flat = [p.transpose(1, 2).reshape(-1, Hkv, D).cpu() for p in pools]
    at = t.slots[live]
    assert between16(flat[0][at], v[live], REL * size[live], dtype).all()
    assert torch.equal(flat[1][at], t.x[:, (Hq + Hkv) * D:].reshape(t.n, Hkv, D)[live])
    rest = np.setdiff1d(np.arange(t.pages * t.ps), at)
    assert all((f[rest] == 7.0).all() for f in flat)


@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[4]], ids=lambda c: f"{c[0]}-D{c[3]}")
def test_norm_rope_append_fp8(case):
    dtype, Hq, Hkv, D = case[:4]
    t = Tokens(dtype, Hq, Hkv, D, n=37, seed=3)
    norm, rope, want = setup(t, case)
    pools = [torch.full((t.pages, Hkv, t.ps, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q_out = torch.zeros((t.n, Hq, D), dtype=TDT[dtype], device="cuda")
    bsp.norm_rope_append_kv_fp8(t.plan, norm, rope, t.pos(), t.q, t.k, t.v, t.loc(), *pools, k_mul=3.0, v_mul=0.7, q_out=q_out)
    assert bsp.read_device_status(t.plan) == (0, 0)
    v, size = want("q")
    assert between16(q_out.cpu(), v, REL * size, dtype).all()
    flat = [cache.DECODE[p.transpose(1, 2).reshape(-1, Hkv, D).cpu().numpy()] for p in pools]
    v, size = want("k")
    between8(flat[0][t.slots], 3.0 * v, 3.0 * REL * size)
    between8(flat[1][t.slots], float(np.float32(0.7)) * t.rows("v"), 2.0 ** -23 * np.abs(t.rows("v")))
    rest = np.setdiff1d(np.arange(t.pages * t.ps), t.slots)
    assert all((f[rest] == cache.DECODE[0x55]).all() for f in flat)


def between8(got, v, delta):
    lo, hi = cache.DECODE[cache.round_e4m3(v - delta)], cache.DECODE[cache.round_e4m3(v + delta)]
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), (np.argwhere(~ok)[:3], got[~ok][:3], v[~ok][:3])


def check_blocks(t, block, new, size, before, after, eb, ea):
    """Pools and exponents (codes [pages, heads, slots, D], bytes [pages, heads, blocks]) before and after a call that
    wrote rows `new` [n, heads, D], off by REL * size, to t.slots."""
    ps = t.ps
    rows = lambda x: x.transpose(0, 2, 1, 3).reshape(-1, t.Hkv, t.D)  # noqa: E731 - [slots of the pool][heads][D]
    exps = lambda x: x.transpose(0, 2, 1).reshape(-1, t.Hkv)  # noqa: E731 - [blocks of the pool][heads]
    b4, got, eb, ea = rows(before), rows(after), exps(eb), exps(ea)
    touched_rows, touched_blocks = np.zeros(len(b4), bool), np.zeros(len(eb), bool)
    found = cache.runs(t.slots, block, t.pages * ps)
    heads = [t.slots[i] // block for i, _ in found]
    for i, j in found:
        blk, off = t.slots[i] // block, t.slots[i] % block
        touched_blocks[blk] = True
        first = blk * block
        if heads.count(blk) > 1:  # parted by a skipped token, which the call reports: unspecified
            touched_rows[first:first + block] = True
            continue
        for h in range(t.Hkv):
            v, d = new[i:j, h], REL * size[i:j, h]
            mag = np.abs(np.where(np.isnan(v), 0, v))
            want = {cache.exponent(x, t.dtype) for x in ((mag - np.nan_to_num(d, posinf=0)).max(), mag.max(), (mag + np.nan_to_num(d, posinf=0)).max())}
            old = eb[blk, h] if off else 0
            e = int(ea[blk, h])
            assert e in {max(x, int(old)) for x in want}, (blk, h, e, want, old)
            s = t.slots[i:j]
            nan = np.isnan(v)
            assert np.isnan(cache.DECODE[got[s, h]])[nan].all()
            scale = 2.0 ** (127 - e)
            with np.errstate(invalid="ignore"):
                lo, hi = (cache.DECODE[cache.round_e4m3(np.where(nan, 0, x) * scale)] for x in (v - np.nan_to_num(d, posinf=0), v + np.nan_to_num(d, posinf=0)))
            g = cache.DECODE[got[s, h]]
            assert ((g >= lo) & (g <= hi) | nan).all(), (blk, h)
            lead = np.arange(first, first + off)
            if off and old and e > old:
                np.testing.assert_array_equal(cache.DECODE[got[lead, h]], cache.DECODE[cache.round_e4m3(cache.DECODE[b4[lead, h]] * 2.0 ** (int(old) - e))])
            else:
                np.testing.assert_array_equal(got[lead, h], b4[lead, h])
            touched_rows[lead] = True
        touched_rows[t.slots[i:j]] = True
    np.testing.assert_array_equal(got[~touched_rows], b4[~touched_rows])
    np.testing.assert_array_equal(ea[~touched_blocks], eb[~touched_blocks])


def run_blocks(t, block, norm=None, rope=None, want=None, seed=0, empty=False, q=True):
    rs = np.random.RandomState(seed)
    shape = (t.pages, t.Hkv, t.ps, t.D)
    codes = [rs.randint(0, 0x7f, shape).astype(np.uint8) | (rs.randint(0, 2, shape) << 7).astype(np.uint8) for _ in range(2)]
    exps = [np.zeros((t.pages, t.Hkv, t.ps // block), np.uint8) if empty else rs.randint(113, 126, (t.pages, t.Hkv, t.ps // block)).astype(np.uint8) for _ in range(2)]
    kp, vp = (torch.from_numpy(c).cuda() for c in codes)
    scales = bsp.BlockScales(t.geo, block, k=torch.from_numpy(exps[0]).cuda(), v=torch.from_numpy(exps[1]).cuda())
    q_out = torch.zeros((t.n, t.Hq, t.D), dtype=TDT[t.dtype], device="cuda") if q else None
    bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, t.loc(), kp, vp, scales, norm=norm, rope=rope, positions=t.pos() if rope else None,
                             q=t.q if q else None, q_out=q_out)
    flags = bsp.read_device_status(t.plan)[1]
    k, ksize = want("k") if want else (t.rows("k"), np.zeros_like(t.rows("k")))
    check_blocks(t, block, k, ksize, codes[0], kp.cpu().numpy(), exps[0], scales.k.cpu().numpy())
    v = t.rows("v")
    check_blocks(t, block, v, np.zeros_like(v), codes[1], vp.cpu().numpy(), exps[1], scales.v.cpu().numpy())
    return q_out, flags


def prompt_slots(t, starts, rs):
    """Slots of prompts one after another: request r of len_r tokens from position starts[r], pages in random order."""
    ids = rs.permutation(t.pages)
    out, page0, n = [], 0, t.n
    share = -(-n // len(starts))
    for s in starts:
        m = min(share, n - len(out))
        pos = s + np.arange(m)
        out += list(ids[page0 + pos // t.ps] * t.ps + pos % t.ps)
        page0 += (s + m) // t.ps + 1
    t.slots = np.array(out, np.int32)


@pytest.mark.parametrize("case,ps,block,n,starts", [
    (CASES[0], 32, 32, 200, (0, 5)),            # a scale per page; the second prompt begins inside a block
    (CASES[1], 32, 8, 131, (3, 0, 30)),
    (CASES[2], 16, 1, 77, (0,)),                # a scale per token
    (CASES[3], 64, 32, 97, (31,)),              # a run of one token, then whole blocks over the windows' ends
    (CASES[4], 8, 4, 65, (2, 6)),
    (CASES[5], 128, 32, 300, (17, 100)),
    (CASES[6], 32, 16, 33, (0,)),
], ids=lambda x: str(x) if isinstance(x, (int, tuple)) and not (isinstance(x, tuple) and isinstance(x[0], str)) else "")
@pytest.mark.parametrize("prefill", [False, True])
def test_block_append_of_prompts(case, ps, block, n, starts, prefill):
    dtype, Hq, Hkv, D = case[:4]
    t = Tokens(dtype, Hq, Hkv, D, ps=ps, pages=max(6, 4 * n // ps + 8), n=n, seed=n, prefill=prefill)
    prompt_slots(t, starts, np.random.RandomState(n))
    norm, rope, want = setup(t, case)
    q_out, flags = run_blocks(t, block, norm, rope, want, seed=n)
    assert flags == 0
    v, size = want("q")
    assert between16(q_out.cpu(), v, REL * size, dtype).all()


@pytest.mark.parametrize("dtype,D,block,spread", [("bf16", 128, 8, 3.0), ("fp16", 64, 16, 1.0), ("bf16", 256, 2, 2.0), ("fp16", 128, 1, 1.0)])
@pytest.mark.parametrize("prefill", [False, True])
def test_block_append_of_single_tokens(dtype, D, block, spread, prefill):
    """A token per beam into blocks that hold rows: scales that grow, and that stay."""
    t = Tokens(dtype, 4, 2, D, ps=16, pages=90, n=83, seed=5, spread=spread, prefill=prefill)
    rs = np.random.RandomState(6)
    t.slots = (rs.permutation(90)[:83] * 16 + rs.randint(0, 16, 83)).astype(np.int32)
    _, flags = run_blocks(t, block, seed=7)
    assert flags == 0
    run_blocks(t, block, seed=8, empty=True)


@pytest.mark.parametrize("prefill", [False, True])
def test_block_append_extremes(prefill):
    """Zeros, infinities, NaN, the largest and smallest values, and skipped tokens that part a run."""
    for dtype in ("bf16", "fp16"):
        t = Tokens(dtype, 2, 1, 64, ps=32, pages=8, n=40, seed=9, prefill=prefill)
        t.slots = np.arange(35, 75).astype(np.int32)
        x = t.x.view(t.n, 4, 64)
        x[0:3] = 0
        x[4, :, 0], x[6, :, 1] = float("inf"), float("nan")
        x[7, 2:] = float("nan")
        x[30] = 0
        x[31:35] = torch.finfo(TDT[dtype]).smallest_subnormal if hasattr(torch.finfo(TDT[dtype]), "smallest_subnormal") else torch.finfo(TDT[dtype]).tiny
        x[38] = torch.finfo(TDT[dtype]).max
        t.dev.copy_(t.x)
        for block in (1, 4, 32):
            run_blocks(t, block, seed=10)
        t.slots[[8, 20]] = [-5, 8 * 32]
        _, flags = run_blocks(t, 8, seed=11)
        assert flags == bsp.DEVFLAG_PAGE_INDEX


def test_block_append_again_and_one_by_one():
    """The same call again changes nothing; a prompt token by token reaches the exponents of the prompt at once."""
    t = Tokens("bf16", 2, 2, 128, ps=32, pages=6, n=64, seed=12)
    t.slots = np.arange(32, 96).astype(np.int32)
    pools = [torch.zeros((6, 2, 32, 128), dtype=torch.uint8, device="cuda") for _ in range(4)]
    one, two = (bsp.BlockScales(t.geo, 32) for _ in range(2))
    loc = t.loc()
    for _ in range(2):
        bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, loc, pools[0], pools[1], one)
        kept = [x.clone() for x in (pools[0], pools[1], one.k, one.v)]
    bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, loc, pools[0], pools[1], one)
    assert all(torch.equal(a, b) for a, b in zip(kept, (pools[0], pools[1], one.k, one.v)))
    for i in range(t.n):
        bsp.append_kv_fp8_blocks(t.plan, t.k[i:i + 1], t.v[i:i + 1], loc[i:i + 1], pools[2], pools[3], two)
    assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v)
    # a code brought to a larger scale was rounded twice: a step of its value, half a step of the direct one
    a, b = (cache.dequantise(p.cpu().numpy(), s.cpu().numpy()) for p, s in ((pools[0], one.k), (pools[2], two.k)))
    assert (np.abs(a - b) <= 2.0 ** -3 * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -9 * np.repeat(cache.scale_of(one.k.cpu().numpy()), 32, 2)[..., None]).all()


@pytest.mark.parametrize("kind", [None, "linear", "base", "bands", "ramp"])
def test_scaled_tables(kind):
    for n, rot, base in ((3000, 128, 1e6), (77, 48, 1e4), (9, 16, 500.0)):
        kw = SCALED.get(kind, {})
        r = bsp.Rope(n, rot, base, scaling=None if kind is None else bsp.RopeScaling(kind, **kw))
        theta = cache.frequencies(rot, base, kind, kw.get("factor", 1.0), kw.get("original_positions", 0), kw.get("low", 0), kw.get("high", 0))
        angle = np.arange(n)[:, None] * theta
        want = np.concatenate([np.cos(angle), np.sin(angle)], 1) * kw.get("amplitude", 1.0)
        # half an fp32 step of values up to 1.25, and what an angle of 3000 loses in 64 bits
        assert np.abs(r.cos_sin.double().cpu().numpy() - want).max() <= 2.0 ** -24 + 1e-11


def test_no_tokens_and_one():
    t = Tokens("bf16", 2, 2, 64, n=1, pages=3)
    pools = [torch.zeros((3, 2, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    bsp.norm_rope_append_kv(t.plan, bsp.QkNorm(), None, None, None, t.k[:0], t.v[:0], none, *pools)
    assert all((p == 0).all() for p in pools)
    bsp.norm_rope_append_kv(t.plan, bsp.QkNorm(eps=0.0), None, None, None, t.k, t.v, t.loc(), *pools)
    v, size = cache.norm_rotate(t.rows("k"), None, 0.0, 0.0, None, None, 0, False)
    got = pools[0].transpose(1, 2).reshape(-1, 2, 64).cpu()[t.slots]
    assert between16(got, v, REL * size, "bf16").all()


def test_refusals_on_the_device():
    t = Tokens("bf16", 4, 2, 64, n=8)
    pools = [torch.zeros((t.pages, 2, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    call = lambda **kw: bsp.norm_rope_append_kv(  # noqa: E731
        t.plan, kw.pop("norm", bsp.QkNorm()), None, None, kw.pop("q", t.q), kw.pop("k", t.k), kw.pop("v", t.v), t.loc(), *pools, **kw)
    for bad in (dict(q_out=t.dev[:, 128:384]),                       # over q and k, not q itself
                dict(norm=bsp.QkNorm(torch.ones(64, dtype=torch.bfloat16))),  # host memory
                dict(q_out=torch.zeros((8, 4, 64), dtype=torch.bfloat16)),
                dict(norm=bsp.QkNorm(eps=-1.0))):
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):
            call(**bad)
    assert all((p == 0).all() for p in pools)
    with pytest.raises(bsp.BspError, match="UNSUPPORTED"):  # a block larger than the limit
        t64 = Tokens("bf16", 2, 1, 64, ps=64, n=4)
        z = torch.zeros((t64.pages, 1, 64, 64), dtype=torch.uint8, device="cuda")
        bsp.append_kv_fp8_blocks(t64.plan, t64.k, t64.v, t64.loc(), z, z.clone(), bsp.BlockScales(t64.geo, 64))


def test_replayed_on_another_stream_and_in_a_prefill():
    t = Tokens("fp16", 4, 2, 128, n=50, seed=14, prefill=True)
    t.slots = np.arange(50).astype(np.int32)
    loc, pos = t.loc(), t.pos()
    rope = bsp.Rope(500, 128, 1e4)
    norm = bsp.QkNorm(t.qw.half().cuda(), t.kw.half().cuda())
    kp, vp = (torch.zeros((t.pages, 2, 32, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = bsp.BlockScales(t.geo, 16)
    q_out = torch.zeros((50, 4, 128), dtype=torch.float16, device="cuda")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, loc, kp, vp, scales, norm=norm, rope=rope, positions=pos, q=t.q, q_out=q_out)
    assert (kp == 0).all()
    g.replay()
    torch.cuda.synchronize()
    want = [x.clone() for x in (kp, vp, scales.k, scales.v, q_out)]
    kp.zero_(), vp.zero_(), scales.k.zero_(), scales.v.zero_(), q_out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        bsp.append_kv_fp8_blocks(t.plan, t.k, t.v, loc, kp, vp, scales, norm=norm, rope=rope, positions=pos, q=t.q, q_out=q_out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (kp, vp, scales.k, scales.v, q_out)))
    assert not (kp == 0).all()
