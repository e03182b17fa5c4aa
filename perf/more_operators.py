"""The paged cache around the attention, as a user calls it, and its plain forms.

Five operators that write, read and keep the pages of the K/V cache:

* append: the step's (or a prompt's) keys and queries normalised per head and rotated by their positions,
  keys and values written to their slots of 16-bit pools, queries to a buffer of their own;
* append8: the same into 8-bit (E4M3) pools with a power-of-two scale for each block of tokens and head;
* attend: a beam step's attention over such pools, prompt and tails;
* fork: beams become sequences of their own: full prompt pages shared, fresh pages taken for the rest and
  filled with the prompt's last rows and the beam's tail rows;
* compact: the pages of finished sequences given back and the live pages moved to the lowest page ids.

``own`` chooses between the framework's calls and elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
TAIL = 8  # positions that a beam's own pages have room for
E4M3_MAX = 448.0
# exponents of the block scales that a write chooses: every product of a code and its scale is a number of
# the 16-bit type (fp16: a multiple of 2^-24 below 2^16; bf16: far from its ends)
EXPONENTS = {"bf16": (-100, 15), "fp16": (-15, 7)}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one interactive request of four beams
        dict(name="append_b1_w4_d128_bf16", op="append", kind="decode", batch=1, beam=4, q_heads=16, kv_heads=8, dim=128,
             dtype="bf16", page=32, lo=500, hi=500, rotary=128, interleaved=False, scaled=False),
        # a served step of a small dense layer
        dict(name="append_b64_w30_d128_bf16", op="append", kind="decode", batch=64, beam=30, q_heads=16, kv_heads=8,
             dim=128, dtype="bf16", page=32, lo=400, hi=600, rotary=128, interleaved=False, scaled=False),
        # ragged prompts at far positions of a model stretched beyond its trained length, half of each head rotated
        dict(name="append_prefill_b4_s1024_d128_fp16", op="append", kind="prefill", batch=4, beam=1, q_heads=32,
             kv_heads=8, dim=128, dtype="fp16", page=32, lo=800, hi=1024, rotary=64, interleaved=True, scaled=True),
        # every beam of the widest step into 8-bit pages, blocks of 8 tokens partly filled
        dict(name="append8_b128_w96_d128_bf16_block8", op="append8", kind="decode", batch=128, beam=96, q_heads=16,
             kv_heads=8, dim=128, dtype="bf16", page=8, block=8, lo=2800, hi=3200, rotary=128, interleaved=False,
             scaled=False),
        # prompts into 8-bit pages, one scale for each page and head
        dict(name="append8_prefill_b4_s1024_d128_fp16_block32", op="append8", kind="prefill", batch=4, beam=1,
             q_heads=32, kv_heads=8, dim=128, dtype="fp16", page=32, block=32, lo=800, hi=1024, rotary=128,
             interleaved=False, scaled=False),
        # one long prompt, few beams; a served batch; the widest step
        dict(name="attend_b1_w4_p10000_d128_fp16_block32", op="attend", batch=1, beam=4, q_heads=32, kv_heads=8, dim=128,
             dtype="fp16", page=32, block=32, lo=10000, hi=10000, tail_lo=3, tail_hi=3),
        dict(name="attend_b64_w30_p500_d128_bf16_block32", op="attend", batch=64, beam=30, q_heads=16, kv_heads=8,
             dim=128, dtype="bf16", page=32, block=32, lo=400, hi=600, tail_lo=0, tail_hi=4),
        dict(name="attend_b128_w96_p3000_d128_bf16_block8", op="attend", batch=128, beam=96, q_heads=16, kv_heads=8,
             dim=128, dtype="bf16", page=32, block=8, lo=2800, hi=3200, tail_lo=0, tail_hi=3),
        # the two best of four hypotheses go on by themselves; every beam of a served batch does
        dict(name="fork_b1_w4_n2_d128_bf16", op="fork", batch=1, beam=4, forks=2, q_heads=16, kv_heads=8, dim=128,
             dtype="bf16", page=32, lo=500, hi=500, tail_lo=5, tail_hi=5, spare=64),
        dict(name="fork_b64_w30_n30_d128_bf16", op="fork", batch=64, beam=30, forks=30, q_heads=16, kv_heads=8, dim=128,
             dtype="bf16", page=32, lo=400, hi=600, tail_lo=4, tail_hi=8, spare=4000),
        # a small pool, and one of a gigabyte that half of its sequences leave
        dict(name="compact_n96_d128_fp16", op="compact", pages=96, rows=4, cols=12, done=0.5, kv_heads=8, dim=128,
             dtype="fp16", page=32),
        dict(name="compact_n8192_d128_bf16", op="compact", pages=8192, rows=256, cols=28, done=0.5, kv_heads=8, dim=128,
             dtype="bf16", page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    # no dearer than the listed ones, and its pools within a few gigabytes
    while case["op"] != "compact" and case["batch"] * case["beam"] > 1:
        w, rows = work(case), case["batch"] * case["beam"]
        pool = (rows * (case["page"] + TAIL) + case["batch"] * case["hi"] + case.get("spare", 0) * case["page"])
        if w["bytes"] < 6e8 and w["flops"] < 2e11 and pool * case["kv_heads"] * case["dim"] < 1e9:
            break
        which = "batch" if case["batch"] > 1 else "beam"
        case[which] = max(1, case[which] // 2)
        if case["op"] == "fork":
            case["forks"] = min(case["forks"], case["beam"])
            case["spare"] = 2 * case["batch"] * case["beam"] + 5
    return case


def _draw(rng):
    op = rng.choice(["append", "append8", "attend", "fork", "compact"])
    page = rng.choice([8, 16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8])
    if op == "compact":
        dim = rng.choice([64, 128, 256])
        most = int(5e8 / (page * kv * dim * 2))
        pages = _log(rng, 10, max(11, min(20000, most)))
        cols = rng.randint(1, max(1, min(40, pages // 2)))
        return dict(op=op, pages=pages, rows=max(1, int(pages * rng.uniform(0.3, 0.95) / cols)), cols=cols,
                    done=rng.uniform(0.05, 0.95), kv_heads=kv, dim=dim, dtype=dtype, page=page)
    if op in ("append", "append8"):
        dim = rng.choice([64, 128, 256])
        kind = rng.choice(["prefill", "decode"])
        hi = _log(rng, 1, 4000)
        batch = _log(rng, 1, 128) if kind == "decode" else _log(rng, 1, max(2, 4000 // hi))
        case = dict(op=op, kind=kind, batch=batch, beam=_log(rng, 1, 96) if kind == "decode" else 1,
                    q_heads=kv * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv, dim=dim, dtype=dtype, page=page,
                    lo=max(1, hi // rng.randint(1, 4)), hi=hi, rotary=16 * rng.randint(1, dim // 16),
                    interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5)
        if op == "append8":
            case["block"] = rng.choice([n for n in (1, 2, 4, 8, 16, 32) if n <= page])
        return case
    hi = _log(rng, 1, 8000)
    case = dict(op=op, batch=min(_log(rng, 1, 64), max(1, 200000 // hi)), beam=_log(rng, 1, 96),
                q_heads=kv * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv, dim=rng.choice([64, 128]), dtype=dtype, page=page,
                lo=max(1, hi // rng.randint(1, 4)), hi=hi, tail_lo=0, tail_hi=rng.randint(0, TAIL))
    if op == "attend":
        case["block"] = rng.choice([n for n in (1, 2, 4, 8, 16, 32) if n <= page])
    else:
        case.update(forks=rng.randint(1, case["beam"]), spare=2 * case["batch"] * case["beam"] + rng.randint(0, 200))
    return case


# ---------------------------------------------------------------- what a program holds before a call

def _pages(case, rs, lens, spare):
    """A beam step's pages: the full pages of each prompt shared by its beams, the page of the prompt's last rows
    and those of the tail private to each beam (of them beam 0's hold the prompt's). [batch][..] prompt pages,
    [batch * beam][..] pages of each beam (-1 behind the last), pages in all."""
    page, beam = case["page"], case["beam"]
    full = lens // page
    mine = -(-(lens + TAIL) // page) - full
    wide = int((full + mine).max())
    total = int((full + mine * beam).sum()) + spare
    ids = rs.permutation(total).astype(np.int32)
    of_beam = np.full((len(lens), beam, wide), -1, np.int32)
    at = 0
    for b in range(len(lens)):
        f, m = int(full[b]), int(mine[b])
        of_beam[b, :, :f] = ids[at:at + f]
        at += f
        of_beam[b, :, f:f + m] = ids[at:at + m * beam].reshape(beam, m)
        at += m * beam
    prompt = of_beam[:, 0].copy()
    prompt[np.arange(wide)[None] >= -(-lens // page)[:, None]] = -1
    return prompt, of_beam.reshape(-1, wide), total


def _codes(shape, gen):
    """Random E4M3 codes as bytes: what normally distributed values become."""
    x = (torch.randn(shape, generator=gen, device="cuda") * 70).clamp_(-E4M3_MAX, E4M3_MAX)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _exponents(shape, gen, lo=119, hi=123):
    """Random block scales: the exponents e of 2^(e - 127), a byte each."""
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.uint8)


def _angles(case, positions):
    """cos and sin of the rotation by a stretched model's frequencies, [positions][rotary / 2] each, computed in
    64 bits and rounded once."""
    rot, base = case["rotary"], 1e6
    j = torch.arange(rot // 2, dtype=torch.float64)
    theta = base ** (-2 * j / rot)
    amplitude = 1.0
    if case["scaled"]:
        factor, trained = 8.0, 4096
        edge = lambda turns: rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(edge(32.0))), min(rot - 1, math.ceil(edge(1.0)))
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        theta = theta / factor * ramp + theta * (1 - ramp)
        amplitude = 0.1 * math.log(factor) + 1
    angle = torch.arange(positions, dtype=torch.float64)[:, None].cuda() * theta.cuda()
    return torch.cos(angle) * amplitude, torch.sin(angle) * amplitude


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    op, dt = case["op"], DTYPES[case["dtype"]]
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    s = dict(case=case)
    bsp = None
    if own:
        from beam_search_shared_gb300 import bsp
        s["bsp"] = bsp
    if op == "compact":
        return _prepare_compact(case, s, gen, rs, bsp)
    batch, beam = case["batch"], case["beam"]
    q_heads = case["q_heads"]
    # the lengths go by the case, so that every seed's outputs have the same shapes
    sizes = np.random.RandomState(7 * case["hi"] + case["lo"] + batch)
    lens = sizes.randint(case["lo"], case["hi"] + 1, batch).astype(np.int32)
    zero = np.zeros(batch, np.int32)
    if op in ("append", "append8"):
        prompt, of_beam, total = _pages(case, rs, lens, 3)
        if case["kind"] == "decode":
            pos = np.repeat(lens + rs.randint(0, TAIL, batch), beam)  # each beam's next position
            row = np.arange(batch * beam)
        else:
            pos = np.concatenate([np.arange(n) for n in lens])
            row = np.repeat(np.arange(batch), lens)
        n = len(pos)
        s["slots"] = torch.from_numpy((of_beam[row, pos // page].astype(np.int64) * page + pos % page).astype(np.int32)).cuda()
        if case["scaled"]:
            pos = pos + rs.randint(0, 24000)
        s["positions"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        # one projection's output: queries, keys and values of a token side by side
        width = (q_heads + 2 * kv) * dim
        x = torch.randn((n, width), generator=gen, device="cuda") * torch.exp(
            torch.randn((n, 1), generator=gen, device="cuda"))
        x = x.to(dt)
        s["q"], s["k"], s["v"] = x.split([q_heads * dim, kv * dim, kv * dim], 1)
        s["q_weight"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).to(dt)
        s["k_weight"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).to(dt)
        s["eps"] = 1e-6
        s["q_out"] = torch.empty((n, q_heads, dim), dtype=dt, device="cuda")
        most = int(pos.max()) + 1
        shape = (total, kv, page, dim)
        if op == "append":
            s["k_pool"] = torch.zeros(shape, dtype=dt, device="cuda")
            s["v_pool"] = torch.zeros(shape, dtype=dt, device="cuda")
        else:
            s["k_pool"], s["v_pool"] = _codes(shape, gen), _codes(shape, gen)
            blocks = (total, kv, page // case["block"])
            s["k_scale"], s["v_scale"] = _exponents(blocks, gen), _exponents(blocks, gen)
        if own:
            geo = bsp.geometry(q_heads, kv, dim, page, total, case["dtype"])
            table = prompt if prompt.shape[1] else np.zeros((batch, 1), np.int32)
            if case["kind"] == "decode":
                s["ws"] = bsp.Workspace(geo, batch, beam, table.shape[1])
                s["plan"] = s["ws"].plan(geo, batch, beam, lens, zero, table)
            else:
                s["ws"] = bsp.Workspace(geo, batch, int(lens.max()), table.shape[1])
                s["plan"] = bsp.plan_prefill(geo, batch, zero, lens, table, True, s["ws"])
            s["norm"] = bsp.QkNorm(s["q_weight"], s["k_weight"], s["eps"])
            scaling = None
            if case["scaled"]:
                scaling = bsp.RopeScaling("ramp", factor=8.0, original_positions=4096, low=1.0, high=32.0,
                                          amplitude=0.1 * math.log(8.0) + 1)
            s["rope"] = bsp.Rope(most, case["rotary"], 1e6, interleaved=case["interleaved"], scaling=scaling)
            if op == "append8":
                s["scales"] = bsp.BlockScales(geo, case["block"], k=s["k_scale"], v=s["v_scale"])
        else:
            c, sn = _angles(case, most)
            s["cos"], s["sin"] = c.float(), sn.float()
        return s

    tails = sizes.randint(case["tail_lo"], case["tail_hi"] + 1, batch).astype(np.int32)
    if op == "fork":
        tails = np.maximum(tails, 1)
    prompt, of_beam, total = _pages(case, rs, lens, case.get("spare", 3))
    s["lens"], s["tails"] = torch.from_numpy(lens).cuda(), torch.from_numpy(tails).cuda()
    s["prompt_pages"], s["beam_pages"] = torch.from_numpy(prompt).cuda(), torch.from_numpy(of_beam).cuda()
    s["most"] = int(lens.max())
    s["indirection"] = torch.randint(0, beam, (batch, beam, s["most"] + TAIL + 1), generator=gen, device="cuda",
                                     dtype=torch.int32)
    shape = (total, kv, page, dim)
    if op == "attend":
        s["k_pool"], s["v_pool"] = _codes(shape, gen), _codes(shape, gen)
        blocks = (total, kv, page // case["block"])
        s["k_scale"], s["v_scale"] = _exponents(blocks, gen), _exponents(blocks, gen)
        rows = batch * beam
        s["q"] = torch.randn((rows, q_heads, dim), generator=gen, device="cuda").to(dt)
        s["o"] = torch.empty((rows, q_heads, dim), dtype=dt, device="cuda")
        s["lse"] = torch.empty((rows, q_heads), device="cuda")
        s["scale"] = dim ** -0.5
        if own:
            geo = bsp.geometry(q_heads, kv, dim, page, total, case["dtype"], kv_dtype=bsp.KV_DTYPE_E4M3)
            s["ws"] = bsp.Workspace(geo, batch, beam, prompt.shape[1])
            s["plan"] = s["ws"].plan(geo, batch, beam, lens, tails, prompt)
            s["scales"] = bsp.BlockScales(geo, case["block"], k=s["k_scale"], v=s["v_scale"])
        return s
    s["k_pool"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    s["v_pool"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    s["refs"] = torch.zeros(total, dtype=torch.int32, device="cuda")
    s["refs"][s["beam_pages"][s["beam_pages"] >= 0].long()] = 1
    s["forks"] = torch.from_numpy(np.stack([rs.permutation(beam)[:case["forks"]] for _ in range(batch)]).astype(np.int32)).cuda()
    n = batch * case["forks"]
    s["refs_out"] = torch.zeros_like(s["refs"])
    s["pages_out"] = torch.full((n, -(-(s["most"] + TAIL) // page)), -1, dtype=torch.int32, device="cuda")
    if own:
        geo = bsp.geometry(q_heads, kv, dim, page, total, case["dtype"])
        s["ws"] = bsp.Workspace(geo, batch, beam, prompt.shape[1])
        s["plan"] = s["ws"].plan(geo, batch, beam, lens, tails, prompt)
        s["fork_ws"] = bsp.fork_workspace(batch, case["forks"])
    return s


def _prepare_compact(case, s, gen, rs, bsp):
    pages, rows, cols = case["pages"], case["rows"], case["cols"]
    kv, dim, page, dt = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    ids = rs.permutation(pages)
    need = min(rows * cols, pages)
    table = np.full(rows * cols, -1, np.int32)
    table[:need] = ids[:need]
    table = table.reshape(rows, cols)
    # every second sequence holds its first page together with the one before
    table[1::2, 0] = table[0:rows - 1:2, 0][:len(table[1::2])]
    length = rs.randint(1, cols + 1, rows)
    table[np.arange(cols)[None] >= length[:, None]] = -1
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    done = rs.random_sample(rows) < case["done"]
    s["tables"] = torch.from_numpy(table).cuda()
    s["finished"] = torch.from_numpy(np.where(done[:, None], table, -1)).cuda()
    s["refs"] = torch.from_numpy(refs).cuda()
    s["refs_freed"] = torch.zeros_like(s["refs"])
    s["refs_out"] = torch.zeros_like(s["refs"])
    s["live"] = torch.from_numpy(np.where(done[:, None], -1, table)).cuda()
    s["live_out"] = torch.zeros_like(s["live"])
    shape = (pages, kv, page, dim)
    s["k_pool"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    s["v_pool"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    if own:
        geo = bsp.geometry(kv, kv, dim, page, pages, case["dtype"])
        s["ws"] = bsp.Workspace(geo, 1, 1, 1)
        s["plan"] = s["ws"].plan(geo, 1, 1, [1], [0], np.zeros((1, 1), np.int32))
        s["moves"] = bsp.PageMoves(pages)
    return s


# ---------------------------------------------------------------- plain forms

def _turn(s, x, weight):
    """Rows [tokens][heads][dim] normalised per head and rotated, in fp32."""
    case = s["case"]
    rot = case["rotary"]
    x = x.float()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    at = s["positions"].long()
    c, sn = s["cos"][at][:, None], s["sin"][at][:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    case = s["case"]
    dt, page = DTYPES[case["dtype"]], case["page"]
    n, kv, dim = len(s["slots"]), case["kv_heads"], case["dim"]
    s["q_out"].copy_(_turn(s, s["q"].unflatten(1, (-1, dim)), s["q_weight"]))
    at, slot = (s["slots"] // page).long(), (s["slots"] % page).long()
    s["k_pool"][at, :, slot] = _turn(s, s["k"].unflatten(1, (kv, dim)), s["k_weight"]).to(dt)
    s["v_pool"][at, :, slot] = s["v"].unflatten(1, (kv, dim))
    return s["q_out"], s["k_pool"], s["v_pool"]


def _write8(s, pool, scale, x):
    """Rows x [tokens][kv heads][dim] into an E4M3 pool. A block that the call begins at its first slot starts anew;
    another keeps its rows. Its scale is the smallest power of two, but none smaller than it was, with which the new
    rows' largest magnitude is at most 448; rows that were there are brought to a larger scale."""
    case = s["case"]
    page, block = case["page"], case["block"]
    lo, hi = EXPONENTS[case["dtype"]]
    slots = s["slots"].long()
    blocks, of = torch.unique(slots // block, return_inverse=True)
    nb, kv = len(blocks), case["kv_heads"]
    top = torch.zeros((nb, kv), device="cuda").scatter_reduce_(0, of[:, None].expand(-1, kv), x.abs().amax(-1), "amax")
    first = torch.full((nb,), block, dtype=torch.int64, device="cuda").scatter_reduce_(0, of, slots % block, "amin")
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(lo, hi) + 127
    e = torch.where(top == 0, 0, e)
    at, which = blocks // (page // block), blocks % (page // block)
    old = torch.where(first[:, None] == 0, 0, scale[at, :, which].int())
    new = torch.maximum(e, old)
    # the rows that were there: [blocks][kv heads][block][dim]
    row = which[:, None] * block + torch.arange(block, device="cuda")
    was = pool[at[:, None], :, row].view(torch.float8_e4m3fn).float()  # [blocks][block][kv heads][dim]
    held = (was * torch.exp2((old - new).float())[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (torch.arange(block, device="cuda") < first[:, None])[..., None, None] & ((new > old) & (old > 0))[:, None, :, None]
    pool[at[:, None], :, row] = torch.where(keep, held, was.to(torch.float8_e4m3fn).view(torch.uint8))
    scale[at, :, which] = new.to(torch.uint8)
    y = (x * torch.exp2(127.0 - new[of].float())[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    pool[(slots // page), :, slots % page] = y.view(torch.uint8)


def _values8(s):
    """8-bit pools and scales as the numbers that they hold."""
    return (s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn),
            s["k_scale"].view(torch.float8_e8m0fnu), s["v_scale"].view(torch.float8_e8m0fnu))


def _append8(s):
    case = s["case"]
    kv, dim = case["kv_heads"], case["dim"]
    s["q_out"].copy_(_turn(s, s["q"].unflatten(1, (-1, dim)), s["q_weight"]))
    _write8(s, s["k_pool"], s["k_scale"], _turn(s, s["k"].unflatten(1, (kv, dim)), s["k_weight"]))
    _write8(s, s["v_pool"], s["v_scale"], s["v"].unflatten(1, (kv, dim)).float())
    return (s["q_out"], *_values8(s))


def _attend(s):
    case = s["case"]
    batch, beam, kv, dim, page, block = (case[k] for k in ("batch", "beam", "kv_heads", "dim", "page", "block"))
    group = case["q_heads"] // kv
    pages = s["prompt_pages"].clamp(min=0).long()
    most = pages.shape[1] * page
    # each beam's tail: pages through the indirection, [rows][TAIL]
    t = torch.arange(TAIL, device="cuda")
    pos = s["lens"][:, None].long() + t
    source = s["indirection"].gather(2, pos[:, None].expand(batch, beam, TAIL)).long()
    source = source + beam * torch.arange(batch, device="cuda")[:, None, None]
    col = (pos // page)[:, None].expand(batch, beam, TAIL).clamp(max=s["beam_pages"].shape[1] - 1)
    at, slot = s["beam_pages"][source, col].clamp(min=0).long(), (pos % page)[:, None].expand(batch, beam, TAIL)

    def prompt(pool, scale):
        x = pool[pages].view(torch.float8_e4m3fn).float()  # [batch][pages][kv][page][dim]
        x = x.unflatten(3, (-1, block)) * torch.exp2(scale[pages].float() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(batch, kv, most, dim)

    def tail(pool, scale):
        x = pool[at, :, slot].view(torch.float8_e4m3fn).float()  # [batch][beam][TAIL][kv][dim]
        return x * torch.exp2(scale[at, :, slot // block].float() - 127)[..., None]

    q = s["q"].float().view(batch, beam, kv, group, dim)
    a = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(batch, kv, beam * group, dim),
                     prompt(s["k_pool"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    a = a.masked_fill((torch.arange(most, device="cuda") >= s["lens"][:, None])[:, None, None], -math.inf)
    b = (q[:, :, None] * tail(s["k_pool"], s["k_scale"])[:, :, :, :, None]).sum(-1) * s["scale"]
    b = b.masked_fill((t >= s["tails"][:, None])[:, None, :, None, None], -math.inf)  # [batch][beam][TAIL][kv][group]
    b = b.permute(0, 3, 1, 4, 2).reshape(batch, kv, beam * group, TAIL)
    top = torch.maximum(a.amax(-1), b.amax(-1))
    safe = torch.where(top == -math.inf, 0, top)[..., None]
    a, b = torch.exp(a - safe), torch.exp(b - safe)
    total = a.sum(-1) + b.sum(-1)
    o = torch.matmul(a, prompt(s["v_pool"], s["v_scale"])).view(batch, kv, beam, group, dim)
    w = b.view(batch, kv, beam, group, TAIL).permute(0, 2, 4, 1, 3)[..., None]
    o = o.permute(0, 2, 1, 3, 4) + (w * tail(s["v_pool"], s["v_scale"])[:, :, :, :, None]).sum(2)
    total = total.view(batch, kv, beam, group).permute(0, 2, 1, 3)
    s["o"].copy_((o / torch.where(total == 0, 1, total)[..., None]).reshape(s["o"].shape))
    s["lse"].copy_((torch.log(total) + safe[..., 0].view(batch, kv, beam, group).permute(0, 2, 1, 3)).reshape(s["lse"].shape))
    return s["o"], s["lse"]


def _fork(s):
    """Fresh pages: the lowest free ones, in the order of the forked rows."""
    case = s["case"]
    batch, beam, forks, page = case["batch"], case["beam"], case["forks"], case["page"]
    lens, tails = s["lens"].long(), s["tails"].long()
    full = lens // page
    need = -(-(lens + tails) // page) - full
    mine = need[:, None].expand(batch, forks).reshape(-1)
    first = torch.cumsum(mine, 0) - mine
    free = (s["refs"] == 0).nonzero()[:, 0]
    col = torch.arange(s["pages_out"].shape[1], device="cuda")
    shared = s["prompt_pages"][:, None].expand(batch, forks, -1).reshape(batch * forks, -1).long()
    shared = torch.nn.functional.pad(shared, (0, max(0, len(col) - shared.shape[1])))[:, :len(col)]
    lead = full[:, None].expand(batch, forks).reshape(-1, 1)
    nth = first[:, None] + col - lead
    own_page = (col >= lead) & (col < lead + mine[:, None])
    pages = torch.where(col < lead, shared, torch.where(own_page, free[nth.clamp(0, len(free) - 1)], -1))
    out = s["pages_out"]
    out.copy_(torch.where(pages >= 0, pages.int(), out))
    s["refs_out"].copy_(s["refs"])
    taken = (pages >= 0).flatten()
    s["refs_out"].index_add_(0, pages.flatten()[taken], torch.ones_like(pages.flatten()[taken], dtype=torch.int32))
    # rows from the last full page's end to the sequence's
    i = torch.arange(page + TAIL, device="cuda")
    pos = full[:, None, None] * page + i
    pos = pos.expand(batch, forks, -1)
    end = (lens + tails)[:, None, None]
    w = s["forks"].long()[:, :, None].expand_as(pos)
    b = torch.arange(batch, device="cuda")[:, None, None].expand_as(pos)
    seat = pos.clamp(max=s["indirection"].shape[2] - 1)
    source = torch.where(pos < lens[:, None, None], 0, s["indirection"][b, w, seat].long())
    cols = s["beam_pages"].shape[1]
    at = s["beam_pages"][b * beam + source, (pos // page).clamp(max=cols - 1)].long()
    to = pages.view(batch, forks, -1).gather(2, (pos // page).clamp(max=len(col) - 1))
    live = pos < end
    at, to, slot = at[live], to[live], (pos % page)[live]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[to, :, slot] = pool[at, :, slot]
    return s["refs_out"], out, s["k_pool"], s["v_pool"]


def _compact(s):
    """The i-th live page behind the first L (L pages are live) goes to the i-th free page of those."""
    gone = s["finished"].flatten()
    gone = gone[gone >= 0].long()
    s["refs_freed"].copy_(s["refs"])
    s["refs_freed"].index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    refs = s["refs_freed"]
    live = refs > 0
    at = torch.arange(len(refs), device="cuda")
    front = at < live.sum()
    to, of = (~live & front).nonzero()[:, 0], (live & ~front).nonzero()[:, 0]
    where = at.clone()
    where[of] = to
    s["live_out"].copy_(torch.where(s["live"] >= 0, where[s["live"].clamp(min=0).long()].int(), s["live"]))
    s["refs_out"].copy_(refs)
    s["refs_out"][to] = refs[of]
    s["refs_out"][of] = 0
    for pool in (s["k_pool"], s["v_pool"]):
        pool[to] = pool[of]
    return s["refs_freed"], s["refs_out"], s["live_out"], s["k_pool"], s["v_pool"]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "append8": _append8, "attend": _attend, "fork": _fork, "compact": _compact}[op](s)
    bsp = s["bsp"]
    if op == "append":
        bsp.norm_rope_append_kv(s["plan"], s["norm"], s["rope"], s["positions"], s["q"], s["k"], s["v"], s["slots"],
                                s["k_pool"], s["v_pool"], q_out=s["q_out"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    if op == "append8":
        bsp.append_kv_fp8_blocks(s["plan"], s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["scales"],
                                 norm=s["norm"], rope=s["rope"], positions=s["positions"], q=s["q"], q_out=s["q_out"])
        return (s["q_out"], *_values8(s))
    if op == "attend":
        bsp.decode_attn_fp8_blocks(s["plan"], s["q"], s["k_pool"], s["v_pool"], s["scales"], s["beam_pages"],
                                   s["indirection"], s["scale"], s["o"], s["lse"])
        return s["o"], s["lse"]
    if op == "fork":
        bsp.fork_tables(s["plan"], s["forks"], s["refs"], s["refs_out"], s["pages_out"], s["fork_ws"])
        bsp.fork_rows(s["plan"], s["forks"], s["pages_out"], s["beam_pages"], s["indirection"], s["k_pool"], s["v_pool"])
        return s["refs_out"], s["pages_out"], s["k_pool"], s["v_pool"]
    bsp.free_pages(s["plan"], s["finished"], s["refs"], s["refs_freed"])
    bsp.compact_tables(s["plan"], s["refs_freed"], s["refs_out"], s["moves"], s["live"], s["live_out"])
    bsp.copy_pages(s["plan"], s["moves"], s["k_pool"], s["v_pool"])
    return s["refs_freed"], s["refs_out"], s["live_out"], s["k_pool"], s["v_pool"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "compact":
        n = case["rows"] * case["cols"] / 2  # pages in the tables: lengths are even over 1 .. cols
        live = min(n, case["pages"]) * (1 - case["done"])
        moved = live * max(0.0, 1 - live / case["pages"])
        return {"bytes": int(moved * kv * page * dim * 2 * 4 + 4 * (3 * case["pages"] + 3 * case["rows"] * case["cols"])),
                "flops": case["pages"]}
    batch, beam, q_heads = case["batch"], case["beam"], case["q_heads"]
    mean = (case["lo"] + case["hi"]) / 2
    if case["op"] in ("append", "append8"):
        n = batch * (beam if case["kind"] == "decode" else mean)
        write = 2 if case["op"] == "append" else 1
        far = batch * (1 if case["kind"] == "decode" else mean)  # distinct positions at most
        scales = 0 if case["op"] == "append" else 2 * 2 * kv * (n if case["kind"] == "decode" else n / case["block"])
        return {"bytes": int(n * dim * (q_heads * 4 + 2 * kv * (2 + write)) + 8 * n + 4 * far * case["rotary"] + scales),
                "flops": int(n * dim * (q_heads + kv) * 8)}
    tail = (case["tail_lo"] + case["tail_hi"]) / 2
    if case["op"] == "attend":
        rows, keys = batch * beam, batch * mean
        held = 2 * kv * (keys + rows * tail) * (dim + 1 / case["block"])
        return {"bytes": int(held + rows * q_heads * (4 * dim + 4)),
                "flops": int(4 * dim * q_heads * rows * (mean + tail))}
    n = batch * case["forks"]
    rows = n * ((page - 1) / 2 + tail)
    cols = -(-(mean + tail) // page)
    return {"bytes": int(rows * kv * dim * 2 * 4 + 4 * n * cols + 8 * batch * mean * (1 + beam / page)), "flops": int(n)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(case, s, x, weight):
    """Normalised and rotated rows [tokens][heads][dim] in 64 bits, each pair as a complex number."""
    rot = case["rotary"]
    c, sn = _angles(case, int(s["positions"].max()) + 1)
    turn = torch.complex(c, sn)[s["positions"].long()][:, None]
    x = x.double()
    x = x * weight.double() * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_write8(case, slots, pool, scale, x):
    """append8 block by block: values (of the codes) and scales in 64 bits."""
    page, block = case["page"], case["block"]
    lo, hi = EXPONENTS[case["dtype"]]
    value = pool.view(torch.float8_e4m3fn).double()
    power = torch.exp2(scale.double() - 127)
    which = (slots // block).tolist()
    begin = [i for i in range(len(which)) if i == 0 or which[i] != which[i - 1]] + [len(which)]
    for i, j in zip(begin, begin[1:]):
        slot = int(slots[i])
        p, r = slot // page, slot % page
        first = r // block * block
        top = x[i:j].abs().amax((0, 2))  # [kv]
        e = torch.full_like(top, lo)
        for n in range(lo, hi):
            e += top > E4M3_MAX * 2.0 ** n
        new = torch.where(top > 0, torch.exp2(e), 2.0 ** -127)
        if r > first:
            new = torch.maximum(new, power[p, :, r // block])
            value[p, :, first:r] *= (power[p, :, r // block] / new)[:, None, None]
            value[p, :, first:r] = value[p, :, first:r].float().to(torch.float8_e4m3fn).double()
        power[p, :, r // block] = new
        value[p, :, r:r + j - i] = (x[i:j] / new[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).transpose(0, 1).float().to(
            torch.float8_e4m3fn).double()
    return value, power


def exact(case, seed):
    s = prepare(case, seed)
    op, kv, dim, page = case["op"], case["kv_heads"], case["dim"], case["page"]
    if op in ("append", "append8"):
        n = len(s["slots"])
        q = _exact_rows(case, s, s["q"].reshape(n, -1, dim), s["q_weight"])
        k = _exact_rows(case, s, s["k"].reshape(n, kv, dim), s["k_weight"])
        v = s["v"].reshape(n, kv, dim).double()
        if op == "append":
            pools = []
            for pool, x in ((s["k_pool"], k), (s["v_pool"], v)):
                flat = pool.double().transpose(1, 2).reshape(-1, kv, dim)
                flat[s["slots"].long()] = x
                pools.append(flat.view(-1, page, kv, dim).transpose(1, 2).contiguous())
            return q, pools[0], pools[1]
        if n > 5000:
            return q, None, None, None, None
        slots = s["slots"].cpu()
        kval, kpow = _exact_write8(case, slots, s["k_pool"], s["k_scale"], k)
        vval, vpow = _exact_write8(case, slots, s["v_pool"], s["v_scale"], v)
        return q, kval, vval, kpow, vpow
    if op == "attend":
        batch, beam, q_heads, block = case["batch"], case["beam"], case["q_heads"], case["block"]
        group = q_heads // kv
        o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b in range(batch):
            n, t = int(s["lens"][b]), int(s["tails"][b])
            pos = torch.arange(n + t, device="cuda")
            rows = torch.arange(b * beam, (b + 1) * beam, device="cuda")
            pages = s["beam_pages"][b * beam + s["indirection"][b, :, n:n + t].long(), (pos[n:] // page)[None]]
            head = s["prompt_pages"][b, (pos[:n] // page)]

            def held(pool, power, at, slot, g):
                x = pool[at.long(), g, slot].view(torch.float8_e4m3fn).double()
                return x * torch.pow(2.0, power[at.long(), g, slot // block].double() - 127)[..., None]

            for g in range(kv):
                heads = slice(g * group, (g + 1) * group)
                q = s["q"][rows, heads].double()  # [beam][group][dim]
                k1, v1 = (held(s[p + "_pool"], s[p + "_scale"], head, pos[:n] % page, g) for p in "kv")
                k2, v2 = (held(s[p + "_pool"], s[p + "_scale"], pages, (pos[n:] % page).expand(beam, t), g) for p in "kv")
                x = torch.cat((torch.einsum("wgd,kd->wgk", q, k1), torch.einsum("wgd,wtd->wgt", q, k2)), -1) * s["scale"]
                lse[rows, heads] = torch.logsumexp(x, -1)
                p = torch.softmax(x, -1)
                o[rows, heads] = torch.einsum("wgk,kd->wgd", p[..., :n], v1) + torch.einsum("wgt,wtd->wgd", p[..., n:], v2)
        return o, lse
    if op == "fork":
        batch, beam, forks = case["batch"], case["beam"], case["forks"]
        lens, tails, table = s["lens"].tolist(), s["tails"].tolist(), s["beam_pages"].cpu()
        ci, chosen = s["indirection"].cpu(), s["forks"].tolist()
        free = (i for i, r in enumerate(s["refs"].tolist()) if r == 0)
        old = {n: s[n + "_pool"].double() for n in "kv"}
        new = {n: x.clone() for n, x in old.items()}
        for b in range(batch):
            end, full = lens[b] + tails[b], lens[b] // page
            for w in chosen[b]:
                mine = [next(free) for _ in range(-(-end // page) - full)]
                pos = list(range(full * page, end))
                of = [int(table[b * beam + (0 if p < lens[b] else int(ci[b, w, p])), p // page]) for p in pos]
                to = [mine[p // page - full] for p in pos]
                slot = [p % page for p in pos]
                for n in "kv":
                    new[n][to, :, slot] = old[n][of, :, slot]
        return None, None, new["k"], new["v"]
    refs = s["refs"].cpu().numpy().copy()
    gone = s["finished"].cpu().numpy()
    np.subtract.at(refs, gone[gone >= 0], 1)
    held = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(held)
    taken = set(held)
    pairs = list(zip([p for p in range(n) if p not in taken], [p for p in held if p >= n]))
    pools = []
    for name in ("k_pool", "v_pool"):
        x = s[name].double()
        if pairs:
            to, of = (torch.tensor(i, device="cuda") for i in zip(*pairs))
            x[to] = x[of]
        pools.append(x)
    return None, None, None, pools[0], pools[1]
