"""Plain 64-bit restatements of the paged cache's writes and page bookkeeping (numpy, on the host): normalised and
rotated rows, blocks of E4M3 codes with a power-of-two scale, forked, freed and compacted pages."""
import math

import numpy as np

from . import e4m3_to_double

DECODE = np.array([e4m3_to_double(i) for i in range(256)])
_POSITIVE = DECODE[:0x7f]  # 0 .. 448, ascending with the code


def round_e4m3(x):
    """Nearest E4M3 codes of an array: ties to the even code, magnitudes past 448 to 448, NaN to a NaN code."""
    x = np.asarray(x, np.float64)
    m = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.searchsorted(_POSITIVE, m)            # first code with a value of at least m
    lo = np.maximum(hi - 1, 0)
    below, above = m - _POSITIVE[lo], _POSITIVE[hi] - m
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 0x7f, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def frequencies(rot, base, kind=None, factor=1.0, original=0, low=0.0, high=0.0):
    """theta_j of the rotation's pairs, by the definitions of bsp_rope_scaling."""
    if kind == "base":
        base = base * factor ** (rot / (rot - 2))
    theta = np.array([base ** (-2.0 * j / rot) for j in range(rot // 2)])
    if kind == "linear":
        return theta / factor
    if kind == "bands":
        out = []
        for t in theta:
            s = min(max((original * t / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            out.append(t * ((1 - s) / factor + s))
        return np.array(out)
    if kind == "ramp":
        index = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
        s = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return theta / factor * s + theta * (1 - s)
    return theta


def norm_rotate(x, weight, eps, offset, positions, theta, rot, interleaved, amplitude=1.0):
    """Rows x [n, heads, D] (float64) normalised (eps None: not; weight None: ones) and rotated (theta None: not), and for
    each value the sum of magnitudes that a rounding error of the computation is relative to."""
    x = np.asarray(x, np.float64)
    if eps is not None:
        w = 1.0 if weight is None else np.asarray(weight, np.float64) + offset
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, size = x.copy(), np.abs(x)
    if theta is not None:
        angle = np.asarray(positions, np.float64)[:, None] * theta
        c, s = np.cos(angle)[:, None] * amplitude, np.sin(angle)[:, None] * amplitude
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
        both = (np.abs(x[..., i]) + np.abs(x[..., j])) * amplitude
        size[..., i], size[..., j] = both, both
    return y, size


def exponent(top, dtype):
    """The exponent byte of a block whose new rows reach `top`."""
    if not top > 0:
        return 0
    lo, hi = (27, 142) if dtype == "bf16" else (112, 134)
    e = lo
    while e < hi and top > 448.0 * 2.0 ** (e - 127):
        e += 1
    return e


def runs(slots, block, num_slots):
    """[(first token, one past the last)] of the runs of a call, -1 or slots outside the pool belonging to none."""
    out = []
    for i, s in enumerate(slots):
        if not 0 <= s < num_slots:
            continue
        if out and out[-1][1] == i and slots[i - 1] // block == s // block:
            out[-1][1] = i + 1
        else:
            out.append([i, i + 1])
    return out


def scale_of(exps):
    return np.exp2(np.asarray(exps, np.float64) - 127)


def dequantise(pool, exps):
    """Values of codes [pages, heads, slots, D] with exponent bytes [pages, heads, blocks]."""
    block = pool.shape[2] // exps.shape[2]
    return DECODE[pool] * np.repeat(scale_of(exps), block, 2)[..., None]


def free_pages(refs, tables):
    refs = refs.copy()
    for p in tables.ravel():
        if 0 <= p < len(refs) and refs[p] > 0:
            refs[p] -= 1
    return refs


def compact(refs, tables):
    """(refs, pairs, live, remap, tables) after a compaction."""
    live = [p for p in range(len(refs)) if refs[p] > 0]
    L = len(live)
    holes = [p for p in range(L) if refs[p] <= 0]
    pairs = list(zip([p for p in live if p >= L], holes))
    remap = np.arange(len(refs))
    out = np.maximum(refs, 0)
    for a, b in pairs:
        remap[a] = b
        out[b], out[a] = refs[a], 0
    inside = (tables >= 0) & (tables < len(refs))
    return out, pairs, L, remap, np.where(inside, remap[np.where(inside, tables, 0)], tables)


def fork_tables(prefix, tail, prefix_pages, beams, W, ps, refs, pages_out):
    """(refs, pages_out, served) of bsp_fork_tables."""
    refs, out = refs.copy(), pages_out.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    forks = beams.shape[1]
    used, short = 0, False
    served = np.zeros(beams.size, bool)
    for i in range(beams.size):
        b, w = i // forks, beams.ravel()[i]
        L, full = prefix[b] + tail[b], prefix[b] // ps
        n = -(-L // ps) - full
        row = np.full(full + n, -1)
        if 0 <= w < W:
            # (what a row that came too late would have taken is counted as taken)
            if used + n <= len(free):
                row[:full] = prefix_pages[b][:full]
                row[full:] = free[used:used + n]
                refs[row[:full]] += 1
                refs[row[full:]] = 1
                served[i] = True
            else:
                short = True
            used += n
        out[i, :full + n] = row
    return refs, out, served, short


def fork_sources(prefix, tail, prefix_pages, beam_pages, ci, beams, W, ps):
    """For each row, [(position, source page)] of the rows that its fresh pages take."""
    out = []
    for i, w in enumerate(beams.ravel()):
        b = i // beams.shape[1]
        P, L = prefix[b], prefix[b] + tail[b]
        rows = []
        if 0 <= w < W:
            for pos in range(P // ps * ps, L):
                rows.append((pos, prefix_pages[b][pos // ps] if pos < P else beam_pages[b * W + ci[b, w, pos], pos // ps]))
        out.append(rows)
    return out
