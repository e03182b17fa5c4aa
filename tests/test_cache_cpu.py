"""Host-side tests of the cache's appends of normalised rows, block scales and page bookkeeping: what the C entry points
and the binding refuse before a launch, the limits and structs that the header states, and the restatements against
their definitions (no CUDA device needed)."""
import ctypes as c
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import oracle
from beam_search_shared_gb300 import bsp, build
from oracle import cache
from test_step_cpu import BUF, CAPACITY, INVALID, OK, ROOT, STALE, UNSUPPORTED, Staged, ptr


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsp.load()


b = ptr(BUF)
ROPE = bsp.RopeConfig(BUF.ctypes.data, 100, 64, 0, 0)


def norm(**kw):
    n = bsp._QkNorm(BUF.ctypes.data, BUF.ctypes.data, 1e-6, 0.0, 0, 0)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def scales(**kw):
    s = bsp._BlockScales(BUF.ctypes.data, BUF.ctypes.data, 16, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


KEEP = []


def staged(**kw):
    """The plan of a Staged, whose staging header lives on."""
    KEEP.append(Staged(**kw))
    return KEEP[-1].plan


def ref(x):
    return None if x is None else c.byref(x)


def head(plan, nrm, rope, q, q_stride, out_stride, stride, q_out=b):
    return (c.byref(plan), ref(nrm), ref(rope), b, b if q else None, q_stride, q_out if q else None, out_stride, b, b, stride)


def append(lib, plan, nrm=norm(), rope=ROPE, q=True, q_stride=1024, out_stride=1024, stride=512, n=4):  # noqa: B008
    return lib.bsp_norm_rope_append_kv(*head(plan, nrm, rope, q, q_stride, out_stride, stride), b, n, b, b, None, None)


def append8(lib, plan, nrm=norm(), rope=ROPE, q=True, q_stride=1024, out_stride=1024, stride=512, n=4, mul=1.0):  # noqa: B008
    return lib.bsp_norm_rope_append_kv_fp8(*head(plan, nrm, rope, q, q_stride, out_stride, stride), mul, 1.0, b, n, b, b, None, None)


def blocks(lib, plan, nrm=norm(), rope=ROPE, q=True, q_stride=1024, out_stride=1024, stride=512, n=4, sc=scales()):  # noqa: B008
    return lib.bsp_append_kv_fp8_blocks(*head(plan, nrm, rope, q, q_stride, out_stride, stride), b, n, b, b, ref(sc), None, None)


def attend(lib, plan, sc=scales(), scale=0.1, flags=0):  # noqa: B008
    return lib.bsp_decode_attn_fp8_blocks(c.byref(plan), b, b, b, ref(sc), b, 10, b, 200, scale, flags, b, b, None, None)


def tables(lib, plan, stride=2, forks=2, out_stride=4, cols=4, ws=1 << 20):
    return lib.bsp_fork_tables(c.byref(plan), b, stride, forks, b, b, b, out_stride, cols, b, ws, None)


def rows(lib, plan, stride=2, forks=2, out_stride=4, cols=4, bps=4, max_seq=200, sc=None):
    return lib.bsp_fork_rows(c.byref(plan), b, stride, forks, b, out_stride, cols, b, bps, b, max_seq, b, b, ref(sc), None)


def free(lib, plan, stride=4, n=3, cols=4):
    return lib.bsp_free_pages(c.byref(plan), b, stride, n, cols, b, b, None)


def compact(lib, plan, stride=4, n=3, cols=4):
    return lib.bsp_compact_tables(c.byref(plan), b, b, b, b, b, b, b, stride, n, cols, None)


def copy(lib, plan, n=3, sc=None):
    return lib.bsp_copy_pages(c.byref(plan), b, b, n, b, b, ref(sc), None)


E4M3 = bsp.KV_DTYPE_E4M3
CALLS = [(append, 0), (append8, 0), (blocks, 0), (attend, E4M3), (tables, 0), (rows, 0), (free, 0), (compact, 0), (copy, 0)]


@pytest.mark.parametrize("call,kv", CALLS)
def test_unstaged_stale_and_host_memory(lib, call, kv):
    s = Staged(kv_dtype=kv)
    assert call(lib, s.plan) == INVALID  # host memory
    s.host[1] = 8
    assert call(lib, s.plan) == STALE
    s.plan.generation = 0
    assert call(lib, s.plan) == INVALID
    assert call(lib, bsp.Plan()) == INVALID


@pytest.mark.parametrize("call", [append, append8, blocks])
def test_append_refusals(lib, call):
    s = Staged()
    assert call(lib, s.plan, n=0) == OK
    for bad in (dict(n=-1), dict(n=9), dict(stride=511), dict(stride=516), dict(q_stride=1023), dict(out_stride=1016),
                dict(out_stride=1028), dict(q_stride=2048)):  # (the last: in place with another stride)
        assert call(lib, s.plan, **bad) == INVALID, bad
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("inf")),
               dict(weight_fp32=2), dict(reserved=1)):
        assert call(lib, s.plan, nrm=norm(**kw), n=0) == INVALID, kw
    for kw in (dict(rotary_dim=8), dict(rotary_dim=144), dict(rotary_dim=24), dict(max_position=0), dict(interleaved=2),
               dict(reserved=1)):
        r = bsp.RopeConfig(BUF.ctypes.data, 100, 64, 0, 0)
        for k, v in kw.items():
            setattr(r, k, v)
        assert call(lib, s.plan, rope=r, n=0) == INVALID, kw


def test_append_pool_types(lib):
    assert append(lib, staged(kv_dtype=E4M3), n=0) == INVALID  # 16-bit pools
    assert append8(lib, staged(kv_dtype=E4M3), n=0) == OK
    assert append(lib, staged(), nrm=None, n=0) == INVALID and append8(lib, staged(), nrm=None, n=0) == INVALID
    assert blocks(lib, staged(), nrm=None, rope=None, n=0) == OK
    for mul in (0.0, -1.0, float("nan"), float("inf")):
        assert append8(lib, staged(), mul=mul, n=0) == INVALID


def test_block_scales_refusals(lib):
    for call, kv in ((lambda p, sc: blocks(lib, p, sc=sc, n=0), 0), (lambda p, sc: attend(lib, p, sc=sc), E4M3),
                     (lambda p, sc: rows(lib, p, sc=sc), E4M3), (lambda p, sc: copy(lib, p, sc=sc), E4M3)):
        s = Staged(kv_dtype=kv)
        p = s.plan
        for kw, want in ((dict(block=0), INVALID), (dict(block=3), INVALID), (dict(block=-4), INVALID), (dict(block=64), UNSUPPORTED),
                         (dict(reserved=1), INVALID)):
            assert call(p, scales(**kw)) == want, kw
    assert blocks(lib, staged(), sc=None) == INVALID and attend(lib, staged(kv_dtype=E4M3), sc=None) == INVALID
    for call in (rows, copy):
        assert call(lib, staged(), sc=scales()) == INVALID  # 16-bit pools have none
    assert attend(lib, staged()) == INVALID
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(flags=bsp.FLAG_ACCUMULATE)):
        assert attend(lib, staged(kv_dtype=E4M3), **bad) == INVALID
    assert attend(lib, staged(prefix=(), tail=(), kv_dtype=E4M3)) == OK


def test_page_calls_refusals(lib):
    s = Staged()
    p = s.plan  # the longest sequence: 65 positions, 3 pages
    for call in (tables, rows):
        for bad in (dict(forks=0), dict(forks=3), dict(cols=2), dict(cols=-1), dict(out_stride=3)):
            assert call(lib, p, **bad) == INVALID, bad
        assert call(lib, staged(prefill=True)) == INVALID
    for bad in (dict(bps=2), dict(max_seq=64)):
        assert rows(lib, p, **bad) == INVALID
    for call in (free, compact):
        for bad in (dict(n=-1), dict(cols=-1), dict(stride=3)):
            assert call(lib, p, **bad) == INVALID, bad
    assert copy(lib, p, n=-1) == INVALID


def test_limits_of_the_header(lib):
    text = open(os.path.join(ROOT, "include", "bsp.h")).read()
    limit = dict(re.findall(r"#define (BSP_MAX_\w+) +([^/\n]+)", text))
    size = c.c_size_t()
    n = eval(limit["BSP_MAX_FORK_ROWS"])  # noqa: S307 - a constant of this repository's header
    assert lib.bsp_fork_workspace_size(1, n, c.byref(size)) == OK and size.value == 12 * n
    assert lib.bsp_fork_workspace_size(1, n + 1, c.byref(size)) == UNSUPPORTED
    for bad in ((-1, 1), (1, 0)):
        assert lib.bsp_fork_workspace_size(*bad, c.byref(size)) == INVALID
    assert lib.bsp_fork_workspace_size(1, 1, None) == INVALID
    for call in (tables, rows):
        assert call(lib, staged(), forks=n // 2, stride=n) == INVALID  # past the limits: host memory
        assert call(lib, staged(), forks=n // 2 + 1, stride=n) == UNSUPPORTED
    most = eval(limit["BSP_MAX_PAGES"])  # noqa: S307
    for call in (tables, rows, free, compact, copy):
        s = Staged()
        s.plan.geo.num_pages = most + 1
        assert call(lib, s.plan) == UNSUPPORTED
    assert int(limit["BSP_MAX_SCALE_BLOCK"]) == 32
    assert blocks(lib, staged(), sc=scales(block=32), n=0) == OK


def scaled(lib, n=10, rot=64, base=1e4, **kw):
    s = bsp._RopeScaling(1, 0, 2.0, 0.0, 0.0, 1.0)
    for k, v in kw.items():
        setattr(s, k, v)
    return lib.bsp_rope_cos_sin_scaled(n, rot, base, c.byref(s), b, None)


def test_scaled_table_refusals(lib):
    assert scaled(lib) == INVALID  # host memory
    for bad in (dict(n=0), dict(rot=0), dict(rot=7), dict(rot=1026), dict(base=1.0), dict(base=float("inf")), dict(factor=0.0),
                dict(factor=float("inf")), dict(amplitude=0.0), dict(amplitude=float("nan")), dict(kind=2, rot=2)):
        assert scaled(lib, **bad) == INVALID, bad
    assert scaled(lib, kind=0) == UNSUPPORTED and scaled(lib, kind=5) == UNSUPPORTED
    good = dict(original_positions=100, low=1.0, high=4.0)
    for kind in (3, 4):
        for bad in (dict(original_positions=0), dict(low=0.0), dict(high=1.0), dict(high=float("inf")), dict(low=float("nan"))):
            assert scaled(lib, kind=kind, **{**good, **bad}) == INVALID, bad
    assert lib.bsp_rope_cos_sin_scaled(10, 64, 1e4, None, b, None) == INVALID
    with pytest.raises(ValueError):
        bsp.RopeScaling("other", 2.0)


def test_structs_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "bsp.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(bsp_qk_norm), '
                   "sizeof(bsp_block_scales), sizeof(bsp_rope_scaling), offsetof(bsp_qk_norm, weight_fp32), "
                   "offsetof(bsp_block_scales, block), offsetof(bsp_rope_scaling, amplitude)); return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [c.sizeof(bsp._QkNorm), c.sizeof(bsp._BlockScales), c.sizeof(bsp._RopeScaling), bsp._QkNorm.weight_fp32.offset,
                   bsp._BlockScales.block.offset, bsp._RopeScaling.amplitude.offset]


def test_binding_refusals(lib):
    s = Staged()
    p, bf = s.plan, torch.bfloat16
    pool, loc = torch.zeros((100, 4, 32, 128), dtype=bf), torch.zeros(4, dtype=torch.int32)
    k, q = torch.zeros((4, 512), dtype=bf), torch.zeros((4, 8, 128), dtype=bf)
    nrm = bsp.QkNorm(torch.ones(128, dtype=bf), None)

    class Stream:
        cuda_stream = 0

    def call(norm=nrm, q=q, k=k, v=k, loc=loc, kp=pool, vp=pool, q_out=None):
        bsp.norm_rope_append_kv(p, norm, None, None, q, k, v, loc, kp, vp, q_out=q_out, stream=Stream)

    with pytest.raises(bsp.BspError):  # all right but for the memory
        call()
    with pytest.raises(bsp.BspError):
        call(k=torch.zeros((4, 1024), dtype=bf)[:, 512:], v=torch.zeros((4, 1024), dtype=bf)[:, :512], q=torch.zeros((4, 2048), dtype=bf)[:, :1024], q_out=q)
    for bad in (dict(k=k.half()), dict(k=k[:3]), dict(k=k[:, :511]), dict(v=torch.zeros((4, 520), dtype=bf)[:, :512]),
                dict(k=torch.zeros((4, 1024), dtype=bf)[:, ::2]), dict(q=q.float()), dict(q=q[:, :7]), dict(q_out=q.half()),
                dict(q=torch.zeros((4, 128, 8), dtype=bf).transpose(1, 2)), dict(q=None, q_out=q), dict(loc=loc.long()),
                dict(kp=pool.half()), dict(vp=pool[:99]), dict(norm=bsp.QkNorm(torch.ones(64, dtype=bf))),
                dict(norm=bsp.QkNorm(torch.ones(128, dtype=torch.float16)))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in ((torch.ones(128), torch.ones(128, dtype=bf)), (torch.ones(128), torch.ones(64)), (torch.ones(128, dtype=torch.float64), None),
                (torch.ones(256)[::2], None)):
        with pytest.raises(ValueError):
            bsp.QkNorm(*bad)
    pool8 = torch.zeros((100, 4, 32, 128), dtype=torch.uint8)
    sc = bsp.BlockScales(s.geo, 16, device="cpu")
    with pytest.raises(bsp.BspError):
        bsp.append_kv_fp8_blocks(p, k, k, loc, pool8, pool8, sc, stream=Stream)
    other = bsp.BlockScales(bsp.geometry(8, 4, 128, 32, 99, "bf16"), 16, device="cpu")
    for kp, x in ((pool, sc), (pool8[:99], sc), (pool8, other)):
        with pytest.raises(ValueError):
            bsp.append_kv_fp8_blocks(p, k, k, loc, kp, pool8, x, stream=Stream)
    for bad in (dict(block=3), dict(block=64), dict(block=0), dict(block=16, k=torch.zeros((100, 4, 1), dtype=torch.uint8)),
                dict(block=16, v=torch.zeros((100, 4, 2), dtype=torch.int8))):
        with pytest.raises(ValueError):
            bsp.BlockScales(s.geo, device="cpu", **bad)
    i32 = torch.int32
    beams, refs, out = torch.zeros((2, 3), dtype=i32), torch.zeros(100, dtype=i32), torch.zeros((6, 4), dtype=i32)
    ws = torch.zeros(100, dtype=torch.uint8)
    with pytest.raises(bsp.BspError):
        bsp.fork_tables(p, beams, refs, refs, out, ws, stream=Stream)
    for bad in ((beams[:1], refs, refs, out), (beams, refs[:99], refs, out), (beams, refs, refs.long(), out), (beams, refs, refs, out[:5])):
        with pytest.raises(ValueError):
            bsp.fork_tables(p, *bad, ws, stream=Stream)
    mv = bsp.PageMoves(100, device="cpu")
    with pytest.raises(bsp.BspError):
        bsp.compact_tables(p, refs, refs, mv, out, stream=Stream)
    for bad in ((refs, refs, bsp.PageMoves(99, device="cpu"), out, None), (refs, refs, mv, out, out.T), (refs, refs, mv, out.long(), None)):
        with pytest.raises(ValueError):
            bsp.compact_tables(p, *bad, stream=Stream)
    with pytest.raises(bsp.BspError):
        bsp.copy_pages(p, mv, pool, pool, stream=Stream)
    with pytest.raises(ValueError):
        bsp.copy_pages(p, mv, pool, pool8, stream=Stream)


def test_round_e4m3_restatement():
    rs = np.random.RandomState(0)
    x = np.concatenate([cache.DECODE[:0x7f], -cache.DECODE[:0x7f], (cache.DECODE[:0x7e] + cache.DECODE[1:0x7f]) / 2,
                        rs.randn(300) * 10.0 ** rs.randint(-4, 4, 300), [449, 465, 1e9, -1e9, np.inf]])
    got = cache.round_e4m3(x)
    assert all(int(g) == oracle.round_e4m3(float(v)) for g, v in zip(got, np.clip(x, -448, 448)))
    assert np.isnan(cache.DECODE[cache.round_e4m3(np.nan)])


def test_exponents_are_the_smallest_that_fit():
    for dtype, lo, hi in (("bf16", 27, 142), ("fp16", 112, 134)):
        for e in range(lo, hi + 1):
            edge = 448.0 * 2.0 ** (e - 127)
            assert cache.exponent(edge, dtype) == e
            assert cache.exponent(np.nextafter(edge, np.inf), dtype) == min(e + 1, hi)
        assert cache.exponent(0.0, dtype) == 0 and cache.exponent(np.inf, dtype) == hi


def test_frequencies_restatement():
    """Where the stretched frequencies are the plain ones, where they are divided by the factor, and in between."""
    plain = cache.frequencies(64, 1e4)
    np.testing.assert_allclose(cache.frequencies(64, 1e4, "linear", 4.0), plain / 4)
    np.testing.assert_allclose(cache.frequencies(64, 1e4, "base", 4.0)[[0, -1]], [1.0, plain[-1] / 4])  # the slowest pair by the factor
    for kind in ("bands", "ramp"):
        f = cache.frequencies(64, 1e4, kind, 4.0, original=4096, low=1.0, high=32.0)
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 4)
        assert np.all(f <= plain * (1 + 1e-15)) and np.all(f >= plain / 4 * (1 - 1e-15)) and np.all(np.diff(f) < 0)
