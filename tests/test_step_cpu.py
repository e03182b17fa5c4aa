"""Host-side tests of the operators around a beam step: argument checks of the C entry points and of the binding
(no CUDA device is needed: every call fails, or returns, before a launch), parameter structs against the header, and
the plain restatements against brute force."""
import ctypes as c
import itertools
import os
import subprocess

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, build
from oracle import steps

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CAPACITY, STALE = 0, 1, 2, 4, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsp.load()


class Staged:
    """A plan that the host checks take for staged: its staging header says so. Its device workspace is an address
    that no call reaches."""

    def __init__(self, W=4, prefix=(64, 0), tail=(1, 0), kv_dtype=0, prefill=False, D=128):
        B = len(prefix)
        self.geo = bsp.geometry(8, 4, D, 32, 100, "bf16", kv_dtype)
        pages = np.zeros((B, 4), np.int32)
        if prefill:
            self.plan, _ = bsp.plan_prefill_build(self.geo, B, [0] * B, prefix, pages, True, 152)
        else:
            self.plan, _ = bsp.plan_build(self.geo, B, W, prefix, tail, pages, 8, 152)
        self.host = np.zeros(256, np.uint64)
        self.host[0], self.host[1], self.host[4] = 0x3150534250534253, 7, 0x1000
        self.plan.generation, self.plan.ws_device, self.plan.ws_host = 7, 0x1000, self.host.ctypes.data


def ptr(a):
    return a.ctypes.data_as(c.c_void_p)


BUF = np.zeros(1 << 16, np.float32)  # host memory: no device pointer


def process(lib, plan, vocab=100, dtype=0, stride=100, params=None, out_stride=100):
    params = bsp._LogitsParams() if params is None else params
    return lib.bsp_process_logits(c.byref(plan), ptr(BUF), dtype, stride, vocab, c.byref(params), ptr(BUF), out_stride, None, None)


def select(lib, plan, vocab=100, dtype=0, stride=100, cum_stride=4, num=4, ws_bytes=1 << 20):
    return lib.bsp_beam_select(c.byref(plan), ptr(BUF), dtype, stride, vocab, ptr(BUF), ptr(BUF), cum_stride, None, num,
                               ptr(BUF), ptr(BUF), ptr(BUF), ptr(BUF), ws_bytes, None)


def advance(lib, plan, stride=4, ci=True, max_seq=200, tok=True, tok_stride=9, tok_cols=9):
    b = ptr(BUF)
    return lib.bsp_beam_advance(c.byref(plan), b, b, stride, b if ci else None, b, max_seq, b if tok else None, b, tok_stride,
                                tok_cols, None, None)


def weigh(lib, plan, scale=0.1, window=0, flags=0, stride=64, fp8=False, k_scale=1.0):
    b = ptr(BUF)
    if fp8:
        return lib.bsp_key_weights_fp8(c.byref(plan), b, b, b, scale, k_scale, window, flags, b, stride, None)
    return lib.bsp_key_weights(c.byref(plan), b, b, b, scale, window, flags, b, stride, None)


def evict(lib, plan, stride=64, sinks=0, recent=0, out_stride=64):
    b = ptr(BUF)
    return lib.bsp_evict_prefix(c.byref(plan), b, stride, None, b, sinks, recent, b, b, b, None, None, out_stride, None)


def test_unstaged_and_stale_plans_are_refused(lib):
    for change, want in ((lambda s: setattr(s.plan, "generation", 0), INVALID), (lambda s: s.host.__setitem__(1, 8), STALE)):
        s = Staged(tail=(0, 0))
        change(s)
        for call in (process, select, advance, weigh, evict):
            assert call(lib, s.plan) == want, call.__name__


def test_process_and_select_refusals(lib):
    s = Staged()
    # host memory reaches no launch, and what is outside the supported set is refused before it is looked at
    assert process(lib, s.plan) == INVALID and select(lib, s.plan) == INVALID
    for call in (process, select):
        assert call(lib, s.plan, dtype=3) == UNSUPPORTED
        assert call(lib, s.plan, vocab=0) == INVALID
        assert call(lib, s.plan, stride=99) == INVALID
        assert call(lib, s.plan, vocab=(1 << 21) + 1, stride=1 << 22) == UNSUPPORTED
        assert call(lib, Staged(prefill=True).plan) == INVALID
    assert process(lib, s.plan, out_stride=99) == INVALID
    assert lib.bsp_process_logits(c.byref(s.plan), ptr(BUF), 0, 100, 100, None, ptr(BUF), 100, None, None) == INVALID
    assert select(lib, s.plan, num=0) == INVALID and select(lib, s.plan, num=513) == UNSUPPORTED
    assert select(lib, s.plan, cum_stride=3) == INVALID
    assert select(lib, Staged(W=3000).plan, vocab=1 << 21, stride=1 << 21, cum_stride=3000) == UNSUPPORTED  # 32-bit places
    empty = Staged(prefix=(), tail=())
    assert process(lib, empty.plan) == OK and select(lib, empty.plan) == OK


def test_workspace_size(lib):
    n = c.c_size_t()
    size = lambda *a: (lib.bsp_beam_select_workspace_size(*a, c.byref(n)), n.value)  # noqa: E731
    for bad in ((-1, 4, 100, 4), (1, 0, 100, 4), (1, 4, 0, 4), (1, 4, 100, 0)):
        assert size(*bad)[0] == INVALID
    assert size(1, 4, (1 << 21) + 1, 4)[0] == UNSUPPORTED and size(1, 4, 100, 513)[0] == UNSUPPORTED
    assert lib.bsp_beam_select_workspace_size(1, 4, 100, 4, None) == INVALID
    for B, W, V, K in itertools.product((1, 3, 128, 2000), (1, 96), (1, 50257, 1 << 21), (1, 60, 512)):
        st, bytes_ = size(B, W, V, K)
        assert st == OK and bytes_ >= (B + 1) * (K + 2) * 8
        assert bytes_ <= (2048 + 2 * B) * (K + 2) * 8


def test_advance_weights_and_evict_refusals(lib):
    s = Staged()
    assert advance(lib, s.plan) == INVALID  # host memory
    assert advance(lib, s.plan, stride=3) == INVALID
    assert advance(lib, Staged(W=16385).plan, stride=1 << 20) == UNSUPPORTED
    assert advance(lib, Staged(prefill=True).plan) == INVALID
    assert advance(lib, s.plan, ci=False) == INVALID  # an output without its input
    assert advance(lib, s.plan, tok=False) == INVALID
    assert weigh(lib, s.plan) == INVALID
    assert weigh(lib, s.plan, flags=16) == INVALID and weigh(lib, s.plan, flags=bsp.FLAG_GRAPH) == INVALID
    assert weigh(lib, s.plan, window=1) == INVALID and weigh(lib, s.plan, stride=63) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert weigh(lib, s.plan, scale=bad) == INVALID
        assert weigh(lib, Staged(kv_dtype=1).plan, fp8=True, k_scale=bad) == INVALID
    assert weigh(lib, s.plan, fp8=True) == INVALID and weigh(lib, Staged(kv_dtype=1).plan) == INVALID
    many = Staged(prefix=(1,) * 4097, tail=(0,) * 4097)
    assert weigh(lib, many.plan) == UNSUPPORTED
    assert evict(lib, s.plan) == INVALID  # tail rows
    s = Staged(tail=(0, 0))
    assert evict(lib, s.plan) == INVALID  # host memory
    assert evict(lib, s.plan, sinks=-1) == INVALID and evict(lib, s.plan, recent=-1) == INVALID
    assert evict(lib, s.plan, stride=63) == INVALID and evict(lib, s.plan, out_stride=63) == INVALID
    empty = Staged(prefix=(), tail=())
    assert advance(lib, empty.plan) == OK and weigh(lib, empty.plan) == OK and evict(lib, empty.plan) == OK


def test_structs_match_header(tmp_path):
    fields = {"bsp_token_mask": (bsp.TokenMask, [f[0] for f in bsp.TokenMask._fields_]),
              "bsp_logits_params": (bsp._LogitsParams, [f[0] for f in bsp._LogitsParams._fields_])}
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"bsp.h\"\nint main(void){\n"
    for name, (_, names) in fields.items():
        src += f'printf("{name} %zu\\n", sizeof({name}));\n'
        for f in names:
            src += f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));\n'
    src += "return 0;}\n"
    (tmp_path / "t.c").write_text(src)
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "t.c"), "-o", exe], check=True)
    told = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, (struct, names) in fields.items():
        assert int(told[name]) == c.sizeof(struct)
        for f in names:
            assert int(told[f"{name}.{f}"]) == getattr(struct, f).offset, f


def test_binding_checks_tables():
    i32 = torch.int32
    t = torch.zeros((4, 6), dtype=i32)
    assert bsp._table("t", t, i32, (4, None)) == 6 and bsp._table("t", t, i32, (4, 6)) == 6
    assert bsp._table("t", t[:, :5], i32, (4, 5)) == 6 and bsp._table("t", t, i32, (4, 3), exact_last=False) == 6
    assert bsp._table("t", t[:1, :2], i32, (1, 2)) == 2
    w = torch.zeros((3, 1, 8), dtype=i32)
    assert bsp._table("w", w[:, :, :7], i32, (3, 1, 7)) == 8
    for bad, shape in ((t.long(), (4, 6)), (t, (5, 6)), (t, (4, 7)), (t.t(), (6, 4)), (t[None], (4, 6))):
        with pytest.raises(ValueError):
            bsp._table("t", bad, i32, shape)
    with pytest.raises(ValueError):  # rows of unequal distance
        bsp._table("w", torch.zeros((3, 4, 8), dtype=i32)[:, :3], i32, (3, 3, 8))
    with pytest.raises(ValueError):
        bsp.LogitsParams(tokens=t)
    with pytest.raises(ValueError):
        bsp.LogitsParams(bias_tokens=t, bias_values=torch.zeros((4, 5)))
    with pytest.raises(ValueError):
        bsp.LogitsParams(temperature=torch.ones(3), presence_penalty=torch.ones(2))
    with pytest.raises(ValueError):
        bsp.LogitsParams(mask=t)


def test_restatements_against_brute_force():
    rng = np.random.default_rng(0)
    # masks
    a = rng.random((3, 77)) < 0.5
    assert all(np.array_equal(steps.unpack_mask(w, 77), r) for w, r in zip(steps.pack_mask(a), a))
    # a row, token by token
    x = rng.normal(size=20)
    got = steps.process_row(x, [3, 3, 99, -1], [5, 5, 7], 2.0, 0.25, 0.5, [(7, 1.0), (7, 9.0), (3, -2.0), (50, 1.0)], 0.5, a[0][:20])
    for t in range(20):
        v = x[t]
        if t in (3, 5, 7):
            v = v / 2 if v > 0 else v * 2
        v -= {5: 0.25 * 2 + 0.5, 7: 0.25 + 0.5}.get(t, 0.0)
        v += {7: 1.0, 3: -2.0}.get(t, 0.0)
        assert got[t] == (v / 0.5 if a[0][t] else -np.inf)
    # the choice: every pair of a small problem, by hand
    for trial in range(50):
        W, V, num = rng.integers(1, 4), rng.integers(1, 6), rng.integers(1, 10)
        x = rng.integers(-2, 3, (W, V)).astype(np.float32)
        lse, cum = rng.integers(0, 2, W).astype(np.float32), rng.choice([0.0, -1.0, -np.inf], W).astype(np.float32)
        s, p, t = steps.select(x, lse, cum, num)
        every = sorted(((-(float(x[w, v]) - float(lse[w]) + float(cum[w])), w, v) for w in range(W) for v in range(V)))
        every = [e for e in every if e[0] < np.inf][:num]
        assert [(-a, b, v) for a, b, v in every] == [(float(s[i]), int(p[i]), int(t[i])) for i in range(len(every))]
        assert (p[len(every):] == -1).all() and (s[len(every):] == -np.inf).all()
    # eviction: the kept set by repeated maxima, and holes filled in order
    for trial in range(50):
        n = int(rng.integers(1, 20))
        w = rng.integers(0, 4, n).astype(float)
        keep, sinks, recent = int(rng.integers(0, n + 2)), int(rng.integers(0, 3)), int(rng.integers(0, 3))
        src = steps.evict(w, keep, sinks, recent)
        v = w.copy()
        v[:sinks] = np.inf
        if recent:
            v[max(0, n - recent):] = np.inf
        live = []
        for _ in range(min(keep, n)):
            i = int(np.argmax(np.where(np.isin(np.arange(n), live), -1.0, v)))
            live.append(i)
        assert sorted(src) == sorted(live)
        k = len(src)
        assert all(src[i] == i for i in range(k) if i in live)
        moved = [s for i, s in enumerate(src) if s != i]
        assert moved == sorted(moved) and all(m >= k for m in moved)
    # weights of all rows' softmaxes sum to the rows
    q, k = rng.normal(size=(3, 2, 8)), rng.normal(size=(11, 8))
    sc = np.einsum("igd,jd->igj", q, k)
    lse = np.log(np.exp(sc).sum(-1))
    assert np.isclose(steps.key_weights(q, k, lse, 1.0).sum(), 6.0)
    lse[1, 1] = -np.inf
    assert np.isclose(steps.key_weights(q, k, lse, 1.0).sum(), 5.0)
    assert (steps.key_weights(q, k, lse, 1.0, [4, 2, 0])[4:] == 0).all()
