"""Arguments of the cache's calls that only the binding can check: buffers' lengths, types and strides (no CUDA device
needed: a call that passes them is told of its host memory by the library)."""
import pytest
import torch

from beam_search_shared_gb300 import bsp, build
from test_step_cpu import Staged

I32, BF = torch.int32, torch.bfloat16


class Stream:
    cuda_stream = 0


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return bsp.load()


def test_counts_of_a_compaction_and_of_copies():
    """The kernel writes two counts and reads one."""
    s = Staged()
    refs, table = torch.zeros(100, dtype=I32), torch.zeros((6, 4), dtype=I32)
    pool = torch.zeros((100, 4, 32, 128), dtype=BF)
    compact = lambda mv: bsp.compact_tables(s.plan, refs, refs, mv, table, stream=Stream)  # noqa: E731
    for n in (2, 5):
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):
            compact(bsp.PageMoves(100, device="cpu", count=torch.zeros(n, dtype=I32)))
    for n in (0, 1):
        with pytest.raises(ValueError, match="count"):
            compact(bsp.PageMoves(100, device="cpu", count=torch.zeros(n, dtype=I32)))
    short = bsp.PageMoves(100, device="cpu")
    short.pairs = short.pairs[:49]
    with pytest.raises(ValueError, match="pairs"):
        compact(short)
    pairs = torch.zeros((3, 2), dtype=I32)
    with pytest.raises(bsp.BspError, match="INVALID_ARG"):
        bsp.copy_pages(s.plan, bsp.PageMoves(100, pairs=pairs, count=torch.zeros(1, dtype=I32)), pool, pool, stream=Stream)
    with pytest.raises(ValueError, match="count"):
        bsp.copy_pages(s.plan, bsp.PageMoves(100, pairs=pairs, count=torch.zeros(0, dtype=I32)), pool, pool, stream=Stream)


def test_buffers_of_the_attention_over_blocks():
    """Types, contiguity and lengths of what the call goes by the address of; rows may be counted by any dimensions."""
    s = Staged(prefix=(64, 32), tail=(1, 0), kv_dtype=bsp.KV_DTYPE_E4M3)   # 8 rows, 8 heads of 128, 65 positions
    pool = torch.zeros((100, 4, 32, 128), dtype=torch.uint8)
    scales = bsp.BlockScales(s.geo, 16, device="cpu")
    good = dict(q=torch.zeros((8, 8, 128), dtype=BF), o=torch.zeros((8, 8, 128), dtype=BF), lse=torch.zeros((8, 8)),
                pages=torch.zeros((8, 3), dtype=I32), ci=torch.zeros((2, 4, 65), dtype=I32))

    def call(plan=s.plan, flags=0, **kw):
        a = {**good, **kw}
        bsp.decode_attn_fp8_blocks(plan, a["q"], pool, pool, scales, a["pages"], a["ci"], 0.1, a["o"], a["lse"], flags=flags, stream=Stream)

    for kw in ({}, dict(q=good["q"].view(8, 1024)), dict(q=good["q"].view(2, 4, 8, 128)), dict(q=torch.zeros((9, 8, 128), dtype=BF)),
               dict(lse=torch.zeros(64)), dict(lse=torch.zeros((2, 4, 8))), dict(pages=torch.zeros((2, 4, 3), dtype=I32)),
               dict(ci=torch.zeros((8, 65), dtype=I32))):
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):   # all right but for the memory
            call(**kw)
    wide = torch.zeros((8, 2048), dtype=BF)
    for kw in (dict(q=good["q"].half()), dict(q=good["q"].float()), dict(q=wide[:, :1024]), dict(q=good["q"][:7]),
               dict(q=torch.zeros((8, 128, 8), dtype=BF)), dict(q=good["q"].transpose(0, 1)), dict(o=good["o"].float()),
               dict(o=good["o"][:, :7]), dict(o=wide[:, 1024:]), dict(lse=good["lse"].bfloat16()), dict(lse=torch.zeros((8, 7))),
               dict(lse=torch.zeros((8, 16))[:, ::2]), dict(pages=good["pages"].long()), dict(pages=torch.zeros((7, 3), dtype=I32)),
               dict(pages=torch.zeros((8, 6), dtype=I32)[:, :3]), dict(ci=good["ci"].long()), dict(ci=torch.zeros((2, 3, 65), dtype=I32)),
               dict(ci=torch.zeros((2, 4, 130), dtype=I32)[..., :65])):
        with pytest.raises(ValueError):
            call(**kw)
    none = Staged(prefix=(64, 32), tail=(0, 0), kv_dtype=bsp.KV_DTYPE_E4M3)
    with pytest.raises(bsp.BspError, match="INVALID_ARG"):       # without tails these are not read
        call(plan=none.plan, pages=torch.zeros((1, 3), dtype=I32))
    with pytest.raises(ValueError):                              # a replay may have some
        call(plan=none.plan, pages=torch.zeros((1, 3), dtype=I32), flags=bsp.FLAG_GRAPH)


def test_columns_of_the_forked_beams_pages(monkeypatch):
    """A column slice of a wider table has its own columns only, though the library goes by the rows' stride."""
    s = Staged(prefix=(64, 32), tail=(1, 0))   # 65 positions: 3 pages
    beams, out = torch.zeros((2, 3), dtype=I32), torch.zeros((6, 4), dtype=I32)
    ci = torch.zeros((2, 4, 65), dtype=I32)
    pool = torch.zeros((100, 4, 32, 128), dtype=BF)
    wide = torch.zeros((8, 10), dtype=I32)
    call = lambda pages: bsp.fork_rows(s.plan, beams, out, pages, ci, pool, pool, stream=Stream)  # noqa: E731
    for pages in (wide, wide[:, :3], wide[:, 2:5], wide[:, :3].contiguous()):
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):   # all right but for the memory
            call(pages)
    for pages in (wide[:, :2], wide[:, :2].contiguous()):
        with pytest.raises(ValueError, match="columns"):
            call(pages)
    monkeypatch.setattr(bsp, "_captured", lambda t: True)
    for pages in (wide, wide[:, :3], wide[:, :3].contiguous()):
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):
            call(pages)
    with pytest.raises(ValueError, match="stride"):              # (a replay may read ten columns of the last row)
        call(wide[:, 2:5])
