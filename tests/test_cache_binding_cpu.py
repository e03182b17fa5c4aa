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
