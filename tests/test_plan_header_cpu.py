"""The header of a plan image names what a captured launch depends on: rows, place of the page table, geometry."""
import numpy as np
import pytest

from beam_search_shared_gb300 import bsp, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def header(img):
    return img[:64].view(np.int32)


def test_header_of_prefill_plans():
    geo = bsp.geometry(8, 4, 128, 32, 100, "bf16")
    seen = set()
    for prompt in ([100, 100], [400, 900], [1500, 64]):
        plan, img = bsp.plan_prefill_build(geo, 2, [0, 0], prompt, np.zeros((2, 64), np.int32), True, 152)
        h = header(img)
        # one batch, width and kind throughout; the rest tells the images apart
        assert (h[2], h[4], h[6]) == (2, 1, 1)
        assert h[8] == plan.total_rows == sum(prompt) and h[9] == plan.off_pages - bsp.STATUS_BYTES
        assert list(h[10:14]) == [8, 4, 32, 128]
        seen.add((int(h[8]), int(h[9])))
    assert len(seen) == 3


def test_header_of_decode_plans():
    # one layout for all lengths of a shape; another geometry of the same batch and width is another layout
    layouts = []
    for Hq, Hkv, D, ps in ((8, 4, 128, 32), (8, 8, 128, 32), (16, 4, 64, 16)):
        geo = bsp.geometry(Hq, Hkv, D, ps, 100, "bf16")
        at = set()
        for lens in ([64, 0], [500, 900]):
            plan, img = bsp.plan_build(geo, 2, 40, lens, [1, 0], np.zeros((2, 64), np.int32), 8, 152)
            h = header(img)
            assert h[8] == plan.total_rows == 80 and h[9] == plan.off_pages - bsp.STATUS_BYTES
            assert list(h[10:14]) == [Hq, Hkv, ps, D]
            at.add(tuple(int(v) for v in h[8:14]))
        assert len(at) == 1
        layouts.append(at.pop())
    assert len(set(layouts)) == 3
