"""What the merge of partial states chooses its kernel by: the most splits of a request, as the plan image has them."""
import numpy as np
import pytest

from beam_search_shared_gb300 import bsp, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("prefix", [(10000,), (10000, 40, 0), (300,) * 10, (500,) * 64, (0, 0), ()])
@pytest.mark.parametrize("W,Hq,Hkv,D", [(4, 32, 8, 128), (30, 8, 2, 64), (96, 16, 8, 128), (60, 4, 1, 256)])
def test_most_splits_of_a_request(prefix, W, Hq, Hkv, D):
    B = len(prefix)
    geo = bsp.geometry(Hq, Hkv, D, 32, 20000, "bf16")
    pages = np.zeros((B, max(1, -(-max(prefix, default=0) // 32))), np.int32)
    plan, img = bsp.plan_build(geo, B, W, prefix, [2] * B, pages, 8, 152)
    assert plan.max_splits == (bsp.plan_requests(plan, img)[:, 2].max() if B else 0)
    if prefix == (10000,):
        assert plan.max_splits > 5
