"""Plans whose row blocks outnumber the SMs (very wide beams)."""
import numpy as np
import pytest

from beam_search_shared_gb300 import bsp, build


@pytest.mark.parametrize("W", [9728, 9729, 16385, 40000])
def test_plan_of_more_row_blocks_than_sms(W):
    build.build()
    geo = bsp.geometry(8, 4, 128, 32, 100, "bf16")
    plan, img = bsp.plan_build(geo, 2, W, [64, 0], [1, 0], np.zeros((2, 4), np.int32), 8, 152)
    assert plan.num_units == plan.row_blocks * 4  # each (kv head, row block) of the request with a prompt, once
    lo = plan.off_units - bsp.STATUS_BYTES
    units = img[lo:lo + plan.num_units * 32].view(np.int32).reshape(-1, 8)
    assert len({(u[1], u[2]) for u in units}) == plan.num_units and (units[:, 0] == 0).all()
