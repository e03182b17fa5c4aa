"""The binding refuses pools that are not of the plan's geometry before it takes their address (no CUDA device needed)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


STREAM = SimpleNamespace(cuda_stream=0)


def state(kv_dtype=0, dtype="bf16", pages=6):
    geo = bsp.geometry(4, 2, 64, 16, pages, dtype, kv_dtype)
    plan, _ = bsp.plan_build(geo, 1, 3, [20], [0], np.zeros((1, 2), np.int32), 8, 152)
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    return plan, dict(q=torch.zeros((3, 4, 64), dtype=t), lse=torch.zeros((3, 4)), w=torch.zeros((1, 2, 20)),
                      keep=torch.zeros(1, dtype=torch.int32), kept=torch.zeros((1, 2, 20), dtype=torch.int32))


def calls(plan, s, k, v):
    """Each call's refusal: a ValueError of the binding, or a BspError of the library behind it."""
    weigh = (lambda: bsp.key_weights_fp8(plan, s["q"], k, s["lse"], 0.1, 1.0, s["w"], stream=STREAM)) if plan.geo.kv_dtype else (
        lambda: bsp.key_weights(plan, s["q"], k, s["lse"], 0.1, s["w"], stream=STREAM))
    out = []
    for call in (weigh, lambda: bsp.evict_prefix(plan, s["w"], s["keep"], 0, 0, k, v, s["kept"], stream=STREAM)):
        with pytest.raises((ValueError, bsp.BspError)) as e:
            call()
        out.append(e.type)
    return out


GOOD = [bsp.BspError, bsp.BspError]  # past the binding: the plan is not staged


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_16_bit_pools(dtype):
    plan, s = state(dtype=dtype)
    t, other = (torch.bfloat16, torch.float16) if dtype == "bf16" else (torch.float16, torch.bfloat16)
    pool = torch.zeros((6, 2, 16, 64), dtype=t)
    assert calls(plan, s, pool, pool) == GOOD
    assert calls(plan, s, torch.zeros((9, 2, 16, 64), dtype=t), pool.view(-1)) == GOOD  # more pages; another view
    for bad in (pool.to(other), pool.float(), pool.to(torch.uint8), pool[:5], torch.zeros((6, 2, 16, 128), dtype=t)[..., :64],
                torch.zeros((6, 16, 2, 64), dtype=t), torch.zeros((6, 16, 2, 64), dtype=t).transpose(1, 2), pool.view(-1)[1:]):
        assert calls(plan, s, bad, pool) == [ValueError, ValueError], (bad.dtype, bad.shape)
        assert calls(plan, s, pool, bad) == [bsp.BspError, ValueError]


def test_e4m3_pools():
    plan, s = state(kv_dtype=bsp.KV_DTYPE_E4M3)
    pool = torch.zeros((6, 2, 16, 64), dtype=torch.uint8)
    assert calls(plan, s, pool, pool) == GOOD
    assert calls(plan, s, pool.view(torch.float8_e4m3fn), pool) == GOOD
    for bad in (pool.to(torch.bfloat16), pool[:5], pool.view(torch.int8)):
        assert calls(plan, s, bad, pool) == [ValueError, ValueError]
