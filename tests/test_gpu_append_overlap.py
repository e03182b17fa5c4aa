"""Where the query rows of an append may go (q_out): a column slice of the buffer that holds the inputs, but over none of
the call's inputs."""
import pytest
import torch

from beam_search_shared_gb300 import bsp
from test_gpu_norm_append import TDT, Tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n", [("bf16", 8), ("fp16", 1), ("bf16", 300)])
@pytest.mark.parametrize("order", ["oqkv", "qokv", "qkvo"])
def test_a_slice_of_the_inputs_buffer(dtype, n, order):
    t = Tokens(dtype, 4, 2, 64, n=n, seed=n)
    norm, rope = bsp.QkNorm(eps=1e-5), bsp.Rope(500, 64, 1e4)
    want = torch.empty((n, 256), dtype=TDT[dtype], device="cuda")
    pools = [torch.zeros((t.pages, 2, 32, 64), dtype=TDT[dtype], device="cuda") for _ in range(4)]
    bsp.norm_rope_append_kv(t.plan, norm, rope, t.pos(), t.q, t.k, t.v, t.loc(), *pools[:2], q_out=want)
    parts = dict(o=torch.zeros_like(want), q=t.q, k=t.k, v=t.v)
    wide = torch.cat([parts[x] for x in order], 1)
    got = dict(zip(order, wide.split([parts[x].shape[1] for x in order], 1)))
    bsp.norm_rope_append_kv(t.plan, norm, rope, t.pos(), got["q"], got["k"], got["v"], t.loc(), *pools[2:], q_out=got["o"])
    assert torch.equal(got["o"], want) and torch.equal(pools[2], pools[0]) and torch.equal(pools[3], pools[1])
    assert all(torch.equal(got[x], parts[x]) for x in "qkv")
    assert bsp.read_device_status(t.plan) == (0, 0)


def test_over_an_input_is_refused():
    """8 elements of a row (addresses are multiples of 16 bytes) at its end, at its beginning and of the row behind; rows
    of another stride among them; the slots, positions, table and weights."""
    bf, i32 = torch.bfloat16, torch.int32
    t = Tokens("bf16", 4, 2, 64, n=8)
    pools = [torch.zeros((t.pages, 2, 32, 64), dtype=bf, device="cuda") for _ in range(2)]
    rope = bsp.Rope(100, 64, 1e4)
    flat = torch.zeros(16 * 1024, dtype=bf, device="cuda")
    rows = lambda at, width, stride=1024: flat[at:].as_strided((8, width), (stride, 1), at)  # noqa: E731
    apart = torch.zeros((8, 1024), dtype=bf, device="cuda")[:, :128]
    out = flat[:8 * 256].view(8, 256)
    calls = dict(
        k_begins_in_it=dict(k=rows(248, 128), v=apart, q_out=rows(0, 256)),
        k_ends_in_it=dict(k=rows(0, 128), v=apart, q_out=rows(120, 256)),
        v_begins_in_it=dict(k=apart, v=rows(248, 128), q_out=rows(0, 256)),
        k_of_the_row_behind=dict(k=rows(1024 + 120, 128), v=apart, q_out=rows(896, 256)),
        q_of_the_row_behind=dict(q=rows(1024 + 120, 256), q_out=rows(896, 256)),
        last_row_alone=dict(k=rows(7 * 1024 + 248, 128), v=apart, q_out=rows(0, 256)),
        another_stride=dict(q=rows(256, 256, 512), q_out=rows(0, 256)),
        slots=dict(loc=out.view(i32).flatten()[1016:], q_out=out),
        positions=dict(positions=out.view(i32).flatten()[:8], q_out=out),
        k_weight=dict(norm=bsp.QkNorm(None, out.flatten()[64:128]), q_out=out),
        q_weight=dict(norm=bsp.QkNorm(flat[8 * 256 - 8:].view(torch.float32)[:64], None), q_out=out),
        table=dict(q_out=rope.cos_sin.view(bf).flatten()[-8 * 256:].view(8, 256)),
    )
    for name, kw in calls.items():
        a = dict(norm=bsp.QkNorm(), positions=t.pos(), q=t.q, k=t.k, v=t.v, loc=t.loc())
        a.update(kw)
        with pytest.raises(bsp.BspError, match="INVALID_ARG"):
            bsp.norm_rope_append_kv(t.plan, a["norm"], rope, a["positions"], a["q"], a["k"], a["v"], a["loc"], *pools,
                                    q_out=a["q_out"])
            pytest.fail(name)
    torch.cuda.synchronize()
    assert all((p == 0).all() for p in pools)
