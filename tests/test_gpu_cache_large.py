"""Pools whose byte offsets pass 32 bits: rows appended into blocks of the last pages, attended, forked, moved to the front
and attended again. The keys and values that the attention sees are compared bit for bit with the same rows in a small pool
of the same contents, and the attention with itself over them."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu

Hq, Hkv, D, ps, block, W, P, T = 4, 1, 128, 128, 32, 2, 200, 3


def run(pages, at):
    """Prompt pages at[0], at[1]; the beams' second pages at[2], at[3]; the pool's other pages hold references but for
    the two before the last of those."""
    geo = bsp.geometry(Hq, Hkv, D, ps, pages, "bf16", bsp.KV_DTYPE_E4M3)
    k_pool, v_pool = (torch.empty((pages, Hkv, ps, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, ws = bsp.BlockScales(geo, block), bsp.Workspace(geo, 1, W, 2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((P + W * T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").bfloat16()
    own = [[-1, at[2]], [-1, at[3]]]
    slots = [at[i // ps] * ps + i % ps for i in range(P)] + [own[w][1] * ps + (P + t) % ps for w in range(W) for t in range(T)]
    first = bsp.geometry(Hq, Hkv, D, ps, pages, "bf16")
    pws = bsp.Workspace(first, 1, P + W * T, 3)
    plan = bsp.plan_prefill(first, 1, [0], [P + W * T], [[at[0], at[1], at[1]]], True, pws)
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
    loc = torch.tensor(slots, dtype=torch.int32, device="cuda")
    bsp.append_kv_fp8_blocks(plan, k, v, loc, k_pool, v_pool, scales, norm=bsp.QkNorm())
    assert bsp.read_device_status(plan) == (0, 0)
    rows = [(k_pool.view(-1, D)[loc.long()], v_pool.view(-1, D)[loc.long()])]
    plan = ws.plan(geo, 1, W, [P], [T], [at[:2]])
    ci = torch.arange(W, dtype=torch.int32, device="cuda")[None, :, None].expand(1, W, 2 * ps).contiguous()
    pg = torch.tensor(own, dtype=torch.int32, device="cuda")

    def attend(pl, qr, p, c):
        o, lse = torch.empty((len(qr), Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((len(qr), Hq), device="cuda")
        bsp.decode_attn_fp8_blocks(pl, qr.reshape(-1, Hq, D).contiguous(), k_pool, v_pool, scales, p, c, D ** -0.5, o, lse)
        assert bsp.read_device_status(pl) == (0, 0)
        return o, lse

    rows.append(attend(plan, q[:W], pg, ci))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[:max(at) - 2] = 1
    refs[torch.tensor(at, device="cuda")] = 1
    refs[max(at) - 1] = 0   # the fork's page: just below the last
    table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    beams = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    free = int((refs == 0).nonzero()[0])
    bsp.fork_tables(plan, beams, refs, refs, table, bsp.fork_workspace(1, 1))
    assert table.tolist() == [[at[0], free]]
    bsp.fork_rows(plan, beams, table, pg, ci, k_pool, v_pool, scales=scales)
    one = ws.plan(geo, 1, 1, [P + T], [0], table.cpu().numpy())
    rows.append(attend(one, q[1:2], None, None))
    refs.zero_()
    refs[table[0].long()] = 1
    moves = bsp.PageMoves(pages)
    bsp.compact_tables(one, refs, refs, moves, table)
    bsp.copy_pages(one, moves, k_pool, v_pool, scales=scales)
    assert sorted(table[0].tolist()) == [0, 1]
    one = ws.plan(geo, 1, 1, [P + T], [0], table.cpu().numpy())
    rows.append(attend(one, q[1:2], None, None))
    assert all(torch.equal(a, b) for a, b in zip(rows[-1], rows[-2]))
    return [t.cpu() for r in rows for t in r]


def test_offsets_past_32_bits():
    pages = 270_000
    assert pages * Hkv * ps * D > 2 ** 32
    far = run(pages, [pages - 9, pages - 4, pages - 2, pages - 6])
    near = run(40, [31, 36, 38, 34])
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    assert all(np.isfinite(t.float().numpy()).all() for t in far[2:])
