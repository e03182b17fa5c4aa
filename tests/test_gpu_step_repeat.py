"""Repeated calls of the operators around a step agree bit for bit: no result depends on the order of arrival."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,W,V,dtype", [(3, 4, 50_001, torch.bfloat16), (1, 2, 8_192, torch.float32),
                                         (40, 30, 20_000, torch.float16)])
def test_processing_and_selection_repeat(B, W, V, dtype):
    gen = torch.Generator(device="cuda").manual_seed(V)
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    plan = ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))
    x = (torch.randn((B * W, V), generator=gen, device="cuda") * 3).to(dtype)
    # more marked vectors than are put aside, in runs and scattered
    prompt = torch.randint(0, V, (B, 3000), generator=gen, dtype=torch.int32, device="cuda")
    prompt[:, :1500] = torch.arange(1500, device="cuda", dtype=torch.int32) * 4 + 7
    lens = torch.full((B,), 3000, dtype=torch.int32, device="cuda")
    bias = torch.randint(0, V, (B, 200), generator=gen, dtype=torch.int32, device="cuda")
    params = bsp.LogitsParams(prompt_tokens=prompt, prompt_token_len=lens, bias_tokens=bias,
                              bias_values=torch.randn((B, 200), generator=gen, device="cuda"),
                              repetition_penalty=torch.full((B,), 1.2, device="cuda"),
                              temperature=torch.full((B,), 0.7, device="cuda"))
    K = 2 * W
    cum = torch.randn((B, W), generator=gen, device="cuda")
    sel = bsp.beam_select_workspace(B, W, V, K)
    first = None
    for _ in range(15):
        out, lse = torch.empty_like(x), torch.empty(B * W, device="cuda")
        scores, parents, tokens = (torch.empty((B, K), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
        bsp.process_logits(plan, x, params, out, lse)
        bsp.beam_select(plan, out, lse, cum, scores, parents, tokens, sel)
        got = [out.view(torch.uint8), lse.view(torch.int32), scores.view(torch.int32), parents, tokens]
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))
