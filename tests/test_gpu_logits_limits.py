"""Logits processing at the limits of its lists and vocabularies together, against the plain restatement."""
import numpy as np
import pytest
import torch

from beam_search_shared_gb300 import bsp
from oracle import steps

pytestmark = pytest.mark.gpu


# bias entries and generated tokens (under a frequency penalty) share BSP_MAX_LISTED = 8192; in one run of ids, which one
# slice of the vocabulary holds, or scattered
@pytest.mark.parametrize("V,bias,made,scattered,masked", [
    (1 << 21, 8192, 0, False, True), (1 << 21, 4096, 4096, False, True), (1 << 21, 8192, 0, True, False),
    (1 << 21, 4000, 0, False, True), (410_000, 8192, 0, False, True), (420_000, 8192, 0, True, True),
    (1_250_001, 5000, 3000, False, False), (151_936, 8192, 0, False, True), (8192, 8192, 0, False, True)])
def test_long_lists_over_large_vocabularies(V, bias, made, scattered, masked):
    B, W = 1, 2
    rng = np.random.default_rng(V + bias)
    gen = torch.Generator(device="cuda").manual_seed(V)
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    plan = ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))
    x = torch.randn((B * W, V), generator=gen, device="cuda")
    at = 0 if V < 20000 else V // 3
    ids = (rng.permutation(V)[:bias] if scattered else at + rng.permutation(bias)).astype(np.int32)
    kw = dict(bias_tokens=ids[None], bias_values=rng.normal(0, 2, (1, bias)).astype(np.float32),
              repetition_penalty=np.array([1.25], np.float32))
    prompt = rng.integers(0, V, (1, 500)).astype(np.int32)
    kw.update(prompt_tokens=prompt, prompt_token_len=np.array([500], np.int32))
    tokens = None
    if made:
        tokens = (at + bias + rng.integers(0, made, (B * W, made))).astype(np.int32)
        kw.update(tokens=tokens, token_len=np.array([made, made // 2], np.int32), frequency_penalty=np.array([0.125], np.float32))
    allowed = None
    if masked:
        allowed = rng.random((1, V)) < 0.7
        kw.update(mask=steps.pack_mask(allowed), mask_index=np.array([0, -1], np.int32))
    params = bsp.LogitsParams(**{k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in kw.items()})
    out, lse = torch.empty_like(x), torch.empty(B * W, device="cuda")
    bsp.process_logits(plan, x, params, out, lse)
    assert bsp.read_device_status(plan) == (0, 0)
    src, got = x.double().cpu().numpy(), out.double().cpu().numpy()
    pairs = list(zip(ids, kw["bias_values"][0].astype(float)))
    for r in range(B * W):
        n = 0 if tokens is None else int(kw["token_len"][r])
        count = 0 if tokens is None or not n else np.bincount(tokens[r, :n]).max()
        want = steps.process_row(src[r], prompt[0], () if tokens is None else tokens[r, :n], 1.25,
                                 0.125 if made else None, None, pairs, None, allowed[0] if masked and r == 0 else None)
        fin = np.isfinite(want)
        assert np.array_equal(fin, np.isfinite(got[r]))
        # four fp32 roundings (penalty, product, difference, bias) of values below |x| 1.25 + 0.125 count + |bias|
        size = np.abs(src[r]).max() * 1.25 + 0.125 * count + np.abs(kw["bias_values"]).max()
        assert np.abs(got[r][fin] - want[fin]).max() <= 4 * 2.0 ** -24 * size
        # the sum of V positive terms in some V / 512 additions a thread and a slice's eighth, as in the other tests
        ref = steps.log_sum_exp(got[r])
        assert abs(float(lse[r]) - ref) <= 2.0 ** -22 + 64 * 2.0 ** -22 + (V / 512 + 40) * 2.0 ** -24 + 3 * 2.0 ** -24 * (abs(ref) + 20)


def small_step(B, W):
    geo = bsp.geometry(2, 1, 64, 32, 1, "bf16")
    ws = bsp.Workspace(geo, B, W, 1)
    return ws, ws.plan(geo, B, W, np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros((B, 1), np.int32))


def test_one_listed_token_too_many():
    ws, plan = small_step(1, 1)
    x = torch.zeros((1, 100), device="cuda")
    i32 = torch.int32
    bias = dict(bias_tokens=torch.zeros((1, 8000), dtype=i32, device="cuda"), bias_values=torch.ones((1, 8000), device="cuda"))
    made = lambda n: dict(tokens=torch.ones((1, n), dtype=i32, device="cuda"), token_len=torch.full((1,), n, dtype=i32, device="cuda"))  # noqa: E731
    rep, pen = dict(repetition_penalty=torch.ones(1, device="cuda")), dict(presence_penalty=torch.full((1,), 0.5, device="cuda"))
    out = torch.empty_like(x)
    bsp.process_logits(plan, x, bsp.LogitsParams(**bias, **made(192), **pen), out)
    assert out[0, 0] == 1.0 and out[0, 1] == -0.5 and (out[0, 2:] == 0).all()
    with pytest.raises(bsp.BspError) as e:
        bsp.process_logits(plan, x, bsp.LogitsParams(**bias, **made(193), **pen), out)
    assert e.value.status == 2
    # histories that only the repetition penalty reads are no part of the limit
    bsp.process_logits(plan, x, bsp.LogitsParams(**bias, **made(5000), **rep), out)
    assert out[0, 0] == 1.0 and (out[0, 1:] == 0).all()


def test_extreme_temperatures():
    """From 2^-127, whose reciprocal is finite (a denormal), to 2^126: powers of two scale exactly."""
    ws, plan = small_step(3, 1)
    k = torch.arange(-50, 50, device="cuda").float()
    x = torch.stack([k * 2.0 ** -130, k, k * 2.0 ** 100])
    temperature = torch.tensor([2.0 ** -127, 0.25, 2.0 ** 126], device="cuda")
    out, lse = torch.empty_like(x), torch.empty(3, device="cuda")
    bsp.process_logits(plan, x, bsp.LogitsParams(temperature=temperature), out, lse)
    want = torch.stack([k / 8, k * 4, k * 2.0 ** -26])
    assert torch.equal(out, want)
    # the other tests' bound: exponentials and their arguments, a few additions, and three roundings of the size of the
    # result (-m log2(e) as one fp32 number: 2^-24 |m|; the last sum: half a step of the result, 2^-17 alone where the
    # result is 196; the logarithm): 3 x 2^-24 (|result| + 20)
    ref = torch.logsumexp(want.double(), -1)
    assert ((lse - ref).abs() <= 2.0 ** -22 + 64 * 2.0 ** -22 + 41 * 2.0 ** -24 + 3 * 2.0 ** -24 * (ref.abs() + 20)).all()
