"""The bits of the attention's weights, which a bound that sums worst cases cannot see.

Scores are exact (one dimension of the queries and keys is not zero) and positions come in
pairs of nearly the same weight and opposite values, so the sums of products nearly cancel
and an output's own rounding is a hundredth of what rounding the weights to 16 bits leaves.

Tolerance for the root mean square over all outputs, before any run: twice what rounding
the exact outputs to the type gives; a relative error of each weight of 2^-20 in fp16 and
2^-15 in bf16 (two 16-bit parts keep 2^-22 and 2^-16, the exponent's rounding at 2^4 is
2^-21, the exponential's 2^-22), which adds up to twice that times the root of
sum w^2 v^2; and for the sums in FP32 2^-22 of the largest product in each of n / 16
matrix products."""
from __future__ import annotations

import random

import pytest
import torch

WEIGHTS = {torch.float16: 2.0 ** -20, torch.bfloat16: 2.0 ** -15}
TYPES = [torch.float16, torch.bfloat16]
HEADS, DIM = 2, 64


def make(n, dtype, seed):
    """(q [1, 2, DIM], scores' keys [n], values [n, DIM]) on the CPU; n is even."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(1, HEADS, DIM)
    q[0, :, 0] = torch.tensor([1.0, 0.5])
    first = torch.randint(-64, 64, (n // 2,), generator=g) / 32.0
    keys = torch.stack([first, first + 2.0 ** -7], 1).flatten()
    half = torch.randn(n // 2, DIM, generator=g).to(dtype).double()
    values = torch.stack([half, -half], 1).flatten(0, 1)
    assert torch.equal(keys.to(dtype).float(), keys)
    return q.to(dtype), keys.to(dtype), values.to(dtype)


def exact(q, keys, values):
    w = torch.softmax(q[0, :, :1].double() * keys.double(), 1)
    return w, w @ values.double()


def close(out, q, keys, values) -> bool:
    w, want = exact(q, keys, values)
    v, n = values.double(), keys.numel()
    rms = lambda x: x.square().mean().sqrt().item()  # noqa: E731
    tol = (2 * rms(want.to(out.dtype).double() - want)
           + 2 * WEIGHTS[out.dtype] * rms((w.square() @ v.square()).sqrt())
           + n / 16 * 2.0 ** -22 * (w.max() * v.abs().max()).item())
    return rms(out.double() - want) <= tol


def down(x, dtype):
    """Positive x rounded towards zero."""
    r = x.to(dtype)
    return torch.where(r.double() > x, (r.view(torch.int16) - 1).view(dtype), r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [2048, 6000])
def test_the_criterion_sees_a_lost_part(dtype, n):
    """Weights in two 16-bit parts pass, in one they do not; nor do outputs one position short."""
    q, keys, values = make(n, dtype, seed=n)
    x = q[0, :, :1].double() * keys.double()
    p = torch.exp(x - x.amax(1, keepdim=True)) * 2.0 ** 12
    first = down(p, dtype)
    second = (p - first.double()).to(dtype)
    sums, v = p.sum(1, keepdim=True), values.double()
    both = ((first.double() + second.double()) @ v / sums).to(dtype)
    assert close(both, q, keys, values)
    assert not close((first.double() @ v / sums).to(dtype), q, keys, values)
    assert not close((p.to(dtype).double() @ v / sums).to(dtype), q, keys, values)
    assert not close((p[:, 1:] @ v[1:] / sums).to(dtype), q, keys, values)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [None, 4000], ids=["clusters", "line"])
@pytest.mark.parametrize("page", [16, 13])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [2048, 6000])
def test_weights_keep_their_bits(w4lib, n, dtype, page, width):
    import w4a16_weight_only_gemm_gb300 as w4
    q, keys, values = make(n, dtype, seed=n)
    used = -(-n // page)
    order = random.Random(n).sample(range(used), used)
    k = torch.zeros(used, page, 1, DIM, dtype=dtype)
    v = torch.zeros_like(k)
    at = torch.tensor(order).repeat_interleave(page)[:n], torch.arange(n) % page
    k[at[0], at[1], 0, 0] = keys
    v[at[0], at[1], 0] = values
    tables = torch.full((1, width or used), -1, dtype=torch.int32)
    tables[0, :used] = torch.tensor(order, dtype=torch.int32)
    out = w4.paged_attention(q.cuda(), k.cuda(), v.cuda(), tables.cuda(),
                             torch.tensor([n], dtype=torch.int32).cuda(), scale=1.0)
    assert close(out[0].cpu(), q, keys, values)
