"""The bits that the weights keep in the attention of chunks, which a bound that sums worst
cases cannot see.

Scores are exact (two dimensions of the queries and keys are not zero) and positions come in
pairs of nearly the same weight and opposite values, so the sums of products nearly cancel
and an output's own rounding is a hundredth of what rounding the weights to 16 bits leaves.
The last dimension of the values is 1 throughout: its output is 1, whatever the weights.

Tolerance for the root mean square over all outputs but those ones, before any run.  A weight
of mantissa m in [1, 2) that is rounded to nearest is off by up to u / m of itself (u = 2^-11
for fp16, 2^-8 for bf16), evenly spread: u / m / sqrt 3 in the root mean square, and as
mantissas are spread over their logarithm, E[1 / m^2] = 3 / (8 ln 2): R = 0.4248 u.  Errors of
different positions are independent: an output is off by R sqrt(sum w^2 v^2).  A lost bit makes
it twice that; allowed is sqrt 2 of it, half way.  To that come twice what rounding the exact
outputs to the type gives, and for the sums in FP32 2^-22 of the largest product in each of
n / 16 matrix products.  The output that is 1 has the mean of the weights' errors, R sqrt(sum w^2)
with a sum w^2 of 2^-7 at most: under u / 6 at four times its spread, and what is within u / 2 of 1
is rounded to 1."""
from __future__ import annotations

import math
import random

import pytest
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float16, torch.bfloat16]
HEADS = 2


def make(n, new, dim, dtype, seed):
    """(q [new, 2, dim], keys [n, dim], values [n, dim]) on the CPU; n is even."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(new, HEADS, dim)
    q[..., 0] = torch.randint(2, 5, (new, HEADS), generator=g) / 4.0
    q[..., 1] = 2.0 ** -7
    k = torch.zeros(n, dim)
    k[:, 0] = (torch.randint(-64, 64, (n // 2,), generator=g) / 32.0).repeat_interleave(2)
    k[:, 1] = (torch.randint(64, 128, (n // 2,), generator=g) / 64.0).repeat_interleave(2)
    k[1::2, 1] += 1.0
    half = torch.randn(n // 2, dim, generator=g).to(dtype)
    values = torch.stack([half, -half], 1).flatten(0, 1)
    values[:, -1] = 1.0
    assert torch.equal(k.to(dtype).float(), k)
    return q.to(dtype), k.to(dtype), values


def scores(q, keys):
    """[new, 2, n], -infinity where a token does not see."""
    new, n = q.shape[0], keys.shape[0]
    x = torch.einsum("thd,pd->thp", q.double(), keys.double())
    seen = torch.arange(n) <= torch.arange(n - new, n)[:, None]
    return x.masked_fill(~seen[:, None], -math.inf)


def close(out, q, keys, values) -> bool:
    w, v, u = torch.softmax(scores(q, keys), -1), values.double(), UNIT[out.dtype]
    assert w.square().sum(-1).max() <= 2.0 ** -7
    if not (out[..., -1] == 1).all():
        return False
    out, v = out[..., :-1], v[:, :-1]
    want = w @ v
    rms = lambda x: x.square().mean().sqrt().item()  # noqa: E731
    tol = (math.sqrt(2) * math.sqrt(1 / (8 * math.log(2))) * u * rms((w.square() @ v.square()).sqrt())
           + 2 * rms(want.to(out.dtype).double() - want)
           + keys.shape[0] / 16 * 2.0 ** -22 * (w.max() * v.abs().max()).item())
    return rms(out.double() - want) <= tol


def kept(p, dtype, lost):
    """Positive p rounded to nearest in the type, `lost` bits short of it."""
    mantissa, exponent = torch.frexp(p)
    one = 2.0 ** ({torch.float16: 11, torch.bfloat16: 8}[dtype] - lost)
    return torch.ldexp((mantissa * one).round() / one, exponent)


def down(p, dtype):
    """Positive p rounded towards zero."""
    r = p.to(dtype)
    return torch.where(r.double() > p, (r.view(torch.int16) - 1).view(dtype), r).double()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, new", [(1030, 100), (6000, 5), (6000, 1)])
@pytest.mark.parametrize("stale", [0.0, 1.3], ids=["maximum", "old maximum"])
def test_the_criterion_sees_a_lost_bit(dtype, n, new, stale):
    """Weights rounded once pass, whichever of their sums divides; with a bit less, in the other
    type, rounded towards zero or a position short they do not."""
    q, keys, values = make(n, new, 64, dtype, seed=n + new)
    x, v = scores(q, keys), values.double()
    p = torch.exp(x - x.amax(-1, keepdim=True) + stale) * (2.0 ** 12 if dtype == torch.float16 else 1)
    p = p.float().double()
    sums = p.sum(-1, keepdim=True)

    def passes(weights, divisor=sums, v=v):
        return close((weights @ v / divisor).to(dtype), q, keys, values)

    once = p.to(dtype).double()
    assert torch.equal(once, kept(p, dtype, 0))
    assert passes(p) and passes(once) and passes(once, once.sum(-1, keepdim=True))
    for lost in (1, 2, 3):
        assert not passes(kept(p, dtype, lost))
        assert not passes(kept(p, dtype, lost), kept(p, dtype, lost).sum(-1, keepdim=True))
    assert not passes(down(p, dtype))
    assert not passes(once[..., 1:], v=v[1:])
    if dtype == torch.float16:
        assert not passes(p.bfloat16().double())


ITEMS = {"one tile, cut": (1, 6000, 5), "one token, cut": (1, 6000, 1), "one tile, whole": (1000, 1030, 5),
         "two tiles, cut": (1, 6000, 100), "two tiles, whole": (1000, 1030, 100)}


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 13])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("items", ITEMS)
def test_weights_keep_their_bits(w4lib, items, dtype, page, dim):
    """Rows that are alike share their pages: many of them are not cut, a single one is."""
    import w4a16_weight_only_gemm_gb300 as w4
    rows, n, new = ITEMS[items]
    q, keys, values = make(n, new, dim, dtype, seed=n + new)
    used = -(-n // page)
    order = random.Random(n).sample(range(used), used)
    k, v = (torch.zeros(used, page, 1, dim, dtype=dtype) for _ in range(2))
    at = torch.tensor(order).repeat_interleave(page)[:n], torch.arange(n) % page
    k[at[0], at[1], 0], v[at[0], at[1], 0] = keys, values
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.paged_chunk_attention(q.cuda().repeat(rows, 1, 1), k.cuda(), v.cuda(),
                                   ints([order] * rows), ints([n] * rows),
                                   ints([b * new for b in range(rows + 1)]), scale=1.0)
    out = out.view(rows, new, HEADS, dim)
    assert close(out[0].cpu(), q, keys, values)
    assert (out == out[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 1000], ids=["cut", "whole"])
@pytest.mark.parametrize("later", [0.6875, 1.5625, -1.5625, 4.9375])
def test_an_average_of_equal_values(w4lib, later, rows, dtype):
    """Weights that are alike are all rounded alike: behind 256 scores of 0, 1244 of another.
    Each is off by u of itself at most, and so is their average over one value; the output
    is rounded once more."""
    import w4a16_weight_only_gemm_gb300 as w4
    n, new, page, u = 1500, 3, 16, UNIT[dtype]
    value = torch.randn(64, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    q, k = (torch.zeros(*shape, 64, dtype=dtype, device="cuda")
            for shape in ((rows * new, HEADS), (94, page, 1)))
    q[..., 0], k[16:, ..., 0] = 1.0, later
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.paged_chunk_attention(q, k, value.expand_as(k).contiguous(), ints([list(range(94))] * rows),
                                   ints([n] * rows), ints([b * new for b in range(rows + 1)]), scale=1.0)
    value = value.double()
    assert ((out.double() - value).abs() <= ((1 + u) ** 2 - 1 + 2.0 ** -16) * value.abs() + 2.0 ** -25).all()
