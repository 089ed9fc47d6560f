"""Token scores against the 64-bit definition: types, vocabulary sizes,
alignments, masks, ties, rows without a number.

Tolerance, from the arithmetic: x - m and its exponential are off by a few units
of 2^-24 each, a sum of n terms in at least 256 partial sums by at most n / 256
more; so a logarithm of the sum is off by at most 2^-24 (n / 256 + 64), a log
probability by 2^-22 of itself besides, and the entropy, an average of such
terms, by (1 + H + ln n) times as much."""
from __future__ import annotations

import math
import random

import pytest
import torch

import paged_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]


def check(logits, tokens, top):
    got = w4.token_logprobs(logits, tokens, top=top)
    torch.cuda.synchronize()
    want = ref.scores(logits, tokens, top)
    n = logits.shape[1]
    tol = 2.0 ** -24 * (n / 256 + 64)
    assert [g.dtype for g in got] == [torch.float32, torch.float32, torch.int32, torch.float32]
    assert torch.equal(got[2].cpu().long(), want[2])
    for g, w, t in ((got[0], want[0], tol + 2.0 ** -22 * want[0].abs()),
                    (got[1], want[1], tol * (1 + want[1].abs() + math.log(n))),
                    (got[3], want[3], tol + 2.0 ** -22 * want[3].abs())):
        g = g.cpu().double()
        assert torch.equal(torch.isnan(g), torch.isnan(w))
        whole = torch.isfinite(w)
        assert torch.equal(g[~whole].nan_to_num(), w[~whole].nan_to_num())
        assert ((g - w).abs() <= t)[whole].all(), (g - w).abs()[whole].max()
    return got


def random_logits(rows, n, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * 3
    return x.to(dtype).cuda(), torch.randint(0, n, (rows,), generator=g).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 31, 32, 33, 255, 1000, 4099, 8192, 50257, 128256])
@pytest.mark.parametrize("rows", [1, 5])
def test_sizes(w4lib, rows, n, dtype):
    for top in {0, 1, min(n, 5), min(n, 32)}:
        check(*random_logits(rows, n, dtype, seed=n + rows), top)


@pytest.mark.parametrize("rows", [2, 16, 17, 151, 400])
@pytest.mark.parametrize("n", [3001, 32003])
def test_many_rows(w4lib, rows, n):
    check(*random_logits(rows, n, torch.float16, seed=rows), 10)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
def test_alignment_and_strides(w4lib, dtype, shift):
    """Rows that start anywhere, with foreign values between them."""
    x, tokens = random_logits(6, 5003, dtype, seed=shift)
    wide = torch.full((6, 5003 + 11), 99.0, device="cuda").to(dtype)
    wide[:, shift:shift + 5003] = x
    a = check(wide[:, shift:shift + 5003], tokens, 20)
    b = w4.token_logprobs(x, tokens.int(), top=20)
    for s, t in zip(a, b):
        assert torch.allclose(s, t, rtol=0, atol=2.0 ** -18) and (s.dtype != torch.int32 or torch.equal(s, t))
    one = x[:1].expand(6, -1)                   # one row read by all
    check(one, tokens, 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lowest_index(w4lib, dtype):
    x = torch.zeros(4, 9001, device="cuda").to(dtype)
    x[1, 4000:] = 1.0
    x[2, ::97] = 2.0
    x[2, 1::2] = -0.0
    x[3, 8990:] = 5.0
    check(x, torch.tensor([0, 1, 2, 9000], device="cuda"), 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["up", "down"])
def test_sorted_logits(w4lib, dtype, order):
    """Every logit a new maximum, or none after the first."""
    x = torch.linspace(-8, 8, 30011, device="cuda")
    x = (x if order == "up" else x.flip(0)).to(dtype).repeat(3, 1)
    check(x, torch.tensor([0, 17, 30010], device="cuda"), 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_masks(w4lib, dtype):
    x, tokens = random_logits(8, 6007, dtype, seed=4)
    low = torch.finfo(dtype).min
    x[0, 100:] = -math.inf                      # a few left
    x[1, :] = -math.inf                         # nothing left
    x[2, 1:] = -math.inf                        # one left
    x[3, 5:] = low                              # masked by the type's lowest value
    x[4, :] = low
    x[5, :3000] = -math.inf                     # whole parts of the row masked
    x[6, 1000:] = -math.inf
    x[6, 6006] = 4.0
    x[7, :3] = low                              # both kinds together
    x[7, 3:] = -math.inf
    tokens[1] = 3
    tokens[2] = 0
    check(x, tokens, 10)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_a_number(w4lib, dtype):
    x, tokens = random_logits(6, 3003, dtype, seed=5)
    x[0, 17] = math.nan
    x[1, 2000] = math.inf
    x[2, 5] = math.inf
    x[2, 9] = math.nan
    x[3, :] = math.nan
    x[4, :] = -math.inf
    x[4, 8] = math.nan
    check(x, tokens, 5)


def test_large_and_small_logits(w4lib):
    x, tokens = random_logits(4, 4001, torch.float32, seed=6)
    x[0] *= 1e4
    x[1] *= 1e-6
    x[2] += 1e6
    x[3, 7] = 3e38
    x[3, 8] = -3e38
    check(x, tokens, 5)


def test_tokens_outside(w4lib):
    x, _ = random_logits(4, 100, torch.float16, seed=7)
    check(x, torch.tensor([-1, 100, 2 ** 40, 99], device="cuda"), 2)
    check(x, torch.tensor([-1, 100, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda"), 2)


def test_repeat_streams_and_graph(w4lib):
    x, tokens = random_logits(3, 128256, torch.float16, seed=8)
    first = w4.token_logprobs(x, tokens, top=20)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        again = w4.token_logprobs(x, tokens, top=20, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.token_logprobs(x, tokens, top=20)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_past_32_bit_offsets(w4lib):
    x = torch.zeros(17000, 128256, dtype=torch.float16, device="cuda")   # 2.2 G logits
    x[-1, 128255] = 9.0
    x[-1, 5] = 8.0
    tokens = torch.full((17000,), 128255, device="cuda")
    got = w4.token_logprobs(x, tokens, top=2)
    want = ref.scores(x[-1:], tokens[-1:], 2)
    assert got[2][-1].tolist() == [128255, 5] and got[2][0].tolist() == [0, 1]
    assert abs(got[0][-1].item() - want[0].item()) < 1e-4


@pytest.mark.parametrize("seed", range(40))
def test_random_rows(w4lib, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = rng.choice((3, 9, 513, 2047, 4096, 16384, 32767, 32768, 70001, 131072, 300001))
    rows = min(rng.choice((1, 2, 19, 38, 76, 77, 151, 160, 305)),
               max(1, (100_000 if n <= 4096 else 3_000_000) // n))
    dtype, shift = rng.choice(TYPES), rng.randrange(0, 9)
    wide = torch.randn(rows, n + shift + rng.randrange(0, 5), generator=g, device="cuda")
    wide *= rng.choice((0.01, 1.0, 4.0, 30.0))
    kind = seed % 5
    if kind == 1:
        wide = (wide * 0.3).round()
    elif kind == 2:
        wide[:, rng.randrange(0, 12):] = -math.inf
    elif kind == 3:
        wide[torch.rand(wide.shape, generator=g, device="cuda") < 0.7] = -math.inf
    elif kind == 4:
        wide[torch.rand(wide.shape, generator=g, device="cuda") < 0.9] = torch.finfo(dtype).min
    tokens = torch.randint(-1, n + 1, (rows,), generator=g, device="cuda")
    check(wide.to(dtype)[:, shift:shift + n], tokens, rng.randrange(0, min(n, 32) + 1))


def test_refusals(w4lib):
    x, tokens = random_logits(2, 100, torch.float16)
    for bad in ((x.double(), tokens, 0), (x.cpu(), tokens, 0), (x[0], tokens, 0),
                (x.t(), tokens, 0), (x, tokens[:1], 0), (x, tokens.float(), 0),
                (x, tokens, 33), (x, tokens, -1), (x[:, :3], tokens, 4)):
        with pytest.raises(ValueError):
            w4.token_logprobs(bad[0], bad[1], top=bad[2])
    none = w4.token_logprobs(x[:0], tokens[:0], top=3)
    assert [list(t.shape) for t in none] == [[0], [0], [0, 3], [0, 3]]
