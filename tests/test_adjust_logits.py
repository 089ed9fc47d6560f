"""Penalties, biases and masks on logits against the definition in 64 bits.

Tolerance, from the arithmetic: a quotient or product, a fused product and
differences, and one sum a bias are FP32, each off by 2^-24 of what is summed so far:
(3 + biases of the token) 2^-24 (|x| r + f c + |p| + sum |b|) at most, r the larger of the
penalty and its inverse.  The result is rounded once, by u of it (u = 2^-11 for fp16, 2^-8
for bf16, 2^-24 for fp32).  What nothing applies to keeps its bits."""
from __future__ import annotations

import math

import pytest
import torch

import prompt_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = list(UNIT)
gpu = pytest.mark.gpu


def make(rows, vocabulary, width, dtype, biases=0, masked=False, seed=0, wide=False):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocabulary, generator=g) * 3).to(dtype).cuda()
    tokens = (torch.rand(rows, width, generator=g) ** 4 * vocabulary).int()
    lengths = torch.randint(0, width + 1, (rows,), generator=g).int()
    s = {"tokens": (tokens.long() if wide else tokens).cuda(), "lengths": lengths.cuda(),
         "prompts": (lengths * torch.rand(rows, generator=g)).int().cuda(),
         "repetition": (torch.rand(rows, generator=g) * 0.5 + 0.9).cuda(),
         "presence": torch.randn(rows, generator=g).cuda(),
         "frequency": torch.rand(rows, generator=g).cuda()}
    if biases:
        # some of tokens that were said, some listed twice, some outside the vocabulary
        ids = torch.randint(-3, vocabulary + 3, (rows, biases), generator=g).int()
        ids[:, ::3] = tokens[:, torch.arange(0, biases, 3) % width]
        if biases > 4:
            ids[:, 4] = ids[:, 1]
        s["bias_ids"], s["biases"] = ids.cuda(), torch.randn(rows, biases, generator=g).cuda()
    if masked:
        words = -(-vocabulary // 32)
        mask = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=g).int()
        mask[:, words // 3:words // 2] = 0
        mask[:, words // 2:] = -1
        s["mask"] = mask.cuda()
    return x, s


def near(x, got, want, s):
    got, want, x = got.cpu(), want, x.cpu().double()
    value = lambda n: s[n].cpu().double()[:, None] if isinstance(s.get(n), torch.Tensor) \
        else torch.tensor(float(s.get(n, n == "repetition")))  # noqa: E731
    r = value("repetition")
    width = s["tokens"].shape[1] if s.get("tokens") is not None else 0
    scale = x.abs() * torch.maximum(r, 1 / r) + value("frequency").abs() * width \
        + value("presence").abs()
    sums = 3
    if s.get("biases") is not None:
        scale = scale + s["biases"].cpu().double().abs().sum(1, keepdim=True)
        sums += s["biases"].shape[1]
    assert torch.equal(got == -math.inf, want == -math.inf)
    live = want > -math.inf
    far = (got.double() - want).abs() - UNIT[got.dtype] * want.abs() - sums * 2.0 ** -24 * scale
    assert far[live].max() <= (2.0 ** -25 if got.dtype == torch.float16 else 0.0)


def check(x, s, **kw):
    before = x.clone()
    got = w4.adjust_logits(x, **s, **kw)
    torch.cuda.synchronize()
    want = ref.adjusted(before, **s)
    near(before, got, want, s)
    same = want == before.cpu().double()
    bits = torch.int32 if x.dtype == torch.float32 else torch.int16
    assert torch.equal(got.cpu().view(bits)[same], before.cpu().view(bits)[same])
    return got


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocabulary", [1, 7, 31, 33, 1000, 1027, 4099])
@pytest.mark.parametrize("masked", [False, True])
def test_sizes(w4lib, vocabulary, masked, dtype):
    for rows, width, biases in ((1, 1, 0), (3, 50, 1), (5, 700, 40)):
        x, s = make(rows, vocabulary, width, dtype, biases, masked, seed=vocabulary + rows)
        check(x, s)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, vocabulary, width", [(1, 128256, 2000), (2, 151000, 9000),
                                                     (40, 50001, 300)])
def test_large(w4lib, rows, vocabulary, width, dtype):
    x, s = make(rows, vocabulary, width, dtype, 300, True, seed=rows, wide=rows == 2)
    s["mask"] = s["mask"] if rows < 40 else None     # the definition's loop over a mask is slow
    check(x, s)


@gpu
def test_every_slice_size(w4lib):
    """Rows and vocabularies on both sides of each change in how a row is cut, each row the
    same as alone."""
    for rows, vocabulary in ((1, 600000), (3, 700001), (17, 130001), (300, 33001), (2000, 5003)):
        x, s = make(rows, vocabulary, 64, torch.bfloat16, 5, True, seed=rows)
        got = w4.adjust_logits(x, **s)
        for r in (0, rows // 2, rows - 1):
            one = {n: t[r:r + 1] for n, t in s.items()}
            assert torch.equal(w4.adjust_logits(x[r:r + 1], **one), got[r:r + 1])
        near(x[:1], got[:1], ref.adjusted(x[:1], **{n: t[:1] for n, t in s.items()}),
             {n: t[:1] for n, t in s.items()})


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("masked", [False, True])
def test_in_place(w4lib, dtype, masked):
    x, s = make(6, 5003, 200, dtype, 20, masked, seed=4)
    want = w4.adjust_logits(x, **s)
    same = x.clone()
    got = w4.adjust_logits(same, **s, out=same)
    assert got.data_ptr() == same.data_ptr() and torch.equal(same, want)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(w4lib, dtype):
    """Rows that begin anywhere: of a wider tensor, a value past its start, in and out alike
    or not; wider tables of tokens, biases and words."""
    x, s = make(5, 3001, 90, dtype, 12, True, seed=5)
    want = check(x, s)
    for pad, first, out_first in ((7, 0, 0), (8, 1, 1), (16, 3, 5), (5, 2, 0)):
        wide = torch.full((5, 3001 + pad), 3.0, device="cuda", dtype=dtype)
        wide[:, first:first + 3001] = x
        out = torch.full((5, 3001 + pad), 9.0, device="cuda", dtype=dtype)
        got = w4.adjust_logits(wide[:, first:first + 3001], **s,
                               out=out[:, out_first:out_first + 3001])
        assert torch.equal(got, want)
        assert (out[:, :out_first] == 9).all() and (out[:, out_first + 3001:] == 9).all()
    apart = dict(s)
    for name in ("tokens", "bias_ids", "biases", "mask"):
        t = s[name]
        w = torch.zeros(5, t.shape[1] + 9, dtype=t.dtype, device="cuda")
        w[:, 3:3 + t.shape[1]] = t
        apart[name] = w[:, 3:3 + t.shape[1]]
    assert torch.equal(w4.adjust_logits(x, **apart), want)


@gpu
def test_parts_alone(w4lib):
    x, s = make(4, 900, 60, torch.float32, 9, True, seed=6)
    for names in ((), ("mask",), ("bias_ids", "biases"), ("tokens",), ("tokens", "lengths"),
                  ("tokens", "prompts"), ("tokens", "repetition"), ("tokens", "frequency"),
                  ("tokens", "lengths", "prompts", "presence")):
        check(x, {n: s[n] for n in names})
    check(x, {"tokens": s["tokens"], "repetition": 1.25, "presence": -0.5, "frequency": 0.75})
    assert w4.adjust_logits(x[:0]).shape == (0, 900)


@gpu
def test_tokens_out_of_range(w4lib):
    """Tokens and biases outside the vocabulary, lengths and prompts outside the width."""
    x, s = make(4, 500, 40, torch.float16, 5, seed=7)
    s["tokens"][0, :5] = torch.tensor([-1, 500, 2 ** 31 - 1, -2 ** 31, 499]).int()
    s["lengths"] = torch.tensor([40, -3, 10 ** 9, 0], dtype=torch.int32, device="cuda")
    s["prompts"] = torch.tensor([-7, 5, 50, 3], dtype=torch.int32, device="cuda")
    check(x, s)
    s["tokens"] = s["tokens"].long()
    s["tokens"][0, 5:8] = torch.tensor([2 ** 32 + 1, -2 ** 62, 2 ** 62])
    check(x, s)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite(w4lib, dtype):
    """Masked logits of -infinity and of the type's lowest value, NaN in one place."""
    x = torch.zeros(2, 40, device="cuda", dtype=dtype)
    x[:, 1], x[:, 2], x[:, 3], x[0, 4] = -math.inf, torch.finfo(dtype).min, math.inf, math.nan
    tokens = torch.tensor([[1, 2, 3, 4], [1, 2, 3, 5]], dtype=torch.int32, device="cuda")
    mask = torch.tensor([[-1, -1], [-1 & ~(1 << 3), 0]], dtype=torch.int32, device="cuda")
    y = w4.adjust_logits(x, tokens, repetition=2.0, frequency=0.5, mask=mask)
    assert (y[:, 1] == -math.inf).all() and (y[:, 2] == -math.inf).all()
    assert y[0, 3] == math.inf and y[1, 3] == -math.inf and torch.isnan(y[0, 4])
    assert (y[0, 5:] == 0).all() and y[1, 5] == -0.5 and (y[1, 6:32] == 0).all()
    assert (y[1, 32:] == -math.inf).all()


@gpu
def test_a_token_said_very_often(w4lib):
    tokens = torch.zeros(1, 200000, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 64, device="cuda")
    prompts = torch.tensor([50000], dtype=torch.int32, device="cuda")
    y = w4.adjust_logits(x, tokens, prompts=prompts, frequency=0.5, presence=1.0)
    assert y[0, 0] == -75001.0 and (y[0, 1:] == 0).all()


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("width", [60, 900, 9000, 20000])
def test_in_place_with_tokens_said_again(w4lib, width, wide):
    """Few and many finds of a thread, words of 16 and of 32 bits."""
    x, s = make(3, 9001, width, torch.float32, 20, True, seed=width, wide=wide)
    want = check(x, s)
    assert torch.equal(w4.adjust_logits(x, **s, out=x), want)


@gpu
def test_streams_graphs_and_repeats(w4lib):
    x, s = make(8, 20011, 500, torch.bfloat16, 30, True, seed=8)
    want = w4.adjust_logits(x, **s)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = w4.adjust_logits(x, **s, stream=stream)
    stream.synchronize()
    with torch.cuda.stream(stream):
        assert torch.equal(got, want)
    torch.cuda.synchronize()
    a, b = x.clone(), x.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph, t in zip(graphs, (a, b)):
        with torch.cuda.graph(graph):
            outs.append(w4.adjust_logits(t, **s))
    b.mul_(0.5)
    half = w4.adjust_logits(b, **s)
    for graph in graphs + graphs[::-1]:
        graph.replay()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], half)


def test_refused_calls():
    x = torch.zeros(3, 40).half()
    t, n = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    ids, values = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    for bad in (dict(logits=x[0]), dict(logits=x.double()), dict(logits=x.t()),
                dict(tokens=t.float()), dict(tokens=t[:2]), dict(tokens=t.t()), dict(lengths=n),
                dict(prompts=n), dict(tokens=t, lengths=n.long()), dict(tokens=t, prompts=n[:2]),
                dict(repetition=0.0), dict(repetition=math.nan), dict(presence=torch.zeros(3).half()),
                dict(frequency=torch.zeros(2)), dict(repetition=torch.zeros(3, 1)),
                dict(bias_ids=ids), dict(biases=values), dict(bias_ids=ids[:, :3], biases=values),
                dict(bias_ids=ids.long(), biases=values), dict(bias_ids=ids, biases=values.half()),
                dict(bias_ids=torch.zeros(3, 1025, dtype=torch.int32),
                     biases=torch.zeros(3, 1025)),
                dict(mask=t), dict(mask=ids[:, :2].long()), dict(mask=ids[:2, :2]),
                dict(out=x.float()), dict(out=x[:, :39]), dict(out=torch.zeros(40, 3).half().t()),
                dict()):
        with pytest.raises(ValueError):
            w4.adjust_logits(**{"logits": x, **bad})
