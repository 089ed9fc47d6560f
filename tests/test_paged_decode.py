"""The serving operators together: the example's best-of-n decoding against a
dense forward pass of the same decoder that keeps every key and value.

The dense pass shares the example's layers, so both round the same
activations to fp16 at the same places; they differ by the attention's own
rounding (2^-11 of its output) and what later layers make of it, a few units of
2^-11 of a logit of order 1 each.  A summed log probability over `steps` tokens
is off by at most steps * 2 * 8 * 2^-11 * max|logit|."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import w4a16_weight_only_gemm_gb300 as w4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import paged_decode  # noqa: E402

pytestmark = pytest.mark.gpu


def dense_logits(model, tokens):
    """Logits at every position of one sequence, attention in FP32 over all of it."""
    n = len(tokens)
    group = model.q_heads // model.kv_heads

    def attend(layer, q, k, v):
        k, v = (t.float().repeat_interleave(group, 1) for t in (k, v))
        x = torch.einsum("ihd,jhd->hij", q.float(), k) * model.head_dim ** -0.5
        later = torch.ones(n, n, device="cuda").triu(1).bool()
        p = torch.softmax(x.masked_fill(later, -torch.inf), -1)
        return torch.einsum("hij,jhd->ihd", p, v).half()

    return model.forward(paged_decode.ints(tokens), paged_decode.ints(list(range(n))), attend)


@pytest.mark.parametrize("page_size, n, steps", [(16, 4, 12), (1, 2, 5), (13, 3, 20)])
def test_best_of_n(w4lib, page_size, n, steps):
    model = paged_decode.Decoder()
    prompts = [[(7 * i + j * j) % 1024 for j in range(m)] for i, m in enumerate((37, 1, 64, 16))]
    cache = w4.PagedCache(len(model.layers), len(prompts) * n, 2000 // page_size, model.kv_heads,
                          model.head_dim, page_size=page_size, max_length=128)
    answers, rows = paged_decode.best_of(model, cache, prompts, n, steps, seed=n)
    for prompt, (tokens, score) in zip(prompts, answers):
        logits = dense_logits(model, prompt + tokens[:-1])[len(prompt) - 1:].float()
        want = torch.log_softmax(logits.double(), 1)[range(steps), tokens].sum().item()
        assert abs(score - want) <= steps * 2 * 8 * 2.0 ** -11 * logits.abs().max().item()
    # the kept rows alone hold pages, each its own, drawn together from 0 on
    assert [r for r, m in enumerate(cache.lengths.tolist()) if m] == rows
    assert cache.lengths[rows].tolist() == [len(p) + steps - 1 for p in prompts]
    pages = sum(-(-(len(p) + steps - 1) // page_size) for p in prompts)
    assert sorted(p for p in cache.tables.flatten().tolist() if p >= 0) == list(range(pages))
    assert cache.refs.tolist() == [1] * pages + [0] * (cache.refs.numel() - pages)


def test_too_few_pages(w4lib):
    model = paged_decode.Decoder(layers=1)
    cache = w4.PagedCache(1, 4, 3, model.kv_heads, model.head_dim, max_length=64)
    with pytest.raises(RuntimeError, match="prompts"):
        paged_decode.best_of(model, cache, [[1] * 60], 4, 3)
    with pytest.raises(RuntimeError, match="branches"):
        paged_decode.best_of(model, cache, [[1] * 20], 4, 3)


def test_the_example_runs(w4lib, capsys):
    paged_decode.main()
    assert "pages held" in capsys.readouterr().out


def test_a_decode_step_in_a_graph(w4lib):
    """Room, append and attention of a step captured once and replayed, as eager calls leave
    the cache and their outputs; also all of it on a stream of its own."""
    def fresh():
        cache = w4.PagedCache(2, 5, 40, 2, 64, page_size=8, max_length=64)
        g = torch.Generator(device="cuda").manual_seed(1)
        cache.pool.normal_(generator=g)
        cache.extend(paged_decode.ints([0, 1, 3]), paged_decode.ints([7, 8, 30]))
        return cache

    g = torch.Generator(device="cuda").manual_seed(2)
    steps = [torch.randn(3, 5, 2, 64, generator=g, device="cuda").half() for _ in range(4)]
    rows = torch.arange(5, dtype=torch.int32, device="cuda")

    def step(cache, x, stream=None):
        starts = cache.lengths.clone()
        done = cache.extend(rows, (starts > 0).int(), stream=stream)
        outs = []
        for layer in range(2):
            cache.append(layer, x[0], x[1], starts, stream=stream)
            q = x[2].repeat_interleave(4, 1).contiguous()
            outs.append(cache.attend(layer, q, stream=stream))
        return (done, *outs)

    eager = fresh()
    want = [[t.clone() for t in step(eager, x)] for x in steps]
    captured = fresh()
    x = steps[0].clone()
    books = [t.clone() for t in (captured.refs, captured.tables, captured.lengths)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(captured, x)
    for t, b in zip((captured.refs, captured.tables, captured.lengths), books):
        assert torch.equal(t, b)               # a capture runs nothing
    for now, values in zip(steps, want):
        x.copy_(now)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, values))
    aside = fresh()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for now, values in zip(steps, want):
        with torch.cuda.stream(stream):
            got = step(aside, now, stream)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, values))
    for cache in (captured, aside):
        for t, b in zip((cache.refs, cache.tables, cache.lengths, cache.pool),
                        (eager.refs, eager.tables, eager.lengths, eager.pool)):
            assert torch.equal(t, b)


def test_listed_rows_on_another_stream(w4lib):
    """The listed rows' tables and lengths are taken on the call's stream, not on the current
    one, which is busy with something else."""
    cache = w4.PagedCache(1, 6, 30, 2, 64, page_size=16, max_length=64)
    g = torch.Generator(device="cuda").manual_seed(3)
    cache.pool.normal_(generator=g)
    cache.extend(paged_decode.ints([0, 2, 5]), paged_decode.ints([40, 20, 9]))
    rows = paged_decode.ints([5, 0])
    q = torch.randn(2, 8, 64, generator=g, device="cuda").half()
    k, v = (torch.randn(2, 2, 64, generator=g, device="cuda").half() for _ in range(2))
    starts = paged_decode.ints([8, 39])
    want = cache.pool.clone()
    for i, (r, p) in enumerate(((5, 8), (0, 39))):
        page = int(cache.tables[r, p // 16])
        want[0, page, p % 16], want[1, page, p % 16] = k[i], v[i]
    x = w4.paged_attention(q, want[0], want[1], cache.tables[[5, 0]], cache.lengths[[5, 0]])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)             # some 50 ms on the current stream
    cache.append(0, k, v, starts, rows=rows, stream=stream)
    out = cache.attend(0, q, rows=rows, stream=stream)
    stream.synchronize()
    with torch.cuda.stream(stream):
        assert torch.equal(out, x) and torch.equal(cache.pool, want)


def test_too_few_pages_while_decoding(w4lib):
    """A prompt of 20 and a branch fit in 4 pages of 16; the 13th step of the two does not."""
    model = paged_decode.Decoder(layers=1)

    def cache():
        return w4.PagedCache(1, 2, 4, model.kv_heads, model.head_dim, max_length=64)

    assert paged_decode.best_of(model, cache(), [[1] * 20], 2, 12)[1]
    with pytest.raises(RuntimeError, match="decoding"):
        paged_decode.best_of(model, cache(), [[1] * 20], 2, 16)
