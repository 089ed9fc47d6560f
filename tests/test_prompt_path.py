"""The prompt-side operators together: the example's chunked serving against a dense
forward pass of the same decoder that keeps every key and value, and a mixed step
captured in a graph.

The dense pass shares the example's layers, so both round the same activations to
fp16 at the same places; they differ by the attention's own rounding and the
rotation's (2^-11 of what they give, twice: weights and output), and what later layers
make of it, some units of 2^-11 of a logit of order 1 each.  A row's logits are off by
at most 32 * 2^-11 * max|logit|: twice what the single-token path is held to."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import prompt_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import chunked_serving  # noqa: E402
from chunked_serving import ChunkedDecoder, Server, ints  # noqa: E402

pytestmark = pytest.mark.gpu


def dense_logits(model, tokens):
    """Logits at every position of one sequence; positions and attention by their definitions."""
    n, r = len(tokens), model.rotary
    group = model.q_heads // model.kv_heads
    c, s = (t.cuda() for t in ref.turns(range(n), r.rates))

    def turn(x):
        a, b = x.double().chunk(2, -1)
        return torch.cat([a * c[:, None] - b * s[:, None], a * s[:, None] + b * c[:, None]], -1).half()

    def attend(layer, q, k, v):
        q, k = turn(q).float(), turn(k).float()
        k, v = (t.float().repeat_interleave(group, 1) for t in (k, v))
        x = torch.einsum("ihd,jhd->hij", q, k) * model.head_dim ** -0.5
        later = torch.ones(n, n, device="cuda").triu(1).bool()
        p = torch.softmax(x.masked_fill(later, -torch.inf), -1)
        return torch.einsum("hij,jhd->ihd", p, v).half()

    return model.forward(ints(tokens), None, attend)


@pytest.mark.parametrize("page_size, chunk", [(16, 50), (1, 7), (13, 1000), (64, 33)])
def test_chunks_against_a_dense_pass(w4lib, page_size, chunk):
    """Each step's logits, before they are adjusted, are the dense pass's at that position."""
    model = ChunkedDecoder()
    prompts = [[(7 * i + j * j) % 1024 for j in range(m)] for i, m in enumerate((137, 1, 64, 90))]
    cache = w4.PagedCache(len(model.layers), len(prompts), 2000 // page_size, model.kv_heads,
                          model.head_dim, page_size=page_size, max_length=400)
    read = [0] * len(prompts)
    text = [list(p) for p in prompts]
    for p in text:
        p += [3 * len(p) % 1024, 5, 6]           # a few tokens after the prompt, one a step
    seen = []
    while min(n - len(t) for n, t in zip(read, text)) < 0:
        rows = [r for r, n in enumerate(read) if n < len(text[r])]
        pieces = [text[r][read[r]:read[r] + chunk] if read[r] < len(prompts[r])
                  else text[r][read[r]:read[r] + 1] for r in rows]
        logits = chunked_serving.step(model, cache, rows, pieces)
        for r, piece, x in zip(rows, pieces, logits):
            read[r] += len(piece)
            seen.append((r, read[r] - 1, x))
    for r in range(len(prompts)):
        want = dense_logits(model, text[r]).float()
        for row, at, x in seen:
            if row == r:
                assert (x.float() - want[at]).abs().max() <= 32 * 2.0 ** -11 * want[at].abs().max()
    assert cache.lengths.tolist() == [len(t) for t in text]


def test_the_server_takes_what_its_rules_leave(w4lib):
    """Every answer's token is the likeliest by the adjusted logits' definition, or one as likely
    up to the logits' own rounding; a masked row gives even tokens only."""
    model = ChunkedDecoder(layers=1)
    prompts = [[(7 * i + j * j) % 1024 for j in range(m)] for i, m in enumerate((70, 3, 41))]
    cache = w4.PagedCache(1, 3, 64, model.kv_heads, model.head_dim, max_length=256)
    server = Server(model, cache, prompts, chunk=32, even_rows=(1,))
    for _ in range(9):
        server.step()
    assert [len(a) for a in server.answers] == [7, 9, 8]
    assert all(t % 2 == 0 for t in server.answers[1])
    for r, (prompt, answer) in enumerate(zip(prompts, server.answers)):
        logits = dense_logits(model, prompt + answer[:-1])[len(prompt) - 1:]
        slack = 2 * 32 * 2.0 ** -11 * logits.float().abs().max().item() * 1.3
        for i, token in enumerate(answer):
            said = ints([prompt + answer[:i]])
            x = ref.adjusted(logits[i:i + 1], said, prompts=ints([len(prompt)]), repetition=1.3,
                             frequency=0.2, mask=server.mask[r:r + 1])[0]
            assert x[token] >= x.max() - slack


def test_the_example_runs(w4lib, capsys):
    chunked_serving.main()
    assert capsys.readouterr().out.count("log probability") == 4


def test_a_mixed_step_in_a_graph(w4lib):
    """Room, rotated append, attention of chunks and adjusted logits captured once and replayed on
    other inputs, as eager calls leave the cache and give their outputs."""
    counts, kv, heads, dim = [1, 40, 0, 7], 2, 8, 64
    rotary = w4.Rotary(dim)
    offsets = ints([0, 1, 41, 41, 48])
    rows, news = ints([0, 1, 2, 3]), ints(counts)
    said = torch.randint(0, 500, (4, 30), device="cuda", dtype=torch.int32)

    def fresh():
        cache = w4.PagedCache(2, 4, 60, kv, dim, page_size=8, max_length=200)
        g = torch.Generator(device="cuda").manual_seed(1)
        cache.pool.normal_(generator=g)
        cache.extend(ints([0, 1, 3]), ints([70, 3, 9]))
        return cache

    def step(cache, qkv, logits, stream=None):
        starts = cache.lengths.clone()
        done = cache.extend(rows, news, stream=stream)
        outs = []
        for layer in range(2):
            q = cache.append_rotary(layer, qkv[:, heads:heads + kv], qkv[:, heads + kv:], starts,
                                    rotary, offsets, q=qkv[:, :heads], stream=stream)
            outs.append(cache.attend_chunks(layer, q, offsets, stream=stream))
        return (done, *outs, w4.adjust_logits(logits, said, frequency=0.5, stream=stream))

    g = torch.Generator(device="cuda").manual_seed(2)
    inputs = [(torch.randn(48, heads + 2 * kv, dim, generator=g, device="cuda").half(),
               torch.randn(4, 500, generator=g, device="cuda").half()) for _ in range(3)]
    eager = fresh()
    want = [[t.clone() for t in step(eager, *x)] for x in inputs]
    captured = fresh()
    now = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(captured, *now)
    for x, values in zip(inputs, want):
        for t, value in zip(now, x):
            t.copy_(value)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, values))
    aside, stream = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for x, values in zip(inputs, want):
        with torch.cuda.stream(stream):
            got = step(aside, *x, stream)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, values))
    for cache in (captured, aside):
        for name in ("refs", "tables", "lengths", "pool"):
            assert torch.equal(getattr(cache, name), getattr(eager, name))


def test_listed_rows_out_of_range(w4lib):
    """A listed row that is none: its tokens go nowhere, its queries are rotated to where the call
    says, its attention is zeros."""
    cache = w4.PagedCache(1, 3, 20, 2, 64, page_size=8, max_length=64)
    cache.pool.normal_()
    cache.extend(ints([0, 1, 2]), ints([20, 20, 20]))
    before = cache.pool.clone()
    listed, offsets = ints([1, 7, -1]), ints([0, 2, 5, 6])
    qkv = torch.randn(6, 8, 64, device="cuda").half()
    q = cache.append_rotary(0, qkv[:, 4:6], qkv[:, 6:], ints([18, 3, 0]), w4.Rotary(64), offsets,
                            q=qkv[:, :4], rows=listed)
    touched = (cache.pool != before).any(0).flatten(1).any(1)
    assert set(touched.nonzero()[:, 0].tolist()) <= set(cache.tables[1].tolist())
    turned = w4.rotate(qkv[:, :4], ints([18, 19, 3, 4, 5, 0]), w4.Rotary(64))
    assert torch.equal(q, turned)
    out = cache.attend_chunks(0, q, offsets, rows=listed)
    assert (out[2:] == 0).all() and out[:2].abs().sum() > 0
