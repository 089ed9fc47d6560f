#!/usr/bin/env python3
"""Serving with prompts in chunks: every step takes one token of each row that is
decoding and the next piece of each prompt that is not yet read, all in one pass.

The decoder is that of paged_decode.py, with its positions rotated on the way into
the cache and for longer contexts than its base allows.  What a row has said is
penalised before the next token is taken, and a grammar (here: even tokens only)
may be laid over a row's answers:

    python examples/chunked_serving.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_weight_only_gemm_gb300 as w4  # noqa: E402
from paged_decode import Decoder, ints  # noqa: E402


class ChunkedDecoder(Decoder):
    """paged_decode's layers; queries and keys reach `attend` as the linear layer left them."""

    def __init__(self, rotary: w4.Rotary | None = None, **sizes):
        super().__init__(**sizes)
        self.rotary = rotary or w4.Rotary(self.head_dim, scaling="ramp", factor=4.0, original=64,
                                          device="cuda")

    def forward(self, tokens, positions, attend) -> torch.Tensor:
        x = self.embedding[tokens.long()].float()
        heads, kv, d = self.q_heads, self.kv_heads, self.head_dim
        for i, layer in enumerate(self.layers):
            qkv = layer["qkv"](self.norm(x)).unflatten(1, (heads + 2 * kv, d))
            o = attend(i, qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:])
            x = x + layer["out"](o.flatten(1)).float()
            gate, up = layer["up"](self.norm(x)).float().chunk(2, -1)
            x = x + layer["down"]((torch.nn.functional.silu(gate) * up).half()).float()
        return self.head(self.norm(x))


def step(model: ChunkedDecoder, cache: w4.PagedCache, rows: list[int], pieces: list[list[int]]):
    """One pass over the next tokens of the listed rows (one or many of each); the logits of each
    row's last one."""
    listed, counts = ints(rows), [len(p) for p in pieces]
    starts = cache.lengths.index_select(0, listed)
    if not cache.extend(listed, ints(counts)).all():
        raise RuntimeError("the cache has too few free pages")
    offsets = ints([sum(counts[:i]) for i in range(len(counts) + 1)])

    def attend(layer, q, k, v):
        q = cache.append_rotary(layer, k, v, starts, model.rotary, offsets, q=q, rows=listed)
        return cache.attend_chunks(layer, q, offsets, rows=listed)

    tokens = ints([t for p in pieces for t in p])
    return model.forward(tokens, None, attend)[offsets[1:].long() - 1]


class Server:
    """Rows of a cache, each with a prompt partly read and an answer partly given."""

    def __init__(self, model: ChunkedDecoder, cache: w4.PagedCache, prompts: list[list[int]],
                 chunk: int, repetition=1.3, frequency=0.2, even_rows=()):
        self.model, self.cache, self.chunk = model, cache, chunk
        self.prompts, self.answers = prompts, [[] for _ in prompts]
        self.read = [0] * len(prompts)
        self.scores = [0.0] * len(prompts)
        self.repetition, self.frequency = repetition, frequency
        vocabulary = model.embedding.shape[0]
        self.mask = torch.full((len(prompts), -(-vocabulary // 32)), -1, dtype=torch.int32,
                               device="cuda")
        for r in even_rows:
            self.mask[r] = 0x55555555

    def step(self) -> None:
        """The next token of every row that answers, the next piece of every prompt."""
        pieces = []
        for prompt, answer, n in zip(self.prompts, self.answers, self.read):
            pieces.append(prompt[n:n + self.chunk] if n < len(prompt) else answer[-1:])
        logits = step(self.model, self.cache, list(range(len(pieces))), pieces)
        self.read = [n + len(p) for n, p in zip(self.read, pieces)]
        done = [r for r, n in enumerate(self.read) if n >= len(self.prompts[r])]
        if not done:
            return
        said = [self.prompts[r] + self.answers[r] for r in done]
        width = max(map(len, said))
        logits = logits[done]
        adjusted = w4.adjust_logits(
            logits, ints([s + [0] * (width - len(s)) for s in said]), ints([len(s) for s in said]),
            ints([len(self.prompts[r]) for r in done]), repetition=self.repetition,
            frequency=self.frequency, mask=self.mask[done])
        tokens = adjusted.argmax(1)
        logprobs, _, _, _ = w4.token_logprobs(adjusted, tokens)
        for r, token, score in zip(done, tokens.tolist(), logprobs.tolist()):
            self.answers[r].append(token)
            self.scores[r] += score


def main() -> None:
    model = ChunkedDecoder()
    prompts = [[(7 * i + j * j) % 1024 for j in range(n)] for i, n in enumerate((137, 5, 64, 218))]
    cache = w4.PagedCache(layers=len(model.layers), rows=len(prompts), pages=64,
                          kv_heads=model.kv_heads, head_dim=model.head_dim, page_size=16,
                          max_length=512)
    server = Server(model, cache, prompts, chunk=50, even_rows=(1,))
    for _ in range(16):
        server.step()
    for prompt, answer, score in zip(prompts, server.answers, server.scores):
        print(f"prompt of {len(prompt):3d} tokens: log probability {score:8.3f}, {answer}")


if __name__ == "__main__":
    main()
