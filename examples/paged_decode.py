#!/usr/bin/env python3
"""Best-of-n decoding with quantized linear layers and a paged cache.

A small decoder with random weights (W4A16 linear layers, grouped query heads)
takes prompts of uneven lengths, branches each into n continuations that share
the prompt's pages, decodes them side by side, scores what was sampled, keeps
each prompt's likeliest branch, gives the other pages back and draws the rest
together:

    python examples/paged_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_weight_only_gemm_gb300 as w4  # noqa: E402
from w4a16_weight_only_gemm_gb300 import synthetic  # noqa: E402


def ints(values) -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Decoder:
    """Pre-norm transformer layers: attention over a PagedCache, then a gated MLP."""

    def __init__(self, layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=64, mlp=1024,
                 vocabulary=1024, seed=0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim

        def linear(n, k, i):
            return w4.W4A16Linear(synthetic.master_weight(n, k, seed + i).cuda())

        qkv = (q_heads + 2 * kv_heads) * head_dim
        self.layers = [{"qkv": linear(qkv, hidden, 10 * i + 1),
                        "out": linear(hidden, q_heads * head_dim, 10 * i + 2),
                        "up": linear(2 * mlp, hidden, 10 * i + 3),
                        "down": linear(hidden, mlp, 10 * i + 4)} for i in range(layers)]
        self.head = linear(vocabulary, hidden, 9999)
        g = torch.Generator().manual_seed(seed)
        self.embedding = torch.randn(vocabulary, hidden, generator=g).half().cuda()

    @staticmethod
    def norm(x: torch.Tensor) -> torch.Tensor:
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).half()

    @staticmethod
    def rotate(x: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
        """Rotary positions on [tokens, heads, head_dim], halves paired."""
        half = x.shape[-1] // 2
        rate = 10000.0 ** (-torch.arange(half, device=x.device) / half)
        angle = positions[:, None, None].float() * rate
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()],
                         -1).half()

    def forward(self, tokens, positions, attend) -> torch.Tensor:
        """Logits of tokens [n] at positions [n]; attend(layer, q, k, v) puts k and v where
        they belong and returns the attention's output [n, q_heads, head_dim]."""
        x = self.embedding[tokens.long()].float()
        heads, kv, d = self.q_heads, self.kv_heads, self.head_dim
        for i, layer in enumerate(self.layers):
            qkv = layer["qkv"](self.norm(x)).unflatten(1, (heads + 2 * kv, d))
            q = self.rotate(qkv[:, :heads], positions)
            k = self.rotate(qkv[:, heads:heads + kv], positions)
            o = attend(i, q, k, qkv[:, heads + kv:])
            x = x + layer["out"](o.flatten(1)).float()
            gate, up = layer["up"](self.norm(x)).float().chunk(2, -1)
            x = x + layer["down"]((torch.nn.functional.silu(gate) * up).half()).float()
        return self.head(self.norm(x))


def prefill(model: Decoder, cache: w4.PagedCache, prompts: list[list[int]], rows) -> torch.Tensor:
    """Prompts into the listed rows; logits of each prompt's last token."""
    counts = [len(p) for p in prompts]
    starts = cache.lengths.index_select(0, rows)
    if not cache.extend(rows, ints(counts)).all():
        raise RuntimeError("the cache has too few free pages for the prompts")
    offsets = ints([sum(counts[:i]) for i in range(len(counts) + 1)])
    row = torch.repeat_interleave(torch.arange(len(prompts), device="cuda"), ints(counts).long())
    tokens = ints([t for p in prompts for t in p])
    positions = ints([i for n in counts for i in range(n)]) + starts[row]
    tables = cache.tables.index_select(0, rows)

    def attend(layer, q, k, v):
        cache.append(layer, k, v, starts, offsets, rows=rows)
        # each token of a prompt is a row of its own that ends with it
        return w4.paged_attention(q, cache.keys(layer), cache.values(layer), tables[row],
                                  positions + 1)

    return model.forward(tokens, positions, attend)[offsets[1:].long() - 1]


def decode(model: Decoder, cache: w4.PagedCache, tokens: torch.Tensor):
    """One token of every row of the cache; the next token's logits, and PagedCache.extend's
    answer.  A row of length 0 takes no part, and one whose answer is 0 found no page for its
    token (or was listed after such a row): their logits say nothing."""
    rows = torch.arange(cache.tables.shape[0], dtype=torch.int32, device="cuda")
    starts = cache.lengths.clone()
    done = cache.extend(rows, (starts > 0).int())

    def attend(layer, q, k, v):
        cache.append(layer, k, v, starts)
        return cache.attend(layer, q)

    return model.forward(tokens, starts, attend), done


def best_of(model: Decoder, cache: w4.PagedCache, prompts: list[list[int]], n: int, steps: int,
            seed: int = 0):
    """n sampled continuations of each prompt; (tokens, summed log probability) of the likeliest,
    and the rows that hold them.  The cache has len(prompts) * n rows, all empty."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    count = len(prompts)
    first = ints([i * n for i in range(count)])
    logits = prefill(model, cache, prompts, first)
    parents = [i * n for i in range(count) for _ in range(n - 1)]
    children = [i * n + j for i in range(count) for j in range(1, n)]
    if not cache.fork(ints(parents), ints(children)).all():
        raise RuntimeError("the cache has too few free pages for the branches")
    logits = logits.repeat_interleave(n, 0)
    total = torch.zeros(count * n, device="cuda")
    sampled = []
    placed = torch.ones(count * n, dtype=torch.int32, device="cuda")
    for step in range(steps):
        if step:
            logits, done = decode(model, cache, sampled[-1])
            placed &= done                     # looked at once, after the last step
        noise = torch.rand(logits.shape, generator=g, device="cuda").clamp_min(1e-9)
        tokens = (logits.float() - torch.log(-torch.log(noise))).argmax(1)
        logprobs, _, _, _ = w4.token_logprobs(logits, tokens, top=4)
        total += logprobs
        sampled.append(tokens)
    if not placed.all():
        raise RuntimeError("the cache ran out of free pages while decoding")
    best = total.view(count, n).argmax(1) + torch.arange(count, device="cuda") * n
    kept = best.tolist()
    cache.free(ints([r for r in range(count * n) if r not in kept]))
    cache.compact()
    text = torch.stack(sampled, 1)
    return [(text[r].tolist(), total[r].item()) for r in kept], kept


def main() -> None:
    model = Decoder()
    prompts = [[(7 * i + j * j) % 1024 for j in range(n)] for i, n in enumerate((37, 5, 64, 18))]
    cache = w4.PagedCache(layers=len(model.layers), rows=16, pages=64, kv_heads=model.kv_heads,
                          head_dim=model.head_dim, page_size=16, max_length=256)
    answers, rows = best_of(model, cache, prompts, n=4, steps=12)
    for prompt, (tokens, score) in zip(prompts, answers):
        print(f"prompt of {len(prompt):3d} tokens: log probability {score:8.3f}, {tokens}")
    held = int((cache.refs > 0).sum())
    print(f"{held} pages held, the highest number {int(cache.tables.max())}, "
          f"rows {rows} of lengths {cache.lengths[rows].tolist()}")


if __name__ == "__main__":
    main()
