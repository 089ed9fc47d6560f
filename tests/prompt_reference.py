"""Plain 64-bit definitions of the prompt-side serving operators, for their tests:
on the CPU, sharing nothing with the library."""
from __future__ import annotations

import math
import random
from fractions import Fraction

import torch

INVERSE_TURN = Fraction(10 ** 50, 628318530717958647692528676655900576839433879875021)


def turns(positions, rates):
    """cos and sin [positions, rates] of position * rate, the angle reduced exactly."""
    angle = [[float(2 * math.pi * ((p * Fraction(r) * INVERSE_TURN) % 1)) for r in rates]
             for p in positions]
    angle = torch.tensor(angle, dtype=torch.float64).view(len(positions), len(rates))
    return angle.cos(), angle.sin()


def rotate(x, positions, rates, interleaved, magnitude=1.0):
    """(rotated, bound): bound is |a| + |b| of each value's pair times the magnitude, 0 where
    nothing is rotated."""
    x = x.detach().cpu().double()
    out, bound, n = x.clone(), torch.zeros_like(x), len(rates)
    c, s = turns(list(map(int, positions)), rates)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        ci, si = c[:, i, None] * magnitude, s[:, i, None] * magnitude
        out[..., a] = x[..., a] * ci - x[..., b] * si
        out[..., b] = x[..., a] * si + x[..., b] * ci
        bound[..., a] = bound[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(magnitude)
    return out, bound


def chunk_attention(q, k_pool, v_pool, tables, lengths, offsets, scale):
    """(out, lse, bound, mass): bound is max_p sum_d |q k| scale over what a head sees, mass the
    weighted average of |v|."""
    q, k_pool, v_pool = (t.detach().cpu().double() for t in (q, k_pool, v_pool))
    pages, ps, kv, d = k_pool.shape
    tokens, heads = q.shape[:2]
    group = heads // kv
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    bound = torch.zeros((tokens, heads), dtype=torch.float64)
    offsets = offsets.tolist()
    for b, (row, n) in enumerate(zip(tables.tolist(), lengths.tolist())):
        n = min(max(n, 0), len(row) * ps)
        held = [(row[p // ps], p % ps, p) for p in range(n) if 0 <= row[p // ps] < pages]
        if not held:
            continue
        g, s, at = (torch.tensor(x) for x in zip(*held))
        first, last = offsets[b], offsets[b + 1]
        if first == last:
            continue
        position = torch.arange(n - (last - first), n)
        seen = at <= position[:, None]
        for h in range(heads):
            k, v = k_pool[g, s, h // group], v_pool[g, s, h // group]
            x = (q[first:last, h] @ k.T) * scale
            x = torch.where(seen, x, -math.inf)
            one = torch.logsumexp(x, 1)
            w = torch.where(seen, torch.exp(x - torch.where(one > -math.inf, one, 0)[:, None]), 0.0)
            lse[first:last, h] = one
            out[first:last, h] = w @ v
            mass[first:last, h] = w @ v.abs()
            bound[first:last, h] = torch.where(
                seen, (q[first:last, h].abs() @ k.abs().T) * abs(scale), 0.0).amax(1)
    return out, lse, bound, mass


def adjusted(logits, tokens=None, lengths=None, prompts=None, repetition=1.0, presence=0.0,
             frequency=0.0, bias_ids=None, biases=None, mask=None):
    """The adjusted logits in binary64, by loops over lists."""
    x = logits.detach().cpu().double()
    rows, n = x.shape
    of = lambda v, r: v[r].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    for r in range(rows):
        said = [] if tokens is None else tokens[r].tolist()
        if lengths is not None:
            said = said[:max(0, int(lengths[r]))]
        first = 0 if prompts is None else max(0, int(prompts[r]))
        counts = {}
        for i, t in enumerate(said):
            if 0 <= t < n:
                counts[t] = counts.get(t, 0) + (i >= first)
        for t, c in counts.items():
            v = x[r, t].item()
            v = v / of(repetition, r) if v > 0 else v * of(repetition, r)
            if c:
                v -= of(frequency, r) * c + of(presence, r)
            x[r, t] = v
        if bias_ids is not None:
            for t, v in zip(bias_ids[r].tolist(), biases[r].tolist()):
                if 0 <= t < n:
                    x[r, t] += v
        if mask is not None:
            words = mask[r].tolist()
            for t in range(n):
                if not words[t // 32] >> (t % 32) & 1:
                    x[r, t] = -math.inf
    return x


def cache(rows, kv_heads, dim, page, dtype, layout="slots", seed=0, spare=3, garbage=math.nan,
          width=None):
    """(k_pool, v_pool, tables, lengths, offsets) of rows of (held, new) tokens on scattered
    pages; every slot that no row holds is filled with `garbage`."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    lengths = [held + new for held, new in rows]
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    width = width or max(1, max(need))
    order = rng.sample(range(pages), sum(need))
    tables, at = [], 0
    for n in need:
        tables.append(order[at:at + n] + [-1] * (width - n))
        at += n
    pools = []
    for _ in range(2):
        p = torch.full((pages, page, kv_heads, dim), garbage)
        for row, n in zip(tables, lengths):
            for t in range(0, n, page):
                m = min(page, n - t)
                p[row[t // page], :m] = torch.randn(m, kv_heads, dim, generator=g)
        pools.append(p.to(dtype))
    if layout == "heads":
        pools = [p.transpose(1, 2).contiguous().cuda().transpose(1, 2) for p in pools]
    elif layout == "both":  # keys and values of a page side by side
        both = torch.stack(pools, 1).cuda()
        pools = [both[:, 0], both[:, 1]]
    else:
        pools = [p.cuda() for p in pools]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets = [0]
    for _, new in rows:
        offsets.append(offsets[-1] + new)
    return *pools, ints(tables), ints(lengths), ints(offsets)
