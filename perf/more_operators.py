"""Cases of the prompt-side serving operators: rotary positions, new keys and
values rotated on their way into the paged cache, the attention of chunks of
new tokens over that cache, and the adjustments of logits before sampling.

Each case is one call that a decoding program makes between the quantized linear
layers.  ``run`` makes it in plain torch operations in 32 bits, angles in 64
(``own`` false), or through this package's entry points (``own`` true);
``exact`` has the same answer in 64 bits.  Head counts, head size and
vocabulary are those of ``workloads.py``: 32 query and 8 key-value heads of 128
(or 28 and 4), a vocabulary of 128256.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed() -> list[dict]:
    far = {"base": 500000.0, "scaling": "ramp", "factor": 8.0, "original": 8192, "magnitude": 1.0}
    near = {"base": 10000.0, "scaling": "none", "factor": 1.0, "original": 0, "magnitude": 1.0}
    return [
        # The query and key heads of one token of one user: latency alone.
        {"name": "rotate_1", "op": "rotate", "tokens": 1, "heads": 40, "dim": 128, "part": 128,
         "interleaved": False, "far": 4000, "dtype": "float16", **near},
        # A batch of prompts without a cache, half of each head rotated, neighbours paired, at
        # positions that only a stretched rotation reaches.
        {"name": "rotate_16381", "op": "rotate", "tokens": 16381, "heads": 40, "dim": 128,
         "part": 64, "interleaved": True, "far": 120000, "dtype": "bfloat16", **far},
        # A decode step of sixteen sequences: one token each, queries rotated, keys rotated into
        # their pages, values copied.
        {"name": "place_16x1", "op": "place", "batch": 16, "kv_heads": 8, "group": 4, "dim": 128,
         "part": 128, "interleaved": False, "page": 16, "tokens": 16, "held": 4000,
         "dtype": "float16", "head_major": False, **near},
        # The same for a batch of prompts of uneven lengths, cut from the qkv product.
        {"name": "place_prompts", "op": "place", "batch": 23, "kv_heads": 8, "group": 4,
         "dim": 128, "part": 128, "interleaved": False, "page": 16, "tokens": 32749,
         "held": 48, "dtype": "bfloat16", "head_major": False, **far},
        # Five drafted tokens checked at once behind a short conversation: latency.
        {"name": "chunk_1x5", "op": "chunk", "batch": 1, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "new": 5, "held": 700, "singles": 0, "ragged": False, "dtype": "float16",
         "head_major": False},
        # Uneven prompts without anything held before: the lower triangle alone.
        {"name": "chunk_prompts", "op": "chunk", "batch": 23, "kv_heads": 8, "group": 4,
         "dim": 128, "page": 16, "new": 1531, "held": 0, "singles": 0, "ragged": True,
         "dtype": "float16", "head_major": False},
        # A server's mixed step: most rows bring one token, some a piece of a prompt; seven query
        # heads to a key-value head, pages stored head by head.
        {"name": "chunk_mixed", "op": "chunk", "batch": 48, "kv_heads": 4, "group": 7, "dim": 128,
         "page": 32, "new": 509, "held": 8191, "singles": 40, "ragged": True, "dtype": "bfloat16",
         "head_major": True},
        # One piece of a very long document: the tensor cores' work.
        {"name": "chunk_1x2048", "op": "chunk", "batch": 1, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 64, "new": 2048, "held": 129023, "singles": 0, "ragged": False,
         "dtype": "bfloat16", "head_major": False},
        # One user's logits before sampling: penalties over a conversation, a few biases.
        {"name": "adjust_1", "op": "adjust", "rows": 1, "vocabulary": 128256, "history": 2000,
         "prompt": 0.6, "biases": 20, "masked": False, "dtype": "float16"},
        # A server's batch, every row with penalties of its own.
        {"name": "adjust_64", "op": "adjust", "rows": 64, "vocabulary": 128256, "history": 4093,
         "prompt": 0.5, "biases": 300, "masked": False, "dtype": "float32"},
        # A large batch under a grammar: most of the vocabulary is not allowed.
        {"name": "adjust_512_masked", "op": "adjust", "rows": 512, "vocabulary": 128256,
         "history": 8191, "prompt": 0.8, "biases": 8, "masked": True, "dtype": "bfloat16"},
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def _draw_rotation(rng: random.Random, dim: int) -> dict:
    scaling = rng.choice(("none", "linear", "base", "ramp"))
    return {"part": rng.choice((dim, dim, dim // 2, dim // 4)), "interleaved": rng.random() < 0.5,
            "base": rng.choice((10000.0, 500000.0, 1000000.0)), "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 7.5, 32.0)),
            "original": rng.choice((4096, 8192)) if scaling == "ramp" else 0,
            "magnitude": rng.choice((1.0, 1.2)) if scaling == "ramp" else 1.0}


def draw(rng: random.Random) -> dict:
    op = rng.choice(("rotate", "place", "chunk", "chunk", "adjust"))
    if op == "rotate":
        dim = rng.choice((64, 80, 96, 128, 256))
        return {"op": op, "tokens": _log_int(rng, 1, 16381), "dim": dim,
                "heads": _log_int(rng, 1, 40 * 128 // dim), "far": _log_int(rng, 1, 1000000),
                "dtype": rng.choice(("float16", "bfloat16", "float32")),
                **_draw_rotation(rng, dim)}
    if op == "place":
        tokens, dim = _log_int(rng, 1, 32749), rng.choice((64, 96, 128))
        kv_heads = rng.choice((1, 2, 4, 8))
        return {"op": op, "batch": _log_int(rng, 1, min(tokens, 64)), "kv_heads": kv_heads,
                "group": rng.choice([g for g in (1, 2, 4, 7, 8) if g * kv_heads <= 32]), "dim": dim,
                "page": rng.choice((1, 8, 13, 16, 32, 64)), "tokens": tokens,
                "held": _log_int(rng, 1, 8191 if tokens < 1000 else 64),
                "dtype": rng.choice(("float16", "bfloat16")),
                "head_major": rng.random() < 0.5, **_draw_rotation(rng, dim)}
    if op == "chunk":
        kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 96, 128, 256))
        group = rng.choice([g for g in (1, 2, 4, 7, 8, 16) if g * kv_heads <= 32])
        batch, held = _log_int(rng, 1, 48), rng.choice((0, 1))
        # keys and values of at most 2^30 values, at most a quarter of the longest case's products
        most = min(131071, (1 << 29) // (batch * kv_heads * dim))
        held = held and _log_int(rng, 1, most - 1)
        new = min(_log_int(rng, 1, 4096), most - held)
        cost = 4 * batch * new * (new + held) * kv_heads * group * dim
        new = max(1, min(new, int(new * 1.1e12 / cost)))
        return {"op": op, "batch": batch, "kv_heads": kv_heads, "group": group, "dim": dim,
                "page": rng.choice((1, 8, 13, 16, 32, 64, 128)), "new": new, "held": held,
                "singles": rng.choice((0, 0, batch // 2)), "ragged": rng.random() < 0.7,
                "dtype": rng.choice(("float16", "bfloat16")), "head_major": rng.random() < 0.5}
    vocabulary = _log_int(rng, 1000, 256000)
    return {"op": op, "rows": _log_int(rng, 1, min(512, 512 * 64000 // vocabulary)),
            "vocabulary": vocabulary, "history": _log_int(rng, 1, 8191),
            "prompt": rng.choice((0.0, 0.5, 1.0)), "biases": rng.choice((0, 1, 33, 300)),
            "masked": rng.random() < 0.5, "dtype": rng.choice(("float16", "bfloat16", "float32"))}


def _spread(n: int, longest: int, ragged: bool) -> list[int]:
    """n lengths, the same for every seed up to their order: 1/n, 2/n, ... of the longest."""
    if not ragged:
        return [longest] * n
    return [max(min(1, longest), longest * (i + 1) // n - (i * 7) % 5) for i in range(n)]


def _chunks(case: dict) -> list[tuple[int, int]]:
    """(held, new) tokens of each row."""
    n, singles = case["batch"], case["singles"]
    held = _spread(n, case["held"], case["ragged"])
    new = [1] * singles + _spread(n - singles, case["new"], case["ragged"])
    return [(held[i], new[(i * 7 + 3) % n if math.gcd(7, n) == 1 else i]) for i in range(n)]


def _counts(case: dict) -> list[int]:
    """New tokens of each sequence of an append, uneven, summing to case["tokens"]."""
    n, total = case["batch"], case["tokens"]
    weights = [1 + (i * 5) % 7 for i in range(n)]
    counts = [1 + (total - n) * w // sum(weights) for w in weights]
    counts[0] += total - sum(counts)
    return counts


def _rates(case: dict) -> list[float]:
    """Radians a position, of each pair of the rotated dimensions."""
    n, base, factor = case["part"], case["base"], case["factor"]
    if case["scaling"] == "base":
        base *= factor ** (n / (n - 2))
    rates = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":
        return [r / factor for r in rates]
    if case["scaling"] == "ramp":  # what turns often keeps its rate, what turns less than once does not
        keep = [min(1.0, max(0.0, (case["original"] * r / (2 * math.pi) - 1.0) / (4.0 - 1.0)))
                for r in rates]
        return [r * k + r / factor * (1.0 - k) for r, k in zip(rates, keep)]
    return rates


# ---------------------------------------------------------------------------
# What a program has in hand before the call
# ---------------------------------------------------------------------------
def _int32(values) -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _normal(g: torch.Generator, *shape, dtype) -> torch.Tensor:
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype)


def _rotation(case: dict) -> dict:
    """The rotation that a program sets up once for its model."""
    s = {"part": case["part"], "interleaved": case["interleaved"],
         "magnitude": case["magnitude"], "rates": None, "rotary": None}
    if own:
        import w4a16_weight_only_gemm_gb300 as w4
        scaling = None if case["scaling"] == "none" else case["scaling"]
        s["rotary"] = w4.Rotary(case["part"], base=case["base"], interleaved=case["interleaved"],
                                scaling=scaling, factor=case["factor"],
                                original=case["original"] or None, low=1.0, high=4.0,
                                magnitude=case["magnitude"], device=DEVICE)
    else:
        s["rates"] = torch.tensor(_rates(case), dtype=torch.float64, device=DEVICE)
    return s


def _scattered(rng: random.Random, pages_of: list[int], pool: int, width: int) -> list[list[int]]:
    """Page tables of rows that hold pages_of[b] pages each, taken from all over the pool."""
    order = rng.sample(range(pool), sum(pages_of))
    rows, at = [], 0
    for n in pages_of:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return rows


def _pool(g: torch.Generator, pages: int, case: dict) -> torch.Tensor:
    """[pages, page, kv_heads, dim], stored token by token or head by head."""
    t, h, d = case["page"], case["kv_heads"], case["dim"]
    if case["head_major"]:
        return _normal(g, pages, h, t, d, dtype=DTYPES[case["dtype"]]).transpose(1, 2)
    return _normal(g, pages, t, h, d, dtype=DTYPES[case["dtype"]])


def _prepare_rotate(case, rng, g):
    n = case["tokens"]
    # runs of positions, as packed sequences have them, that end somewhere up to `far`
    positions, run = [], -(-n // 5)
    for first in range(0, n, run):
        count = min(run, n - first)
        start = max(0, rng.randrange(case["far"] // 2, case["far"] + 1) - count)
        positions += range(start, start + count)
    x = _normal(g, n, case["heads"] + 8, case["dim"], dtype=DTYPES[case["dtype"]])
    # the query and key heads of a qkv product: the values lie behind them
    return {"x": x[:, :case["heads"]], "positions": _int32(positions), **_rotation(case)}


def _prepare_place(case, rng, g):
    page, h, d = case["page"], case["kv_heads"], case["dim"]
    heads = h * case["group"]
    # what each sequence holds already, the same for every seed up to the order
    news = [(case["held"] * (i * 11 % 17 + 1) // 17, n) for i, n in enumerate(_counts(case))]
    rng.shuffle(news)
    starts, counts = [s for s, _ in news], [n for _, n in news]
    pages_of = [-(-(s + n) // page) for s, n in zip(starts, counts)]
    pages = sum(pages_of) + 5
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    qkv = _normal(g, case["tokens"], heads + 2 * h, d, dtype=DTYPES[case["dtype"]])
    return {"q": qkv[:, :heads], "k": qkv[:, heads:heads + h], "v": qkv[:, heads + h:],
            "k_pool": _pool(g, pages, case), "v_pool": _pool(g, pages, case),
            "tables": _int32(_scattered(rng, pages_of, pages, max(pages_of))),
            "starts": _int32(starts), "offsets": _int32(offsets), **_rotation(case)}


def _prepare_chunk(case, rng, g):
    rows = _chunks(case)
    rng.shuffle(rows)
    lengths = [held + new for held, new in rows]
    pages_of = [-(-n // case["page"]) for n in lengths]
    pages = sum(pages_of) + 5
    offsets = [0]
    for _, new in rows:
        offsets.append(offsets[-1] + new)
    q_heads = case["kv_heads"] * case["group"]
    # queries as a norm and a rotation leave them: some heads attend sharply
    q = _normal(g, offsets[-1], q_heads, case["dim"], dtype=torch.float32)
    q = q * torch.rand(q_heads, 1, generator=g, device=DEVICE).mul_(2.0).add_(0.5)
    return {"q": q.to(DTYPES[case["dtype"]]), "k_pool": _pool(g, pages, case),
            "v_pool": _pool(g, pages, case), "rows": rows,
            "tables": _int32(_scattered(rng, pages_of, pages, max(pages_of))),
            "lengths": _int32(lengths), "offsets": _int32(offsets)}


def _prepare_adjust(case, rng, g):
    m, v, width = case["rows"], case["vocabulary"], case["history"]
    # logits of a trained model: a broad body and a few high ones
    x = _normal(g, m, v, dtype=torch.float32)
    x = x.mul_(2.5)
    at = torch.randint(0, v, (m, 8), generator=g, device=DEVICE)
    x.scatter_add_(1, at, torch.rand(m, 8, generator=g, device=DEVICE) * 12)
    # histories of uneven lengths; a few tokens come often, most seldom
    lengths = [max(1, width * (i + 1) // m) for i in range(m)]
    rng.shuffle(lengths)
    tokens = (torch.rand(m, width, generator=g, device=DEVICE, dtype=torch.float64) ** 3 * v).int()
    tokens = (tokens * 7919) % v
    prompts = [int(n * case["prompt"]) for n in lengths]
    s = {"logits": x.to(DTYPES[case["dtype"]]), "tokens": tokens, "lengths": _int32(lengths),
         "prompts": _int32(prompts),
         "repetition": torch.rand(m, generator=g, device=DEVICE) * 0.5 + 1.0,
         "presence": torch.rand(m, generator=g, device=DEVICE) * 2.0 - 0.5,
         "frequency": torch.rand(m, generator=g, device=DEVICE),
         "bias_ids": None, "biases": None, "mask": None}
    if case["biases"]:
        n = case["biases"]
        first = torch.randint(0, v - n + 1, (m, 1), generator=g, device=DEVICE)
        step = torch.randint(1, max(2, (v - 1) // n), (m, 1), generator=g, device=DEVICE)
        s["bias_ids"] = ((first + step * torch.arange(n, device=DEVICE)) % v).int()
        s["biases"] = torch.randn(m, n, generator=g, device=DEVICE) * 5.0
    if case["masked"]:
        # every thirtieth row is under no grammar, the others allow a twentieth of the tokens
        words = -(-v // 32)
        mask = torch.randint(-2 ** 31, 2 ** 31, (m, words), generator=g, device=DEVICE).int()
        mask *= (torch.rand(m, words, generator=g, device=DEVICE) < 0.1).int()
        mask[::30] = -1
        s["mask"] = mask
    return s


_PREPARE = {"rotate": _prepare_rotate, "place": _prepare_place, "chunk": _prepare_chunk,
            "adjust": _prepare_adjust}


def prepare(case: dict, seed: int) -> dict:
    rng = random.Random(seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    return {"op": case["op"], **_PREPARE[case["op"]](case, rng, g)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state: dict):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _own_rotate(s):
    import w4a16_weight_only_gemm_gb300 as w4
    return w4.rotate(s["x"], s["positions"], s["rotary"])


def _own_place(s):
    import w4a16_weight_only_gemm_gb300 as w4
    q = w4.paged_append_rotary(s["k"], s["v"], s["k_pool"], s["v_pool"], s["tables"], s["starts"],
                               s["rotary"], offsets=s["offsets"], q=s["q"])
    return q, s["k_pool"], s["v_pool"]


def _own_chunk(s):
    import w4a16_weight_only_gemm_gb300 as w4
    return w4.paged_chunk_attention(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lengths"],
                                    s["offsets"])


def _own_adjust(s):
    import w4a16_weight_only_gemm_gb300 as w4
    return w4.adjust_logits(s["logits"], s["tokens"], s["lengths"], s["prompts"],
                            repetition=s["repetition"], presence=s["presence"],
                            frequency=s["frequency"], bias_ids=s["bias_ids"], biases=s["biases"],
                            mask=s["mask"])


_OWN = {"rotate": _own_rotate, "place": _own_place, "chunk": _own_chunk, "adjust": _own_adjust}


def _rotate(x: torch.Tensor, positions: torch.Tensor, s: dict) -> torch.Tensor:
    """x [tokens, heads, dim] with its first dimensions rotated, angles in 64 bits."""
    angle = positions.double()[:, None] * s["rates"]
    c = (angle.cos() * s["magnitude"]).float()[:, None]
    z = (angle.sin() * s["magnitude"]).float()[:, None]
    n, f = s["part"], x.float()
    if s["interleaved"]:
        a, b = f[..., 0:n:2], f[..., 1:n:2]
        turned = torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2)
    else:
        a, b = f[..., :n // 2], f[..., n // 2:n]
        turned = torch.cat([a * c - b * z, a * z + b * c], -1)
    return torch.cat([turned, f[..., n:]], -1).to(x.dtype)


def _plain_rotate(s):
    return _rotate(s["x"], s["positions"], s)


def _plain_place(s):
    token = torch.arange(s["k"].shape[0], device=s["k"].device, dtype=torch.int32)
    row = torch.searchsorted(s["offsets"], token, right=True) - 1
    position = s["starts"][row] + token - s["offsets"][row]
    ps = s["k_pool"].shape[1]
    page = s["tables"][row, (position // ps).long()].long()
    s["k_pool"][page, (position % ps).long()] = _rotate(s["k"], position, s)
    s["v_pool"][page, (position % ps).long()] = s["v"]
    return _rotate(s["q"], position, s), s["k_pool"], s["v_pool"]


def _plain_chunk(s):
    kv, ps, d = s["k_pool"].shape[2], s["k_pool"].shape[1], s["q"].shape[2]
    group = s["q"].shape[1] // kv
    out, at = torch.empty_like(s["q"]), 0
    for b, (held, new) in enumerate(s["rows"]):
        pages = s["tables"][b, :-(-(held + new) // ps)].long()
        seen = torch.arange(held, held + new, device=out.device)[:, None]
        later = torch.arange(held + new, device=out.device) > seen
        for h in range(kv):
            k = s["k_pool"][pages, :, h].flatten(0, 1)[:held + new].float()
            v = s["v_pool"][pages, :, h].flatten(0, 1)[:held + new].float()
            q = s["q"][at:at + new, h * group:(h + 1) * group].float()
            x = (q.transpose(0, 1).flatten(0, 1) @ k.T).unflatten(0, (group, new))
            x = x.mul_(1.0 / math.sqrt(d)).masked_fill_(later, -math.inf)
            e = x.sub_(x.amax(-1, keepdim=True)).exp_()
            o = (e.flatten(0, 1) @ v).unflatten(0, (group, new)) / e.sum(-1, keepdim=True)
            out[at:at + new, h * group:(h + 1) * group] = o.transpose(0, 1).to(out.dtype)
        at += new
    return out


def _plain_adjust(s):
    x = s["logits"].float()
    tokens = s["tokens"].long()
    place = torch.arange(tokens.shape[1], device=x.device)
    held = place < s["lengths"][:, None]
    fresh = held & (place >= s["prompts"][:, None])
    seen = torch.zeros(x.shape, dtype=torch.int32, device=x.device)
    seen.scatter_add_(1, tokens, held.int())
    count = torch.zeros(x.shape, dtype=torch.int32, device=x.device)
    count.scatter_add_(1, tokens, fresh.int())
    r = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["biases"] is not None:
        x.scatter_add_(1, s["bias_ids"].long(), s["biases"])
    if s["mask"] is not None:
        bit = torch.arange(32, device=x.device, dtype=torch.int32)
        allowed = (s["mask"][:, :, None] >> bit & 1).flatten(1)[:, :x.shape[1]] > 0
        x = x.masked_fill(~allowed, -math.inf)
    return x.to(s["logits"].dtype)


_PLAIN = {"rotate": _plain_rotate, "place": _plain_place, "chunk": _plain_chunk,
          "adjust": _plain_adjust}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case: dict) -> dict:
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"],
                "flops": 3 * n * case["part"]}
    if case["op"] == "place":
        h, q = case["kv_heads"], case["kv_heads"] * case["group"]
        return {"bytes": 2 * case["tokens"] * (q + 2 * h) * case["dim"] * size + 12 * case["batch"],
                "flops": 3 * case["tokens"] * (q + h) * case["part"]}
    if case["op"] == "chunk":
        rows, heads = _chunks(case), case["kv_heads"] * case["group"]
        positions, tokens = sum(h + n for h, n in rows), sum(n for _, n in rows)
        pairs = sum(n * h + n * (n + 1) // 2 for h, n in rows)
        return {"bytes": 2 * positions * case["kv_heads"] * case["dim"] * size
                + 2 * tokens * heads * case["dim"] * size + 8 * case["batch"]
                + 4 * sum(-(-(h + n) // case["page"]) for h, n in rows),
                "flops": 4 * pairs * heads * case["dim"]}
    m, v = case["rows"], case["vocabulary"]
    history = sum(max(1, case["history"] * (i + 1) // m) for i in range(m))
    return {"bytes": 2 * m * v * size + 4 * history + 20 * m + 8 * m * case["biases"]
            + (4 * m * -(-v // 32) if case["masked"] else 0), "flops": m * v}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case: dict, seed: int):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_rotated(case, x, positions):
    """Each pair as a complex number, times one of the magnitude and the position's angle."""
    out, n = x.double(), case["part"]
    first = range(0, n, 2) if case["interleaved"] else range(n // 2)
    step = 1 if case["interleaved"] else n // 2
    p = positions.double()
    for i, rate in zip(first, _rates(case)):
        turn = torch.polar(torch.full_like(p, case["magnitude"]), p * rate)
        z = torch.complex(out[..., i], out[..., i + step]) * turn[:, None]
        out[..., i], out[..., i + step] = z.real, z.imag
    return out


def _exact_rotate(case, s):
    return _exact_rotated(case, s["x"], s["positions"])


def _exact_place(case, s):
    tables, offsets, starts = (s[n].tolist() for n in ("tables", "offsets", "starts"))
    ps, pages, slots, positions = case["page"], [], [], []
    for b, start in enumerate(starts):
        for p in range(start, start + offsets[b + 1] - offsets[b]):
            pages.append(tables[b][p // ps])
            slots.append(p % ps)
            positions.append(p)
    at = torch.tensor(pages, device=DEVICE), torch.tensor(slots, device=DEVICE)
    positions = torch.tensor(positions, device=DEVICE)
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    k_pool.index_put_(at, _exact_rotated(case, s["k"], positions))
    v_pool.index_put_(at, s["v"].double())
    return _exact_rotated(case, s["q"], positions), k_pool, v_pool


def _exact_chunk(case, s):
    ps, d, kv, group = case["page"], case["dim"], case["kv_heads"], case["group"]
    tables, offsets, lengths = (s[n].tolist() for n in ("tables", "offsets", "lengths"))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lengths):
        pages = torch.tensor(tables[b][:-(-n // ps)], device=DEVICE)
        first, last = offsets[b], offsets[b + 1]
        for h in range(kv):
            k, v = (s[x][:, :, h].index_select(0, pages).reshape(-1, d)[:n].double()
                    for x in ("k_pool", "v_pool"))
            for t in range(first, last, 256):  # some tokens at a time: scores of 64 bits are large
                e = min(last, t + 256)
                q = s["q"][t:e, h * group:(h + 1) * group].double()
                x = torch.einsum("tgd,pd->tgp", q, k) * d ** -0.5
                limit = torch.arange(n - last + t, n - last + e, device=DEVICE)[:, None, None]
                x = torch.where(torch.arange(n, device=DEVICE) <= limit, x, -math.inf)
                out[t:e, h * group:(h + 1) * group] = torch.softmax(x, -1) @ v
    return out


def _exact_adjust(case, s):
    x = s["logits"].double()
    m, v = x.shape
    lengths, prompts = s["lengths"].tolist(), s["prompts"].tolist()
    for r in range(m):
        said = s["tokens"][r, :lengths[r]].long()
        seen = torch.bincount(said, minlength=v) > 0
        count = torch.bincount(said[prompts[r]:], minlength=v).double()
        p = s["repetition"][r].double()
        x[r] = torch.where(seen & (x[r] > 0), x[r] / p, torch.where(seen, x[r] * p, x[r]))
        x[r] -= s["frequency"][r].double() * count + s["presence"][r].double() * count.clamp(max=1)
        if s["biases"] is not None:
            x[r].index_add_(0, s["bias_ids"][r].long(), s["biases"][r].double())
        if s["mask"] is not None:
            words = s["mask"][r].long() & 0xFFFFFFFF
            j = torch.arange(v, device=DEVICE)
            x[r][(words[j // 32] >> (j % 32)) % 2 == 0] = -math.inf
    return x


_EXACT = {"rotate": _exact_rotate, "place": _exact_place, "chunk": _exact_chunk,
          "adjust": _exact_adjust}
