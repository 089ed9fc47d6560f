"""Cases of the serving operators: the paged key-value cache, the attention of a
new token over it, the care of its pages, and the scores of sampled tokens.

Each case is one call that a decoding program makes between the quantized linear
layers.  ``run`` makes it in plain torch operations in 32 bits (``own`` false) or
through this package's entry points (``own`` true); ``exact`` has the same answer
in 64 bits.  Head counts, head size and vocabulary are those of
``workloads.py``: 32 query and 8 key-value heads of 128 (or 28 and 4), 32 layers,
a vocabulary of 128256.
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
    return [
        # One user's decode step after a 512-token prompt: latency alone.
        {"name": "attend_1x512", "op": "attend", "batch": 1, "kv_heads": 8, "group": 4, "dim": 128,
         "page": 16, "longest": 512, "ragged": False, "empty": 0, "dtype": "float16",
         "head_major": False},
        # A small server's batch: sequences of very different lengths, seven query heads to a
        # key-value head, bf16.
        {"name": "attend_16_ragged", "op": "attend", "batch": 16, "kv_heads": 4, "group": 7,
         "dim": 128, "page": 16, "longest": 4093, "ragged": True, "empty": 0, "dtype": "bfloat16",
         "head_major": False},
        # One very long document: the length has to be split over the whole GPU.
        {"name": "attend_1x131071", "op": "attend", "batch": 1, "kv_heads": 8, "group": 4,
         "dim": 128, "page": 64, "longest": 131071, "ragged": False, "empty": 0,
         "dtype": "float16", "head_major": False},
        # A full server's batch, slots without a sequence among it, pages stored head by head.
        {"name": "attend_128_ragged", "op": "attend", "batch": 128, "kv_heads": 8, "group": 4,
         "dim": 128, "page": 32, "longest": 8191, "ragged": True, "empty": 3, "dtype": "float16",
         "head_major": True},
        # A decode step's new keys and values: one token a sequence.
        {"name": "append_16x1", "op": "append", "batch": 16, "kv_heads": 8, "dim": 128, "page": 16,
         "tokens": 16, "dtype": "float16", "head_major": False},
        # The keys and values of a batch of prompts of uneven lengths, cut from the qkv product.
        {"name": "append_prompts", "op": "append", "batch": 24, "kv_heads": 8, "dim": 128,
         "page": 16, "tokens": 32749, "dtype": "float16", "head_major": False},
        # Best-of-four sampling: four branches of one prompt, the last round's branches dropped.
        {"name": "branch_4", "op": "branch", "parents": 1, "children": 4, "tokens": 509,
         "planes": 64, "page": 16, "page_values": 16384, "pages": 256, "dtype": "float16"},
        # Many branches at once over a pool of many pages.
        {"name": "branch_250", "op": "branch", "parents": 50, "children": 250, "tokens": 250,
         "planes": 64, "page": 16, "page_values": 16384, "pages": 2000, "dtype": "float16"},
        # A little pool drawn together after its users left.
        {"name": "compact_64", "op": "compact", "planes": 64, "page_values": 16384, "pages": 64,
         "used": 30, "moves": 13, "rows": 8, "dtype": "float16"},
        # A large pool, half of it free, drawn together before it shrinks.
        {"name": "compact_2000", "op": "compact", "planes": 64, "page_values": 16384,
         "pages": 2000, "used": 901, "moves": 473, "rows": 64, "dtype": "float16"},
        # The score of one sampled token with the twenty likeliest.
        {"name": "score_1", "op": "score", "rows": 1, "vocabulary": 128256, "top": 20,
         "dtype": "float16", "masked": 0},
        # The scores of a whole prompt's tokens, a part of the vocabulary masked.
        {"name": "score_2047", "op": "score", "rows": 2047, "vocabulary": 128256, "top": 5,
         "dtype": "float16", "masked": 1000},
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng: random.Random) -> dict:
    op = rng.choice(("attend", "attend", "append", "branch", "compact", "score"))
    if op == "attend":
        kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 96, 128, 256))
        batch = _log_int(rng, 1, 128)
        most = 128 * 8191 * 8 * 128 // (batch * kv_heads * dim)
        return {"op": op, "batch": batch, "kv_heads": kv_heads, "group": rng.choice((1, 2, 4, 7, 8, 16)),
                "dim": dim, "page": rng.choice((1, 8, 13, 16, 32, 64, 128)),
                "longest": _log_int(rng, 1, min(131071, most)), "ragged": rng.random() < 0.7,
                "empty": rng.choice((0, 0, 1)) if batch > 1 else 0,
                "dtype": rng.choice(("float16", "bfloat16")), "head_major": rng.random() < 0.5}
    if op == "append":
        tokens = _log_int(rng, 1, 32749)
        return {"op": op, "batch": _log_int(rng, 1, min(tokens, 64)), "kv_heads": rng.choice((1, 2, 4, 8)),
                "dim": rng.choice((64, 96, 128)), "page": rng.choice((1, 8, 13, 16, 32, 64)),
                "tokens": tokens, "dtype": rng.choice(("float16", "bfloat16")),
                "head_major": rng.random() < 0.5}
    if op == "branch":
        parents = _log_int(rng, 1, 50)
        children = max(parents, _log_int(rng, 1, 250))
        page = rng.choice((8, 16, 32))
        tokens = _log_int(rng, 1, 250)
        # the pool: parents' pages, a last page each for old and new branches, some spare
        pages = parents * (-(-tokens // page)) + 2 * children + _log_int(rng, 1, 300)
        return {"op": op, "parents": parents, "children": children, "tokens": tokens,
                "planes": rng.choice((2, 8, 56, 64)), "page": page,
                "page_values": page * rng.choice((512, 1024)) // (2 if page == 32 else 1),
                "pages": pages, "dtype": rng.choice(("float16", "bfloat16"))}
    if op == "compact":
        pages = _log_int(rng, 16, 2000)
        used = rng.randrange(max(1, pages // 4), pages // 2 + 1)
        return {"op": op, "planes": rng.choice((2, 8, 56, 64)),
                "page_values": rng.choice((2048, 4096, 8192, 16384)), "pages": pages, "used": used,
                "moves": rng.randrange(0, used + 1), "rows": _log_int(rng, 1, 64),
                "dtype": rng.choice(("float16", "bfloat16"))}
    vocabulary = _log_int(rng, 1000, 256000)
    return {"op": op, "rows": _log_int(rng, 1, min(2047, 2047 * 64000 // vocabulary)),
            "vocabulary": vocabulary, "top": rng.choice((1, 3, 5, 10, 20, 32)),
            "dtype": rng.choice(("float16", "bfloat16", "float32")),
            "masked": rng.choice((0, vocabulary // 3))}


def _lengths(case: dict) -> list[int]:
    """The sequences' lengths, the same for every seed up to their order."""
    n, longest = case["batch"], case["longest"]
    if not case["ragged"]:
        lengths = [longest] * n
    else:  # evenly spread from short to long: 1/n, 2/n, ... of the longest, off the round sizes
        lengths = [max(1, longest * (i + 1) // n - (i * 7) % 5) for i in range(n)]
    for i in range(case["empty"]):
        lengths[i * n // max(1, case["empty"])] = 0
    return lengths


def _counts(case: dict) -> list[int]:
    """New tokens of each sequence of an append, uneven, summing to case["tokens"]."""
    n, total = case["batch"], case["tokens"]
    weights = [1 + (i * 5) % 7 for i in range(n)]
    counts = [1 + (total - n) * w // sum(weights) for w in weights]
    counts[0] += total - sum(counts)
    return counts


# ---------------------------------------------------------------------------
# What a program has in hand before the call
# ---------------------------------------------------------------------------
def _int32(values) -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _normal(g: torch.Generator, *shape, dtype) -> torch.Tensor:
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype)


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


def _prepare_attend(case, rng, g):
    lengths = _lengths(case)
    rng.shuffle(lengths)
    pages_of = [-(-n // case["page"]) for n in lengths]
    width = max(1, max(pages_of))
    pages = sum(pages_of) + 5
    dtype = DTYPES[case["dtype"]]
    q_heads = case["kv_heads"] * case["group"]
    # queries as a norm and a rotation leave them: some heads attend sharply
    q = _normal(g, case["batch"], q_heads, case["dim"], dtype=torch.float32)
    q = q * torch.rand(q_heads, 1, generator=g, device=DEVICE).mul_(2.0).add_(0.5)
    return {"q": q.to(dtype), "k_pool": _pool(g, pages, case), "v_pool": _pool(g, pages, case),
            "tables": _int32(_scattered(rng, pages_of, pages, width)), "lengths": _int32(lengths)}


def _prepare_append(case, rng, g):
    page = case["page"]
    # what each sequence holds already: up to three pages, the same for every seed up to the order
    news = [(i * 11 % (3 * page), n) for i, n in enumerate(_counts(case))]
    rng.shuffle(news)
    starts, counts = [s for s, _ in news], [n for _, n in news]
    pages_of = [-(-(s + n) // page) for s, n in zip(starts, counts)]
    pages = sum(pages_of) + 5
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    # keys and values as the qkv product leaves them: columns behind the queries'
    h, d = case["kv_heads"], case["dim"]
    qkv = _normal(g, case["tokens"], 6 * h * d, dtype=DTYPES[case["dtype"]])
    return {"k": qkv[:, 4 * h * d:5 * h * d].unflatten(1, (h, d)),
            "v": qkv[:, 5 * h * d:].unflatten(1, (h, d)),
            "k_pool": _pool(g, pages, case), "v_pool": _pool(g, pages, case),
            "tables": _int32(_scattered(rng, pages_of, pages, max(pages_of))),
            "starts": _int32(starts), "offsets": _int32(offsets)}


def _prepare_branch(case, rng, g):
    """Slots: the parents, then the last round's branches (dropped now), then empty ones for
    the new branches.  Old branches share their parent's full pages and own a last page."""
    page, n, m = case["page"], case["parents"], case["children"]
    # parents differ in length a little; at least one page position is partly filled in most
    lengths = [max(1, case["tokens"] - i % 3) for i in range(n)]
    pages_of = [-(-t // page) for t in lengths]
    width = max(pages_of) + 1
    order = rng.sample(range(case["pages"]), sum(pages_of) + m)
    spare = iter(order[sum(pages_of):])
    tables, refs, at = [], [0] * case["pages"], 0
    for k in pages_of:
        tables.append(order[at:at + k] + [-1] * (width - k))
        at += k
        for p in tables[-1][:k]:
            refs[p] += 1
    old = [i % n for i in range(m)]
    for p in old:
        full = lengths[p] // page
        row = tables[p][:full]
        for x in row:
            refs[x] += 1
        if lengths[p] % page:
            row = row + [next(spare)]
            refs[row[-1]] += 1
        tables.append(row + [-1] * (width - len(row)))
        lengths.append(lengths[p])
    tables += [[-1] * width] * m
    lengths += [0] * m
    parents = [i % n for i in range(m)]
    rng.shuffle(parents)
    return {"pool": _normal(g, case["planes"], case["pages"], case["page_values"],
                            dtype=DTYPES[case["dtype"]]),
            "refs": _int32(refs), "tables": _int32(tables), "lengths": _int32(lengths),
            "drop": _int32(list(range(n, n + m))), "parents": _int32(parents),
            "children": _int32(list(range(n + m, n + 2 * m))), "page": page}


def _prepare_compact(case, rng, g):
    pages, used = case["pages"], case["used"]
    moves = min(case["moves"], pages - used)
    low = rng.sample(range(used), used - moves)
    high = rng.sample(range(used, pages), moves)
    held = low + high
    rng.shuffle(held)
    # the first row's first page is shared by every row, as a common prompt's is
    per = -(-(used - 1) // case["rows"])
    rows = [held[:1] + held[1 + i * per:1 + (i + 1) * per] for i in range(case["rows"])]
    refs = [0] * pages
    for r in rows:
        for p in r:
            refs[p] += 1
    return {"pool": _normal(g, case["planes"], pages, case["page_values"],
                            dtype=DTYPES[case["dtype"]]),
            "refs": _int32(refs), "tables": _int32([r + [-1] * (per + 3 - len(r)) for r in rows])}


def _prepare_score(case, rng, g):
    m, v = case["rows"], case["vocabulary"]
    # logits of a trained model: a broad body and a few high ones
    x = _normal(g, m, v, dtype=torch.float32)
    x = x.mul_(2.5)
    at = torch.randint(0, v, (m, 8), generator=g, device=DEVICE)
    x.scatter_add_(1, at, torch.rand(m, 8, generator=g, device=DEVICE) * 12)
    x = x.to(DTYPES[case["dtype"]])
    if case["masked"]:
        first = rng.randrange(0, v - case["masked"])
        x[:, first:first + case["masked"]] = -math.inf
    # most sampled tokens are among the likely ones, and none is masked
    tokens = torch.where(torch.rand(m, generator=g, device=DEVICE) < 0.7, x.argmax(1),
                         torch.randint(0, v, (m,), generator=g, device=DEVICE))
    if case["masked"]:
        inside = (tokens >= first) & (tokens < first + case["masked"])
        tokens = torch.where(inside, x.argmax(1), tokens)
    return {"logits": x, "tokens": tokens, "top": case["top"]}


_PREPARE = {"attend": _prepare_attend, "append": _prepare_append, "branch": _prepare_branch,
            "compact": _prepare_compact, "score": _prepare_score}


def prepare(case: dict, seed: int) -> dict:
    rng = random.Random(seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    return {"op": case["op"], **_PREPARE[case["op"]](case, rng, g)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state: dict):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _own_attend(s):
    import w4a16_weight_only_gemm_gb300 as w4
    return w4.paged_attention(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lengths"])


def _own_append(s):
    import w4a16_weight_only_gemm_gb300 as w4
    w4.paged_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["tables"], s["starts"],
                    s["offsets"])
    return s["k_pool"], s["v_pool"]


def _own_branch(s):
    import w4a16_weight_only_gemm_gb300 as w4
    refs, tables, lengths = w4.pages_free(s["refs"], s["tables"], s["lengths"], s["drop"])
    refs, tables, lengths, done = w4.pages_fork(s["pool"], refs, tables, lengths, s["parents"],
                                                s["children"], s["page"])
    return refs, tables, lengths, done, s["pool"]


def _own_compact(s):
    import w4a16_weight_only_gemm_gb300 as w4
    refs, tables, used = w4.pages_compact(s["pool"], s["refs"], s["tables"])
    return refs, tables, used, s["pool"]


def _own_score(s):
    import w4a16_weight_only_gemm_gb300 as w4
    return w4.token_logprobs(s["logits"], s["tokens"], top=s["top"])


_OWN = {"attend": _own_attend, "append": _own_append, "branch": _own_branch,
        "compact": _own_compact, "score": _own_score}


def _plain_attend(s):
    q, tables, lengths = s["q"], s["tables"], s["lengths"]
    b, heads, d = q.shape
    kv = s["k_pool"].shape[2]
    at = tables.clamp(min=0).long()
    k = s["k_pool"][at].flatten(1, 2).float()  # [b, positions, kv, d]
    v = s["v_pool"][at].flatten(1, 2).float()
    x = torch.einsum("bhgd,bthd->bhgt", q.float().view(b, kv, heads // kv, d), k) / math.sqrt(d)
    there = torch.arange(k.shape[1], device=q.device) < lengths[:, None]
    x = x.masked_fill(~there[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - top)
    o = torch.einsum("bhgt,bthd->bhgd", e, v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(b, heads, d).to(q.dtype)


def _plain_append(s):
    token = torch.arange(s["k"].shape[0], device=s["k"].device, dtype=torch.int32)
    row = torch.searchsorted(s["offsets"], token, right=True) - 1
    position = s["starts"][row] + token - s["offsets"][row]
    ps = s["k_pool"].shape[1]
    page = s["tables"][row, (position // ps).long()].long()
    s["k_pool"][page, (position % ps).long()] = s["k"]
    s["v_pool"][page, (position % ps).long()] = s["v"]
    return s["k_pool"], s["v_pool"]


def _plain_branch(s):
    page, width = s["page"], s["tables"].shape[1]
    refs, tables, lengths = s["refs"].clone(), s["tables"].clone(), s["lengths"].clone()
    drop, parents, children = s["drop"].long(), s["parents"].long(), s["children"].long()
    # free: one holder fewer of each page of the dropped rows
    rows = tables[drop]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).int().flatten())
    tables[drop] = -1
    lengths[drop] = 0
    # fork: full pages are shared, a partly filled last page is copied to the lowest free one
    length = lengths[parents]
    full, part = length // page, (length % page > 0).int()
    free = torch.argsort((refs > 0).int(), stable=True).int()
    nth = part.cumsum(0)
    done = (nth <= (refs == 0).sum()).int()
    fresh = free[(nth - 1).clamp(0, refs.numel() - 1)]
    column = torch.arange(width, device=refs.device)
    rows = tables[parents]
    shared = (column < full[:, None]) & (done > 0)[:, None]
    copied = (column == full[:, None]) & ((part > 0) & (done > 0))[:, None]
    tables[children] = torch.where(shared, rows, torch.where(copied, fresh[:, None], -1))
    lengths[children] = torch.where(done > 0, length, 0)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), shared.int().flatten())
    chosen = copied.any(1)
    source = rows.gather(1, full.clamp(max=width - 1)[:, None].long())[:, 0][chosen].long()
    target = fresh[chosen].long()
    refs[target] = 1
    s["pool"][:, target] = s["pool"][:, source]
    return refs, tables, lengths, done, s["pool"]


def _plain_compact(s):
    refs, tables = s["refs"], s["tables"]
    held = refs > 0
    used = held.sum().int().view(1)
    page = torch.arange(refs.numel(), device=refs.device)
    holes = page[~held & (page < used)]
    movers = page[held & (page >= used)]
    to = page.int()
    to[movers] = holes.int()
    s["pool"][:, holes] = s["pool"][:, movers]
    new_refs = refs.clone()
    new_refs[holes] = refs[movers]
    new_refs[movers] = 0
    new_tables = torch.where(tables >= 0, to[tables.clamp(min=0).long()], tables)
    return new_refs, new_tables, used, s["pool"]


def _ordered(x: torch.Tensor) -> torch.Tensor:
    """fp32 values as integers of the same order, -0 equal to 0."""
    bits = (x + 0.0).view(torch.int32)
    return bits ^ ((bits >> 31) & 0x7FFFFFFF)


def _plain_score(s):
    x, tokens = s["logits"].float(), s["tokens"].long()
    m, v = x.shape
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total)
    logprob = d.gather(1, tokens[:, None])[:, 0] - lse[:, 0]
    entropy = lse[:, 0] - (torch.where(e > 0, d, 0.0) * e).sum(1) / total[:, 0]
    # the likeliest, of equal ones the lowest index: one integer that holds both
    key = _ordered(x).long() * (1 << 20) + ((1 << 20) - 1 - torch.arange(v, device=x.device))
    best = key.topk(s["top"], dim=1).values
    ids = ((1 << 20) - 1 - (best & ((1 << 20) - 1)))
    return logprob, entropy, ids.int(), d.gather(1, ids) - lse


_PLAIN = {"attend": _plain_attend, "append": _plain_append, "branch": _plain_branch,
          "compact": _plain_compact, "score": _plain_score}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case: dict) -> dict:
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "attend":
        tokens, heads = sum(_lengths(case)), case["kv_heads"] * case["group"]
        per = case["kv_heads"] * case["dim"] * size
        pages = sum(-(-n // case["page"]) for n in _lengths(case))
        return {"bytes": 2 * tokens * per + 2 * case["batch"] * heads * case["dim"] * size
                + 4 * pages + 4 * case["batch"], "flops": 4 * tokens * heads * case["dim"]}
    if case["op"] == "append":
        return {"bytes": 4 * case["tokens"] * case["kv_heads"] * case["dim"] * size
                + 12 * case["batch"], "flops": 0}
    if case["op"] == "branch":
        n, page = case["parents"], case["page"]
        lengths = [max(1, case["tokens"] - i % 3) for i in range(n)]
        copies = sum(1 for i in range(case["children"]) if lengths[i % n] % page)
        width = max(-(-t // page) for t in lengths) + 1
        rows = n + 2 * case["children"]
        return {"bytes": 2 * copies * case["planes"] * case["page_values"] * size
                + 8 * case["pages"] + 8 * rows * (width + 1) + 16 * case["children"], "flops": 0}
    if case["op"] == "compact":
        moves = min(case["moves"], case["pages"] - case["used"])
        per = -(-(case["used"] - 1) // case["rows"]) + 3
        return {"bytes": 2 * moves * case["planes"] * case["page_values"] * size
                + 8 * case["pages"] + 8 * case["rows"] * per, "flops": 0}
    return {"bytes": case["rows"] * (case["vocabulary"] * size + 16 + 8 * case["top"]),
            "flops": 5 * case["rows"] * case["vocabulary"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case: dict, seed: int):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_attend(s):
    q, lengths, tables = s["q"].double(), s["lengths"].tolist(), s["tables"].tolist()
    kv, ps = s["k_pool"].shape[2], s["k_pool"].shape[1]
    group, d = q.shape[1] // kv, q.shape[2]
    out = torch.zeros_like(q)
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        pages = torch.tensor(tables[b][:-(-n // ps)], device=q.device)
        k = s["k_pool"].index_select(0, pages).double().reshape(-1, kv, d)[:n]
        v = s["v_pool"].index_select(0, pages).double().reshape(-1, kv, d)[:n]
        for h in range(kv):
            x = q[b, h * group:(h + 1) * group] @ k[:, h].T * d ** -0.5
            p = torch.softmax(x, -1)
            out[b, h * group:(h + 1) * group] = p @ v[:, h]
    return out


def _exact_append(s):
    k_pool, v_pool, tables = s["k_pool"].clone(), s["v_pool"].clone(), s["tables"].tolist()
    offsets, ps = s["offsets"].tolist(), k_pool.shape[1]
    pages, slots = [], []
    for b, start in enumerate(s["starts"].tolist()):
        for p in range(start, start + offsets[b + 1] - offsets[b]):
            pages.append(tables[b][p // ps])
            slots.append(p % ps)
    pages, slots = (torch.tensor(t, device=k_pool.device) for t in (pages, slots))
    k_pool.index_put_((pages, slots), s["k"])
    v_pool.index_put_((pages, slots), s["v"])
    return k_pool, v_pool


def _exact_branch(s):
    page, pool = s["page"], s["pool"]
    refs, tables, lengths = s["refs"].tolist(), s["tables"].tolist(), s["lengths"].tolist()
    for r in s["drop"].tolist():
        for p in tables[r]:
            if p >= 0:
                refs[p] -= 1
        tables[r], lengths[r] = [-1] * len(tables[r]), 0
    free = [p for p, n in enumerate(refs) if n == 0]
    done, wanted, copies = [], 0, []
    for parent, child in zip(s["parents"].tolist(), s["children"].tolist()):
        full, part = divmod(lengths[parent], page)
        wanted += part > 0
        done.append(int(wanted <= len(free)))
        if not done[-1]:
            continue
        row = tables[parent][:full]
        for p in row:
            refs[p] += 1
        if part:
            copies.append((tables[parent][full], free[wanted - 1]))
            row = row + [free[wanted - 1]]
            refs[row[-1]] = 1
        tables[child] = row + [-1] * (len(tables[child]) - len(row))
        lengths[child] = lengths[parent]
    for source, target in copies:
        pool[:, target].copy_(pool[:, source])
    return [_int32(t) for t in (refs, tables, lengths, done)] + [pool]


def _exact_compact(s):
    refs, tables, pool = s["refs"].tolist(), s["tables"].tolist(), s["pool"]
    used = sum(n > 0 for n in refs)
    holes = iter([p for p in range(used) if refs[p] == 0])
    to = {}
    for p in range(used, len(refs)):
        if refs[p] > 0:
            to[p] = next(holes)
            refs[to[p]], refs[p] = refs[p], 0
            pool[:, to[p]].copy_(pool[:, p])
    tables = [[to.get(p, p) for p in row] for row in tables]
    return [_int32(refs), _int32(tables), _int32([used]), pool]


def _exact_score(s):
    x = s["logits"].double()
    lse = torch.logsumexp(x, 1, keepdim=True)
    logp = x - lse
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    return (logp.gather(1, s["tokens"][:, None])[:, 0], entropy, ids.int(), logp.gather(1, ids))


_EXACT = {"attend": _exact_attend, "append": _exact_append, "branch": _exact_branch,
          "compact": _exact_compact, "score": _exact_score}
