"""Attention of chunks of new tokens over the paged cache, against the 64-bit
definition: types, head layouts, page sizes, chunks and lengths from none to many
tiles, strides, pages that are not there, and garbage wherever a token may not look.

Tolerance, from the arithmetic: products of 16-bit values are exact in FP32 and
summed there, with 2 bits to spare for a tensor core's truncation, so a score is
off by at most E = dim * 2^-22 * sum |q k| scale (+ 2^-20 for the exponential); a
softmax average of V then moves by at most 4 E max|V|.  Each weight enters the
product with V rounded by u (2^-11 for fp16, 2^-8 for bf16) of itself, so the average
by u times that of |V|, and the output is rounded once, by u |out|.  In fp16 a weight
below 2^-36 of the largest may count as 0: n 2^-36 max|V| for n positions."""
from __future__ import annotations

import math

import pytest
import torch

import prompt_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

gpu = pytest.mark.gpu
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def queries(offsets, heads, dim, dtype, seed=0, scale=1.5):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(int(offsets[-1]), heads, dim, generator=g) * scale).to(dtype).cuda()


def near(out, lse, want, want_lse, bound, mass, v_pool, positions, dim):
    if out.numel() == 0:
        return
    u = UNIT[out.dtype]
    error = dim * 2.0 ** -22 * bound + 2.0 ** -20
    v = torch.nan_to_num(v_pool.cpu().double(), 0, 0, 0).abs().max()
    far = (out.cpu().double() - want).abs() - u * (want.abs() + (1 + u) * mass) \
        - 4 * error[..., None] * v - positions * 2.0 ** -36 * v
    assert torch.isfinite(out).all()
    assert far.max() <= 2.0 ** -24, f"off by {far.max():.3g} beyond the bound"
    held = want_lse > -math.inf
    assert torch.equal(lse.cpu() > -math.inf, held)
    off = (lse.cpu().double() - want_lse)[held].abs()
    assert (off <= error[held] + 2.0 ** -20 * (1 + want_lse[held].abs())).all()
    assert (out.cpu()[~held] == 0).all()


def check(q, k_pool, v_pool, tables, lengths, offsets, scale=None, **kw):
    out, lse = w4.paged_chunk_attention(q, k_pool, v_pool, tables, lengths, offsets, scale=scale,
                                        return_lse=True, **kw)
    torch.cuda.synchronize()
    assert w4.device_status() == 0
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want = ref.chunk_attention(q, k_pool, v_pool, tables, lengths, offsets, scale)
    near(out, lse, *want, v_pool, tables.shape[1] * k_pool.shape[1], q.shape[2])
    return out


def make(rows, kv_heads, group, dim, page, dtype, **kw):
    parts = ref.cache(rows, kv_heads, dim, page, dtype, **kw)
    return queries(parts[-1], kv_heads * group, dim, dtype, kw.get("seed", 0)), *parts


# (positions held, new tokens): none, one, tiles' edges and past them, long and short
ROWS = [(0, 1), (0, 0), (5, 3), (0, 130), (127, 1), (128, 129), (300, 64), (700, 17), (0, 257),
        (63, 2), (64, 0), (255, 1), (256, 2), (0, 64), (1, 31)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv_heads, group, dim", [(8, 4, 128), (4, 7, 128), (1, 1, 64), (2, 8, 64),
                                                  (2, 16, 128), (1, 32, 128), (3, 5, 96),
                                                  (1, 12, 256), (2, 2, 256), (1, 71, 64),
                                                  (5, 3, 8), (1, 9, 136), (1, 300, 64)])
def test_heads_and_sizes(w4lib, kv_heads, group, dim, dtype):
    rows = ROWS if group < 30 else ROWS[:7]
    check(*make(rows, kv_heads, group, dim, 16, dtype, seed=dim + group))


@gpu
@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 3, 8, 13, 16, 24, 32, 48, 64, 128, 256])
def test_pages_and_layouts(w4lib, page, layout):
    check(*make(ROWS, 2, 4, 128, page, torch.float16, layout=layout, seed=page))


@gpu
@pytest.mark.parametrize("rows", [[(0, 1)], [(0, 128)], [(0, 129)], [(0, 1000)], [(4096, 5)],
                                  [(20011, 3)], [(9000, 300)], [(3, 20), (20011, 1), (0, 0), (0, 70)],
                                  [(0, 0), (0, 0)], [(5000, 1)] * 40,
                                  [(i * 3, i % 5) for i in range(150)], [(63, 1)] * 700],
                         ids=lambda rows: f"{len(rows)}x{rows[-1]}")
@pytest.mark.parametrize("kv_heads, group", [(8, 4), (1, 7)])
def test_lengths(w4lib, rows, kv_heads, group):
    if kv_heads == 8 and rows[0] == (9000, 300):
        kv_heads = 2                             # the definition takes its time
    check(*make(rows, kv_heads, group, 64, 16, torch.float16, seed=len(rows)))


@gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tables_much_wider_than_the_rows(w4lib, dim):
    check(*make(ROWS, 2, 4, dim, 16, torch.bfloat16, seed=dim, width=4000))


@gpu
@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
def test_garbage_where_no_row_is(w4lib, garbage):
    check(*make(ROWS, 2, 4, 128, 32, torch.float16, garbage=garbage))


# a row of two tiles and one of one; the first among many others, so that no item is cut; rows of
# one tile, whose steps two groups of warps share
SPOILT = {"cut": [(40, 150), (100, 100)], "whole": [(40, 150)] + [(0, 260)] * 90,
          "one tile": [(40, 20), (700, 9)]}


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", SPOILT)
@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
def test_garbage_that_only_later_tokens_see(w4lib, garbage, rows, dim, dtype):
    """A key or a value that is not finite spoils the tokens that see it, and no other."""
    rows = SPOILT[rows]
    args = make(rows, 2, 4, dim, 16, dtype, garbage=0.0, seed=3)
    q, k, v, tables, lengths, offsets = args
    plain, held, new = w4.paged_chunk_attention(*args), *rows[0]
    for pool, at in ((k, held + new // 3), (v, held + new // 3), (v, held + new - 2)):
        spoilt = pool.clone()
        page, slot = int(tables[0, at // 16]), at % 16
        spoilt[page, slot, 1, 3] = garbage
        pools = (spoilt, v) if pool is k else (k, spoilt)
        out, lse = w4.paged_chunk_attention(q, *pools, tables, lengths, offsets, return_lse=True)
        seeing = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        seeing[at - held:new, 4:] = True
        assert torch.equal(out[~seeing], plain[~seeing])
        if pool is v:                            # one dimension of V, of all tokens that see it
            assert not torch.isfinite(out[seeing][:, 3]).any()
            assert torch.equal(out[..., :3], plain[..., :3])
            assert torch.equal(out[..., 4:], plain[..., 4:])
        elif math.isnan(garbage):
            assert torch.isnan(out[seeing]).all() and torch.isnan(lse[seeing]).all()
        else:                                    # a score of either infinity, by the query's sign
            up = (q[..., 3] > 0) == (garbage > 0)
            assert torch.isnan(out[seeing & up]).all()
            assert torch.isfinite(out[seeing & ~up]).all()


@gpu
def test_values_that_all_tokens_see(w4lib):
    """Not finite before the chunk: every token's dimension, and only that."""
    args = make([(300, 20)], 1, 4, 128, 16, torch.float16, garbage=0.0, seed=4)
    q, k, v, tables, lengths, offsets = args
    plain = w4.paged_chunk_attention(*args)
    v[int(tables[0, 7]), 2, 0, 9] = math.inf
    out = w4.paged_chunk_attention(*args)
    assert not torch.isfinite(out[..., 9]).any()
    out[..., 9] = plain[..., 9]
    assert torch.equal(out, plain)


@gpu
@pytest.mark.parametrize("page", [8, 13, 16, 64])
def test_pages_that_are_not_there(w4lib, page):
    q, k, v, tables, lengths, offsets = make([(300, 100), (200, 100), (0, 200)], 2, 4, 128, page,
                                             torch.float16, seed=3)
    tables[0, 1] = -1
    tables[0, 2] = k.shape[0]                  # one past the pool
    tables[0, 3] = 2 ** 31 - 1
    tables[0, -1] = -1                         # the last tokens' own page
    tables[1, :] = -7                          # a row with no page at all
    tables[2, 0] = -1                          # the first tokens have nothing left to see
    check(q, k, v, tables, lengths, offsets)


@gpu
def test_lengths_out_of_range(w4lib):
    """Rows with more tokens than positions, below 0, and past the table."""
    q, k, v, tables, _, _ = make([(28, 20), (28, 20), (28, 20), (0, 48)], 2, 4, 64, 16,
                                 torch.float16, seed=6, garbage=0.0)
    q = q[:68]
    check(q, k, v, tables, ints([5, -5, 1 << 30, 48]), ints([0, 20, 40, 60, 68]))
    check(q, k, v, tables, ints([0, 0, 0, 0]), ints([0, 20, 40, 60, 68]))


@gpu
@pytest.mark.parametrize("dim", [64, 128])
def test_tokens_of_no_row(w4lib, dim):
    """Before the first row and behind the last, whatever lies there; the rest as without them."""
    args = make([(10, 30), (0, 0), (140, 7)], 2, 4, dim, 16, torch.bfloat16, seed=7)
    plain = check(*args)
    q = torch.full((50, 8, dim), math.nan, device="cuda").bfloat16()
    q[6:43] = args[0]
    out = torch.full((50, 8, dim), 7.0, device="cuda").bfloat16()
    got, lse = w4.paged_chunk_attention(q, *args[1:5], args[5] + 6, out=out, return_lse=True)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out[6:43], plain)
    for t in (out[:6], out[43:]):
        assert (t == 0).all()
    assert (lse[:6] == -math.inf).all() and (lse[43:] == -math.inf).all()
    none = w4.paged_chunk_attention(q, *args[1:5], torch.zeros_like(args[5]))
    assert (none == 0).all()
    assert w4.paged_chunk_attention(q[:0], *args[1:5], torch.zeros_like(args[5])).shape == (0, 8, dim)


@gpu
def test_large_scores_and_scale(w4lib):
    """Scores of some hundreds, where the running maximum has to carry the sum."""
    q, *rest = make([(600, 100), (0, 333)], 2, 4, 128, 16, torch.float16, seed=5, garbage=0.)
    rest[0] *= 4
    check(q * 8, *rest)
    check(q, *rest, scale=0.0)
    check(q, *rest, scale=-0.25)


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rising", [True, False])
def test_ordered_scores(w4lib, rising, dtype):
    """The maximum found last, or first."""
    q, k, v, tables, lengths, offsets = make([(1400, 100)], 1, 2, 64, 16, dtype, seed=7, garbage=0.)
    q.fill_(0.5)
    at = torch.arange(1500, device="cuda") / 50.0
    at = at if rising else at.flip(0)
    for p in range(0, 1500, 16):
        n = min(16, 1500 - p)
        k[tables[0, p // 16], :n, 0] = at[p:p + n, None].to(dtype)
    check(q, k, v, tables, lengths, offsets)


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_small_weights_beside_a_large_one(w4lib, dtype):
    """A position that draws nearly all attention, and many whose weights are 1.5 * 2^-24 of it."""
    n = 100_000
    q, k, v, tables, lengths, offsets = make([(n - 1, 1)], 1, 2, 64, 16, dtype, garbage=0.0)
    q.zero_()
    q[:, :, 0] = 1.0
    k.zero_()
    v.fill_(1.0)
    page = int(tables[0, 0])
    k[page, 3, 0, 0] = math.log(2.0 ** 24 / 1.5)
    v[page, 3] = 0.0
    check(q, k, v, tables, lengths, offsets, scale=1.0)


@gpu
def test_strided_query_and_output(w4lib):
    q, *rest = make(ROWS, 4, 7, 128, 16, torch.bfloat16, seed=8)
    plain = check(q, *rest)
    n = q.shape[0]
    wide = torch.randn(n, 36, 128, device="cuda").bfloat16()
    wide[:, :28] = q
    out = torch.full((n, 40, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    got = w4.paged_chunk_attention(wide[:, :28], *rest, out=out[:, 4:32])
    assert torch.equal(got, plain) and torch.equal(out[:, 4:32], plain)
    assert (out[:, :4] == 7).all() and (out[:, 32:] == 7).all()
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(w4.paged_chunk_attention(turned, *rest), plain)
    tables = torch.full((len(ROWS), rest[2].shape[1] + 20), 10 ** 9, dtype=torch.int32,
                        device="cuda")
    tables[:, :rest[2].shape[1]] = rest[2]
    rest[2] = tables[:, :rest[2].shape[1]]
    assert torch.equal(w4.paged_chunk_attention(q, *rest), plain)


@gpu
@pytest.mark.parametrize("page", [16, 13])
def test_heads_and_pages_of_stride_zero(w4lib, page):
    """Key-value heads that are one head seen several times, and a table of one page repeated."""
    q, k, v, tables, lengths, offsets = make([(100, 40), (3, 200)], 1, 8, 64, page, torch.float16,
                                             seed=14, garbage=0.0)
    four = [t.expand(-1, -1, 4, -1) for t in (k, v)]
    assert four[0].stride(2) == 0
    # (two heads to each of four: other tiles than eight to one, so other sums, each within the bound)
    check(q, *four, tables, lengths, offsets)
    same = tables.clone()
    same[:] = tables[0, 0]
    check(q, k, v, same, lengths, offsets)


@gpu
def test_offsets_that_make_no_sense(w4lib):
    """Descending, below 0 and past the tokens: whatever comes out, nothing else is touched and the
    next call is right."""
    args = make([(100, 40), (3, 200), (0, 30)], 2, 4, 64, 16, torch.float16, seed=15, garbage=0.0)
    plain = w4.paged_chunk_attention(*args)
    wide = torch.full((272, 9, 64), 7.0, device="cuda").half()
    for bad in ([0, 240, 40, 270], [-5, 40, 10 ** 9, 270], [270, 0, 0, 0], [2 ** 31 - 1] * 4,
                [-2 ** 31] * 4, [0, 0, 0, 2 ** 31 - 1]):
        w4.paged_chunk_attention(*args[:5], ints(bad), out=wide[1:271, :8])
        torch.cuda.synchronize()
        assert w4.device_status() == 0
        assert (wide[0] == 7).all() and (wide[271] == 7).all() and (wide[:, 8] == 7).all()
    assert torch.equal(w4.paged_chunk_attention(*args), plain)


@gpu
def test_one_token_a_row_is_paged_attention(w4lib):
    q, *rest = make([(n, 1) for n in (0, 5, 63, 64, 127, 500, 3000)], 4, 7, 128, 16,
                    torch.float16, seed=9)
    chunk = w4.paged_chunk_attention(q, *rest)
    single = w4.paged_attention(q, *rest[:4])
    assert (chunk.float() - single.float()).abs().max() <= 2.0 ** -10 * rest[1].float().nan_to_num().abs().max()


@gpu
def test_chunk_by_chunk(w4lib):
    """A prompt at once, and the same prompt in pieces: each token sees the same positions."""
    q, k, v, tables, lengths, offsets = make([(0, 700)], 2, 4, 128, 16, torch.float16, seed=10)
    whole = w4.paged_chunk_attention(q, k, v, tables, lengths, offsets)
    for cut in (1, 128, 200, 511):
        for first, last in ((0, cut), (cut, 700)):
            part = w4.paged_chunk_attention(q[first:last], k, v, tables, ints([last]),
                                            ints([0, last - first]))
            far = (part.float() - whole[first:last].float()).abs().max()
            assert far <= 4 * UNIT[torch.float16] * v.float().nan_to_num().abs().max()


@gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_repeats_streams_and_graphs(w4lib, dim):
    """The same bits again, from calls in turn on two streams and in two graphs that share
    what the allocator gives them."""
    first = make([(3000, 40), (0, 300), (77, 1)], 2, 4, dim, 16, torch.float16, seed=11, garbage=0.)
    second = make([(128, 129), (9000, 9)], 2, 4, dim, 16, torch.float16, seed=12, garbage=0.)
    want = [check(*first), check(*second)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for args, stream in zip((first, second), streams):
            got.append(w4.paged_chunk_attention(*args, stream=stream))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [], []
    for args in (first, second):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(w4.paged_chunk_attention(*args))
        graphs.append(graph)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])
    # other lengths for the captured call
    q, k, v, tables, lengths, offsets = first
    lengths -= 7
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], w4.paged_chunk_attention(*first))


@gpu
def test_far_pages(w4lib):
    """Pools of more than 2^32 bytes: pages on both sides of the border."""
    pages, page, kv, dim = 70000, 32, 8, 128
    k_pool = torch.empty(pages, page, kv, dim, device="cuda", dtype=torch.float16)
    v_pool = torch.empty_like(k_pool)
    assert k_pool.numel() * 2 > 2 ** 32
    rows = [(100, 30), (0, 64)]
    small = ref.cache(rows, kv, dim, page, torch.float16, seed=13, garbage=0.0)
    q = queries(small[-1], 32, dim, torch.float16, 13)
    want = check(q, *small)
    where = torch.linspace(0, pages - 1, small[0].shape[0]).long().cuda()
    k_pool[where], v_pool[where] = small[0], small[1]
    tables = torch.where(small[2] >= 0, where[small[2].clamp(min=0).long()].int(), -1)
    got = w4.paged_chunk_attention(q, k_pool, v_pool, tables, *small[3:])
    assert torch.equal(got, want)


@gpu
def test_many_sizes(w4lib):
    """Seeded draws over everything at once."""
    import random
    rng = random.Random(0)
    for seed in range(40):
        dim = rng.choice((16, 64, 96, 128, 200, 256))
        kv = rng.choice((1, 2, 3))
        group = rng.choice((1, 2, 3, 4, 7, 8, 20))
        rows = [(rng.choice((0, 0, rng.randrange(3000))), rng.choice((0, 1, rng.randrange(400))))
                for _ in range(rng.choice((1, 2, 5, 20)))]
        if sum(new for _, new in rows) * group * kv > 20000:
            rows = rows[:2]
        check(*make(rows, kv, group, dim, rng.choice((1, 8, 13, 16, 64)),
                    rng.choice((torch.float16, torch.bfloat16)),
                    layout=rng.choice(("slots", "heads", "both")), seed=seed))


def test_refused_calls():
    q, pool = torch.zeros(9, 8, 64).half(), torch.zeros(4, 16, 2, 64).half()
    tables, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    at = torch.zeros(4, dtype=torch.int32)
    good = dict(q=q, k_pool=pool, v_pool=pool, tables=tables, lengths=n, offsets=at)
    for bad in (dict(q=q[0]), dict(q=q.bfloat16()), dict(q=q[..., :32]), dict(v_pool=pool[:3]),
                dict(tables=tables.long()), dict(lengths=n[:2]), dict(lengths=n.long()),
                dict(offsets=n), dict(offsets=at.long()), dict(out=q[:8]), dict(out=q.float()),
                dict(q=q.transpose(1, 2)), dict()):
        with pytest.raises(ValueError):
            w4.paged_chunk_attention(**{**good, **bad})
