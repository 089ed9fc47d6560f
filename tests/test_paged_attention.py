"""The paged cache and the attention of a new token over it, against the 64-bit
definition: types, head layouts, page sizes, lengths from none to many splits,
strides, pages that are not there, and garbage in places that no row holds.

Tolerance, from the arithmetic: products of 16-bit values are exact in FP32 and
summed there, with 2 bits to spare for a tensor core's truncation, so a score is
off by at most E = dim * 2^-22 * sum |q k| scale (+ 2^-20 for the exponential);
a softmax average of V then moves by at most 4 E max|V|, and the output is
rounded once, by u |out| (u = 2^-11 for fp16, 2^-8 for bf16)."""
from __future__ import annotations

import math
import random

import pytest
import torch

import paged_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(lengths, kv_heads, group, dim, page, dtype, layout="slots", seed=0, spare=3,
         garbage=math.nan, width=None):
    """A cache whose rows hold `lengths` positions on scattered pages; every slot
    that no row holds is filled with `garbage`."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
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
    q = torch.randn(len(lengths), kv_heads * group, dim, generator=g) * 1.5
    return (q.to(dtype).cuda(), *pools, torch.tensor(tables, dtype=torch.int32).cuda(),
            torch.tensor(lengths, dtype=torch.int32).cuda())


def check(q, k_pool, v_pool, tables, lengths, scale=None, **kw):
    out, lse = w4.paged_attention(q, k_pool, v_pool, tables, lengths, scale=scale,
                                  return_lse=True, **kw)
    torch.cuda.synchronize()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, bound = ref.attention(q, k_pool, v_pool, tables, lengths, scale)
    error = q.shape[2] * 2.0 ** -22 * bound + 2.0 ** -20
    v = torch.nan_to_num(v_pool.cpu().double(), 0, 0, 0).abs().max()
    far = (out.cpu().double() - want).abs() - UNIT[q.dtype] * want.abs() - 4 * error[..., None] * v
    assert torch.isfinite(out).all()
    assert far.max() <= 2.0 ** -24, f"off by {far.max():.3g} beyond the bound"
    held = want_lse > -math.inf
    assert torch.equal(lse.cpu() > -math.inf, held)
    off = (lse.cpu().double() - want_lse)[held].abs()
    assert (off <= error[held] + 2.0 ** -20 * (1 + want_lse[held].abs())).all()
    assert (out.cpu()[~held] == 0).all()
    return out


ODD = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 0, 511]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv_heads, group, dim", [(8, 4, 128), (4, 7, 128), (1, 1, 64), (2, 8, 64),
                                                  (2, 16, 128), (1, 32, 128), (3, 5, 96),
                                                  (1, 12, 256), (2, 2, 256), (1, 71, 64),
                                                  (5, 3, 8), (1, 9, 136)])
def test_heads_and_sizes(w4lib, kv_heads, group, dim, dtype):
    check(*make(ODD, kv_heads, group, dim, 16, dtype, seed=dim + group))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv_heads, group, dim", [(8, 4, 128), (4, 7, 128), (1, 1, 64), (2, 8, 64),
                                                  (2, 16, 128), (3, 5, 96), (1, 12, 256),
                                                  (2, 2, 256), (1, 71, 64), (5, 3, 8)])
def test_tables_much_wider_than_the_rows(w4lib, kv_heads, group, dim, dtype):
    """Room for 64000 positions, so rows are cut into parts wherever they end."""
    check(*make(ODD + [1500, 70], kv_heads, group, dim, 16, dtype, seed=dim, width=4000))


@pytest.mark.parametrize("page", [1, 13, 24, 32])
@pytest.mark.parametrize("rows", [1, 2, 7, 29, 60])
def test_rows_and_widths(w4lib, rows, page):
    """Tables on both sides of every change in how the work is split."""
    for positions in (64, 500, 1030, 2100, 4200):
        lengths = [positions * (i + 1) // rows - i % 3 for i in range(rows)]
        q, k, v, tables, n = make(lengths, 2, 4, 64, page, torch.float16, seed=rows)
        narrow = check(q, k, v, tables, n)
        wide = torch.cat([tables, torch.full((rows, 70000 // page), -1, dtype=torch.int32,
                                             device="cuda")], 1)
        other = w4.paged_attention(q, k, v, wide, n)
        # split elsewhere: sums in another order, so a rounding of the output apart at most
        assert ((narrow.double() - other.double()).abs()
                <= 2 * UNIT[q.dtype] * narrow.double().abs() + 1e-4).all()
    lengths[0] = 0
    check(*make(lengths, 2, 4, 64, page, torch.float16, seed=rows))


@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 48, 64, 128, 256])
def test_pages_and_layouts(w4lib, page, layout):
    check(*make(ODD, 2, 4, 128, page, torch.float16, layout, seed=page))


@pytest.mark.parametrize("lengths", [[1], [16], [17], [512], [4096, 1], [20011], [3, 20011, 0, 700],
                                     [0], [0, 0, 0], list(range(150)), [64] * 700])
@pytest.mark.parametrize("kv_heads, group", [(8, 4), (1, 7)])
def test_lengths(w4lib, lengths, kv_heads, group):
    check(*make(lengths, kv_heads, group, 64, 16, torch.float16, seed=len(lengths)))


@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
def test_garbage_where_no_row_is(w4lib, garbage):
    check(*make(ODD, 2, 4, 128, 32, torch.float16, garbage=garbage))


def test_lengths_out_of_range(w4lib):
    q, k, v, tables, lengths = make([32, 48, 16], 2, 4, 64, 16, torch.float16, width=3)
    lengths[0] = -5
    lengths[1] = 1 << 30                       # counts as 3 pages of 16
    check(q, k, v, tables, lengths)


@pytest.mark.parametrize("page", [8, 16, 64])
def test_pages_that_are_not_there(w4lib, page):
    q, k, v, tables, lengths = make([400, 300, 200], 2, 4, 128, page, torch.float16, seed=3)
    tables[0, 1] = -1
    tables[0, 2] = k.shape[0]                  # one past the pool
    tables[0, 3] = 2 ** 31 - 1
    tables[1, :] = -7                          # a row with no page at all
    check(q, k, v, tables, lengths)


def test_large_scores_and_scale(w4lib):
    """Scores of some hundreds, where the running maximum has to carry the sum."""
    q, k, v, tables, lengths = make([700, 33], 2, 4, 128, 16, torch.float16, seed=5, garbage=0.)
    check(q * 8, k * 4, v, tables, lengths)
    check(q, k, v, tables, lengths, scale=0.0)
    check(q, k, v, tables, lengths, scale=-0.25)


def test_equal_scores_average(w4lib):
    """A query of zeros weighs all positions alike: the average of V."""
    q, k, v, tables, lengths = make([1000], 1, 4, 64, 16, torch.float16, seed=6, garbage=0.)
    q.zero_()
    check(q, k, v, tables, lengths)


@pytest.mark.parametrize("width", [None, 30000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_small_weights_beside_a_large_one(w4lib, dtype, width):
    """A position that draws nearly all attention, and a hundred thousand others whose
    weights, each 1.5 * 2^-24 of it, are a hundredth of the sum."""
    n = 100_000
    q, k, v, tables, lengths = make([n], 1, 2, 64, 16, dtype, seed=12, garbage=0.0, width=width)
    q.zero_()
    q[:, :, 0] = 1.0
    k.zero_()
    v.fill_(1.0)
    page = int(tables[0, 0])
    k[page, 3, 0, 0] = math.log(2.0 ** 24 / 1.5)
    v[page, 3] = 0.0
    check(q, k, v, tables, lengths, scale=1.0)


@pytest.mark.parametrize("rising", [True, False])
def test_ordered_scores(w4lib, rising):
    """The maximum found last, or first."""
    q, k, v, tables, lengths = make([1500], 1, 2, 64, 16, torch.float16, seed=7, garbage=0.)
    q.fill_(0.5)
    at = torch.arange(1500, device="cuda") / 100.0
    at = at if rising else at.flip(0)
    for p in range(0, 1500, 16):
        n = min(16, 1500 - p)
        k[tables[0, p // 16], :n, 0] = at[p:p + n, None].half()
    check(q, k, v, tables, lengths)


def test_strided_query_and_output(w4lib):
    q, k, v, tables, lengths = make(ODD, 4, 7, 128, 16, torch.bfloat16, seed=8)
    plain = check(q, k, v, tables, lengths)
    wide = torch.randn(len(ODD), 36, 128, device="cuda").bfloat16()
    wide[:, :28] = q
    out = torch.full((len(ODD), 40, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    got = w4.paged_attention(wide[:, :28], k, v, tables, lengths, out=out[:, 4:32])
    assert torch.equal(got, plain) and torch.equal(out[:, 4:32], plain)
    assert (out[:, :4] == 7).all() and (out[:, 32:] == 7).all()
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(w4.paged_attention(turned, k, v, tables[:, :], lengths), plain)


def test_a_slice_of_a_wider_table(w4lib):
    q, k, v, tables, lengths = make(ODD, 2, 4, 64, 16, torch.float16, seed=9, width=40)
    wide = torch.full((len(ODD), 64), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :40] = tables
    check(q, k, v, wide[:, :40], lengths)


def test_repeat_and_streams(w4lib):
    """The same bits again, also from calls in turn on two streams and in a graph."""
    # zeros for garbage: the graph's lengths below reach into slots that no row held
    case = make([9000, 100, 0, 4000], 8, 4, 128, 16, torch.float16, seed=10, garbage=0.0)
    first = w4.paged_attention(*case)
    other = make([300, 2000, 17, 1], 8, 4, 128, 16, torch.float16, seed=11)
    second = w4.paged_attention(*other)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((w4.paged_attention(*case, stream=a), w4.paged_attention(*other, stream=b)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) and torch.equal(y, second) for x, y in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.paged_attention(*case)
    case[4].copy_(torch.tensor([1, 8999, 50, 0]))   # lengths change between replays
    graph.replay()
    torch.cuda.synchronize()
    now = check(*case)
    assert torch.equal(out, now)


def test_past_32_bit_offsets(w4lib):
    """Pages that start beyond 2^31 elements of the pool."""
    pages, page, kv, dim = 70000, 16, 8, 256
    pool = torch.empty(2, pages, page, kv, dim, dtype=torch.float16, device="cuda")
    assert pages * page * kv * dim > 2 ** 31
    tables = torch.tensor([[69999, 5, 66001, 69998]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([55], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(55, kv, dim, generator=g, device="cuda").half() for _ in range(2))
    w4.paged_append(k, v, pool[0], pool[1], tables, torch.zeros_like(lengths),
                    torch.tensor([0, 55], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 4 * kv, dim, generator=g, device="cuda").half()
    out = w4.paged_attention(q, pool[0], pool[1], tables, lengths)
    small = torch.empty(2, 4, page, kv, dim, dtype=torch.float16, device="cuda")
    for i, p in enumerate(tables[0].tolist()):
        small[:, i] = pool[:, p]
    near = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    assert torch.equal(out, check(q, small[0], small[1], near, lengths))


@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append(w4lib, page, layout, dtype):
    """Ragged new tokens, cut from a wider product, and nothing else written."""
    counts, starts = [3, 0, 70, 1, 18], [0, 9, 5, 31, 16]
    held = [s + n for s, n in zip(starts, counts)]
    _, k_pool, v_pool, tables, _ = make(held, 3, 1, 40, page, dtype, layout, garbage=2.0)
    qkv = torch.randn(sum(counts), 4 * 3 * 40).to(dtype).cuda()
    k, v = (qkv[:, i * 120:(i + 1) * 120].unflatten(1, (3, 40)) for i in (2, 3))
    want = [k_pool.clone(), v_pool.clone()]
    t = 0
    for b, (s, n) in enumerate(zip(starts, counts)):
        for p in range(s, s + n):
            want[0][tables[b, p // page], p % page] = k[t]
            want[1][tables[b, p // page], p % page] = v[t]
            t += 1
    offsets = torch.tensor([sum(counts[:i]) for i in range(6)], dtype=torch.int32, device="cuda")
    w4.paged_append(k, v, k_pool, v_pool, tables,
                    torch.tensor(starts, dtype=torch.int32, device="cuda"), offsets)
    torch.cuda.synchronize()
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])


def test_append_one_token_a_row(w4lib):
    q, k_pool, v_pool, tables, lengths = make([5, 16, 100, 33], 2, 1, 64, 16, torch.float16,
                                              garbage=0.0, width=9, spare=20)
    tables[1, 1] = int(set(range(k_pool.shape[0])).difference(tables.flatten().tolist()).pop())
    k, v = (torch.randn(4, 2, 64, device="cuda").half() for _ in range(2))
    want = [k_pool.clone(), v_pool.clone()]
    for b, n in enumerate([5, 16, 100, 33]):
        want[0][tables[b, n // 16], n % 16] = k[b]
        want[1][tables[b, n // 16], n % 16] = v[b]
    w4.paged_append(k, v, k_pool, v_pool, tables, lengths)
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])


def test_append_leaves_out_what_has_no_place(w4lib):
    _, k_pool, v_pool, tables, _ = make([16, 16, 16, 16], 1, 1, 64, 16, torch.float16, garbage=0.0)
    before = k_pool.clone(), v_pool.clone()
    tables[1, 0] = -1
    tables[2, 0] = k_pool.shape[0]
    k = torch.randn(4, 1, 64, device="cuda").half()
    starts = torch.tensor([-1, 3, 3, 16], dtype=torch.int32, device="cuda")
    w4.paged_append(k, k, k_pool, v_pool, tables, starts)
    # tokens before the first offset and past the last belong to no row
    offsets = torch.tensor([2, 2, 2, 2, 2], dtype=torch.int32, device="cuda")
    w4.paged_append(k, k, k_pool, v_pool, tables, torch.zeros_like(starts), offsets)
    torch.cuda.synchronize()
    assert torch.equal(k_pool, before[0]) and torch.equal(v_pool, before[1])


def test_append_nothing_and_many(w4lib):
    _, k_pool, v_pool, tables, _ = make([0] * 3 + [9000] + [0] * 4, 2, 1, 64, 16, torch.float16,
                                        garbage=0.0)
    starts = torch.zeros(8, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    w4.paged_append(none, none, k_pool, v_pool, tables, starts,
                    torch.zeros(9, dtype=torch.int32, device="cuda"))
    k, v = (torch.randn(9000, 2, 64, device="cuda").half() for _ in range(2))
    offsets = torch.tensor([0, 0, 0, 0] + [9000] * 5, dtype=torch.int32, device="cuda")
    w4.paged_append(k, v, k_pool, v_pool, tables, starts, offsets)
    pages = tables[3].long()
    assert torch.equal(k_pool[pages].flatten(0, 1)[:9000], k)
    assert torch.equal(v_pool[pages].flatten(0, 1)[:9000], v)


@pytest.mark.parametrize("seed", range(30))
def test_random_caches(w4lib, seed):
    rng = random.Random(seed)
    kv_heads, group = rng.choice((1, 2, 3, 8)), rng.choice((1, 2, 5, 7, 8, 9, 16, 17, 33))
    dim = rng.choice((8, 40, 64, 72, 96, 128, 136, 200, 256))
    page = rng.choice((1, 2, 5, 16, 17, 32, 48, 64, 100, 128))
    rows = rng.choice((1, 2, 3, 9, 40, 130))
    longest = rng.choice((1, 17, 100, 300, 1500 if rows < 10 else 200))
    lengths = [rng.choice((0, rng.randint(0, longest), longest)) for _ in range(rows)]
    need = max(1, max(-(-n // page) for n in lengths))
    case = make(lengths, kv_heads, group, dim, page, rng.choice((torch.float16, torch.bfloat16)),
                rng.choice(("slots", "heads", "both")), seed=seed,
                width=rng.choice((None, need + rng.randint(0, 50), need + 70000 // page)),
                garbage=rng.choice((math.nan, math.inf, 0.0)))
    if rng.random() < 0.2:
        case[3][rng.randrange(rows), 0] = rng.choice((-1, case[1].shape[0], 2 ** 31 - 1))
    check(*case, scale=rng.choice((None, None, 0.3, -0.1)))


@pytest.mark.parametrize("seed", range(20))
def test_append_to_many_rows(w4lib, seed):
    """Rows by the thousand, most without a token, tokens before the first row and past the last."""
    rng = random.Random(seed)
    rows, page = rng.choice((1, 2, 31, 32, 33, 1000, 1025, 3000)), rng.choice((1, 7, 16))
    counts = [rng.choice((0, 0, 1, rng.randint(0, 9))) for _ in range(rows)]
    counts[rng.randrange(rows)] += rng.choice((0, 500))
    starts = [rng.randint(0, 2 * page) for _ in range(rows)]
    _, k_pool, v_pool, tables, _ = make([s + n for s, n in zip(starts, counts)], 2, 1, 24, page,
                                        torch.float16, rng.choice(("slots", "heads")), seed=seed,
                                        garbage=2.0)
    first, past = rng.choice((0, 3)), rng.choice((0, 5))
    offsets = [first]
    for n in counts:
        offsets.append(offsets[-1] + n)
    k, v = (torch.randn(offsets[-1] + past, 2, 24, device="cuda").half() for _ in range(2))
    at = [(b, s + i) for b, (s, n) in enumerate(zip(starts, counts)) for i in range(n)]
    want = [k_pool.clone(), v_pool.clone()]
    if at:
        row, position = (torch.tensor(x, device="cuda") for x in zip(*at))
        pages = tables[row, position // page].long()
        for pool, new in zip(want, (k, v)):
            pool[pages, position % page] = new[first:offsets[-1]]
    w4.paged_append(k, v, k_pool, v_pool, tables,
                    torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert torch.equal(k_pool, want[0]) and torch.equal(v_pool, want[1])


def test_refusals(w4lib):
    q, k, v, tables, lengths = make([20, 5], 2, 2, 64, 16, torch.float16, garbage=0.0)
    good = (q, k, v, tables, lengths)

    def bad(error, **change):
        names = ("q", "k_pool", "v_pool", "tables", "lengths")
        with pytest.raises(error):
            w4.paged_attention(**{**dict(zip(names, good)), **change})

    bad(ValueError, q=q.float())
    bad(ValueError, q=q.cpu())
    bad(ValueError, q=q[:, :, :32])
    bad(ValueError, q=q[:1])
    bad(ValueError, q=q.transpose(1, 2))
    bad(ValueError, k_pool=k.float())
    bad(ValueError, v_pool=v.bfloat16())
    bad(ValueError, v_pool=v.transpose(1, 2).contiguous().transpose(1, 2))
    bad(ValueError, v_pool=v[:-1])
    bad(ValueError, tables=tables.long())
    bad(ValueError, tables=tables[0])
    bad(ValueError, lengths=lengths[:1])
    bad(ValueError, lengths=lengths.float())
    bad(ValueError, out=torch.empty_like(q).float())
    bad(ValueError, out=torch.empty_like(q)[:, :2])
    bad(w4._native.W4A16Error, q=q[:, :3].contiguous())           # 3 heads over 2
    flat = torch.zeros(q.numel() + 1, dtype=torch.float16, device="cuda")
    bad(w4._native.W4A16Error, q=flat[1:].view(q.shape))            # 2-byte aligned
    bad(w4._native.W4A16Error, scale=math.nan)
    ones = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    starts = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        w4.paged_append(ones, ones.float(), k, v, tables, starts)
    with pytest.raises(ValueError):
        w4.paged_append(ones, ones, k, v, tables, starts, starts)  # 3 offsets, not 2
    with pytest.raises(w4._native.W4A16Error):
        w4.paged_append(ones[:1], ones[:1], k, v, tables, starts)  # one token, two rows


def test_no_rows(w4lib):
    q, k, v, tables, lengths = make([20], 2, 2, 64, 16, torch.float16)
    out, lse = w4.paged_attention(q[:0], k, v, tables[:0], lengths[:0], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    w4.paged_append(q[:0, :2], q[:0, :2], k, v, tables[:0], lengths[:0])


@pytest.mark.parametrize("page, width", [(14322, 149943), (8176, 262657)])
def test_lengths_up_to_the_last_31_bit_position(w4lib, page, width):
    """A table for 2^31 - 2 and for 2^31 - 16 positions, all on one page but the last.  Head 0
    weighs all alike: sums of whole numbers below 2^24 a warp, so what is off is the join of at
    most 1024 parts (2^-14) and the output's rounding.  Head 1 sees the last position alone."""
    total = page * width
    assert 2 ** 31 - 64 < total < 2 ** 31
    q = torch.zeros(1, 2, 8, dtype=torch.float16)
    q[0, 1] = 1.0
    k = torch.zeros(2, page, 1, 8, dtype=torch.float16)
    k[1, -1] = 6.0                              # a score of 48 = 2 ln 2^31 and more
    v = (torch.arange(page) % 8)[None, :, None, None].expand(2, -1, 1, 8).half().contiguous()
    v[1, -1] = 100.0
    tables = torch.zeros(1, width, dtype=torch.int32)
    tables[0, -1] = 1
    mean = ((v[0, :, 0, 0].double().sum() * width + 100 - v[0, -1, 0, 0]) / total).item()
    for length in (total, 2 ** 31 - 1):
        out, lse = w4.paged_attention(q.cuda(), k.cuda(), v.cuda(), tables.cuda(),
                                      torch.tensor([length], dtype=torch.int32).cuda(),
                                      scale=1.0, return_lse=True)
        assert ((out[0, 0].cpu().double() - mean).abs() <= mean * (2.0 ** -11 + 2.0 ** -13)).all()
        assert abs(lse[0, 0].item() - math.log(total)) <= 2.0 ** -13
        assert (out[0, 1] == 100).all() and abs(lse[0, 1].item() - 48) <= 2.0 ** -12
