"""The books of a paged cache and its page copies against list definitions:
whole numbers, equal in every place."""
from __future__ import annotations

import random

import pytest
import torch

import paged_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(pages, rows, width, ps, used, seed=0):
    """Books with `used` pages held, some by several rows, and the rest free."""
    rng = random.Random(seed)
    held = rng.sample(range(pages), used)
    refs, tables, lengths, at = [0] * pages, [], [], 0
    for r in range(rows):
        n = rng.randint(0, width - 1) if rng.random() < 0.8 else 0
        n = min(n, used - at)
        row, at = held[at:at + n], at + n
        if tables and rng.random() < 0.3:      # a prefix shared with an earlier row
            other = rng.choice(tables)
            row = ([p for p in other if p >= 0][:rng.randint(0, 3)] + row)[:width - 1]
        for p in row:
            refs[p] += 1
        lengths.append(max(0, len(row) * ps - rng.randrange(ps)) if row else 0)
        tables.append(row + [-1] * (width - len(row)))
    return refs, tables, lengths


def same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), torch.tensor(w, dtype=torch.int32).view(g.shape))


def books(b, in_place, wide=False):
    """Input tensors of the books (tables a slice of a wider tensor when asked) and `out`."""
    refs, tables, lengths = (ints(t) for t in b)
    if wide:
        big = torch.full((tables.shape[0], tables.shape[1] + 5), -3, dtype=torch.int32,
                         device="cuda")
        big[:, :tables.shape[1]] = tables
        tables = big[:, :tables.shape[1]]
    ins = refs, tables, lengths
    return ins, (ins if in_place else None)


SIZES = [(1, 1, 2, 1), (40, 6, 5, 16), (511, 40, 12, 16), (512, 33, 20, 4), (2000, 64, 70, 16),
         (16384, 100, 130, 1), (16385, 300, 33, 32), (140000, 50, 999, 16)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages, rows, width, ps", SIZES)
def test_free(w4lib, pages, rows, width, ps, in_place):
    b = make(pages, rows, width, ps, pages * 3 // 4, seed=pages)
    rng = random.Random(1)
    listed = [rng.randrange(rows) for _ in range(rows // 2 + 1)] + [-1, rows, 2 ** 31 - 1]
    ins, out = books(b, in_place, wide=True)
    got = w4.pages_free(*ins, ints(listed), out=out)
    same(got, ref.free(*b, listed))
    if not in_place:
        same(ins, b)


def test_free_of_foreign_numbers_and_nothing(w4lib):
    b = [1, 2, 1], [[0, -1, 7, 2 ** 31 - 1], [1, -5, 1, -1]], [4, 2]
    ins, _ = books(b, False)
    same(w4.pages_free(*ins, ints([0, 1])), ref.free(*b, [0, 1]))
    same(w4.pages_free(*ins, ints([])), b)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages, rows, width, ps", SIZES)
def test_extend(w4lib, pages, rows, width, ps, in_place):
    b = make(pages, rows, width, ps, pages // 2, seed=pages + 1)
    rng = random.Random(2)
    n = min(rows, 2500)
    listed = rng.sample(range(rows), n) + [rng.randrange(rows), -1, rows, 0]
    counts = [rng.choice((0, 1, 2, ps, 3 * ps, rng.randrange(width * ps + 2))) for _ in range(n)]
    counts += [1, 1, 1, -4]
    ins, out = books(b, in_place, wide=True)
    got = w4.pages_extend(*ins, ints(listed), ints(counts), ps, out=out)
    same(got, ref.extend(*b, listed, counts, ps))


def test_extend_until_none_is_left(w4lib):
    b = [0, 1, 0, 0], [[1, -1, -1], [-1] * 3, [-1] * 3], [3, 0, 0]
    for listed, counts in (([1, 2, 0], [8, 5, 1]), ([2, 0, 1], [12, 1, 1]), ([0], [9]), ([], [])):
        ins, _ = books(b, False)
        got = w4.pages_extend(*ins, ints(listed), ints(counts), 4)
        same(got, ref.extend(*b, listed, counts, 4))


def test_extend_long_lists(w4lib):
    """More requests than a block has threads."""
    rows = 3000
    b = [0] * 4000, [[-1] * 3 for _ in range(rows)], [0] * rows
    listed = list(range(rows))
    counts = [(i * 7) % 9 for i in listed]
    ins, out = books(b, True)
    same(w4.pages_extend(*ins, ints(listed), ints(counts), 4, out=out),
         ref.extend(*b, listed, counts, 4))


def fill(planes, pages, shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(planes, pages, *shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages, rows, width, ps", SIZES)
def test_fork(w4lib, pages, rows, width, ps, in_place):
    b = make(pages, rows, width, ps, pages // 2, seed=pages + 2)
    rng = random.Random(3)
    empty = [r for r, n in enumerate(b[2]) if n == 0]
    children = empty + empty[:2] + [0, rows - 1, -1, rows]
    rng.shuffle(children)
    parents = [rng.randrange(rows) for _ in children]
    parents[0] = rows
    pool = fill(2, pages, (8,), torch.float16)
    want = pool.clone()
    ins, out = books(b, in_place, wide=True)
    got = w4.pages_fork(pool, *ins, ints(parents), ints(children), ps, out=out)
    *books_want, copies = ref.fork(*b, parents, children, ps)
    same(got, books_want)
    for a, z in copies:
        want[:, z] = want[:, a]
    assert torch.equal(pool, want)


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_long_lists_with_requests_that_are_refused(w4lib, in_place):
    """More requests than a block has threads; every third past the first thousand names a row
    that is not there, behind requests of the same thread that were granted."""
    rows, ps = 2600, 4
    b = [1] * 3 + [0] * 3000, [[0, 1, 2, -1]] + [[-1] * 4 for _ in range(rows - 1)], \
        [11] + [0] * (rows - 1)
    children = list(range(1, 2500))
    parents = [0] * len(children)
    for i in range(1024, len(children), 3):
        if i % 2:
            parents[i] = rows + i
        else:
            children[i] = -1 - i
    pool = fill(2, 3003, (8,), torch.float16)
    want = pool.clone()
    ins, out = books(b, in_place)
    got = w4.pages_fork(pool, *ins, ints(parents), ints(children), ps, out=out)
    *books_want, copies = ref.fork(*b, parents, children, ps)
    same(got, books_want)
    for a, z in copies:
        want[:, z] = want[:, a]
    assert torch.equal(pool, want)


def test_fork_exhausts_and_chains(w4lib):
    """Too few pages for all; a child that is also listed as an (empty) parent."""
    b = [1, 1, 0, 0], [[0, 1, -1]] + [[-1] * 3 for _ in range(5)], [6, 0, 0, 0, 0, 0]
    for parents, children in (([0, 0, 0, 0], [1, 2, 3, 4]), ([0, 1, 2], [1, 2, 3]),
                              ([5, 0], [1, 5]), ([0], [0]), ([], [])):
        for in_place in (False, True):
            pool = fill(3, 4, (4, 2, 8), torch.bfloat16, seed=4)
            want = pool.clone()
            ins, out = books(b, in_place)
            got = w4.pages_fork(pool, *ins, ints(parents), ints(children), 4, out=out)
            *books_want, copies = ref.fork(*b, parents, children, 4)
            same(got, books_want)
            for a, z in copies:
                want[:, z] = want[:, a]
            assert torch.equal(pool, want)


def test_fork_whose_parent_lacks_its_last_page(w4lib):
    b = [1, 0, 0], [[0, -1], [7, 0], [-1, -1], [-1, -1]], [6, 3, 0, 0]
    pool = fill(1, 3, (8,), torch.float16)
    before = pool.clone()
    ins, _ = books(b, False)
    got = w4.pages_fork(pool, *ins, ints([0, 1]), ints([2, 3]), 4)
    same(got, ref.fork(*b, [0, 1], [2, 3], 4)[:4])
    assert got[3].tolist() == [0, 0] and torch.equal(pool, before)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("used", [0.0, 0.3, 0.7, 1.0])
@pytest.mark.parametrize("pages, rows, width, ps", SIZES)
def test_compact(w4lib, pages, rows, width, ps, used, in_place):
    b = make(pages, rows, width, ps, int(pages * used), seed=pages + 3)
    pool = fill(3, pages, (8,), torch.float16)
    want = pool.clone()
    ins, out = books(b, in_place, wide=True)
    got = w4.pages_compact(pool, *ins[:2], out=out[:2] if out else None)
    *books_want, copies = ref.compact(*b[:2])
    same(got, books_want)
    for a, z in copies:
        want[:, z] = want[:, a]
    assert torch.equal(pool, want)


def test_compact_passes_over_numbers_that_nothing_holds(w4lib):
    b = [0, 1, 0, 0, 2, 1], [[4, 5, 3, -1], [4, 1, 9, -8]]
    pool = fill(2, 6, (8,), torch.float16)
    want = pool.clone()
    got = w4.pages_compact(pool, ints(b[0]), ints(b[1]))
    *books_want, copies = ref.compact(*b)
    same(got, books_want)
    for a, z in copies:
        want[:, z] = want[:, a]
    assert torch.equal(pool, want)


@pytest.mark.parametrize("values", [8, 24, 1000, 16384, 40008])
def test_page_sizes_of_a_copy(w4lib, values):
    """Pages of 16 bytes to many pieces, in planes and pages with gaps between."""
    wide = fill(5, 9, (values + 8,), torch.float16)
    pool = wide[1:4, :, :values]
    want = wide.clone()
    sources, targets = [0, 3, -1, 5, 9, 2], [1, 8, 4, 6, 7, 12]
    for a, z in ((0, 1), (3, 8), (5, 6)):
        want[1:4, z, :values] = want[1:4, a, :values]
    w4.pages_copy(pool, ints(sources), ints(targets))
    torch.cuda.synchronize()
    assert torch.equal(wide, want)
    w4.pages_copy(pool, ints([]), ints([]))
    assert torch.equal(wide, want)


def test_copy_many_pages(w4lib):
    pool = fill(7, 600, (2, 16, 40), torch.bfloat16)
    want = pool.clone()
    order = random.Random(5).sample(range(600), 600)
    sources, targets = order[:300], order[300:]
    want[:, targets] = want[:, sources]
    w4.pages_copy(pool, ints(sources), ints(targets))
    assert torch.equal(pool, want)


def test_copy_past_32_bit_offsets(w4lib):
    pool = torch.zeros(2, 1200, 1 << 20, dtype=torch.float16, device="cuda")  # 2.5 G values
    pool[:, 1199, -5:] = 3.0
    w4.pages_copy(pool, ints([1199]), ints([1]))
    assert (pool[:, 1, -5:] == 3).all() and (pool[:, 1, :-5] == 0).all()


@pytest.mark.parametrize("seed", range(60))
def test_random_books(w4lib, seed):
    """Sizes on both sides of every change in how the work is done, lists with rows out of
    range and twice, in place and apart."""
    rng = random.Random(seed)
    pages = rng.choice((1, 2, 31, 33, 511, 513, 4095, 4096, 4097, 16384, 16385, 40000))
    rows = rng.choice((1, 7, 100, 257, 1023, 1025, 4096, 4097))
    width, ps = rng.choice((2, 3, 9, 33, 70)), rng.choice((1, 3, 16))
    b = make(pages, rows, width, ps, rng.randrange(0, pages + 1), seed=seed)
    ins, out = books(b, rng.random() < 0.4, wide=rng.random() < 0.5)
    n = rng.choice((0, 1, 5, 255, 256, 257, 1024, 1025, 3000))
    listed = [rng.randrange(-1, rows + 1) for _ in range(n)]
    empty = [r for r, m in enumerate(b[2]) if m == 0] or [0]
    children = [rng.choice(empty) if rng.random() < 0.8 else rng.randrange(-1, rows + 1)
                for _ in range(n)]
    counts = [rng.choice((-1, 0, 1, 2, ps, 3 * ps, width * ps)) for _ in range(n)]
    pool = fill(2, pages, (8,), torch.float16, seed=seed)
    moved, copies = pool.clone(), []
    what = seed % 4
    if what == 0:
        got, want = w4.pages_free(*ins, ints(listed), out=out), ref.free(*b, listed)
    elif what == 1:
        got = w4.pages_extend(*ins, ints(listed), ints(counts), ps, out=out)
        want = ref.extend(*b, listed, counts, ps)
    elif what == 2:
        got = w4.pages_fork(pool, *ins, ints(listed), ints(children), ps, out=out)
        *want, copies = ref.fork(*b, listed, children, ps)
    else:
        got = w4.pages_compact(pool, *ins[:2], out=out[:2] if out else None)
        *want, copies = ref.compact(*b[:2])
    same(got, want)
    if copies:
        sources, targets = (torch.tensor(t, device="cuda") for t in zip(*copies))
        moved[:, targets] = moved[:, sources]
    assert torch.equal(pool, moved)
    if out is None:
        same(ins, b)


def test_life_of_a_cache(w4lib):
    """Random lives of rows through PagedCache, its books checked at every step."""
    rng = random.Random(6)
    ps, rows, pages, layers = 4, 12, 64, 2
    cache = w4.PagedCache(layers, rows, pages, 2, 16, page_size=ps, max_length=60)
    b = [0] * pages, [[-1] * 15 for _ in range(rows)], [0] * rows
    content = [[] for _ in range(rows)]        # the value of each position of each row
    stamp = 0
    for step in range(120):
        what = rng.choice(("extend", "extend", "fork", "free", "compact"))
        if what == "extend":
            listed = rng.sample(range(rows), rng.randint(1, rows))
            counts = [rng.randint(0, 9) for _ in listed]
            starts = [b[2][r] for r in listed]
            done = cache.extend(ints(listed), ints(counts))
            *b, want = ref.extend(*b, listed, counts, ps)
            assert done.tolist() == want
            counts = [c if d else 0 for c, d in zip(counts, want)]
            new = [list(range(stamp + 1 + sum(counts[:i]), stamp + 1 + sum(counts[:i + 1])))
                   for i in range(len(listed))]
            stamp += sum(counts)
            for r, x in zip(listed, new):
                content[r] = content[r] + x
            flat = torch.tensor([y % 2000 for x in new for y in x], device="cuda").half()
            k = flat.view(-1, 1, 1).expand(-1, 2, 16).contiguous()
            offsets = [sum(counts[:i]) for i in range(len(counts) + 1)]
            for layer in range(layers):
                cache.append(layer, k + layer, k - layer, ints(starts), ints(offsets),
                             rows=ints(listed))
        elif what == "fork":
            children = rng.sample(range(rows), 4)
            parents = [rng.randrange(rows) for _ in children]
            done = cache.fork(ints(parents), ints(children))
            old = [list(c) for c in content]
            *b, want, _ = ref.fork(*b, parents, children, ps)
            assert done.tolist() == want
            for a, c, d in zip(parents, children, want):
                if d:
                    content[c] = old[a]
        elif what == "free":
            listed = rng.sample(range(rows), rng.randint(1, 4))
            cache.free(ints(listed))
            b = ref.free(*b, listed)
            for r in listed:
                content[r] = []
        else:
            used = cache.compact()
            refs, tables, want, _ = ref.compact(b[0], b[1])
            b = refs, tables, b[2]
            assert used.item() == want
        same((cache.refs, cache.tables, cache.lengths), b)
        for r in range(rows):
            assert b[2][r] == len(content[r])
            for layer in range(layers):
                pages_of = [p for p in b[1][r] if p >= 0]
                got = cache.pool[2 * layer][pages_of].flatten(0, 1)[:b[2][r], 1, 3]
                assert got.tolist() == [x % 2000 + layer for x in content[r]]


def test_refusals(w4lib):
    b = make(8, 4, 3, 4, 4)
    (refs, tables, lengths), _ = books(b, False)
    pool = fill(2, 8, (8,), torch.float16)
    one = ints([1])
    with pytest.raises(ValueError):
        w4.pages_free(refs.long(), tables, lengths, one)
    with pytest.raises(ValueError):
        w4.pages_free(refs, tables, lengths[:2], one)
    with pytest.raises(ValueError):
        w4.pages_free(refs, tables, lengths, one.long())
    with pytest.raises(ValueError):
        w4.pages_free(refs, tables, lengths, one, out=(refs, tables))
    with pytest.raises(ValueError):
        w4.pages_extend(refs, tables, lengths, one, ints([1, 2]), 4)
    with pytest.raises(w4._native.W4A16Error):
        w4.pages_extend(refs, tables, lengths, one, one, 0)
    with pytest.raises(ValueError):
        w4.pages_fork(pool[:, :5], refs, tables, lengths, one, one, 4)
    with pytest.raises(ValueError):
        w4.pages_fork(pool.cpu(), refs, tables, lengths, one, one, 4)
    with pytest.raises(ValueError):
        w4.pages_compact(fill(2, 8, (4, 8), torch.float16).transpose(2, 3), refs, tables)
    with pytest.raises(w4._native.W4A16Error):
        w4.pages_compact(fill(2, 8, (7,), torch.float16), refs, tables)     # 14-byte pages
    with pytest.raises(ValueError):
        w4.pages_copy(pool, one, ints([1, 2]))


# (values of a page, planes): one piece of 16 KB and several, the last one partly filled; 52 and
# 53 planes are on both sides of 128 MB of copies by 32 pages of 80016 bytes.
POOLS = [(8, 3), (1000, 3), (8192, 2), (8200, 2), (16384, 5), (40008, 1), (40008, 52), (40008, 53)]


def gapped(planes, pages, values, seed):
    """A pool with foreign planes around it and gaps between its pages, and all of its memory."""
    wide = fill(planes + 2, pages, (values + 8,), torch.float16, seed=seed)
    return wide[1:-1, :, :values], wide


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("values, planes", POOLS)
def test_compact_moves_whole_pages(w4lib, values, planes, gaps, in_place):
    b = make(64, 12, 9, 16, 40, seed=values)
    pool, wide = gapped(planes, 64, values, planes)
    if not gaps:
        pool = wide = pool.contiguous()
    want = wide.clone()
    inner = want[1:-1, :, :values] if gaps else want
    ins, out = books(b, in_place)
    got = w4.pages_compact(pool, *ins[:2], out=out[:2] if out else None)
    *books_want, copies = ref.compact(*b[:2])
    assert len(copies) > 3
    same(got, books_want)
    for a, z in copies:
        inner[:, z] = inner[:, a]
    assert torch.equal(wide, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("values, planes", POOLS)
def test_fork_copies_whole_pages(w4lib, values, planes, gaps, in_place):
    """32 branches, some of parents that end on a page's edge and copy nothing, and too few free
    pages for the last ones."""
    ps, parents_of = 16, [5, 16, 40, 33, 0, 64, 1, 20]
    tables, refs = [], [0] * 64
    for i, n in enumerate(parents_of):
        row = [(i * 7 + j * 11) % 64 for j in range(-(-n // ps))]
        for p in row:
            refs[p] += 1
        tables.append(row + [-1] * (5 - len(row)))
    free = [p for p in range(64) if refs[p] == 0]
    for p in free[18:]:
        refs[p] = 1                                # held by rows elsewhere
    tables += [[-1] * 5 for _ in range(32)]
    b = refs, tables, parents_of + [0] * 32
    parents, children = [i * 3 % 8 for i in range(32)], list(range(8, 40))
    random.Random(values).shuffle(children)
    pool, wide = gapped(planes, 64, values, planes)
    if not gaps:
        pool = wide = pool.contiguous()
    want = wide.clone()
    inner = want[1:-1, :, :values] if gaps else want
    ins, out = books(b, in_place)
    got = w4.pages_fork(pool, *ins, ints(parents), ints(children), ps, out=out)
    *books_want, copies = ref.fork(*b, parents, children, ps)
    assert len(copies) == 18 and 0 in books_want[3]
    same(got, books_want)
    for a, z in copies:
        inner[:, z] = inner[:, a]
    assert torch.equal(wide, want)


@pytest.mark.parametrize("aside", [False, True])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_listed_rows_out_of_range(w4lib, dtype, aside):
    """A PagedCache passes them over: no token of theirs is written, and their attention is that
    of an empty row; the rows beside them are served."""
    cache = w4.PagedCache(1, 3, 12, 2, 64, page_size=16, max_length=64)
    g = torch.Generator(device="cuda").manual_seed(4)
    cache.pool.normal_(generator=g)
    cache.extend(ints([0, 2]), ints([20, 33]))
    listed = torch.tensor([-1, 2, 3, 0, 2 ** 31 - 1, -2 ** 31], dtype=dtype, device="cuda")
    starts, offsets = ints([0, 30, 0, 18, 5, 3]), ints([0, 4, 7, 9, 11, 12, 20])
    k, v = (torch.randn(20, 2, 64, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(6, 8, 64, generator=g, device="cuda").half()
    want = cache.pool.clone()
    for row, start, first, count in ((2, 30, 4, 3), (0, 18, 9, 2)):
        for i in range(count):
            page = int(cache.tables[row, (start + i) // 16])
            want[0, page, (start + i) % 16] = k[first + i]
            want[1, page, (start + i) % 16] = v[first + i]
    x = w4.paged_attention(q[[1, 3]], want[0], want[1], cache.tables[[2, 0]], cache.lengths[[2, 0]])
    stream = torch.cuda.Stream() if aside else None
    torch.cuda.synchronize()
    cache.append(0, k, v, starts, offsets, rows=listed, stream=stream)
    out = cache.attend(0, q, rows=listed, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(cache.pool, want)
    assert torch.equal(out[[1, 3]], x) and (out[[0, 2, 4, 5]] == 0).all()
    assert starts.tolist() == [0, 30, 0, 18, 5, 3]


@pytest.mark.parametrize("width", [1, 3, 1023, 1025, 5000])
def test_listed_rows_of_wide_tables(w4lib, width):
    """More rows and columns than one piece, from a slice of a wider table."""
    g = torch.Generator(device="cuda").manual_seed(width)
    cache = w4.PagedCache(1, 70, 4 * width, 1, 8, page_size=1, max_length=width)
    wide = torch.randint(0, 4 * width, (70, width + 3), generator=g, device="cuda").int()
    cache.tables = wide[:, 1:width + 1]
    cache.lengths.random_(0, width + 1, generator=g)
    cache.pool.normal_(generator=g)
    listed = torch.randint(-3, 73, (300,), generator=g, device="cuda").int()
    q = torch.randn(300, 2, 8, generator=g, device="cuda").half()
    out = cache.attend(0, q, rows=listed)
    inside = (listed >= 0) & (listed < 70)
    at = listed[inside].long()
    want = w4.paged_attention(q[inside], cache.keys(0), cache.values(0),
                              cache.tables[at].contiguous(), cache.lengths[at])
    assert torch.allclose(out[inside].float(), want.float(), rtol=2.0 ** -9, atol=2.0 ** -12)
    assert (out[~inside] == 0).all()
