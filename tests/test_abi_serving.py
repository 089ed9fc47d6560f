"""The serving entry points of the C ABI on a CPU-only host: bad arguments are
refused synchronously, before any device is touched."""
from __future__ import annotations

import math
import struct

import pytest

from w4a16_weight_only_gemm_gb300 import _native, build

FAKE = 0x10000        # an aligned non-null pointer value; never dereferenced here
MISALIGNED = 0x10008


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def cache(pages=10, page=16, kv=2, dim=64, type=0, page_stride=2048, slot=128, head=64, batch=3,
          width=4, stride=4):
    return struct.pack("11q", pages, page, kv, dim, type, page_stride, slot, head, batch, width,
                       stride)


def query(heads=8, q_row=512, q_head=64, o_row=512, o_head=64, scale=0.125):
    return struct.pack("5qd", heads, q_row, q_head, o_row, o_head, scale)


BAD_CACHES = [dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(page=65537), dict(kv=0),
              dict(kv=1025), dict(dim=0), dict(dim=12), dict(dim=264), dict(type=2), dict(type=-1),
              dict(page_stride=4), dict(slot=-8), dict(head=9), dict(batch=0), dict(batch=65536),
              dict(width=0), dict(width=1 << 25), dict(width=1 << 24, page=128), dict(stride=-1)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_cache_shapes(lib, bad):
    c = cache(**bad)
    assert lib.w4a16_paged_append(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, c, 5, 128, 64, 128, 64,
                                  None) == 2
    assert lib.w4a16_paged_attention(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, c, query(),
                                     None) == 2
    assert lib.w4a16_paged_attention_workspace(c, 8) == -1


def test_append_arguments(lib):
    c = cache()

    def call(*p, tokens=5, strides=(128, 64, 128, 64), offsets=FAKE):
        p = p or (FAKE,) * 6
        return lib.w4a16_paged_append(*p, offsets, c, tokens, *strides, None)

    for i in range(6):
        assert call(*(None if j == i else FAKE for j in range(6))) == 1
    for i in range(4):
        assert call(*(MISALIGNED if j == i else FAKE for j in range(6))) == 3
        assert call(strides=tuple(4 if j == i else 64 for j in range(4))) == 2
        assert call(strides=tuple(-8 if j == i else 64 for j in range(4))) == 2
    assert call(tokens=-1) == 2
    assert call(offsets=None) == 2                               # 5 tokens, 3 rows
    assert call(None, None, None, None, None, None, tokens=0) == 0
    assert lib.w4a16_paged_append(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 5, 128, 64, 128,
                                  64, None) == 1


def test_attention_arguments(lib):
    pointers = [FAKE] * 6 + [None, FAKE]

    def call(p=pointers, c=cache(), q=query()):
        return lib.w4a16_paged_attention(*p, c, q, None)

    for i in (0, 1, 2, 3, 4, 5, 7):
        assert call([None if j == i else p for j, p in enumerate(pointers)]) == 1
    for i in (0, 1, 2, 5, 7):
        assert call([MISALIGNED if j == i else p for j, p in enumerate(pointers)]) == 3
    assert call(c=None) == 1 and call(q=None) == 1
    for bad in (dict(heads=0), dict(heads=7), dict(heads=1026), dict(q_row=5), dict(q_head=-8),
                dict(o_row=4), dict(o_head=1), dict(scale=math.nan)):
        assert call(q=query(**bad)) == 2


def books(pages=10, rows=4, width=3, in_stride=3, out_stride=3, page=16):
    return struct.pack("6q", pages, rows, width, in_stride, out_stride, page)


def pool(planes=2, plane=1600, page=160, size=160):
    return struct.pack("4q", planes, plane, page, size)


@pytest.mark.parametrize("bad", [dict(pages=0), dict(pages=1 << 31), dict(rows=0),
                                 dict(rows=(1 << 24) + 1), dict(width=0), dict(width=(1 << 24) + 1),
                                 dict(in_stride=-1), dict(out_stride=2), dict(page=0),
                                 dict(page=65537), dict(width=1 << 20, out_stride=1 << 20,
                                                        page=4096)], ids=str)
def test_books_shapes(lib, bad):
    b = books(**bad)
    assert lib.w4a16_pages_workspace(b, 2) == -1
    assert lib.w4a16_pages_free(*[FAKE] * 4, 2, *[FAKE] * 3, b, None) == 2
    assert lib.w4a16_pages_extend(*[FAKE] * 5, 2, *[FAKE] * 5, b, None) == 2
    assert lib.w4a16_pages_fork(*[FAKE] * 6, 2, *[FAKE] * 5, b, pool(), None) == 2
    assert lib.w4a16_pages_compact(*[FAKE] * 7, b, pool(), None) == 2


@pytest.mark.parametrize("bad", [dict(planes=0), dict(plane=8), dict(page=-16), dict(page=20),
                                 dict(size=0), dict(size=24)], ids=str)
def test_pool_shapes(lib, bad):
    p = pool(**bad)
    assert lib.w4a16_pages_fork(*[FAKE] * 6, 2, *[FAKE] * 5, books(), p, None) == 2
    assert lib.w4a16_pages_compact(*[FAKE] * 7, books(), p, None) == 2
    assert lib.w4a16_pages_copy(FAKE, FAKE, FAKE, 2, 10, p, None) == 2


def test_pages_arguments(lib):
    assert lib.w4a16_pages_workspace(None, 0) == -1
    assert lib.w4a16_pages_workspace(books(), -1) == -1
    assert lib.w4a16_pages_workspace(books(), 0) > 0
    for i in range(7):
        p = [None if j == i else FAKE for j in range(7)]
        assert lib.w4a16_pages_free(*p[:4], 2, *p[4:], books(), None) == 1
        assert lib.w4a16_pages_compact(*p, books(), pool(), None) == 1
    for i in range(10):
        p = [None if j == i else FAKE for j in range(10)]
        assert lib.w4a16_pages_extend(*p[:5], 2, *p[5:], books(), None) == 1
    for i in range(11):
        p = [None if j == i else FAKE for j in range(11)]
        assert lib.w4a16_pages_fork(*p[:6], 2, *p[6:], books(), pool(), None) == 1
    for i in range(3):
        p = [None if j == i else FAKE for j in range(3)]
        assert lib.w4a16_pages_copy(*p, 2, 10, pool(), None) == 1
    assert lib.w4a16_pages_free(*[FAKE] * 4, -1, *[FAKE] * 3, books(), None) == 2
    assert lib.w4a16_pages_extend(*[FAKE] * 5, (1 << 24) + 1, *[FAKE] * 5, books(), None) == 2
    assert lib.w4a16_pages_copy(FAKE, FAKE, FAKE, 2, 0, pool(), None) == 2
    assert lib.w4a16_pages_copy(MISALIGNED, FAKE, FAKE, 2, 10, pool(), None) == 3
    assert lib.w4a16_pages_fork(MISALIGNED, *[FAKE] * 5, 2, *[FAKE] * 5, books(), pool(), None) == 3
    assert lib.w4a16_pages_compact(*[FAKE] * 6, MISALIGNED, books(), pool(), None) == 3


def test_logprobs_arguments(lib):
    def call(*p, rows=2, n=100, stride=100, type=0, wide=1, top=5):
        return lib.w4a16_token_logprobs(*(p or [FAKE] * 6), rows, n, stride, type, wide, top, None)

    for i in range(6):
        assert call(*(None if j == i else FAKE for j in range(6))) == 1
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(n=0), dict(n=(1 << 30) + 1),
                dict(stride=-1), dict(type=3), dict(type=-1), dict(wide=2), dict(top=-1),
                dict(top=33), dict(n=4, top=5)):
        assert call(**bad) == 2
    assert call(FAKE + 1, *[FAKE] * 5) == 3
    assert call(FAKE + 2, *[FAKE] * 5, type=2) == 3


def test_pages_workspaces(lib):
    """Small pools need none where the books are written apart; else both ask for some."""
    fork, compact = lib.w4a16_pages_fork_workspace, lib.w4a16_pages_compact_workspace
    assert fork(books(), pool(), 2, 1) == 0 and compact(books(), pool(), 1) == 0
    assert fork(books(), pool(), 2, 0) > 0 and compact(books(), pool(), 0) > 0
    large = books(pages=100000)
    assert fork(large, pool(), 2, 1) > 0 and compact(large, pool(), 1) > 0
    assert fork(books(pages=0), pool(), 2, 1) == -1 and fork(books(), pool(size=8), 2, 1) == -1
    assert fork(books(), pool(), -1, 1) == -1 and fork(None, pool(), 2, 1) == -1
    assert compact(books(), None, 1) == -1


def test_listed_rows_arguments(lib):
    def call(p, b=books(), count=2):
        return lib.w4a16_pages_rows(*p[:3], count, *p[3:], b, None)

    for i in (0, 1, 2, 3):                       # a NULL lengths_out asks for none
        assert call([None if j == i else FAKE for j in range(5)]) == 1
    assert call([FAKE] * 5, None) == 1
    assert call([FAKE] * 5, count=-1) == 2 and call([FAKE] * 5, count=(1 << 24) + 1) == 2
    for bad in (dict(rows=0), dict(width=0), dict(in_stride=-1), dict(out_stride=2)):
        assert call([FAKE] * 5, books(**bad)) == 2
