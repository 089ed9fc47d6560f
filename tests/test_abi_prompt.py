"""The prompt-side entry points of the C ABI on a CPU-only host: bad arguments are
refused synchronously, before any device is touched."""
from __future__ import annotations

import math
import struct

import pytest

from w4a16_weight_only_gemm_gb300 import _native, build
from test_abi_serving import BAD_CACHES, FAKE, MISALIGNED, cache, query


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


def rotary(dims=64, interleaved=0, magnitude=1.0):
    return struct.pack("2qd", dims, interleaved, magnitude)


def heads(tokens=5, heads=8, dim=64, type=0, row=512, head=64, o_row=512, o_head=64):
    return struct.pack("8q", tokens, heads, dim, type, row, head, o_row, o_head)


BAD_ROTARIES = [dict(dims=0), dict(dims=7), dict(dims=66), dict(interleaved=2),
                dict(magnitude=math.nan), dict(magnitude=math.inf)]
BAD_HEADS = [dict(heads=0), dict(heads=1025), dict(dim=0), dict(dim=12), dict(dim=264),
             dict(row=4), dict(row=-8), dict(head=9), dict(o_row=1), dict(o_head=-8)]


def test_rotate_arguments(lib):
    def call(p=(FAKE,) * 4, r=rotary(), h=heads()):
        return lib.w4a16_rotate(*p, r, h, None)

    for i in range(4):
        assert call([None if j == i else FAKE for j in range(4)]) == 1
    for i in (0, 3):
        p = [FAKE] * 3 + [FAKE + 16]
        p[i] = MISALIGNED
        assert call(p) == 3
    assert call(r=None) == 1 and call(h=None) == 1
    for bad in BAD_ROTARIES:
        assert call(r=rotary(**bad)) == 2
    for bad in BAD_HEADS + [dict(tokens=-1), dict(tokens=(1 << 31) + 1), dict(type=3),
                            dict(type=-1)]:
        assert call(h=heads(**bad)) == 2
    # the input's place with other strides
    assert call(h=heads(o_row=1024)) == 2 and call(h=heads(o_head=128)) == 2
    assert call((None,) * 4, h=heads(tokens=0)) == 0


def test_append_rotary_arguments(lib):
    def call(p=(FAKE,) * 7, at=FAKE, q=(FAKE, FAKE + 16), c=cache(), r=rotary(), h=heads(),
             strides=(128, 64, 128, 64)):
        return lib.w4a16_paged_append_rotary(*p, at, *q, c, r, h, *strides, None)

    for i in range(7):
        assert call([None if j == i else FAKE for j in range(7)]) == 1
    for i in (0, 1, 3, 4):
        assert call([MISALIGNED if j == i else FAKE for j in range(7)]) == 3
    assert call(q=(FAKE, None)) == 1 and call(q=(None, FAKE)) == 1
    assert call(q=(MISALIGNED, FAKE)) == 3 and call(q=(FAKE, MISALIGNED)) == 3
    assert call(c=None) == 1 and call(r=None) == 1 and call(h=None) == 1
    assert call(at=None) == 2                                    # 5 tokens, 3 rows
    for i in range(4):
        assert call(strides=tuple(4 if j == i else 64 for j in range(4))) == 2
        assert call(strides=tuple(-8 if j == i else 64 for j in range(4))) == 2
    for bad in BAD_CACHES:
        assert call(c=cache(**bad)) == 2
    for bad in BAD_ROTARIES:
        assert call(r=rotary(**bad)) == 2
    for bad in BAD_HEADS + [dict(tokens=-1), dict(type=1), dict(dim=128)]:
        assert call(h=heads(**bad)) == 2
    assert call(q=(FAKE, FAKE), h=heads(o_row=1024)) == 2
    assert call((None,) * 7, None, (None, None), c=cache(batch=3), h=heads(tokens=0)) == 2
    assert call((None,) * 7, FAKE, (None, None), h=heads(tokens=0)) == 0


def test_chunk_arguments(lib):
    pointers = [FAKE] * 7 + [None, FAKE]

    def call(p=pointers, c=cache(), q=query(), tokens=5):
        return lib.w4a16_paged_chunk_attention(*p, c, q, tokens, None)

    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        assert call([None if j == i else p for j, p in enumerate(pointers)]) == 1
    for i in (0, 1, 2, 6, 8):
        assert call([MISALIGNED if j == i else p for j, p in enumerate(pointers)]) == 3
    assert call(c=None) == 1 and call(q=None) == 1
    for bad in BAD_CACHES:
        assert call(c=cache(**bad)) == 2
        assert lib.w4a16_paged_chunk_workspace(cache(**bad), 8, 5) == -1
    for bad in (dict(heads=0), dict(heads=7), dict(heads=1026), dict(q_row=5), dict(q_head=-8),
                dict(o_row=4), dict(o_head=1), dict(scale=math.nan)):
        assert call(q=query(**bad)) == 2
    for tokens in (-1, (1 << 24) + 1):
        assert call(tokens=tokens) == 2
        assert lib.w4a16_paged_chunk_workspace(cache(), 8, tokens) == -1
    assert call(c=cache(kv=1, head=64), q=query(heads=1024), tokens=1 << 22) == 2
    assert lib.w4a16_paged_chunk_workspace(None, 8, 5) == -1
    assert lib.w4a16_paged_chunk_workspace(cache(), 7, 5) == -1
    assert call([None] * 9, tokens=0) == 0


def tensors(**given):
    names = ("logits", "tokens", "lengths", "prompts", "repetition", "presence", "frequency",
             "bias_ids", "biases", "mask", "out")
    return struct.pack("11Q", *({"logits": FAKE, "out": FAKE + 64, **given}.get(n, 0)
                                for n in names))


def sizes(rows=3, vocabulary=100, type=0, stride=100, out=100, wide=0, width=5, tokens=5, biases=4,
          bias=4, mask=4):
    return struct.pack("11q3d", rows, vocabulary, type, stride, out, wide, width, tokens, biases,
                       bias, mask, 1.0, 0.0, 0.0)


def test_adjust_arguments(lib):
    def call(t=tensors(), s=sizes()):
        return lib.w4a16_adjust_logits(t, s, None)

    assert call(t=None) == 1 and call(s=None) == 1
    assert call(tensors(logits=0)) == 1 and call(tensors(out=0)) == 1
    assert call(tensors(bias_ids=FAKE)) == 1
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(vocabulary=0),
                dict(vocabulary=(1 << 30) + 1), dict(type=3), dict(type=-1), dict(stride=-1),
                dict(out=-1), dict(wide=2), dict(width=-1), dict(width=1 << 30), dict(tokens=-1),
                dict(biases=-1), dict(biases=1025), dict(bias=-4), dict(mask=-4)):
        assert call(s=sizes(**bad)) == 2
    assert call(tensors(out=FAKE), sizes(out=104)) == 2          # the input's place, another stride
    assert call(tensors(logits=FAKE + 1)) == 3 and call(tensors(out=FAKE + 1)) == 3
    assert call(tensors(logits=FAKE + 2), sizes(type=2)) == 3


# Strides of 5 tokens of 8 heads of 64 (tokens, heads) in which heads share values, and ones in
# which none do.
SHARED = [(0, 64), (512, 0), (0, 0), (512, 56), (504, 64), (448, 64), (64, 312), (56, 320), (64, 0)]
APART = [(512, 64), (520, 64), (1024, 128), (64, 320), (72, 352)]


def test_outputs_that_share_values_are_refused(lib):
    for row, head in SHARED:
        h = heads(o_row=row, o_head=head)
        assert lib.w4a16_rotate(*(FAKE,) * 3, FAKE + 16, rotary(), h, None) == 2
        assert lib.w4a16_paged_append_rotary(*(FAKE,) * 7, FAKE, FAKE, FAKE + 16, cache(), rotary(),
                                             h, 128, 64, 128, 64, None) == 2
        assert lib.w4a16_paged_chunk_attention(*[FAKE] * 7, None, FAKE, cache(),
                                               query(o_row=row, o_head=head), 5, None) == 2
    for out in (0, 1, 99):
        assert lib.w4a16_adjust_logits(tensors(), sizes(out=out), None) == 2


def test_outputs_that_share_no_value_are_taken(lib):
    # (told by the check behind the strides', of the alignment)
    for row, head in APART + [(0, 64)]:
        tokens = 5 if row else 1
        h = heads(tokens=tokens, o_row=row, o_head=head)
        assert lib.w4a16_rotate(*(FAKE,) * 3, MISALIGNED, rotary(), h, None) == 3
        assert lib.w4a16_paged_append_rotary(*(FAKE,) * 7, FAKE, FAKE, MISALIGNED, cache(), rotary(),
                                             h, 128, 64, 128, 64, None) == 3
        assert lib.w4a16_paged_chunk_attention(*[FAKE] * 6, MISALIGNED, None, FAKE, cache(),
                                               query(o_row=row, o_head=head), tokens, None) == 3
    assert lib.w4a16_adjust_logits(tensors(out=FAKE + 1), sizes(out=100), None) == 3
    assert lib.w4a16_adjust_logits(tensors(out=FAKE + 1), sizes(rows=1, out=0), None) == 3
