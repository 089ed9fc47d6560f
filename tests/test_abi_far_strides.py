"""Strides so far apart that their products pass 64 bits, on a CPU-only host: what shares
values is refused, and what does not is taken (told by the check behind it, of the alignment)."""
from __future__ import annotations

import pytest

from test_abi_prompt import MISALIGNED, FAKE, cache, heads, lib, query, rotary  # noqa: F401

FAR = 1 << 40
# (tokens, token stride, heads, head stride): tokens - 1 strides are 2^64, 2^65, 2^63 or just past
SHARED = [((1 << 24) + 1, FAR, 1024, 1 << 31), ((1 << 25) + 1, FAR, 1024, 1 << 31),
          ((1 << 23) + 1, FAR, 1024, 1 << 31), ((1 << 24) + 2, FAR, 512, 1 << 32),
          ((1 << 31) - 1, FAR, 2, FAR), (1 << 31, FAR - 8, 1024, FAR)]
APART = [((1 << 24) + 1, FAR, 1024, 1 << 30), (1 << 24, 64, 1024, 1 << 30),
         ((1 << 31) - 1, 64, 2, 1 << 37), (1 << 31, FAR, 1, 0)]


def call(lib, tokens, row, n, head, out):
    h = heads(tokens=tokens, heads=n, row=64 * n, o_row=row, o_head=head)
    return {lib.w4a16_rotate(FAKE, FAKE, FAKE, out, rotary(), h, None),
            lib.w4a16_paged_append_rotary(*(FAKE,) * 7, FAKE, FAKE, out, cache(), rotary(), h, 128, 64,
                                          128, 64, None)}


@pytest.mark.parametrize("sizes", SHARED)
def test_far_heads_that_share_values_are_refused(lib, sizes):  # noqa: F811
    assert call(lib, *sizes, MISALIGNED) == {2}


@pytest.mark.parametrize("sizes", APART)
def test_far_heads_that_share_none_are_taken(lib, sizes):  # noqa: F811
    assert call(lib, *sizes, MISALIGNED) == {3}


def test_the_attentions_outputs(lib):  # noqa: F811
    def attend(tokens, row, head, n=32):
        return lib.w4a16_paged_chunk_attention(*[FAKE] * 6, MISALIGNED, None, FAKE, cache(),
                                               query(heads=n, o_row=row, o_head=head), tokens, None)

    assert attend(1 << 24, FAR, 1 << 38) == 2
    assert attend((1 << 23) + 1, FAR, 1 << 36) == 2
    assert attend(1 << 24, FAR, 1 << 34) == 3
    assert attend(1 << 24, 64, 1 << 30) == 3
