"""Tokens that the attention of chunks has nothing for: of rows with fewer positions than
tokens, in any number and beside any rows; tolerances as in test_chunk_attention."""
from __future__ import annotations

import math

import pytest
import torch

import w4a16_weight_only_gemm_gb300 as w4
from test_chunk_attention import check, ints, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv_heads, group, dim", [(8, 4, 128), (4, 7, 64), (1, 1, 8), (2, 9, 136),
                                                  (1, 300, 64), (3, 5, 96)])
def test_rows_with_fewer_positions_than_tokens(w4lib, kv_heads, group, dim, dtype):
    """From none to all of a row's tokens, with items' edges on both sides of position 0."""
    rows = [(40, 20), (0, 300), (0, 257), (100, 1), (0, 130), (0, 64), (0, 5), (64, 64)]
    if group > 30:
        rows = rows[:1] + rows[3:]
    q, k, v, tables, lengths, offsets = make(rows, kv_heads, group, dim, 16, dtype, seed=dim,
                                             garbage=0.0)
    all_there = w4.paged_chunk_attention(q, k, v, tables, lengths, offsets)
    for short in (1, 32, 63, 100, 129, 10 ** 6):
        less = torch.where(torch.arange(len(rows), device="cuda") % 2 == 1,
                           (lengths - short).clamp(min=0), lengths).int()
        out = check(q, k, v, tables, less, offsets)
        for b, (held, n) in enumerate(rows):
            at = slice(int(offsets[b]), int(offsets[b + 1]))
            none = max(n - int(less[b]), 0)
            assert (out[at][:none] == 0).all()
            if b % 2 == 0:
                u = 2.0 ** -10 if dtype == torch.float16 else 2.0 ** -7
                far = (out[at].float() - all_there[at].float()).abs().max()
                assert far <= 2 * u * v.abs().max()


def test_a_long_chunk_on_a_row_of_no_length(w4lib):
    """512 MB of zeros beside two rows whose attention waits for nothing: well within a limit of
    5 ms on every wait, and strided outputs are left alone elsewhere."""
    n = 65536
    q, k, v, tables, lengths, offsets = make([(700, 64), (0, 0), (300, 9)], 8, 4, 128, 16,
                                             torch.float16, garbage=0.0)
    plain = w4.paged_chunk_attention(q, k, v, tables, lengths, offsets)
    q = torch.cat([q[:64], torch.full((n, 32, 128), math.nan, device="cuda").half(), q[64:]])
    offsets = ints([0, 64, 64 + n, 73 + n])
    out = torch.full((n + 73, 33, 128), 7.0, device="cuda", dtype=torch.float16)
    w4.set_wait_timeout_ns(5_000_000)
    try:
        _, lse = w4.paged_chunk_attention(q, k, v, tables, lengths, offsets, out=out[:, :32],
                                          return_lse=True)
        torch.cuda.synchronize()
    finally:
        w4.set_wait_timeout_ns(2_000_000_000)
    assert w4.device_status() == 0
    assert not out[64:64 + n, :32].any() and (out[:, 32] == 7).all()
    assert (lse[64:64 + n] == -math.inf).all() and torch.isfinite(lse[:64]).all()
    far = 4 * 2.0 ** -11 * v.abs().max()
    assert (out[:64, :32].float() - plain[:64].float()).abs().max() <= far
    assert (out[64 + n:, :32].float() - plain[64:].float()).abs().max() <= far


def test_listed_rows_that_are_out_of_range(w4lib):
    """PagedCache.attend_chunks: a row that does not exist has no positions."""
    cache = w4.PagedCache(layers=1, rows=2, pages=40, kv_heads=2, head_dim=64, max_length=256)
    assert cache.extend(ints([0, 1]), ints([30, 200])).tolist() == [1, 1]
    g = torch.Generator().manual_seed(5)
    kv = torch.randn(230, 4, 64, generator=g).half().cuda()
    cache.append(0, kv[:, :2], kv[:, 2:], ints([0, 0]), ints([0, 30, 230]))
    q = torch.randn(5000, 8, 64, generator=g).half().cuda()
    out = cache.attend_chunks(0, q, ints([0, 10, 4990, 5000]), rows=ints([0, 9, 1]))
    one = cache.attend_chunks(0, q[:10], ints([0, 10]), rows=ints([0]))
    two = cache.attend_chunks(0, q[4990:], ints([0, 10]), rows=ints([1]))
    assert not out[10:4990].any() and torch.isfinite(out).all()
    for got, want in ((out[:10], one), (out[4990:], two)):
        assert (got.float() - want.float()).abs().max() <= 4 * 2.0 ** -11 * kv.abs().max()
