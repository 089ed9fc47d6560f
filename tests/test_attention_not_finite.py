"""Attention over queries, keys and values that are not finite, by clusters (tables as
wide as the rows) and by the cut line (tables much wider), against the 64-bit definition.

A head with a score that is NaN or +infinity has no softmax: NaN in its output and its
logarithm.  A position of score -infinity has no weight, as if it were masked: a head with
no other has zeros and -infinity, as in a row of length 0.  What is finite keeps the
tolerance of finite inputs, taken from the same case before anything was planted in it: a
score is off by at most E = dim * 2^-22 * sum |q k| scale (+ 2^-20 for the exponential),
the output by 4 E max|V| and its rounding."""
from __future__ import annotations

import math

import pytest
import torch

import paged_reference as ref
import w4a16_weight_only_gemm_gb300 as w4
from test_paged_attention import UNIT, make

pytestmark = pytest.mark.gpu

LENGTHS = [65, 1, 700, 64, 130, 0, 449, 1500]     # parts of one step, one position, many steps
KV, GROUP, DIM, PAGE = 2, 4, 64, 16


def spot(tables, row, position):
    return int(tables[row, position // PAGE]), position % PAGE


def check(case, planted):
    """The kernel on `planted` = (q, k_pool, v_pool); `case` is the finite one it came from."""
    _, _, v_clean, tables, lengths = case
    scale = DIM ** -0.5
    out, lse = w4.paged_attention(*planted, tables, lengths, return_lse=True)
    torch.cuda.synchronize()
    want, want_lse, _ = ref.attention(*planted, tables, lengths, scale)
    want[want_lse == -math.inf] = 0.0
    error = DIM * 2.0 ** -22 * ref.attention(*case, scale)[2] + 2.0 ** -20
    out, lse = out.cpu().double(), lse.cpu().double()
    # +infinity: its weight would be infinity / infinity
    none = torch.isnan(want_lse) | (want_lse == math.inf)
    assert torch.equal(torch.isnan(lse), none)
    held = torch.isfinite(want_lse)
    assert torch.equal(lse[~held & ~none], want_lse[~held & ~none])      # -infinity: no position
    off = (lse - want_lse)[held].abs()
    assert (off <= error[held] + 2.0 ** -20 * (1 + want_lse[held].abs())).all()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    infinite = torch.isinf(want)
    assert torch.equal(torch.isinf(out), infinite)
    assert torch.equal(out[infinite], want[infinite])
    v = torch.nan_to_num(v_clean.cpu().double(), 0, 0, 0).abs().max()
    far = (out - want).abs() - UNIT[case[0].dtype] * want.abs() - 4 * error[..., None] * v
    assert far[torch.isfinite(want)].max() <= 2.0 ** -24


@pytest.fixture(params=[torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def dtype(request):
    return request.param


@pytest.fixture(params=[None, 4000], ids=["clusters", "line"])
def case(w4lib, dtype, request):
    return make(LENGTHS, KV, GROUP, DIM, PAGE, dtype, seed=21, width=request.param)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_query(case, value):
    q = case[0].clone()
    q[0, 3, 5] = value
    q[2, 6, :] = value
    q[4, 0, 63] = value
    q[5, 1, 0] = value                             # of a row without a position
    check(case, (q, *case[1:3]))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["newest", "first", "middle"])
def test_one_key(case, value, where):
    """One held key; the newest of 65 positions is alone in its step."""
    k, tables = case[1].clone(), case[3]
    for row in (0, 1, 2, 4, 7):
        n = LENGTHS[row]
        page, slot = spot(tables, row, {"newest": n - 1, "first": 0, "middle": n // 2}[where])
        k[page, slot, 1, 7] = value
    check(case, (case[0], k, case[2]))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_all_keys_of_a_head(case, value):
    k, tables = case[1].clone(), case[3]
    for row in (0, 1, 2, 4):
        for p in range(LENGTHS[row]):
            page, slot = spot(tables, row, p)
            k[page, slot, 0, 3] = value
    q = case[0].clone()
    q[:, :KV * GROUP, 3] = q[:, :KV * GROUP, 3].abs() + 0.5    # all scores +infinity or -infinity
    check(case, (q, k, case[2]))


@pytest.mark.parametrize("values", [[math.inf], [-math.inf], [math.nan], [math.inf, math.inf],
                                    [math.inf, -math.inf], [math.inf, math.nan]], ids=str)
def test_values(case, values):
    """Infinite and missing values in held places: weights are above 0, so an infinity shows
    as it is, beside an opposite one or a NaN as NaN, in its own dimension alone."""
    v, tables = case[2].clone(), case[3]
    for row in (0, 1, 2, 4, 7):
        n = LENGTHS[row]
        for i, value in enumerate(values[:n]):
            for p in (n - 1 - i, i * (n // 3)):    # side by side, and steps apart
                page, slot = spot(tables, row, p)
                v[page, slot, 1, 9 + p % 5] = value
                v[page, slot, 0, 63] = value
    check(case, (*case[:2], v))


def test_values_of_equal_weight(w4lib, dtype):
    """Weights that 16 bits hold exactly, so that nothing is left over for a second part."""
    case = make(LENGTHS, KV, GROUP, DIM, PAGE, dtype, seed=22)
    case[0].zero_()
    v, tables = case[2].clone(), case[3]
    for row in (0, 1, 2, 4):
        page, slot = spot(tables, row, LENGTHS[row] - 1)
        v[page, slot, 0, :32] = math.inf
        v[page, slot, 0, 32:] = -math.inf
    check(case, (*case[:2], v))
