"""Rotary positions, alone and on the way into the paged cache, against the 64-bit
definition with angles reduced exactly.

Tolerance, from the arithmetic: an angle's fraction of a turn is rounded to FP32
(2^-24 of at most pi) and its cosine and sine are off by an ulp more, so each is off
by at most 2^-22; two products and a sum add 2^-23 of |a| + |b| at most.  So a value
is off by 2^-21 (|a| + |b|) m, and is rounded once, by u |out| (u = 2^-11 for fp16,
2^-8 for bf16, 2^-24 for fp32)."""
from __future__ import annotations

import math

import pytest
import torch

import prompt_reference as ref
import w4a16_weight_only_gemm_gb300 as w4

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = list(UNIT)
gpu = pytest.mark.gpu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def near(got, want, bound):
    got = got.cpu()
    far = (got.double() - want).abs() - UNIT[got.dtype] * want.abs() - 2.0 ** -21 * bound
    # below fp16's normal numbers a rounding is half of 2^-24
    assert far.max() <= (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -140)


def check(x, positions, rotary, **kw):
    before = x.clone()
    got = w4.rotate(x, positions, rotary, **kw)
    torch.cuda.synchronize()
    want, bound = ref.rotate(before, positions.tolist(), rotary.rates, rotary.interleaved,
                             rotary.magnitude)
    near(got, want, bound)
    n = rotary.dim
    assert torch.equal(got[..., n:], before[..., n:])
    return got


# --- the rates (CPU) ---------------------------------------------------------
def test_rates():
    plain = w4.Rotary(8, base=100.0, device="cpu")
    assert plain.rates == pytest.approx([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rel=1e-15)
    linear = w4.Rotary(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert linear.rates == pytest.approx([r / 4 for r in plain.rates], rel=1e-15)
    base = w4.Rotary(8, base=100.0, scaling="base", factor=16.0, device="cpu")
    assert base.rates[0] == 1.0
    assert base.rates[3] == pytest.approx(plain.rates[3] / 16.0, rel=1e-14)
    ramp = w4.Rotary(8, base=100.0, scaling="ramp", factor=4.0, original=60, low=1.0, high=5.0,
                     device="cpu")
    turns = [60 * r / (2 * math.pi) for r in plain.rates]   # 9.55, 3.02, 0.95, 0.30
    assert ramp.rates[0] == plain.rates[0]
    keep = (turns[1] - 1) / 4
    assert ramp.rates[1] == pytest.approx(plain.rates[1] * (keep + (1 - keep) / 4), rel=1e-14)
    assert ramp.rates[2:] == pytest.approx([r / 4 for r in plain.rates[2:]], rel=1e-15)
    own = w4.Rotary(4, rates=[0.25, -3.0], device="cpu")
    assert own.rates == [0.25, -3.0]
    # a fraction of a turn times 2^64, off by half of its last bit
    for t, r in zip(own.turns.tolist(), own.rates):
        exact = r * ref.INVERSE_TURN * 2 ** 64
        assert abs((t - exact + 2 ** 63) % 2 ** 64 - 2 ** 63) <= 0.5 + 1e-6


@pytest.mark.parametrize("bad", [dict(dim=0), dict(dim=7), dict(base=0.0), dict(factor=0.0),
                                 dict(scaling="other"), dict(dim=2, scaling="base"),
                                 dict(scaling="ramp"), dict(scaling="ramp", original=-1),
                                 dict(scaling="ramp", original=9, low=4.0, high=4.0),
                                 dict(rates=[1.0]), dict(rates=[1.0, math.inf, 0.0, 0.0]),
                                 dict(rates=[1.0] * 4, scaling="linear"),
                                 dict(magnitude=math.nan)], ids=str)
def test_refused_rotations(bad):
    with pytest.raises(ValueError):
        w4.Rotary(**{"dim": 8, "device": "cpu", **bad})


def test_refused_calls():
    r = w4.Rotary(8, device="cpu")
    x, p = torch.zeros(3, 2, 16).half(), torch.zeros(3, dtype=torch.int32)
    for bad in (lambda: w4.rotate(x[0], p, r), lambda: w4.rotate(x.double(), p, r),
                lambda: w4.rotate(x[..., :4], p, r), lambda: w4.rotate(x, p.long(), r),
                lambda: w4.rotate(x, p[:2], r), lambda: w4.rotate(x, p, r),
                lambda: w4.rotate(x, p, r, out=x[:2]),
                lambda: w4.rotate(x.transpose(1, 2), p, w4.Rotary(2, device="cpu"))):
        with pytest.raises(ValueError):
            bad()
    pool, tables = torch.zeros(4, 16, 2, 16).half(), torch.zeros(3, 2, dtype=torch.int32)
    for bad in (dict(q=x[:2]), dict(q=x[..., :8]), dict(out=x), dict(q=x, out=x[:, :1]),
                dict(starts=p.long()), dict(offsets=p), dict(k=x[:2], v=x[:2]),
                dict(k=x[:, :1]), dict(rotary=w4.Rotary(32, device="cpu")), dict(v=x.bfloat16()),
                dict()):
        args = dict(k=x, v=x, k_pool=pool, v_pool=pool, tables=tables, starts=p, rotary=r)
        with pytest.raises(ValueError):
            w4.paged_append_rotary(**{**args, **bad})


# --- rotate ------------------------------------------------------------------
@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim, part", [(8, 2), (8, 8), (16, 6), (64, 64), (64, 12), (80, 20),
                                       (96, 24), (96, 96), (128, 128), (128, 64), (256, 256),
                                       (256, 34), (136, 130)])
def test_sizes(w4lib, dim, part, interleaved, dtype):
    g = torch.Generator().manual_seed(dim + part)
    for tokens, heads in ((1, 1), (3, 40), (70, 5)):
        x = torch.randn(tokens, heads, dim, generator=g).to(dtype).cuda()
        positions = ints(torch.randint(0, 9000, (tokens,), generator=g).tolist())
        check(x, positions, w4.Rotary(part, interleaved=interleaved, magnitude=1.25))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_far_positions(w4lib, dtype):
    """Also at the ends of 32 bits, and rates above half a turn."""
    positions = [0, 1, -1, 131071, -131072, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]
    x = torch.randn(len(positions), 3, 64, generator=torch.Generator().manual_seed(1))
    rates = [10000.0 ** (-i / 30) for i in range(28)] + [3.2, 6.5, -2.0, 1e-12]
    for interleaved in (False, True):
        check(x.to(dtype).cuda(), ints(positions),
              w4.Rotary(64, interleaved=interleaved, rates=rates))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_in_place(w4lib, dtype):
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(50, 14, 96, generator=g).to(dtype).cuda()
    positions, r = ints(list(range(100, 150))), w4.Rotary(48)
    plain = check(wide[:, 2:9].contiguous(), positions, r)
    assert torch.equal(w4.rotate(wide[:, 2:9], positions, r), plain)
    turned = wide.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(w4.rotate(turned[:, 2:9], positions, r), plain)
    kept = wide.clone()
    out = torch.full((50, 9, 104), 7.0, device="cuda", dtype=dtype)
    got = w4.rotate(wide[:, 2:9], positions, r, out=out[:, 1:8, :96])
    assert torch.equal(got, plain) and (out[:, 0] == 7).all() and (out[:, 8] == 7).all()
    assert (out[:, :, 96:] == 7).all()
    some = w4.rotate(wide[:, 2:9], positions, r, out=wide[:, 2:9])
    assert some.data_ptr() == wide[:, 2:9].data_ptr() and torch.equal(wide[:, 2:9], plain)
    assert torch.equal(wide[:, :2], kept[:, :2]) and torch.equal(wide[:, 9:], kept[:, 9:])
    with pytest.raises(w4._native.W4A16Error):     # the input's place with other strides
        w4.rotate(wide[:7, :7], positions[:7], r, out=wide[:7, :7].transpose(0, 1))


@gpu
def test_a_rotation_and_its_gradient(w4lib):
    """Back to where it was by the opposite positions, and the definition's gradient."""
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(20, 4, 32, generator=g).cuda() for _ in range(2))
    positions, r = ints(list(range(0, 200, 10))), w4.Rotary(24, interleaved=True, magnitude=1.5)
    back = w4.rotate(w4.rotate(x, positions, r), -positions, r)
    assert (back[..., :24] / 2.25 - x[..., :24]).abs().max() < 2.0 ** -18
    # sum(dy * rotate(x)) is linear in x: its gradient by the definition, one basis at a time
    dx = w4.rotate(dy, -positions, r).cpu().double()
    for d in range(32):
        e = torch.zeros(20, 4, 32, dtype=torch.float64)
        e[..., d] = 1.0
        turned, _ = ref.rotate(e, positions.tolist(), r.rates, True, 1.5)
        want = (turned * dy.cpu().double()).sum(-1)
        assert (dx[..., d] - want).abs().max() <= 2.0 ** -20 * dy.abs().max().item() * 3


@gpu
def test_what_is_not_finite_stays_in_its_pair(w4lib):
    x = torch.ones(4, 2, 16, device="cuda").half()
    x[0, 0, 3], x[1, 1, 4], x[2, 0, 15] = math.nan, math.inf, -math.inf
    y = w4.rotate(x, ints([0, 5, 6, 7]), w4.Rotary(8))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 7]] = want[1, 1, [0, 4]] = want[2, 0, 15] = True
    assert torch.equal(bad, want)


@gpu
def test_many_tokens(w4lib):
    """Every block size, against the same call a token at a time in a few places."""
    r = w4.Rotary(64)
    for tokens in (600, 1217, 5000, 20011):
        x = torch.randn(tokens, 6, 64, device="cuda").bfloat16()
        positions = torch.randint(0, 10 ** 6, (tokens,), device="cuda", dtype=torch.int32)
        y = w4.rotate(x, positions, r)
        for t in (0, 1, tokens // 2, tokens - 1):
            assert torch.equal(w4.rotate(x[t:t + 1], positions[t:t + 1], r), y[t:t + 1])
    assert w4.rotate(x[:0], positions[:0], r).shape == (0, 6, 64)


# --- the append --------------------------------------------------------------
ROWS = [(0, 1), (0, 0), (5, 3), (63, 2), (0, 130), (127, 1), (128, 33), (1000, 17)]


def append(rows, kv_heads, group, dim, page, dtype, r, layout="slots", offsets=True, seed=0,
           q_heads=None):
    """One call, checked against the definition; (arguments, outputs)."""
    k_pool, v_pool, tables, lengths, at = ref.cache(rows, kv_heads, dim, page, dtype, layout, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q_heads = kv_heads * group if q_heads is None else q_heads
    tokens = int(at[-1])
    qkv = torch.randn(tokens, q_heads + 2 * kv_heads, dim, generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    starts = ints([held for held, _ in rows])
    want_k, want_v = k_pool.clone(), v_pool.clone()
    out = w4.paged_append_rotary(k, v, k_pool, v_pool, tables, starts, r,
                                 offsets=at if offsets else None, q=q)
    torch.cuda.synchronize()
    positions = [p for held, new in rows for p in range(held, held + new)]
    row = [b for b, (_, new) in enumerate(rows) for _ in range(new)]
    where = [(int(tables[b, p // page]), p % page) for b, p in zip(row, positions)]
    near(out, *ref.rotate(q, positions, r.rates, r.interleaved, r.magnitude))
    turned, bound = ref.rotate(k, positions, r.rates, r.interleaved, r.magnitude)
    g_, s_ = (torch.tensor(x) for x in zip(*where))
    near(k_pool[g_, s_], turned, bound)
    want_v[g_, s_] = v
    assert torch.equal(v_pool[g_, s_], v)
    assert torch.equal(v_pool.view(torch.int16), want_v.view(torch.int16))
    k_pool[g_, s_] = 0
    want_k[g_, s_] = 0                           # nothing else was touched
    assert torch.equal(k_pool.view(torch.int16), want_k.view(torch.int16))


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv_heads, group, dim, part", [(8, 4, 128, 128), (4, 7, 128, 64),
                                                        (1, 1, 64, 64), (3, 5, 96, 24),
                                                        (2, 2, 256, 256), (2, 8, 64, 10),
                                                        (1, 1, 8, 2)])
def test_append(w4lib, kv_heads, group, dim, part, dtype):
    r = w4.Rotary(part, interleaved=group % 2 == 1, magnitude=1.0 + group / 8)
    append(ROWS, kv_heads, group, dim, 16, dtype, r, seed=dim)


@gpu
@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("page", [1, 8, 13, 64])
def test_append_pages(w4lib, page, layout):
    append(ROWS, 2, 4, 64, page, torch.float16, w4.Rotary(64), layout, seed=page)


@gpu
def test_append_one_token_a_row(w4lib):
    append([(7 * i, 1) for i in range(50)], 2, 4, 64, 16, torch.bfloat16, w4.Rotary(64),
           offsets=False)


@gpu
def test_append_agrees_with_its_parts(w4lib):
    """rotate, then paged_append: the same bits in the pools and the queries."""
    rows = [(i % 37, 1 + 97 * i % 300) for i in range(20)]
    k_pool, v_pool, tables, _, at = ref.cache(rows, 2, 128, 16, torch.float16, garbage=0.0)
    n = int(at[-1])
    qkv = torch.randn(n, 12, 128, device="cuda").half()
    starts, r = ints([h for h, _ in rows]), w4.Rotary(128, scaling="linear", factor=4.0)
    positions = ints([p for h, m in rows for p in range(h, h + m)])
    held, pools = k_pool.clone(), (k_pool.clone(), v_pool.clone())
    turned = w4.rotate(qkv[:, :10], positions, r)
    w4.paged_append(turned[:, 8:], qkv[:, 10:], *pools, tables, starts, at)
    got = w4.paged_append_rotary(qkv[:, 8:10], qkv[:, 10:], k_pool, v_pool, tables, starts, r, at,
                                 q=qkv[:, :8])
    assert torch.equal(got, turned[:, :8])
    assert torch.equal(k_pool, pools[0]) and torch.equal(v_pool, pools[1])
    # without queries, and with them in place
    k_pool.copy_(held)
    assert w4.paged_append_rotary(qkv[:, 8:10], qkv[:, 10:], k_pool, v_pool, tables, starts, r,
                                  at) is None
    assert torch.equal(k_pool, pools[0])
    same = w4.paged_append_rotary(qkv[:, 8:10], qkv[:, 10:], k_pool, v_pool, tables, starts, r, at,
                                  q=qkv[:, :8], out=qkv[:, :8])
    assert same.data_ptr() == qkv.data_ptr() and torch.equal(qkv[:, :8], turned[:, :8])


@gpu
def test_append_what_has_no_place(w4lib):
    """Tokens of no row, positions past the table and below 0, pages that are not there."""
    k_pool, v_pool, tables, _, _ = ref.cache([(20, 0), (20, 0), (20, 0)], 1, 64, 8, torch.float16,
                                             garbage=0.0)
    tables[2, 1] = -1
    tables[2, 2] = k_pool.shape[0]
    starts = ints([22, -2, 7])                   # 24 positions a row
    offsets = ints([2, 6, 10, 15])
    qkv = torch.randn(18, 4, 64, device="cuda").half()
    r = w4.Rotary(64)
    out = torch.full((18, 2, 64), 7.0, device="cuda").half()
    w4.paged_append_rotary(qkv[:, 2:3], qkv[:, 3:], k_pool, v_pool, tables, starts, r, offsets,
                           q=qkv[:, :2], out=out)
    assert (out[:2] == 0).all() and (out[15:] == 0).all()
    positions = [22, 23, 24, 25, -2, -1, 0, 1, 7, 8, 9, 10, 11]
    near(out[2:15], *ref.rotate(qkv[2:15, :2], positions, r.rates, False))
    held = {(0, 22): 2, (0, 23): 3, (1, 0): 8, (1, 1): 9, (2, 7): 10}
    untouched, *_ = ref.cache([(20, 0), (20, 0), (20, 0)], 1, 64, 8, torch.float16, garbage=0.0)
    slots = {(int(tables[b, p // 8]), p % 8): t for (b, p), t in held.items()}
    for g in range(k_pool.shape[0]):
        for s in range(8):
            if (g, s) in slots:
                assert torch.equal(v_pool[g, s], qkv[slots[g, s], 3:])
            else:
                assert torch.equal(k_pool[g, s], untouched[g, s])
