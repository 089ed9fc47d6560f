"""The rotation of a model's queries and keys by their positions, set up once.

Pair i of the rotated dimensions turns by position * rate[i].  The usual rates
are base ** (-2 i / dim); for contexts longer than a model was trained on they
are made slower in one of three ways:

  "linear"  every rate divided by the factor;
  "base"    the base times factor ** (dim / (dim - 2)), so that the fastest rate
            stays and the slowest is divided by the factor;
  "ramp"    a rate that turns more than `high` times over the `original` length
            stays, one that turns less than `low` times is divided by the factor,
            and those between are blended linearly in their turns (Peng et al.,
            "YaRN: Efficient Context Window Extension of Large Language Models",
            2023), whose magnitude 0.1 ln(factor) + 1 is for the caller to give.
"""
from __future__ import annotations

import math
import struct
from fractions import Fraction

import torch

# 2^192 / (2 pi)
_TURN = int(Fraction("0.159154943091895335768883763372514362034459645740456448747667344058896797634")
            * 2 ** 192)
_SCALINGS = (None, "linear", "base", "ramp")
_SHAPE = struct.Struct("2qd").pack


def _rates(dim, base, scaling, factor, original, low, high) -> list[float]:
    if not base > 0 or not factor > 0:
        raise ValueError(f"base and factor must be above 0, got {base} and {factor}")
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {_SCALINGS}, got {scaling!r}")
    if scaling == "base":
        if dim == 2:
            raise ValueError("scaling 'base' needs more than one pair")
        base = base * factor ** (dim / (dim - 2))
    rates = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [r / factor for r in rates]
    if scaling == "ramp":
        if original is None or original <= 0 or not low < high:
            raise ValueError("scaling 'ramp' needs the original length, and low below high")
        turns = [original * r / (2.0 * math.pi) for r in rates]
        keep = [min(1.0, max(0.0, (t - low) / (high - low))) for t in turns]
        return [r * k + r / factor * (1.0 - k) for r, k in zip(rates, keep)]
    return rates


def _turn(rate: float) -> int:
    """rate / (2 pi) as a fraction of a turn times 2^64, rounded."""
    n, d = rate.as_integer_ratio()
    return ((n * _TURN // d >> 127) + 1 >> 1) % 2 ** 64


class Rotary:
    """The rotation of the first `dim` dimensions of a head, for rotate and
    paged_append_rotary: neighbours (2i, 2i + 1) are paired where `interleaved`,
    else (i, i + dim / 2).  `rates` (dim / 2 numbers, radians a position) takes
    the place of base and scaling.  What is rotated is multiplied by `magnitude`.

    `rates` holds the numbers used, `turns` (int64 [dim / 2], on the device) each
    as a fraction of a turn times 2^64, so that a position's angle is reduced by
    an integer product alone.  What describes a rotation is read-only; it may be
    copied and pickled like any object that holds a tensor."""

    def __init__(self, dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str | None = None, factor: float = 1.0, original: int | None = None,
                 low: float = 1.0, high: float = 4.0, magnitude: float = 1.0, rates=None,
                 device="cuda"):
        if dim < 2 or dim % 2:
            raise ValueError(f"dim must be even and at least 2, got {dim}")
        if rates is None:
            rates = _rates(dim, base, scaling, factor, original, low, high)
        elif scaling is not None:
            raise ValueError("rates are given: scaling must be None")
        rates = [float(r) for r in rates]
        if len(rates) != dim // 2 or not all(map(math.isfinite, rates)):
            raise ValueError(f"rates must be {dim // 2} finite numbers")
        if not math.isfinite(magnitude):
            raise ValueError(f"magnitude must be finite, got {magnitude}")
        self._dim, self._interleaved, self._magnitude = dim, bool(interleaved), float(magnitude)
        self._rates = tuple(rates)
        turns = [_turn(r) for r in rates]
        self._turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns],
                                   dtype=torch.int64, device=device)
        self._shape = _SHAPE(dim, self._interleaved, self._magnitude)

    dim = property(lambda self: self._dim)
    interleaved = property(lambda self: self._interleaved)
    magnitude = property(lambda self: self._magnitude)
    rates = property(lambda self: list(self._rates))
    turns = property(lambda self: self._turns)

    def _held(self) -> tuple[int, int]:
        """The device and the address of `turns` as they are now: a copy of this object has
        memory of its own, and torch may give a tensor another."""
        turns = self._turns
        if turns.dtype is not torch.int64 or turns.shape != (self._dim // 2,) or (
                not turns.is_contiguous()):
            raise ValueError(f"the rotation's turns must be a dense int64 tensor "
                             f"[{self._dim // 2}], got {turns.dtype} {list(turns.shape)}")
        return turns.get_device(), turns.data_ptr()
