"""A rotation that is copied, pickled or changed: each call reads the tensor that the
object holds at that time, and what describes the rotation cannot come apart from it."""
from __future__ import annotations

import copy
import pickle

import pytest
import torch

import prompt_reference as ref
import w4a16_weight_only_gemm_gb300 as w4
from w4a16_weight_only_gemm_gb300 import serving

COPIES = {"copy": copy.copy, "deepcopy": copy.deepcopy,
          "pickle": lambda r: pickle.loads(pickle.dumps(r)),
          "in a list": lambda r: copy.deepcopy({"layers": [r, r]})["layers"][1]}


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded in the place of being made (on CPU tensors)."""
    made = []
    monkeypatch.setattr(serving, "_run", lambda dev, stream, name, *args: made.append(args))
    monkeypatch.setattr(serving, "_device", lambda stream, **named: -1)
    return made


def rotate(r):
    return w4.rotate(torch.zeros(3, 2, 16).half(), torch.zeros(3, dtype=torch.int32), r)


def append(r):
    x, pool = torch.zeros(3, 2, 16).half(), torch.zeros(4, 16, 2, 16).half()
    return w4.paged_append_rotary(x, x, pool, pool, torch.zeros(3, 2, dtype=torch.int32),
                                  torch.zeros(3, dtype=torch.int32), r)


@pytest.mark.parametrize("how", COPIES)
def test_a_copy_is_read_where_it_lies(calls, how):
    r = w4.Rotary(8, interleaved=True, magnitude=1.5, device="cpu")
    c = COPIES[how](r)
    assert (c.turns.data_ptr() == r.turns.data_ptr()) == (how == "copy")
    assert (c.dim, c.interleaved, c.magnitude, c.rates) == (8, True, 1.5, r.rates)
    assert torch.equal(c.turns, r.turns)
    for one in (r, c):
        for call in (rotate, append):
            calls.clear()
            call(one)
            assert calls[0][2] == one.turns.data_ptr()


def test_memory_that_torch_gave_anew_is_read(calls):
    r = w4.Rotary(8, device="cpu")
    before = r.turns.data_ptr()
    r.turns.data = r.turns.clone()
    assert r.turns.data_ptr() != before
    rotate(r), append(r)
    assert [args[2] for args in calls] == [r.turns.data_ptr()] * 2


@pytest.mark.parametrize("name, value", [("dim", 4), ("interleaved", True), ("magnitude", 2.0),
                                         ("rates", [1.0] * 4),
                                         ("turns", torch.zeros(4, dtype=torch.int64))])
def test_what_describes_a_rotation_is_read_only(name, value):
    r = w4.Rotary(8, device="cpu")
    with pytest.raises(AttributeError):
        setattr(r, name, value)
    r.rates[0] = 7.0
    assert r.rates[0] == 1.0


@pytest.mark.parametrize("data", [torch.zeros(3, dtype=torch.int64), torch.zeros(4),
                                  torch.zeros(2, 2, dtype=torch.int64),
                                  torch.zeros(8, dtype=torch.int64)[::2]],
                         ids=["short", "float", "square", "apart"])
def test_turns_that_are_not_the_rotations_are_refused(calls, data):
    r = w4.Rotary(8, device="cpu")
    r.turns.data = data
    for call in (rotate, append):
        with pytest.raises(ValueError):
            call(r)
    assert not calls


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_a_copy_outlives_its_original(w4lib, how):
    """The original's memory is given to another tensor before the copy rotates: the same bits."""
    x = torch.randn(20, 3, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    positions = torch.arange(20, dtype=torch.int32, device="cuda") * 1000
    r = w4.Rotary(64)
    want = w4.rotate(x, positions, r)
    c, size = COPIES[how](r), r.turns.numel()
    del r
    others = [torch.full((size,), -1, dtype=torch.int64, device="cuda") for _ in range(8)]
    assert torch.equal(w4.rotate(x, positions, c), want)
    exact, bound = ref.rotate(x, positions.tolist(), c.rates, False)
    assert ((want.cpu().double() - exact).abs() <= 2.0 ** -11 * exact.abs()
            + 2.0 ** -21 * bound + 2.0 ** -25).all()
    assert all((t == -1).all() for t in others)
