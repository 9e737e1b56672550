"""The comparison of strict.py on the host: one value that is not finite is enough."""
import numpy as np
import pytest
import torch

from . import seq_ref, strict


def test_one_value_is_enough():
    ref, bound = np.linspace(-2.0, 2.0, 12).reshape(3, 4), np.full((3, 4), 1e-6)
    good = torch.from_numpy(ref).float()
    strict.within(good, ref, bound, "f32", "good")
    strict.within(good[:0], ref[:0], bound[:0], "f32", "nothing")
    for value in (float("nan"), float("inf"), float("-inf"), 5.0):
        bad = good.clone()
        bad[1, 2] = value
        with pytest.raises(AssertionError, match="1 values"):
            strict.within(bad, ref, bound, "f32", "output")
        with pytest.raises(AssertionError):
            strict.within(bad[None], ref, bound, "f32", "shape")
    with pytest.raises(AssertionError, match="12 values"):
        strict.within(torch.full((3, 4), float("nan")), ref, bound, "f32", "all")
    for name in ("ref", "bound"):
        for value in (np.nan, np.inf):
            a = dict(ref=ref.copy(), bound=bound.copy())
            a[name][0, 0] = value
            with pytest.raises(AssertionError, match="reference"):
                strict.within(good, a["ref"], a["bound"], "f32", name)


def test_room_is_the_bound_and_half_a_step():
    ref, bound = np.array([1.0, -4.0]), np.array([1e-3, 0.0])
    half = seq_ref.HALF_STEP["bf16"]
    strict.within(torch.tensor([1.0 + 1e-3 + half, -4.0 * (1 - half)], dtype=torch.float64), ref, bound, "bf16", "edge")
    with pytest.raises(AssertionError, match="1 values"):
        strict.within(torch.tensor([1.0, -4.0 * (1 + 1.01 * half)], dtype=torch.float64), ref, bound, "bf16", "beyond")
