"""Comparison with a reference and its bound that no NaN passes: neither one in the output, where a difference that
is NaN is not above anything, nor one in the reference or its bound, which would make any output good."""
import numpy as np

from . import seq_ref
from .gpu_cases import to_np


def within(out, ref, bound, dtype, what):
    out, ref, bound = to_np(out), np.asarray(ref), np.asarray(bound)
    assert out.shape == ref.shape, f"{what}: {out.shape} against {ref.shape}"
    assert np.isfinite(ref).all() and np.isfinite(bound).all(), f"{what}: the reference is not finite"
    room = bound + seq_ref.HALF_STEP[dtype] * (np.abs(ref) + bound)
    bad = ~(np.abs(out - ref) <= room)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} values, the first {out[at]} against {ref[at]} at {at}")
