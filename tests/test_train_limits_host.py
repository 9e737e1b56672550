"""Limits of the training-step operators' sizes, refused on the host (the addresses are made up: every
call here has to be one that is refused, on a machine with a GPU too)."""
import ctypes

import pytest

from implicit_gemm_conv2d_gb300 import build, train

OK = 0x1000


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


@pytest.mark.parametrize("B", [2 ** 31 - 2 ** 25, 2 ** 31 - 1000, 2 ** 31 - 1])
def test_samples_that_32_bit_steps_cannot_count(L, B):
    """One group a sample, so B * G is within its limit; the kernels' steps over samples are not."""
    d = train.GnDesc(B, 1, 1, 1, 0, 0, 1, 1e-5)
    r = ctypes.addressof(d)
    assert L.conv_gn_fwd(r, OK, None, None, OK, None, None, OK, 1 << 40, None) == -3
    assert L.conv_gn_bwd(r, OK, OK, None, None, OK, OK, OK, OK, OK, OK, 1 << 40, None) == -3
    assert L.conv_gn_fwd_workspace_size(r) == 0 and L.conv_gn_bwd_workspace_size(r) == 0
