"""Layer norm of a residual sum on the host (no GPU): arguments are refused before any CUDA call, and the
fp64 reference's gradients agree with central differences."""
import ctypes

import numpy as np
import pytest

from implicit_gemm_conv2d_gb300 import build, train

from . import seq_ref

OK, ODD = 0x1000, 0x1008


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


def desc(**kw):
    a = dict(N=4, D=100, rms=0, dtype=0, eps=1e-5)
    a.update(kw)
    return train.LnDesc(a["N"], a["D"], a["rms"], a["dtype"], a["eps"])


# The addresses are made up: every call here has to be one that is refused.
def fwd(L, d, x=OK, residual=OK, gamma=OK, beta=OK, y=OK, total=OK, mean=OK, rstd=OK):
    return L.conv_ln_fwd(ctypes.addressof(d), x, residual, gamma, beta, y, total, mean, rstd, None)


def bwd(L, d, x=OK, dy=OK, gamma=OK, mean=OK, rstd=OK, dtotal=OK, dx=OK, dgamma=OK, dbeta=OK, ws=OK, size=1 << 40):
    return L.conv_ln_bwd(ctypes.addressof(d), x, dy, gamma, mean, rstd, dtotal, dx, dgamma, dbeta, ws, size, None)


@pytest.mark.parametrize("bad,code", [(dict(N=-1), -2), (dict(D=0), -2), (dict(rms=2), -2), (dict(dtype=2), -2),
                                      (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
                                      (dict(N=1 << 31), -3), (dict(D=1 << 30), -3)])
def test_descriptor_refused(L, bad, code):
    d = desc(**bad)
    assert (fwd(L, d), bwd(L, d)) == (code, code)
    assert L.conv_ln_bwd_workspace_size(ctypes.addressof(d)) == 0


def test_pointers_and_alignment(L):
    for name in ("x", "y", "total", "residual", "mean", "rstd"):   # the last four: one without the other
        assert fwd(L, desc(), **{name: None}) == -1
    for name in ("x", "y", "total", "residual", "mean", "rstd", "gamma", "beta"):
        assert fwd(L, desc(), **{name: ODD}) == -4
    for name in ("x", "dy", "mean", "rstd", "dx", "dgamma", "dbeta"):
        assert bwd(L, desc(), **{name: None}) == -1
    for name in ("x", "dy", "mean", "rstd", "dx", "dgamma", "dbeta", "gamma", "dtotal", "ws"):
        assert bwd(L, desc(), **{name: ODD}) == -4
    rms = desc(rms=1)
    assert fwd(L, rms, mean=None) == -2 and fwd(L, rms, beta=None) == -2          # beta, and mean, with rms
    assert bwd(L, rms, mean=None) == -2 and bwd(L, rms, dbeta=None) == -2
    assert L.conv_ln_fwd(None, *[OK] * 8, None) == -1 and L.conv_ln_bwd(None, *[OK] * 10, 0, None) == -1
    empty = desc(N=0)
    assert fwd(L, empty, *[None] * 8) == 0
    assert bwd(L, empty, *[None] * 7, OK, None) == -1


def test_outputs_over_what_is_still_read(L):
    assert fwd(L, desc(), y=OK + 16, total=OK + 16) == -2
    assert bwd(L, desc(), x=OK + 16, dx=OK + 16) == -2


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        train.layer_norm(x)                       # a CPU tensor
    with pytest.raises(ValueError):
        train.layer_norm(x.double())
    with pytest.raises(ValueError):
        train.layer_norm_bwd(x, x, None, None, x[:, 0])
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode(allow_non_fake_inputs=True):
        x, r = torch.empty((2, 8), device="cuda:1"), torch.empty(2, device="cuda:1")
        with pytest.raises(ValueError, match="not the current device"):
            train.layer_norm(x)
        with pytest.raises(ValueError, match="not the current device"):
            train.layer_norm_bwd(x, x, None, r, r)


@pytest.mark.parametrize("rms", [False, True])
def test_reference_gradient_against_differences(rms):
    rng = np.random.default_rng(8)
    N, D, eps = 3, 7, 1e-3
    x, dy, dt = (rng.normal(size=(N, D)) for _ in range(3))
    gamma, beta = rng.normal(size=D), None if rms else rng.normal(size=D)

    def loss():
        return float((seq_ref.ln_fwd(x, gamma, beta, eps, rms)[0][0] * dy).sum() + (x * dt).sum())

    mean, rstd = seq_ref.ln_stats(x, eps, rms)
    (dx, _), (dg, _), (db, _) = seq_ref.ln_bwd(x, dy, gamma, mean, rstd, dt, rms)
    h = 1e-6
    for a, grad in ((x, dx), (gamma, dg)) + (() if rms else ((beta, db),)):
        for k in range(a.size):
            old = a.flat[k]
            a.flat[k] = old + h
            hi = loss()
            a.flat[k] = old - h
            lo = loss()
            a.flat[k] = old
            # central difference: h^2 f''' / 6 and 2^-52 |f| / h, both below 1e-8 here
            assert abs((hi - lo) / (2 * h) - grad.flat[k]) < 1e-6
