"""Layer norm of rows that are not finite, each kind in a call of its own, against what the formulas give: NaN; an
infinity, with a mean and without; finite values whose squares are not.  The other rows are as without them."""
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import test_gpu_ln
from .gpu_cases import TORCH_DT

pytestmark = pytest.mark.gpu
ROW, KEEP = 5, [0, 1, 2, 3, 4, 6, 7, 8]


def passes(t, x, rms, dy):
    beta = None if rms else t["beta"]
    y, total, mean, rstd = train.layer_norm(x, t["gamma"], beta, t["residual"], test_gpu_ln.EPS, rms)
    return y, rstd, train.layer_norm_bwd(total, dy, t["gamma"], mean, rstd, t["dtotal"])


def setting(D, dtype):
    t = test_gpu_ln.inputs((9, D), dtype)
    quiet = t["dy"].clone()   # the row adds nothing to the parameters' gradients
    quiet[ROW] = 0
    return t, quiet


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [20, 33, 256, 1430, 10001, 40000])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_one_infinity(value, D, rms, dtype):
    t, quiet = setting(D, dtype)
    at = D // 3
    x = t["x"].clone()
    x[ROW, at] = value
    clean, silent = passes(t, t["x"], rms, t["dy"]), passes(t, t["x"], rms, quiet)
    y, rstd, (dx, dgamma, dbeta) = passes(t, x, rms, t["dy"])
    assert torch.equal(y[KEEP], clean[0][KEEP]) and torch.equal(rstd[KEEP], clean[1][KEEP])
    assert torch.equal(dx[KEEP], clean[2][0][KEEP]) and bool(torch.isnan(dx[ROW]).all())
    others = torch.arange(D, device="cuda") != at
    if rms:
        assert float(rstd[ROW]) == 0.0
        assert bool(torch.isnan(y[ROW, at])) and not bool(y[ROW][others].any())
        assert bool(torch.isnan(dgamma[at])) and torch.equal(dgamma[others], silent[2][1][others])
        assert dbeta is None
    else:
        assert bool(torch.isnan(rstd[ROW])) and bool(torch.isnan(y[ROW]).all()) and bool(torch.isnan(dgamma).all())
        assert torch.equal(dbeta, clean[2][2])   # a sum of dy alone


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [20, 33, 256, 1430, 10001, 40000])
def test_one_nan(D, rms, dtype):
    t, _ = setting(D, dtype)
    x = t["x"].clone()
    x[ROW, D // 3] = float("nan")
    clean = passes(t, t["x"], rms, t["dy"])
    y, rstd, (dx, dgamma, dbeta) = passes(t, x, rms, t["dy"])
    assert torch.equal(y[KEEP], clean[0][KEEP]) and torch.equal(dx[KEEP], clean[2][0][KEEP])
    assert bool(torch.isnan(rstd[ROW])) and all(bool(torch.isnan(v).all()) for v in (y[ROW], dx[ROW], dgamma))
    assert rms or torch.equal(dbeta, clean[2][2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [20, 33, 1430, 10001])
def test_one_nan_in_the_gradient(D, rms, dtype):
    """dy: its row of dx, and its column of the parameters' gradients."""
    t, _ = setting(D, dtype)
    at = D // 3
    dy = t["dy"].clone()
    dy[ROW, at] = float("nan")
    clean = passes(t, t["x"], rms, t["dy"])[2]
    dx, dgamma, dbeta = passes(t, t["x"], rms, dy)[2]
    others = torch.arange(D, device="cuda") != at
    assert torch.equal(dx[KEEP], clean[0][KEEP]) and bool(torch.isnan(dx[ROW]).all())
    for got, want in ((dgamma, clean[1]), (dbeta, clean[2])):
        if want is not None:
            assert bool(torch.isnan(got[at])) and torch.equal(got[others], want[others])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [20, 33, 1430, 10001])
def test_squares_beyond_the_range(D, rms, dtype):
    """Values of +-1e30: rstd is 0, y is beta, and dx what came around the norm."""
    t, quiet = setting(D, dtype)
    x = t["x"].clone()
    x[ROW] = torch.where(torch.arange(D, device="cuda") % 2 == 0, 1e30, -1e30).to(x.dtype)
    clean, silent = passes(t, t["x"], rms, t["dy"]), passes(t, t["x"], rms, quiet)
    y, rstd, (dx, dgamma, dbeta) = passes(t, x, rms, t["dy"])
    assert float(rstd[ROW]) == 0.0 and torch.equal(y[KEEP], clean[0][KEEP])
    assert torch.equal(y[ROW], torch.zeros_like(y[ROW]) if rms else t["beta"])
    assert torch.equal(dx[KEEP], clean[2][0][KEEP]) and torch.equal(dx[ROW], t["dtotal"][ROW])
    assert torch.equal(dgamma, silent[2][1]) and (rms or torch.equal(dbeta, clean[2][2]))
    assert t["x"].dtype == TORCH_DT[dtype]
