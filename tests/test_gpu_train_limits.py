"""The training-step operators at the largest sizes that they accept."""
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1
POSITIONS = MOST - 2 ** 20


@pytest.mark.parametrize("T", [5, 600])
def test_table_of_the_most_rows(T):
    """In one launch, and sorted."""
    V = MOST
    rows = torch.tensor([0, V - 1, 12345, V - 1, -1], device="cuda", dtype=torch.int64).repeat(T // 5)
    dy = torch.ones((T, 1), device="cuda", dtype=torch.bfloat16)
    dt = train.embed_bwd(rows, dy, V)
    n = T // 5
    assert dt[0] == n and dt[V - 1] == 2 * n and dt[12345] == n
    assert int(torch.count_nonzero(dt.view(-1)[:2 ** 30])) + int(torch.count_nonzero(dt.view(-1)[2 ** 30:])) == 3
    y = train.embed(rows, dt).view(-1)
    assert torch.equal(y[:5], torch.tensor([n, 2 * n, n, 2 * n, 0], device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_norm_of_the_most_positions(layout):
    P = POSITIONS
    shape = (1, 1, P) if layout == "nchw" else (1, P, 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    y, mean, rstd = train.group_norm(x, 1, None, None, 1e-5, "none", layout)
    v = x.view(-1)
    parts = [(a, min(P, a + 2 ** 28)) for a in range(0, P, 2 ** 28)]
    m = sum(float(v[a:b].double().sum()) for a, b in parts) / P
    r = (sum(float((v[a:b].double() - m).square().sum()) for a, b in parts) / P + 1e-5) ** -0.5
    assert abs(float(mean) - m) <= 1e-5 and abs(float(rstd) / r - 1.0) <= 1e-5
    z = y.view(-1)
    for a, b in parts:
        want = (v[a:b].float() - m) * r
        assert float((z[a:b].float() - want).abs().max()) <= 8e-3 * float(want.abs().max())
    dx, dg, db = train.group_norm_bwd(x, x, 1, None, None, mean, rstd, "none", layout)
    # dy = x: dbeta = sum x, dgamma = sum x * xhat = P (1 - eps r^2) / r, dx = 0 but for eps and rounding
    assert abs(float(db) - P * m) <= 1e-5 * P
    assert abs(float(dg) / (P * (1.0 - 1e-5 * r * r) / r) - 1.0) <= 8e-3
    assert max(float(dx.view(-1)[a:b].abs().max()) for a, b in parts) <= 1e-3
