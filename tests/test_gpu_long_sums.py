"""Long sums of equal values with a full mantissa, for which each rounding of a chain of additions
goes the same way: a chain of n loses up to 1.5e-8 n of its sum (700 additions: 1e-5).  Every sum
over tokens, samples and positions stays within the fp32 tolerance, 1e-5 of the sum of |term|,
however long it is."""
import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

pytestmark = pytest.mark.gpu
TOL = 1e-5
VALUES = [1.00412, 1.706299, 1.913085]  # the worst of 2000 values in [1, 2) for chains of 1023, 4825, 16384


def rel(out, want):
    return float((out.double() / want - 1.0).abs().max())


#        tokens,     V,    D
TOKENS = {
    "whole_table_one_block_a_window": (19300, 300, 2500),
    "whole_table_wide": (65536, 128, 1216),
    "whole_table_long": (4_000_000, 128, 32),
    "sorted_in_a_cluster": (60000, 20000, 32),
    "sorted_by_kernels": (300000, 20000, 64),
    "one_column": (1 << 25, 2000, 1),
}


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("name", list(TOKENS))
def test_table_gradient_of_one_row(name, value):
    T, V, D = TOKENS[name]
    idx = torch.full((T,), V // 2, dtype=torch.int32, device="cuda")
    dy = torch.full((T, D), value, device="cuda")
    dt = train.embed_bwd(idx, dy, V)
    off = rel(dt[V // 2], T * float(np.float32(value)))
    assert off <= TOL, f"{off:.2e}"
    assert torch.count_nonzero(dt).item() == D


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("length", [700, 1023])
def test_table_gradient_of_runs_over_two_chunks(length, value):
    """Every row the same number of tokens, so that runs begin at every place of a chunk."""
    T, D = 240000, 1024
    V = T // length + 1
    idx = (torch.arange(T, device="cuda") // length).to(torch.int32)
    dy = torch.full((T, D), value, device="cuda")
    dt = train.embed_bwd(idx, dy, V)
    count = torch.bincount(idx.long(), minlength=V).double()
    off = rel(dt[count > 0], count[count > 0][:, None] * float(np.float32(value)))
    assert off <= TOL, f"{off:.2e}"


#                B,      C,   P,      G, layout
SHAPES = {
    "teams": (160000, 1024, 2, 1024, "nchw"),
    "teams_of_one_group": (400000, 16, 4, 1, "nchw"),
    "clusters": (3000, 64, 64, 4, "nhwc"),
    "tiles": (1, 1024, 280000, 16, "nhwc"),
    "pieces": (1, 4, 2_000_000, 2, "nchw"),
}


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_channel_sums(shape, value):
    """dy constant and xhat 1 everywhere: dbeta and dgamma are both B * P * dy."""
    B, C, P, G, layout = SHAPES[shape]
    x = torch.ones((B, C, P) if layout == "nchw" else (B, P, C), device="cuda")
    dy = torch.full_like(x, value)
    mean, rstd = torch.zeros((B, G), device="cuda"), torch.ones((B, G), device="cuda")
    dx, dgamma, dbeta = train.group_norm_bwd(x, dy, G, None, None, mean, rstd, "none", layout)
    want = B * P * float(np.float32(value))
    for name, out in (("dgamma", dgamma), ("dbeta", dbeta)):
        off = rel(out, want)
        assert off <= TOL, f"{name} {off:.2e}"


@pytest.mark.parametrize("layout,C,P,G", [("nchw", 64, 16, 8), ("nchw", 64, 64, 8), ("nhwc", 64, 64, 8),
                                          ("nchw", 4096, 400, 4096), ("nhwc", 4096, 64, 256)])
def test_no_block_walks_more_than_256_samples(layout, C, P, G):
    """A block adds up its samples' channel sums one after another and leaves one row of partial sums:
    (2, C) fp32 a row of the workspace."""
    for B in (1 << 17, min(1 << 20, (1 << 30) // G)):
        d = train.make_gn_desc(B, C, P, G, "none", layout, torch.float32)
        rows = train.conv_gn_bwd_workspace_size(d) // (8 * C)
        per = 1 if C // G * P > 384 else max(1, 256 // G)  # teams: up to so many samples side by side
        assert rows * 256 * per >= B, f"{B} samples, {rows} rows"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", VALUES)
def test_gradient_norm(value, dtype):
    g = torch.full((300_000_000,), value, device="cuda").to(dtype)
    want = (300_000_000 * float(g[0]) ** 2) ** 0.5
    assert abs(float(train.grad_norm([g])) / want - 1.0) <= TOL


@pytest.mark.parametrize("value", VALUES)
def test_statistics_of_many_pieces(value):
    """2^29 + 1 equal values of one channel, in 262145 pieces: mean is the value, y is 0."""
    x = torch.full((1, 1, 2 ** 29 + 1), value, device="cuda")
    y, mean, rstd = train.group_norm(x, 1, None, None, 1e-5, "none", "nchw")
    assert abs(float(mean) / float(x[0, 0, 0]) - 1.0) <= TOL
    dx, dg, db = train.group_norm_bwd(x, x, 1, None, None, torch.zeros_like(mean), torch.ones_like(rstd), "none")
    v = float(x[0, 0, 0])  # xhat = dy = v: dx = v - v - v * v * v
    assert float((dx.double() / -v ** 3 - 1.0).abs().max()) <= TOL
