"""Group norm's statistics on values that single-pass sums get wrong: all equal but for a few that
are far off, at the start of a sample (a border) or at regular distances.  mean and rstd against
64 bits: the mean to 1e-5 of the largest magnitude, rstd to 1e-5 of itself (the conv tests' fp32
figure: a few hundred roundings of 2^-24 at the worst).  The values are the kernel's own inputs in
either type, and the statistics are fp32 in both."""
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from .gpu_cases import TORCH_DT

pytestmark = pytest.mark.gpu
EPS = 1e-5
TOL = 1e-5

#                B,    C,      P,  G, layout
SHAPES = {
    # a cluster holds the group: up to 128 values a thread and place
    "cluster_f32_single": (1, 5, 40000, 1, "nhwc", "f32"),
    "cluster_bf16_single": (1, 5, 76000, 1, "nhwc", "bf16"),
    "cluster_f32_pairs": (2, 6, 36000, 1, "nhwc", "f32"),
    "cluster_bf16_pairs": (2, 6, 70000, 1, "nhwc", "bf16"),
    "cluster_two_groups_a_vector": (1, 20, 22000, 4, "nhwc", "bf16"),
    "cluster_rows_f32": (1, 1, 200001, 1, "nchw", "f32"),
    "cluster_rows_bf16": (1, 1, 400001, 1, "nchw", "bf16"),
    "cluster_wide_bf16": (2, 64, 5184, 2, "nhwc", "bf16"),
    # two passes over row tiles: 64 to 1024 rows a thread
    "tiles_f32": (1, 1024, 17000, 16, "nhwc", "f32"),
    "tiles_bf16": (1, 2048, 17000, 32, "nhwc", "bf16"),
    "tiles_long_f32": (1, 1024, 140000, 16, "nhwc", "f32"),
    "tiles_narrow_f32": (1, 8, 1 << 20, 1, "nhwc", "f32"),
    # pieces of rows, teams
    "pieces": (1, 2, 3_000_003, 1, "nchw", "f32"),
    "team": (64, 16, 24, 2, "nchw", "f32"),
}
PATTERNS = {"first": lambda i: i == 0, "border": lambda i: i < 8, "border_long": lambda i: i < 40,
            "period": lambda i: i % 100 == 0}


@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_few_values_far_off(shape, pattern):
    B, C, P, G, layout, dtype = SHAPES[shape]
    at = PATTERNS[pattern](torch.arange(P, device="cuda"))
    v = torch.where(at, 100.0, 0.3).to(TORCH_DT[dtype])
    x = v.view(1, 1, P).expand(B, C, P) if layout == "nchw" else v.view(1, P, 1).expand(B, P, C)
    x = x.contiguous()
    y, mean, rstd = train.group_norm(x, G, None, None, EPS, "none", layout)
    d = v.double()
    want = d.mean()
    want_rstd = 1.0 / torch.sqrt(((d - want) ** 2).mean() + EPS)
    off = (mean.double() - want).abs().max() / d.abs().max()
    assert float(off) <= TOL, f"mean off by {float(off):.2e}"
    off = (rstd.double() / want_rstd - 1.0).abs().max()
    assert float(off) <= TOL, f"rstd off by {float(off):.2e}"
