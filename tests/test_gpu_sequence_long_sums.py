"""Sums over the longest rows that the sequence operators take, of terms that are all alike: every addition of a
chain then rounds the same way, which no chain may carry far."""
import math

import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import seq_ref, test_gpu_distill, test_gpu_ln

pytestmark = pytest.mark.gpu
U = seq_ref.U


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 2 ** 30 - 1), (torch.float32, 2 ** 30 - 1),
                                     (torch.bfloat16, 2 ** 27 + 5), (torch.float32, 50_000_017)], ids=str)
def test_loss_over_logits_alike(dtype, V):
    """Logits of -1.5, and of 0 here and there, so that every thread has met the largest one early."""
    z = torch.full((1, V), -1.5, dtype=dtype, device="cuda")
    for k in range(64):
        z[0, k * (V // 64):][:4096] = 0.0
    low = 5000
    ids = torch.tensor([[0, V - 1]], device="cuda")
    assert float(z[0, low]) == float(z[0, V - 1]) == -1.5
    q = torch.zeros((1, 2), device="cuda")
    log = math.log(64 * 4096 + (V - 64 * 4096) * math.exp(-1.5))
    # exp's argument: 4 U of 1.5, 2^x: 4 U; a chain of 256 additions, of up to 512 chains, and a tree of 16 steps;
    # the logarithm: 2 U of itself
    room = (10 + 256 + 512 + 16 + 2 * log) * U
    loss, zmax, zlog = train.distill(z, ids, q)
    assert float(zmax) == 0.0 and abs(float(zlog) - log) <= room
    want = math.log(0.5) + log + 0.75           # log p - log P at 0 and at -1.5, half each
    assert abs(float(loss) - want) <= room + 8 * U * (log + 2)
    # P at -1.5: the same room, its own exponential's argument (3 U of 1.5 + log) and its rounding as it is kept
    half = seq_ref.HALF_STEP["bf16" if dtype == torch.bfloat16 else "f32"]
    P = math.exp(-1.5 - log)
    back = train.distill_bwd(z, ids, q, zmax, zlog)
    assert abs(float(back[0, low]) / P - 1) <= room + (3 * (1.5 + log) + 8) * U + half
    del back
    loss, dz = train.distill_grad(z, ids, q)
    assert abs(float(loss) - want) <= room + 8 * U * (log + 2)
    assert abs(float(dz[0, low]) / P - 1) <= room + (3 * (1.5 + log) + 8) * U + half


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 2_200_003, 9), (1, 4_300_001, 5), (3, 5_000_000, 3)], ids=str)
def test_loss_where_chains_begin(size, dtype):
    """Rows a little longer than one chain a thread."""
    z, ids, q, w = test_gpu_distill.inputs(size, dtype, 23)
    test_gpu_distill.all_ways(z, ids, q, w, 1.0, dtype, f"{size} {dtype}")


@pytest.mark.parametrize("dtype,D", [(torch.float32, 2 ** 29 - 1), (torch.float32, 2 ** 29 - 4), (torch.bfloat16, 2 ** 30 - 8),
                                     (torch.bfloat16, 2 ** 29 - 1), (torch.bfloat16, 2 ** 29 - 2)], ids=str)
def test_norm_of_values_alike(dtype, D):
    """A mean, a mean square, and the backward's two sums over one row.  A vector has up to 8 values, a chain 256
    vectors, the tree over a block's threads 12 steps."""
    sum_room = (8 + 256 + 12) * U
    x = torch.full((1, D), 0.1, dtype=dtype, device="cuda")
    value = float(x[0, 0])
    _, _, mean, _ = train.layer_norm(x)
    assert abs(float(mean) / value - 1) <= sum_room + 2 * U          # the division's two roundings
    _, _, _, rstd = train.layer_norm(x, eps=0.0, rms=True)
    assert abs(float(rstd) * value - 1) <= (sum_room + 3 * U) / 2 + 2 * U
    dy = torch.full_like(x, 0.7)
    e = float(dy[0, 0])
    r = torch.full((1,), 1.0 / value, device="cuda")
    # dx / (r e) = 1 - (mean of e) / e, and without a mean 1 - xhat (mean of e xhat) / e, xhat = 1: both 0
    dx, _, _ = train.layer_norm_bwd(x, dy, None, r * 0 + value, r, param_grads=False)
    assert float(dx.abs().max()) <= float(r) * e * (sum_room + 4 * U)
    dx, _, _ = train.layer_norm_bwd(x, dy, None, None, r, param_grads=False)
    assert float(dx.abs().max()) <= float(r) * e * (sum_room + 12 * U)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("size,dtype", [((2, 270_001), "f32"), ((1, 530_002), "f32"), ((1, 1_050_000), "f32"),
                                        ((2, 270_001), "bf16"), ((1, 530_002), "bf16"), ((1, 2_100_000), "bf16")], ids=str)
def test_norm_where_chains_begin(size, dtype, rms):
    """Rows a little longer than one chain a thread, by one, two and four or eight values a vector."""
    test_gpu_ln.both_ways(size, dtype, rms)
