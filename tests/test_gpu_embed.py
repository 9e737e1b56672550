"""Embedding lookup and its gradient on the GPU against the fp64 reference: both index and value
types, vector widths down to one value, tables from one row to many, tokens from none to many,
all equal, all different, padding and out-of-range tokens, more digits than one pass of the sort.

Lookup: one fp32 product and one rounding, so fp32 is exact to 2^-24 and bf16 to 2^-9 (tolerances
2^-23, 2^-8).  Gradient: tests/gpu_cases.py's 1e-5 / 8e-3 of the sum of |term|."""
import numpy as np
import pytest
import torch

import oracle
from implicit_gemm_conv2d_gb300 import train

from . import train_ref
from .gpu_cases import TOL, to_dev, to_np

pytestmark = pytest.mark.gpu

#      T,     V,    D, distribution
CASES = {
    "one_token": (1, 7, 16, "uniform"),
    "encoder": (20 * 47, 128, 32, "zipf"),
    "one_row": (3000, 1, 8, "uniform"),
    "all_equal": (9000, 300, 40, "equal"),
    "all_equal_wide": (2500, 9, 1040, "equal"),
    "all_different": (4097, 4097, 24, "permutation"),
    "odd_width": (1000, 77, 51, "uniform"),
    "width_one": (5000, 500, 1, "zipf"),
    "width_two": (700, 33, 2, "uniform"),
    "wide": (300, 1000, 4100, "zipf"),
    "two_digits": (30000, 70001, 8, "zipf"),
    "three_digits": (6000, 700001, 4, "uniform"),
    "many_tokens": (200000, 130, 12, "zipf"),
    "few_rows_two_windows": (20000, 100, 40, "zipf"),
    "few_rows_equal": (9000, 3, 33, "equal"),
    "few_rows_most": (40000, 512, 7, "zipf"),
    "bins_511": (10000, 511, 16, "uniform"),
    "bins_512": (10000, 512, 16, "uniform"),
    "tile_end": (2048, 60, 16, "uniform"),
    "tile_end_plus": (2049, 60, 16, "uniform"),
}


def tokens(T, V, dist, rng):
    if dist == "equal":
        return np.full(T, V // 2)
    if dist == "permutation":
        return rng.permutation(V)[:T]
    if dist == "zipf":
        return np.minimum(V - 1, (np.exp(rng.uniform(size=T) * np.log(V + 1.0)) - 1).astype(np.int64)) * 7919 % V
    return rng.integers(0, V, size=T)


def make(case, dtype, index, seed=0):
    T, V, D, dist = CASES[case]
    rng = np.random.default_rng(seed)
    idx = tokens(T, V, dist, rng)
    table, dy = to_dev(rng.normal(size=(V, D)), dtype), to_dev(rng.normal(size=(T, D)), dtype)
    return torch.from_numpy(idx).to("cuda", getattr(torch, index)), idx, table, dy


def check_bwd(dt, idx, dy, V, scale, padding, dtype, what):
    ref, den = train_ref.embed_bwd(idx, to_np(dy), V, scale, padding)
    err = oracle.normalised_error(to_np(dt), ref, den)
    assert err <= TOL[dtype], f"{what}: {err:.3e}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("index", ["int32", "int64"])
@pytest.mark.parametrize("case", list(CASES))
def test_both_ways(case, index, dtype):
    didx, idx, table, dy = make(case, dtype, index)
    scale = 1.7320508
    y = train.embed(didx, table, scale)
    ref = train_ref.embed_fwd(idx, to_np(table), np.float32(scale), -1)
    assert (np.abs(to_np(y) - ref) <= (2.0 ** -23 if dtype == "f32" else 2.0 ** -8) * np.abs(ref)).all()
    dt = train.embed_bwd(didx, dy, table.shape[0], scale)
    check_bwd(dt, idx, dy, table.shape[0], np.float32(scale), -1, dtype, f"{case} {index} {dtype}")
    assert torch.equal(dt, train.embed_bwd(didx, dy, table.shape[0], scale))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("index", ["int32", "int64"])
def test_padding_and_tokens_outside_the_table(index, dtype):
    rng = np.random.default_rng(5)
    V, D, T = 40, 24, 3000
    idx = rng.integers(-3, V + 3, size=(T,))
    idx[:7] = [-2**31, 2**31 - 1, V, -1, 0, 11, 11]
    if index == "int64":
        idx[7:10] = [2**40 + 3, -2**50, 2**32]  # the low 32 bits name rows
    didx = torch.from_numpy(idx).to("cuda", getattr(torch, index))
    table, dy = to_dev(rng.normal(size=(V, D)), dtype), to_dev(rng.normal(size=(T, D)), dtype)
    y = train.embed(didx, table, 0.5, padding_idx=11)
    ref = train_ref.embed_fwd(idx, to_np(table), 0.5, 11)
    assert np.array_equal(to_np(y), ref)  # a power of two: exact
    dt = train.embed_bwd(didx, dy, V, 0.5, padding_idx=11)
    check_bwd(dt, idx, dy, V, 0.5, 11, dtype, "padding")
    assert not dt[11].any()


@pytest.mark.parametrize("T", [5, 5000])
def test_no_token_names_a_row(T):
    idx = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    dy = torch.full((T, 8), float("nan"), device="cuda")
    dt = train.embed_bwd(idx, dy, 100)
    assert torch.count_nonzero(dt).item() == 0 and not torch.isnan(dt).any()
    y = train.embed(idx, torch.full((3, 8), float("nan"), device="cuda"))
    assert torch.count_nonzero(y).item() == 0


def test_no_tokens():
    idx = torch.empty((0,), dtype=torch.int64, device="cuda")
    assert train.embed(idx, torch.ones((3, 4), device="cuda")).shape == (0, 4)
    dt = train.embed_bwd(idx, torch.empty((0, 4), device="cuda"), 3)
    assert torch.count_nonzero(dt).item() == 0


def test_non_finite_gradients_stay_in_their_row():
    rng = np.random.default_rng(6)
    idx = torch.from_numpy(rng.integers(0, 50, size=(4000,))).cuda()
    dy = torch.randn((4000, 16), device="cuda")
    clean = train.embed_bwd(idx, dy, 50)
    dy[123, 3] = float("inf")
    dt = train.embed_bwd(idx, dy, 50)
    row = int(idx[123])
    assert torch.isinf(dt[row, 3])
    dt[row, 3] = clean[row, 3]
    assert torch.equal(dt, clean)


def test_shapes_and_stream():
    idx = torch.randint(0, 128, (6, 47), device="cuda", dtype=torch.int32)
    table = torch.randn((128, 32), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = train.embed(idx, table, stream=s)
    dt = train.embed_bwd(idx, y, 128, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert y.shape == (6, 47, 32) and torch.equal(y, table[idx.long()])
    assert torch.equal(dt, train.embed_bwd(idx, y, 128))


def test_gradient_against_differences():
    """The lookup is linear in the table: <dtable, v> is the difference of <dy, y> exactly."""
    rng = np.random.default_rng(8)
    idx = rng.integers(0, 60, size=(2000,))
    dy, v = rng.normal(size=(2000, 20)).astype(np.float32), rng.normal(size=(60, 20))
    dt = train.embed_bwd(torch.from_numpy(idx).cuda(), to_dev(dy, "f32"), 60, 0.25)
    want = (dy.astype(np.float64) * train_ref.embed_fwd(idx, v, 0.25, -1)).sum()
    den = (np.abs(dy) * np.abs(train_ref.embed_fwd(idx, v, 0.25, -1))).sum()
    assert abs((to_np(dt) * v).sum() - want) <= 1e-5 * den


def test_small_workspace_refused():
    desc = train.make_embed_desc(1000, 50, 8, torch.int32, torch.float32)
    idx = torch.zeros(1000, dtype=torch.int32, device="cuda")
    dy, dt = torch.zeros((1000, 8), device="cuda"), torch.zeros((50, 8), device="cuda")
    size = train.conv_embed_bwd_workspace_size(desc)
    for ws in (None, torch.empty(size - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(train.binding.ConvError) as e:
            train.conv_embed_bwd(desc, idx, dy, dt, ws)
        assert e.value.status == -5


# Around the one-launch path's limits: 512 tokens, 4096 blocks of a token and 32 vectors (513 x 40,
# 128 x 8192 in fp32 and 512 x 257 are beyond them), tables of many rows a filling block, widths that
# end inside a window.
FEW = {
    "most": (512, 60187, 40, "zipf"),
    "most_plus": (513, 60187, 40, "zipf"),
    "most_one_row": (512, 1, 136, "equal"),
    "most_equal": (512, 90, 1032, "equal"),
    "odd_width": (511, 400001, 3, "uniform"),
    "many_rows": (40, 900000, 5, "uniform"),
    "windows": (300, 4410, 1088, "zipf"),
    "windows_most": (128, 700, 8192, "zipf"),
    "windows_odd": (455, 100, 257, "zipf"),
    "windows_odd_plus": (512, 512, 257, "permutation"),
    "two": (2, 3, 33, "equal"),
    "warp_shares": (257, 31, 64, "uniform"),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("index", ["int32", "int64"])
@pytest.mark.parametrize("case", list(FEW))
def test_few_tokens(case, index, dtype):
    T, V, D, dist = FEW[case]
    rng = np.random.default_rng(9)
    idx = tokens(T, V, dist, rng)
    if T > 40 and V > 3:
        idx[[3, 20, T - 1]] = [-1, V, V // 3]
    didx = torch.from_numpy(idx).to("cuda", getattr(torch, index))
    dy = to_dev(rng.normal(size=(T, D)), dtype)
    padding = V // 3 if V > 3 else -1
    dt = train.embed_bwd(didx, dy, V, 1.25, padding_idx=padding)
    check_bwd(dt, idx, dy, V, 1.25, padding, dtype, f"{case} {index} {dtype}")
    rows = np.zeros(V, dtype=bool)
    rows[[i for i in idx if 0 <= i < V and i != padding]] = True
    assert not dt[torch.from_numpy(~rows).cuda()].any()
    assert torch.equal(dt, train.embed_bwd(didx, dy, V, 1.25, padding_idx=padding))
