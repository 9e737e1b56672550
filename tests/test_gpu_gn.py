"""Group norm with an activation on the GPU against the fp64 reference: both layouts and types,
every activation, groups of one value up to groups that no block holds, vector widths from 16
bytes down to one value, missing gamma and beta, no statistics, in place, another stream,
non-finite values, run to run.

Tolerances are the conv tests' (tests/gpu_cases.py): the error of an element over the sum of the
magnitudes it is computed from, 1e-5 in fp32 (a few hundred roundings of 2^-24 at the worst; the
sums here are trees and short chains) and 8e-3 in bf16 (one rounding to 2^-9 on top)."""
import numpy as np
import pytest
import torch

import oracle
from implicit_gemm_conv2d_gb300 import train

from . import train_ref
from .gpu_cases import TOL, TORCH_DT, to_dev, to_np

pytestmark = pytest.mark.gpu
EPS = 1e-5

#      B,   C,   P,   G
SHAPES = {
    "encoder1": (37, 128, 12, 16),
    "encoder2": (9, 128, 2, 8),
    "one_value_a_group": (5, 8, 1, 8),
    "two_positions_one_group": (3, 6, 2, 1),
    "odd_everything": (3, 15, 7, 5),
    "one_channel_groups": (4, 3, 331, 3),
    "five_groups_of_three": (7, 15, 35, 5),
    "position_165": (6, 60, 165, 4),
    "block_team": (3, 64, 257, 8),
    "block_team_wide": (2, 128, 64, 1),
    "long_rows": (2, 32, 3001, 4),
    "long_rows_even": (1, 24, 4096, 3),
    "one_channel_long": (1, 2, 30011, 1),
    "wide_short": (2, 1280, 9, 1),
    "many_channels": (1, 2304, 40, 3),
    "thin_groups": (2, 96, 700, 32),
    "one_sample_one_group": (1, 40, 999, 1),
}


def inputs(shape, layout, dtype, seed=0, offset=0.0):
    B, C, P, G = SHAPES[shape] if isinstance(shape, str) else shape
    rng = np.random.default_rng(seed)
    sh = (B, C, P) if layout == "nchw" else (B, P, C)
    dev = {"x": rng.normal(size=sh) * 1.7 + offset, "dy": rng.normal(size=sh),
           "gamma": 1 + 0.3 * rng.normal(size=C), "beta": 0.3 * rng.normal(size=C)}
    dev = {k: to_dev(v, dtype) for k, v in dev.items()}
    return dev, {k: to_np(v) for k, v in dev.items()}, G


def check(out, ref, den, dtype, what, tol=None):
    err = oracle.normalised_error(to_np(out), ref, den)
    assert err <= (tol or TOL[dtype]), f"{what}: {err:.3e}"


def f32_mask(host, mean, rstd, G, layout):
    """z > 0 with the kernels' individually rounded fp32 operations."""
    C = host["gamma"].size
    m, r = (np.repeat(t.astype(np.float32), C // G, axis=1) for t in (mean, rstd))
    ch = (slice(None), slice(None), None) if layout == "nchw" else (slice(None), None, slice(None))
    x = host["x"].astype(np.float32)
    one = (None, slice(None), None) if layout == "nchw" else (None, None, slice(None))
    z = (x - m[ch]) * r[ch] * host["gamma"].astype(np.float32)[one] + host["beta"].astype(np.float32)[one]
    assert z.dtype == np.float32
    return z > 0


def both_ways(shape, layout, dtype, act, seed=0, offset=0.0):
    dev, host, G = inputs(shape, layout, dtype, seed, offset)
    y, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, act, layout)
    torch.cuda.synchronize()
    ry, den, rmean, rrstd = train_ref.gn_fwd(host["x"], host["gamma"], host["beta"], G, EPS, act, layout)
    what = f"{shape} {layout} {dtype} {act}"
    check(y, ry, den, dtype, what + " y")
    v = train_ref.to_bcp(host["x"], layout).reshape(*rmean.shape, -1)
    check(mean, rmean, np.abs(v).max(axis=2), "f32", what + " mean")
    # rstd: relative, where the spread is not lost in the values' own fp32 rounding
    check(rstd, rrstd, rrstd * (1 + np.abs(v).max(axis=2) * rrstd), "f32", what + " rstd")
    # the backward from the reference's statistics, rounded to fp32
    mean32, rstd32 = rmean.astype(np.float32), rrstd.astype(np.float32)
    dx, dg, db = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], to_dev(mean32, "f32"),
                                      to_dev(rstd32, "f32"), act, layout)
    torch.cuda.synchronize()
    mask = f32_mask(host, mean32, rstd32, G, layout) if act == "relu" else None
    ref = train_ref.gn_bwd(host["x"], host["dy"], host["gamma"], host["beta"], mean32, rstd32, G, act, layout, mask)
    for out, (r, d), name in zip((dx, dg, db), ref, ("dx", "dgamma", "dbeta")):
        check(out, r, d, dtype, f"{what} {name}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_shapes(shape, layout, dtype):
    both_ways(shape, layout, dtype, "silu")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("shape,layout", [("encoder1", "nchw"), ("block_team", "nchw"), ("long_rows", "nchw"),
                                          ("long_rows", "nhwc"), ("odd_everything", "nhwc")])
def test_activations(shape, layout, act, dtype):
    both_ways(shape, layout, dtype, act)


@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed, layout):
    """Sizes over the whole range, vector widths and group sizes as they fall."""
    rng = np.random.default_rng(100 + seed)
    while True:
        G = int(rng.choice([1, 2, 3, 4, 5, 8, 16, 32]))
        C, P, B = G * int(np.exp(rng.uniform(0, 4.5))), int(np.exp(rng.uniform(0, 9))), int(np.exp(rng.uniform(0, 5)))
        if 64 <= B * C * P <= 3_000_000:
            break
    both_ways((B, C, P, G), layout, "bf16" if seed % 2 else "f32", ["none", "relu", "silu", "gelu"][seed % 4], seed)


@pytest.mark.parametrize("shape", ["encoder1", "block_team", "long_rows"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_large_common_offset(shape, layout):
    """An offset of 1000 standard deviations: a variance from the mean of squares would be lost
    (1e6 * 2^-24 of it); from the squares about the mean it is not.  The x that both sides see
    are the same fp32 values."""
    both_ways(shape, layout, "f32", "none", offset=1700.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,layout", [("encoder1", "nchw"), ("long_rows", "nhwc"), ("long_rows", "nchw"),
                                          ("wide_short", "nchw")])
def test_optional_arguments(shape, layout, dtype):
    dev, host, G = inputs(shape, layout, dtype)
    ry, den, rmean, rrstd = train_ref.gn_fwd(host["x"], None, None, G, EPS, "relu", layout)
    y, mean, rstd = train.group_norm(dev["x"], G, None, None, EPS, "relu", layout, stats=False)
    assert mean is None and rstd is None
    check(y, ry, den, dtype, "no gamma, beta, stats")
    m, r = to_dev(rmean, "f32"), to_dev(rrstd, "f32")
    dx, dg, db = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], m, r, "silu", layout,
                                      param_grads=False)
    assert dg is None and db is None
    full = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], m, r, "silu", layout)
    assert torch.equal(dx, full[0])
    dx, dg, db = train.group_norm_bwd(dev["x"], dev["dy"], G, None, None, m, r, "gelu", layout)
    ref = train_ref.gn_bwd(host["x"], host["dy"], None, None, to_np(m), to_np(r), G, "gelu", layout)
    for out, (a, d) in zip((dx, dg, db), ref):
        check(out, a, d, dtype, "no gamma, beta")


@pytest.mark.parametrize("shape,layout", [("encoder1", "nchw"), ("long_rows", "nhwc"), ("long_rows", "nchw"),
                                          ("block_team", "nhwc")])
def test_in_place_and_run_to_run(shape, layout):
    dev, host, G = inputs(shape, layout, "bf16")
    y, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", layout)
    again = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", layout)
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd), again))
    g = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], mean, rstd, "silu", layout)
    g2 = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], mean, rstd, "silu", layout)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))
    B, C, P, _ = SHAPES[shape]
    desc = train.make_gn_desc(B, C, P, G, "silu", layout, torch.bfloat16, EPS)
    n = max(train.conv_gn_fwd_workspace_size(desc), train.conv_gn_bwd_workspace_size(desc), 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    d = dev["dy"].clone()
    dg, db = torch.empty_like(g[1]), torch.empty_like(g[2])
    train.conv_gn_bwd(desc, dev["x"], d, dev["gamma"], dev["beta"], mean, rstd, d, dg, db, ws)
    assert torch.equal(d, g[0]) and torch.equal(dg, g[1]) and torch.equal(db, g[2])
    x = dev["x"].clone()
    train.conv_gn_fwd(desc, x, dev["gamma"], dev["beta"], x, None, None, ws)
    assert torch.equal(x, y)


@pytest.mark.parametrize("shape,layout", [("encoder1", "nchw"), ("encoder1", "nhwc"), ("long_rows", "nhwc"),
                                          ("long_rows", "nchw")])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_values_stay_in_their_group(shape, layout, bad):
    dev, host, G = inputs(shape, layout, "f32")
    B, C, P, _ = SHAPES[shape]
    clean = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", layout)
    x = dev["x"].clone()
    x.view(-1)[5] = bad  # the first sample's first group in either layout
    y, mean, rstd = train.group_norm(x, G, dev["gamma"], dev["beta"], EPS, "silu", layout)
    v, c = (t if layout == "nchw" else t.transpose(1, 2) for t in (y, clean[0]))
    v, c = v.reshape(B, G, -1), c.reshape(B, G, -1)
    hit = 0 if layout == "nchw" else 5 // (C // G)
    assert torch.isnan(v[0, hit]).all() and torch.isnan(rstd[0, hit])
    keep = torch.ones((B, G), dtype=torch.bool, device="cuda")
    keep[0, hit] = False
    assert torch.equal(v[keep], c[keep])


def test_constant_group_and_zero_spread():
    x = torch.full((2, 8, 6), 3.25, device="cuda")
    beta = torch.arange(8, device="cuda", dtype=torch.float32)
    y, mean, rstd = train.group_norm(x, 2, None, beta, EPS, "none", "nchw")
    assert torch.equal(y, beta.view(1, 8, 1).expand(2, 8, 6)) and (mean == 3.25).all()
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


def test_empty_batch():
    x = torch.empty((0, 8, 6), device="cuda")
    y, mean, rstd = train.group_norm(x, 2, None, None)
    assert y.shape == x.shape and mean.shape == (0, 2)
    dx, dg, db = train.group_norm_bwd(x, x, 2, None, None, mean, rstd)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()


def test_another_stream():
    dev, host, G = inputs("long_rows", "nchw", "f32")
    ref = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", stream=s) for _ in range(5)]
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_small_workspace_refused():
    desc = train.make_gn_desc(2, 32, 3001, 4, "silu", "nchw", torch.float32, EPS)
    x = torch.zeros((2, 32, 3001), device="cuda")
    for size, call in ((train.conv_gn_fwd_workspace_size(desc),
                        lambda ws: train.conv_gn_fwd(desc, x, None, None, x, None, None, ws)),
                       (train.conv_gn_bwd_workspace_size(desc),
                        lambda ws: train.conv_gn_bwd(desc, x, x, None, None, x.view(-1)[:8], x.view(-1)[:8], x,
                                                     x.view(-1)[:32], x.view(-1)[:32], ws))):
        if size:
            for ws in (None, torch.empty(size - 1, dtype=torch.uint8, device="cuda")):
                with pytest.raises(train.binding.ConvError) as e:
                    call(ws)
                assert e.value.status == -5


@pytest.mark.parametrize("shape,layout", [("odd_everything", "nchw"), ("thin_groups", "nhwc")])
def test_gradient_against_differences(shape, layout):
    """<dx, v> of the kernel against the fp64 reference loss's central difference along v.  The
    difference is off by h^2/6 |f'''| and 2^-52 |f| / h (h = 1e-5: both below 1e-7 of the sum of
    magnitudes), the kernel by its 1e-5 tolerance."""
    dev, host, G = inputs(shape, layout, "f32")
    x = host["x"]
    y, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", layout)
    dx, dg, db = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], mean, rstd, "silu", layout)
    rng = np.random.default_rng(9)
    v, vg, vb = rng.normal(size=x.shape), rng.normal(size=host["gamma"].shape), rng.normal(size=host["beta"].shape)

    def loss(h):
        out = train_ref.gn_fwd(x + h * v, host["gamma"] + h * vg, host["beta"] + h * vb, G, EPS, "silu", layout)[0]
        return float((out * host["dy"]).sum())

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [to_np(dx) * v, to_np(dg) * vg, to_np(db) * vb]
    ref = train_ref.gn_bwd(x, host["dy"], host["gamma"], host["beta"], to_np(mean), to_np(rstd), G, "silu", layout)
    den = sum((d * np.abs(t)).sum() for (_, d), t in zip(ref, (v, vg, vb)))
    assert abs(sum(t.sum() for t in terms) - want) <= 1e-5 * den


# Sizes at which a team or a cluster walks several samples (its next one is read, or copied into the
# slots of the last, while it works on this one), and tiles of many groups in two passes.
MANY = {
    "teams": ((6000, 32, 12, 4), "relu"),
    "blocks": ((6000, 8, 131, 2), "gelu"),
    "clusters": ((40, 64, 4096, 4), "relu"),
    "vectors_of_two_groups": ((1500, 160, 60, 16), "silu"),
    "many_groups_a_tile": ((1, 1088, 3860, 32), "relu"),
    "long_tiles": ((2, 224, 13115, 8), "gelu"),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("case", list(MANY))
def test_many_samples_and_long_tiles(case, layout, dtype):
    shape, act = MANY[case]
    both_ways(shape, layout, dtype, act, seed=11)


@pytest.mark.parametrize("shape", ["block_team", (40, 64, 512, 4), (8192, 64, 12, 8)])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
def test_relu_at_zero(shape, layout):
    """beta = -fl(fl((x - mean) rstd) gamma) at one position of each channel and group: z is 0 there
    when its product and its sum are rounded apart, and the product's rounding error when they are
    not, so y and the gradient through that position show it."""
    dev, host, G = inputs(shape, layout, "f32", 12)
    x = host["x"].astype(np.float32)
    C = host["gamma"].size
    _, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "relu", layout)
    m, r = to_np(mean).astype(np.float32), to_np(rstd).astype(np.float32)
    at = (0, slice(None), 1) if layout == "nchw" else (0, 1, slice(None))  # sample 0, position 1, every channel
    rep = C // G
    xhat = (x[at] - np.repeat(m[0], rep)) * np.repeat(r[0], rep)
    beta = -(xhat * host["gamma"].astype(np.float32))
    assert beta.dtype == np.float32
    dbeta_in = to_dev(beta, "f32")
    y, mean2, rstd2 = train.group_norm(dev["x"], G, dev["gamma"], dbeta_in, EPS, "relu", layout)
    assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    assert not to_np(y)[at].any()
    # a gradient at those positions only: the mask stops all of it
    dy = torch.zeros_like(dev["x"])
    dy[at] = 1.0
    dx, dg, db = train.group_norm_bwd(dev["x"], dy, G, dev["gamma"], dbeta_in, mean, rstd, "relu", layout)
    assert not dx.any() and not dg.any() and not db.any()
