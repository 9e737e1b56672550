"""The training-step operators on paths and in settings that the other files leave out: groups of
more channels than a window or a cluster takes, long tiles, z at 0 and non-finite values on every
path of the norm, calls inside a captured graph, tensors of more than 2^31 elements."""
import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from .gpu_cases import to_dev, to_np
from .test_gpu_gn import EPS, both_ways, inputs

pytestmark = pytest.mark.gpu

WIDE = {
    "windows_a_group": (2, 4096, 40, 1),
    "odd_channels": (2, 2051, 33, 1),
    "uneven_windows": (2, 1282, 50, 2),
    "one_position": (3, 6144, 1, 2),
    "short_rows": (3, 4200, 9, 2),
    "long_tiles": (1, 768, 20011, 12),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("shape", list(WIDE))
def test_wide_groups_and_long_tiles(shape, layout, dtype):
    act = ("none", "relu", "silu", "gelu")[list(WIDE).index(shape) % 4]
    both_ways(WIDE[shape], layout, dtype, act, seed=21)
    dev, host, G = inputs(WIDE[shape], layout, dtype, 21)
    y, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, act, layout)
    a, b = (train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], mean, rstd, act, layout)
            for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


# Each path of the norm, by sizes that it takes in fp32.
PATHS = {
    "team": ((37, 128, 12, 16), "nchw"),
    "cluster_nchw": ((3, 64, 257, 8), "nchw"),
    "cluster_nhwc": ((3, 64, 257, 8), "nhwc"),
    "pieces": ((2, 4200, 9, 2), "nchw"),
    "pieces_long": ((1, 2, 300_011, 1), "nchw"),
    "tiles": ((1, 768, 20011, 12), "nhwc"),
    "tiles_of_windows": ((2, 4096, 40, 1), "nhwc"),
}


@pytest.mark.parametrize("path", list(PATHS))
def test_relu_at_zero_on_every_path(path):
    """beta = -fl(fl((x - mean) rstd) gamma) at one position of each channel: z is 0 there, y is 0 and
    no gradient passes."""
    shape, layout = PATHS[path]
    dev, host, G = inputs(shape, layout, "f32", 12)
    rep = shape[1] // G
    _, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "relu", layout)
    m, r = to_np(mean).astype(np.float32), to_np(rstd).astype(np.float32)
    at = (0, slice(None), 0) if layout == "nchw" else (0, 0, slice(None))
    xhat = (host["x"].astype(np.float32)[at] - np.repeat(m[0], rep)) * np.repeat(r[0], rep)
    beta = -(xhat * host["gamma"].astype(np.float32))
    assert beta.dtype == np.float32
    b = to_dev(beta, "f32")
    y, mean2, rstd2 = train.group_norm(dev["x"], G, dev["gamma"], b, EPS, "relu", layout)
    assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    assert not to_np(y)[at].any()
    dy = torch.zeros_like(dev["x"])
    dy[at] = 1.0
    out = train.group_norm_bwd(dev["x"], dy, G, dev["gamma"], b, mean, rstd, "relu", layout)
    assert not any(t.any() for t in out)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("path", list(PATHS))
def test_non_finite_gradient_stays_in_its_group(path, act):
    shape, layout = PATHS[path]
    B, C, P, G = shape
    dev, host, _ = inputs(shape, layout, "f32", 13)
    beta = dev["beta"] + 20.0  # no ReLU is off, no slope is 0
    y, mean, rstd = train.group_norm(dev["x"], G, dev["gamma"], beta, EPS, act, layout)
    clean = train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], beta, mean, rstd, act, layout)
    dy = dev["dy"].clone()
    at = (B - 1, C - 1, P - 1) if layout == "nchw" else (B - 1, P - 1, C - 1)
    dy[at] = float("nan")
    dx, dg, db = train.group_norm_bwd(dev["x"], dy, G, dev["gamma"], beta, mean, rstd, act, layout)
    v, c = (t if layout == "nchw" else t.transpose(1, 2) for t in (dx, clean[0]))
    v, c = v.reshape(B, G, -1), c.reshape(B, G, -1)
    assert torch.isnan(v[-1, -1]).all()
    keep = torch.ones((B, G), dtype=torch.bool, device="cuda")
    keep[-1, -1] = False
    assert torch.equal(v[keep], c[keep])
    for a, b in ((dg, clean[1]), (db, clean[2])):
        assert torch.isnan(a[-1]) and torch.equal(a[:-1], b[:-1])


def captured(call):
    """The call's results from a replay of a graph of it, and from the call itself."""
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = call()
    for t in (out if isinstance(out, tuple) else (out,)):
        t.fill_(-7.0)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    return (out, want) if isinstance(out, tuple) else ((out,), (want,))


@pytest.mark.parametrize("path", list(PATHS))
def test_norm_in_a_graph(path):
    shape, layout = PATHS[path]
    dev, host, G = inputs(shape, layout, "bf16", 14)
    out, want = captured(lambda: train.group_norm(dev["x"], G, dev["gamma"], dev["beta"], EPS, "silu", layout))
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    mean, rstd = want[1], want[2]
    out, want = captured(lambda: train.group_norm_bwd(dev["x"], dev["dy"], G, dev["gamma"], dev["beta"], mean, rstd,
                                                      "silu", layout))
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T,V,D", [(300, 700, 16), (20000, 100, 32), (20000, 5000, 64), (200000, 40000, 16)])
def test_embedding_in_a_graph(T, V, D):
    """One launch, whole tables, the sort by a cluster, the sort by kernels (behind a memset)."""
    rng = np.random.default_rng(15)
    idx = torch.from_numpy(rng.integers(0, V, size=T)).cuda()
    table, dy = to_dev(rng.normal(size=(V, D)), "f32"), to_dev(rng.normal(size=(T, D)), "f32")
    for call in (lambda: train.embed(idx, table), lambda: train.embed_bwd(idx, dy, V)):
        out, want = captured(call)
        assert torch.equal(out[0], want[0])


def test_clipping_in_a_graph():
    grads = [torch.randn(n, device="cuda") for n in (7, 100_000, 3_000_001)]
    outs = [torch.empty_like(g) for g in grads]
    out, want = captured(lambda: train.clip_grads(grads, 0.5, out=outs))
    assert torch.equal(out[0], want[0])
    coef = 0.5 / (float(want[0]) + 1e-6)
    assert all(torch.allclose(o, g * coef, rtol=1e-5) for o, g in zip(outs, grads))


# ---- more than 2^31 elements -----------------------------------------------------------------
BIG = 2 ** 31


@pytest.mark.parametrize("layout,C,P,G", [("nchw", 16, 12, 4), ("nchw", 32, 4096, 2), ("nhwc", 32, 4096, 2),
                                          ("nchw", 8, 1 << 20, 1), ("nhwc", 64, 1 << 18, 2)])
def test_norm_beyond_32_bits(layout, C, P, G):
    """The first and the last samples beside calls on them alone: the same bits, and in dgamma and
    dbeta the gradient of the last sample, as the others' is 0."""
    B = BIG // (C * P) + 3
    shape = (B, C, P) if layout == "nchw" else (B, P, C)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    gamma, beta = (torch.randn(C, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    assert x.numel() > BIG
    y, mean, rstd = train.group_norm(x, G, gamma, beta, EPS, "silu", layout)
    dy = torch.zeros_like(x)
    dy[-2:].copy_(torch.randn(dy[-2:].shape, generator=g, device="cuda"))
    dx, dg, db = train.group_norm_bwd(x, dy, G, gamma, beta, mean, rstd, "silu", layout)
    for part in (slice(0, 2), slice(B - 2, B)):
        y2, mean2, rstd2 = train.group_norm(x[part].contiguous(), G, gamma, beta, EPS, "silu", layout)
        a = train.group_norm_bwd(x[part].contiguous(), dy[part].contiguous(), G, gamma, beta, mean2, rstd2, "silu",
                                 layout)
        # another number of samples may be cut up in another way: equal to a rounding or two
        assert torch.allclose(mean[part], mean2, atol=1e-5) and torch.allclose(rstd[part], rstd2, rtol=1e-5)
        for u, v in ((y[part], y2), (dx[part], a[0])):
            assert (u.float() - v.float()).abs().max() <= 2.0 ** -7 * v.float().abs().max()
    for u, v in ((dg, a[1]), (db, a[2])):
        assert (u.float() - v.float()).abs().max() <= 2.0 ** -7 * v.float().abs().max()


def test_lookup_and_gradient_beyond_32_bits():
    T, D = 2 ** 23 + 5, 256
    V = T
    idx = torch.arange(T, device="cuda", dtype=torch.int64).flip(0)
    dy = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16)[:, None].expand(T, D).contiguous()
    dt = train.embed_bwd(idx, dy, V)
    assert dt.numel() > BIG and torch.equal(dt, dy.flip(0))
    assert torch.equal(train.embed(idx, dt), dy)


def test_clipping_beyond_32_bits():
    n = BIG + 12345
    g = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    norm = train.clip_grads([g], 0.5 * n ** 0.5)
    assert abs(float(norm) / n ** 0.5 - 1.0) <= 1e-5
    assert bool((g == 0.5).all())
