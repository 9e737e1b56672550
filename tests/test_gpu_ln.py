"""Layer norm of a residual sum on the GPU against the fp64 reference, with and without a mean: one value a
row to rows that no block holds, odd sizes, one row to hundreds of thousands, missing gamma, beta and
statistics, the gradient that came around the norm, in place, values far off and not finite, another
stream, a captured graph, run to run.  Tolerances: the bound that comes with the reference plus the
rounding of the result as it is kept (seq_ref)."""
import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import seq_ref
from .gpu_cases import TORCH_DT, to_np
from .test_gpu_scan import within

pytestmark = pytest.mark.gpu
EPS = 1e-5

#     rows, values
SIZES = [(1, 1), (5, 2), (3, 16), (1000, 16), (257, 33), (96, 512), (130, 100), (70, 1024), (9, 1430), (33, 1023),
         (12, 2048), (5, 3001), (4, 4094), (3, 8192), (2, 8193), (3, 12000), (3, 12275), (3, 6140), (2, 70001), (1, 131072), (20011, 24)]


def inputs(size, dtype, seed=0, residual=True, offset=0.0):
    N, D = size
    rng = np.random.default_rng(seed + N + 11 * D)

    def dev(a):
        return torch.from_numpy(np.asarray(a)).float().cuda().to(TORCH_DT[dtype])

    t = dict(x=dev(rng.normal(size=size) * 1.5 + offset), dy=dev(rng.normal(size=size)),
             gamma=dev(1 + 0.3 * rng.normal(size=D)), beta=dev(0.3 * rng.normal(size=D)), residual=None, dtotal=None)
    if residual:
        t["residual"], t["dtotal"] = dev(rng.normal(size=size) + 0.3), dev(rng.normal(size=size))
    return t


def both_ways(size, dtype, rms, residual=True, gamma=True, seed=0, offset=0.0):
    t = inputs(size, dtype, seed, residual, offset)
    what = f"{size} {dtype} rms {rms} residual {residual} gamma {gamma}"
    if not gamma:
        t["gamma"] = t["beta"] = None
    if rms:
        t["beta"] = None
    y, total, mean, rstd = train.layer_norm(t["x"], t["gamma"], t["beta"], t["residual"], EPS, rms)
    assert (total is None) == (not residual) and (mean is None) == rms
    n = {k: None if v is None else to_np(v) for k, v in t.items()}
    kept = t["x"] if total is None else total
    if residual:
        s = n["x"] + n["residual"]
        within(total, s, seq_ref.U * np.abs(s), dtype, what + " total")
    s = to_np(kept)
    (ry, by), (rm, bm), (rr, br) = seq_ref.ln_fwd(s, n["gamma"], n["beta"], EPS, rms)
    within(y, ry, by, dtype, what + " y")
    within(rstd, rr, br, "f32", what + " rstd")
    if not rms:
        within(mean, rm, bm, "f32", what + " mean")
    dx, dgamma, dbeta = train.layer_norm_bwd(kept, t["dy"], t["gamma"], mean, rstd, t["dtotal"])
    refs = seq_ref.ln_bwd(s, n["dy"], n["gamma"], None if rms else to_np(mean), to_np(rstd), n["dtotal"], rms)
    within(dx, *refs[0], dtype, what + " dx")
    within(dgamma, *refs[1], dtype, what + " dgamma")
    assert (dbeta is None) == rms
    if not rms:
        within(dbeta, *refs[2], dtype, what + " dbeta")
    return t, (y, total, mean, rstd), (dx, dgamma, dbeta)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("rms", [False, True])
def test_against_the_reference(rms, size, dtype):
    i = SIZES.index(size)
    both_ways(size, dtype, rms, residual=True)
    both_ways(size, dtype, rms, residual=False, gamma=i % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(300_001, 16), (400_000, 24), (150_000, 7), (100_003, 130)], ids=str)
def test_many_rows(size, dtype):
    both_ways(size, dtype, False)


@pytest.mark.parametrize("D", [4104, 6001, 8192])
def test_many_long_rows(D):
    """Rows of one team a block, so many that a thread's sums are handed over in between."""
    N = 45_000
    g = torch.Generator(device="cuda").manual_seed(D)
    x, dy = (torch.empty((N, D), device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(D, device="cuda", generator=g).bfloat16()
    _, _, mean, rstd = train.layer_norm(x, gamma)
    dx, dgamma, dbeta = train.layer_norm_bwd(x, dy, gamma, mean, rstd)
    dg, db, mg, mb = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(4))
    for a in range(0, N, 5000):
        xh = (x[a:a + 5000].double() - mean[a:a + 5000, None]) * rstd[a:a + 5000, None]
        y = dy[a:a + 5000].double()
        dg += (y * xh).sum(0)
        db += y.sum(0)
        mg += (y * xh).abs().sum(0)
        mb += y.abs().sum(0)
    # chains of 256, of 2 of those and of the blocks' sums, and xhat's three roundings
    for got, want, size in ((dgamma, dg, mg), (dbeta, db, mb)):
        room = (256 + 2 + 152 + 16) * seq_ref.U * size + seq_ref.HALF_STEP["bf16"] * want.abs()
        assert bool(((got.double() - want).abs() <= room).all())
    refs = seq_ref.ln_bwd(to_np(x[-3:]), to_np(dy[-3:]), to_np(gamma), to_np(mean[-3:]), to_np(rstd[-3:]), None, False)
    within(dx[-3:], *refs[0], "bf16", "dx")


def test_sums_over_equal_rows():
    """Rows whose terms are all alike: every addition of a chain rounds the same way, which no chain may carry far."""
    N, D = 2_000_000, 8
    x = torch.tensor([1.1, -0.9] * 4, device="cuda").repeat(N, 1)
    dy = torch.full((N, D), 0.1, device="cuda")
    _, _, mean, rstd = train.layer_norm(x, eps=EPS)
    _, dgamma, dbeta = train.layer_norm_bwd(x, dy, None, mean, rstd)
    xh = (to_np(x[:1]) - float(mean[0])) * float(rstd[0])
    term = float(dy[0, 0])
    # chains of up to 360 additions, half a step each, and xhat's own three roundings
    assert float(np.abs(to_np(dbeta) / (N * term) - 1).max()) <= 400 * seq_ref.U
    assert float(np.abs(to_np(dgamma) / (N * term * xh[0]) - 1).max()) <= 410 * seq_ref.U + 8 * seq_ref.U


@pytest.mark.parametrize("D", [512, 9001])
def test_values_far_off(D):
    """Rows around 1000 with a spread of one: mean and deviations, not a difference of squares."""
    both_ways((20, D), "f32", False, residual=False, offset=1000.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(7, 48), (6, 1024), (5, 20001)], ids=str)
def test_in_place_and_without_statistics(size, dtype):
    t, (y, total, mean, rstd), (dx, dgamma, dbeta) = both_ways(size, dtype, False)
    d = train.make_ln_desc(*size, TORCH_DT[dtype], EPS)
    x, r = t["x"].clone(), t["residual"].clone()
    train.conv_ln_fwd(d, x, r, t["gamma"], t["beta"], x, r, None, None)   # y over x, total over the residual
    assert torch.equal(x, y) and torch.equal(r, total)
    x, r = t["x"].clone(), t["residual"].clone()
    train.conv_ln_fwd(d, x, r, t["gamma"], t["beta"], r, x, None, None)
    assert torch.equal(r, y) and torch.equal(x, total)
    got = train.layer_norm(t["x"], t["gamma"], t["beta"], t["residual"], EPS, stats=False)
    assert torch.equal(got[0], y) and got[2] is None and got[3] is None
    ws = torch.empty(train.conv_ln_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    for name in ("dy", "dtotal"):
        g = {k: t[k].clone() for k in ("dy", "dtotal")}
        dg, db = torch.empty_like(dgamma), torch.empty_like(dbeta)
        ws.fill_(255)
        train.conv_ln_bwd(d, total, g["dy"], t["gamma"], mean, rstd, g["dtotal"], g[name], dg, db, ws)
        assert torch.equal(g[name], dx) and torch.equal(dg, dgamma) and torch.equal(db, dbeta)
    only = train.layer_norm_bwd(total, t["dy"], t["gamma"], mean, rstd, t["dtotal"], param_grads=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [20, 256, 1430, 10001])
def test_a_row_that_is_not_finite(D, rms, dtype):
    t = inputs((9, D), dtype)
    beta = None if rms else t["beta"]
    want = train.layer_norm(t["x"], t["gamma"], beta, t["residual"], EPS, rms)
    bad = t["x"].clone()
    bad[2, D // 2], bad[5, 0] = float("nan"), float("inf")
    y, total, mean, rstd = train.layer_norm(bad, t["gamma"], beta, t["residual"], EPS, rms)
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(y[keep], want[0][keep]) and torch.equal(rstd[keep], want[3][keep])
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[5]).any())
    good = train.layer_norm_bwd(want[1], t["dy"], t["gamma"], want[2], want[3], t["dtotal"])
    dx, dgamma, _ = train.layer_norm_bwd(total, t["dy"], t["gamma"], mean, rstd, t["dtotal"])
    assert torch.equal(dx[keep], good[0][keep]) and bool(torch.isnan(dx[2]).all()) and bool(torch.isnan(dgamma).all())


def test_no_rows_and_shapes():
    x = torch.zeros((0, 12), device="cuda")
    y, total, mean, rstd = train.layer_norm(x)
    assert y.shape == (0, 12) and total is None and mean.shape == rstd.shape == (0,)
    dx, dgamma, dbeta = train.layer_norm_bwd(x, x, None, mean, rstd)
    assert dx.shape == (0, 12) and not bool(dgamma.any()) and not bool(dbeta.any())
    t = inputs((24, 40), "bf16")
    flat = train.layer_norm(t["x"], t["gamma"], t["beta"], t["residual"])
    cube = train.layer_norm(t["x"].view(4, 6, 40), t["gamma"], t["beta"], t["residual"].view(4, 6, 40))
    assert cube[2].shape == (4, 6) and torch.equal(cube[0].view(24, 40), flat[0])
    one = train.layer_norm(t["x"][3], t["gamma"], t["beta"], t["residual"][3])
    assert torch.equal(one[0], flat[0][3]) and one[3].shape == ()


def test_refusals():
    t = inputs((6, 32), "f32")
    x, g, b, r = t["x"], t["gamma"], t["beta"], t["residual"]
    _, _, mean, rstd = train.layer_norm(x)
    for bad in (lambda: train.layer_norm(x.t(), g, b), lambda: train.layer_norm(x, g[:8], b),
                lambda: train.layer_norm(x, g.bfloat16(), b), lambda: train.layer_norm(x, g, b, r[:3]),
                lambda: train.layer_norm(x.half()), lambda: train.layer_norm(x.cpu()),
                lambda: train.layer_norm_bwd(x, r[:3], g, mean, rstd), lambda: train.layer_norm_bwd(x, r, g, mean[:2], rstd),
                lambda: train.layer_norm_bwd(x, r, g, mean, rstd.double()),
                lambda: train.layer_norm_bwd(x, r, g, mean, rstd, dtotal=r.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: train.layer_norm(x, g, b, rms=True), lambda: train.layer_norm(x, eps=-1.0),
                lambda: train.layer_norm(x, eps=float("nan")), lambda: train.layer_norm(x.view(-1)[1:161].view(5, 32))):
        with pytest.raises(train.binding.ConvError):
            bad()


@pytest.mark.parametrize("size", [(5000, 24), (2000, 1024), (300, 5001)], ids=str)
def test_run_to_run_on_a_stream_and_in_a_graph(size):
    t, fwd, bwd = both_ways(size, "bf16", False)

    def calls(stream=None):
        a = train.layer_norm(t["x"], t["gamma"], t["beta"], t["residual"], EPS, stream=stream)
        return (*a, *train.layer_norm_bwd(a[1], t["dy"], t["gamma"], a[2], a[3], t["dtotal"], stream=stream))

    want = (*fwd, *bwd)
    assert all(torch.equal(u, v) for u, v in zip(calls(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = calls(s)
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(2):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_beyond_32_bits():
    """More than 2^31 values: the last rows, and a gradient that every row adds to."""
    N, D = 2_200_000, 1000
    x = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    t = inputs((3, D), "bf16")
    x[-3:] = t["x"]
    y, _, mean, rstd = train.layer_norm(x, t["gamma"], t["beta"], stats=True)
    (ry, by), _, _ = seq_ref.ln_fwd(to_np(t["x"]), to_np(t["gamma"]), to_np(t["beta"]), EPS, False)
    within(y[-3:], ry, by, "bf16", "y")
    assert torch.equal(y[:3], t["beta"].expand(3, D))
    dx, dgamma, dbeta = train.layer_norm_bwd(x, y, t["gamma"], mean, rstd)
    want = seq_ref.ln_bwd(to_np(t["x"]), to_np(y[-3:]), to_np(t["gamma"]), to_np(mean[-3:]), to_np(rstd[-3:]), None, False)
    within(dx[-3:], *want[0], "bf16", "dx")
    within(dgamma, *want[1], "bf16", "dgamma")   # (the others' xhat is 0)
