"""The loss against a teacher's top logits and its gradient on the GPU against the fp64 reference: one
logit to a million, rows that begin anywhere, one entry to 1024, both types and index types, entries
that name nothing, ids that occur twice, rows of padding with NaN in them, infinite and lowest logits,
strided rows, in place, another stream, a captured graph, run to run.  Tolerances: the bound that comes
with the reference plus the rounding of the result as it is kept (seq_ref)."""
import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import seq_ref
from .gpu_cases import TORCH_DT, to_np
from .test_gpu_scan import within

pytestmark = pytest.mark.gpu

#     rows, logits, entries
SIZES = [(1, 1, 1), (3, 2, 1), (5, 7, 3), (9, 33, 40), (64, 128, 8), (37, 1000, 64), (300, 257, 5), (6, 1021, 256),
         (5, 900, 300), (4, 2049, 16), (3, 5003, 40), (2, 50021, 64), (700, 3001, 20), (1, 131071, 256), (2, 300007, 1024),
         (2, 1000003, 7)]


def inputs(size, dtype, seed=0, teacher_dtype="f32", index=torch.int32, tau=1.0, spread=2.0, pad=0.1):
    N, V, K = size
    rng = np.random.default_rng(seed + N + 3 * V + 7 * K)
    z = torch.from_numpy(rng.normal(size=(N, V)) * spread).float().cuda().to(TORCH_DT[dtype])
    ids = rng.integers(0, V, size=(N, K))
    if K > 2:
        again = rng.random((N, K)) < 0.1          # ids that occur twice
        ids = np.where(again, np.roll(ids, 1, axis=1), ids)
    gone = rng.random((N, K)) < pad               # entries that name nothing
    ids = np.where(gone, rng.choice([-1, -7, V, V + 5], size=(N, K)), ids)
    if N > 2:
        ids[1] = -1                               # a row of padding
    q = torch.from_numpy(rng.normal(size=(N, K)) * 3.0 + 5.0).float().cuda().to(TORCH_DT[teacher_dtype])
    w = torch.from_numpy(rng.normal(size=N)).float().cuda()
    return z, torch.from_numpy(ids).to(index).cuda(), q, w


def all_ways(z, ids, q, w, tau, dtype, what, scale=0.25):
    loss, zmax, zlog = train.distill(z, ids, q, tau)
    dz = train.distill_bwd(z, ids, q, zmax, zlog, w, scale, tau)
    loss2, dz2 = train.distill_grad(z, ids, q, w, scale, tau)
    nz, ni, nq = to_np(z), ids.cpu().numpy().astype(np.int64), to_np(q)
    nw = None if w is None else to_np(w)
    (rl, bl), rm, (rg, bg) = seq_ref.distill_fwd(nz, ni, nq, tau)
    assert np.array_equal(to_np(zmax), rm), what + " zmax"
    within(zlog, rg, bg, "f32", what + " zlog")
    within(loss, rl, bl, "f32", what + " loss")
    within(loss2, rl, bl, "f32", what + " loss at once")
    ref, bound = seq_ref.distill_bwd(nz, ni, nq, rm, to_np(zlog), nw, scale, tau)
    within(dz, ref, bound, dtype, what + " dz")
    ref, bound = seq_ref.distill_bwd(nz, ni, nq, rm, rg, nw, scale, tau, bg)
    within(dz2, ref, bound, dtype, what + " dz at once")
    return loss, dz, loss2, dz2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_against_the_reference(size, dtype):
    i = SIZES.index(size)
    tau = (1.0, 2.0, 0.7, 4.0)[i % 4]
    z, ids, q, w = inputs(size, dtype, 0, ("f32", "bf16")[i % 2], (torch.int32, torch.int64)[i // 2 % 2])
    all_ways(z, ids, q, None if i % 3 == 2 else w, tau, dtype, f"{size} {dtype} tau {tau}")


@pytest.mark.parametrize("size", [(64, 128, 8), (3, 5003, 40), (2, 50021, 64)], ids=str)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("teacher", ["f32", "bf16"])
def test_types_of_the_teacher(size, index, teacher):
    z, ids, q, w = inputs(size, "bf16", 1, teacher, index)
    all_ways(z, ids, q, w, 1.0, "bf16", f"{size} {index} {teacher}")


@pytest.mark.parametrize("size", [(40, 796, 152), (700, 11516, 64), (700, 11500, 65), (9, 23000, 33)], ids=str)
def test_blocks_of_48_kilobytes(size):
    """Rows whose part in shared memory ends at what a launch may ask for without opting in."""
    z, ids, q, w = inputs(size, "f32", 11)
    all_ways(z, ids, q, w, 1.0, "f32", str(size))


def test_a_teacher_that_is_not_finite():
    z, ids, q, w = inputs((6, 900, 5), "f32", 12, pad=0.0)
    ids = torch.arange(5, device="cuda", dtype=torch.int32).repeat(6, 1) * 100
    clean = train.distill_grad(z, ids, q, w)
    q[1, 2], q[4, 0] = float("nan"), float("inf")
    loss, dz = train.distill_grad(z, ids, q, w)
    keep = [0, 2, 3, 5]
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(dz[keep], clean[1][keep])
    assert bool(torch.isnan(loss[[1, 4]]).all())
    named = torch.zeros(900, dtype=torch.bool, device="cuda")
    named[::100][:5] = True
    for row in (1, 4):
        assert bool(torch.isnan(dz[row][named]).all()) and bool(torch.isfinite(dz[row][~named]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [130, 4099, 60001])
def test_rows_apart_and_in_place(V, dtype):
    """Rows of a wider array: only their own logits are read and written; dz in z's place."""
    z, ids, q, w = inputs((9, V, 20), dtype, 2)
    for pad in (1, 8, 13):
        wide = torch.full((9, V + pad), float("nan"), dtype=z.dtype, device="cuda")
        wide[:, :V] = z
        view = wide[:, :V]
        loss, dz, loss2, dz2 = all_ways(view, ids, q, w, 1.0, dtype, f"{V} + {pad}")
        assert dz.stride() == view.stride()
        own = train.distill(view, ids, q)
        out = train.distill_bwd(view, ids, q, own[1], own[2], w, 0.25, out=view)
        assert out is view and torch.equal(view, dz) and bool(torch.isnan(wide[:, V:]).all())
        view.copy_(z)
        got, out = train.distill_grad(view, ids, q, w, 0.25, out=view)
        assert out is view and torch.equal(view, dz2) and torch.equal(got, loss2)
        assert bool(torch.isnan(wide[:, V:]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 500, 9001])
def test_one_entry_is_the_cross_entropy(V, dtype):
    z, _, _, _ = inputs((50, V, 1), dtype, 3)
    label = torch.randint(0, V, (50, 1), device="cuda")
    label[::7] = -100
    loss, dz = train.distill_grad(z, label, torch.full((50, 1), -3.25, device="cuda"))
    zd = z.double().requires_grad_()
    want = torch.nn.functional.cross_entropy(zd, label[:, 0], reduction="none", ignore_index=-100)
    want.sum().backward()
    # log sum exp and one difference: a few hundred roundings at the worst
    assert float((loss.double() - want.detach()).abs().max()) <= 100 * seq_ref.U * 16
    room = 100 * seq_ref.U * 16 + seq_ref.HALF_STEP[dtype] * zd.grad.abs()
    assert bool(((dz.double() - zd.grad).abs() <= room).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 300, 5003, 60001])
def test_an_id_many_times(V, dtype):
    """All entries the same id, and ids that only share low bits: one gradient each, in full."""
    N, K = 6, 130
    z, _, q, w = inputs((N, V, K), dtype, 4)
    ids = torch.full((N, K), V - 1, dtype=torch.int32, device="cuda")
    ids[1] = torch.arange(K, device="cuda") % 3
    ids[2] = torch.arange(K, device="cuda") * 8192 % V
    ids[3] = (torch.arange(K, device="cuda") // 2 * 2048) % V
    all_ways(z, ids, q, w, 1.0, dtype, f"V {V}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [64, 1024, 7001, 120001])
def test_rows_that_count_for_nothing(V, dtype):
    """No entry, entries of -inf, weight 0: zeros, also where z is NaN or infinite; other rows are as without them."""
    N, K = 8, 12
    z, ids, q, w = inputs((N, V, K), dtype, 5, pad=0.0)
    ids = ids.abs() % V
    clean = train.distill_grad(z, ids, q, w)
    ids[2] = -1
    q[3] = -float("inf")
    w[4] = 0.0
    z[2], z[3], z[4] = float("nan"), float("inf"), float("-inf")
    loss, dz = train.distill_grad(z, ids, q, w)
    first, zmax, zlog = train.distill(z, ids, q)
    back = train.distill_bwd(z, ids, q, zmax, zlog, w)
    for d in (dz, back):
        assert not bool(d[2:5].any()) and bool(torch.isfinite(d).all())
    for got in (loss, first):
        assert not bool(got[2:4].any()) and bool(torch.isnan(got[4]))
    keep = [0, 1, 5, 6, 7]
    assert torch.equal(dz[keep], clean[1][keep]) and torch.equal(loss[keep], clean[0][keep])
    # a row that is not finite, and counts, is NaN, and the others are not
    w[4] = 1.0
    loss, dz = train.distill_grad(z, ids, q, w)
    assert bool(torch.isnan(dz[4]).all()) and torch.equal(dz[keep], clean[1][keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 2000, 70001])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_masked_logits(tau, V, dtype):
    """-inf and the type's lowest value among the logits; all of a row at the lowest value."""
    low = torch.finfo(TORCH_DT[dtype]).min
    z, ids, q, w = inputs((6, V, 5), dtype, 6, pad=0.0)
    ids = torch.arange(5, device="cuda", dtype=torch.int32).repeat(6, 1) * 7 % V
    z[0, 40:] = -float("inf")
    z[1, 40:] = low
    z[2, :] = low
    z[3, :3] = -float("inf")       # ids 0 among them: an infinite loss
    z[4, -1] = 80.0 if dtype == "f32" else 64.0
    named = list(range(6))
    named.remove(3)
    loss, zmax, zlog = train.distill(z, ids, q, tau)
    loss2, dz = train.distill_grad(z, ids, q, w, 1.0, tau)
    assert bool(torch.isinf(loss[3])) and bool(loss[3] > 0) and bool(torch.isinf(loss2[3]))
    n = [to_np(t) for t in (z, ids, q, w)]
    n[1] = n[1].astype(np.int64)
    (rl, bl), rm, (rg, bg) = seq_ref.distill_fwd(n[0], n[1], n[2], tau)
    within(loss[named], rl[named], bl[named], "f32", "loss")
    within(loss2[named], rl[named], bl[named], "f32", "loss at once")
    ref, bound = seq_ref.distill_bwd(n[0], n[1], n[2], rm, rg, n[3], 1.0, tau, bg)
    within(dz, ref, bound, dtype, "dz at once")
    within(train.distill_bwd(z, ids, q, zmax, zlog, w, 1.0, tau), ref, bound, dtype, "dz")


@pytest.mark.parametrize("size", [(5, 130, 7), (5, 4099, 40), (3, 60001, 64)], ids=str)
def test_ids_whose_low_half_is_in_range(size):
    """64-bit ids beyond 32 bits are outside of the vocabulary, whatever their low half says."""
    z, _, q, w = inputs(size, "bf16", 15)
    ids = torch.arange(size[2], device="cuda").repeat(size[0], 1)
    far = ids.clone()
    far[:, ::3] += 1 << 32
    far[:, 1::3] -= 1 << 32
    out = ids.clone()
    out[:, ::3], out[:, 1::3] = -1, size[1]
    for a, b in zip(train.distill_grad(z, far, q, w), train.distill_grad(z, out, q, w)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tau", [2.0 ** -60, 2.0 ** 60])
def test_temperatures_at_their_limits(tau):
    """The largest logit takes all of P, or every logit the same: the losses and gradients stay finite."""
    z, ids, q, w = inputs((4, 5003, 6), "f32", 16, pad=0.0)
    ids = torch.arange(6, device="cuda", dtype=torch.int32).repeat(4, 1)
    loss, dz = train.distill_grad(z, ids, q, w, temperature=tau)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dz).all())
    if tau > 1:  # P = 1 / V, p = 1 / K
        want = tau * tau * np.log(5003 / 6)
        assert float((loss / want - 1).abs().max()) <= 1e-5


def test_no_rows_and_refusals():
    z = torch.zeros((0, 10), device="cuda")
    ids, q = torch.zeros((0, 2), dtype=torch.int32, device="cuda"), torch.zeros((0, 2), device="cuda")
    assert train.distill(z, ids, q)[0].shape == (0,)
    loss, dz = train.distill_grad(z, ids, q)
    assert loss.shape == (0,) and dz.shape == (0, 10)
    z, ids, q, w = inputs((4, 30, 3), "f32")
    for bad in (lambda: train.distill(z, ids.float(), q), lambda: train.distill(z, ids, q[:, :2]),
                lambda: train.distill(z.t().contiguous().t(), ids, q), lambda: train.distill(z.half(), ids, q),
                lambda: train.distill(z, ids[:3], q[:3]), lambda: train.distill_grad(z, ids, q, w.double()),
                lambda: train.distill_grad(z, ids, q, w, out=z.bfloat16()), lambda: train.distill(z, ids.cpu(), q),
                lambda: train.distill_bwd(z, ids, q, w[:3], w), lambda: train.distill_grad(z, ids, q, out=z[:, :29])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: train.distill(z, ids, q, 0.0), lambda: train.distill(z, ids, q, float("nan")),
                lambda: train.distill_grad(z, ids, q, scale=float("inf")),
                lambda: train.distill(z.view(-1)[1:91].view(3, 30), ids[:3], q[:3])):
        with pytest.raises(train.binding.ConvError):
            bad()


def test_run_to_run_on_a_stream_and_in_a_graph():
    z, ids, q, w = inputs((40, 20011, 64), "bf16", 7)
    want = train.distill_grad(z, ids, q, w)
    first = train.distill(z, ids, q)
    back = train.distill_bwd(z, ids, q, first[1], first[2], w)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(train.distill_grad(z, ids, q, w), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = train.distill_grad(z, ids, q, w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = train.distill(z, ids, q)
        b = train.distill_bwd(z, ids, q, a[1], a[2], w)
        c = train.distill_grad(z, ids, q, w)
    for _ in range(2):
        for t in (*a, b, *c):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip((*a, b, *c), (*first, back, *want)))


def test_beyond_32_bits():
    """More than 2^31 logits: the last rows are computed at their own place."""
    N, V = 70_000, 32_003
    z = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    z[-3:] = inputs((3, V, 9), "bf16", 8)[0]
    ids = torch.arange(9, device="cuda", dtype=torch.int32).repeat(N, 1) * 3000
    q = torch.zeros((N, 9), device="cuda")
    n = to_np(z[-3:]), ids[-3:].cpu().numpy().astype(np.int64), to_np(q[-3:])
    loss, out = train.distill_grad(z, ids, q, out=z)
    # (the order of a row's sums, and so its bits, go by the number of rows: the reference's bounds hold for any)
    (rl, bl), rm, (rg, bg) = seq_ref.distill_fwd(*n, 1.0)
    within(loss[-3:], rl, bl, "f32", "loss")
    within(out[-3:], *seq_ref.distill_bwd(*n, rm, rg, None, 1.0, 1.0, bg), "bf16", "dz")
    # even logits: log V - log 9 each
    assert float((loss[:-3] - (np.log(V) - np.log(9))).abs().max()) < 1e-4


def test_c_entry_points():
    z, ids, q, w = inputs((5, 3001, 17), "bf16", 9)
    d = train.make_distill_desc(z, ids, q, 2.0)
    loss, zmax, zlog = (torch.empty(5, device="cuda") for _ in range(3))
    dz, dz2 = torch.empty_like(z), torch.empty_like(z)
    train.conv_distill_fwd(d, z, ids, q, loss, zmax, zlog)
    train.conv_distill_bwd(d, z, ids, q, zmax, zlog, None, 0.5, dz)
    want = train.distill(z, ids, q, 2.0)
    assert all(torch.equal(a, b) for a, b in zip((loss, zmax, zlog), want))
    assert torch.equal(dz, train.distill_bwd(z, ids, q, zmax, zlog, None, 0.5, 2.0))
    train.conv_distill_grad(d, z, ids, q, w, 0.5, loss, dz2)
    assert torch.equal(dz2, train.distill_grad(z, ids, q, w, 0.5, 2.0)[1])
