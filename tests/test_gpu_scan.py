"""The gated scan on the GPU against the fp64 reference, forward and backward: lengths from nothing to
thousands of steps, odd numbers of steps and channels, padded rows, resets, strided and time-first
inputs, infinities and NaN behind a reset or a row's end, the state kept in place, another stream, a
captured graph, run to run.  Tolerances: the bound that comes with the reference plus the rounding of
the result as it is kept (seq_ref)."""
import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import seq_ref
from .gpu_cases import TORCH_DT, to_np

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (3, 1, 5), (96, 1, 130), (1, 2, 2), (7, 5, 33), (300, 9, 8), (2, 17, 33), (1, 129, 64), (40, 64, 16),
         (5, 777, 31), (1, 1000, 1), (2, 1025, 72), (1, 2500, 16), (1, 3000, 260), (3, 4099, 6), (700, 40, 3),
         (1000, 37, 130), (20000, 21, 6), (40, 200, 520),
         (1, 9001, 24), (2, 20011, 9), (1, 5000, 70)]
OPTIONS = {
    "plain": {},
    "state": dict(h0=True),
    "packed": dict(reset=0.05),
    "padded": dict(lengths=True, h0=True),
    "everything": dict(reset=0.1, lengths=True, h0=True, layout="joined"),
    "time_first": dict(h0=True, layout="time_first"),
    "joined": dict(layout="joined"),
}


def lay(a, dtype, layout, other=None):
    """The array on the GPU: dense, time first, or the first part of a joined one."""
    t = torch.from_numpy(np.ascontiguousarray(a)).float().cuda().to(TORCH_DT[dtype])
    if layout == "time_first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "joined":
        both = torch.full((*t.shape[:2], 2 * t.shape[2] + 1), float("nan"), dtype=t.dtype, device="cuda")
        view = both[..., :t.shape[2]] if other is None else both[..., t.shape[2]:2 * t.shape[2]]
        view.copy_(t)
        return view
    return t


def inputs(size, dtype, seed=0, h0=False, reset=0.0, lengths=False, layout="dense"):
    B, T, D = size
    rng = np.random.default_rng(seed + B + 7 * T + 31 * D)
    dev = {"x": lay(rng.normal(size=size), dtype, layout),
           "gate": lay(rng.normal(size=size) * 1.5 - 4.0 * rng.random(D), dtype, layout, True),
           "dh": lay(rng.normal(size=size), dtype, layout)}
    side = {"h0": None, "reset": None, "lengths": None, "dlast": None}
    if h0:
        side["h0"] = torch.from_numpy(rng.normal(size=(B, D))).float().cuda()
        side["dlast"] = torch.from_numpy(rng.normal(size=(B, D))).float().cuda()
    if reset:
        side["reset"] = torch.from_numpy(rng.random((B, T)) < reset).cuda()
    if lengths:
        n = rng.integers(-1, T + 2, size=B)
        n[0] = T
        side["lengths"] = torch.from_numpy(n).int().cuda()
    return dev, side


def numbers(t):
    return None if t is None else t.cpu().numpy() if not t.is_floating_point() else to_np(t)


def within(out, ref, bound, dtype, what):
    out = to_np(out)
    room = bound + seq_ref.HALF_STEP[dtype] * (np.abs(ref) + bound)
    bad = np.abs(out - ref) > room
    assert out.shape == ref.shape and not bad.any(), \
        f"{what}: {np.abs(out - ref)[bad].max():.3e} at {np.argwhere(bad)[0]} of room {room[bad].min():.3e}"


def both_ways(size, dtype, **options):
    dev, side = inputs(size, dtype, **options)
    what = f"{size} {dtype} {options}"
    h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"], side["lengths"])
    n = {k: numbers(v) for k, v in {**dev, **side}.items()}
    rh, rl, bh, bl = seq_ref.scan_fwd(n["x"], n["gate"], n["h0"], n["reset"], n["lengths"])
    within(h, rh, bh, dtype, what + " h")
    within(last, rl, bl, "f32", what + " last")
    dx, dgate, dh0 = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"], side["reset"],
                                          side["lengths"])
    refs = seq_ref.scan_bwd(n["x"], n["gate"], to_np(h), n["dh"], n["h0"], n["dlast"], n["reset"], n["lengths"])
    for name, out, (ref, bound) in zip(("dx", "dgate"), (dx, dgate), refs):
        within(out, ref, bound, dtype, f"{what} {name}")
    assert (dh0 is None) == (side["h0"] is None)
    if dh0 is not None:
        within(dh0, *refs[2], "f32", what + " dh0")
    return dev, side, (h, last, dx, dgate)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("options", list(OPTIONS))
def test_against_the_reference(options, size, dtype):
    both_ways(size, dtype, **OPTIONS[options])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(140, 150, 260), (250, 33, 75), (60, 700, 70), (30, 700, 70), (330, 65, 64), (3, 700, 1030), (2, 900, 778), (1, 9000, 70)], ids=str)
@pytest.mark.parametrize("options", ["plain", "everything"])
def test_walks_from_shared_memory_and_clusters_of_each_size(options, size, dtype):
    both_ways(size, dtype, **OPTIONS[options])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_steps_no_rows(dtype):
    dev, side = inputs((4, 0, 6), dtype, h0=True)
    h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"])
    assert h.shape == (4, 0, 6) and torch.equal(last, side["h0"])
    assert not train.gated_scan(dev["x"], dev["gate"])[1].any()
    dx, dgate, dh0 = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"])
    assert dx.shape == dgate.shape == (4, 0, 6) and torch.equal(dh0, side["dlast"])
    dev, side = inputs((0, 5, 6), dtype)
    h, last = train.gated_scan(dev["x"], dev["gate"])
    assert h.shape == (0, 5, 6) and last.shape == (0, 6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_run_to_run(dtype):
    dev, side = inputs((2, 5000, 70), dtype, h0=True, reset=0.01)
    runs = []
    for _ in range(3):
        h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"])
        runs.append((h, last, *train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"],
                                                    side["reset"])))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


@pytest.mark.parametrize("T", [1, 30, 3000, 20000])
def test_state_in_place_and_outputs_given(T):
    dev, side = inputs((5, T, 44), "bf16", h0=True, layout="joined")
    h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"])
    state = side["h0"].clone()
    room = torch.full((T, 5, 44), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    h2, last2 = train.gated_scan(dev["x"], dev["gate"], state, out=room, last=state)
    assert h2 is room and last2 is state and torch.equal(h, room) and torch.equal(last, state)
    dx, dgate, _ = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"])
    grad = torch.full((5, T, 89), 7.0, dtype=torch.bfloat16, device="cuda")
    train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], dx=grad[..., :44], dgate=grad[..., 44:88])
    assert torch.equal(grad[..., :44], dx) and torch.equal(grad[..., 44:88], dgate) and bool((grad[..., 88] == 7).all())


@pytest.mark.parametrize("size", [(300, 9, 8), (1000, 37, 130), (40, 200, 520), (5, 777, 31), (2, 1025, 72), (1, 9001, 24)],
                         ids=str)
def test_side_arrays_anywhere(size):
    """States, lengths and flags at addresses that are only their elements'; flags of any value but 0."""
    dev, side, (h, last, dx, dgate) = both_ways(size, "bf16", h0=True, reset=0.05, lengths=True)

    def moved(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        room[1:] = t.reshape(-1)
        return room[1:].view(t.shape)

    flags = side["reset"].to(torch.uint8) * torch.randint(1, 256, side["reset"].shape, device="cuda").to(torch.uint8)
    h0, lengths, dlast = moved(side["h0"]), moved(side["lengths"]), moved(side["dlast"])
    h2, last2 = train.gated_scan(dev["x"], dev["gate"], h0, moved(flags), lengths, last=moved(side["h0"]))
    assert torch.equal(h2, h) and torch.equal(last2, last)
    got = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], h0, dlast, moved(flags), lengths)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dgate)


def test_outputs_over_inputs_are_refused():
    dev, side = inputs((3, 20, 8), "f32")
    h, _ = train.gated_scan(dev["x"], dev["gate"])
    for bad in (lambda: train.gated_scan(dev["x"], dev["gate"], out=dev["x"]),
                lambda: train.gated_scan(dev["x"], dev["gate"], out=dev["gate"]),
                lambda: train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], dx=dev["dh"]),
                lambda: train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], dgate=h)):
        with pytest.raises(train.binding.ConvError):
            bad()


def test_steps_one_by_one_are_the_sequence():
    """A rollout's steps with the state kept in place: step t's state is the sequence's, within both bounds."""
    dev, side = inputs((6, 50, 20), "f32", h0=True)
    n = {k: numbers(v) for k, v in {**dev, **side}.items()}
    rh, _, bh, _ = seq_ref.scan_fwd(n["x"], n["gate"], n["h0"])
    state = side["h0"].clone()
    for t in range(50):
        h, _ = train.gated_scan(dev["x"][:, t:t + 1], dev["gate"][:, t:t + 1], state, last=state)
        within(h, rh[:, t:t + 1], bh[:, t:t + 1], "f32", f"step {t}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 100, 3000])
def test_what_is_not_finite_stays_in_its_sequence(T, dtype):
    """NaN and infinities in front of a reset, and behind a row's end, reach nothing else."""
    B, D, cut, end = 3, 40, T // 2, T - 1
    dev, side = inputs((B, T, D), dtype, h0=True)
    side["reset"] = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    side["reset"][:, cut] = True
    side["lengths"] = torch.full((B,), end, dtype=torch.int32, device="cuda")
    clean = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"], side["lengths"])
    cleanb = train.gated_scan_bwd(dev["x"], dev["gate"], clean[0], dev["dh"], side["h0"], side["dlast"], side["reset"],
                                  side["lengths"])
    bad = {k: v.clone() for k, v in dev.items()}
    for k, v in zip(("x", "gate", "dh"), (float("nan"), float("inf"), float("-inf"))):
        bad[k][:, end:] = v
    h, last = train.gated_scan(bad["x"], bad["gate"], side["h0"], side["reset"], side["lengths"])
    hb = h.clone()
    hb[:, end:] = float("nan")
    back = train.gated_scan_bwd(bad["x"], bad["gate"], hb, bad["dh"], side["h0"], side["dlast"], side["reset"],
                                side["lengths"])
    assert torch.equal(h, clean[0]) and torch.equal(last, clean[1])
    assert all(torch.equal(a, b) for a, b in zip(back, cleanb))
    # the old sequence's values: nothing beyond the reset changes
    bad["x"][:, cut - 1] = float("nan")
    h0 = torch.full_like(side["h0"], float("inf"))
    h, last = train.gated_scan(bad["x"], bad["gate"], h0, side["reset"], side["lengths"])
    assert torch.equal(h[:, cut:], clean[0][:, cut:]) and torch.equal(last, clean[1])
    assert not bool(torch.isfinite(h[:, :cut]).any())
    # and a gradient that is not finite behind the reset does not flow in front of it
    dlast = torch.full_like(side["dlast"], float("nan"))
    dx, dgate, dh0 = train.gated_scan_bwd(dev["x"], dev["gate"], clean[0], dev["dh"], side["h0"], dlast, side["reset"],
                                          side["lengths"])
    assert torch.equal(dx[:, :cut], cleanb[0][:, :cut]) and torch.equal(dgate[:, :cut], cleanb[1][:, :cut])
    assert torch.equal(dh0, cleanb[2])


def test_gates_at_the_ends_of_their_range():
    """z exactly 0 keeps the state, z exactly 1 replaces it, and neither gives a NaN in the gradient."""
    g = torch.tensor([-float("inf"), -1e30, -200.0, -90.0, 90.0, 200.0, 1e30, float("inf")], device="cuda")
    gate = g.view(1, 1, 8).repeat(2, 6, 1)
    x = torch.randn((2, 6, 8), device="cuda")
    h0 = torch.randn((2, 8), device="cuda")
    h, last = train.gated_scan(x, gate, h0)
    assert torch.equal(h[..., :4], h0[:, None, :4].expand(2, 6, 4))
    within(h[..., 4:], to_np(x[..., 4:]), np.abs(to_np(x[..., 4:])) * 4 * seq_ref.U + 8 * seq_ref.U * 4, "f32", "z = 1")
    dx, dgate, dh0 = train.gated_scan_bwd(x, gate, h, torch.ones_like(x), h0, torch.ones_like(h0))
    assert bool(torch.isfinite(dx).all()) and bool((dgate.abs() < 1e-37).all()) and bool(torch.isfinite(dh0).all())
    assert bool((dx[..., :4].abs() < 1e-36).all()) and torch.equal(dh0[:, :4], torch.full((2, 4), 7.0, device="cuda"))


def test_on_another_stream_and_in_a_graph():
    dev, side = inputs((3, 1500, 48), "bf16", h0=True, reset=0.02)
    want = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"])
    grads = train.gated_scan_bwd(dev["x"], dev["gate"], want[0], dev["dh"], side["h0"], side["dlast"], side["reset"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"], stream=s)
    back = train.gated_scan_bwd(dev["x"], dev["gate"], got[0], dev["dh"], side["h0"], side["dlast"], side["reset"], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"])
        out = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"], side["reset"])
    for _ in range(2):
        for t in (h, last, *out):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((h, last, *out), (*want, *grads)))


def test_rows_beyond_32_bits():
    """Rows whose offsets pass 2^31 elements, in a view of few of them."""
    base = torch.zeros((2 ** 31 + 8192,), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (2, 70, 24), (2 ** 31, 40, 1))
    gate = torch.as_strided(base, (2, 70, 24), (2 ** 31, 40, 1), 3000)
    dev, _ = inputs((2, 70, 24), "bf16")
    x.copy_(dev["x"])
    gate.copy_(dev["gate"] - 3.0)
    h, last = train.gated_scan(x, gate)
    want = train.gated_scan(x.contiguous(), gate.contiguous())
    assert torch.equal(h, want[0]) and torch.equal(last, want[1])
    dx = torch.as_strided(base, (2, 70, 24), (2 ** 31, 40, 1))
    back = train.gated_scan_bwd(dev["x"], gate, h, dev["dh"], dx=dx)
    wantb = train.gated_scan_bwd(dev["x"], gate.contiguous(), h, dev["dh"])
    assert torch.equal(dx, wantb[0]) and torch.equal(back[1], wantb[1])


def test_pieces_of_time():
    """Few channels over many steps, in pieces: what is not finite in one stays in its sequence, and a workspace that
    is too small is refused."""
    B, T, D = 1, 20000, 24
    dev, side = inputs((B, T, D), "f32", h0=True)
    side["reset"] = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    side["reset"][:, [9000, 9001, 15000]] = True
    d = train.make_scan_desc(dev["x"], dev["gate"], dev["x"], dev["dh"], dev["x"], dev["x"])
    need = train.conv_scan_fwd_workspace_size(d)
    assert need > 0 and train.conv_scan_bwd_workspace_size(d) > 0
    clean = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"])
    back = train.gated_scan_bwd(dev["x"], dev["gate"], clean[0], dev["dh"], side["h0"], side["dlast"], side["reset"])
    bad = dev["x"].clone()
    bad[:, 5000] = float("nan")
    h, last = train.gated_scan(bad, dev["gate"], side["h0"], side["reset"])
    assert torch.equal(h[:, :5000], clean[0][:, :5000]) and torch.equal(h[:, 9000:], clean[0][:, 9000:])
    assert bool(torch.isnan(h[:, 5000:9000]).all()) and torch.equal(last, clean[1])
    bad = dev["dh"].clone()
    bad[:, 12000] = float("inf")
    dx, dgate, dh0 = train.gated_scan_bwd(dev["x"], dev["gate"], clean[0], bad, side["h0"], side["dlast"], side["reset"])
    assert torch.equal(dx[:, 12001:], back[0][:, 12001:]) and torch.equal(dx[:, :9001], back[0][:, :9001])
    assert torch.equal(dgate[:, :9001], back[1][:, :9001]) and torch.equal(dh0, back[2])
    assert not bool(torch.isfinite(dx[:, 9001:12001]).any())
    out, ws = torch.empty_like(dev["x"]), torch.empty(need, dtype=torch.uint8, device="cuda")
    for room in (None, ws[:need - 8]):
        with pytest.raises(train.binding.ConvError, match="(?i)workspace"):
            train.conv_scan_fwd(d, dev["x"], dev["gate"], None, None, None, out, None, room)
    train.conv_scan_fwd(d, dev["x"], dev["gate"], side["h0"], side["reset"].view(torch.uint8), None, out, None, ws.fill_(255))
    assert torch.equal(out, clean[0])


def test_c_entry_points():
    dev, side = inputs((3, 90, 26), "bf16", h0=True, reset=0.05, layout="joined")
    want = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"])
    grads = train.gated_scan_bwd(dev["x"], dev["gate"], want[0], dev["dh"], side["h0"], side["dlast"], side["reset"])
    h = torch.empty((90, 3, 26), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    dx, dgate = torch.empty_like(want[0]), torch.empty_like(want[0])
    d = train.make_scan_desc(dev["x"], dev["gate"], h, dev["dh"], dx, dgate)
    reset = side["reset"].view(torch.uint8)
    last = torch.empty_like(side["h0"])
    train.conv_scan_fwd(d, dev["x"], dev["gate"], side["h0"], reset, None, h, last, None)
    assert torch.equal(h, want[0]) and torch.equal(last, want[1])
    train.conv_scan_fwd(d, dev["x"], dev["gate"], side["h0"], reset, None, h, None, None)
    dh0 = torch.empty_like(side["h0"])
    train.conv_scan_bwd(d, dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"], reset, None, dx, dgate, dh0, None)
    assert all(torch.equal(a, b) for a, b in zip((dx, dgate, dh0), grads))
