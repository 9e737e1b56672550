"""The sequence operators at the largest sizes that they accept, and with several calls at once."""
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import test_gpu_distill, test_gpu_ln, test_gpu_scan

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1
STEPS = MOST - 2 ** 20 - 1


def pattern(n, dtype=torch.bfloat16):
    """1, 2, .. 7, 1, ..: values that bf16 holds."""
    return (torch.arange(7, device="cuda") + 1).to(dtype).repeat(n // 7 + 1)[:n]


def same(a, b):
    """Equal, looked at in parts (some torch operations count with 32 bits)."""
    a, b = a.reshape(-1), b.reshape(-1)
    return all(torch.equal(u, v) for u, v in zip(a.split(2 ** 30), b.split(2 ** 30)))


def test_norm_of_the_most_rows():
    """Rows of one value without a mean: y = x / sqrt(x^2 + eps)."""
    x = pattern(MOST).view(MOST, 1)
    y, _, _, rstd = train.layer_norm(x, eps=0.0, rms=True)
    assert all(bool((t == 1).all()) for t in y.view(-1).split(2 ** 30))
    dy = torch.zeros_like(x)
    dy[-5:] = 1
    dx, dgamma, _ = train.layer_norm_bwd(x, dy, None, None, rstd)
    assert float(dgamma) == 5.0
    assert not any(bool(t.any()) for t in dx[:-5].view(-1).split(2 ** 30)) and float(dx[-5:].abs().max()) <= 2.0 ** -8


def test_loss_of_the_most_rows():
    N = 2 ** 27 - 1
    z = torch.zeros((N, 2), device="cuda")
    ids = torch.ones((N, 1), dtype=torch.int32, device="cuda")
    loss, dz = train.distill_grad(z, ids, torch.zeros((N, 1), device="cuda"))
    assert float((loss - 0.6931472).abs().max()) <= 1e-6
    assert float((dz[:, 0] - 0.5).abs().max()) <= 1e-6 and float((dz[:, 1] + 0.5).abs().max()) <= 1e-6


def test_loss_over_the_most_logits():
    """All alike: every partial sum is a whole number that fp32 holds, the last is 2^30 - 1 to a rounding."""
    V = 2 ** 30 - 1
    z = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0, V - 1, V, -1]], device="cuda")
    q = torch.zeros((1, 4), device="cuda")
    want = 30 * 0.6931472 - 0.6931472
    for loss, zmax, zlog in [train.distill(z, ids, q)]:
        assert abs(float(loss) - want) <= 1e-5 and float(zmax) == 0.0
        dz = train.distill_bwd(z, ids, q, zmax, zlog)
    loss, dz2 = train.distill_grad(z, ids, q)
    assert abs(float(loss) - want) <= 1e-5
    for d in (dz, dz2):
        assert float(d[0, 0]) == float(d[0, -1]) == -0.5
        assert abs(float(d[0, 1]) * 2.0 ** 30 - 1) <= 2.0 ** -7 and bool((d[0, 1:-1] == d[0, 1]).all())


@pytest.mark.parametrize("size", [(1, STEPS, 1), (STEPS, 1, 1), (1, 1, STEPS), (1, STEPS // 16, 16)], ids=str)
def test_scan_of_the_most(size):
    """A gate of 40 is open (z = 1): every state is its step's x, and dx is dh."""
    x = pattern(size[0] * size[1] * size[2]).view(size)
    gate = torch.full_like(x, 40.0)
    h, last = train.gated_scan(x, gate)
    assert same(h, x)
    assert same(last.to(torch.bfloat16), x[:, -1])
    del last
    dx, dgate, _ = train.gated_scan_bwd(x, gate, h, x)
    assert same(dx, x)


# ---- several calls at once ---------------------------------------------------------------------
def scan_calls(size, dtype, **options):
    dev, side = test_gpu_scan.inputs(size, dtype, **options)

    def call():
        h, last = train.gated_scan(dev["x"], dev["gate"], side["h0"], side["reset"], side["lengths"])
        dx, dgate, dh0 = train.gated_scan_bwd(dev["x"], dev["gate"], h, dev["dh"], side["h0"], side["dlast"],
                                              side["reset"], side["lengths"])
        return h, last, dx, dgate, dh0
    return call


def loss_calls(size, dtype):
    z, ids, q, w = test_gpu_distill.inputs(size, dtype, 21)

    def call():
        loss, zmax, zlog = train.distill(z, ids, q)
        return loss, train.distill_bwd(z, ids, q, zmax, zlog, w), *train.distill_grad(z, ids, q, w)
    return call


def norm_calls(size, dtype):
    t = test_gpu_ln.inputs(size, dtype, 22)

    def call():
        a = train.layer_norm(t["x"], t["gamma"], t["beta"], t["residual"])
        return (*a, *train.layer_norm_bwd(a[1], t["dy"], t["gamma"], a[2], a[3], t["dtotal"]))
    return call


CALLS = {
    "pieces": lambda: scan_calls((1, 9001, 24), "bf16", h0=True, reset=0.01),
    "clusters": lambda: scan_calls((4, 3000, 130), "f32", h0=True, lengths=True),
    "walks": lambda: scan_calls((140, 150, 260), "bf16", h0=True),
    "loss": lambda: loss_calls((40, 30011, 40), "bf16"),
    "loss_short": lambda: loss_calls((3000, 700, 9), "f32"),
    "norm": lambda: norm_calls((4000, 1430), "f32"),
    "norm_long": lambda: norm_calls((40, 9001), "bf16"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_calls_on_two_streams_and_two_graphs_at_once(name):
    call = CALLS[name]()
    want = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, kept = [], []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kept.append(call())
        graphs.append(g)
    got = []
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                got.append(call())
                g.replay()
    torch.cuda.synchronize()
    for out in got + kept:
        assert all(torch.equal(a, b) for a, b in zip((t for t in out if t is not None), want))
    assert train.binding.conv_device_status() == 0
