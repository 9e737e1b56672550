"""The gated scan on the host (no GPU): arguments are refused before any CUDA call, and the fp64
reference's gradients agree with central differences."""
import ctypes

import numpy as np
import pytest

from implicit_gemm_conv2d_gb300 import build, train

from . import seq_ref

OK, ODD = 0x1000, 0x1001
ARRAYS = ("x", "gate", "h", "dh", "dx", "dgate")


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


def desc(rows=None, **kw):
    a = dict(B=4, T=10, D=6, dtype=0)
    a.update(kw)
    d = train.ScanDesc(a["B"], a["T"], a["D"], a["dtype"])
    for n in ARRAYS:
        setattr(d, n, train.Rows(60, 6))
    for n, r in (rows or {}).items():
        setattr(d, n, train.Rows(*r))
    return d


# The addresses are made up: every call here has to be one that is refused.
def fwd(L, d, x=OK, gate=OK, h0=None, lengths=None, h=OK, last=OK, ws=None):
    return L.conv_scan_fwd(ctypes.addressof(d), x, gate, h0, None, lengths, h, last, ws, 0, None)


def bwd(L, d, x=OK, gate=OK, h=OK, dh=OK, h0=None, dlast=None, lengths=None, dx=OK, dgate=OK, dh0=None, ws=None):
    return L.conv_scan_bwd(ctypes.addressof(d), x, gate, h, dh, h0, dlast, None, lengths, dx, dgate, dh0, ws, 0, None)


@pytest.mark.parametrize("bad,code", [(dict(B=-1), -2), (dict(T=-1), -2), (dict(D=0), -2), (dict(dtype=2), -2),
                                      (dict(B=2 ** 31 - 1), -3), (dict(T=2 ** 31 - 1, B=1), -3),
                                      (dict(B=1 << 20, D=1 << 17, rows={n: (1 << 21, 1 << 17) for n in ARRAYS}), -3),
                                      (dict(rows=dict(x=(-60, 6))), -2), (dict(rows=dict(gate=(60, -6))), -2),
                                      (dict(rows=dict(x=(1 << 62, 6))), -3)])
def test_descriptor_refused(L, bad, code):
    d = desc(**bad)
    assert (fwd(L, d), bwd(L, d)) == (code, code)
    assert L.conv_scan_fwd_workspace_size(ctypes.addressof(d)) == 0
    assert L.conv_scan_bwd_workspace_size(ctypes.addressof(d)) == 0


@pytest.mark.parametrize("rows", [(59, 6), (60, 5), (0, 6), (6, 23), (5, 60), (60, 0)])
def test_outputs_whose_rows_overlap_are_refused(L, rows):
    assert fwd(L, desc(rows=dict(h=rows))) == -2
    assert bwd(L, desc(rows=dict(dx=rows))) == -2
    assert bwd(L, desc(rows=dict(dgate=rows))) == -2


def test_pointers_and_alignment(L):
    for name in ("x", "gate", "h"):
        assert fwd(L, desc(), **{name: None}) == -1
        assert fwd(L, desc(), **{name: ODD}) == -4
        assert fwd(L, desc(dtype=1), **{name: ODD}) == -4
    for name in ("x", "gate", "h", "dh", "dx", "dgate"):
        assert bwd(L, desc(), **{name: None}) == -1
        assert bwd(L, desc(), **{name: ODD + 1}) == -4
    for name in ("h0", "last", "lengths", "ws"):
        assert fwd(L, desc(), **{name: ODD}) == -4
    for name in ("h0", "dlast", "dh0", "lengths", "ws"):
        assert bwd(L, desc(), **{name: ODD}) == -4
    assert L.conv_scan_fwd(None, OK, OK, None, None, None, OK, OK, None, 0, None) == -1
    assert L.conv_scan_bwd(None, OK, OK, OK, OK, None, None, None, None, OK, OK, None, None, 0, None) == -1
    assert fwd(L, desc(B=0), None, None, None, None, None, None) == 0
    assert bwd(L, desc(B=0), None, None, None, None, None, None, None, None, None, None) == 0


def test_outputs_over_inputs_are_refused(L):
    a, b, c, e, f, g = (OK + 0x1000 * i for i in range(6))
    for name in ("x", "gate"):
        assert fwd(L, desc(), **{**dict(x=a, gate=b, h=c), name: c}) == -2
    for out in ("dx", "dgate"):
        for name in ("x", "gate", "h", "dh", "dx", "dgate"):
            if name != out:
                args = dict(x=a, gate=b, h=c, dh=e, dx=f, dgate=g)
                assert bwd(L, desc(), **{**args, out: args[name]}) == -2


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 8, 3))
    with pytest.raises(ValueError):
        train.gated_scan(x, x)                       # CPU tensors
    with pytest.raises(ValueError):
        train.gated_scan(x[0], x[0])
    with pytest.raises(ValueError):
        train.gated_scan(x.double(), x.double())
    with pytest.raises(ValueError):
        train.gated_scan_bwd(x, x, x, x)
    with pytest.raises(ValueError):
        train.make_scan_desc(x, x[:, :4], x)
    d = train.make_scan_desc(x, x.transpose(0, 1).contiguous().transpose(0, 1), x[:1].expand(2, 8, 3))
    assert [(r.batch, r.step) for r in (d.x, d.gate, d.h)] == [(24, 3), (3, 6), (0, 3)]


def test_wrong_companions_are_refused():
    """Sizes and dtypes that do not fit x, on tensors that have a device and no memory."""
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode

    build.build()
    with FakeTensorMode(allow_non_fake_inputs=True):
        def f(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:1")

        with pytest.raises(ValueError, match="not the current device"):
            train.gated_scan(f(2, 8, 4), f(2, 8, 4))
        with pytest.raises(ValueError, match="not the current device"):
            train.gated_scan_bwd(f(2, 8, 4), f(2, 8, 4), f(2, 8, 4), f(2, 8, 4))


@pytest.mark.parametrize("options", [{}, dict(reset=True), dict(lengths=True), dict(reset=True, lengths=True)])
def test_reference_gradient_against_differences(options):
    rng = np.random.default_rng(5)
    B, T, D = 3, 7, 2
    x, gate = rng.normal(size=(B, T, D)), rng.normal(size=(B, T, D))
    h0, dh, dlast = rng.normal(size=(B, D)), rng.normal(size=(B, T, D)), rng.normal(size=(B, D))
    reset = rng.random((B, T)) < 0.3 if options.get("reset") else None
    lengths = np.array([7, 0, 4]) if options.get("lengths") else None

    def loss():
        h, last, _, _ = seq_ref.scan_fwd(x, gate, h0, reset, lengths)
        return float((h * dh).sum() + (last * dlast).sum())

    h = seq_ref.scan_fwd(x, gate, h0, reset, lengths)[0]
    (dx, _), (dg, _), (dh0, _) = seq_ref.scan_bwd(x, gate, h, dh, h0, dlast, reset, lengths)
    step = 1e-6
    for a, grad in ((x, dx), (gate, dg), (h0, dh0)):
        for k in range(a.size):
            old = a.flat[k]
            a.flat[k] = old + step
            hi = loss()
            a.flat[k] = old - step
            lo = loss()
            a.flat[k] = old
            # central difference: step^2 f''' / 6 and 2^-52 |f| / step, both below 1e-8 here
            assert abs((hi - lo) / (2 * step) - grad.flat[k]) < 1e-7
