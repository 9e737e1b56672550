"""The loss against a teacher's top logits on the host (no GPU): arguments are refused before any CUDA
call, and the fp64 reference's gradient agrees with central differences."""
import ctypes

import numpy as np
import pytest

from implicit_gemm_conv2d_gb300 import build, train

from . import seq_ref

OK, ODD = 0x1000, 0x1008


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


def desc(**kw):
    a = dict(N=4, ld=100, V=100, K=5, dtype=0, index_dtype=0, teacher_dtype=0, temperature=1.0)
    a.update(kw)
    return train.DistillDesc(**a)


# The addresses are made up: every call here has to be one that is refused.
def calls(L, d, at=None, value=None, scale=1.0):
    def args(*names):
        return [value if name == at else OK for name in names]

    r = ctypes.addressof(d)
    head = ("z", "ids", "teacher")
    out = set()
    if at not in ("weight", "dz"):
        out.add(L.conv_distill_fwd(r, *args(*head, "loss", "zmax", "zlog"), None))
    if at != "loss":
        out.add(L.conv_distill_bwd(r, *args(*head, "zmax", "zlog", "weight"), scale, *args("dz"), None))
    if at not in ("zmax", "zlog"):
        out.add(L.conv_distill_grad(r, *args(*head, "weight"), scale, *args("loss", "dz"), None))
    return out


@pytest.mark.parametrize("bad,code", [(dict(N=-1), -2), (dict(V=0), -2), (dict(K=0), -2), (dict(ld=99), -2),
                                      (dict(dtype=2), -2), (dict(teacher_dtype=2), -2), (dict(index_dtype=2), -2),
                                      (dict(temperature=0.0), -2), (dict(temperature=-1.0), -2),
                                      (dict(temperature=float("nan")), -2), (dict(temperature=float("inf")), -2),
                                      (dict(temperature=1e-45), -2), (dict(temperature=2.0 ** -61), -2),
                                      (dict(temperature=2.0 ** 61), -2), (dict(N=1 << 27), -3),
                                      (dict(V=1 << 30, ld=1 << 30), -3), (dict(K=1025), -3), (dict(ld=1 << 32), -3)])
def test_descriptor_refused(L, bad, code):
    assert calls(L, desc(**bad)) == {code}


def test_pointers_alignment_and_scale(L):
    for name in ("z", "ids", "teacher", "loss", "zmax", "zlog", "dz"):
        assert calls(L, desc(), name, None) == {-1}
        assert calls(L, desc(), name, ODD) == {-4}
    assert calls(L, desc(), "weight", ODD) == {-4}
    r = ctypes.addressof(desc())
    for scale in (float("nan"), float("inf")):
        assert L.conv_distill_bwd(r, OK, OK, OK, OK, OK, OK, scale, OK, None) == -2
        assert L.conv_distill_grad(r, OK, OK, OK, OK, scale, OK, OK, None) == -2
    assert L.conv_distill_fwd(None, OK, OK, OK, OK, OK, OK, None) == -1
    empty = desc(N=0)
    assert L.conv_distill_fwd(ctypes.addressof(empty), None, None, None, None, None, None, None) == 0
    assert L.conv_distill_grad(ctypes.addressof(empty), None, None, None, None, 1.0, None, None, None) == 0


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    z, ids, q = torch.zeros((2, 8)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 3))
    with pytest.raises(ValueError):
        train.distill(z, ids, q)                       # CPU tensors
    with pytest.raises(ValueError):
        train.distill(z.double(), ids, q)
    with pytest.raises(ValueError):
        train.distill_grad(z, ids[:1], q)
    with pytest.raises(ValueError):
        train.distill_bwd(z, ids, q, z[:, 0], None)
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode(allow_non_fake_inputs=True):
        z, ids, q = (torch.empty(s, dtype=t, device="cuda:1") for s, t in
                     (((2, 8), torch.float32), ((2, 3), torch.int32), ((2, 3), torch.float32)))
        for call in (train.distill, train.distill_grad):
            with pytest.raises(ValueError, match="not the current device"):
                call(z, ids, q)


@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_reference_gradient_against_differences(tau):
    rng = np.random.default_rng(6)
    N, V, K = 4, 9, 5
    z, q, w = rng.normal(size=(N, V)), rng.normal(size=(N, K)), rng.normal(size=N)
    ids = rng.integers(0, V, size=(N, K))
    ids[0, 1] = ids[0, 0]
    ids[1] = -1
    ids[2, 0] = V

    def loss():
        return float((seq_ref.distill_fwd(z, ids, q, tau)[0][0] * w).sum() * 0.7)

    _, m, (log, _) = seq_ref.distill_fwd(z, ids, q, tau)
    dz, _ = seq_ref.distill_bwd(z, ids, q, m, log, w, 0.7, tau)
    assert not dz[1].any()
    h = 1e-6
    for k in range(z.size):
        old = z.flat[k]
        z.flat[k] = old + h
        hi = loss()
        z.flat[k] = old - h
        lo = loss()
        z.flat[k] = old
        # central difference: h^2 f''' / 6 and 2^-52 |f| / h, both below 1e-8 here
        assert abs((hi - lo) / (2 * h) - dz.flat[k]) < 1e-7
