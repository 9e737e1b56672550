"""The training-step operators on the host (no GPU): the library exports what
include/conv_train.h declares, arguments are checked before any CUDA call, and the fp64
references' gradients agree with central differences."""
import ctypes
import os
import re

import numpy as np
import pytest

from implicit_gemm_conv2d_gb300 import build, train

from . import train_ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "conv_train.h")
OK, ODD = 0x1000, 0x1008


@pytest.fixture(scope="module")
def L():
    build.build()
    return train.lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(conv_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(train.EXPORTS)
    for n in names:
        assert hasattr(L, n), f"{n} declared in include/conv_train.h but not exported"


def gn_desc(**kw):
    a = dict(B=4, C=32, P=12, G=8, act=1, layout=0, dtype=0, eps=1e-5)
    a.update(kw)
    return train.GnDesc(**a)


def gn_calls(L, d, x=OK, ws=OK):
    r = ctypes.addressof(d)
    return (L.conv_gn_fwd(r, x, OK, OK, OK, OK, OK, ws, 1 << 40, None),
            L.conv_gn_bwd(r, x, OK, OK, OK, OK, OK, OK, OK, OK, ws, 1 << 40, None))


@pytest.mark.parametrize("bad", [dict(B=-1), dict(C=0), dict(P=0), dict(G=0), dict(G=5), dict(act=4), dict(act=-1),
                                 dict(layout=2), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(eps=float("inf"))])
def test_gn_descriptor_refused(L, bad):
    d = gn_desc(**bad)
    assert gn_calls(L, d) == (-2, -2)
    assert L.conv_gn_fwd_workspace_size(ctypes.addressof(d)) == 0
    assert L.conv_gn_bwd_workspace_size(ctypes.addressof(d)) == 0


def test_gn_limits_pointers_alignment(L):
    assert gn_calls(L, gn_desc(C=1 << 16, G=1, P=1 << 15)) == (-3, -3)
    assert gn_calls(L, gn_desc(B=1 << 30, C=32, G=8, P=1)) == (-3, -3)
    desc = gn_desc()
    d = ctypes.addressof(desc)
    assert gn_calls(L, gn_desc(), x=None) == (-1, -1)
    assert gn_calls(L, gn_desc(), x=ODD) == (-4, -4)
    assert gn_calls(L, gn_desc(), ws=ODD) == (-4, -4)
    assert L.conv_gn_fwd(None, OK, OK, OK, OK, OK, OK, OK, 0, None) == -1
    assert L.conv_gn_fwd(d, OK, OK, OK, None, OK, OK, OK, 0, None) == -1
    assert L.conv_gn_fwd(d, OK, OK, OK, OK, OK, None, OK, 0, None) == -1  # mean without rstd
    assert L.conv_gn_fwd(d, OK, ODD, OK, OK, OK, OK, OK, 0, None) == -4
    assert L.conv_gn_bwd(d, OK, OK, OK, OK, OK, OK, OK, OK, None, OK, 0, None) == -1  # dgamma without dbeta
    assert L.conv_gn_bwd(d, OK, OK, OK, OK, None, OK, OK, OK, OK, OK, 0, None) == -1
    assert L.conv_gn_bwd(d, OK, OK, OK, OK, OK, OK, OK, ODD, OK, OK, 0, None) == -4
    empty = gn_desc(B=0)
    assert L.conv_gn_fwd(ctypes.addressof(empty), None, None, None, None, None, None, None, 0, None) == 0


def embed_desc(**kw):
    a = dict(T=100, V=50, D=24, padding_idx=-1, index_dtype=0, dtype=0, scale=1.0)
    a.update(kw)
    return train.EmbedDesc(**a)


@pytest.mark.parametrize("bad,code", [(dict(T=-1), -2), (dict(V=0), -2), (dict(D=0), -2), (dict(index_dtype=2), -2),
                                      (dict(dtype=3), -2), (dict(scale=float("inf")), -2), (dict(T=1 << 31), -3),
                                      (dict(D=(1 << 24) + 1), -3)])
def test_embed_descriptor_refused(L, bad, code):
    d = embed_desc(**bad)
    r = ctypes.addressof(d)
    assert L.conv_embed_fwd(r, OK, OK, OK, None) == code
    assert L.conv_embed_bwd(r, OK, OK, OK, OK, 1 << 40, None) == code
    assert L.conv_embed_bwd_workspace_size(r) == 0


def test_embed_pointers_alignment(L):
    d = embed_desc()
    r = ctypes.addressof(d)
    assert L.conv_embed_fwd(None, OK, OK, OK, None) == -1
    for i in range(3):
        a = [OK] * 3
        a[i] = None
        assert L.conv_embed_fwd(r, *a, None) == -1
        assert L.conv_embed_bwd(r, *a, OK, 1 << 40, None) == -1
        a[i] = ODD
        assert L.conv_embed_fwd(r, *a, None) == -4
        assert L.conv_embed_bwd(r, *a, OK, 1 << 40, None) == -4
    assert L.conv_embed_bwd(r, OK, OK, OK, ODD, 1 << 40, None) == -4
    d0 = embed_desc(T=0)
    assert L.conv_embed_fwd(ctypes.addressof(d0), None, None, None, None) == 0
    assert L.conv_embed_bwd(ctypes.addressof(d0), None, None, None, None, 0, None) == -1  # dtable is still written


def test_grads_refused(L):
    def one(grad=OK, out=OK, n=10, dtype=0):
        return (train.Grad * 1)(train.Grad(grad, out, n, dtype))

    # The addresses are made up: every call here has to be one that is refused.
    def clip(a, count=1, norm=OK, max_norm=1.0):
        p = ctypes.addressof(a) if a is not None else None
        return L.conv_grad_clip(p, count, max_norm, norm, OK, 1 << 40, None)

    def calls(a, count=1, norm=OK):
        p = ctypes.addressof(a) if a is not None else None
        return L.conv_grad_norm(p, count, norm, OK, 1 << 40, None), clip(a, count, norm)

    assert calls(one(n=-1)) == (-2, -2)
    assert calls(one(dtype=2)) == (-2, -2)
    assert calls(one(), count=-1) == (-2, -2)
    assert calls(one(), count=(1 << 20) + 1) == (-3, -3)
    assert calls(one(n=1 << 40)) == (-3, -3)
    assert calls(None) == (-1, -1)
    assert calls(one(grad=None)) == (-1, -1)
    assert clip(one(out=None)) == -1
    assert calls(one(grad=0x1002)) == (-4, -4)          # fp32 off its element
    assert clip(one(out=0x1002)) == -4
    assert calls(one(grad=0x1001, dtype=1)) == (-4, -4)
    assert calls(one(), norm=None) == (-1, -1)
    for m in (-1.0, float("nan"), float("inf")):
        assert clip(one(), max_norm=m) == -2


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 8, 3))
    with pytest.raises(ValueError):
        train.group_norm(x.double(), 2)
    with pytest.raises(ValueError):
        train.group_norm(x, 2, act="tanh")
    with pytest.raises(ValueError):
        train.group_norm(x, 2, layout="nwhc")
    with pytest.raises(ValueError):
        train.group_norm(x, 2, gamma=torch.zeros(7))
    with pytest.raises(ValueError):
        train.group_norm(x, 2)                      # a CPU tensor
    with pytest.raises(ValueError):
        train.embed(torch.zeros(3), torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        train.embed_bwd(torch.zeros(3, dtype=torch.int64), torch.zeros((2, 5)), 4)
    with pytest.raises(ValueError):
        train.grad_norm([])
    with pytest.raises(ValueError):
        train.clip_grads([torch.zeros(3)], 1.0, out=[])
    with pytest.raises(ValueError):
        train.grad_norm([torch.zeros(3)])


# ---- the references' gradients against central differences, in fp64 --------------------------
@pytest.mark.parametrize("layout", ["nchw", "nhwc"])
@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_reference_gn_gradient_against_differences(kind, layout):
    rng = np.random.default_rng(3)
    B, C, P, G, eps = 2, 6, 5, 3, 1e-5
    x = rng.normal(size=(B, C, P) if layout == "nchw" else (B, P, C))
    gamma, beta = rng.normal(size=C), rng.normal(size=C)
    dy = rng.normal(size=x.shape)

    def loss(x, gamma, beta):
        return float((train_ref.gn_fwd(x, gamma, beta, G, eps, kind, layout)[0] * dy).sum())

    mean, rstd = train_ref.gn_stats(x, G, eps, layout)
    (dx, _), (dg, _), (db, _) = train_ref.gn_bwd(x, dy, gamma, beta, mean, rstd, G, kind, layout)
    h = 1e-6
    for a, grad in ((x, dx), (gamma, dg), (beta, db)):
        for k in rng.choice(a.size, size=min(a.size, 12), replace=False):
            old = a.flat[k]
            a.flat[k] = old + h
            hi = loss(x, gamma, beta)
            a.flat[k] = old - h
            lo = loss(x, gamma, beta)
            a.flat[k] = old
            # central difference: h^2 f''' / 6 and 2^-52 |f| / h, both below 1e-8 here
            assert abs((hi - lo) / (2 * h) - grad.flat[k]) < 1e-6


def test_reference_embedding_gradient_is_the_adjoint():
    rng = np.random.default_rng(4)
    idx = rng.integers(-2, 9, size=(5, 7))
    table, dy = rng.normal(size=(7, 3)), rng.normal(size=(5, 7, 3))
    y = train_ref.embed_fwd(idx, table, 1.5, 2)
    dt, _ = train_ref.embed_bwd(idx, dy, 7, 1.5, 2)
    assert abs((y * dy).sum() - (table * dt).sum()) < 1e-12
    assert not dt[2].any()
