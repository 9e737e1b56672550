"""Global gradient norm and clipping on the GPU against fp64: lists of one to many hundred
tensors, both types mixed, empty tensors, views that start off a 16-byte boundary, in place and
into other tensors, norms below and above the limit, non-finite gradients, run to run.

Tolerances: the norm to 1e-5 relative (the conv tests' fp32 figure; squares are added in short
chains and trees); a clipped value to 1e-5 (fp32) or 8e-3 (bf16) relative to itself."""
import math

import numpy as np
import pytest
import torch

from implicit_gemm_conv2d_gb300 import train

from . import train_ref
from .gpu_cases import TOL, TORCH_DT, to_np

pytestmark = pytest.mark.gpu

LISTS = {
    "one_value": [1],
    "one": [1000],
    "encoder": [128 * 59 * 25, 128, 128 * 128 * 9, 128, 128, 128, 4096, 33, 1],
    "tile_edges": [16383, 16384, 16385, 32768, 7, 8, 9],
    "with_empty": [0, 17, 0, 0, 40000, 0],
    "all_empty": [0, 0],
    "many": [1 + 37 * (i % 19) for i in range(1300)],
    "large": [3_000_001, 12, 5_000_000],
}


def make(sizes, dtype, seed=0, odd=False):
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtype if dtype != "mixed" else ("f32", "bf16")[i % 2]
        off = 1 + i % 7 if odd else 0
        base = torch.from_numpy(rng.normal(size=n + off).astype(np.float32)).cuda().to(TORCH_DT[dt])
        out.append(base[off:])
    return out


def rel(a, b):
    return abs(a - b) / b if b else abs(a)


def check_clip(grads, outs, max_norm, norm, host):
    want = train_ref.grad_norm(host)
    assert rel(float(norm), want) <= 1e-5
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o, h in zip(grads, outs, host):
        tol = TOL["f32" if o.dtype == torch.float32 else "bf16"]
        assert (np.abs(to_np(o) - h * coef) <= tol * np.abs(h * coef)).all()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("name", list(LISTS))
def test_norm_and_clip(name, dtype, odd):
    grads = make(LISTS[name], dtype, odd=odd)
    host = [to_np(g) for g in grads]
    n1, n2 = train.grad_norm(grads), train.grad_norm(grads)
    assert torch.equal(n1, n2) and n1.shape == ()
    assert rel(float(n1), train_ref.grad_norm(host)) <= 1e-5
    for limit in (0.37, 1e6):
        out = [torch.full_like(g, 7.0) for g in grads]
        norm = train.clip_grads(grads, limit, out=out)
        assert torch.equal(norm, n1)
        check_clip(grads, out, limit, norm, host)
        if limit == 1e6:
            assert all(torch.equal(g, o) for g, o in zip(grads, out))
    mine = [g.clone() for g in grads]
    train.clip_grads(mine, 0.37)
    out = [torch.empty_like(g) for g in grads]
    train.clip_grads(grads, 0.37, out=out)
    assert all(torch.equal(a, b) for a, b in zip(mine, out))


def test_in_place_on_views_leaves_the_neighbours():
    flat = torch.randn(100_003, device="cuda")
    keep = flat.clone()
    cuts = [0, 3, 20, 21, 40_000, 99_999]
    views = [flat[a + 1:b] for a, b in zip(cuts[:-1], cuts[1:])]
    host = [to_np(v) for v in views]
    norm = train.clip_grads(views, 1.0)
    check_clip(views, views, 1.0, norm, host)
    for c in cuts:
        assert flat[c] == keep[c]
    assert torch.equal(flat[99_999:], keep[99_999:])


def test_other_alignment_of_output():
    g = torch.randn(50_000, device="cuda", dtype=torch.bfloat16)
    o = torch.zeros(50_003, device="cuda", dtype=torch.bfloat16)
    norm = train.clip_grads([g], 0.5, out=[o[3:]])
    check_clip([g], [o[3:]], 0.5, norm, [to_np(g)])
    assert not o[:3].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_non_finite(dtype):
    grads = make([1000, 40_000], dtype)
    grads[1][77] = float("inf")
    out = [torch.empty_like(g) for g in grads]
    norm = train.clip_grads(grads, 1.0, out=out)
    assert math.isinf(float(norm)) and torch.isnan(out[1][77])
    out[1][77] = 0
    assert not any(o.any() for o in out)
    grads[1][77] = float("nan")
    norm = train.clip_grads(grads, 1.0, out=out)
    assert math.isnan(float(norm)) and all(torch.isnan(o).all() for o in out)


def test_zero_gradients_and_zero_limit():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(5, device="cuda", dtype=torch.bfloat16)]
    assert float(train.clip_grads(grads, 1.0)) == 0.0 and not any(g.any() for g in grads)
    grads = make([3000], "f32")
    train.clip_grads(grads, 0.0)
    assert not grads[0].any()


def test_follows_the_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = [torch.randn(100_000, device="cuda") for _ in range(3)]
        want = train_ref.grad_norm([to_np(t) for t in g])
    norm = train.clip_grads(g, 1.0, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert rel(float(norm), want) <= 1e-5
    assert rel(float(train.grad_norm(g)), 1.0 / (1 + 1e-6 / want)) <= 1e-5


def test_small_workspace_refused():
    g = make([100_000], "f32")
    arr = train.make_grads(g)
    norm = torch.zeros((), device="cuda")
    size = train.conv_grad_norm_workspace_size(arr, 1)
    for ws in (None, torch.empty(size - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(train.binding.ConvError) as e:
            train.conv_grad_norm(arr, 1, norm, ws)
        assert e.value.status == -5
