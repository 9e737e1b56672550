"""A call runs on the current device: tensors on another one are refused before anything is
allocated or enqueued.  The tensors here have a device and sizes but no memory (torch's fake
tensors), so no GPU is needed and none is touched."""
import pytest

torch = pytest.importorskip("torch")

from torch._subclasses.fake_tensor import FakeTensorMode  # noqa: E402

from implicit_gemm_conv2d_gb300 import binding, train  # noqa: E402

OTHER = "cuda:1"


@pytest.fixture(scope="module")
def t():
    train.binding._build.build()
    with FakeTensorMode(allow_non_fake_inputs=True):
        def f(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=OTHER)

        return dict(x=f(2, 8, 6), gamma=f(8), stat=f(2, 2), idx=f(10, dtype=torch.int32), table=f(4, 8), rows=f(10, 8))


CALLS = {
    "group_norm": lambda t: train.group_norm(t["x"], 2, t["gamma"], t["gamma"]),
    "group_norm_bwd": lambda t: train.group_norm_bwd(t["x"], t["x"], 2, t["gamma"], t["gamma"], t["stat"], t["stat"]),
    "embed": lambda t: train.embed(t["idx"], t["table"]),
    "embed_bwd": lambda t: train.embed_bwd(t["idx"], t["rows"], 4),
    "grad_norm": lambda t: train.grad_norm([t["x"], t["gamma"]]),
    "clip_grads": lambda t: train.clip_grads([t["x"]], 1.0),
    "clip_grads out": lambda t: train.clip_grads([t["x"]], 1.0, out=[t["x"]]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_allocating_functions_refuse_another_device(t, name):
    with pytest.raises(ValueError, match="not the current device"):
        CALLS[name](t)


def test_c_entry_points_refuse_another_device(t, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="not the current device"):
        binding._ptr(t["x"])
    with pytest.raises(ValueError, match="not the current device"):
        train.make_grads([t["x"]])
