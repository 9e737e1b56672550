"""The gradient of the loss against a teacher's top logits is laid out as the logits are: another layout, which would
be written behind its end, is refused before the library is called.  No GPU: tensors with a device and no memory."""
import pytest

from implicit_gemm_conv2d_gb300 import build, train


def test_another_layout_is_refused():
    torch = pytest.importorskip("torch")
    from torch._subclasses.fake_tensor import FakeTensorMode

    build.build()
    with FakeTensorMode(allow_non_fake_inputs=True):
        def f(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:1")

        wide, ids, q, row = f(5, 120), f(5, 3, dtype=torch.int32), f(5, 3), f(5)
        z = wide[:, :100]
        d = train.make_distill_desc(z, ids, q)
        assert (d.N, d.V, d.ld) == (5, 100, 120)
        for dz in (torch.empty_like(z, memory_format=torch.contiguous_format), f(4, 120)[:, :100], wide,
                   f(5, 121)[:, :100], f(500)):
            with pytest.raises(ValueError, match="z's sizes and distances"):
                train.conv_distill_bwd(d, z, ids, q, row, row, None, 1.0, dz)
            with pytest.raises(ValueError, match="z's sizes and distances"):
                train.conv_distill_grad(d, z, ids, q, None, 1.0, row, dz)
