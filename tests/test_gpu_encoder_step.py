"""The example training step: its loss, gradients, norm and update against the same step in fp64
by autograd on the CPU, and a few steps that have to bring the loss down."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("encoder_step", os.path.join(ROOT, "examples", "encoder_step.py"))
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules[spec.name] = mod  # dataclasses look their module up
    spec.loader.exec_module(mod)
    return mod


def _reference(ex, p, batch):
    """Loss and gradients in fp64."""
    q = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items()}
    F = torch.nn.functional
    x, idx, B = batch.x.double().cpu(), batch.idx.long().cpu(), batch.x.shape[0]
    h = F.conv2d(x, q["w1"], q["b1"], ex.S1)
    h = torch.relu(F.group_norm(h, ex.GROUPS, q["gamma1"], q["beta1"], ex.EPS))
    h = F.conv2d(h, q["w2"], q["b2"], ex.S2)
    h = F.silu(F.group_norm(h, ex.GROUPS, q["gamma2"], q["beta2"], ex.EPS))
    attr = q["table"][idx] * ex.WIDTH ** -0.5 * (idx != ex.PADDING)[..., None]
    out = torch.cat((h.reshape(B, -1), attr.reshape(B, -1)), 1) @ q["head"]
    loss = ((out - batch.target.double().cpu()) ** 2).mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in q.items()}


# Relative error of a gradient in the 2-norm.  fp32: the convs' 3xTF32 products and fp32 sums are
# within 1e-5 of fp64 by themselves, a chain of six operators with a norm's division between them
# within ten times that; a ReLU whose z lies within rounding of 0 may switch, one of 1e5 values or
# so, which moves a gradient by up to 1e-3.  bf16: every stored tensor is rounded to 2^-9, eight of
# them in a row and their sums' conditions give a few per cent; a wrong term is of order 1.  The
# biases before a norm have a gradient of exactly 0 plus what the group's other channels leave;
# they are measured against the norm of all gradients instead.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-3), (torch.bfloat16, 1e-1)])
def test_gradients_and_update(dtype, tol):
    ex = _example()
    p, batch = ex.make_params(dtype, "cuda"), ex.make_batch(37, dtype, "cuda")
    want_loss, want = _reference(ex, p, batch)
    loss, grads = ex.loss_and_grads(p, batch)
    assert abs(loss.item() - want_loss.item()) <= tol * want_loss.item()
    total = torch.sqrt(sum((g * g).sum() for g in want.values())).item()
    for name, g in grads.items():
        diff = (g.double().cpu() - want[name]).norm().item()
        scale = total if name in ("b1", "b2") else want[name].norm().item()
        assert diff <= tol * scale, (name, diff, scale)
    before = {k: v.clone() for k, v in p.items()}
    _, norm = ex.step(p, batch, lr=0.5, max_norm=0.25 * total)
    assert abs(norm.item() - total) <= tol * total
    moved = torch.sqrt(sum((p[k].double() - before[k].double()).square().sum() for k in p)).item()
    # the clipped gradient has norm 0.25 total; in bf16 the parameters' own rounding adds noise
    if dtype == torch.float32:
        assert abs(moved - 0.125 * total) <= 2 * tol * 0.125 * total


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_loss_falls(dtype):
    ex = _example()
    p, batch = ex.make_params(dtype, "cuda"), ex.make_batch(64, dtype, "cuda")
    losses = [ex.step(p, batch, 0.05, 1.0)[0].item() for _ in range(30)]
    assert losses[-1] < 0.5 * losses[0]


def test_command_runs(capsys):
    _example().main(["--batch", "32", "--steps", "3"])
    assert "ms a step" in capsys.readouterr().out
