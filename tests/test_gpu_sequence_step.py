"""The example training step of the sequence model: its loss and gradients against the same step in fp64 by
autograd on the CPU, the update, and the same states whether a sequence runs at once or token by token."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("sequence_step", os.path.join(ROOT, "examples", "sequence_step.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod  # dataclasses look their module up
    spec.loader.exec_module(mod)
    return mod


def _logits(ex, q, tokens, fresh):
    F, B, T = torch.nn.functional, *tokens.shape
    stream = q["table"][tokens.long()] * ex.WIDTH ** 0.5
    for k in range(ex.LAYERS):
        y = F.layer_norm(stream, (ex.WIDTH,), q[f"gamma{k}"], q[f"beta{k}"], ex.EPS)
        both = y @ q[f"in{k}"]
        x, z = both[..., :ex.WIDTH], torch.sigmoid(both[..., ex.WIDTH:])
        h, state = [], torch.zeros((B, ex.WIDTH), dtype=torch.float64)
        for t in range(T):
            state = state.masked_fill(fresh[:, t, None], 0.0)
            state = state + z[:, t] * (x[:, t] - state)
            h.append(state)
        stream = stream + torch.stack(h, 1) @ q[f"out{k}"]
    return F.layer_norm(stream, (ex.WIDTH,), q["gamma"], q["beta"], ex.EPS).reshape(B * T, -1) @ q["head"]


def _reference(ex, p, batch):
    """Loss and gradients in fp64."""
    q = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items()}
    ids, tau = batch.ids.long().cpu(), ex.TEMPERATURE
    logp = torch.log_softmax(_logits(ex, q, batch.tokens.cpu(), batch.fresh.cpu()) / tau, dim=1)
    teacher = torch.softmax(batch.teacher.double().cpu() / tau, dim=1)
    rows = (teacher * (teacher.log() - logp.gather(1, ids.clamp(min=0)))).sum(dim=1) * (ids[:, 0] >= 0)
    loss = tau * tau * rows.mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in q.items()}


# Relative error of a gradient in the 2-norm.  fp32: about twenty operators and products one behind the other, each
# within 1e-5 of fp64 by itself.  bf16: every stored tensor is rounded by up to 2^-8, some twenty of them in a row with
# random signs give 2^-8 * sqrt(20) < 2 %, and a norm's division, which takes a part of a value away, up to a few times
# that; a wrong term is of order 1.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-4), (torch.bfloat16, 1e-1)])
def test_gradients_and_update(dtype, tol):
    ex = _example()
    p, batch = ex.make_params(dtype, "cuda"), ex.make_batch(5, 77, "cuda")
    want_loss, want = _reference(ex, p, batch)
    loss, grads = ex.loss_and_grads(p, batch)
    assert abs(loss.item() - want_loss.item()) <= tol * want_loss.item()
    assert list(grads) == list(p)
    for name, g in grads.items():
        diff, scale = (g.double().cpu() - want[name]).norm().item(), want[name].norm().item()
        assert diff <= tol * scale, (name, diff, scale)
    total = torch.sqrt(sum((g * g).sum() for g in want.values())).item()
    before = {k: v.clone() for k, v in p.items()}
    _, norm = ex.step(p, batch, lr=0.5, max_norm=0.25 * total)
    assert abs(norm.item() - total) <= tol * total
    # the clipped gradient has norm 0.25 total; in bf16 the parameters' own rounding adds noise
    if dtype == torch.float32:
        moved = torch.sqrt(sum((p[k].double() - before[k].double()).square().sum() for k in p)).item()
        assert abs(moved - 0.125 * total) <= 2 * tol * 0.125 * total


def test_step_in_a_graph_while_an_eager_one_lives():
    """The whole backward in a captured graph, beside the results of an eager run of the same parameters."""
    ex = _example()
    p, batch = ex.make_params(torch.bfloat16, "cuda"), ex.make_batch(3, 200, "cuda")
    loss, grads = ex.loss_and_grads(p, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ex.loss_and_grads(p, batch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss2, grads2 = ex.loss_and_grads(p, batch)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, loss2) and all(torch.equal(grads[k], grads2[k]) for k in grads)


def test_token_by_token():
    """fp32: the logits behind each token are those of the sequence at once.  A logit is a sum of 256 products of
    normed values, within a few hundred roundings of its terms' size (about 1) either way."""
    ex = _example()
    p, batch = ex.make_params(torch.float32, "cuda"), ex.make_batch(4, 40, "cuda")
    at_once, _ = ex.forward(p, batch.tokens)
    at_once = at_once.view(4, 40, -1)
    states = [torch.zeros((4, ex.WIDTH), device="cuda") for _ in range(ex.LAYERS)]
    for t in range(40):
        logits, _ = ex.forward(p, batch.tokens[:, t:t + 1].contiguous(), states=states)
        assert float((logits - at_once[:, t]).abs().max()) <= 1e-3
    assert ex.generate(p, batch.tokens[:, :10].contiguous(), 5).shape == (4, 5)


def test_command_runs(capsys):
    _example().main(["--batch", "2", "--length", "64", "--steps", "3", "--dtype", "bf16"])
    out = capsys.readouterr().out
    assert "ms a step" in out and "generated" in out
