"""Training steps of a small encoder on the library's operators (one GPU):

    conv1 + bias -> group norm, ReLU -> conv2 + bias -> group norm, SiLU -> map features
    attributes (47 a sample) -> embedding table                           -> attribute features
    head: one dot product of both feature sets a sample;  loss: mean squared error
    backward -> global norm of all gradients, clipped -> SGD

The conv shapes are PufferLib PR #522's encoder's (59 -> 128 channels, 11 x 15, K = 5, S = 3; then
128 -> 128, K = 3, S = 1), the table its 128 rows of 32.  The head and the update are torch calls;
everything else is this library's.  Data and weights are synthetic.

    python examples/encoder_step.py --batch 1024 --steps 50 --dtype bf16
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from implicit_gemm_conv2d_gb300 import binding, train  # noqa: E402

ATTRIBUTES, ROWS, WIDTH = 47, 128, 32
IC, OC, H, W = 59, 128, 11, 15
K1, S1, K2, S2 = 5, 3, 3, 1
H1, W1 = (H - K1) // S1 + 1, (W - K1) // S1 + 1
H2, W2 = (H1 - K2) // S2 + 1, (W1 - K2) // S2 + 1
GROUPS = 16
EPS = 1e-5
PADDING = 0   # the attribute value that stands for "none"


@dataclass
class Batch:
    x: torch.Tensor       # (B, IC, H, W)
    idx: torch.Tensor     # (B, ATTRIBUTES), int32
    target: torch.Tensor  # (B,), fp32


def make_params(dtype, device, seed: int = 0) -> dict:
    """Kept in the order of the update; gammas start at 1 and betas at 0."""
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, scale):
        return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)

    def const(v):
        return torch.full((OC,), v, dtype=dtype, device=device)

    return {
        "w1": rand(OC, IC, K1, K1, scale=(IC * K1 * K1) ** -0.5), "b1": const(0.0),
        "gamma1": const(1.0), "beta1": const(0.0),
        "w2": rand(OC, OC, K2, K2, scale=(OC * K2 * K2) ** -0.5), "b2": const(0.0),
        "gamma2": const(1.0), "beta2": const(0.0),
        "table": rand(ROWS, WIDTH, scale=1.0),
        "head": rand(OC * H2 * W2 + ATTRIBUTES * WIDTH, scale=(OC * H2 * W2 + ATTRIBUTES * WIDTH) ** -0.5),
    }


def make_batch(B: int, dtype, device, seed: int = 1) -> Batch:
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand((B, IC, H, W), generator=g) < 0.1).to(dtype)
    idx = torch.randint(0, ROWS, (B, ATTRIBUTES), generator=g, dtype=torch.int32)
    return Batch(x.to(device), idx.to(device), torch.randn(B, generator=g).to(device))


def loss_and_grads(p: dict, batch: Batch):
    """The mean squared error (a device scalar) and the gradient of every parameter."""
    B = batch.x.shape[0]
    # forward
    a1 = binding.fwd(batch.x, p["w1"], S1, False, bias=p["b1"])
    h1, mean1, rstd1 = train.group_norm(a1, GROUPS, p["gamma1"], p["beta1"], EPS, "relu")
    a2 = binding.fwd(h1, p["w2"], S2, False, bias=p["b2"])
    h2, mean2, rstd2 = train.group_norm(a2, GROUPS, p["gamma2"], p["beta2"], EPS, "silu")
    attr = train.embed(batch.idx, p["table"], WIDTH ** -0.5, PADDING)
    feats = torch.cat((h2.reshape(B, -1), attr.reshape(B, -1)), 1)
    err = (feats @ p["head"]).float() - batch.target
    loss = (err * err).mean()
    # backward
    g = {}
    dout = (2.0 / B * err).to(feats.dtype)
    g["head"] = feats.t() @ dout
    dfeats = dout[:, None] * p["head"][None, :]
    split = OC * H2 * W2
    dh2 = dfeats[:, :split].reshape(B, OC, H2, W2).contiguous()
    dattr = dfeats[:, split:].reshape(B, ATTRIBUTES, WIDTH).contiguous()
    g["table"] = train.embed_bwd(batch.idx, dattr, ROWS, WIDTH ** -0.5, PADDING)
    da2, g["gamma2"], g["beta2"] = train.group_norm_bwd(a2, dh2, GROUPS, p["gamma2"], p["beta2"], mean2, rstd2, "silu")
    g["b2"] = binding.bwd_bias(da2, None, False)
    g["w2"] = binding.bwd_filter(h1, da2, None, K2, S2, False)
    dh1 = binding.bwd_data(da2, p["w2"], None, H1, W1, S2, False)
    da1, g["gamma1"], g["beta1"] = train.group_norm_bwd(a1, dh1, GROUPS, p["gamma1"], p["beta1"], mean1, rstd1, "relu")
    g["b1"] = binding.bwd_bias(da1, None, False)
    g["w1"] = binding.bwd_filter(batch.x, da1, None, K1, S1, False)
    return loss, {name: g[name] for name in p}


def step(p: dict, batch: Batch, lr: float, max_norm: float):
    """One update in place; the loss and the gradients' norm before clipping (device scalars)."""
    loss, g = loss_and_grads(p, batch)
    norm = train.clip_grads(list(g.values()), max_norm)
    torch._foreach_add_(list(p.values()), list(g.values()), alpha=-lr)
    return loss, norm


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--lr", type=float, default=0.05)
    ap.add_argument("--max-norm", type=float, default=1.0)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args(argv)
    dtype = torch.float32 if a.dtype == "f32" else torch.bfloat16
    p, batch = make_params(dtype, "cuda"), make_batch(a.batch, dtype, "cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == min(5, a.steps - 1):
            start.record()
        loss, norm = step(p, batch, a.lr, a.max_norm)
        if i % max(1, a.steps // 10) == 0 or i == a.steps - 1:
            print(f"step {i}: loss {loss.item():.5f}, gradient norm {norm.item():.4f}")
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end) / max(1, a.steps - min(5, a.steps - 1)):.3f} ms a step, batch {a.batch}, {a.dtype}")


if __name__ == "__main__":
    main()
