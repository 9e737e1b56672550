"""Training steps of a small recurrent sequence model on the library's operators (one GPU), taught by
another model's top logits:

    tokens -> embedding table -> layers of [norm of the residual sum -> projection -> gated scan -> projection]
    -> norm -> logits;  loss: distance from the teacher's distribution over its K best tokens
    backward -> global norm of all gradients, clipped -> SGD

Rows hold several sequences one behind the other; the scan starts anew at each one's first token.  The
projections are torch products; everything else is this library's.  ``generate`` runs the model token
by token, each layer's state kept in place.  Data, teacher and weights are synthetic.

    python examples/sequence_step.py --batch 16 --length 512 --steps 50 --dtype bf16
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

from implicit_gemm_conv2d_gb300 import train  # noqa: E402

ROWS, WIDTH, LAYERS, K = 1000, 256, 2, 16
TEMPERATURE = 2.0
EPS = 1e-5


@dataclass
class Batch:
    tokens: torch.Tensor    # (B, T), int32
    fresh: torch.Tensor     # (B, T), bool: a sequence begins here
    ids: torch.Tensor       # (B * T, K), int32: the teacher's best tokens; -1 in a row that is not to be learnt
    teacher: torch.Tensor   # (B * T, K), fp32: its logits at them


def make_params(dtype, device, seed: int = 0) -> dict:
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, scale):
        return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)

    p = {"table": rand(ROWS, WIDTH, scale=WIDTH ** -0.5)}
    for k in range(LAYERS):
        p[f"gamma{k}"] = torch.ones(WIDTH, dtype=dtype, device=device)
        p[f"beta{k}"] = torch.zeros(WIDTH, dtype=dtype, device=device)
        p[f"in{k}"] = rand(WIDTH, 2 * WIDTH, scale=WIDTH ** -0.5)
        p[f"out{k}"] = rand(WIDTH, WIDTH, scale=WIDTH ** -0.5)
    p["gamma"], p["beta"] = torch.ones(WIDTH, dtype=dtype, device=device), torch.zeros(WIDTH, dtype=dtype, device=device)
    p["head"] = rand(WIDTH, ROWS, scale=WIDTH ** -0.5)
    return p


def make_batch(B: int, T: int, device, seed: int = 1) -> Batch:
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, ROWS, (B, T), generator=g, dtype=torch.int32)
    fresh = torch.rand((B, T), generator=g) < 1.0 / 64.0
    fresh[:, 0] = True
    # a teacher that knows its answer by the last token: K ids from it on
    ids = (tokens.long().reshape(-1, 1) * 7 + torch.arange(K) * 13) % ROWS
    ids[torch.rand(B * T, generator=g) < 0.05] = -1
    teacher = 6.0 - torch.arange(K) * 0.7 + 0.3 * torch.randn((B * T, K), generator=g)
    return Batch(tokens.to(device), fresh.to(device), ids.int().to(device), teacher.to(device))


def forward(p: dict, tokens, fresh=None, states=None):
    """The logits (B * T, ROWS) and what the backward takes.  states: the layers' (B, WIDTH), which the
    sequences begin with and which are brought up to date in place."""
    B, T = tokens.shape
    kept = []
    stream, delta = None, train.embed(tokens, p["table"], WIDTH ** 0.5)
    for k in range(LAYERS):
        y, total, mean, rstd = train.layer_norm(delta, p[f"gamma{k}"], p[f"beta{k}"], residual=stream, eps=EPS)
        stream = delta if total is None else total
        both = (y.view(B * T, WIDTH) @ p[f"in{k}"]).view(B, T, 2 * WIDTH)
        state = None if states is None else states[k]
        h, _ = train.gated_scan(both[..., :WIDTH], both[..., WIDTH:], state, reset=fresh, last=state)
        delta = (h.view(B * T, WIDTH) @ p[f"out{k}"]).view(B, T, WIDTH)
        kept.append((stream, y, mean, rstd, both, h))
    y, total, mean, rstd = train.layer_norm(delta, p["gamma"], p["beta"], residual=stream, eps=EPS)
    logits = y.view(B * T, WIDTH) @ p["head"]
    return logits, (kept, total, y, mean, rstd)


def loss_and_grads(p: dict, batch: Batch):
    """The mean loss (a device scalar) and the gradient of every parameter."""
    B, T = batch.tokens.shape
    logits, (kept, total, y, mean, rstd) = forward(p, batch.tokens, batch.fresh)
    losses, dz = train.distill_grad(logits, batch.ids, batch.teacher, scale=1.0 / (B * T), temperature=TEMPERATURE,
                                    out=logits)
    g = {"head": y.view(B * T, WIDTH).t() @ dz}
    dy = (dz @ p["head"].t()).view(B, T, WIDTH)
    # the gradient of the stream, which is that of the layer's own output too
    flow, g["gamma"], g["beta"] = train.layer_norm_bwd(total, dy, p["gamma"], mean, rstd)
    for k in reversed(range(LAYERS)):
        stream, y, mean, rstd, both, h = kept[k]
        ddelta = flow.view(B * T, WIDTH)
        g[f"out{k}"] = h.view(B * T, WIDTH).t() @ ddelta
        dh = (ddelta @ p[f"out{k}"].t()).view(B, T, WIDTH)
        dboth = torch.empty_like(both)
        train.gated_scan_bwd(both[..., :WIDTH], both[..., WIDTH:], h, dh, reset=batch.fresh, dx=dboth[..., :WIDTH],
                             dgate=dboth[..., WIDTH:])
        dboth = dboth.view(B * T, 2 * WIDTH)
        g[f"in{k}"] = y.view(B * T, WIDTH).t() @ dboth
        dy = (dboth @ p[f"in{k}"].t()).view(B, T, WIDTH)
        flow, g[f"gamma{k}"], g[f"beta{k}"] = train.layer_norm_bwd(stream, dy, p[f"gamma{k}"], mean, rstd, dtotal=flow)
    g["table"] = train.embed_bwd(batch.tokens, flow, ROWS, WIDTH ** 0.5)
    return losses.mean(), {name: g[name] for name in p}


def step(p: dict, batch: Batch, lr: float, max_norm: float):
    """One update in place; the loss and the gradients' norm before clipping (device scalars)."""
    loss, g = loss_and_grads(p, batch)
    norm = train.clip_grads(list(g.values()), max_norm)
    torch._foreach_add_(list(p.values()), list(g.values()), alpha=-lr)
    return loss, norm


def generate(p: dict, tokens, count: int):
    """The next ``count`` tokens (the likeliest each) behind the sequences ``tokens`` (B, T): the sequences at
    once, then a token at a time."""
    B = tokens.shape[0]
    states = [torch.zeros((B, WIDTH), device=tokens.device) for _ in range(LAYERS)]
    logits, _ = forward(p, tokens, states=states)
    token = logits.view(B, -1, ROWS)[:, -1].argmax(dim=1, keepdim=True).int()
    out = [token]
    for _ in range(count - 1):
        logits, _ = forward(p, token, states=states)
        token = logits.argmax(dim=1, keepdim=True).int()
        out.append(token)
    return torch.cat(out, 1)


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--length", type=int, default=512)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--max-norm", type=float, default=1.0)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args(argv)
    dtype = torch.float32 if a.dtype == "f32" else torch.bfloat16
    p, batch = make_params(dtype, "cuda"), make_batch(a.batch, a.length, "cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == min(5, a.steps - 1):
            start.record()
        loss, norm = step(p, batch, a.lr, a.max_norm)
        if i % max(1, a.steps // 10) == 0 or i == a.steps - 1:
            print(f"step {i}: loss {loss.item():.5f}, gradient norm {norm.item():.4f}")
    end.record()
    torch.cuda.synchronize()
    steps = max(1, a.steps - min(5, a.steps - 1))
    print(f"{start.elapsed_time(end) / steps:.3f} ms a step, {a.batch} x {a.length} tokens, {a.dtype}")
    print("generated:", generate(p, batch.tokens[:2, :32].contiguous(), 8).tolist())


if __name__ == "__main__":
    main()
