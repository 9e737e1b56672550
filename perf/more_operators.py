"""What the sequence operators are measured on: the gated scan over time (forward, one step, and
backward), the loss against a teacher's top logits (its value, its gradient, both at once), and
the layer norm of a residual sum (forward and backward).

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a
case's inputs on the GPU, ``run()`` makes one pass through the operator and ``exact()`` computes
the same in 64 bits.  With ``own`` false ``run`` computes the operators' plain form out of
elementary torch operations in fp32; with ``own`` true it calls the framework's kernels."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # One step of every agent of a rollout: the state goes in and comes out.
        dict(name="scan_step_f32", op="scan_fwd", B=96, T=1, D=512, h0=True, resets=0, lengths=False, joined=False,
             dtype="f32"),
        # A training segment of many agents: 64 steps, episodes that end inside it.
        dict(name="scan_fwd_segment_f32", op="scan_fwd", B=1024, T=64, D=128, h0=True, resets=20, lengths=False,
             joined=False, dtype="f32"),
        # Two long sequences, values and gates being halves of one projection.
        dict(name="scan_fwd_long_bf16", op="scan_fwd", B=2, T=32768, D=1024, h0=False, resets=0, lengths=False,
             joined=True, dtype="bf16"),
        # Backward over rows of packed sequences, some 200 steps each.
        dict(name="scan_bwd_packed_bf16", op="scan_bwd", B=8, T=4096, D=1024, h0=False, resets=200, lengths=False,
             joined=False, dtype="bf16"),
        # Backward of a padded batch, an odd number of steps and of channels.
        dict(name="scan_bwd_padded_f32", op="scan_bwd", B=5, T=1999, D=777, h0=True, resets=0, lengths=True,
             joined=False, dtype="f32"),
        # Evaluation of a few positions over a large vocabulary.
        dict(name="distill_fwd_few_f32", op="distill_fwd", N=24, V=131071, K=128, temperature=1.0, dtype="f32"),
        # The gradient alone, for a loss whose weights follow from its values.
        dict(name="distill_bwd_vocab_f32", op="distill_bwd", N=1024, V=50021, K=32, temperature=1.0, dtype="f32"),
        # A training batch: the loss and its gradient over the same vocabulary.
        dict(name="distill_grad_vocab_bf16", op="distill_grad", N=8192, V=50021, K=64, temperature=2.0, dtype="bf16"),
        # The norm in front of a rollout's step.
        dict(name="norm_fwd_step_f32", op="norm_fwd", N=96, D=512, residual=True, rms=False, dtype="f32"),
        # A training batch of tokens.
        dict(name="norm_fwd_tokens_bf16", op="norm_fwd", N=32768, D=1024, residual=True, rms=False, dtype="bf16"),
        # Its backward, with the gradient that came around it.
        dict(name="norm_bwd_tokens_bf16", op="norm_bwd", N=32768, D=1024, residual=True, rms=False, dtype="bf16"),
        # Backward of the form without a mean, an odd number of rows.
        dict(name="norm_bwd_rms_f32", op="norm_bwd", N=6001, D=1430, residual=False, rms=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "distill_fwd", "distill_bwd", "distill_grad",
                     "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("scan_fwd", "scan_bwd"):
        cap = 67_000_000 if op == "scan_fwd" else 33_000_000
        while True:
            B, T, D = _log(rng, 1, 2048), _log(rng, 1, 65536), _log(rng, 16, 4096)
            if rng.random() < 0.7:
                D = (D + 7) // 8 * 8
            if 10_000 <= B * T * D <= (cap if dtype == "bf16" else cap // 2):
                return dict(op=op, B=B, T=T, D=D, h0=rng.random() < 0.5,
                            resets=rng.choice([0, 0, _log(rng, 10, 1000)]), lengths=rng.random() < 0.3,
                            joined=rng.random() < 0.5, dtype=dtype)
    if op in ("distill_fwd", "distill_bwd", "distill_grad"):
        while True:
            N, V = _log(rng, 1, 32768), _log(rng, 100, 200_000)
            if 10_000 <= N * V <= 200_000_000:
                return dict(op=op, N=N, V=V, K=min(V, _log(rng, 1, 256)),
                            temperature=rng.choice([1.0, 1.0, 2.0, 0.7, 4.0]), dtype=dtype)
    while True:
        N, D = _log(rng, 1, 200_000), _log(rng, 16, 8192)
        if rng.random() < 0.7:
            D = (D + 7) // 8 * 8
        if 10_000 <= N * D <= 33_000_000:
            return dict(op=op, N=N, D=D, residual=rng.random() < 0.6, rms=rng.random() < 0.4, dtype=dtype)


# ---- inputs ----------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _row_lengths(case):
    """From half of the steps to all of them."""
    B, T = case["B"], case["T"]
    return [T - (T // 2) * b // max(1, B - 1) for b in range(B)]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D = case["B"], case["T"], case["D"]
        # each channel remembers for a time of its own: from two steps to some hundred
        x, gate = _normal(g, B, T, D), _normal(g, B, T, D).sub_(5.0 * _uniform(g, D))
        if case["joined"]:
            both = torch.cat((x, gate), 2).to(dt)
            x, gate = both[..., :D], both[..., D:]
        else:
            x, gate = x.to(dt), gate.to(dt)
        s = dict(case, x=x, gate=gate, h0=_normal(g, B, D) * 0.5 if case["h0"] else None, reset=None, lengths=None)
        if case["resets"]:
            s["reset"] = _uniform(g, B, T) * case["resets"] < 1.0
        if case["lengths"]:
            order = torch.randperm(B, generator=g, device="cuda")
            s["lengths"] = torch.tensor(_row_lengths(case), dtype=torch.int32, device="cuda")[order]
        if op == "scan_bwd":
            s["h"] = _plain_scan(s)["h"]
            s["dh"] = (0.01 * _normal(g, B, T, D)).to(dt)
            s["dlast"] = 0.01 * _normal(g, B, D) if case["h0"] else None
        return s
    if op in ("distill_fwd", "distill_bwd", "distill_grad"):
        N, V, K = case["N"], case["V"], case["K"]
        z = _normal(g, N, V).mul_(2.0)
        # the teacher's K entries: any of the vocabulary, each once, falling from the first on
        step = next(p for p in (7919, 7907, 7901) if V % p)
        first = torch.randint(V, (N, 1), generator=g, device="cuda")
        rank = torch.arange(K, device="cuda")
        ids = (first + rank * step) % V
        teacher = 12.0 - 1.5 * torch.log2(1.0 + rank.float()) + 0.5 * _normal(g, N, K)
        z.scatter_add_(1, ids, 0.6 * teacher)  # a student that has learnt something already
        ids[_uniform(g, N) < 1.0 / 16.0] = -1  # rows that are padding
        s = dict(case, z=z.to(dt), ids=ids.to(torch.int32), teacher=teacher, weight=0.5 + _uniform(g, N), scale=1.0 / N)
        if op == "distill_bwd":
            zf = s["z"].float()
            s["zmax"] = zf.max(dim=1).values
            s["zlog"] = ((zf - s["zmax"][:, None]) / case["temperature"]).exp().sum(dim=1).log()
        return s
    N, D = case["N"], case["D"]
    # activations: a level and a spread of each row's own
    level, spread = 0.3 * _normal(g, N, 1), 0.5 + _normal(g, N, 1).abs()
    s = dict(case, x=(_normal(g, N, D) * spread + level).to(dt), gamma=(1.0 + 0.2 * _normal(g, D)).to(dt),
             beta=None if case["rms"] else (0.2 * _normal(g, D)).to(dt), other=None)
    if case["residual"]:
        s["other"] = ((0.01 if op == "norm_bwd" else 1.0) * _normal(g, N, D)).to(dt)
    if op == "norm_bwd":
        s["dy"] = (0.01 * _normal(g, N, D)).to(dt)
        v = s["x"].double()
        mean = torch.zeros((N,), dtype=torch.float64, device="cuda") if case["rms"] else v.mean(dim=1)
        s["rstd"] = torch.rsqrt((v - mean[:, None]).square().mean(dim=1) + EPS).float()
        s["mean"] = None if case["rms"] else mean.float()
    return s


# ---- one pass --------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from implicit_gemm_conv2d_gb300 import train

    op = s["op"]
    if op == "scan_fwd":
        h, last = train.gated_scan(s["x"], s["gate"], s["h0"], reset=s["reset"], lengths=s["lengths"])
        return {"h": h, "last": last}
    if op == "scan_bwd":
        dx, dgate, dh0 = train.gated_scan_bwd(s["x"], s["gate"], s["h"], s["dh"], s["h0"], dlast=s["dlast"],
                                              reset=s["reset"], lengths=s["lengths"])
        return {"dx": dx, "dgate": dgate, "dh0": dh0}
    if op == "distill_fwd":
        loss, zmax, zlog = train.distill(s["z"], s["ids"], s["teacher"], temperature=s["temperature"])
        return {"loss": loss, "zmax": zmax, "zlog": zlog}
    if op == "distill_bwd":
        return train.distill_bwd(s["z"], s["ids"], s["teacher"], s["zmax"], s["zlog"], s["weight"], scale=s["scale"],
                                 temperature=s["temperature"])
    if op == "distill_grad":
        loss, dz = train.distill_grad(s["z"], s["ids"], s["teacher"], s["weight"], scale=s["scale"],
                                      temperature=s["temperature"])
        return {"loss": loss, "dz": dz}
    if op == "norm_fwd":
        y, total, mean, rstd = train.layer_norm(s["x"], s["gamma"], s["beta"], residual=s["other"], eps=EPS,
                                                rms=s["rms"])
        return {"y": y, "total": total, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = train.layer_norm_bwd(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], dtotal=s["other"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _run_plain(s):
    op = s["op"]
    if op == "scan_fwd":
        return _plain_scan(s)
    if op == "scan_bwd":
        return _plain_scan_bwd(s)
    if op in ("distill_fwd", "distill_bwd", "distill_grad"):
        return _plain_distill(s)
    return _plain_norm(s) if op == "norm_fwd" else _plain_norm_bwd(s)


def _doubling(a, b):
    """v[t] = a[t] v[t-1] + b[t] along dimension 1, v[-1] = 0, in about log2 T steps."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat((b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return b


def _inside(s):
    """(B, T, 1): the steps that a row has."""
    steps = torch.arange(s["x"].shape[1], device="cuda")
    return (steps[None, :] < s["lengths"][:, None])[:, :, None]


def _plain_scan(s):
    x, gate = s["x"].float(), s["gate"].float()
    keep, take = 1.0 / (1.0 + torch.exp(gate)), 1.0 / (1.0 + torch.exp(-gate))
    b = take * x
    if s["reset"] is not None:
        keep = torch.where(s["reset"][:, :, None], torch.zeros_like(keep), keep)
    if s["lengths"] is not None:
        inside = _inside(s)
        keep, b = torch.where(inside, keep, torch.ones_like(keep)), torch.where(inside, b, torch.zeros_like(b))
    if s["h0"] is not None:
        b = torch.cat((b[:, :1] + keep[:, :1] * s["h0"][:, None], b[:, 1:]), 1)
    h = _doubling(keep, b)
    last = h[:, -1].clone()
    if s["lengths"] is not None:
        h = torch.where(inside, h, torch.zeros_like(h))
    return {"h": h.to(s["x"].dtype), "last": last}


def _plain_scan_bwd(s):
    x, gate, h, dh = s["x"].float(), s["gate"].float(), s["h"].float(), s["dh"].float()
    keep, take = 1.0 / (1.0 + torch.exp(gate)), 1.0 / (1.0 + torch.exp(-gate))
    slope = keep * take
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0])
    before = torch.cat((h0[:, None], h[:, :-1]), 1)
    if s["reset"] is not None:
        cut = s["reset"][:, :, None]
        keep, before = torch.where(cut, torch.zeros_like(keep), keep), torch.where(cut, torch.zeros_like(h), before)
    if s["dlast"] is not None:
        ends = s["lengths"] - 1 if s["lengths"] is not None else torch.full((x.shape[0],), x.shape[1] - 1, device="cuda")
        at = torch.arange(x.shape[1], device="cuda")[None, :] == ends[:, None]
        dh = dh + at[:, :, None] * s["dlast"][:, None]
    if s["lengths"] is not None:
        inside = _inside(s)
        dh, keep = torch.where(inside, dh, torch.zeros_like(dh)), torch.where(inside, keep, torch.zeros_like(keep))
    after = torch.cat((keep[:, 1:], torch.zeros_like(keep[:, :1])), 1)
    lam = _doubling(after.flip(1), dh.flip(1)).flip(1)
    dgate = lam * (x - before) * slope
    dt = s["x"].dtype
    return {"dx": (take * lam).to(dt), "dgate": dgate.to(dt),
            "dh0": keep[:, 0] * lam[:, 0] if s["h0"] is not None else None}


def _plain_distill(s):
    op, tau = s["op"], s["temperature"]
    z, ids = s["z"].float(), s["ids"].long()
    if op == "distill_bwd":
        zmax, zlog = s["zmax"], s["zlog"]
    else:
        zmax = z.max(dim=1).values
        zlog = torch.log(torch.exp((z - zmax[:, None]) / tau).sum(dim=1))
    logp = (z - zmax[:, None]) / tau - zlog[:, None]
    named = ids >= 0
    q = torch.where(named, s["teacher"].float() / tau, torch.full_like(s["teacher"], -math.inf, dtype=torch.float32))
    qmax = torch.where(named.any(dim=1), q.max(dim=1).values, torch.zeros_like(zmax))[:, None]
    e = torch.exp(q - qmax)
    total = e.sum(dim=1, keepdim=True)
    some = total > 0
    p = torch.where(some, e / total, torch.zeros_like(e))
    safe = torch.where(named, ids, torch.zeros_like(ids))
    out = {}
    if op != "distill_bwd":
        term = p * (q - qmax - torch.log(total) - torch.gather(logp, 1, safe))
        out["loss"] = tau * tau * torch.where(p > 0, term, torch.zeros_like(term)).sum(dim=1)
    if op == "distill_fwd":
        return {**out, "zmax": zmax, "zlog": zlog}
    c = (tau * s["scale"]) * s["weight"][:, None]
    dz = torch.where(some, torch.exp(logp), torch.zeros_like(logp))
    dz = (c * dz.scatter_add(1, safe, -p)).to(s["z"].dtype)
    return dz if op == "distill_bwd" else {**out, "dz": dz}


def _plain_norm(s):
    x = s["x"].float()
    total = None
    if s["other"] is not None:
        total = (x + s["other"].float()).to(s["x"].dtype)
        x = total.float()
    mean = None if s["rms"] else x.mean(dim=1)
    v = x if s["rms"] else x - mean[:, None]
    rstd = torch.rsqrt(v.square().mean(dim=1) + EPS)
    y = v * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "total": total, "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    dt = s["x"].dtype
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (x if s["rms"] else x - s["mean"][:, None]) * rstd
    e = dy * s["gamma"].float()
    dx = e - xhat * (e * xhat).mean(dim=1, keepdim=True)
    if not s["rms"]:
        dx = dx - e.mean(dim=1, keepdim=True)
    dx = rstd * dx
    if s["other"] is not None:
        dx = dx + s["other"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * xhat).sum(dim=0).to(dt),
            "dbeta": None if s["rms"] else dy.sum(dim=0).to(dt)}


# ---- the work of a pass ----------------------------------------------------------------------
def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "f32" else 2
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D = case["B"], case["T"], case["D"]
        every = B * T * D
        read = sum(_row_lengths(case)) * D if case["lengths"] else every
        flags = (B * T if case["resets"] else 0) + (4 * B if case["lengths"] else 0)
        if op == "scan_fwd":  # x, gate; h; the states
            return {"bytes": (2 * read + every) * es + flags + 4 * B * D * (2 if case["h0"] else 1), "flops": 12 * read}
        # x, gate, h, dh; dx, dgate; the states
        return {"bytes": (4 * read + 2 * every) * es + flags + 4 * B * D * (3 if case["h0"] else 0), "flops": 20 * read}
    if op in ("distill_fwd", "distill_bwd", "distill_grad"):
        N, V, K = case["N"], case["V"], case["K"]
        passes = 1 if op == "distill_fwd" else 2
        return {"bytes": passes * N * V * es + N * K * 8 + 12 * N, "flops": 4 * passes * N * V + 8 * N * K}
    N, D = case["N"], case["D"]
    stats = 4 * N * (1 if case["rms"] else 2)
    params = D * es * (1 if case["rms"] else 2)
    if op == "norm_fwd":  # x, the residual; y, the sum
        return {"bytes": N * D * es * (4 if case["residual"] else 2) + stats + params, "flops": 8 * N * D}
    # x, dy, the sum's gradient; dx; gamma; dgamma, dbeta
    return {"bytes": N * D * es * (4 if case["residual"] else 3) + stats + params + D * es, "flops": 14 * N * D}


# ---- the same in 64 bits ---------------------------------------------------------------------
def exact(case, seed):
    """Step by step in time (the scan), row block by row block from the definitions (the loss, the
    norm), all in fp64."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_fwd":
        return _exact_scan(s)
    if op == "scan_bwd":
        return _exact_scan_bwd(s)
    if op in ("distill_fwd", "distill_bwd", "distill_grad"):
        return _exact_distill(s)
    return _exact_norm(s) if op == "norm_fwd" else _exact_norm_bwd(s)


def _at(s, t):
    """What step t starts anew, and which rows have it: (B, 1) or None."""
    fresh = s["reset"][:, t, None] if s["reset"] is not None else None
    there = s["lengths"][:, None] > t if s["lengths"] is not None else None
    return fresh, there


def _exact_scan(s):
    B, T, D = s["x"].shape
    state = torch.zeros((B, D), dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    h = torch.zeros((B, T, D), dtype=torch.float64, device="cuda")
    for t in range(T):
        fresh, there = _at(s, t)
        z = torch.sigmoid(s["gate"][:, t].double())
        old = state if fresh is None else state.masked_fill(fresh, 0.0)
        new = old + z * (s["x"][:, t].double() - old)
        state = new if there is None else torch.where(there, new, state)
        h[:, t] = new if there is None else new * there
    return {"h": h, "last": state}


def _exact_scan_bwd(s):
    B, T, D = s["x"].shape
    flow = torch.zeros((B, D), dtype=torch.float64, device="cuda") if s["dlast"] is None else s["dlast"].double()
    dx, dgate = (torch.zeros((B, T, D), dtype=torch.float64, device="cuda") for _ in range(2))
    for t in range(T - 1, -1, -1):
        fresh, there = _at(s, t)
        z = torch.sigmoid(s["gate"][:, t].double())
        if t > 0:
            old = s["h"][:, t - 1].double()
        else:
            old = torch.zeros_like(flow) if s["h0"] is None else s["h0"].double()
        lam = flow + s["dh"][:, t].double()
        back = lam - lam * z
        if fresh is not None:
            old, back = old.masked_fill(fresh, 0.0), back.masked_fill(fresh, 0.0)
        grads = lam * z, lam * (s["x"][:, t].double() - old) * (z - z * z)
        if there is not None:
            back, grads = torch.where(there, back, flow), tuple(v * there for v in grads)
        dx[:, t], dgate[:, t] = grads
        flow = back
    return {"dx": dx, "dgate": dgate, "dh0": flow if s["h0"] is not None else None}


def _exact_distill(s):
    op, tau = s["op"], s["temperature"]
    rows = max(1, 50_000_000 // s["V"])
    parts = []
    for a in range(0, s["N"], rows):
        z = s["z"][a:a + rows].double()
        ids = s["ids"][a:a + rows].long()
        padding = ids[:, 0] < 0  # the cases have whole rows of padding
        p = torch.softmax(s["teacher"][a:a + rows].double() / tau, dim=1)
        p[padding] = 0.0
        ids = ids.clamp(min=0)
        top = z.amax(dim=1)
        if op == "distill_bwd":
            top, log = s["zmax"][a:a + rows].double(), s["zlog"][a:a + rows].double()
        else:
            log = torch.logsumexp(z / tau, dim=1) - top / tau
        norm = top / tau + log
        loss = (torch.xlogy(p, p) - p * (z.gather(1, ids) / tau - norm[:, None])).sum(dim=1) * tau ** 2
        if op == "distill_fwd":
            parts.append((loss, top, log))
            continue
        dz = torch.exp(z / tau - norm[:, None])
        dz[padding] = 0.0
        dz.scatter_add_(1, ids, -p)
        dz *= s["weight"][a:a + rows, None].double() * (tau * s["scale"])
        parts.append((loss, dz))
    out = [torch.cat(v) for v in zip(*parts)]
    if op == "distill_fwd":
        return {"loss": out[0], "zmax": out[1], "zlog": out[2]}
    return out[1] if op == "distill_bwd" else {"loss": out[0], "dz": out[1]}


def _exact_norm(s):
    x = s["x"].double()
    total = None
    if s["other"] is not None:
        total = x + s["other"].double()
        x = total.float().to(s["x"].dtype).double()  # what is normalised is the sum as it is kept
    if s["rms"]:
        mean, var = None, torch.linalg.vecdot(x, x) / x.shape[1]
    else:
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        x = x - mean[:, None]
    rstd = (var + EPS) ** -0.5
    y = s["gamma"].double() * (x * rstd[:, None])
    return {"y": y if s["beta"] is None else y + s["beta"].double(), "total": total, "mean": mean, "rstd": rstd}


def _exact_norm_bwd(s):
    x, dy, rstd = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    D = x.shape[1]
    xhat = x * rstd if s["rms"] else (x - s["mean"].double()[:, None]) * rstd
    e = dy * s["gamma"].double()
    dx = e - xhat * (torch.linalg.vecdot(e, xhat) / D)[:, None]
    if not s["rms"]:
        dx -= e.sum(dim=1, keepdim=True) / D
    dx *= rstd
    if s["other"] is not None:
        dx += s["other"].double()
    ones = torch.ones((x.shape[0],), dtype=torch.float64, device="cuda")
    return {"dx": dx, "dgamma": ones @ (dy * xhat), "dbeta": None if s["rms"] else ones @ dy}
