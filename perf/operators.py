"""What the training-step operators are measured on: group norm with an activation (forward
and backward, NCHW and channels last), the embedding lookup and its gradient, and the global
gradient norm with clipping.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a
case's inputs on the GPU, ``run()`` makes one pass through the operator and ``exact()`` computes
the same in 64 bits.  With ``own`` false ``run`` computes the operators' plain form out of
elementary torch operations in fp32; with ``own`` true it calls the framework's kernels."""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
MAX_NORM = 0.6


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # Second encoder layer's output during a rollout: small batch, 8 or 16 values a group.
        dict(name="gn_fwd_rollout_f32", op="gn_fwd", B=256, C=128, P=2, G=8, act="relu", layout="nchw", dtype="f32"),
        # First encoder layer's output (3x4 positions) at the training batch.
        dict(name="gn_fwd_encoder_bf16", op="gn_fwd", B=32768, C=128, P=12, G=16, act="silu", layout="nchw",
             dtype="bf16"),
        # Channels-last feature maps of an image-sized network, 10 channels a group.
        dict(name="gn_fwd_map_nhwc_bf16", op="gn_fwd", B=24, C=320, P=72 * 72, G=32, act="silu", layout="nhwc",
             dtype="bf16"),
        # The encoder layer's backward, fp32 training.
        dict(name="gn_bwd_encoder_f32", op="gn_bwd", B=8192, C=128, P=12, G=16, act="relu", layout="nchw",
             dtype="f32"),
        # Channels-last maps with an odd number of positions, backward.
        dict(name="gn_bwd_map_nhwc_bf16", op="gn_bwd", B=12, C=192, P=95 * 101, G=24, act="gelu", layout="nhwc",
             dtype="bf16"),
        # Attribute table of the encoder (128 rows of 32, 47 attributes a sample) in a rollout.
        dict(name="embed_fwd_rollout_f32", op="embed_fwd", T=16 * 47, V=128, D=32, index="i32", dtype="f32"),
        # The same at the training batch.
        dict(name="embed_fwd_encoder_bf16", op="embed_fwd", T=32768 * 47, V=128, D=32, index="i32", dtype="bf16"),
        # Its gradient: every row of the table is the sum of about ten thousand tokens.
        dict(name="embed_bwd_encoder_f32", op="embed_bwd", T=32768 * 47, V=128, D=32, index="i32", dtype="f32"),
        # A token vocabulary: most rows get no token, a few get very many.
        dict(name="embed_bwd_vocab_bf16", op="embed_bwd", T=16384, V=50021, D=1024, index="i64", dtype="bf16"),
        # The encoder's own parameters: two conv layers with bias and norm, the attribute table.
        dict(name="clip_encoder_f32", op="clip", count=9, total=341_000, shuffle=1, dtype="f32"),
        # A network of hundreds of millions of parameters, sizes over four orders of magnitude.
        dict(name="clip_large_bf16", op="clip", count=48, total=400_000_000, shuffle=2, dtype="bf16"),
        # The norm alone, for logging: many tensors of both types.
        dict(name="norm_many_mixed", op="norm", count=300, total=60_000_000, shuffle=3, dtype="mixed"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "embed_fwd", "embed_bwd", "clip", "norm"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("gn_fwd", "gn_bwd"):
        act = rng.choice(["none", "relu", "silu", "gelu"])
        layout = rng.choice(["nchw", "nhwc"])
        cap = 50_000_000 if op == "gn_fwd" else 25_000_000
        while True:
            G = rng.choice([1, 2, 3, 4, 8, 8, 16, 16, 32, 32])
            C = G * _log(rng, 1, 64)
            P = _log(rng, 1, 300) if rng.random() < 0.6 else _log(rng, 256, 40_000)
            B = _log(rng, 1, 32768)
            # a group of one or two values has nothing to normalise
            if C <= 1280 and C // G * P >= 4 and 20_000 <= B * C * P <= cap:
                return dict(op=op, B=B, C=C, P=P, G=G, act=act, layout=layout, dtype=dtype)
    if op in ("embed_fwd", "embed_bwd"):
        cap = 100_000_000
        while True:
            T, V, D = _log(rng, 100, 1_600_000), _log(rng, 50, 200_000), _log(rng, 8, 4096)
            if rng.random() < 0.7:
                D = (D + 7) // 8 * 8
            if T * D <= cap and V * D <= cap:
                return dict(op=op, T=T, V=V, D=D, index=rng.choice(["i32", "i64"]), dtype=dtype)
    count = _log(rng, 1, 60) if op == "clip" else _log(rng, 1, 400)
    total = max(50 * count, _log(rng, 10_000, 200_000_000))
    return dict(op=op, count=count, total=total, shuffle=rng.randrange(1000),
                dtype=rng.choice(["f32", "bf16", "mixed"]))


def _sizes(case):
    """The list's tensor sizes: a few large ones hold most of the total, many small ones the rest."""
    r = random.Random(case["shuffle"])
    w = [math.exp(r.uniform(0.0, math.log(1e4))) for _ in range(case["count"])]
    s = sum(w)
    n = [max(1, int(case["total"] * v / s)) for v in w]
    dts = [case["dtype"] if case["dtype"] != "mixed" else r.choice(["f32", "bf16"]) for _ in n]
    return n, [DTYPES[d] for d in dts]


# ---- inputs ----------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _per_channel(case, v):
    return v.view(1, -1, 1) if case["layout"] == "nchw" else v.view(1, 1, -1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        dt = DTYPES[case["dtype"]]
        B, C, P = case["B"], case["C"], case["P"]
        shape = (B, C, P) if case["layout"] == "nchw" else (B, P, C)
        # a conv's output: every channel with an offset and a spread of its own
        x = _normal(g, *shape)
        x.mul_(_per_channel(case, 0.5 + _normal(g, C).abs())).add_(_per_channel(case, 0.5 * _normal(g, C)))
        s = dict(case, x=x.to(dt), gamma=(1.0 + 0.2 * _normal(g, C)).to(dt), beta=(0.2 * _normal(g, C)).to(dt))
        if op == "gn_bwd":
            s["dy"] = (0.01 * _normal(g, *shape)).to(dt)
            v = _grouped(s, s["x"].float())
            mean = v.mean(dim=2)
            s["mean"] = mean
            s["rstd"] = torch.rsqrt((v - mean.unsqueeze(2)).square().mean(dim=2) + EPS)
        return s
    if op in ("embed_fwd", "embed_bwd"):
        dt = DTYPES[case["dtype"]]
        T, V, D = case["T"], case["V"], case["D"]
        # a few tokens make up much of a text or of an observation: P(rank k) ~ 1 / k
        u = torch.rand((T,), generator=g, device="cuda", dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        step = next(p for p in (7919, 7907, 7901) if V % p)
        idx = (rank * step + int(torch.randint(V, (1,), generator=g, device="cuda"))) % V
        s = dict(case, idx=idx.to(torch.int32 if case["index"] == "i32" else torch.int64), scale=math.sqrt(D))
        if op == "embed_fwd":
            s["table"] = (0.02 * _normal(g, V, D)).to(dt)
        else:
            s["dy"] = (0.01 * _normal(g, T, D)).to(dt)
        return s
    n, dts = _sizes(case)
    scale = 2.0 / math.sqrt(case["total"])  # a norm of about two: above the limit, so that it is clipped
    grads = [(scale * _normal(g, k)).to(dt) for k, dt in zip(n, dts)]
    s = dict(case, grads=grads)
    if op == "clip":
        s["out"] = [torch.empty_like(t) for t in grads]
    return s


# ---- one pass --------------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from implicit_gemm_conv2d_gb300 import train

    op = s["op"]
    if op == "gn_fwd":
        y, mean, rstd = train.group_norm(s["x"], s["G"], s["gamma"], s["beta"], eps=EPS, act=s["act"],
                                         layout=s["layout"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "gn_bwd":
        dx, dgamma, dbeta = train.group_norm_bwd(s["x"], s["dy"], s["G"], s["gamma"], s["beta"], s["mean"], s["rstd"],
                                                 act=s["act"], layout=s["layout"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "embed_fwd":
        return train.embed(s["idx"], s["table"], scale=s["scale"])
    if op == "embed_bwd":
        return train.embed_bwd(s["idx"], s["dy"], s["V"], scale=s["scale"])
    if op == "clip":
        norm = train.clip_grads(s["grads"], MAX_NORM, out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    return train.grad_norm(s["grads"])


def _grouped(s, t):
    """(B, G, values of the group)"""
    B, C, P, G = s["B"], s["C"], s["P"], s["G"]
    if s["layout"] == "nchw":
        return t.view(B, G, C // G * P)
    return t.view(B, P, G, C // G).transpose(1, 2).reshape(B, G, P * (C // G))


def _spread(s, v):
    """(B, G) -> one value for each element's channel"""
    c = v.repeat_interleave(s["C"] // s["G"], dim=1)
    return c.unsqueeze(2) if s["layout"] == "nchw" else c.unsqueeze(1)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    return torch.ones_like(z)


def _run_plain(s):
    op = s["op"]
    if op == "gn_fwd":
        x = s["x"].float()
        v = _grouped(s, x)
        mean = v.mean(dim=2)
        rstd = torch.rsqrt((v - mean.unsqueeze(2)).square().mean(dim=2) + EPS)
        z = (x - _spread(s, mean)) * _spread(s, rstd)
        z = z * _per_channel(s, s["gamma"].float()) + _per_channel(s, s["beta"].float())
        return {"y": _act(z, s["act"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "gn_bwd":
        dt = s["x"].dtype
        gamma, beta = _per_channel(s, s["gamma"].float()), _per_channel(s, s["beta"].float())
        rstd = _spread(s, s["rstd"])
        xhat = (s["x"].float() - _spread(s, s["mean"])) * rstd
        dz = s["dy"].float()
        if s["act"] != "none":
            dz = dz * _act_slope(xhat * gamma + beta, s["act"])
        dims = (0, 2) if s["layout"] == "nchw" else (0, 1)
        dgamma, dbeta = (dz * xhat).sum(dim=dims), dz.sum(dim=dims)
        dxhat = dz * gamma
        m1 = _spread(s, _grouped(s, dxhat).mean(dim=2))
        m2 = _spread(s, _grouped(s, dxhat * xhat).mean(dim=2))
        dx = rstd * (dxhat - m1 - xhat * m2)
        return {"dx": dx.to(dt), "dgamma": dgamma.to(dt), "dbeta": dbeta.to(dt)}
    if op == "embed_fwd":
        table = s["table"]
        return (table[s["idx"].long()].float() * s["scale"]).to(table.dtype)
    if op == "embed_bwd":
        acc = torch.zeros((s["V"], s["D"]), dtype=torch.float32, device="cuda")
        acc.index_add_(0, s["idx"].long(), s["dy"].float())
        return (acc * s["scale"]).to(s["dy"].dtype)
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    if op == "norm":
        return norm
    coef = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * coef)
    return {"norm": norm, "grads": s["out"]}


# ---- the work of a pass ----------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        es = 4 if case["dtype"] == "f32" else 2
        n = case["B"] * case["C"] * case["P"]
        stats = 8 * case["B"] * case["G"]
        if op == "gn_fwd":
            return {"bytes": 2 * n * es + stats + 2 * case["C"] * es, "flops": 10 * n}
        return {"bytes": 3 * n * es + stats + 4 * case["C"] * es, "flops": 20 * n}
    if op in ("embed_fwd", "embed_bwd"):
        es = 4 if case["dtype"] == "f32" else 2
        idx = case["T"] * (4 if case["index"] == "i32" else 8)
        tokens, rows = case["T"] * case["D"], case["V"] * case["D"]
        if op == "embed_fwd":  # no more of the table than the tokens name
            return {"bytes": idx + es * (tokens + min(tokens, rows)), "flops": tokens}
        return {"bytes": idx + es * (tokens + rows), "flops": tokens}
    n, dts = _sizes(case)
    size = sum(k * (4 if d == torch.float32 else 2) for k, d in zip(n, dts))
    total = sum(n)
    return {"bytes": size * (2 if op == "clip" else 1) + 4, "flops": total * (3 if op == "clip" else 2)}


# ---- the same in 64 bits ---------------------------------------------------------------------
def exact(case, seed):
    """Sample by sample (group norm), by one-hot products in blocks of rows (the embedding's
    gradient) and tensor by tensor, all in fp64 from the definitions."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        return _exact_gn(s)
    if op == "embed_fwd":
        return torch.index_select(s["table"].double(), 0, s["idx"].long()).mul_(s["scale"])
    if op == "embed_bwd":
        order = torch.argsort(s["idx"].long(), stable=True)
        rows, count = torch.unique_consecutive(s["idx"].long()[order], return_counts=True)
        out = torch.zeros((s["V"], s["D"]), dtype=torch.float64, device="cuda")
        ends = torch.cumsum(count, 0)
        cols = max(1, 200_000_000 // s["T"])  # running sums of a block of columns, differenced at the rows' ends
        for c in range(0, s["D"], cols):
            run_sum = torch.cumsum(s["dy"][:, c:c + cols].double()[order], 0)[ends - 1]
            out[rows, c:c + cols] = torch.diff(run_sum, dim=0, prepend=torch.zeros_like(run_sum[:1])) * s["scale"]
        return out
    total = math.fsum(float(torch.dot(t.double(), t.double())) for t in s["grads"])
    norm = torch.tensor(math.sqrt(total), dtype=torch.float64)
    if op == "norm":
        return norm
    coef = min(1.0, MAX_NORM / (float(norm) + 1e-6))
    return {"norm": norm, "grads": [t.double() * coef for t in s["grads"]]}


def _exact_gn(s):
    B, C, P, G = s["B"], s["C"], s["P"], s["G"]
    K = C // G
    gamma, beta = s["gamma"].double().view(1, G, K, 1), s["beta"].double().view(1, G, K, 1)

    def four(t):  # (b, G, K, P)
        t = t.double()
        return t.view(-1, G, K, P) if s["layout"] == "nchw" else t.view(-1, P, G, K).permute(0, 2, 3, 1)

    def back(t):
        return t.reshape(-1, C, P) if s["layout"] == "nchw" else t.permute(0, 3, 1, 2).reshape(-1, P, C)

    step = max(1, 40_000_000 // (C * P))
    parts, dgamma, dbeta = [], 0.0, 0.0
    for b in range(0, B, step):
        x = four(s["x"][b:b + step])
        if s["op"] == "gn_fwd":
            var, mean = torch.var_mean(x, dim=(2, 3), keepdim=True, unbiased=False)
            rstd = 1.0 / torch.sqrt(var + EPS)
        else:
            mean = s["mean"][b:b + step].double().view(-1, G, 1, 1)
            rstd = s["rstd"][b:b + step].double().view(-1, G, 1, 1)
        xhat = (x - mean) * rstd
        z = xhat * gamma + beta
        if s["op"] == "gn_fwd":
            parts.append((back(_exact_act(z, s["act"])), mean.view(-1, G), rstd.view(-1, G)))
            continue
        dz = four(s["dy"][b:b + step]) * _exact_slope(z, s["act"])
        dgamma = dgamma + (dz * xhat).sum(dim=(0, 3)).view(C)
        dbeta = dbeta + dz.sum(dim=(0, 3)).view(C)
        e = dz * gamma
        dx = (e - e.mean(dim=(2, 3), keepdim=True) - xhat * (e * xhat).mean(dim=(2, 3), keepdim=True)) * rstd
        parts.append((back(dx),))
    out = [torch.cat(p) for p in zip(*parts)]
    if s["op"] == "gn_fwd":
        return {"y": out[0], "mean": out[1], "rstd": out[2]}
    return {"dx": out[0], "dgamma": dgamma, "dbeta": dbeta}


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z


def _exact_slope(z, act):
    if act == "relu":
        return (z > 0.0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1.0 - p)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(z)
