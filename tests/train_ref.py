"""fp64 references of the training-step operators (numpy), from their definitions, and the sums
of |term| that the tests' normalised errors divide by (as oracle's ``den``)."""
import math

import numpy as np
from scipy.special import erf

SLOPE_MOST = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + erf(z / math.sqrt(2.0)))
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        p = 1.0 / (1.0 + np.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if kind == "gelu":
        return 0.5 * (1.0 + erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def to_bcp(a, layout):
    return a if layout == "nchw" else np.swapaxes(a, 1, 2)


def gn_stats(x, G, eps, layout):
    v = to_bcp(x.astype(np.float64), layout)
    B, C, P = v.shape
    v = v.reshape(B, G, -1)
    mean = v.mean(axis=2)
    var = ((v - mean[:, :, None]) ** 2).mean(axis=2)
    return mean, 1.0 / np.sqrt(var + eps)


def gn_fwd(x, gamma, beta, G, eps, kind, layout):
    """y and its den, mean, rstd; x (B, C, P) or (B, P, C)."""
    v = to_bcp(x.astype(np.float64), layout)
    B, C, P = v.shape
    K = C // G
    mean, rstd = gn_stats(x, G, eps, layout)
    m, r = (np.repeat(t, K, axis=1)[:, :, None] for t in (mean, rstd))
    ga = np.ones(C) if gamma is None else gamma.astype(np.float64)
    be = np.zeros(C) if beta is None else beta.astype(np.float64)
    z = (v - m) * r * ga[None, :, None] + be[None, :, None]
    amax = np.repeat(np.abs(v.reshape(B, G, -1)).max(axis=2), K, axis=1)[:, :, None]
    den = (np.abs(v) + amax) * r * np.abs(ga)[None, :, None] + np.abs(be)[None, :, None]
    return to_bcp(act(z, kind), layout), to_bcp(den, layout), mean, rstd


def gn_bwd(x, dy, gamma, beta, mean, rstd, G, kind, layout, mask=None):
    """dx, dgamma, dbeta, each with its den.  mean, rstd: (B, G).  mask: the ReLU's, where given."""
    v, d = to_bcp(x.astype(np.float64), layout), to_bcp(dy.astype(np.float64), layout)
    B, C, P = v.shape
    K, M = C // G, C // G * P
    m, r = (np.repeat(np.asarray(t, np.float64), K, axis=1)[:, :, None] for t in (mean, rstd))
    ga = (np.ones(C) if gamma is None else gamma.astype(np.float64))[None, :, None]
    be = (np.zeros(C) if beta is None else beta.astype(np.float64))[None, :, None]
    xh = (v - m) * r
    s = slope(xh * ga + be, kind) if mask is None else to_bcp(mask, layout).astype(np.float64)
    dz = d * s
    # the terms as magnitudes; the slope moves by at most its own size plus that of z's error
    xh_abs = (np.abs(v) + np.abs(m)) * r
    dz_abs = np.abs(d) * SLOPE_MOST[kind]

    def group_mean(t):
        return np.repeat(t.reshape(B, G, -1).sum(axis=2) / M, K, axis=1)[:, :, None]

    e, e_abs = dz * ga, dz_abs * np.abs(ga)
    dx = r * (e - group_mean(e) - xh * group_mean(e * xh))
    dx_den = r * (e_abs * (1 + xh_abs) + group_mean(e_abs * (1 + xh_abs)) + xh_abs * group_mean(e_abs * (1 + xh_abs)))
    out = [(to_bcp(dx, layout), to_bcp(dx_den, layout))]
    out.append(((dz * xh).sum(axis=(0, 2)), (dz_abs * (xh_abs + 1)).sum(axis=(0, 2))))
    out.append((dz.sum(axis=(0, 2)), (dz_abs * (1 + xh_abs)).sum(axis=(0, 2))))
    return out


def embed_fwd(idx, table, scale, padding):
    V, D = table.shape
    ok = (idx >= 0) & (idx < V) & (idx != padding)
    out = np.zeros(idx.shape + (D,))
    out[ok] = table.astype(np.float64)[idx[ok]] * scale
    return out


def embed_bwd(idx, dy, V, scale, padding):
    """dtable and the sums of |term|."""
    D = dy.shape[-1]
    idx, dy = idx.reshape(-1), dy.reshape(-1, D).astype(np.float64)
    ok = (idx >= 0) & (idx < V) & (idx != padding)
    out, den = np.zeros((V, D)), np.zeros((V, D))
    np.add.at(out, idx[ok], dy[ok] * scale)
    np.add.at(den, idx[ok], np.abs(dy[ok] * scale))
    return out, den


def grad_norm(grads):
    return math.sqrt(math.fsum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
