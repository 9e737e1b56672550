"""fp64 references of the sequence operators (numpy), from their definitions, and bounds of the error
that fp32 arithmetic in any order of the products may leave (the tests' tolerances)."""
import numpy as np

U = 2.0 ** -24                                   # half a step of fp32
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # of a result as it is kept


def sigmoid(g):
    return 0.5 * (1.0 + np.tanh(0.5 * g))


def _steps(x, lengths):
    B, T, _ = x.shape
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    return np.arange(T)[None, :] < n[:, None]


def scan_fwd(x, gate, h0=None, reset=None, lengths=None):
    """h, last, and a bound of each one's error.

    A step rounds x - h (U), its product with z, whose own error is that of exp and of the quotient
    ((4 + 1.5 |gate|) U relative), and the sum (U of it); what a step leaves decays with the state, by
    1 - z a step.  Joining stretches rounds as often again, so all of it counts twice."""
    B, T, D = x.shape
    inside = _steps(x, lengths)
    s = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    e = np.zeros((B, D))
    h, eh = np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T):
        z = sigmoid(gate[:, t])
        there = inside[:, t][:, None]
        if reset is not None:
            fresh = (reset[:, t] != 0)[:, None] & there
            s, e = np.where(fresh, 0.0, s), np.where(fresh, 0.0, e)
        new = s + z * (x[:, t] - s)
        err = (1 - z) * e + 2 * U * (z * (6 + 1.5 * np.abs(gate[:, t])) * (np.abs(x[:, t]) + np.abs(s)) + np.abs(s)
                                     + np.abs(new))
        s, e = np.where(there, new, s), np.where(there, err, e)
        h[:, t], eh[:, t] = np.where(there, s, 0.0), np.where(there, e, 0.0)
    return h, s, eh, e


def scan_bwd(x, gate, h, dh, h0=None, dlast=None, reset=None, lengths=None):
    """(dx, bound), (dgate, bound), (dh0, bound)."""
    B, T, D = x.shape
    inside = _steps(x, lengths)
    flow = np.zeros((B, D)) if dlast is None else dlast.astype(np.float64)
    e = np.zeros((B, D))
    dx, dg, ex, eg = (np.zeros((B, T, D)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        z = sigmoid(gate[:, t])
        there = inside[:, t][:, None]
        old = h[:, t - 1] if t > 0 else (np.zeros((B, D)) if h0 is None else h0)
        fresh = np.zeros((B, 1), bool) if reset is None else (reset[:, t] != 0)[:, None]
        old = np.where(fresh, 0.0, old)
        lam = dh[:, t] + flow
        el = e + 2 * U * (np.abs(dh[:, t]) + np.abs(flow))
        rel = (8 + 3 * np.abs(gate[:, t])) * U   # of z and of z (1 - z)
        dx[:, t] = np.where(there, z * lam, 0.0)
        ex[:, t] = np.where(there, z * (el + rel * np.abs(lam)), 0.0)
        slope, d = z * (1 - z), x[:, t] - old
        dg[:, t] = np.where(there, lam * d * slope, 0.0)
        eg[:, t] = np.where(there, slope * (el * np.abs(d) + np.abs(lam) * (rel + 4 * U) * (np.abs(x[:, t]) + np.abs(old))),
                            0.0)
        back = np.where(fresh, 0.0, lam - z * lam)
        eb = np.where(fresh, 0.0, (1 - z) * el + 2 * U * (2 + z * (8 + 3 * np.abs(gate[:, t]))) * np.abs(lam))
        flow, e = np.where(there, back, flow), np.where(there, eb, e)
    return (dx, ex), (dg, eg), (flow, e)


def teacher_probabilities(ids, teacher, V, tau):
    """p (0 where the entry counts for nothing), log p, and which rows have entries that count."""
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where((ids >= 0) & (ids < V), teacher, -np.inf) / tau
        some = (q > -np.inf).any(axis=1)
        x = q - np.where(some, q.max(axis=1, initial=-np.inf), 0.0)[:, None]
        e = np.where(some[:, None], np.exp(x), 0.0)
        s = np.where(some, e.sum(axis=1), 1.0)[:, None]
        return e / s, x - np.log(s), some, np.where(e > 0, np.abs(x), 0.0)


def distill_fwd(z, ids, teacher, tau):
    """(loss, bound), zmax, (zlog, bound).

    exp's argument (z - m) / tau is off by 3 U of itself and 2^x by 4 U; x exp(-x) is below 1, so the terms
    leave 8 U of the sum, and its additions (64 + V / 512) U: a tree over chains of a few hundred
    vectors.  log p and log P are off by 4 U of their terms."""
    N, V = z.shape
    K = ids.shape[1]
    m = z.max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        log = np.log(np.exp((z - m[:, None]) / tau).sum(axis=1))
        blog = (72 + V / 512) * U + 2 * U * np.abs(log)
        p, logp, some, x = teacher_probabilities(ids, teacher, V, tau)
        zk = (np.take_along_axis(z, np.clip(ids, 0, V - 1), 1) - m[:, None]) / tau
        logs = zk - log[:, None]
        term = np.where(p > 0, p * (logp - logs), 0.0)
        rel = (x + K / 16 + 16) * U
        err = np.where(p > 0, rel * np.abs(term) + p * (rel + 4 * U * (np.abs(zk) + np.abs(logp) + 1) + blog[:, None]), 0.0)
        return (tau * tau * term.sum(axis=1), tau * tau * (err.sum(axis=1) + (K / 16 + 16) * U * np.abs(term).sum(axis=1))), \
            m, (log, blog)


def distill_bwd(z, ids, teacher, m, log, weight, scale, tau, blog=0.0):
    """dz and its bound; blog: of log's own error."""
    N, V = z.shape
    p, _, some, x = teacher_probabilities(ids, teacher, V, tau)
    w = np.ones(N) if weight is None else weight
    c = (scale * tau * w * some)[:, None]
    a = (z - m[:, None]) / tau
    P = np.exp(a - log[:, None])
    relP = np.where(P > 0, 3 * U * np.abs(a), 0.0) + (3 * np.abs(log)[:, None] + 10) * U + np.reshape(blog, (-1, 1))
    t, bt = np.zeros((N, V)), np.zeros((N, V))
    for k in range(ids.shape[1]):
        rows = np.flatnonzero((ids[:, k] >= 0) & (ids[:, k] < V))
        np.add.at(t, (rows, ids[rows, k]), p[rows, k])
        np.add.at(bt, (rows, ids[rows, k]), p[rows, k] * (x[rows, k] + ids.shape[1] / 8 + 20) * U)
    dz = np.where(c != 0, c * (P - t), 0.0)
    return dz, np.where(c != 0, np.abs(c) * (P * relP + bt + 1.2e-38) + 4 * U * np.abs(dz), 0.0)


def ln_stats(x, eps, rms):
    mean = np.zeros(x.shape[0]) if rms else x.mean(axis=1)
    return mean, 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)


def ln_fwd(x, gamma, beta, eps, rms):
    """(y, bound), (mean, bound), (rstd, bound) of x, the sum as it is kept.

    A row's sums are trees over chains of at most 64 + D / 1024 values: n U of the sum of magnitudes.  The mean's
    error is common to the row's deviations, and adds its square to their mean square."""
    D = x.shape[1]
    n = (72 + D / 512) * U
    mean, rstd = ln_stats(x, eps, rms)
    em = np.zeros_like(mean) if rms else (n + 2 * U) * np.abs(x).mean(axis=1) + U * np.abs(mean)
    d = x - mean[:, None]
    ed = em[:, None] + U * (np.abs(x) + np.abs(mean)[:, None])
    var = (d * d).mean(axis=1)
    ev = (2 * np.abs(d) * ed + ed * ed).mean(axis=1) + n * var
    er = rstd * (0.51 * ev * rstd * rstd + 3 * U)
    xh = d * rstd[:, None]
    exh = ed * rstd[:, None] + np.abs(d) * er[:, None] + 2 * U * np.abs(xh)
    ga = np.ones(D) if gamma is None else gamma
    be = np.zeros(D) if beta is None else beta
    y = xh * ga + be
    return (y, exh * np.abs(ga) + U * (np.abs(xh * ga) + np.abs(y))), (mean, em), (rstd, er)


def ln_bwd(x, dy, gamma, mean, rstd, dtotal, rms):
    """(dx, bound), (dgamma, bound), (dbeta, bound), from the statistics as they are kept."""
    N, D = x.shape
    n = (72 + D / 512) * U
    m, r = np.zeros((N, 1)) if rms else mean[:, None], rstd[:, None]
    ga = np.ones(D) if gamma is None else gamma
    xh = (x - m) * r
    exh = (np.abs(x) + np.abs(m)) * r * 3 * U
    e = dy * ga
    ee = U * np.abs(e)
    m1 = np.zeros((N, 1)) if rms else e.mean(axis=1, keepdims=True)
    em1 = np.zeros((N, 1)) if rms else (n + 2 * U) * np.abs(e).mean(axis=1, keepdims=True)
    m2 = (e * xh).mean(axis=1, keepdims=True)
    em2 = (np.abs(e) * exh + (n + 4 * U) * np.abs(e * xh)).mean(axis=1, keepdims=True)
    inner = e - m1 - xh * m2
    t = np.zeros_like(x) if dtotal is None else dtotal
    dx = r * inner + t
    edx = r * (ee + em1 + np.abs(xh) * em2 + exh * np.abs(m2) + 3 * U * (np.abs(e) + np.abs(m1) + np.abs(xh * m2))) \
        + 2 * U * (np.abs(r * inner) + np.abs(dx))
    # the rows' sums: chains of 256, of their sums, and of the blocks'
    c = (256 + 64 + N / 65536 + 40) * U
    dg, db = (dy * xh).sum(axis=0), dy.sum(axis=0)
    return (dx, edx), (dg, (np.abs(dy) * exh).sum(axis=0) + c * np.abs(dy * xh).sum(axis=0)), \
        (db, c * np.abs(dy).sum(axis=0))
