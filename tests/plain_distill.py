"""The distillation loss and its gradient from the definition, in 64 bits, row by
row (numpy)."""
import numpy as np


def _logsumexp(x):
    if x.size == 0 or np.isneginf(x).all():
        return -np.inf
    m = x.max()
    return m + np.log(np.exp(x - m).sum())


def row(z, idx, t, tau=1.0, lse=None, g=1.0):
    """(loss, dz) of one row."""
    z = np.asarray(z, np.float64) / tau
    v = z.size
    idx, t = np.asarray(idx), np.asarray(t, np.float64) / tau
    keep = (idx >= 0) & (idx < v)
    idx, t = idx[keep], t[keep]
    if idx.size == 0:
        return 0.0, np.zeros(v)
    bad = np.isnan(z).any() or np.isposinf(z).any()
    if bad:
        return np.nan, np.zeros(v) if g == 0 else np.full(v, np.nan)
    la = _logsumexp(z)
    log_q = np.full(v, -np.inf) if np.isneginf(la) else z - la
    lt = _logsumexp(t) if lse is None else float(lse)
    log_p = t - lt if np.isfinite(lt) else np.full(t.shape, -np.inf)
    p = np.exp(log_p)
    loss = float(sum(a * (b - c) for a, b, c in zip(p, log_p, log_q[idx]) if a != 0))
    d = np.exp(log_q)
    d[idx] -= p
    if lse is not None:
        rest = np.ones(v, bool)
        rest[idx] = False
        lr = _logsumexp(z[rest])
        left = max(0.0, 1.0 - p.sum())
        if not np.isneginf(lr):
            if left > 0:
                loss += left * (np.log(left) - (lr - la))
            d[rest] -= left * np.exp(z[rest] - lr)
    return loss, np.zeros(v) if g == 0 else d * g / tau


def rows(z, idx, t, tau=1.0, lse=None, g=None):
    n = len(z)
    out = [row(z[i], idx[i], t[i], tau, None if lse is None else lse[i], 1.0 if g is None else float(g[i])) for i in range(n)]
    return np.array([o[0] for o in out]), np.stack([o[1] for o in out]) if n else np.zeros((0, z.shape[1]))
