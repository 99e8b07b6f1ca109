"""Float64 layer norm, sliding-window attention with visible first tokens and
distillation from a teacher's top logits: each formula written out plainly,
with the derivatives of the same formulas. Used by tests only; shares no code
with the GPU library.
"""

import numpy as np


# --- layer norm ------------------------------------------------------------

def layer_norm_fwd(x, w, b, eps):
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def layer_norm_bwd(x, w, dy, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(axis=1)[:, None] - xh * (g * xh).mean(axis=1)[:, None])
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# --- attention -------------------------------------------------------------

def visible(n_queries, n_keys, window, sinks):
    """[queries, keys] truth values: queries stand at the end of the keys."""
    pos = np.arange(n_queries)[:, None] + (n_keys - n_queries)
    j = np.arange(n_keys)[None, :]
    return (j <= pos) & ((j > pos - window) | (j < sinks))


def attention(q, k, v, window, sinks, scale):
    """One head of one sequence: q [n, D], k and v [m, D] -> (o, lse, p); a query that sees nothing has
    o = 0, lse = -inf, p = 0."""
    see = visible(q.shape[0], k.shape[0], window, sinks)
    s = np.where(see, scale * (q @ k.T), -np.inf)
    top = np.max(s, axis=1, initial=-np.inf)
    some = np.isfinite(top)
    e = np.where(see, np.exp(s - np.where(some, top, 0.0)[:, None]), 0.0)
    total = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(some, top + np.log(total), -np.inf)
    p = e / np.where(some, total, 1.0)[:, None]
    return p @ v, lse, p


def attention_bwd(q, k, v, p, delta, d_o, scale):
    """(dq, dk, dv) of one head from its probabilities and delta = sum over d of d_o o."""
    ds = p * (d_o @ v.T - delta[:, None])
    return scale * (ds @ k), scale * (ds.T @ q), p.T @ d_o


# --- distillation ----------------------------------------------------------

def topk_distill(z, val, idx, tau, t_lse=None, weight=None):
    """(loss [M], lse [M], dz [M, V]) of logits z [M, V] against entries val, idx [M, K]."""
    M, V = z.shape
    loss, lse, dz = np.zeros(M), np.zeros(M), np.zeros((M, V))
    for m in range(M):
        zz = z[m] / tau
        lse[m] = zz.max() + np.log(np.exp(zz - zz.max()).sum())
        has = (idx[m] >= 0) & (idx[m] < V) & ~np.isneginf(val[m])
        if not has.any():
            continue
        t, at = val[m][has] / tau, idx[m][has]
        log_p = t - (t.max() + np.log(np.exp(t - t.max()).sum()) if t_lse is None else t_lse[m])
        p = np.exp(log_p)
        loss[m] = tau * tau * (p * (log_p - zz[at] + lse[m])).sum()
        w = 1.0 if weight is None else weight[m]
        if w == 0.0:
            continue
        g = p.sum() * np.exp(zz - lse[m])
        np.subtract.at(g, at, p)
        dz[m] = w * tau * g
    return loss, lse, dz
