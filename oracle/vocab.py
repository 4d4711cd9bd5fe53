"""64-bit forms of the operators over rows of vocabulary logits: log
probabilities with entropy and top alternatives, their way back, and
distillation from a teacher's lists."""
from __future__ import annotations

import numpy as np


def log_softmax(x, tau=1.0):
    """ln p of each logit.  A row of nothing but -inf has p = 0 throughout; one
    with a NaN or +inf is NaN."""
    z = np.asarray(x, dtype=np.float64) / tau
    out = np.full(z.shape, np.nan)
    for t, row in enumerate(z):
        top = row.max()
        if top == -np.inf:
            out[t] = -np.inf
        elif np.isfinite(top):
            out[t] = row - top - np.log(np.exp(row - top).sum())
    return out


def logsumexp(x, tau=1.0):
    z = np.asarray(x, dtype=np.float64) / tau
    out = np.full(len(z), np.nan)
    for t, row in enumerate(z):
        top = row.max()
        if top == -np.inf:
            out[t] = -np.inf
        elif np.isfinite(top):
            out[t] = top + np.log(np.exp(row - top).sum())
    return out


def ranked(x, k):
    """Indices of the k largest of each row, best first: a NaN before every
    number, -0 as 0, equal ones by index."""
    x = np.asarray(x, dtype=np.float64)
    order = [sorted(range(x.shape[1]), key=lambda v: (not np.isnan(row[v]), -row[v] if row[v] == row[v] else 0, v))
             for row in x]
    return np.array([o[:k] for o in order], dtype=np.int64).reshape(len(x), k)


def token_logprobs(x, tokens=None, keep=None, tau=1.0, k=0):
    T, V = x.shape
    kept = np.ones(T, bool) if keep is None else keep != 0
    lp = log_softmax(x, tau)
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        terms = np.where(p == 0, 0.0, p * lp)
    out = {"lse": np.where(kept, logsumexp(x, tau), 0.0), "entropy": np.where(kept, 0.0 - terms.sum(axis=1), 0.0)}
    if tokens is not None:
        inside = kept & (tokens >= 0) & (tokens < V)
        y = np.where(inside, tokens, 0)
        out["logprob"] = np.where(inside, lp[np.arange(T), y], 0.0)
    if k:
        at = ranked(x, k)
        out["top_index"] = np.where(kept[:, None], at, -1)
        out["top_logprob"] = np.where(kept[:, None], np.take_along_axis(lp, at, axis=1), 0.0)
    return out


def token_logprobs_bwd(x, lse, tokens=None, dlogprob=None, entropy=None, dentropy=None, keep=None, tau=1.0):
    """The gradient of the logits, for lse and entropy as they are given."""
    T, V = x.shape
    g = np.zeros(T) if dlogprob is None else np.asarray(dlogprob, np.float64).copy()
    y = np.full(T, -1) if tokens is None else tokens
    inside = (y >= 0) & (y < V)
    g[~inside] = 0
    h = np.zeros(T) if dentropy is None else np.asarray(dentropy, np.float64)
    H = np.zeros(T) if entropy is None else np.asarray(entropy, np.float64)
    lse = np.asarray(lse, np.float64)
    zero = ((g == 0) & (h == 0)) | (lse == -np.inf)
    if keep is not None:
        zero |= keep == 0
    with np.errstate(invalid="ignore"):
        lp = np.asarray(x, np.float64) / tau - lse[:, None]
        p = np.exp(lp)
        d = -g[:, None] * p - h[:, None] * np.where(p == 0, 0.0, p * (lp + H[:, None]))
    rows = np.nonzero(inside)[0]
    d[rows, y[rows]] += g[rows]
    d[zero] = 0
    return d / tau


def policy_gradient(x, tokens=None, g=None, h=None, tau=1.0):
    """The gradient of sum_t g_t ln p[token_t] + h_t H_t from the logits alone,
    finite ones of any size among them."""
    T, V = x.shape
    lp = log_softmax(x, tau)
    p = np.exp(lp)
    known = np.where(p == 0, 0.0, lp)
    H = -np.where(p == 0, 0.0, p * known).sum(axis=1)
    d = np.zeros((T, V))
    for t in range(T):
        gt = 0.0 if g is None or not 0 <= tokens[t] < V else float(g[t])
        ht = 0.0 if h is None else float(h[t])
        if (gt == 0 and ht == 0) or (lp[t] == -np.inf).all():
            continue
        d[t] = -gt * p[t] - ht * p[t] * (known[t] + H[t])
        if gt:
            d[t, tokens[t]] += gt
    return d / tau


def distill(x, top_index, top_logit, keep=None, tau=1.0, grad_scale=1.0):
    T, V = x.shape
    lp = log_softmax(x, tau)
    out = {"token_loss": np.zeros(T), "dlogits": np.zeros((T, V)), "counted": np.zeros(T, bool)}
    for t in range(T):
        inside = (top_index[t] >= 0) & (top_index[t] < V)
        length = len(inside) if inside.all() else int(np.argmin(inside))
        if length == 0 or (keep is not None and keep[t] == 0):
            continue
        out["counted"][t] = True
        at = top_index[t, :length]
        logq = log_softmax(np.asarray(top_logit[t:t + 1, :length], np.float64), tau)[0]
        q = np.exp(logq)
        with np.errstate(invalid="ignore"):
            out["token_loss"][t] = tau**2 * np.where(q == 0, 0.0, q * (logq - lp[t, at])).sum()
        d = np.exp(lp[t]) * (0.0 if (logq == -np.inf).all() else 1.0)
        np.subtract.at(d, at, q)
        out["dlogits"][t] = tau * d
    n = int(out["counted"].sum())
    out["n"] = n
    out["loss"] = out["token_loss"].sum() / max(n, 1)
    out["dlogits"] *= grad_scale / max(n, 1)
    return out
