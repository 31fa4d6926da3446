"""fp64 oracle of the row operators (layer norm, token log probabilities, distillation), written from
their definitions in include/mhc.h. Inputs are plain float arrays (already widened from the tested
type); nothing here is shared with the library.
"""

import numpy as np


def layer_norm(x, gamma=None, beta=None, eps=1e-6):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def layer_norm_backward(d_y, x, gamma, mean, rstd):
    """From the statistics given (those of the forward pass)."""
    x, d_y = np.asarray(x, np.float64), np.asarray(d_y, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * r
    q = d_y if gamma is None else d_y * np.asarray(gamma, np.float64)
    d_x = r * (q - q.mean(1, keepdims=True) - xh * (q * xh).mean(1, keepdims=True))
    return d_x, (d_y * xh).sum(0), d_y.sum(0)


def _log_softmax(z, temperature):
    """(ln p, m, s); rows without a finite logit give ln p = -inf and s = 0, rows with a NaN or a
    +inf give NaN."""
    z = np.asarray(z, np.float64)
    m = z.max(1)
    dead = np.isnan(z).any(1) | (m == np.inf)
    base = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = (z - base[:, None]) / temperature
        s = np.exp(d).sum(1)
        lp = np.where(s[:, None] > 0, d - np.log(s)[:, None], -np.inf)
    lp[dead], s[dead], m[dead] = np.nan, np.nan, np.nan
    return lp, m, s


def _p(lp):
    with np.errstate(invalid="ignore"):
        return np.exp(lp)


def token_logprobs(z, targets=None, temperature=1.0, top=0):
    """dict of logprob, entropy, top_index, top_logprob, m, s."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    lp, m, s = _log_softmax(z, temperature)
    p = _p(lp)
    with np.errstate(invalid="ignore"):
        entropy = -np.where(p > 0, p * lp, 0.0).sum(1)
    entropy[np.isnan(s)] = np.nan
    out = dict(entropy=entropy, m=m, s=s, lp=lp)
    if targets is not None:
        y = np.asarray(targets)
        v = lp[np.arange(T), np.clip(y, 0, V - 1)]
        out["logprob"] = np.where(y < 0, 0.0, np.where(y >= V, np.nan, v))
    if top:
        order = np.argsort(-z, axis=1, kind="stable")[:, :top]
        top_lp = np.take_along_axis(lp, order, 1)
        order[np.isnan(s)] = -1
        out["top_index"], out["top_logprob"] = order, top_lp
    return out


def token_logprobs_backward(z, targets, temperature, d_logprob=None, d_entropy=None):
    z = np.asarray(z, np.float64)
    T, V = z.shape
    lp, _, s = _log_softmax(z, temperature)
    p = _p(lp)
    g = np.zeros(T) if d_logprob is None else np.asarray(d_logprob, np.float64).copy()
    h = np.zeros(T) if d_entropy is None else np.asarray(d_entropy, np.float64)
    d = np.zeros((T, V))
    if d_logprob is not None:
        y = np.asarray(targets)
        g[y < 0] = 0.0
        g[(y >= V) & (g != 0)] = np.nan
        rows = np.nonzero((y >= 0) & (y < V))[0]
        d[rows, y[rows]] = g[rows]
    d -= g[:, None] * p
    with np.errstate(invalid="ignore"):
        entropy = -np.where(p > 0, p * lp, 0.0).sum(1, keepdims=True)
        d -= h[:, None] * np.where(p > 0, p * (lp + entropy), 0.0)
    d[np.isnan(s)] = np.nan
    d[(s == 0) | ((g == 0) & (h == 0))] = 0.0
    return d / temperature


def distill_topk(z, index, teacher, temperature=1.0):
    """(loss, weights)."""
    index, t = np.asarray(index), np.asarray(teacher, np.float64).copy()
    V = np.shape(z)[1]
    lp, _, _ = _log_softmax(z, temperature)
    t[index < 0] = -np.inf
    bad = (index >= V).any(1)
    top = t.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.where(top == -np.inf, 0.0, np.exp((t - np.where(top == -np.inf, 0, top)) / temperature))
        tot = e.sum(1, keepdims=True)
        w = np.where(tot == 0, 0.0, e / tot)
        w[bad] = np.where(index[bad] < 0, 0.0, np.nan)
        lpk = np.take_along_axis(lp, np.clip(index, 0, V - 1), 1)
        loss = np.where(w != 0, w * (np.log(w) - lpk), 0.0).sum(1)
    return loss, w


def distill_topk_backward(z, index, weights, d_loss, temperature=1.0):
    lp, _, s = _log_softmax(z, temperature)
    p = _p(lp)
    w, index = np.asarray(weights, np.float64), np.asarray(index)
    g = np.asarray(d_loss, np.float64)
    d = p.copy()
    for t in range(d.shape[0]):
        for k in range(index.shape[1]):
            if 0 <= index[t, k] < d.shape[1] and w[t, k] != 0:
                d[t, index[t, k]] -= w[t, k]
    d[np.isnan(w).any(1)] = np.nan
    d = d * g[:, None] / temperature
    d[(s == 0) | (g == 0) | (w == 0).all(1)] = 0.0
    return d
