"""The router's definitions in numpy float64, written from the formulas in include/tmoe.h."""
import numpy as np


def masked(l, mask):
    l = np.array(l, np.float64)
    if mask is not None:
        l[~mask] = -np.inf
    return l


def softmax_rows(l):
    """Softmax of rows whose -inf entries are not available; zeros for a row of -inf."""
    m = l.max(1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    ex = np.exp(l - m)
    s = ex.sum(1, keepdims=True)
    lse = np.where(s > 0, m + np.log(np.where(s > 0, s, 1.0)), -np.inf)[:, 0]
    return ex / np.where(s > 0, s, 1.0), lse


def topk(l, k, renormalize, mask=None):
    l = masked(l, mask)
    p, lse = softmax_rows(l)
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    there = np.take_along_axis(l, order, 1) > -np.inf
    w = np.where(there, np.take_along_axis(p, order, 1), 0.0)
    if renormalize:
        t = w.sum(1, keepdims=True)
        w = w / np.where(t > 0, t, 1.0)
    return np.where(there, order, -1), w, lse


def topk_loss(l, ids, dw, renormalize):
    """sum w * dw with the selection held fixed, as a function of the logits (for differences)."""
    p, _ = softmax_rows(l)
    w = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
    if renormalize:
        t = w.sum(1, keepdims=True)
        w = w / np.where(t > 0, t, 1.0)
    return (w * dw).sum()


def topk_grad(l, ids, w, dw, renormalize):
    g = np.where(ids >= 0, w * np.where(ids >= 0, dw, 0.0), 0.0)
    dot = g.sum(1, keepdims=True)
    d = np.zeros_like(l) if renormalize else -dot * softmax_rows(l)[0]
    t, j = np.nonzero(ids >= 0)
    d[t, ids[t, j]] += (g - w * dot if renormalize else g)[t, j]
    return d


def balance(l, valid, ids, coefficient):
    """(loss, counts, slope, p) with p the probabilities of the valid rows (zero rows elsewhere)."""
    E = l.shape[1]
    p = softmax_rows(np.where(valid[:, None], l, 0.0))[0] * valid[:, None]
    c = np.bincount(ids[(ids >= 0) & (ids < E)].reshape(-1).astype(np.int64), minlength=E)
    n = int(valid.sum())
    f = c / c.sum() if c.sum() else np.zeros(E)
    slope = coefficient * E * f / n if n else np.zeros(E)
    return (slope * p.sum(0)).sum(), c, slope, p


def balance_grad(p, slope, dloss):
    return dloss * p * (slope - (p * slope).sum(1, keepdims=True))
