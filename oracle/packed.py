"""Causal attention of one query head of one sequence, forward and backward, in float64: n queries over m keys, the last
query at the last key, optionally only the last `window` keys."""
import numpy as np


def mask(n, m, window=0):
    t = np.arange(n)[:, None] + m - n
    j = np.arange(m)
    ok = j <= t
    return ok & (j > t - window) if window else ok


def weights(q, k, scale, window=0):
    """(P [n, m], lse [n]); rows that see nothing have P = 0, lse = -inf."""
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    n, m = len(q), len(k)
    s = np.where(mask(n, m, window), scale * (q @ k.T), -np.inf) if m else np.zeros((n, 0))
    top = s.max(1, initial=-np.inf)
    p = np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None])
    z = p.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, np.where(np.isinf(top), 0.0, top) + np.log(z), -np.inf)
    return p / np.where(z > 0, z, 1.0)[:, None], lse


def forward(q, k, v, scale, window=0):
    p, lse = weights(q, k, scale, window)
    return p @ np.asarray(v, np.float64), lse


def backward(q, k, v, do, scale, window=0):
    """(dq, dk, dv)"""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    p, _ = weights(q, k, scale, window)
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdims=True))
    return scale * (ds @ k), scale * (ds.T @ q), p.T @ do
