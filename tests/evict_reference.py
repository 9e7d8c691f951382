"""Plain 64-bit implementations of the eviction operators (numpy, by the formulas of
include/hstu_evict.h)."""
import numpy as np


def key_weights(q, lse, K, causal, alpha):
    """q [n, Nq, D], lse [n, Nq], K [Lk, Nk, D] -> the weights [Nk, Lk] and, for the tolerance, the
    sums of weight times (bound on |score| / |alpha ..| roundings): sum p |alpha| |q| |k|, sum p |lse|."""
    n, Nq, _ = q.shape
    Lk, Nk = K.shape[:2]
    out, size, off = (np.zeros((Nk, Lk)) for _ in range(3))
    for h in range(Nq):
        if not n or not Lk:
            continue
        k = K[:, h // (Nq // Nk)]
        with np.errstate(over="ignore"):
            p = np.exp(alpha * (q[:, h] @ k.T) - lse[:, h, None])
        if causal:
            p = np.where(np.arange(Lk)[None, :] <= (Lk - n + np.arange(n))[:, None], p, 0.0)
        bound = abs(alpha) * np.linalg.norm(q[:, h], axis=1)[:, None] * np.linalg.norm(k, axis=1)[None, :]
        seen = np.isfinite(lse[:, h])
        out[h // (Nq // Nk)] += p[seen].sum(0)
        size[h // (Nq // Nk)] += (p * bound)[seen].sum(0)
        off[h // (Nq // Nk)] += (p[seen] * np.abs(lse[seen, h, None])).sum(0)
    return out, size, off


def select(w, budget, recent):
    """Positions to keep of one sequence and kv head with weights w [Lk]."""
    Lk = len(w)
    keep = min(Lk, budget)
    last = min(recent, keep)
    others = sorted(range(Lk - last), key=lambda j: (np.isnan(w[j]), -w[j] if not np.isnan(w[j]) else 0.0, j))
    return sorted(others[:keep - last]) + list(range(Lk - last, Lk))
