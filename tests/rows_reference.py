"""The operators on rows of logits in 64 bits, from their definitions (numpy)."""
import numpy as np


def kept_order(x, T, k=0, p=1.0, min_p=0.0):
    """Indices of the kept tokens, in the order of falling logits (lower index first on ties)."""
    x = np.asarray(x, np.float64)
    order = np.argsort(-x, kind="stable")
    order = order[: int((x > -np.inf).sum())]
    if T == 0:
        return order[:1]
    if k > 0:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    n = len(order)
    if p < 1:
        n = max(1, int((np.concatenate([[0.0], np.cumsum(w)[:-1]]) < p * np.cumsum(w)[-1]).sum()))
    n = min(n, int((w >= min_p).sum()))
    return order[:n]


def sample_filtered(x, u, T, k=0, p=1.0, min_p=0.0):
    """(token, distance of u * W to the nearest border of the drawn token over W)."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
        return -1, 1.0
    T, p, min_p = (float(np.float32(v)) for v in (T, p, min_p))
    order = kept_order(x, T, int(k), p, min_p)
    if T == 0:
        return int(order[0]), 1.0
    kept = np.sort(order)
    w = np.exp((x[kept] - x[order[0]]) / T)
    kept, w = kept[w > 0], w[w > 0]
    c = np.cumsum(w)
    t = float(np.float32(u)) * c[-1]
    i = min(int(np.searchsorted(c, t, side="right")), len(kept) - 1)
    low = c[i - 1] if i else 0.0
    return int(kept[i]), min(t - low if i else 1.0, c[i] - t) / c[-1]


def top_logits(x, k, T=1.0):
    """(values [k], ids [k], lse) of one row."""
    x = np.asarray(x, np.float64)
    order = np.argsort(-x, kind="stable")[: int((x > -np.inf).sum())][:k]
    values, ids = np.full(k, -np.inf), np.full(k, -1, np.int32)
    values[: len(order)], ids[: len(order)] = x[order], order
    if not len(order):
        return values, ids, -np.inf
    m = x[order[0]]
    T = float(np.float32(T))
    return values, ids, m / T + np.log(np.exp((x - m) / T).sum())


def distill(x, ids, t, lse=None, T=1.0, w=1.0):
    """(loss, (largest, exp-sum), gradient) of one row, everything in 64 bits."""
    x, t = np.asarray(x, np.float64), np.asarray(t, np.float64)
    T, w = float(np.float32(T)), float(np.float32(w))
    if w == 0:
        return 0.0, (0.0, 0.0), np.zeros_like(x)
    live = (ids >= 0) & (ids < len(x)) & (t > -np.inf)
    ids, t = ids[live], t[live]
    m = x.max()
    e = np.exp((x - m) / T)
    S = e.sum()
    if not len(ids):
        return 0.0, (m, S), np.zeros_like(x)
    if lse is None:
        logp = (t - t.max()) / T - np.log(np.exp((t - t.max()) / T).sum())
    else:
        logp = t / T - float(lse)
    p = np.exp(logp)
    loss = w * (p * (logp - ((x[ids] - m) / T - np.log(S)))).sum()
    grad = p.sum() * e / S
    np.subtract.at(grad, ids, p)
    return loss, (m, S), w / T * grad
