"""fp64 references of the router's training operators, with bounds on what fp32
arithmetic may be off by (numpy, no code of the library).

Bounds count roundings of EPS = 2^-24.  A probability exp(z - m) / S: the
subtraction and the product by log2(e) are each off by |z - m| EPS in the
exponent, the exponential by 2 EPS, S (positive terms, at most 16 in a row and 6
tree steps) by 22 EPS, the reciprocal and the product by 2 EPS:
(2 |z - m| + 26) EPS of it.
"""
import numpy as np

EPS = 2.0 ** -24


def softmax_lse(z):
    """Rows of softmax and logsumexp; a row of -inf leaves 0 and 0."""
    m = z.max(axis=1, keepdims=True)
    none = np.isneginf(m)
    m = np.where(none, 0.0, m)
    w = np.exp(z - m)
    s = np.where(none, 1.0, w.sum(axis=1, keepdims=True))
    return w / s, np.where(none, 0.0, m + np.log(s))[:, 0]


def selected_probs(z, ids):
    q = np.take_along_axis(z, ids, axis=1)
    q = np.exp(q - q.max(axis=1, keepdims=True))
    return q / q.sum(axis=1, keepdims=True)


def exponent_span(z):
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(z) & np.isfinite(m), m - z, 0.0)
    # below e^-110 an fp32 exponential is 0, and the probability lost is nothing
    return np.minimum(d, 110.0)


def balance_ref(z, ids, keep):
    """losses [2], counts [E + 1], prob_sums [E] in fp64."""
    z = np.asarray(z, np.float64)
    E, k = z.shape[1], ids.shape[1]
    p, lse = softmax_lse(z)
    hit = ids[keep].reshape(-1)
    hit = hit[(hit >= 0) & (hit < E)]
    counts = np.bincount(hit, minlength=E)
    n = int(keep.sum())
    sums = p[keep].sum(axis=0)
    N = max(n, 1)
    losses = np.array([E / (k * N * N) * (counts * sums).sum(), (lse[keep] ** 2).sum() / N])
    return losses, np.append(counts, n), sums


def balance_bounds(z, ids, keep, in_order):
    """What losses and prob_sums may be off by.  in_order: the most fp32 additions that
    one value passes through."""
    z = np.asarray(z, np.float64)
    E, k = z.shape[1], ids.shape[1]
    p, lse = softmax_lse(z)
    losses, counts, sums = balance_ref(z, ids, keep)
    n = max(int(keep.sum()), 1)
    off = (p * (2 * exponent_span(z) + 26))[keep].sum(axis=0) * EPS + sums * in_order * EPS
    bal = E / (k * n * n) * (counts[:E] * (off + sums * (E / 64 + 40) * EPS)).sum()
    # lse = m + log(s): log(s) in [0, 7] off by 3 of its own roundings and S's 22,
    # the sum by one of the result's
    d = (np.abs(lse) + 7 * 3 + 22) * EPS
    zl = (2 * np.abs(lse) * d + lse ** 2 * (in_order + 4) * EPS)[keep].sum() / n
    # the fp32 smallest normal covers sums of probabilities that underflow
    return np.array([bal, zl]) + 1e-37, off + 1e-37


def route_backward_ref(z, ids, keep, q, d, counts, g):
    """d_logits in fp64 and its bound; q, d or counts, g may be None."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    grad, off = np.zeros((T, E)), np.zeros((T, E))
    if counts is not None:
        k = ids.shape[1]
        n = int(counts[E])
        inv = 1.0 / n if n else 0.0
        p, lse = softmax_lse(z)
        c = g[0] * E * inv * inv / k * (counts[:E] - k * n / E)
        inner = c[None] - (p @ c)[:, None] + 2 * g[1] * inv * lse[:, None]
        grad += np.where(keep[:, None], p * inner, 0.0)
        size = np.abs(c)[None] + (p @ np.abs(c))[:, None] + np.abs(2 * g[1] * inv * lse[:, None])
        span = 2 * exponent_span(z) + 26
        worst = (p * span).sum(axis=1, keepdims=True)        # of the mean's probabilities
        off += np.where(keep[:, None], p * size * (span + worst + 60) * EPS
                        + p * abs(2 * g[1] * inv) * (7 * 3 + 22) * EPS, 0.0)
    if d is not None:
        for t in range(T):
            ok = [(0 <= ids[t, j] < E) and ids[t, j] not in ids[t, :j] for j in range(ids.shape[1])]
            qt, dt = np.where(ok, q[t], 0.0).astype(np.float64), np.where(ok, d[t], 0.0).astype(np.float64)
            dot, mag = (qt * dt).sum(), np.abs(qt * dt).sum()
            for j, use in enumerate(ok):
                if use:
                    grad[t, ids[t, j]] += qt[j] * (dt[j] - dot)
                    off[t, ids[t, j]] += qt[j] * (np.abs(dt[j]) * 3 + mag * 24) * EPS
    return grad, off + np.abs(grad) * 2 * EPS + 1e-37
