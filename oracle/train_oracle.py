"""fp64 restatement of the operators around the layer's training step: the
router's sequence-wise balance loss and z-loss with their gradient, low-rank
adapters of many requests with theirs, and the global gradient norm with
clipping. Plain numpy, one sequence, adapter or tensor at a time."""
import numpy as np


def router_probs(l, score):
    """(p, slope): the normalised scores of a row set and d p_e / d l_j =
    slope_j p_j ([e = j] - p_e)."""
    if score == "softmax":
        e = np.exp(l - l.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True), np.ones_like(l)
    t = np.exp(-np.abs(l))
    s = np.minimum(l, 0) - np.log1p(t)  # log sigmoid: a row's sigmoids may all lie below the smallest number
    s = np.exp(s - s.max(1, keepdims=True))
    return s / s.sum(1, keepdims=True), np.where(l >= 0, t / (1 + t), 1 / (1 + t))


def valid_rows(T, seq_offsets, token_mask):
    keep = np.ones(T, bool) if token_mask is None else np.asarray(token_mask).astype(bool)
    off = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    return [a + np.nonzero(keep[a:b])[0] for a, b in zip(off[:-1], off[1:])]


def balance(logits, topk_idx, k, score="softmax", balance_coeff=1e-2, z_coeff=0.0, seq_offsets=None, token_mask=None,
            dlosses=(1.0, 1.0)):
    """(losses [2], counts [S, E], dlogits [T, E], scale [T, E]): scale bounds
    each gradient's terms before they cancel, for tolerances."""
    T, E = logits.shape
    rows = valid_rows(T, seq_offsets, token_mask)
    filled, n = sum(len(q) > 0 for q in rows), sum(len(q) for q in rows)
    losses, counts = np.zeros(2), np.zeros((len(rows), E), np.int64)
    d, scale = np.zeros((T, E)), np.zeros((T, E))
    for s, q in enumerate(rows):
        if len(q) == 0:
            continue
        l = logits[q].astype(np.float64)
        idx = topk_idx[q].reshape(-1)
        np.add.at(counts[s], idx[(idx >= 0) & (idx < E)], 1)
        f = E * counts[s] / (k * len(q))
        p, slope = router_probs(l, score)
        m = l.max(1, keepdims=True)
        ex = np.exp(l - m)
        lse = (m + np.log(ex.sum(1, keepdims=True)))
        soft = ex / ex.sum(1, keepdims=True)
        losses[0] += balance_coeff / filled * (f * p.mean(0)).sum()
        w = dlosses[0] * balance_coeff / filled * f / len(q)
        d[q] = p * slope * (w - (p * w).sum(1, keepdims=True))
        scale[q] = p * (np.abs(w) + (p * np.abs(w)).sum(1, keepdims=True))
        if z_coeff != 0.0:
            losses[1] += z_coeff / n * (lse ** 2).sum()
            g = 2 * dlosses[1] * z_coeff / n
            d[q] += g * lse * soft
            scale[q] += abs(g) * (np.abs(lse) + 1) * soft
    return losses, counts, d, scale


def adapter(x, A, B, scale, idx, base, dy=None, dx_base=None):
    """{"y", "dx", "dA", "dB"} and, under "size", the same sums of magnitudes:
    u, y, du, dx, dA, dB with every factor replaced by its absolute value."""
    L = A.shape[0]
    out = {"y": base.copy()}
    T, K = x.shape
    r, N = B.shape[1:]
    size = {"u": np.zeros((T, r)), "y": np.zeros((T, N)), "us": np.zeros((T, r))}
    if dy is not None:
        out |= {"dx": dx_base.copy(), "dA": np.zeros((L, K, r)), "dB": np.zeros((L, r, N))}
        size |= {"du": np.zeros((T, r)), "dus": np.zeros((T, r)), "dx": np.zeros((T, K))}
    for a in range(L):
        q = np.nonzero(idx == a)[0]
        if len(q) == 0:
            continue
        c = float(scale[a])
        u = c * (x[q] @ A[a])
        out["y"][q] += u @ B[a]
        size["us"][q] = np.abs(u)
        size["u"][q] = abs(c) * (np.abs(x[q]) @ np.abs(A[a]))
        if dy is not None:
            du = c * (dy[q] @ B[a].T)
            out["dx"][q] += du @ A[a].T
            out["dA"][a] = x[q].T @ du
            out["dB"][a] = u.T @ dy[q]
            size["dus"][q] = np.abs(du)
            size["du"][q] = abs(c) * (np.abs(dy[q]) @ np.abs(B[a]).T)
    return out, size


def grad_norm(tensors, kind="l2"):
    if kind == "max":
        return max([float(np.abs(t).max()) if not np.isnan(t).any() else np.nan for t in tensors if t.size], default=0.0)
    top = max([float(np.abs(t).max()) for t in tensors if t.size], default=0.0)
    if top == 0.0 or not np.isfinite(top):
        return top
    return top * float(np.sqrt(sum(((t.astype(np.float64) / top) ** 2).sum() for t in tensors)))


def clip(tensors, max_norm, kind="l2"):
    n = grad_norm(tensors, kind)
    coef = min(1.0, max_norm / (n + 1e-6))
    return n, [t.astype(np.float64) * coef for t in tensors]
