"""Plain 64-bit references (numpy) of the operators of fine-tuning, for the parity tests."""
import numpy as np

U = 2.0 ** -24  # half a step of a 32-bit number, relative


def probs(logits, sigmoid):
    """(p, s, open, top) of [tokens, experts] logits: probabilities, sigmoid scores, open experts, largest logit."""
    l = np.array(logits, dtype=np.float64)
    is_open = ~(np.isnan(l) | (l == -np.inf))
    l = np.where(is_open, np.minimum(l, float(np.finfo(np.float32).max)), -np.inf)
    top = l.max(axis=1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        s = np.where(is_open, 1.0 / (1.0 + np.exp(-l)), 0.0)
        if sigmoid:
            p = s / (s.sum(axis=1, keepdims=True) + 1e-20)
        else:
            e = np.where(is_open, np.exp(l - top), 0.0)
            p = np.where(is_open, e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300), 0.0)
    return p, s, is_open, top


def balance(logits, ids, coef, sequences, sigmoid):
    """(loss, counts, mean probabilities, tokens) and the shares count * E / (k N)."""
    T, E = logits.shape
    k, seq = ids.shape[1], T // sequences
    p = probs(logits, sigmoid)[0]
    live = ((ids >= 0) & (ids < E)).any(axis=1)
    counts, mean, tokens, loss = np.zeros((sequences, E), dtype=np.int64), np.zeros((sequences, E)), np.zeros(sequences, dtype=np.int64), 0.0
    for s in range(sequences):
        part = slice(s * seq, (s + 1) * seq)
        i = ids[part]
        counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        tokens[s] = live[part].sum()
        if tokens[s]:
            mean[s] = p[part][live[part]].sum(axis=0) / tokens[s]
            loss += (counts[s] * E / (k * tokens[s]) * mean[s]).sum()
    return loss * coef / sequences, counts, mean, tokens


def balance_backward(logits, ids, counts, tokens, coef, sigmoid, dloss=1.0):
    """The gradient by the formula, and how far one in 32 bits may be off (see the comment in the tests)."""
    T, E = logits.shape
    S, k = counts.shape[0], ids.shape[1]
    seq = T // S
    p, s, is_open, top = probs(logits, sigmoid)
    l = np.array(logits, dtype=np.float64)
    live = ((ids >= 0) & (ids < E)).any(axis=1)
    n = np.repeat(counts.astype(np.float64), seq, axis=0)
    N = np.repeat(np.maximum(tokens, 1).astype(np.float64), seq)[:, None]
    c = np.where(live[:, None], coef * dloss * E / (S * k * N * N), 0.0)
    # the count of the expert with the largest logit, from which the differences are taken
    ref = np.where(np.minimum(l, float(np.finfo(np.float32).max)) == top, n, 0.0).max(axis=1, keepdims=True)
    slope = 1.0 / (1.0 + np.exp(np.clip(l, -700, 700))) if sigmoid else 1.0
    mean = (p * n).sum(axis=1, keepdims=True)
    spread = (p * np.abs(n - ref)).sum(axis=1, keepdims=True)
    # differences from ref: what sums to n - mean in exact numbers, without its cancellation
    d = (n - ref) - (p * (n - ref)).sum(axis=1, keepdims=True)
    if sigmoid:
        d = d + ref * (1e-20 / (s.sum(axis=1, keepdims=True) + 1e-20))
    grad = np.where(is_open, c * p * slope * d, 0.0)
    with np.errstate(invalid="ignore"):
        deep = np.where(is_open, np.abs(l - top), 0.0).max(axis=1, keepdims=True) if not sigmoid else 0.0
    rel = (np.minimum(deep, 110.0) + E / 16 + 24) * U
    tol = np.abs(c) * p * slope * (2 * rel * (np.abs(n - ref) + spread) + 4 * U * ref * (1e-20 / (s.sum(axis=1, keepdims=True) + 1e-20) if sigmoid else 0.0))
    return grad, np.where(is_open, tol, 0.0) + 2.0 ** -126


def adapter(x, a, b, scales, owner, base, x_rows):
    """c [rows x N] in 64 bits, and the magnitudes its sums run over.  owner: the adapter of each row (-1: none); x_rows:
    its row of x; a [L, R, K], b [L, N, R]."""
    c, mag = base.copy(), np.abs(base)
    h = np.zeros((len(owner), a.shape[1]))
    for g in range(a.shape[0]):
        at = np.flatnonzero(owner == g)
        if len(at) == 0:
            continue
        rows = x[x_rows[at]]
        h[at] = rows @ a[g].T
        c[at] += scales[g] * (h[at] @ b[g].T)
        mag[at] += np.abs(scales[g]) * ((np.abs(rows) @ np.abs(a[g]).T) @ np.abs(b[g]).T)
    return c, h, mag


def adapter_backward(dc, x, a, b, scales, owner, h, dx_base):
    """(dx, da, db) and the magnitudes of their sums; x's rows are c's."""
    dx, dxm = dx_base.copy(), np.abs(dx_base)
    da, db, dam, dbm = np.zeros_like(a), np.zeros_like(b), np.zeros_like(a), np.zeros_like(b)
    for g in range(a.shape[0]):
        at = np.flatnonzero(owner == g)
        if len(at) == 0:
            continue
        s = scales[g]
        gr, gm = s * (dc[at] @ b[g]), np.abs(s) * (np.abs(dc[at]) @ np.abs(b[g]))
        dx[at] += gr @ a[g]
        dxm[at] += gm @ np.abs(a[g])
        da[g], dam[g] = gr.T @ x[at], gm.T @ np.abs(x[at])
        db[g] = s * (dc[at].T @ h[at])
        dbm[g] = np.abs(s) * (np.abs(dc[at]).T @ (np.abs(x[at]) @ np.abs(a[g]).T))
    return (dx, da, db), (dxm, dam, dbm)
