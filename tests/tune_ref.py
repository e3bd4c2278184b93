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
