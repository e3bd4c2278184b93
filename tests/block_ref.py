"""Plain 64-bit references (numpy) of the operators around the quantized products, for the parity tests."""
import numpy as np


def scores(logits, sigmoid):
    """Scores of [tokens, experts] logits in 64 bits, and which experts are open."""
    l = np.array(logits, dtype=np.float64)
    is_open = ~(np.isnan(l) | (l == -np.inf))
    l = np.where(is_open, np.minimum(l, float(np.finfo(np.float32).max)), -np.inf)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            return np.where(is_open, 1.0 / (1.0 + np.exp(-l)), 0.0), is_open
        e = np.where(is_open, np.exp(l - np.max(l, axis=1, keepdims=True)), 0.0)
        return np.where(is_open, e / e.sum(axis=1, keepdims=True), 0.0), is_open


def _clear(values):
    """Whether the order of falling values is clear at 32 bits: neighbours equal, or 1e-6 apart."""
    v = values[np.isfinite(values)]
    gap = -np.diff(v)
    return bool(np.all((gap == 0) | (gap > 1e-6)))


def route(logits, k, sigmoid=False, renorm=False, sum2=False, bias=None, groups=1, group_k=1, scale=1.0):
    """(ids, weights, clear): clear[t] says that no choice of token t hangs on less than 1e-6."""
    s, is_open = scores(logits, sigmoid)
    T, E = s.shape
    key = np.where(is_open, s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64)), -np.inf)
    key[np.isnan(key)] = -np.inf
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    clear = np.ones(T, dtype=bool)
    for t in range(T):
        kt = key[t].copy()
        if group_k < groups:
            per = np.sort(kt.reshape(groups, -1), axis=1)[:, ::-1]
            value = per[:, 0].copy()
            if sum2 and per.shape[1] > 1:
                value += np.where(np.isfinite(per[:, 1]), per[:, 1], 0.0)
            order = np.argsort(-value, kind="stable")
            clear[t] &= _clear(value[order])
            shut = order[group_k:]
            kt.reshape(groups, -1)[shut] = -np.inf
        order = np.argsort(-kt, kind="stable")
        clear[t] &= _clear(kt[order[:k + 1]])
        for j in range(k):
            if kt[order[j]] > -np.inf:
                ids[t, j] = order[j]
                w[t, j] = s[t, order[j]]
    if renorm:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return ids, w * scale, clear


def route_weights(logits, ids, sigmoid, renorm, scale):
    """The weights for given ids (the differentiable part)."""
    s, _ = scores(logits, sigmoid)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    if renorm:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return w * scale


def route_backward(logits, ids, dweights, sigmoid, renorm, scale):
    s, is_open = scores(logits, sigmoid)
    dl = np.zeros_like(s)
    for t in range(s.shape[0]):
        sel = [j for j in range(ids.shape[1]) if ids[t, j] >= 0]
        p = np.array([s[t, ids[t, j]] for j in sel])
        g = np.array([dweights[t, j] for j in sel], dtype=np.float64) * scale
        if renorm:
            total = p.sum() + 1e-20
            g = g / total - (g * p).sum() / total ** 2
        ds = np.zeros(s.shape[1])
        for j, v in zip(sel, g):
            ds[ids[t, j]] += v
        dl[t] = ds * s[t] * (1 - s[t]) if sigmoid else s[t] * (ds - (ds * s[t]).sum())
    return np.where(is_open, dl, 0.0)


def plan(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in np.flatnonzero(flat == e)]
    rows = np.full(T * k, -1, dtype=np.int64)
    rows[:len(slots)] = slots
    pos = np.full(T * k, -1, dtype=np.int64)
    pos[slots] = np.arange(len(slots))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return offsets, rows, pos.reshape(T, k)


def int8_rows(x):
    """8-bit rows by the definition (scale, reciprocal and product are 32-bit numbers)."""
    x = np.asarray(x, dtype=np.float32)
    s = (np.abs(x).max(axis=1) * (np.float32(1) / np.float32(127))).astype(np.float32)
    s = np.where(s >= np.finfo(np.float32).tiny, s, np.float32(0)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
    return np.rint((x * inv[:, None]).astype(np.float32)).astype(np.int8), s


def block_norm(x, y, w_post, gate, w_pre, alpha, eps, one_plus):
    """(x', n, rstd_post, rstd_pre) in 64 bits; None where there is none."""
    shift = 1.0 if one_plus else 0.0
    x1, n, r1, r2 = x, None, None, None
    if y is not None:
        p = y
        if w_post is not None:
            r1 = 1.0 / np.sqrt((y * y).mean(axis=1) + eps)
            p = y * r1[:, None] * (w_post + shift)
        x1 = x + alpha * (p if gate is None else gate * p)
    if w_pre is not None:
        r2 = 1.0 / np.sqrt((x1 * x1).mean(axis=1) + eps)
        n = x1 * r2[:, None] * (w_pre + shift)
    return x1, n, r1, r2


def block_norm_backward(dx_out, dn, x, y, w_post, gate, w_pre, alpha, eps, one_plus):
    """Gradients by the formulas, as a dict of the ones that exist."""
    shift = 1.0 if one_plus else 0.0
    x1, _, r1, r2 = block_norm(x, y, w_post, gate, w_pre, alpha, eps, one_plus)
    out = {}
    d = np.zeros_like(x) if dx_out is None else dx_out.copy()
    if w_pre is not None:
        xh = x1 * r2[:, None]
        out["dw_pre"] = (dn * xh).sum(axis=0)
        u = dn * (w_pre + shift)
        d = d + r2[:, None] * (u - xh * (u * xh).mean(axis=1, keepdims=True))
    out["dx"] = d
    if y is not None:
        yh = y if w_post is None else y * r1[:, None]
        p = yh if w_post is None else yh * (w_post + shift)
        q = alpha * d
        if gate is not None:
            dg = q * p
            out["dgate"] = dg.sum(axis=0) if gate.ndim == 1 else dg
            q = q * gate
        if w_post is not None:
            out["dw_post"] = (q * yh).sum(axis=0)
            u = q * (w_post + shift)
            q = r1[:, None] * (u - yh * (u * yh).mean(axis=1, keepdims=True))
        out["dy"] = q
    return out
