"""Routing by groups of experts in float64, token by token, from the definition."""
import numpy as np

MASKED = -1e30


def scores(L, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-L))
    m = L.max(axis=1, keepdims=True)
    e = np.where(np.isneginf(L), 0.0, np.exp(L - np.where(np.isneginf(m), 0.0, m)))
    z = e.sum(axis=1, keepdims=True)
    return e / np.where(z == 0, 1.0, z)


def route(L, bias, k, groups, top_groups, score, best, renorm, scale, alpha=0.01):
    """dict(ids, gates, counts, f, P, aux) of logits [T, E]; ties go to the lower index."""
    L = np.asarray(L, np.float64)
    T, E = L.shape
    s = scores(L, score)
    # without a bias the order is that of the logits themselves (exact where s saturates), masked experts behind all of them
    sel = np.where(np.isneginf(L), MASKED, s + (0.0 if bias is None else np.asarray(bias, np.float64)))
    rank = sel if bias is not None else np.where(np.isneginf(L), -np.inf, L)
    ids = np.zeros((T, k), np.int64)
    gates = np.zeros((T, k))
    for t in range(T):
        per = E // groups
        with np.errstate(invalid="ignore"):      # (opposite infinities of the bias: a masked group)
            g = [sum(sorted(sel[t, i * per:(i + 1) * per], reverse=True)[:best]) for i in range(groups)]
        g = [MASKED if np.isnan(v) else v for v in g]
        kept = sorted(range(groups), key=lambda i: (-g[i], i))[:top_groups]
        cand = [e for i in kept for e in range(i * per, (i + 1) * per)]
        ids[t] = sorted(cand, key=lambda e: (-rank[t, e], e))[:k]
        w = s[t, ids[t]]
        gates[t] = scale * w
        if renorm:
            gates[t] = 0.0 if w.sum() == 0 else scale * w / w.sum()
    counts = np.bincount(ids.reshape(-1), minlength=E)
    total = s.sum(axis=1, keepdims=True)
    P = (s / np.where(total == 0, 1.0, total)).mean(axis=0) if T else np.zeros(E)
    f = counts / (k * T) if T else np.zeros(E)
    return dict(ids=ids, gates=gates, counts=counts, f=f, P=P, aux=alpha * E * float((f * P).sum()))


def loss(L, ids, d_gates, f, score, renorm, scale, alpha=0.01, d_aux=1.0):
    """<d_gates, gates> + d_aux * aux with the choice and f held fixed: what moe_group_route_backward differentiates."""
    L = np.asarray(L, np.float64)
    s = scores(L, score)
    w = np.take_along_axis(s, ids, 1)
    S = w.sum(axis=1, keepdims=True)
    gates = scale * (w / np.where(S == 0, 1.0, S) if renorm else w)
    total = s.sum(axis=1, keepdims=True)
    P = (s / np.where(total == 0, 1.0, total)).mean(axis=0)
    return float((gates * d_gates).sum()) + d_aux * alpha * L.shape[1] * float((f * P).sum())


def backward(L, ids, d_gates, f, score, renorm, scale, alpha=0.01, d_aux=1.0):
    L = np.asarray(L, np.float64)
    T, E = L.shape
    s = scores(L, score)
    w = np.take_along_axis(s, ids, 1)
    S = w.sum(axis=1, keepdims=True)
    dw = scale * d_gates
    if renorm:
        Ss = np.where(S == 0, 1.0, S)
        dw = np.where(S == 0, 0.0, scale * (d_gates - (d_gates * w).sum(axis=1, keepdims=True) / Ss) / Ss)
    ds = np.zeros_like(s)
    for j in range(ids.shape[1]):
        np.add.at(ds, (np.arange(T), ids[:, j]), dw[:, j])
    c = d_aux * alpha * E * np.asarray(f, np.float64) / T
    if score == "softmax":
        ds = ds + c
        return s * (ds - (ds * s).sum(axis=1, keepdims=True))
    total = s.sum(axis=1, keepdims=True)
    ts = np.where(total == 0, 1.0, total)
    ds = ds + np.where(total == 0, 0.0, (c - (c * s / ts).sum(axis=1, keepdims=True)) / ts)
    return ds * s * (1.0 - s)
