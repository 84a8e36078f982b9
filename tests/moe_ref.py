"""The mixture-of-experts operators in numpy, from their formulas: routing in
64 bits, products by the oracle's replay of the documented f32 order."""
import numpy as np

import oracle


def route(logits, top, sigmoid=False, bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(idx int32, weight f64) [T, top], one token and one expert at a time."""
    T, E = logits.shape
    idx, weight = np.full((T, top), -1, np.int32), np.zeros((T, top))
    by_logit = not sigmoid and bias is None and (groups == 1 or group_top == 1)
    for t in range(T):
        l = logits[t].astype(np.float64)
        there = [e for e in range(E) if l[e] > -np.inf]
        s = {}
        if sigmoid:
            with np.errstate(over="ignore"):
                s = {e: 1 / (1 + np.exp(-l[e])) for e in there}
        elif there:
            m = max(l[e] for e in there)
            s = {e: 1.0 if l[e] == m else float(np.exp(l[e] - m)) for e in there}
            total = sum(s.values())
            s = {e: v / total for e, v in s.items()}
        if bias is not None:
            there = [e for e in there if bias[e] > -np.inf]
        c = {e: np.float32(logits[t, e]) if by_logit else np.float32(s[e]) for e in there}
        if bias is not None:
            c = {e: np.float32(c[e] + bias[e]) for e in there}
        if groups > 1:
            size = E // groups
            rank = []
            for g in range(groups):
                best = sorted((c[e] for e in there if e // size == g), reverse=True)
                r = best[0] if best else np.float32(-np.inf)
                if group_top == 2 and len(best) > 1:
                    r = np.float32(best[0] + best[1])
                rank.append(r)
            stay = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            there = [e for e in there if e // size in stay]
        best = sorted(there, key=lambda e: (-c[e], e))[:top]
        total = sum(s[e] for e in best)
        for j, e in enumerate(best):
            idx[t, j] = e
            weight[t, j] = scale * ((s[e] / total if total > 0 else 0.0) if renorm else s[e])
    return idx, weight


def product(fmt, blobs, N, K, x, expert):
    """y[p] = W[expert[p]] x[p] in the documented f32 order, zeros without an expert; blobs: one an expert."""
    y = np.zeros((len(expert), N), np.float32)
    for e in range(len(blobs)):
        p = np.flatnonzero(np.asarray(expert) == e)
        if p.size:
            rows = np.ascontiguousarray(x[p])
            y[p] = oracle.matmul_canon_f32(fmt, blobs[e], N, K, oracle.quantize_act(rows), p.size)
    return y


def gateup(fmt, gates, ups, N, K, x, idx):
    T, top = idx.shape
    rows = np.repeat(x, top, 0)
    e = idx.reshape(-1)
    return oracle.swiglu(product(fmt, gates, N, K, rows, e), product(fmt, ups, N, K, rows, e)).reshape(T, top, N)


def down(fmt, blobs, N, K, h, idx, weight):
    """(y, bound): the weighted sum in 64 bits over the products' f32 values, and sum |weight * product|."""
    T, top = idx.shape
    y = product(fmt, blobs, N, K, h.reshape(T * top, K), idx.reshape(-1)).reshape(T, top, N).astype(np.float64)
    on = (idx >= 0) & (idx < len(blobs))
    w = np.where(on, weight.astype(np.float64), 0.0)[..., None]
    return (w * y).sum(1), np.abs(w * y).sum(1)
