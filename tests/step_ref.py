"""Plain numpy definitions of the operators around the quantised products, in
64 bits with the roundings that include/qmv.h states.  Shares no code with the
library or the oracle."""
import numpy as np

NIB = [0, 4, 1, 5, 2, 6, 3, 7]  # the nibble of a K word that holds element e


def rmsnorm(x, w, eps, res=None):
    """(h f32, y f64 before its rounding to f32)."""
    h = x if res is None else (x + res).astype(np.float32)
    hd = h.astype(np.float64)
    r = 1.0 / np.sqrt((hd * hd).sum(-1, keepdims=True) / h.shape[-1] + float(np.float32(eps)))
    return h, hd * r * w.astype(np.float64)


def rotate(x, pos, freq, halves):
    """x [T, heads, D] -> rotated, f64 before its rounding to f32."""
    y = x.astype(np.float64)
    half = len(freq)
    a = pos[:, None, None].astype(np.float64) * freq
    c, s = np.cos(a), np.sin(a)
    i0 = np.arange(half) if halves else 2 * np.arange(half)
    i1 = i0 + half if halves else i0 + 1
    x0, x1 = x[..., i0].astype(np.float64), x[..., i1].astype(np.float64)
    y[..., i0] = x0 * c - x1 * s
    y[..., i1] = x0 * s + x1 * c
    return y


def q4_0(x):
    """x f32 [..., 32 n] -> (codes int [..., n, 32], d f16 [..., n])."""
    b = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    i = np.abs(b).argmax(-1)  # the first of equals
    top = np.take_along_axis(b, i[..., None], -1)
    d = (top / np.float32(-8)).astype(np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        inv = (np.float32(1) / d).astype(np.float32)
    inv = np.where(np.isfinite(inv), inv, np.float32(0)).astype(np.float32)
    t = (b * inv).astype(np.float32) + np.float32(8.5)
    return np.minimum(15, np.trunc(t).astype(np.int64)), d[..., 0].astype(np.float16)


def q4_value(code, d):
    """f64 values [..., 32 n]."""
    v = (code.astype(np.float64) - 8) * d.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


def page_bytes(page, nb):
    return page * 36 * nb


def decode_page(raw, page, nb):
    """One head's bytes of one page -> (K codes, K d, V codes, V d), codes [page, nb, 32]."""
    n = page * 16 * nb
    kb = raw[:n].reshape(page, 4, nb, 4)
    kn = np.stack([kb & 15, kb >> 4], -1).reshape(page, 4, nb, 8)[..., NIB]
    kc = kn.transpose(0, 2, 1, 3).reshape(page, nb, 32)
    vb = raw[n:2 * n].reshape(page // 4, 16, nb, 4)
    vn = np.stack([vb & 15, vb >> 4], -1)              # [page/4, m, b, t, nibble]
    vc = vn.transpose(0, 3, 2, 1, 4).reshape(page, nb, 32)
    sc = raw[2 * n:].view(np.float16).reshape(2, page, nb)
    return kc.astype(np.int64), sc[0], vc.astype(np.int64), sc[1]


def encode_page(kc, kd, vc, vd, page, nb):
    """The inverse of decode_page."""
    inv = np.argsort(NIB)
    kn = kc.reshape(page, nb, 4, 8).transpose(0, 2, 1, 3)[..., inv].reshape(page, 4, nb, 4, 2)
    kb = (kn[..., 0] | (kn[..., 1] << 4)).astype(np.uint8)
    vn = vc.reshape(page // 4, 4, nb, 16, 2).transpose(0, 3, 2, 1, 4)
    vb = (vn[..., 0] | (vn[..., 1] << 4)).astype(np.uint8)
    return np.concatenate([kb.reshape(-1), vb.reshape(-1),
                           np.ascontiguousarray(kd).view(np.uint8).reshape(-1),
                           np.ascontiguousarray(vd).view(np.uint8).reshape(-1)])


def attention(q, k, v, pos, scale, window=0, seen=None):
    """One sequence: q [n, Hq, D], k, v [L, Hkv, D] f64, pos [n].  Returns out
    [n, Hq, D] and sizes that errors are measured by, per row and head: max_t
    sum_d |q k| scale, sum_t p |v| [D], max_t p max_d |v|."""
    n, hq, _ = q.shape
    g = hq // k.shape[1]
    out, amax, pmax = np.zeros(q.shape), np.zeros((n, hq)), np.zeros((n, hq))
    pv = np.zeros(q.shape)
    t = np.arange(len(k))
    for j in range(n):
        vis = t <= pos[j]
        if window:
            vis &= t > pos[j] - window
        if seen is not None:
            vis &= seen
        if not vis.any():
            continue
        for h in range(hq):
            kk, vv = k[vis, h // g], v[vis, h // g]
            s = kk @ q[j, h].astype(np.float64) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[j, h] = p @ vv
            amax[j, h] = (np.abs(kk) @ np.abs(q[j, h].astype(np.float64))).max() * scale
            pv[j, h] = p @ np.abs(vv)
            pmax[j, h] = (p * np.abs(vv).max(-1)).max()
    return out, amax, pv, pmax
