"""Tables, lengths and starts with any contents: what is described comes out right, and not one byte
beside it changes, inside the buffers or around them."""
import numpy as np
import pytest

from step_ref import attention, decode_page, encode_page, q4_0, q4_value
from test_gpu_kv import bound, dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LOW, HIGH = -(1 << 31), (1 << 31) - 1


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


class Guarded:
    """A tensor between two guard areas; `bytes` are all of it, guards included."""
    MARGIN = 4096

    def __init__(self, a):
        a = np.ascontiguousarray(a)
        raw = np.full(a.nbytes + 2 * self.MARGIN, 0x5A, np.uint8)
        raw[self.MARGIN:self.MARGIN + a.nbytes] = a.reshape(-1).view(np.uint8)
        self.all, self.raw = dev(raw), raw
        self.t = self.all[self.MARGIN:self.MARGIN + a.nbytes].view(torch.from_numpy(a[:0]).dtype).view(a.shape)
        self.inside = self.raw[self.MARGIN:self.MARGIN + a.nbytes].view(a.dtype).reshape(a.shape)

    def now(self):
        """The contents, once the guards are seen to be whole."""
        raw = self.all.cpu().numpy()
        assert np.all(raw[:self.MARGIN] == 0x5A) and np.all(raw[-self.MARGIN:] == 0x5A)
        return raw[self.MARGIN:-self.MARGIN].view(self.inside.dtype).reshape(self.inside.shape)


def described(starts, lens, T, max_len):
    """The rows that runs name (row -> sequence, position), every place so named (of a row in two runs
    both), and whether the starts are in order."""
    rows, places = {}, set()
    for b, n in enumerate(lens):
        q0, q1 = starts[b], starts[b + 1]
        if q0 < 0 or q1 < q0 or q1 > T:
            continue
        held = min(max(n, 0), max_len)
        for t in range(q0, q1):
            rows[t] = b, held - (q1 - t)
            places.add(rows[t])
    return rows, places, all(a <= b for a, b in zip(starts, starts[1:]))


def contents(rng, B, T, width, page, n_pages):
    """Starts (in order or not), lengths and a table, with values out of range among them."""
    kind = rng.integers(0, 3)
    cuts = rng.integers(-2, T + 3, B + 1)
    cuts[rng.random(B + 1) < 0.15] = rng.choice([LOW, HIGH, -1, 1 << 20])
    starts = np.sort(cuts) if kind else cuts
    if kind == 2:
        starts = np.clip(starts, 0, T)
    lens = rng.integers(-2, width * page + 3, B)
    lens[rng.random(B) < 0.15] = rng.choice([LOW, HIGH, 0])
    pages = rng.permutation(n_pages)[:B * width].reshape(B, width)
    wrong = rng.random((B, width)) < 0.2
    table = np.where(wrong, rng.choice([-1, LOW, HIGH, n_pages, n_pages + 7], (B, width)), pages)
    return [int(x) for x in starts], [int(x) for x in lens], table.astype(np.int32)


@pytest.mark.parametrize("hq,hkv,d,T,page,kernel,split", [
    (4, 2, 64, 7, 16, 8, False), (6, 1, 96, 24, 16, 16, False), (2, 2, 160, 9, 16, 16, False),
    (64, 64, 32, 900, 16, 64, False), (3, 1, 128, 6, 256, 8, True), (2, 1, 224, 5, 128, 16, True)])
@pytest.mark.parametrize("seed", range(12))
def test_any_contents(g, hq, hkv, d, T, page, kernel, split, seed):
    B, width, nb = 4, 3, d // 32
    rng = np.random.default_rng(1000 * seed + d)
    n_pages, max_len = B * width, width * page - int(rng.integers(0, 5))
    starts, lens, table = contents(rng, B, T, width, page, n_pages)
    print(hq, hkv, d, T, page, seed, starts, lens, table.tolist(), max_len, flush=True)
    assert g.qmv_kv_attention_rows(T, B, True, hq, hkv, d, max_len) == kernel
    assert (g.qmv_kv_attention_bytes(T, B, hq, hkv, d, max_len) > 16) == split
    rows, places, in_order = described(starts, lens, T, max_len)
    pages = np.zeros((n_pages, hkv, page * 36 * nb), np.uint8)
    for p in range(n_pages):
        for h in range(hkv):
            (kc, kd), (vc, vd) = (q4_0(rng.standard_normal((page, d)).astype(np.float32)) for _ in range(2))
            pages[p, h] = encode_page(kc, kd, vc, vd, page, nb)
    pages = Guarded(pages)
    q, k, v = (rng.standard_normal((T, h * d)).astype(np.float32) for h in (hq, hkv, hkv))
    cache = g.KVCache(pages.t.view(-1), page, hkv, d)
    batch = g.KVBatch(dev(table), dev(np.array(lens, np.int32)), dev(np.array(starts, np.int32)), T, max_len)
    q_out, rk, rv, out = (Guarded(np.full((T, h * d), 7.0, np.float32)) for h in (hq, hkv, hkv, hq))
    work = Guarded(np.zeros(g.qmv_kv_attention_bytes(T, B, hq, hkv, d, max_len), np.uint8))

    # append: the rows' keys and values, and nothing else, in the pages
    g.kv_append(cache, batch, dev(q), dev(k), dev(v), q_out=q_out.t)
    stored = {t: (b, p) for t, (b, p) in rows.items() if p >= 0 and 0 <= table[b, p // page] < n_pages}
    held = pages.inside.copy()
    codes = [x.reshape(T, hkv, -1) for x in (k, v)]
    for t, (b, p) in stored.items():
        at = table[b, p // page]
        for h in range(hkv):
            parts = decode_page(held[at, h], page, nb)
            for part, x in zip(parts, (*q4_0(codes[0][t, h]), *q4_0(codes[1][t, h]))):
                part[p % page] = x
            held[at, h] = encode_page(*parts, page, nb)
    got = pages.now()
    if in_order:
        assert np.array_equal(got, held)
    else:  # a row of a run may be left out, or taken by another run
        changed = np.zeros((n_pages, page), bool)
        for b in range(B):
            for p in range(max_len):
                if 0 <= table[b, p // page] < n_pages:
                    changed[table[b, p // page], p % page] = (b, p) in places
        for at in range(n_pages):
            for h in range(min(hkv, 4)):
                for x, y in zip(decode_page(got[at, h], page, nb), decode_page(pages.inside[at, h], page, nb)):
                    assert np.array_equal(x[~changed[at]], y[~changed[at]])

    # the rows that come out: rotated q (here q itself), stored values, attention
    def check(buffer, want, tolerance=None):
        x = buffer.now()
        other = [t for t in range(T) if t not in rows]
        assert np.all(x[other] == 7.0)
        if in_order:
            for t in range(T) if T < 100 else rng.choice(T, 60, replace=False):
                w = want(t) if t in rows else np.full(x.shape[1], 7.0, np.float32)
                assert np.all(np.abs(x[t] - w) <= (tolerance(t) if tolerance and t in rows else 0)), t

    check(q_out, lambda t: q[t] if rows[t][1] >= 0 else np.full(hq * d, 7.0))
    g.kv_read(cache, batch, rk.t, rv.t)
    for buffer, x in ((rk, k), (rv, v)):
        check(buffer, lambda t: q4_value(*q4_0(x[t])) if t in stored else np.full(hkv * d, 7.0))
    scale = float(np.float32(d ** -0.5))
    g.kv_attention(cache, batch, dev(q), scale, out=out.t, work=work.t)
    work.now()
    ks, vs = np.zeros((2, B, max_len, hkv, d))
    seen = np.zeros((B, max_len), bool)
    for b in range(B):
        for p in range(max_len):
            if 0 <= table[b, p // page] < n_pages:
                seen[b, p] = True
    for b in range(B):
        for j in range(width):
            if seen[b, j * page]:
                for h in range(hkv):
                    kc, kd, vc, vd = decode_page(got[table[b, j], h], page, nb)
                    m = min(page, max_len - j * page)
                    ks[b, j * page:j * page + m, h], vs[b, j * page:j * page + m, h] = \
                        q4_value(kc, kd)[:m], q4_value(vc, vd)[:m]
    results = {}

    def want(t):
        b, p = rows[t]
        results[t] = attention(q[t].reshape(1, hq, d), ks[b, :p + 1], vs[b, :p + 1], np.array([p]), scale, 0,
                               seen[b, :p + 1]) if p >= 0 else (np.zeros((1, hq, d)),)
        return results[t][0].reshape(-1)

    check(out, want, lambda t: bound(d, max_len, *results[t][1:]).reshape(-1) if rows[t][1] >= 0 else 0)
    assert np.array_equal(pages.now(), got)  # reading changes nothing
