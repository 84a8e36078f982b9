"""The paged 4-bit cache on the GPU: append with rotation, read back,
attention, against the definitions in 64 bits."""
import numpy as np
import pytest

from step_ref import attention, decode_page, encode_page, q4_0, q4_value, rotate

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A cache with pages in no order, sequences of `lens` tokens whose last `ns` are a call's rows."""

    def __init__(self, lens, ns, page, hkv, d, seed, spare_rows=0, spare_pages=2, spare_table=1):
        self.rng = np.random.default_rng(seed)
        self.lens, self.ns, self.page, self.hkv, self.d, self.nb = lens, ns, page, hkv, d, d // 32
        self.B = len(lens)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare_pages
        order = self.rng.permutation(self.n_pages)
        self.table = np.full((self.B, max(need + [1]) + spare_table), -7, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.spare = order[at:]
        self.starts = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.rows = int(self.starts[-1])
        self.T = self.rows + spare_rows
        self.pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, ns)] or [[]]).astype(np.int64)
        self.seq = np.repeat(np.arange(self.B), ns)
        self.head_bytes = page * 36 * self.nb

    def batch(self, g, max_len=None, starts=True):
        return g.KVBatch(dev(self.table), dev(np.array(self.lens, np.int32)),
                         dev(self.starts) if starts else None, self.T if starts else None,
                         max_len or max(self.lens + [1]))

    def cells(self, raw):
        return raw.reshape(self.n_pages, self.hkv, self.head_bytes)

    def token(self, raw, b, p):
        """(K codes, K d, V codes, V d) of a token, [hkv, ...]."""
        page = self.cells(raw)[self.table[b, p // self.page]]
        parts = [decode_page(page[h], self.page, self.nb) for h in range(self.hkv)]
        return [np.stack([x[i][p % self.page] for x in parts]) for i in range(4)]


def nasty(rng, shape):
    """Keys and values with zero blocks, ties of the largest magnitude and very small ones."""
    x = rng.standard_normal(shape).astype(np.float32)
    f = x.reshape(-1, 32)
    kind = rng.integers(0, 9, len(f))
    f[kind == 0] = 0
    f[kind == 1] *= np.float32(1e-6)
    tie = kind == 2
    f[tie, 5], f[tie, 21] = 4.0, -4.0
    f[kind == 3, 31] = 300.0
    f[kind == 4] *= np.float32(1e-40)  # 1/d is not finite: codes 8, d 0
    return x


APPENDS = [
    # lens, rows of each, page, q heads, kv heads, d, rot, halves
    ([1], [1], 16, 1, 1, 32, 32, False),
    ([777], [1], 64, 32, 8, 128, 128, False),
    ([5, 40, 16, 17], [1, 1, 1, 1], 16, 14, 2, 64, 64, True),
    ([33, 5, 100], [33, 3, 70], 32, 6, 3, 96, 48, True),
    ([50, 30, 0, 20], [20, 0, 0, 20], 16, 5, 1, 160, 160, False),
    ([130], [130], 64, 4, 4, 256, 128, False),
    ([9, 31], [9, 17], 16, 2, 1, 224, 0, False),
    ([20], [20], 16, 3, 1, 192, 192, True),
]


@pytest.mark.parametrize("lens,ns,page,hq,hkv,d,rot,halves", APPENDS)
def test_append(g, lens, ns, page, hq, hkv, d, rot, halves):
    print("append", lens, ns, page, hq, hkv, d, rot, halves, flush=True)
    c = Case(lens, ns, page, hkv, d, 3, spare_rows=3)
    rng = c.rng
    q = rng.standard_normal((c.T, hq * d)).astype(np.float32)
    k, v = nasty(rng, (c.T, hkv * d)), nasty(rng, (c.T, hkv * d))
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    before = rng.integers(0, 256, c.n_pages * hkv * c.head_bytes, dtype=np.uint8)
    pages = dev(before)
    cache, batch = g.KVCache(pages, page, hkv, d), c.batch(g)
    # the three as parts of one buffer, with its row stride
    width = (hq + 2 * hkv) * d + 4
    both = torch.zeros(c.T, width, device="cuda")
    qd, kd, vd = both[:, :hq * d], both[:, hq * d:(hq + hkv) * d], both[:, (hq + hkv) * d:(hq + 2 * hkv) * d]
    qd.copy_(dev(q)); kd.copy_(dev(k)); vd.copy_(dev(v))
    out = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_append(cache, batch, qd, kd, vd, dev(freq) if rot else None, halves=halves, q_out=out)
    torch.cuda.synchronize()
    got, raw = out.cpu().numpy(), pages.cpu().numpy()
    n = c.rows
    # the rotated q: one rounding of what f64 holds to far below an f32 step (a few of its own
    # roundings of the two products)
    want = rotate(q[:n].reshape(n, hq, d), c.pos, freq, halves).reshape(n, -1)
    assert np.all(np.abs(got[:n] - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -45)
    assert np.all(got[n:] == 7.0)  # rows of no sequence
    kr = rotate(k[:n].reshape(n, hkv, d), c.pos, freq, halves).astype(np.float32)
    kc, ks = q4_0(kr)
    vc, vs = q4_0(v[:n].reshape(n, hkv, d))
    touched = np.zeros(c.cells(raw).shape, bool)
    for i in range(n):
        a = c.token(raw, c.seq[i], c.pos[i])
        for x, y in zip(a, (kc[i], ks[i], vc[i], vs[i])):
            assert np.array_equal(x, y), (i, x, y)
        p = int(c.pos[i]) % page
        cell = touched[c.table[c.seq[i], c.pos[i] // page]]
        kcode = np.zeros((page, c.nb, 32), int)
        kcode[p] = 15
        half = np.zeros((page, c.nb), np.float16)
        half.view(np.uint16)[p] = 0xFFFF
        cell |= encode_page(kcode, half, kcode, half, page, c.nb) != 0
    now, was = c.cells(raw), c.cells(before)
    assert np.array_equal(now[~touched], was[~touched])  # every other token's bytes
    # what a reader sees
    rk = torch.full((c.T, hkv * d), 5.0, device="cuda")
    rv = rk.clone()
    g.kv_read(cache, batch, rk, rv)
    assert np.array_equal(rk.cpu().numpy()[:n], q4_value(kc, ks).reshape(n, -1).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy()[:n], q4_value(vc, vs).reshape(n, -1).astype(np.float32))
    assert torch.all(rk[n:] == 5.0) and torch.all(rv[n:] == 5.0)
    # q in place
    q2 = dev(q)
    g.kv_append(cache, batch, q2, dev(k), dev(v), dev(freq) if rot else None, halves=halves, q_out=q2)
    assert torch.equal(q2[:n], out[:n]) and torch.equal(q2[n:], dev(q)[n:])
    assert np.array_equal(pages.cpu().numpy(), raw)


def test_append_is_the_sum_of_its_parts(g):
    """A prompt appended at once, in two calls, and token by token: the same bytes."""
    hq, hkv, d, page, n = 4, 2, 64, 16, 37
    rng = np.random.default_rng(1)
    q, k, v = (dev(rng.standard_normal((n, h * d)).astype(np.float32)) for h in (hq, hkv, hkv))
    freq = dev(10000.0 ** (-np.arange(0, d, 2) / d))
    table = dev(np.array([[2, 0, 1]], np.int32))
    got = []
    for cuts in ([n], [20, 17], [1] * n):
        cache = g.KVCache(torch.zeros(3 * hkv * page * 72, dtype=torch.uint8, device="cuda"), page, hkv, d)
        out, at = [], 0
        for m in cuts:
            batch = g.KVBatch(table, dev(np.array([at + m], np.int32)), dev(np.array([0, m], np.int32)), m, 48)
            out.append(g.kv_append(cache, batch, q[at:at + m], k[at:at + m], v[at:at + m], freq))
            at += m
        got.append((torch.cat(out), cache.pages))
    for o, p in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(p, got[0][1])


def test_append_far_position_and_bad_values(g):
    """Position 10^6: the angle keeps its low bits.  A block with a NaN or an infinity reads as NaN,
    its neighbours do not."""
    d, page = 64, 1024
    pos = 10 ** 6
    table = np.full((1, pos // page + 1), -1, np.int32)
    table[0, pos // page] = 0
    freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((1, d)).astype(np.float32) for _ in range(3))
    v[0, 3], v[0, 40] = np.nan, -np.inf
    cache = g.KVCache(None, page, 1, d, n_pages=1)
    batch = g.KVBatch(dev(table), dev(np.array([pos + 1], np.int32)), max_len=pos + 1)
    out = g.kv_append(cache, batch, dev(q), dev(k), dev(v), dev(freq)).cpu().numpy()
    want = rotate(q.reshape(1, 1, d), np.array([pos]), freq, False).reshape(1, d)
    # the angle, about 10^6, is held to 2^-33 at worst (its f64 rounding): 2^-32 on values of about 1
    assert np.all(np.abs(out - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -31)
    _, rv = g.kv_read(cache, batch)
    rv = rv.cpu().numpy()
    assert np.all(np.isnan(rv))  # one block holds the NaN, the other the infinity
    v2 = v.copy()
    v2[0, 40] = 1.0
    g.kv_append(cache, batch, dev(q), dev(k), dev(v2), dev(freq))
    rk, rv = (x.cpu().numpy() for x in g.kv_read(cache, batch))
    assert np.all(np.isnan(rv[0, :32])) and np.all(np.isfinite(rv[0, 32:])) and np.all(np.isfinite(rk))


def test_untrusted_tables(g):
    """Pages out of range, lengths of zero, below zero and beyond the table, runs of rows outside the
    call: nothing else is touched, and what is named is right."""
    hq, hkv, d, page = 2, 1, 64, 16
    rng = np.random.default_rng(4)
    size = 2 * page * 72
    pages = torch.full((size,), 9, dtype=torch.uint8, device="cuda")
    cache = g.KVCache(pages, page, hkv, d)
    table = np.array([[0, 1], [2, -1], [1 << 30, 5], [-(1 << 31), 1]], np.int32)
    q, k, v = (dev(rng.standard_normal((4, h * d)).astype(np.float32)) for h in (hq, hkv, hkv))
    freq = dev(10000.0 ** (-np.arange(0, d, 2) / d))
    out = torch.full((4, hq * d), 3.0, device="cuda")
    for lens in ([0, 5, 5, 5], [-3, 17, 30, 2], [-(1 << 31), 1, 16, 16]):
        batch = g.KVBatch(dev(table), dev(np.array(lens, np.int32)), max_len=32)
        g.kv_append(cache, batch, q, k, v, freq, q_out=out)
        assert torch.all(pages == 9)
        assert torch.all(out[0] == 3.0)  # no position
        rk = torch.full((4, hkv * d), 4.0, device="cuda")
        g.kv_read(cache, batch, rk, rk.clone())
        assert torch.all(rk == 4.0)
        o = g.kv_attention(cache, batch, q, 0.125)
        assert torch.all(o == 0.0)  # rows that see no position
    # lengths beyond max_len are cut to it: the row stands at position 31, in page 1
    batch = g.KVBatch(dev(table), dev(np.array([2 ** 31 - 1, 0, 0, 0], np.int32)), max_len=32)
    g.kv_append(cache, batch, q, k, v, freq, q_out=out)
    assert torch.all(pages[:page * 72] == 9) and not torch.all(pages == 9)
    # runs of rows outside the call, and not in order
    for starts in ([0, 5, 6, 7, 8], [-1, 2, 3, 4, 4], [4, 3, 2, 1, 0], [0, 2 ** 31 - 1, -(2 ** 31), 0, 0],
                   [9, 9, 9, 9, 9]):
        batch = g.KVBatch(dev(table), dev(np.array([9, 9, 9, 9], np.int32)), dev(np.array(starts, np.int32)), 4, 32)
        g.kv_append(cache, batch, q, k, v, freq, q_out=out)
        g.kv_read(cache, batch, rk, rk.clone())
        g.kv_attention(cache, batch, q, 0.125, out=out)
    torch.cuda.synchronize()


def test_streams_and_capture(g):
    """append + attention captured once; lengths, tables and inputs change between the replays."""
    B, hq, hkv, d, page = 3, 4, 2, 64, 16
    rng = np.random.default_rng(6)
    freq = dev(10000.0 ** (-np.arange(0, d, 2) / d))
    table = dev(rng.permutation(B * 40).reshape(B, 40).astype(np.int32))
    lens = dev(np.ones(B, np.int32))
    q, k, v = (torch.zeros(B, h * d, device="cuda") for h in (hq, hkv, hkv))
    cache = g.KVCache(torch.zeros(B * 40 * hkv * page * 72, dtype=torch.uint8, device="cuda"), page, hkv, d)
    other = g.KVCache(torch.zeros_like(cache.pages), page, hkv, d)
    batch = g.KVBatch(table, lens, max_len=640)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    work = torch.empty(max(16, g.qmv_kv_attention_bytes(B, B, hq, hkv, d, 640)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.kv_append(cache, batch, q, k, v, freq, q_out=qr)
        g.kv_attention(cache, batch, qr, 0.125, out=out, work=work)
    cache.pages.zero_()
    side = torch.cuda.Stream()
    for step in range(30):
        lens.copy_(dev(np.array([step + 1, 600 + step, 0 if step % 3 else 20 + step], np.int32)))
        for t in (q, k, v):
            t.copy_(dev(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
        work.fill_(255)
        graph.replay()
        if step % 5 == 0:
            torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        qs = g.kv_append(other, batch, q, k, v, freq, stream=side)
        o = g.kv_attention(other, batch, qs, 0.125, stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(cache.pages, other.pages)
        assert torch.equal(out, o), step


# ------------------------------------------------------------- attention --

def filled(c, hq, dscale=1.0):
    """Random pages in both forms: raw bytes, and per sequence K, V f64 [L, hkv, d]."""
    rng = c.rng
    cells = np.empty((c.n_pages, c.hkv, c.head_bytes), np.uint8)
    ks, vs = (np.empty((c.n_pages, c.hkv, c.page, c.d)) for _ in range(2))
    for i in range(c.n_pages):
        for h in range(c.hkv):
            kc, kd = q4_0(rng.standard_normal((c.page, c.d)).astype(np.float32))
            vc, vd = q4_0((dscale * rng.standard_normal((c.page, c.d))).astype(np.float32))
            cells[i, h] = encode_page(kc, kd, vc, vd, c.page, c.nb)
            ks[i, h], vs[i, h] = q4_value(kc, kd), q4_value(vc, vd)

    def of(x, b):
        m = -(-c.lens[b] // c.page)
        t = x[c.table[b, :m]].transpose(0, 2, 1, 3).reshape(m * c.page, c.hkv, c.d)
        return t[:c.lens[b]]

    return cells.reshape(-1), [of(ks, b) for b in range(c.B)], [of(vs, b) for b in range(c.B)]


def bound(d, length, amax, pv, pmax):
    """How far an f32 computation may be off.  A score is a sum of d products: each product and each
    of at most d + 8 roundings (scaling and splitting q, the block scales, the sums) is off by half a
    step of a magnitude below sum |q k| scale (amax, natural units), and exp adds 2^-22; both enter
    every weight and their sum.  The weighted sums run over partial sums of at most 64 terms and
    the runs of 512 keys; each is off by half a step of sum p |v|.
    Weights times block scales are split into two f16 numbers in a unit where the largest such term
    of a run, p max_b |d| = p max |v| / 8, is 2^13 at least: one of them is off by at most half of
    f16's smallest step, 2^-25, that is 2^-38 of that largest term, and meets codes of at most 8, so
    each key adds at most 2^-38 max_t (p max |v|) (a weight of e^-69 beside one of 1 is lost so)."""
    delta = (d + 8) * 2.0 ** -24 * amax[..., None] + 2.0 ** -21
    floor = length * 2.0 ** -38 * pmax[..., None]
    return (2 * delta + (80 + length / 512) * 2.0 ** -24) * pv + floor


ATTNS = [
    # lens, rows of each, page, q heads, kv heads, d, window
    ([1], [1], 16, 1, 1, 32, 0),
    ([500], [1], 64, 14, 2, 64, 0),
    ([129, 1, 128, 0, 511, 513, 1030], [1] * 7, 16, 8, 2, 128, 0),
    ([700, 30], [1, 1], 32, 16, 1, 96, 100),
    ([300], [1], 256, 20, 1, 128, 0),           # more query heads than one tile of rows
    ([600], [1], 16, 33, 1, 64, 0),
    ([130, 260], [1, 1], 64, 4, 2, 256, 0),
    ([100], [1], 16, 3, 3, 160, 7),
    ([70, 140], [1, 1], 16, 2, 1, 224, 0),
    ([530], [1], 32, 7, 1, 192, 0),
    ([65], [65], 16, 2, 2, 64, 0),              # a whole prompt
    ([200, 17, 5, 600], [37, 0, 5, 100], 16, 6, 2, 64, 0),
    ([540], [530], 64, 5, 1, 128, 60),
    ([40, 33], [33, 33], 16, 3, 1, 32, 1),      # a window of the row's own position
    ([3], [7], 16, 4, 2, 64, 0),                # more rows than tokens: the first see nothing
    ([90], [50], 32, 1, 1, 256, 40),
]


@pytest.mark.parametrize("lens,ns,page,hq,hkv,d,window", ATTNS)
def test_attention(g, lens, ns, page, hq, hkv, d, window):
    print("attention", lens, ns, page, hq, hkv, d, window, flush=True)
    c = Case(lens, ns, page, hkv, d, 11, spare_rows=0 if ns == [1] * len(ns) else 2)
    raw, ks, vs = filled(c, hq)
    q = (1.5 * c.rng.standard_normal((c.T, hq * d))).astype(np.float32)
    scale = 1 / np.sqrt(d)
    cache = g.KVCache(dev(raw), page, hkv, d)
    one = ns == [1] * len(ns)
    out = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_attention(cache, c.batch(g, starts=not one), dev(q), scale, window=window, out=out)
    got = out.cpu().numpy()
    assert np.all(got[c.rows:] == 7.0)
    check(c, got, q, ks, vs, hq, float(np.float32(scale)), window)
    if one:  # the same rows named by starts
        assert torch.equal(g.kv_attention(cache, c.batch(g), dev(q), scale, window=window), out)


def check(c, got, q, ks, vs, hq, scale, window, seen=None):
    for b in range(c.B):
        lo, hi = c.starts[b], c.starts[b + 1]
        if lo == hi:
            continue
        pos = np.arange(c.lens[b] - c.ns[b], c.lens[b])
        want, *sizes = attention(q[lo:hi].reshape(hi - lo, hq, c.d), ks[b], vs[b], pos, scale, window,
                                   None if seen is None else seen[b])
        x = got[lo:hi].reshape(hi - lo, hq, c.d)
        assert np.all(x[pos < 0] == 0)
        lim = bound(c.d, c.lens[b], *sizes)
        assert np.all(np.abs(x - want) <= lim), (b, np.max(np.abs(x - want) - lim))


@pytest.mark.parametrize("dscale", [1e-6, 1e-3, 1.0, 1e3, 6e4])
def test_value_scales(g, dscale):
    """Values of any size that fp16 scales hold keep their relative accuracy."""
    c = Case([300, 40], [1, 1], 16, 2, 64, 12)
    raw, ks, vs = filled(c, 4, dscale)
    # and tokens with much larger or smaller values than their neighbours
    q = (3 * c.rng.standard_normal((c.T, 4 * 64))).astype(np.float32)
    got = g.kv_attention(g.KVCache(dev(raw), 16, 2, 64), c.batch(g), dev(q), 0.125).cpu().numpy()
    check(c, got, q, ks, vs, 4, 0.125, 0)


def test_masked_places_may_hold_anything(g):
    """NaN and infinite scales behind the last token, in tokens a row does not see, and in pages that
    the table does not name; a page out of range is not seen."""
    hq, hkv, d, page = 4, 2, 64, 16
    c = Case([150, 40], [30, 40], page, hkv, d, 13)
    raw, ks, vs = filled(c, hq)
    q = c.rng.standard_normal((c.T, hq * d)).astype(np.float32)
    cells = c.cells(raw.copy())
    half = page * 32 * c.nb

    def spoil(b, p, bits):
        cell = cells[c.table[b, p // page]]
        for part in range(2):
            at = half + part * page * 2 * c.nb + (p % page) * 2 * c.nb
            cell[:, at:at + 2 * c.nb] = np.array([bits] * c.nb, np.uint16).view(np.uint8)

    for p in range(150, 160):
        spoil(0, p, 0x7E00)
    for p in range(40, 48):
        spoil(1, p, 0x7C00)
    cells[c.spare] = 0xFF
    cache = g.KVCache(dev(cells.reshape(-1)), page, hkv, d)
    got = g.kv_attention(cache, c.batch(g), dev(q), 0.125).cpu().numpy()
    check(c, got, q, ks, vs, hq, 0.125, 0)
    # a NaN token spoils the rows that see it and no other
    spoil(1, 20, 0x7E00)
    cache = g.KVCache(dev(cells.reshape(-1)), page, hkv, d)
    o = g.kv_attention(cache, c.batch(g), dev(q), 0.125).cpu().numpy()
    assert np.array_equal(o[:50], got[:50]) and np.all(np.isnan(o[50:]))
    o = g.kv_attention(cache, c.batch(g), dev(q), 0.125, window=5).cpu().numpy()
    assert np.all(np.isfinite(o[:50])) and np.all(np.isnan(o[50:55])) and np.all(np.isfinite(o[55:]))
    # a hole in the table
    c.table[0, 3] = 1 << 20
    c.table[1, 1] = -1
    got = g.kv_attention(cache, c.batch(g), dev(q), 0.125).cpu().numpy()
    seen = [np.ones(150, bool), np.ones(40, bool)]
    seen[0][48:64] = False
    seen[1][16:32] = False
    check(c, got, q, ks, vs, hq, 0.125, 0, seen)


def test_extreme_scores(g):
    """Scores of hundreds, one key that takes all the weight, and rows of zeros (every weight equal)."""
    c = Case([200], [4], 16, 1, 64, 14)
    raw, ks, vs = filled(c, 2)
    q = c.rng.standard_normal((c.T, 128)).astype(np.float32)
    q[0] *= 300
    q[1] = 0
    q[2] *= np.float32(1e-20)
    q[3, :64] *= np.float32(1e4)
    got = g.kv_attention(g.KVCache(dev(raw), 16, 1, 64), c.batch(g), dev(q), 1.0).cpu().numpy()
    check(c, got, q, ks, vs, 2, 1.0, 0)


def test_shared_pages_and_offsets(g):
    """Two sequences that share their first pages, and pages whose bytes lie beyond 2^32."""
    hkv, d, page, hq = 8, 256, 1024, 8
    one = hkv * page * 36 * 8
    n_pages = (1 << 32) // one + 3
    pages = torch.zeros(n_pages * one, dtype=torch.uint8, device="cuda")
    c = Case([1100, 1030], [1, 1], page, hkv, d, 15, spare_pages=0)
    raw, ks, vs = filled(c, hq)
    last = n_pages - 1
    cells = c.cells(raw)
    table = np.zeros((2, 2), np.int32)
    for i, (b, j) in enumerate([(0, 0), (0, 1), (1, 1)]):
        to = last - i
        pages[to * one:(to + 1) * one] = dev(cells[c.table[b, j]].reshape(-1))
        table[b, j] = to
    table[1, 0] = table[0, 0]
    ks[1][:1024], vs[1][:1024] = ks[0][:1024], vs[0][:1024]
    q = c.rng.standard_normal((2, hq * d)).astype(np.float32)
    cache = g.KVCache(pages, page, hkv, d)
    batch = g.KVBatch(dev(table), dev(np.array(c.lens, np.int32)), max_len=1100)
    got = g.kv_attention(cache, batch, dev(q), 0.0625).cpu().numpy()
    check(c, got, q, ks, vs, hq, 0.0625, 0)
    # an append there
    k, v = (c.rng.standard_normal((2, hkv * d)).astype(np.float32) for _ in range(2))
    g.kv_append(cache, batch, dev(q), dev(k), dev(v))
    rk, rv = g.kv_read(cache, batch)
    assert np.array_equal(rk.cpu().numpy(), q4_value(*q4_0(k)).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), q4_value(*q4_0(v)).astype(np.float32))


@pytest.mark.parametrize("d,hq,hkv,window", [(32, 4, 2, 0), (64, 7, 1, 0), (96, 3, 3, 600), (128, 8, 2, 0),
                                             (128, 40, 2, 90), (160, 4, 4, 0), (192, 4, 1, 0),
                                             (224, 2, 2, 700), (256, 4, 2, 0)])
def test_a_row_does_not_depend_on_its_call(g, d, hq, hkv, window):
    """The same token's row, bit for bit: in a prompt at once, in chunks, alone, beside other
    sequences, with a larger bound of the lengths (another split of the work)."""
    L, n, page = 1100, 37, 16
    c = Case([L, 50, 333], [n, 50, 1], page, hkv, d, 17)
    raw, _, _ = filled(c, hq)
    q = dev((1.5 * c.rng.standard_normal((c.T, hq * d))).astype(np.float32))
    cache, table = g.KVCache(dev(raw), page, hkv, d), dev(c.table)

    def call(q, seqs, lens, ns=None, max_len=None):
        starts = None if ns is None else dev(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32))
        batch = g.KVBatch(table[seqs].contiguous(), dev(np.array(lens, np.int32)), starts,
                          None if ns is None else sum(ns), max_len or max(lens))
        return g.kv_attention(cache, batch, q.contiguous(), d ** -0.5, window=window)

    whole = call(q, [0, 1, 2], [L, 50, 333], [n, 50, 1])
    assert torch.equal(call(q[:n], [0], [L], [n]), whole[:n])
    assert torch.equal(call(q[:n], [0], [L], [n], max_len=c.table.shape[1] * page), whole[:n])
    assert torch.equal(call(q[5:20], [0], [L - n + 20], [15]), whole[5:20])
    rows = [0, 1, 12, n - 1]
    alone = torch.cat([call(q[j:j + 1], [0], [L - n + j + 1]) for j in rows])
    assert torch.equal(alone, whole[rows])
    # as one decode batch of many lengths of the same pages, enough of them to need no split
    js = list(range(n)) * 20
    many = call(q[js], [0] * len(js), [L - n + j + 1 for j in js])
    assert torch.equal(many.view(20, n, -1), whole[:n].expand(20, n, -1))
    assert torch.equal(call(q[n:n + 50], [1], [50], [50]), whole[n:n + 50])
    assert torch.equal(call(q[n + 50:], [2], [333]), whole[n + 50:])


@pytest.mark.parametrize("d,hq,hkv,window", [(32, 64, 64, 0), (64, 64, 32, 0), (96, 64, 32, 200), (128, 64, 32, 0),
                                             (128, 120, 24, 333)])
def test_many_rows(g, d, hq, hkv, window):
    """Prompts long enough for 64 rows a workgroup, ragged, with a hole in the table and a NaN token:
    sampled rows against the definition, and every row bit for bit as in a call of few rows."""
    page = 32
    c = Case([700, 129, 128, 40], [450, 128, 0, 5], page, hkv, d, 18, spare_rows=3)
    raw, ks, vs = filled(c, hq)
    c.table[0, 5] = -1  # positions 160..191
    seen = [np.ones(n, bool) for n in c.lens]
    seen[0][160:192] = False
    q = (1.5 * c.rng.standard_normal((c.T, hq * d))).astype(np.float32)
    cache, scale = g.KVCache(dev(raw), page, hkv, d), float(np.float32(d ** -0.5))
    out = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_attention(cache, c.batch(g), dev(q), scale, window=window, out=out)
    assert torch.all(out[c.rows:] == 7.0)
    got, G = out.cpu().numpy(), hq // hkv
    for i in c.rng.choice(c.rows, 24, replace=False):
        b, heads = int(c.seq[i]), np.sort(c.rng.choice(hq, 3, replace=False))
        kv = heads // G
        want, *sizes = attention(q[i].reshape(1, hq, d)[:, heads], ks[b][:, kv], vs[b][:, kv], c.pos[i:i + 1],
                                 scale, window, seen[b])
        x = got[i].reshape(1, hq, d)[:, heads]
        assert np.all(np.abs(x - want) <= bound(d, c.lens[b], *sizes)), i
    table = dev(c.table)

    def few(lo, hi, b, length):
        batch = g.KVBatch(table[b:b + 1].contiguous(), dev(np.array([length], np.int32)),
                          dev(np.array([0, hi - lo], np.int32)), hi - lo, length)
        return g.kv_attention(cache, batch, dev(q[lo:hi]), scale, window=window)

    for lo, hi in [(0, 1), (1, 8), (8, 40), (40, 99), (200, 231), (440, 450)]:
        assert torch.equal(few(lo, hi, 0, 700 - 450 + hi), out[lo:hi]), (lo, hi)
    assert torch.equal(few(450, 500, 1, 51), out[450:500])
    assert torch.equal(few(578, 583, 3, 40), out[578:583])


def test_many_rows_see_nan_where_it_is(g):
    """A NaN token in the middle of a long prompt: the rows before it and, with a window, those far
    behind it are as without it."""
    d, h, page, n = 64, 64, 64, 600
    c = Case([n], [n], page, h, d, 19)
    raw, _, _ = filled(c, h)
    q = dev((c.rng.standard_normal((n, h * d))).astype(np.float32))
    clean = g.kv_attention(g.KVCache(dev(raw), page, h, d), c.batch(g), q, 0.125, window=100)
    cells = c.cells(raw)
    at = page * 34 * c.nb + (300 % page) * 2 * c.nb
    cells[c.table[0, 300 // page], :, at:at + 2 * c.nb] = np.array([0x7E00] * c.nb, np.uint16).view(np.uint8)
    got = g.kv_attention(g.KVCache(dev(raw), page, h, d), c.batch(g), q, 0.125, window=100)
    assert torch.equal(got[:300], clean[:300]) and torch.equal(got[400:], clean[400:])
    assert torch.all(torch.isnan(got[300:400]))


@pytest.mark.parametrize("d,rot,halves,extra", [(64, 64, False, 1), (64, 64, True, 3), (96, 24, True, 4), (128, 72, True, 2),
                                                (256, 6, False, 1), (32, 32, True, 1)])
def test_append_rows_of_any_alignment(g, d, rot, halves, extra):
    """Rows that start anywhere (no 16-byte loads) and rotations that end inside eight elements."""
    hq, hkv, page, n = 6, 3, 16, 21
    c = Case([n + 4], [n], page, hkv, d, 21)
    width = (hq + 2 * hkv) * d + extra
    both = dev(c.rng.standard_normal((n, width)).astype(np.float32))
    q, k, v = both[:, :hq * d], both[:, hq * d:(hq + hkv) * d], both[:, (hq + hkv) * d:(hq + 2 * hkv) * d]
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    cache = g.KVCache(None, page, hkv, d, n_pages=c.n_pages)
    out = g.kv_append(cache, c.batch(g), q, k, v, dev(freq), halves=halves)
    rk, rv = (x.cpu().numpy().reshape(n, hkv, d) for x in g.kv_read(cache, c.batch(g)))
    q64, k64 = (rotate(x.cpu().numpy().reshape(n, -1, d), c.pos, freq, halves) for x in (q, k))
    # one rounding to f32 of sums of two f64 products of values below 8
    assert np.all(np.abs(out.cpu().numpy().reshape(q64.shape) - q64) <= 2.0 ** -24 * np.abs(q64) + 2.0 ** -47)
    assert np.array_equal(rk, q4_value(*q4_0(k64.astype(np.float32))).astype(np.float32))
    assert np.array_equal(rv, q4_value(*q4_0(v.cpu().numpy().reshape(n, hkv, d))).astype(np.float32))


@pytest.mark.parametrize("halves", [False, True])
def test_append_in_place_of_many_rows(g, halves):
    """Rows enough for a workgroup to take all heads of one, with q rotated where it stands: as in
    calls of few rows into another tensor."""
    hq, hkv, d, page, n = 32, 8, 128, 64, 700
    rng = np.random.default_rng(22)
    q, k, v = (dev(rng.standard_normal((n, h * d)).astype(np.float32)) for h in (hq, hkv, hkv))
    freq, table = dev(10000.0 ** (-np.arange(0, d, 2) / d)), dev(rng.permutation(11).reshape(1, 11).astype(np.int32))
    few = g.KVCache(torch.zeros(11 * hkv * page * 144, dtype=torch.uint8, device="cuda"), page, hkv, d)
    many = g.KVCache(torch.zeros_like(few.pages), page, hkv, d)

    def batch(lo, hi):
        return g.KVBatch(table, dev(np.array([hi], np.int32)), dev(np.array([0, hi - lo], np.int32)), hi - lo, 704)

    parts = [g.kv_append(few, batch(i, i + 100), q[i:i + 100], k[i:i + 100], v[i:i + 100], freq, halves=halves)
             for i in range(0, n, 100)]
    assert g.kv_append(many, batch(0, n), q, k, v, freq, halves=halves, q_out=q) is q
    assert torch.equal(q, torch.cat(parts)) and torch.equal(few.pages, many.pages)


def test_many_sequences(g):
    """More sequences than a wave looks at a time, some without rows, in one call: each as alone;
    q as a part of wider rows."""
    hq, hkv, d, page, B = 6, 2, 64, 16, 200
    rng = np.random.default_rng(23)
    ns = [int(x) for x in rng.choice([0, 1, 1, 2, 5, 19], B)]
    lens = [n + int(x) for n, x in zip(ns, rng.choice([0, 3, 15, 40, 530], B))]
    c = Case(lens, ns, page, hkv, d, 24, spare_rows=2)
    raw, ks, vs = filled(c, hq)
    wide = dev((1.5 * c.rng.standard_normal((c.T, hq * d + 8))).astype(np.float32))
    q = wide[:, 4:4 + hq * d]
    cache = g.KVCache(dev(raw), page, hkv, d)
    out = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_attention(cache, c.batch(g), q, 0.125, out=out)
    assert torch.all(out[c.rows:] == 7.0)
    check(c, out.cpu().numpy(), q.cpu().numpy(), ks, vs, hq, 0.125, 0)
    k, v = (dev(c.rng.standard_normal((c.T, hkv * d)).astype(np.float32)) for _ in range(2))
    qr = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_append(cache, c.batch(g), q, k, v, q_out=qr)
    assert torch.equal(qr[:c.rows], q[:c.rows]) and torch.all(qr[c.rows:] == 7.0)
    rk, rv = g.kv_read(cache, c.batch(g))
    assert np.array_equal(rk[:c.rows].cpu().numpy(), q4_value(*q4_0(k[:c.rows].cpu().numpy())).astype(np.float32))
    assert np.array_equal(rv[:c.rows].cpu().numpy(), q4_value(*q4_0(v[:c.rows].cpu().numpy())).astype(np.float32))


def test_capture_of_a_long_prompt(g):
    """64 rows a workgroup, captured; tables and starts change between the replays, and two calls run
    at once on two streams, each with a workspace of its own."""
    h, d, page, n = 64, 64, 32, 512
    c = Case([n, n], [n, n], page, h, d, 25)
    raw, _, _ = filled(c, h)
    cache = g.KVCache(dev(raw), page, h, d)
    q = dev(c.rng.standard_normal((c.T, h * d)).astype(np.float32))
    table, lens, starts = dev(c.table), dev(np.array(c.lens, np.int32)), dev(c.starts)
    batch = g.KVBatch(table, lens, starts, c.T, n)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.kv_attention(cache, batch, q, 0.125, out=out)
    one = g.KVBatch(table[:1].contiguous(), lens[:1].contiguous(), max_len=n)
    side = torch.cuda.Stream()
    for step in range(6):
        starts.copy_(dev(np.array([0, 512 - 70 * step, 1024 - 100 * step], np.int32)))
        lens.copy_(dev(np.array([512 - step, 512], np.int32)))
        out.fill_(7.0)
        want = torch.full_like(q, 7.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        g.kv_attention(cache, batch, q, 0.125, out=want, stream=side)
        with torch.cuda.stream(side):
            again = g.kv_attention(cache, one, q[:1].contiguous(), 0.125)
        torch.cuda.current_stream().wait_stream(side)
        if step % 2:
            torch.cuda.synchronize()
        assert torch.equal(out, want), step
        assert torch.equal(again, g.kv_attention(cache, one, q[:1].contiguous(), 0.125)), step


@pytest.mark.parametrize("d,hq,hkv,n,where", [(64, 4, 2, 5, "k"), (128, 16, 1, 40, "k"), (64, 64, 64, 1000, "k"),
                                              (64, 4, 2, 5, "v"), (128, 16, 1, 40, "v"), (160, 2, 2, 40, "k")])
@pytest.mark.parametrize("bits", [0x7C00, 0xFC00, 0x7E00])
def test_a_scale_that_is_not_finite(g, d, hq, hkv, n, where, bits):
    """An infinite or NaN scale of one block of one token: the rows that see it are NaN throughout, the
    others as without it."""
    page, at = 32, n - 3
    c = Case([n + 70], [n], page, hkv, d, 26)
    raw, _, _ = filled(c, hq)
    q = dev(c.rng.standard_normal((n, hq * d)).astype(np.float32))
    clean = g.kv_attention(g.KVCache(dev(raw), page, hkv, d), c.batch(g), q, 0.125)
    cells, p = c.cells(raw), 70 + at
    byte = page * (32 if where == "k" else 34) * c.nb + ((p % page) * c.nb + c.nb - 1) * 2
    cells[c.table[0, p // page], :, byte:byte + 2] = np.array([bits], np.uint16).view(np.uint8)
    got = g.kv_attention(g.KVCache(dev(raw), page, hkv, d), c.batch(g), q, 0.125)
    assert torch.equal(got[:at], clean[:at])
    assert torch.all(torch.isnan(got[at:]))
