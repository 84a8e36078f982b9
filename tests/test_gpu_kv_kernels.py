"""The attention's kernels each for itself, at shapes of which the library says
which kernel they run."""
import numpy as np
import pytest

from step_ref import attention, encode_page, q4_0, q4_value
from test_gpu_kv import Case, bound, dev, filled

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


def sampled(c, got, q, ks, vs, hq, scale, window, seen, rows, heads=3):
    """`rows` rows of the call, `heads` heads of each, against the definition."""
    G = hq // c.hkv
    for i in c.rng.choice(c.rows, min(rows, c.rows), replace=False):
        b, h = int(c.seq[i]), np.sort(c.rng.choice(hq, min(heads, hq), replace=False))
        want, *sizes = attention(q[i].reshape(1, hq, c.d)[:, h], ks[b][:, h // G], vs[b][:, h // G], c.pos[i:i + 1],
                                 scale, window, seen[b])
        x = got[i].reshape(1, hq, c.d)[:, h]
        assert np.all(np.abs(x - want) <= bound(c.d, c.lens[b], *sizes)), i


@pytest.mark.parametrize("d,hq,hkv,window", [(32, 128, 128, 0), (32, 192, 64, 150), (64, 128, 64, 0), (64, 128, 128, 77),
                                             (96, 192, 64, 200), (96, 128, 128, 0), (128, 120, 24, 0),
                                             (128, 80, 80, 600)])
def test_64_rows_a_workgroup(g, d, hq, hkv, window):
    """Ragged prompts with a hole in the table, at every head size of the kernel: sampled rows against
    the definition, every row bit for bit as in calls that run the other kernels, and with a NaN value
    scale as without it wherever the token is not seen."""
    print("64 rows", d, hq, hkv, window, flush=True)
    page, lens, ns = 32, [700, 129, 128, 40], [450, 128, 0, 5]
    c = Case(lens, ns, page, hkv, d, 31, spare_rows=3)
    raw, ks, vs = filled(c, hq)
    c.table[0, 5] = -1  # positions 160..191
    seen = [np.ones(n, bool) for n in lens]
    seen[0][160:192] = False
    q = (1.5 * c.rng.standard_normal((c.T, hq * d))).astype(np.float32)
    cache, scale = g.KVCache(dev(raw), page, hkv, d), float(np.float32(d ** -0.5))
    assert g.qmv_kv_attention_rows(c.T, c.B, True, hq, hkv, d, 700) == 64
    out = torch.full((c.T, hq * d), 7.0, device="cuda")
    g.kv_attention(cache, c.batch(g), dev(q), scale, window=window, out=out)
    assert torch.all(out[c.rows:] == 7.0)
    sampled(c, out.cpu().numpy(), q, ks, vs, hq, scale, window, seen, 24)
    table = dev(c.table)

    def few(lo, hi, b, length):
        assert g.qmv_kv_attention_rows(hi - lo, 1, True, hq, hkv, d, length) != 64
        batch = g.KVBatch(table[b:b + 1].contiguous(), dev(np.array([length], np.int32)),
                          dev(np.array([0, hi - lo], np.int32)), hi - lo, length)
        return g.kv_attention(cache, batch, dev(q[lo:hi]), scale, window=window)

    for lo in range(0, 450, 50):
        assert torch.equal(few(lo, lo + 50, 0, 250 + lo + 50), out[lo:lo + 50]), lo
    for lo in range(450, 578, 32):
        assert torch.equal(few(lo, lo + 32, 1, 1 + lo + 32 - 450), out[lo:lo + 32]), lo
    assert torch.equal(few(578, 583, 3, 40), out[578:583])
    # a NaN token: position 400 of the first sequence, whose rows are positions 250 ...
    cells = c.cells(raw.copy())
    at = page * 34 * c.nb + (400 % page) * 2 * c.nb
    cells[c.table[0, 400 // page], :, at:at + 2 * c.nb] = np.array([0x7E00] * c.nb, np.uint16).view(np.uint8)
    got = g.kv_attention(g.KVCache(dev(cells.reshape(-1)), page, hkv, d), c.batch(g), dev(q), scale, window=window)
    sees = (c.pos >= 400) & (c.seq == 0)
    if window:
        sees &= c.pos < 400 + window
    sees = torch.from_numpy(sees).cuda()
    assert torch.all(torch.isnan(got[:c.rows][sees])) and torch.equal(got[:c.rows][~sees], out[:c.rows][~sees])


# a shape of every kernel: lens, rows of each, page, q heads, kv heads, d, rows a workgroup, split over positions
KERNELS = [
    ([200], [1], 16, 4, 1, 64, 8, False),
    ([2000], [1], 16, 4, 1, 128, 8, True),
    ([90], [25], 16, 2, 1, 96, 16, False),
    ([900], [3], 16, 16, 1, 32, 16, True),
    ([200], [3], 32, 3, 1, 160, 16, False),
    ([700], [2], 32, 2, 2, 256, 16, True),
    ([530], [512], 64, 128, 128, 64, 64, False),
]


def shaped(g, kernel, seed):
    """The Case of a shape, whose kernel and split are as it says."""
    lens, ns, page, hq, hkv, d, rows, split = kernel
    print(kernel, flush=True)
    assert g.qmv_kv_attention_rows(sum(ns), len(ns), True, hq, hkv, d, max(lens)) == rows
    assert (g.qmv_kv_attention_bytes(sum(ns), len(ns), hq, hkv, d, max(lens)) > 16) == split
    return Case(lens, ns, page, hkv, d, seed), page, hq, hkv, d


def built(c, kc, kd, vc, vd):
    """The pages of one sequence's tokens [L, hkv, nb, 32] and scales [L, hkv, nb]; -> raw, K, V."""
    cells = np.zeros((c.n_pages, c.hkv, c.head_bytes), np.uint8)
    L = c.lens[0]
    for j in range(-(-L // c.page)):
        t = slice(j * c.page, min(L, (j + 1) * c.page))
        pad = [(0, c.page - (t.stop - t.start))]
        for h in range(c.hkv):
            k, v = (np.pad(x[t, h], pad + [(0, 0)] * 2) for x in (kc, vc))
            a, b = (np.pad(x[t, h], pad + [(0, 0)]) for x in (kd, vd))
            cells[c.table[0, j], h] = encode_page(k, a, v, b, c.page, c.nb)
    return cells.reshape(-1), q4_value(kc, kd), q4_value(vc, vd)


# around the places where 14 is no multiple of a score's step, and up to both ends of f32
SIZES = [x * 2.0 ** e for e in range(23, 31) for x in (1.0, 1.13, 1.37, 1.61, 1.89)] + [
    1e12, 1e20, 5e29, 1e30, 3e30, 1e31, 1e34, 4e37]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(g, kernel, sign):
    """Keys all alike but one, which is twice as long: with positive scores it takes all the weight,
    with negative ones it has none and the others share it, however large the scores are.  Every
    weight is then exact, and so is its product with a value, so that only the sums round: partial
    sums of at most 64 terms and runs of 512 keys, each by half a step of sum p |v|."""
    c, page, hq, hkv, d = shaped(g, kernel, 32)
    L, n, twice = c.lens[0], c.ns[0], c.lens[0] // 3
    k, v = c.rng.standard_normal((1, hkv, d)), c.rng.standard_normal((L, hkv, c.nb, 32))
    kc, kd = (np.repeat(x, L, 0) for x in q4_0(k.astype(np.float32)))
    kd[twice] *= 2
    v = v.clip(-2.9, 2.9)
    v[..., 7] = 3.0  # one scale for all
    vc, vd = q4_0(v.reshape(L, hkv, d).astype(np.float32))
    raw, ks, vs = built(c, kc, kd, vc, vd)
    cache, batch = g.KVCache(dev(raw), page, hkv, d), c.batch(g)
    unit = ks[0] / (ks[0] ** 2).sum(-1, keepdims=True)  # [hkv, d]: a score of 1
    per = n * hq
    sizes = np.resize(SIZES, -(-len(SIZES) // per) * per).reshape(-1, n, hq)
    for size in sizes[:3] if per >= len(SIZES) else sizes:
        q = (sign * size[..., None] * np.repeat(unit, hq // hkv, 0)).astype(np.float32)
        got = g.kv_attention(cache, batch, dev(q.reshape(n, -1)), 1.0).cpu().numpy().reshape(n, hq, d)
        for j in range(n):
            seen = np.arange(c.pos[j] + 1)
            seen = seen[seen == twice] if sign > 0 and c.pos[j] >= twice else seen[seen != twice]
            want, mean = vs[seen].mean(0), np.abs(vs[seen]).mean(0)
            lim = np.repeat((80 + L / 512) * 2.0 ** -24 * mean, hq // hkv, 0)
            assert np.all(np.abs(got[j] - np.repeat(want, hq // hkv, 0)) <= lim), (j, size[j])


def block_bound(c, q, ks, vs, hq, scale, got, row, floor, seen=slice(None)):
    """Checks a row (or some of its heads) by its blocks: the f32 computation of `bound`, and `floor`
    of the largest p max |v| of the element's own block a key."""
    heads = np.arange(hq) if hq <= 8 else np.sort(c.rng.choice(hq, 4, replace=False))
    d = c.d
    for h in heads:
        k, v = (y[:c.pos[row] + 1, h * c.hkv // hq][seen] for y in (ks, vs))
        L, x = len(k), q[row, h].astype(np.float64)
        s = k @ x * scale
        p = np.exp(s - s.max())
        p /= p.sum()
        pv = p @ np.abs(v)
        most = (p[:, None] * np.abs(v).reshape(L, c.nb, 32).max(-1)).max(0).repeat(32)
        delta = (d + 8) * 2.0 ** -24 * (np.abs(k) @ np.abs(x)).max() * scale + 2.0 ** -21
        lim = (2 * delta + (80 + L / 512) * 2.0 ** -24) * pv + L * floor * most
        err = np.abs(got[row, h] - p @ v)
        assert np.all(err <= lim), (row, h, (err / np.maximum(lim, 1e-300)).reshape(c.nb, 32).max(-1))


# exponents of a block's scale, relative to the head's largest
STEPS = np.array([0, 0, -1, -3, -6, -7, -8, -9, -14, -20, -25, -30, -33])


def scales_of(c, how, L):
    """Value scales [L, hkv, nb] and, for some, the key that the queries look for."""
    shape = (L, c.hkv, c.nb)
    e, look = np.zeros(shape), None
    if how == "blocks":      # every token alike, a size for each block
        e += STEPS[(5 + 3 * np.arange(c.nb)) % len(STEPS)]
        e[..., 0] = 0
    elif how == "tokens":    # every block of every token for itself, zeros among them
        e = c.rng.choice(np.append(STEPS, -99), shape)
    elif how == "looked at":  # one token takes nearly all the weight, and has a block as small as can be
        look = L // 2
        e[look, :, c.nb - 1] = -33
        e[look + 1, :, c.nb - 1] = -99
    elif how == "nothing":   # a block of zeros in every token, and tokens of zeros
        e[..., c.nb - 1] = -99
        e[::3] = -99
    d = np.where(e == -99, 0.0, np.ldexp(600 * (1 + c.rng.random(shape)), e.astype(int)))
    return (d * c.rng.choice([-1, 1], shape)).astype(np.float16), look


def case_of(g, kernel, how, seed):
    c, page, hq, hkv, d = shaped(g, kernel, seed)
    L, n = c.lens[0], c.ns[0]
    kc, kd = q4_0(c.rng.standard_normal((L, hkv, d)).astype(np.float32))
    vd, look = scales_of(c, how, L)
    vc = c.rng.integers(0, 16, (L, hkv, c.nb, 32))
    vc[..., 3] = 0  # a code of -8 in every block
    q = 2 * c.rng.standard_normal((n, hq, d))
    if look is not None:  # a score of about 40 there
        k = np.repeat(q4_value(kc, kd)[look], hq // hkv, 0)
        q = q * 0.5 + 40 * d ** 0.5 * k / (k ** 2).sum(-1, keepdims=True)
    return c, page, hq, hkv, d, kc, kd, vc, vd, q.astype(np.float32)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("how", ["blocks", "tokens", "looked at", "nothing"])
def test_value_scales_of_a_head_apart(g, kernel, how):
    """Blocks of one head whose scales are far apart: each keeps the accuracy of an f32 computation of
    its own sums.  Where all scales that a row sees in a run are within 2^-8 of the largest of their
    token, weight times scale is held as two f16 numbers in a unit where the run's largest is 2^13 at
    least, and the block's at that token 2^5: the two are off by at most 2^-24 (half of f16's smallest
    step, once for the weight and once for the product), and meet codes of at most 8 as the block's
    own largest does, so a key adds at most 2^-29 of it.  Elsewhere nothing is lost but f32 roundings."""
    c, page, hq, hkv, d, kc, kd, vc, vd, q = case_of(g, kernel, how, 33)
    raw, ks, vs = built(c, kc, kd, vc, vd)
    n, scale = c.ns[0], float(np.float32(d ** -0.5))
    got = g.kv_attention(g.KVCache(dev(raw), page, hkv, d), c.batch(g), dev(q.reshape(n, -1)), scale)
    got = got.cpu().numpy().reshape(n, hq, d)
    for row in range(n) if n < 30 else c.rng.choice(n, 12, replace=False):
        block_bound(c, q, ks, vs, hq, scale, got, row, 2.0 ** -29)


@pytest.mark.parametrize("kernel", [k for k in KERNELS if k[1][0] > 1] + [([400], [160], 32, 8, 2, 128, 16, False)])
def test_scales_apart_change_no_row_that_does_not_see_them(g, kernel):
    """Bit for bit: rows before such a token as without it, and all rows as in calls of one row."""
    c, page, hq, hkv, d, kc, kd, vc, vd, q = case_of(g, kernel, "tokens", 34)
    L, n, scale = c.lens[0], c.ns[0], d ** -0.5
    from_ = L - n // 2
    vd[:from_] = (c.rng.random(vd[:from_].shape) + 1).astype(np.float16)
    plain = vd.copy()
    plain[from_:] = 1
    qd, batch = dev(q.reshape(n, -1)), c.batch(g)
    with_, without = (g.kv_attention(g.KVCache(dev(built(c, kc, kd, vc, x)[0]), page, hkv, d), batch, qd, scale)
                      for x in (vd, plain))
    rows = from_ - (L - n)
    assert torch.equal(with_[:rows], without[:rows])
    assert not torch.equal(with_[rows:], without[rows:])
    cache, table = g.KVCache(dev(built(c, kc, kd, vc, vd)[0]), page, hkv, d), dev(c.table)
    for j in range(n) if n < 30 else c.rng.choice(n, 12, replace=False):
        one = g.KVBatch(table, dev(np.array([L - n + j + 1], np.int32)), max_len=int(L))
        assert torch.equal(g.kv_attention(cache, one, qd[j:j + 1], scale)[0], with_[j]), j


@pytest.mark.parametrize("kernel", KERNELS)
def test_q_that_is_not_finite(g, kernel):
    """A query's head with a NaN or an infinity is NaN throughout, its other heads and the other rows
    are as without it."""
    c, page, hq, hkv, d = shaped(g, kernel, 35)
    n = c.ns[0]
    raw, _, _ = filled(c, hq)
    cache, batch = g.KVCache(dev(raw), page, hkv, d), c.batch(g)
    q = c.rng.standard_normal((n, hq, d)).astype(np.float32)
    clean = g.kv_attention(cache, batch, dev(q.reshape(n, -1)), 0.1).view(n, hq, d)
    spoilt = c.rng.random((n, hq)) < 0.3
    spoilt[0, 0] = True
    for j, h in np.argwhere(spoilt):
        q[j, h, c.rng.integers(d)] = c.rng.choice([np.nan, np.inf, -np.inf])
    got = g.kv_attention(cache, batch, dev(q.reshape(n, -1)), 0.1).view(n, hq, d)
    spoilt = torch.from_numpy(spoilt).cuda()
    assert torch.all(torch.isnan(got[spoilt])) and torch.equal(got[~spoilt], clean[~spoilt])


def test_q_that_is_not_finite_and_sees_nothing(g):
    """More rows than tokens: the first see no position and are 0 whatever they hold."""
    c = Case([3], [7], 16, 2, 64, 36)
    raw, _, _ = filled(c, 4)
    q = dev(np.full((7, 4 * 64), np.nan, np.float32))
    got = g.kv_attention(g.KVCache(dev(raw), 16, 2, 64), c.batch(g), q, 0.125)
    assert torch.all(got[:4] == 0) and torch.all(torch.isnan(got[4:]))


@pytest.mark.parametrize("kernel", KERNELS[:-1])
@pytest.mark.parametrize("apart", [6, 12, 18])
def test_q_of_sizes_apart(g, kernel, apart):
    """The first block of q 2^apart times the others, that of the keys as much smaller.  Two f16
    parts of q in a unit where the head's largest element is 2^14 at least are off by at most half of
    f16's smallest step, 2^-25: 2^-39 of that element, times the sum of the key's sizes."""
    c, page, hq, hkv, d = shaped(g, kernel, 37)
    L, n, scale = c.lens[0], c.ns[0], float(np.float32(d ** -0.5))
    kc, kd = q4_0(c.rng.standard_normal((L, hkv, d)).astype(np.float32))
    kd[..., 0] *= np.float16(2.0 ** -apart)
    vc, vd = q4_0(c.rng.standard_normal((L, hkv, d)).astype(np.float32))
    raw, ks, vs = built(c, kc, kd, vc, vd)
    q = c.rng.standard_normal((n, hq, d)).astype(np.float32)
    q[..., :32] *= np.float32(2.0 ** apart)
    got = g.kv_attention(g.KVCache(dev(raw), page, hkv, d), c.batch(g), dev(q.reshape(n, -1)), scale)
    got = got.cpu().numpy().reshape(n, hq, d)
    want, amax, pv, pmax = attention(q, ks, vs, c.pos, scale)
    size = np.abs(ks).sum(-1).max(0).repeat(hq // hkv)
    lost = 2.0 ** -39 * np.abs(q).max(-1) * size * scale
    assert np.all(np.abs(got - want) <= bound(d, L, amax, pv, pmax) + 2 * lost[..., None] * pv)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window", [0, 60])
def test_value_scales_apart_behind_masks(g, kernel, window):
    """The same with a window, a hole in the table, and scales that are not finite where no row looks:
    against the definition, and bit for bit as alone."""
    c, page, hq, hkv, d, kc, kd, vc, vd, q = case_of(g, kernel, "tokens", 38)
    L, n, scale = c.lens[0], c.ns[0], float(np.float32(d ** -0.5))
    hole = (L - 40) // page  # a page that rows with a window of 60 see
    raw, ks, vs = built(c, kc, kd, vc, vd)
    cells = c.cells(raw)
    cells[c.table[0, hole]] = 0xFF  # NaN scales
    cells[c.spare] = 0xFF
    c.table[0, hole] = -1
    table = dev(c.table)
    cache, qd = g.KVCache(dev(raw), page, hkv, d), dev(q.reshape(n, -1))
    out = g.kv_attention(cache, c.batch(g), qd, scale, window=window)
    got = out.cpu().numpy().reshape(n, hq, d)
    for row in range(n) if n < 30 else c.rng.choice(n, 12, replace=False):
        t = np.arange(c.pos[row] + 1)
        seen = t // page != hole
        if window:
            seen &= t > c.pos[row] - window
        if seen.any():
            block_bound(c, q, ks, vs, hq, scale, got, row, 2.0 ** -29, seen)
        else:
            assert np.all(got[row] == 0)
        one = g.KVBatch(table, dev(np.array([c.pos[row] + 1], np.int32)), max_len=int(L))
        assert torch.equal(g.kv_attention(cache, one, qd[row:row + 1], scale, window=window)[0], out[row]), row
