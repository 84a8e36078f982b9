"""The attention's kernels each for itself, at shapes of which the library says
which kernel they run."""
import numpy as np
import pytest

from step_ref import attention
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
