"""A run of the operators as a llama-family block uses them: norm, q/k/v
products, rotation and append, attention, output product, norm, feed-forward;
a ragged prompt first, then single tokens, eager and captured.  Every stage is
checked against its definition from what the stage before left."""
import numpy as np
import pytest

import oracle
import synth
from checks import assert_bitwise, assert_tol
from step_ref import attention, q4_0, q4_value, rmsnorm, rotate
from test_gpu_kv import bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS, E, F = 1e-5, 256, 512


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Model:
    """Two blocks; weights, cache and buffers of each."""

    def __init__(self, g, fmt, hq, hkv, d, page, n_pages, seed):
        self.g, self.fmt, self.hq, self.hkv, self.d = g, fmt, hq, hkv, d
        rng = np.random.default_rng(seed)
        self.freq = 10000.0 ** (-np.arange(0, d, 2) / d)
        self.freq_d = dev(self.freq)
        self.shapes = dict(q=(hq * d, E), k=(hkv * d, E), v=(hkv * d, E), o=(E, hq * d), gate=(F, E),
                           up=(F, E), down=(E, F))
        self.layers = []
        for layer in range(2):
            w = {n: synth.weights(fmt, *s, seed + 10 * layer + i, dscale=0.02)[0]
                 for i, (n, s) in enumerate(self.shapes.items())}
            norms = [(1 + 0.2 * rng.standard_normal(E)).astype(np.float32) for _ in range(2)]
            pages = torch.full((g.qmv_kv_bytes(n_pages, page, hkv, d),), 255, dtype=torch.uint8, device="cuda")
            self.layers.append(dict(w=w, wd={n: dev(b) for n, b in w.items()}, norms=norms,
                                    normsd=[dev(x) for x in norms], cache=g.KVCache(pages, page, hkv, d)))

    def product(self, layer, names, xq, rows):
        g, wd = self.g, layer["wd"]
        if rows <= 16:
            return g.matvec_group(self.fmt, [dict(w=wd[n], N=self.shapes[n][0], K=self.shapes[n][1], xq=xq,
                                                  B=rows) for n in names])
        return [g.matmul(self.fmt, wd[n], *self.shapes[n], xq=xq, M=rows) for n in names]

    def block(self, layer, x, res, batch, keep, work=None):
        """x (+ res) -> (what the block adds to the stream, the stream)."""
        g, rows = self.g, x.shape[0]
        n = max(g.qmv_act_bytes(rows, E), g.qmv_gateup_act_bytes(rows, F, E))
        y1, y2 = torch.empty_like(x), torch.empty_like(x)
        xq1, xq2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        h1, _ = g.add_rmsnorm(x, layer["normsd"][0], EPS, res=res, y=y1, xq=xq1)
        h1 = x if h1 is None else h1
        q, k, v = self.product(layer, "qkv", xq1, rows)
        qr = g.kv_append(layer["cache"], batch, q, k, v, self.freq_d)
        a = g.kv_attention(layer["cache"], batch, qr, self.d ** -0.5, work=work)
        aq = g.quantize(a)
        o, = self.product(layer, "o", aq, rows)
        h2, _ = g.add_rmsnorm(o, layer["normsd"][1], EPS, res=h1, y=y2, xq=xq2)
        if rows <= 16:
            h, hq = g.gateup_swiglu_q8(self.fmt, layer["wd"]["gate"], layer["wd"]["up"], F, E, xq=xq2, B=rows)
        else:
            gate, up = self.product(layer, ("gate", "up"), xq2, rows)
            h = torch.nn.functional.silu(gate) * up
            hq = g.quantize(h)
        out, = self.product(layer, ("down",), hq, rows)
        if keep is not None:
            keep.append(dict(x=x, res=res, y1=y1, xq1=xq1, h1=h1, q=q, k=k, v=v, qr=qr, a=a, aq=aq, o=o, y2=y2,
                             xq2=xq2, h2=h2, h=h, hq=hq, out=out, kv=g.kv_read(layer["cache"], batch)))
        return out, h2

    def step(self, x, batch, keep=None, work=None):
        a, r = x, None
        for layer in self.layers:
            a, r = self.block(layer, a, r, batch, keep, work)
        return a + r


def check_norm(s, h, y, xq, x, res, w, rows):
    # h: one f32 addition.  y: f64 up to one rounding to f32 (the f64 sums differ in their last bits)
    want_h, y64 = rmsnorm(s[x], w, EPS, None if res is None else s[res])
    assert_bitwise(s[h], want_h, h)
    assert np.all(np.abs(s[y] - y64) <= np.abs(y64) * 2.0 ** -24 * (1 + 2.0 ** -20))
    blocks = oracle.quantize_act(s[y])
    assert_bitwise(s[xq][:blocks.size], blocks, xq)


def check_block(m, layer, dev_stages, starts, lens, held):
    """held: per sequence the K and V values of the tokens so far, extended by this call's."""
    s = {n: (tuple(x.cpu().numpy() for x in t) if isinstance(t, tuple) else None if t is None else t.cpu().numpy())
         for n, t in dev_stages.items()}
    rows, w = s["x"].shape[0], layer["w"]

    def product(name, xq, y):
        N, K = m.shapes[name]
        blocks = s[xq][:oracle.quantize_act(np.zeros((rows, K), np.float32)).size]
        if rows <= 16:
            assert_bitwise(s[y], oracle.matmul_canon_f32(m.fmt, w[name], N, K, blocks, rows), name)
        y64, A = oracle.matmul_f64(m.fmt, w[name], N, K, blocks, rows)
        assert_tol(s[y], y64, A, what=name)

    check_norm(s, "h1", "y1", "xq1", "x", None if s["res"] is None else "res", layer["norms"][0], rows)
    for n in "qkv":
        product(n, "xq1", n)
    pos = np.concatenate([np.arange(lens[b] - (starts[b + 1] - starts[b]), lens[b]) for b in range(len(lens))])
    q64 = rotate(s["q"].reshape(rows, m.hq, m.d), pos, m.freq, False)
    # one rounding to f32 of sums of two f64 products, whose own errors are below 2^-50 |x|
    near = 2.0 ** -24 * np.abs(q64) + 2.0 ** -50 * np.abs(s["q"]).max()
    assert np.all(np.abs(s["qr"].reshape(q64.shape) - q64) <= near)
    k32 = rotate(s["k"].reshape(rows, m.hkv, m.d), pos, m.freq, False).astype(np.float32)
    k, v = (t.reshape(rows, m.hkv, m.d).astype(np.float64) for t in s["kv"])
    assert np.array_equal(k, q4_value(*q4_0(k32)))
    assert np.array_equal(v, q4_value(*q4_0(s["v"].reshape(v.shape))))
    for b in range(len(lens)):
        r = slice(starts[b], starts[b + 1])
        held[b] = [np.concatenate([old, new[r]]) for old, new in zip(held[b], (k, v))]
        assert len(held[b][0]) == lens[b]
        want, *sizes = attention(s["qr"][r].reshape(-1, m.hq, m.d), *held[b], pos[r], float(np.float32(m.d ** -0.5)))
        err = np.abs(s["a"][r].reshape(want.shape) - want)
        assert np.all(err <= bound(m.d, lens[b], *sizes)), b
    blocks = oracle.quantize_act(s["a"])
    assert_bitwise(s["aq"][:blocks.size], blocks, "aq")
    product("o", "aq", "o")
    check_norm(s, "h2", "y2", "xq2", "o", "h1", layer["norms"][1], rows)
    product("down", "hq", "out")
    if rows <= 16:
        x2 = oracle.quantize_act(s["y2"])
        gate, up = (oracle.matmul_canon_f32(m.fmt, w[n], F, E, x2, rows) for n in ("gate", "up"))
        assert_bitwise(s["h"], oracle.swiglu(gate, up), "h")


@pytest.mark.parametrize("fmt,hq,hkv,d,page", [(synth.Q4_K, 4, 2, 64, 16), (synth.Q8_0, 6, 1, 128, 32)])
def test_prompt_then_tokens(g, fmt, hq, hkv, d, page):
    print("step", fmt, hq, hkv, d, page, flush=True)
    rng = np.random.default_rng(8)
    lens, B, width = np.array([40, 1, 23]), 3, 12
    m = Model(g, fmt, hq, hkv, d, page, B * width, 40)
    table = dev(rng.permutation(B * width).reshape(B, width).astype(np.int32))
    lens_d = dev(lens.astype(np.int32))
    starts = np.concatenate([[0], np.cumsum(lens)])
    held = [[[np.zeros((0, hkv, d))] * 2 for _ in range(B)] for _ in m.layers]

    def x_of(rows):
        return dev(rng.standard_normal((rows, E)).astype(np.float32))

    # the prompts, ragged, in one call
    keep = []
    T = int(starts[-1])
    m.step(x_of(T), g.KVBatch(table, lens_d, dev(starts.astype(np.int32)), T=T, max_len=width * page), keep)
    torch.cuda.synchronize()
    for layer, stages, h in zip(m.layers, keep, held):
        check_block(m, layer, stages, starts, lens, h)

    # one token a sequence, eager
    one = g.KVBatch(table, lens_d, max_len=width * page)
    for _ in range(2):
        lens += 1
        lens_d.copy_(dev(lens.astype(np.int32)))
        keep = []
        m.step(x_of(B), one, keep)
        torch.cuda.synchronize()
        for layer, stages, h in zip(m.layers, keep, held):
            check_block(m, layer, stages, np.arange(B + 1), lens, h)

    # the same captured, beside eager calls on a copy of the caches
    twin = Model(g, fmt, hq, hkv, d, page, B * width, 40)
    for a, b in zip(twin.layers, m.layers):
        a["cache"].pages.copy_(b["cache"].pages)
    x, out = x_of(B), torch.empty(B, E, device="cuda")
    work = torch.empty(max(16, g.qmv_kv_attention_bytes(B, B, hq, hkv, d, width * page)), dtype=torch.uint8,
                       device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out.copy_(m.step(x, one, work=work))
    for i in range(6):
        lens += 1
        lens_d.copy_(dev(lens.astype(np.int32)))
        x.copy_(x_of(B))
        graph.replay()
        want = twin.step(x, one)
        if i % 2:
            torch.cuda.synchronize()
        assert torch.equal(out, want), i
        for a, b in zip(twin.layers, m.layers):
            assert torch.equal(a["cache"].pages, b["cache"].pages), i
