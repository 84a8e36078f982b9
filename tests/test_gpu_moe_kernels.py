"""Each kernel of the experts' products by name, the operators in a row as a
feed-forward block of experts uses them, on streams and in graphs, and the
limits of their sizes."""
import numpy as np
import pytest

import moe_ref
import oracle
import synth
from checks import assert_bitwise
from test_gpu_moe import FORMATS, check_down, check_gateup, dev, expert_blobs, fits, g, pick  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# rows of a workgroup, down, T, top, E, N, K; a Q6_K call of 64 takes 128
CASES = [
    (1, 0, 1, 2, 4, 37, 512), (1, 0, 6, 4, 16, 50, 288), (1, 0, 3, 2, 3, 21, 8192),
    (1, 1, 1, 16, 20, 37, 512), (1, 1, 7, 4, 16, 50, 2048 + 96), (1, 1, 2, 2, 3, 21, 16384),
    (4, 0, 2, 2, 3, 20, 8192 + 256), (4, 0, 1, 2, 3, 35, 8192 + 32), (4, 0, 4, 32, 40, 33, 8192 + 256),
    (4, 1, 2, 17, 20, 50, 512), (4, 1, 4, 17, 20, 20, 288), (4, 1, 1, 1, 2, 9, 16384 + 64),
    (16, 0, 9, 3, 4, 19, 8192 + 256), (16, 0, 70, 2, 4, 35, 512), (16, 0, 70, 2, 4, 64, 96),
    (16, 1, 9, 2, 3, 18, 16384 + 256), (16, 1, 5, 20, 24, 33, 256), (16, 1, 40, 4, 8, 35, 288),
    (64, 0, 150, 2, 3, 70, 512), (64, 0, 130, 1, 1, 129, 96), (64, 1, 150, 2, 3, 129, 512 + 64),
    (128, 0, 260, 2, 2, 68, 512), (128, 0, 270, 1, 1, 33, 288), (128, 1, 150, 4, 2, 130, 256),
]
# one of each kernel (of 4, the down product alone)
SOME = [(1, 6, 4, 16, 36, 256), (4, 4, 17, 20, 36, 256), (16, 70, 2, 4, 36, 256), (64, 150, 2, 3, 36, 256),
        (128, 260, 2, 2, 36, 256)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel,down,T,top,E,N,K", CASES)
def test_the_kernel_of_a_call(g, fmt, kernel, down, T, top, E, N, K):  # noqa: F811
    K = K if fits(fmt, K) else -(-K // 256) * 256
    if fmt == synth.Q6_K and kernel == 64:
        kernel = 128
    assert g.qmv_moe_rows(fmt, down, T, top, E, N, K) == kernel
    check = check_down if down else check_gateup
    for kind in ("any", "none"):
        check(g, fmt, T, top, E, N, K, kind, staged=kind == "any")


class Call:
    """Inputs of one gate/up and one down product over the same pairs; run(): both, from x and h."""

    def __init__(self, g, T, top, E, N, K, seed=0, shift=0, fmt=synth.Q5_0):  # noqa: F811
        self.g, self.fmt, self.N, self.K = g, fmt, N, K
        rng = np.random.default_rng(seed)
        self.w = [dev(np.concatenate(expert_blobs(fmt, E, N, K, seed + 100 * i))) for i in range(3)]
        self.x = self.at(synth.activations(T, K, seed + 1), shift)
        self.h = self.at(synth.activations(T * top, K, seed + 2).reshape(T, top, K), shift)
        self.idx = self.at(pick(rng, T, top, E, "none"), shift)
        self.weight = self.at(rng.random((T, top)).astype(np.float32), shift)
        self.out = self.at(np.zeros((T, top, N), np.float32), shift)
        self.y = self.at(np.zeros((T, N), np.float32), shift)
        self.work = torch.empty(max(g.qmv_moe_gateup_bytes(T, top, E, N, K), g.qmv_moe_down_bytes(T, top, E, N, K)),
                                dtype=torch.uint8, device="cuda")

    @staticmethod
    def at(a, shift):
        """a, `shift` elements behind an aligned address."""
        flat = torch.zeros(a.size + shift, dtype=torch.from_numpy(a).dtype, device="cuda")
        t = flat[shift:].view(a.shape)
        t.copy_(torch.from_numpy(a))
        return t

    def run(self, stream=None):
        self.g.moe_gateup_swiglu(self.fmt, self.w[0], self.w[1], self.N, self.K, self.idx, x=self.x, h=self.out,
                                 work=self.work, stream=stream)
        self.g.moe_down(self.fmt, self.w[2], self.N, self.K, self.idx, self.weight, h=self.h, y=self.y,
                        work=self.work, stream=stream)

    def results(self):
        return self.out.cpu().numpy(), self.y.cpu().numpy()

    def clear(self):
        self.out.fill_(7)
        self.y.fill_(7)


def same(a, b):
    for u, v, what in zip(a, b, "hy"):
        assert_bitwise(u, v, what)


@pytest.mark.parametrize("kernel,T,top,E,N,K", SOME)
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_four_byte_alignment(g, kernel, T, top, E, N, K, shift):  # noqa: F811
    a, b = Call(g, T, top, E, N, K), Call(g, T, top, E, N, K, shift=shift)
    a.run()
    b.run()
    same(b.results(), a.results())


@pytest.mark.parametrize("kernel,T,top,E,N,K", SOME)
def test_two_streams_at_once(g, kernel, T, top, E, N, K):  # noqa: F811
    calls = [Call(g, T, top, E, N, K, seed=s) for s in (0, 1)]
    want = []
    for c in calls:
        c.run()
        want.append(c.results())
        c.clear()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(8):
        for c, s in zip(calls, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        same(c.results(), w)


@pytest.mark.parametrize("kernel,T,top,E,N,K", SOME)
def test_two_graphs_share_a_workspace(g, kernel, T, top, E, N, K):  # noqa: F811
    """Captured on one stream, replayed in turn, with other numbers and rows each time."""
    calls = [Call(g, T, top, E, N, K, seed=s) for s in (0, 1)]
    calls[1].work = calls[0].work
    eager = [Call(g, T, top, E, N, K, seed=s) for s in (0, 1)]
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for c, graph in zip(calls, graphs):
        with torch.cuda.graph(graph):
            c.run()
    for replay in range(4):
        for i, (c, e) in enumerate(zip(calls, eager)):
            rng = np.random.default_rng(50 * replay + i)
            for t in (c, e):
                t.clear()
            idx = dev(pick(rng, T, top, E, ("any", "none", "one", "different" if top <= E else "any")[replay]))
            x = dev(synth.activations(T, K, 60 + replay + i))
            for t in (c, e):
                t.idx.copy_(idx)
                t.x.copy_(x)
            e.run()
        for graph in graphs:
            graph.replay()
        for c, e in zip(calls, eager):
            same(c.results(), e.results())


class Block:
    """The feed-forward of a block of experts: norm, router, routing, gate/up, down."""

    def __init__(self, g, fmt, E, top, D, F, seed):  # noqa: F811
        self.g, self.fmt, self.E, self.top, self.D, self.F = g, fmt, E, top, D, F
        self.norm = (1 + 0.1 * np.random.default_rng(seed).standard_normal(D)).astype(np.float32)
        self.router = synth.weights(synth.Q8_0, E, D, seed + 1)[0]
        self.gates, self.ups = expert_blobs(fmt, E, F, D, seed + 2), expert_blobs(fmt, E, F, D, seed + 200)
        self.downs = expert_blobs(fmt, E, D, F, seed + 400)
        self.normd, self.routerd = dev(self.norm), dev(self.router)
        self.wd = [dev(np.concatenate(b)) for b in (self.gates, self.ups, self.downs)]

    def buffers(self, T):
        g = self.g
        e = lambda *s, d=torch.float32: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
        n = max(g.qmv_moe_gateup_bytes(T, self.top, self.E, self.F, self.D),
                g.qmv_moe_down_bytes(T, self.top, self.E, self.D, self.F))
        return dict(x=e(T, self.D), normed=e(T, self.D), xq=e(g.qmv_act_bytes(T, self.D), d=torch.uint8),
                    logits=e(T, self.E), idx=e(T, self.top, d=torch.int32), weight=e(T, self.top),
                    h=e(T, self.top, self.F), y=e(T, self.D), work=e(n, d=torch.uint8))

    def run(self, b):
        g, T = self.g, b["x"].shape[0]
        g.add_rmsnorm(b["x"], self.normd, 1e-5, y=b["normed"], xq=b["xq"])
        if T <= 16:
            g.matvec(synth.Q8_0, self.routerd, self.E, self.D, xq=b["xq"], B=T, y=b["logits"])
        else:
            g.matmul(synth.Q8_0, self.routerd, self.E, self.D, xq=b["xq"], M=T, y=b["logits"])
        g.moe_route(b["logits"], self.top, idx=b["idx"], weight=b["weight"])
        g.moe_gateup_swiglu(self.fmt, *self.wd[:2], self.F, self.D, b["idx"], xq=b["xq"], h=b["h"], work=b["work"])
        g.moe_down(self.fmt, self.wd[2], self.D, self.F, b["idx"], b["weight"], h=b["h"], y=b["y"], work=b["work"])

    def check(self, b):
        """Every stage from what the stage before left."""
        v = {k: t.cpu().numpy() for k, t in b.items()}
        idx, weight = moe_ref.route(v["logits"], self.top)
        assert np.array_equal(v["idx"], idx)
        # one rounding to f32 (2^-24), and less than that in 64 bits
        assert np.all(np.abs(v["weight"] - weight) <= weight * 2.0 ** -23)
        assert_bitwise(v["h"], moe_ref.gateup(self.fmt, self.gates, self.ups, self.F, self.D, v["normed"], idx), "h")
        ref, bound = moe_ref.down(self.fmt, self.downs, self.D, self.F, v["h"], idx, v["weight"])
        assert np.all(np.abs(v["y"] - ref) <= bound * self.top * 2.0 ** -24)


@pytest.mark.parametrize("fmt", [synth.Q4_K, synth.Q6_K, synth.Q4_0, synth.Q8_0])
@pytest.mark.parametrize("T", [1, 7, 70, 300])
def test_a_block_of_experts(g, fmt, T):  # noqa: F811
    """Eager, then captured and replayed with other rows between eager runs of the same block."""
    block = Block(g, fmt, 4, 2, 256, 512, 31)
    b, e = block.buffers(T), block.buffers(T)
    b["x"].copy_(dev(synth.activations(T, 256, 5)))
    block.run(b)
    block.check(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.run(b)
    for replay in range(3):
        x = dev(synth.activations(T, 256, 80 + replay))
        e["x"].copy_(x)
        block.run(e)
        b["x"].copy_(x)
        b["y"].fill_(7)
        graph.replay()
        for name in ("idx", "weight", "h", "y"):
            assert_bitwise(b[name].cpu().numpy(), e[name].cpu().numpy(), name)
    block.check(b)


# ------------------------------------------------------------------- limits --

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_the_most_tokens(g, score):  # noqa: F811
    T = 1 << 20
    logits = torch.randn(T, 3, device="cuda")
    idx, weight = g.moe_route(logits, 1, score=score, renorm=False)
    l = logits.cpu().numpy()
    s = (torch.softmax(logits.double(), 1) if score == "softmax" else torch.sigmoid(logits.double())).cpu().numpy()
    # a sigmoid is compared rounded to f32, where neighbouring logits can be equal (the lowest number then)
    c = l if score == "softmax" else s.astype(np.float32)
    first = c.argmax(1)
    assert np.array_equal(idx[:, 0].cpu().numpy(), first)
    p = s[np.arange(T), first]
    assert np.all(np.abs(weight[:, 0].cpu().numpy().astype(np.float64) - p) <= p * 2.0 ** -23)


@pytest.mark.parametrize("fmt", [synth.Q4_0, synth.Q6_K])
@pytest.mark.parametrize("E", [1, 3, 1024])
def test_the_most_pairs(g, fmt, E):  # noqa: F811
    """2^20 pairs, E experts; every row is one of 16 times the same expert number in a run of them."""
    T, N, K = 1 << 20, 5, 32 if fmt == synth.Q4_0 else 256
    blobs = expert_blobs(fmt, E, N, K, 3) if E < 9 else expert_blobs(fmt, 8, N, K, 3) * (E // 8)
    x = synth.activations(16, K, 4)
    which = np.arange(E, dtype=np.int32).repeat(-(-T // E))[:T]
    w, xd, idx = dev(np.concatenate(blobs)), dev(x).repeat(T // 16, 1), dev(which[:, None])
    h = g.moe_gateup_swiglu(fmt, w, w, N, K, idx, x=xd)
    y = g.moe_down(fmt, w, N, K, idx, torch.ones(T, 1, device="cuda"), h=xd.view(T, 1, K))
    kinds = min(E, 8)
    p = np.stack([moe_ref.product(fmt, blobs, N, K, x, np.full(16, e)) for e in range(kinds)])     # [kinds][16][N]
    pick_p = dev(p)[idx[:, 0].long() % kinds, torch.arange(T, device="cuda") % 16]
    assert torch.equal(y.view(torch.int32), pick_p.view(torch.int32))
    s = dev(oracle.swiglu(p.reshape(-1, N), p.reshape(-1, N)).reshape(p.shape))
    pick_s = s[idx[:, 0].long() % kinds, torch.arange(T, device="cuda") % 16]
    assert torch.equal(h.view(T, N).view(torch.int32), pick_s.view(torch.int32))


@pytest.mark.parametrize("T,kernel", [(1, 1), (5, 16), (300, 64)])
def test_weights_beyond_4_gib(g, T, kernel):  # noqa: F811
    """The last expert's last rows; the other matrices are zeros."""
    E, N, K, tail = 9, 32768, 16384, 40
    one = N * g.row_bytes(g.Q8_0, K)
    assert (E - 1) * one > 1 << 32
    blob = synth.weights(synth.Q8_0, tail, K, 5)[0]
    w = torch.zeros(E * one, dtype=torch.uint8, device="cuda")
    w[E * one - blob.size:] = dev(blob)
    top = 3 if T == 300 else 2
    assert g.qmv_moe_rows(g.Q8_0, True, T, top, E, N, K) == kernel
    idx = np.full((T, top), E - 1, np.int32)
    idx[:, 0] = -1
    idx[0, 0] = 0
    h = synth.activations(T * top, K, 6).reshape(T, top, K)
    weight = np.full((T, top), 0.5, np.float32)
    y = g.moe_down(g.Q8_0, w, N, K, dev(idx), dev(weight), h=dev(h)).cpu().numpy()
    assert not y[:, :N - tail].any()
    on = np.where(idx == E - 1, 0, -1)
    ref, bound = moe_ref.down(synth.Q8_0, [blob], tail, K, h, on, weight)
    assert np.all(np.abs(y[:, N - tail:] - ref) <= bound * top * 2.0 ** -24)


def test_results_beyond_4_gib(g):  # noqa: F811
    T, N, K, E = 1 << 19, 2100, 32, 2
    blobs = expert_blobs(synth.Q4_0, E, N, K, 3)
    x = synth.activations(16, K, 4)
    w, xd = dev(np.concatenate(blobs)), dev(x).repeat(T // 16, 1)
    idx = torch.full((T, 1), 1, dtype=torch.int32, device="cuda")
    p = moe_ref.product(synth.Q4_0, blobs, N, K, x, np.full(16, 1))
    h = g.moe_gateup_swiglu(g.Q4_0, w, w, N, K, idx, x=xd)
    assert h.numel() * 4 > 1 << 32
    assert (h.view(T // 16, 16, N).view(torch.int32) == dev(oracle.swiglu(p, p)).view(torch.int32)).all()
    del h
    y = g.moe_down(g.Q4_0, w, N, K, idx, torch.ones(T, 1, device="cuda"), h=xd.view(T, 1, K))
    assert (y.view(T // 16, 16, N).view(torch.int32) == dev(p).view(torch.int32)).all()


# ------------------------------------------------------- values that are not finite --


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("where", ["rows", "weights"])
@pytest.mark.parametrize("kernel,down,T,top,E,N,K", [
    (1, 0, 2, 2, 4, 32, 288), (1, 1, 2, 2, 4, 32, 288), (4, 0, 3, 2, 3, 32, 8192 + 288), (4, 1, 2, 17, 20, 32, 288),
    (16, 0, 70, 2, 4, 32, 288), (16, 1, 70, 2, 4, 32, 288), (64, 0, 100, 2, 2, 32, 288), (64, 1, 100, 2, 2, 32, 288),
    (128, 0, 260, 1, 1, 32, 288), (128, 1, 260, 1, 1, 32, 288)])
def test_values_that_are_not_finite(g, fmt, where, kernel, down, T, top, E, N, K):  # noqa: F811
    """Infinities, NaN and magnitudes whose scale overflows fp16, in first and last blocks: as in a single product."""
    K = K if fits(fmt, K) else -(-K // 256) * 256
    assert g.qmv_moe_rows(fmt, down, T, top, E, N, K) in (kernel, 128 if kernel == 64 else kernel)
    rng = np.random.default_rng(9)
    rows = T * top if down else T
    x = synth.activations(rows, K, 3)
    blobs = [np.concatenate(expert_blobs(fmt, E, N, K, s)) for s in (1, 2)]
    if where == "rows":
        bad = [np.inf, -np.inf, np.nan, 3e7, -3e38, 0.0]
        for r in range(0, rows, 2):
            x[r, rng.choice([0, 31, K - 32, K - 1, K // 2])] = bad[(r // 2) % len(bad)]
        x[1, K - 32:] = 0
    else:
        block, size = g.BLOCK[fmt]
        at = size - 2 if fmt == synth.Q6_K else 0
        for b in blobs:
            v = b.reshape(E * N, -1, size)
            for i, bits in enumerate((0x7C00, 0xFC00, 0x7E00, 0x7BFF)):
                v[3 * i + 1, (0, -1)[i & 1], at:at + 2] = np.frombuffer(np.uint16(bits).tobytes(), np.uint8)
    idx = pick(rng, T, top, E, "any")
    w, u, xd = dev(blobs[0]), dev(blobs[1]), dev(x)
    one = N * g.row_bytes(fmt, K)
    pairs = idx.reshape(-1)
    if down:
        weight = rng.random((T, top)).astype(np.float32)
        got = g.moe_down(fmt, w, N, K, dev(idx), dev(weight), h=xd.view(T, top, K)).cpu().numpy()
        p = torch.stack([g.matvec(fmt, w[e * one:(e + 1) * one], N, K, x=xd[i:i + 1])[0] for i, e in enumerate(pairs)])
        p = p.view(T, top, N).double()
        want = torch.zeros(T, N, dtype=torch.float32, device="cuda")
        for j in range(top):   # fma: the product is exact in 64 bits, and the sum rounded there before it is to f32
            want = (dev(weight)[:, j, None].double() * p[:, j] + want.double()).float()
        want = want.cpu().numpy()
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan)
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        fin = ~(nan | inf)
        bound = (dev(weight)[..., None].double() * p).abs().sum(1).cpu().numpy()
        assert np.all(np.abs(got[fin].astype(np.float64) - want[fin]) <= bound[fin] * top * 2.0 ** -23)
    else:
        got = g.moe_gateup_swiglu(fmt, w, u, N, K, dev(idx), x=xd).view(T * top, N).cpu().numpy()
        # (K beyond the pair's fused limit: the two products)
        y = [torch.stack([g.matvec(fmt, m[e * one:(e + 1) * one], N, K, x=xd[i // top:i // top + 1])[0]
                          for i, e in enumerate(pairs)]).double() for m in (w, u)]
        want = (y[0] / (1 + torch.exp(-y[0])) * y[1]).float().cpu().numpy()
        nan, inf = np.isnan(want), np.isinf(want)
        assert np.array_equal(np.isnan(got), nan)
        assert np.array_equal(got[inf], want[inf])
        fin = ~(nan | inf)
        # both in 64 bits, rounded once
        assert np.all(np.abs(got[fin].astype(np.float64) - want[fin]) <= np.abs(want[fin]) * 2.0 ** -22 + 2.0 ** -148)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [2e-5, 1e-6, 1e6])
@pytest.mark.parametrize("T,top,E,N,K", [(2, 2, 4, 32, 512), (70, 2, 4, 32, 512), (100, 2, 2, 32, 512),
                                         (260, 1, 1, 32, 512)])
def test_scales_that_are_subnormal(g, fmt, size, T, top, E, N, K):  # noqa: F811
    """fp16 scales below 2^-14 of weights and activations: as in the documented order, bit for bit."""
    rng = np.random.default_rng(4)
    x = (synth.activations(T, K, 3) * np.float32(size)).astype(np.float32)
    block, bytes_ = g.BLOCK[fmt]
    at = bytes_ - 2 if fmt == synth.Q6_K else 0
    blobs = [b.copy() for b in expert_blobs(fmt, E, N, K, 1)]
    for b in blobs:
        v = b.reshape(N, -1, bytes_)
        bits = rng.integers(1, 0x400, v.shape[:2]).astype("<u2")
        bits[::3] |= 0x3800                                      # of a third of the rows normal ones
        v[:, :, at:at + 2] = bits.view(np.uint8).reshape(*v.shape[:2], 2)
    idx = pick(rng, T, top, E, "any")
    h = g.moe_gateup_swiglu(fmt, *[dev(np.concatenate(blobs))] * 2, N, K, dev(idx), x=dev(x)).cpu().numpy()
    assert_bitwise(h, moe_ref.gateup(fmt, blobs, blobs, N, K, x, idx), "h")
    one = np.ascontiguousarray(idx[:, :1])
    y = g.moe_down(fmt, dev(np.concatenate(blobs)), N, K, dev(one), torch.ones(T, 1, device="cuda"),
                   h=dev(x).view(T, 1, K)).cpu().numpy()
    assert_bitwise(y, moe_ref.product(fmt, blobs, N, K, x, one[:, 0]) + np.float32(0), "y")
