"""Residual add + RMS norm into 8 bits on the GPU, against the formula in 64
bits and against the quantisers of the library (whose blocks the oracle pins)."""
import numpy as np
import pytest

import synth
from checks import assert_bitwise
from step_ref import rmsnorm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-5


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


def inputs(rows, K, seed):
    rng = np.random.default_rng(seed)
    wide = np.where(rng.random(K) < 0.02, 30, 1)
    x = (rng.standard_normal((rows, K)) * 0.4).astype(np.float32)
    res = (rng.standard_normal((rows, K)) * wide).astype(np.float32)
    return x, res, (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)


def dev(a):
    return torch.from_numpy(a).cuda()


def call(g, q8k, x, w, **k):
    return (g.add_rmsnorm_q8k if q8k else g.add_rmsnorm)(x, w, EPS, **k)


def staged(g, q8k, rows, K, fill, y=None, run=None):
    """The whole scratch, filled with a pattern first, as the quantiser (of y) or `run` leaves it."""
    n = g.qmv_act_bytes_q8k(rows, K) if q8k else g.qmv_act_bytes(rows, K)
    xq = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
    if y is not None:
        (g.quantize_q8k if q8k else g.quantize)(y, xq=xq)
    else:
        run(xq)
    return xq.cpu().numpy()


# K: one block, a partial chunk, 1 / 2 / 4 chunks a wave, more than stay in registers
@pytest.mark.parametrize("rows,K", [
    (1, 32), (1, 896), (1, 4096), (2, 4864), (3, 96), (4, 14336), (5, 896), (7, 8192 + 32), (16, 4096),
    (17, 64), (33, 1024), (5, 16384 + 32), (1, 16384 + 32), (40, 16384 + 96), (1, 1 << 20)])
@pytest.mark.parametrize("with_res", [True, False])
def test_q8_0(g, rows, K, with_res):
    check(g, False, rows, K, with_res)


@pytest.mark.parametrize("rows,K", [(1, 256), (3, 4096), (5, 512), (16, 4096), (17, 768), (33, 14336),
                                    (2, 16384 + 256), (1, 1 << 20)])
@pytest.mark.parametrize("with_res", [True, False])
def test_q8_k(g, rows, K, with_res):
    check(g, True, rows, K, with_res)


def check(g, q8k, rows, K, with_res):
    print(f"norm q8k={q8k} rows={rows} K={K} res={with_res}", flush=True)
    x, res, w = inputs(rows, K, rows * 7 + K)
    y = torch.full((rows, K), float("nan"), device="cuda")
    rd = dev(res) if with_res else None
    out = {}
    got = staged(g, q8k, rows, K, 0xA5, run=lambda xq: out.update(
        h=call(g, q8k, dev(x), dev(w), res=rd, y=y, xq=xq)[0]))
    h, y64 = rmsnorm(x, w, EPS, res if with_res else None)
    if with_res:
        assert_bitwise(out["h"].cpu().numpy(), h, "h")
    else:
        assert out["h"] is None
    yh = y.cpu().numpy()
    # one rounding of a value that f64 holds to far below an f32 step
    assert np.all(np.abs(yh - y64) <= 2.0 ** -24 * np.abs(y64) * (1 + 1e-6) + 2.0 ** -150)
    # every byte that the quantiser writes, and no other
    assert_bitwise(got, staged(g, q8k, rows, K, 0xA5, y=y), "scratch")


@pytest.mark.parametrize("q8k", [False, True])
def test_unaligned_and_in_place(g, q8k):
    rows, K = 6, 1024
    x, res, w = inputs(rows, K, 5)
    h0, q0 = call(g, q8k, dev(x), dev(w), res=dev(res))

    def shifted(a):  # 4-byte aligned only
        t = torch.empty(a.size + 1, device="cuda")[1:]
        return t.copy_(dev(a).reshape(-1)).view(a.shape)

    xs, rs = shifted(x), shifted(res)
    h, q = call(g, q8k, xs, shifted(w), res=rs, h=shifted(np.zeros_like(x)), y=shifted(x))
    assert torch.equal(h, h0)
    n = rows * K // 256 * 292 if q8k else rows * K // 32 * 34
    assert torch.equal(q[:n], q0[:n])
    for which in ("x", "res"):
        xd, rd = dev(x), dev(res)
        h, q = call(g, q8k, xd, dev(w), res=rd, h=xd if which == "x" else rd)
        assert h.data_ptr() == (xd if which == "x" else rd).data_ptr()
        assert torch.equal(h, h0) and torch.equal(q[:n], q0[:n])
    # in place beyond what stays in registers
    x, res, w = inputs(2, 16384 + 256, 9)
    h0, q0 = call(g, q8k, dev(x), dev(w), res=dev(res))
    rd = dev(res)
    h, q = call(g, q8k, dev(x), dev(w), res=rd, h=rd)
    n = 2 * (16384 + 256) // 256 * 292 if q8k else 2 * (16384 + 256) // 32 * 34
    assert torch.equal(h, h0) and torch.equal(q[:n], q0[:n])


@pytest.mark.parametrize("q8k", [False, True])
def test_a_row_does_not_depend_on_the_others(g, q8k):
    rows, K = 40, 4096
    x, res, w = inputs(rows, K, 6)
    res[3, 17] = np.inf  # a row without a norm leaves the others alone
    res[7] = 0
    x[7] = 0             # a row of zeros: y = 0
    y = torch.empty(rows, K, device="cuda")
    call(g, q8k, dev(x), dev(w), res=dev(res), y=y)
    assert torch.equal(y[7], torch.zeros(K, device="cuda"))
    for lo, hi in [(0, 1), (4, 8), (10, 26), (8, 40)]:
        part = torch.empty(hi - lo, K, device="cuda")
        call(g, q8k, dev(x[lo:hi]), dev(w), res=dev(res[lo:hi]), y=part)
        assert torch.equal(part, y[lo:hi])


def test_extremes(g):
    # huge and tiny rows: the sum of squares leaves f32's range, not f64's
    K = 512
    x = np.stack([np.full(K, 3e38), np.full(K, -1e30), np.full(K, 1e-30), np.linspace(-1, 1, K)]).astype(np.float32)
    w = np.ones(K, np.float32)
    y = torch.empty(4, K, device="cuda")
    g.add_rmsnorm(dev(x), dev(w), 0.0, y=y)
    _, y64 = rmsnorm(x, w, 0.0)
    assert np.all(np.abs(y.cpu().numpy() - y64) <= 2.0 ** -24 * np.abs(y64) * (1 + 1e-6))


@pytest.mark.parametrize("rows", [1, 4, 5, 16, 33])
def test_feeds_the_products(g, rows):
    N, K = 48, 1024
    x, res, w = inputs(rows, K, 8)
    y = torch.empty(rows, K, device="cuda")
    _, xq = g.add_rmsnorm(dev(x), dev(w), EPS, res=dev(res), y=y)
    blob = dev(synth.weights(synth.Q4_K, N, K, seed=1)[0])
    if rows <= 16:
        a = g.matvec(synth.Q4_K, blob, N, K, xq=xq, B=rows)
    else:
        a = g.matmul(synth.Q4_K, blob, N, K, xq=xq, M=rows)
    assert torch.equal(a, g.matmul(synth.Q4_K, blob, N, K, x=y))
    _, xq = g.add_rmsnorm_q8k(dev(x), dev(w), EPS, res=dev(res), y=y)
    a = g.matmul_q8k(synth.Q4_K, blob, N, K, xq=xq, M=rows)
    assert torch.equal(a, g.matmul_q8k(synth.Q4_K, blob, N, K, x=y))


def test_streams_and_capture(g):
    rows, K = 5, 4096
    w = dev(inputs(rows, K, 1)[2])
    x, res = (torch.zeros(rows, K, device="cuda") for _ in range(2))
    h, y = torch.empty_like(x), torch.empty_like(x)
    xq = g.act_buffer(rows, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        g.add_rmsnorm(x, w, EPS, res=res, h=h, y=y, xq=xq)
    for seed in range(3):
        a, b, _ = inputs(rows, K, 20 + seed)
        x.copy_(dev(a))
        res.copy_(dev(b))
        graph.replay()
        torch.cuda.synchronize()
        y1, q1 = y.clone(), xq.clone()
        y2 = torch.empty_like(y)
        h2, q2 = g.add_rmsnorm(x, w, EPS, res=res, y=y2, xq=torch.empty_like(xq).copy_(xq))
        assert torch.equal(h2, h) and torch.equal(y1, y2) and torch.equal(q1, q2)
    # on a stream given to the call, as an object and as a handle
    with torch.cuda.stream(s):
        a, b = x * 2, res * 3
    h3, q3 = g.add_rmsnorm(a, w, EPS, res=b, stream=s)
    h4, q4 = g.add_rmsnorm(a, w, EPS, res=b, stream=s.cuda_stream)
    torch.cuda.synchronize()
    h5, _ = g.add_rmsnorm(a, w, EPS, res=b)
    assert torch.equal(h3, h5) and torch.equal(h4, h5)
