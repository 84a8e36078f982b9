"""CPU tests of what the mixture-of-experts entry points decide on the host:
the kernel of a call at the limits of its sizes, and buffers that overlap
(addresses are never dereferenced: every call here is refused)."""
import os

import pytest

import gguf_quantized_matvec_amd as g

pytestmark = pytest.mark.skipif(not os.path.exists(g.LIB_PATH), reason="libqmv.so not built")


@pytest.mark.parametrize("top,K,most", [
    # a row a wave, 6 waves of 64 a workgroup: 384 N threads below 2^32
    (6, 8224, ((1 << 32) - 1) // 384),
    # two rows a wave, 8 waves: 512 threads for two rows; 2^24 rows are 2^32 threads
    (8, 5632, (1 << 24) - 2),
    # a row a wave, two units of 4 waves: the same
    (4, 8224, (1 << 24) - 2),
    # a row a wave, two units of 3 waves: 192 threads a row are never as many
    (3, 8224, 1 << 24),
])
def test_no_grid_beyond_its_dimension(top, K, most):
    """The down products of a token whose matrix-vector launch would pass 2^32 threads go to the rows kernel."""
    assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, most, K) == 1
    if most < 1 << 24:
        assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, most + 1, K) == 4
        assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, 1 << 24, K) == 4


PTR = -3
GIB = 1 << 30
T, TOP, E, N, K = 5, 3, 8, 48, 64
ROW = K // 32 * 18                                     # of Q4_0
BUFFERS = {  # entry: name -> bytes, the outputs first
    "route": dict(idx=T * TOP * 4, weight=T * TOP * 4, logits=T * E * 4, bias=E * 4),
    "gateup": dict(h=T * TOP * N * 4, work=None, x=T * K * 4, xq=T * K // 32 * 34, idx=T * TOP * 4,
                   w_gate=E * N * ROW, w_up=E * N * ROW),
    "down": dict(y=T * N * 4, work=None, h=T * TOP * K * 4, hq=T * TOP * K // 32 * 34, idx=T * TOP * 4,
                 weight=T * TOP * 4, w=E * N * ROW),
}


def buffers(entry):
    b = dict(BUFFERS[entry])
    if entry != "route":
        b["work"] = {"gateup": g.qmv_moe_gateup_bytes, "down": g.qmv_moe_down_bytes}[entry](T, TOP, E, N, K)
    return b


def call(entry, a):
    L = g.lib()
    if entry == "route":
        return L.qmv_moe_route(a["logits"], T, E, 0, a["bias"], 1, 1, 1, TOP, 1, 1.0, a["idx"], a["weight"], None)
    if entry == "gateup":
        return L.qmv_moe_gateup_swiglu(g.Q4_0, a["w_gate"], a["w_up"], E, N, K, a["idx"], T, TOP, a["x"], a["xq"], a["h"],
                                       a["work"], None)
    return L.qmv_moe_down(g.Q4_0, a["w"], E, N, K, a["idx"], a["weight"], T, TOP, a["h"], a["hq"], a["y"], a["work"], None)


@pytest.mark.parametrize("entry", list(BUFFERS))
@pytest.mark.parametrize("where", ["same", "first in last", "last in first"])
def test_outputs_over_other_buffers(entry, where):
    """An output (or the workspace) that shares its first, its last or all bytes with another buffer is refused."""
    b = buffers(entry)
    names = list(b)
    for i, out in enumerate(names[:2]):
        for other in names[i + 1:]:
            a = {n: (k + 1) * GIB for k, n in enumerate(names)}
            rows = {"route": (), "gateup": ("x", "xq"), "down": ("h", "hq")}[entry]
            if rows:
                a[rows[0] if other == rows[1] else rows[1]] = None   # one of the two forms
            last = lambda n: (b[n] - 1) // 16 * 16               # noqa: E731  the last aligned place inside
            a[out] = {"same": a[other], "first in last": a[other] + last(other), "last in first": a[other] - last(out)}[where]
            assert call(entry, a) == PTR, (out, other)


def test_the_kernels_that_other_tests_name():
    """Both products of the shapes that tests of streams, graphs and alignment run: of 4 rows the gate/up pair is the
    single tokens' kernel."""
    pytest.importorskip("torch")
    from test_gpu_moe_kernels import SOME
    got = [tuple(g.qmv_moe_rows(g.Q5_0, down, *shape) for down in (0, 1)) for _, *shape in SOME]
    assert got == [(1, 1), (1, 4), (16, 16), (64, 64), (128, 128)]


@pytest.mark.parametrize("type,N,K,code", [(99, 16, 32, -1), (4, 16, 32, -1), (g.Q4_K, 16, 896, -2), (g.Q6_K, 16, 32, -2),
                                           (g.Q4_0, 16, 48, -2), (g.Q4_0, 0, 32, -2), (g.Q4_0, -16, -32, -2)])
def test_python_types_and_shapes(type, N, K, code):
    """The library's own codes, also from the helpers, which need the bytes of a row before they call it."""
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 16)
    for f, w in ((g.moe_gateup_swiglu, (t, t)), (g.moe_down, (t,))):
        with pytest.raises(g.QmvError) as e:
            f(type, *w, N, K, *((t,) if f is g.moe_gateup_swiglu else (t, t)), t)
        assert e.value.code == code
