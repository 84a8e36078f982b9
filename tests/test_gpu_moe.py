"""Routing to experts and the experts' products on the GPU, against the
formulas in 64 bits and the oracle's replay of the documented f32 order."""
import numpy as np
import pytest

import moe_ref
import synth
from checks import assert_bitwise

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FORMATS = [synth.Q4_0, synth.Q4_1, synth.Q5_0, synth.Q5_1, synth.Q8_0, synth.Q8_1, synth.Q4_K, synth.Q6_K]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gguf_quantized_matvec_amd as g
    g.lib()
    return g


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ routing --

def check_route(g, logits, top, bias=None, sigmoid=False, **k):
    idx, weight = g.moe_route(dev(logits), top, score="sigmoid" if sigmoid else "softmax",
                              bias=None if bias is None else dev(bias), **k)
    ref_idx, ref = moe_ref.route(logits, top, sigmoid=sigmoid, bias=bias, **k)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    # in 64 bits and rounded once: half a step, and the 64-bit sums' own error of some 2^-50
    assert np.all(np.abs(weight.cpu().numpy() - ref) <= np.abs(ref) * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -149)
    return idx, weight


@pytest.mark.parametrize("T,E,top", [
    (1, 1, 1), (1, 8, 2), (3, 8, 8), (5, 60, 4), (1, 64, 8), (7, 65, 6), (2, 128, 8), (33, 160, 6), (4, 256, 8),
    (3, 257, 1), (2, 512, 16), (2, 513, 32), (1, 1024, 32), (1000, 16, 4)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(g, T, E, top, sigmoid, biased, renorm):
    rng = np.random.default_rng(T * 1000 + E)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if biased else None
    check_route(g, logits, top, bias, sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("T,E,top,groups,top_groups", [
    (5, 256, 8, 8, 4), (3, 160, 6, 8, 3), (4, 64, 6, 64, 8), (9, 96, 4, 3, 1), (2, 1024, 8, 64, 64), (6, 30, 5, 5, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_groups(g, T, E, top, groups, top_groups, sigmoid, biased, group_top):
    rng = np.random.default_rng(T * 1000 + E + groups)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if biased else None
    check_route(g, logits, top, bias, sigmoid, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_ties_go_to_the_lowest(g, sigmoid, groups, group_top):
    rng = np.random.default_rng(3)
    logits = rng.integers(-1, 2, (40, 96)).astype(np.float32)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0
    check_route(g, logits, 8, None, sigmoid, groups=groups, top_groups=(groups + 1) // 2, group_top=group_top)
    check_route(g, logits, 8, np.zeros(96, np.float32), sigmoid, groups=groups, top_groups=groups, group_top=group_top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
def test_route_values_that_are_not_finite(g, sigmoid, renorm, groups, biased):
    rng = np.random.default_rng(4)
    E = 72
    logits = (rng.standard_normal((12, E)) * 3).astype(np.float32)
    logits[0] = -np.inf                                    # nothing is available
    logits[1, 5:] = -np.inf                                # fewer than top are
    logits[2, :] = np.nan
    logits[3, ::3] = np.nan
    logits[4, 17] = np.inf
    logits[5, [9, 40]] = np.inf
    logits[6] = np.finfo(np.float32).min                   # the type's lowest value: available
    logits[7, :70] = np.finfo(np.float32).min
    logits[8] = np.finfo(np.float32).max
    logits[9, 60:] = [-np.inf, np.inf, np.nan, 1, 2, 3, 4, 5, 6, -1e30, 1e30, 0]
    logits[10] = -1000.0                                   # a sigmoid of 0 in 64 bits too
    bias = None
    if biased:
        bias = (rng.standard_normal(E) * 0.2).astype(np.float32)
        bias[[3, 50]] = -np.inf
        bias[[7, 51]] = np.nan
        bias[20] = np.inf
    with np.errstate(invalid="ignore"):
        check_route(g, logits, 8, bias, sigmoid, renorm=renorm, groups=groups, top_groups=groups, group_top=1)
        check_route(g, logits, 8, bias, sigmoid, renorm=renorm, groups=groups, top_groups=max(1, groups // 2), group_top=2)


# ----------------------------------------------------------------- products --

def expert_blobs(fmt, E, N, K, seed, **k):
    return [synth.weights(fmt, N, K, seed + e, **k)[0] for e in range(E)]


def pick(rng, T, top, E, kind):
    """Expert numbers: different ones a token, all the same, any (twice in a token too), some that are none."""
    if kind == "different":
        return np.stack([rng.permutation(E)[:top] for _ in range(T)]).astype(np.int32)
    if kind == "one":
        return np.full((T, top), E - 1, np.int32)
    idx = rng.integers(0, E, (T, top)).astype(np.int32)
    if kind == "none":
        idx[rng.random((T, top)) < 0.4] = rng.choice([-1, E, 1 << 30, -(1 << 31)])
        if T > 1:
            idx[0] = -1
    return idx


def guarded(shape, dtype=torch.float32, fill=0xA5):
    """A tensor between guard bytes: (tensor, the whole buffer's bytes)."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
    return whole[256:256 + n].view(dtype).view(shape), whole


def guards_hold(whole, n, fill=0xA5):
    raw = whole.cpu().numpy()
    return (raw[:256] == fill).all() and (raw[256 + n:] == fill).all()


def check_gateup(g, fmt, T, top, E, N, K, kind, seed=0, staged=False, **k):
    rng = np.random.default_rng(seed + T * 7 + N)
    gates, ups = expert_blobs(fmt, E, N, K, seed + 10, **k), expert_blobs(fmt, E, N, K, seed + 500, **k)
    x, idx = synth.activations(T, K, seed + 3), pick(rng, T, top, E, kind)
    h, whole = guarded((T, top, N))
    n = g.qmv_moe_gateup_bytes(T, top, E, N, K)
    work, wwhole = guarded((n,), torch.uint8)
    xd = dev(x)
    k = dict(xq=g.quantize(xd)) if staged else dict(x=xd)
    g.moe_gateup_swiglu(fmt, dev(np.concatenate(gates)), dev(np.concatenate(ups)), N, K, dev(idx), h=h, work=work, **k)
    assert_bitwise(h.cpu().numpy(), moe_ref.gateup(fmt, gates, ups, N, K, x, idx), "h")
    assert guards_hold(whole, h.numel() * 4) and guards_hold(wwhole, n)


def check_down(g, fmt, T, top, E, N, K, kind, seed=0, staged=False, **k):
    rng = np.random.default_rng(seed + T * 7 + N)
    blobs = expert_blobs(fmt, E, N, K, seed + 10, **k)
    h = synth.activations(T * top, K, seed + 3).reshape(T, top, K)
    idx = pick(rng, T, top, E, kind)
    weight = rng.random((T, top)).astype(np.float32)
    y, whole = guarded((T, N))
    n = g.qmv_moe_down_bytes(T, top, E, N, K)
    work, wwhole = guarded((n,), torch.uint8)
    hd = dev(h)
    k = dict(hq=g.quantize(hd.view(T * top, K))) if staged else dict(h=hd)
    g.moe_down(fmt, dev(np.concatenate(blobs)), N, K, dev(idx), dev(weight), y=y, work=work, **k)
    ref, bound = moe_ref.down(fmt, blobs, N, K, h, idx, weight)
    # one rounding a slot
    assert np.all(np.abs(y.cpu().numpy() - ref) <= bound * top * 2.0 ** -24)
    if top == 1:   # fma(1, product, 0): the product itself
        ones = torch.ones_like(dev(weight))
        y1 = g.moe_down(fmt, dev(np.concatenate(blobs)), N, K, dev(idx), ones, h=hd)
        assert_bitwise(y1.cpu().numpy(), moe_ref.product(fmt, blobs, N, K, h[:, 0], idx[:, 0]), "y")
    assert guards_hold(whole, y.numel() * 4) and guards_hold(wwhole, n)


# one row of an expert to more than an item holds; one block, short last chunks, several segments; odd numbers of
# rows, so that matrices begin at any even address
SHAPES = [(1, 2, 3, 33, 32), (1, 1, 2, 16, 256), (4, 2, 3, 17, 96), (5, 3, 4, 40, 896), (3, 8, 9, 7, 512),
          (9, 2, 5, 65, 288), (20, 2, 3, 50, 256), (33, 4, 8, 19, 512), (1, 4, 4, 24, 4864), (2, 2, 3, 11, 8192 + 64)]


def fits(fmt, K):
    return K % 256 == 0 or fmt not in (synth.Q4_K, synth.Q6_K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,K", SHAPES)
def test_gateup(g, fmt, T, top, E, N, K):
    check_gateup(g, fmt, T, top, E, N, K if fits(fmt, K) else -(-K // 256) * 256, "none")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,K", SHAPES)
def test_down(g, fmt, T, top, E, N, K):
    check_down(g, fmt, T, top, E, N, K if fits(fmt, K) else -(-K // 256) * 256, "none")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 5, 17, 40, 200])
def test_products_of_one_slot(g, fmt, T):
    check_down(g, fmt, T, 1, 4, 37, 512, "any", seed=T)


@pytest.mark.parametrize("kind", ["different", "one", "any", "none"])
@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("T,top,E", [(1, 4, 6), (6, 4, 6), (16, 4, 6), (17, 4, 6), (70, 6, 12), (130, 1, 2)])
def test_which_experts(g, kind, staged, T, top, E):
    check_gateup(g, synth.Q4_0, T, top, E, 35, 288, kind, staged=staged)
    check_down(g, synth.Q5_1, T, top, E, 35, 288, kind, staged=staged)


def test_no_pair_has_an_expert(g):
    for T, top in [(1, 2), (30, 4)]:
        idx = torch.full((T, top), -1, dtype=torch.int32, device="cuda")
        w = dev(synth.weights(synth.Q8_0, 3 * 20, 64, 1)[0])
        h = g.moe_gateup_swiglu(g.Q8_0, w, w, 20, 64, idx, x=torch.randn(T, 64, device="cuda"))
        assert not h.cpu().numpy().view(np.uint32).any()
        y = g.moe_down(g.Q8_0, w, 20, 64, idx, torch.full((T, top), float("nan"), device="cuda"), h=torch.randn(T, top, 64, device="cuda"))
        assert not y.cpu().numpy().view(np.uint32).any()


# Tiles of 64 and 128 rows of an expert, full and part full; a last tile of a few weight rows; short last chunks, an odd
# number of blocks
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,K", [
    (48, 1, 2, 33, 32), (30, 2, 2, 130, 288), (100, 2, 3, 70, 512), (97, 1, 1, 17, 96), (150, 2, 3, 129, 512 + 64),
    (260, 1, 2, 68, 896)])
@pytest.mark.parametrize("kind", ["any", "none"])
def test_many_rows(g, fmt, T, top, E, N, K, kind):
    K = K if fits(fmt, K) else -(-K // 256) * 256
    check_gateup(g, fmt, T, top, E, N, K, kind, staged=kind == "any")
    check_down(g, fmt, T, top, E, N, K, kind, staged=kind == "any")
    check_down(g, fmt, T * top, 1, E, N, K, kind)


@pytest.mark.parametrize("kind", ["one", "different"])
@pytest.mark.parametrize("T,top,E", [(70, 2, 3), (300, 2, 4)])
def test_many_rows_unevenly(g, kind, T, top, E):
    check_gateup(g, synth.Q4_K, T, top, E, 100, 512, kind)
    check_down(g, synth.Q8_0, T, top, E, 100, 512, kind)


# Q6_K's int8 sub-scales over their whole range (odd ones beyond 64 do not fold into f16), and a few rows of them
@pytest.mark.parametrize("T,top,E", [(3, 2, 3), (40, 2, 3), (70, 1, 2), (200, 2, 2)])
@pytest.mark.parametrize("s_range", [(-128, 127), (-66, 66), (127, 127), (-128, -128)])
def test_q6_k_scales(g, T, top, E, s_range):
    check_gateup(g, synth.Q6_K, T, top, E, 80, 768, "any", s_range=s_range)
    check_down(g, synth.Q6_K, T * top, 1, E, 80, 768, "any", s_range=s_range)


# One token: a row of 1 to 64 chunks, short last ones, several rows a wave and one; 1 to 16 slots, and more
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("top,E,N,K", [(1, 2, 33, 32), (2, 4, 70, 256), (3, 5, 37, 96), (8, 9, 21, 896), (16, 16, 9, 512),
                                       (20, 24, 9, 256), (2, 3, 19, 4864), (2, 3, 10, 8192), (2, 2, 7, 14336)])
@pytest.mark.parametrize("kind", ["none", "any"])
def test_one_token(g, fmt, top, E, N, K, kind):
    K = K if fits(fmt, K) else -(-K // 256) * 256
    for seed in (0, 7):
        check_gateup(g, fmt, 1, top, E, N, K, kind, seed=seed, staged=seed == 7)
        check_down(g, fmt, 1, top, E, N, K, kind, seed=seed, staged=seed == 7)
