"""CPU tests of the mixture-of-experts entry points: sizes and refusals (every
check runs on the host before anything is enqueued)."""
import os

import pytest

import gguf_quantized_matvec_amd as g

pytestmark = pytest.mark.skipif(not os.path.exists(g.LIB_PATH), reason="libqmv.so not built")

P = 1 << 20  # a 16-byte aligned non-NULL address; never dereferenced
TYPE, SHAPE, PTR = -1, -2, -3
NAN, INF = float("nan"), float("inf")

ROUTE = dict(logits=P, T=4, E=16, score=0, bias=P, groups=1, top_groups=1, group_top=1, top=2, renorm=1, scale=1.0,
             idx=P, weight=P)


@pytest.mark.parametrize("bad,code", [
    (dict(T=0), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(T=1 << 20), SHAPE),     # T * top
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(top=0), SHAPE), (dict(top=17), SHAPE),
    (dict(E=64, top=33), SHAPE), (dict(score=2), SHAPE), (dict(score=-1), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(E=130, groups=65), SHAPE),
    (dict(groups=4, top_groups=0), SHAPE), (dict(groups=4, top_groups=5), SHAPE),
    (dict(groups=8, top_groups=1, top=3), SHAPE),                                     # more than the groups hold
    (dict(groups=4, top_groups=2, group_top=0), SHAPE), (dict(groups=4, top_groups=2, group_top=3), SHAPE),
    (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE),
    (dict(logits=None), PTR), (dict(idx=None), PTR), (dict(weight=None), PTR), (dict(logits=P + 2), PTR),
    (dict(bias=P + 1), PTR), (dict(idx=P + 2), PTR), (dict(weight=P + 3), PTR),
])
def test_route_refusals(bad, code):
    assert g.lib().qmv_moe_route(*dict(ROUTE, **bad).values(), None) == code


GATEUP = dict(type=g.Q4_0, w_gate=P, w_up=P, E=8, N=48, K=64, idx=P, T=4, top=2, x=P, xq=None, h=2 * P, work=P)
DOWN = dict(type=g.Q4_0, w=P, E=8, N=48, K=64, idx=P, weight=P, T=4, top=2, h=P, hq=None, y=2 * P, work=P)

SHARED = [
    (dict(type=4), TYPE), (dict(type=10), TYPE), (dict(type=g.Q4_K), SHAPE), (dict(type=g.Q6_K, K=896), SHAPE),
    (dict(K=48), SHAPE), (dict(K=0), SHAPE), (dict(K=(1 << 20) + 32), SHAPE), (dict(N=0), SHAPE),
    (dict(N=(1 << 24) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(T=0), SHAPE),
    (dict(T=1 << 20), SHAPE), (dict(top=0), SHAPE), (dict(top=33), SHAPE),
    (dict(T=1 << 18, K=1 << 15), SHAPE),                                              # 2^33 activations
    (dict(idx=None), PTR), (dict(idx=P + 2), PTR), (dict(work=None), PTR), (dict(work=P + 8), PTR),
]


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(w_gate=None), PTR), (dict(w_up=None), PTR), (dict(w_gate=P + 8), PTR), (dict(w_up=P + 8), PTR),
    (dict(x=None), PTR), (dict(xq=P), PTR), (dict(x=P + 2), PTR), (dict(x=None, xq=P + 8), PTR),
    (dict(h=None), PTR), (dict(h=2 * P + 2), PTR), (dict(h=P), PTR),
])
def test_gateup_refusals(bad, code):
    assert g.lib().qmv_moe_gateup_swiglu(*dict(GATEUP, **bad).values(), None) == code


@pytest.mark.parametrize("bad,code", SHARED + [
    (dict(w=None), PTR), (dict(w=P + 8), PTR), (dict(h=None), PTR), (dict(hq=P), PTR), (dict(h=P + 2), PTR),
    (dict(h=None, hq=P + 8), PTR), (dict(weight=None), PTR), (dict(weight=P + 2), PTR), (dict(y=None), PTR),
    (dict(y=2 * P + 2), PTR), (dict(y=P), PTR),
])
def test_down_refusals(bad, code):
    assert g.lib().qmv_moe_down(*dict(DOWN, **bad).values(), None) == code


def test_workspaces():
    # the Q8_0 blocks of the rows come first; the down products' workspace also holds a row a pair
    assert g.qmv_moe_gateup_bytes(4, 2, 8, 48, 64) >= 4 * 2 * 34
    assert g.qmv_moe_down_bytes(4, 2, 8, 48, 64) >= 8 * 2 * 34 + 8 * 48 * 4
    for bad in [(0, 2, 8, 48, 64), (4, 0, 8, 48, 64), (4, 33, 64, 48, 64), (4, 2, 0, 48, 64), (4, 2, 1025, 48, 64),
                (4, 2, 8, 0, 64), (4, 2, 8, (1 << 24) + 1, 64), (4, 2, 8, 48, 0), (4, 2, 8, 48, 48),
                (4, 2, 8, 48, (1 << 20) + 32), ((1 << 19) + 1, 2, 8, 48, 64), (1 << 18, 1, 8, 48, 1 << 15)]:
        assert g.qmv_moe_gateup_bytes(*bad) == 0
        assert g.qmv_moe_down_bytes(*bad) == 0


def test_the_kernel_of_a_call():
    # type, down, T, top, E, N, K
    assert g.qmv_moe_rows(g.Q4_0, 0, 1, 2, 8, 48, 64) == g.qmv_moe_rows(g.Q4_0, 1, 1, 2, 8, 48, 64) == 1
    assert [g.qmv_moe_rows(g.Q4_0, 0, T, 2, 2, 48, 16384) for T in (4, 5, 95, 96, 255, 256)] == [4, 16, 16, 64, 64, 128]
    assert [g.qmv_moe_rows(g.Q6_K, 1, T, 2, 2, 48, 16384 + 256) for T in (4, 5, 47, 48)] == [4, 16, 16, 128]
    for bad in [(99, 0, 4, 2, 8, 48, 64), (g.Q4_0, 0, 0, 2, 8, 48, 64), (g.Q4_0, 0, 4, 33, 64, 48, 64),
                (g.Q4_0, 1, 4, 2, 0, 48, 64), (g.Q4_0, 1, 4, 2, 8, 0, 64), (g.Q4_0, 1, 4, 2, 8, 48, 48),
                (g.Q4_K, 1, 4, 2, 8, 48, 288), (g.Q4_0, 1, 1 << 18, 1, 8, 48, 1 << 15)]:
        assert g.qmv_moe_rows(*bad) == 0


def test_python_refusals():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 16)
    with pytest.raises(TypeError):
        g.moe_route(t, 2)                                    # not on a device
    with pytest.raises(ValueError):
        g.moe_route(torch.zeros(16), 2)
    with pytest.raises(ValueError):
        g.moe_route(t, 2, score="relu")
    with pytest.raises(TypeError):
        g.moe_gateup_swiglu(g.Q4_0, t, t, 16, 32, t, x=t)
    with pytest.raises(TypeError):
        g.moe_down(g.Q4_0, t, 16, 32, t, t, h=t)
