"""Routing at the ends of its range, and the experts' products in each kernel by
name where the shapes of other tests lead to another one."""
import numpy as np
import pytest

from test_gpu_moe import dev, g  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("E,top", [(8, 8), (70, 5)])
def test_route_sigmoids_that_are_subnormal(g, E, top):  # noqa: F811
    """Logits around -715: s is exp(l), some 1e-311 in 64 bits, and its shares of their sum are ordinary numbers."""
    rng = np.random.default_rng(6)
    logits = rng.uniform(-718, -712, (40, E)).astype(np.float32)
    logits[1::2, :2] = -709.5                                     # on either side of where exp(-l) ends
    logits[1::2, 1] = -708.5
    logits[0] = -800.0                                            # a sigmoid of 0 in 64 bits too
    idx, weight = g.moe_route(dev(logits), top, score="sigmoid")
    # all choices are 0 in 32 bits: the lowest numbers
    assert np.array_equal(idx.cpu().numpy(), np.tile(np.arange(top, dtype=np.int32), (40, 1)))
    s = np.exp(logits[:, :top].astype(np.float64))
    total = s.sum(1, keepdims=True)
    want = np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    assert (want[1:] > 0).all() and not want[0].any()
    # rounded once to 32 bits; s and the sum to steps of 2^-1074, of which the least s, exp(-718), has 2^38
    assert np.all(np.abs(weight.cpu().numpy() - want) <= want * (2.0 ** -24 + 2.0 ** -34))
