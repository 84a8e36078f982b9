"""Routing at the ends of its range, and the experts' products in each kernel by
name where the shapes of other tests lead to another one."""
import numpy as np
import pytest

import moe_ref
import synth
from checks import assert_bitwise
from test_gpu_moe import FORMATS, check_down, check_gateup, dev, expert_blobs, fits, g, pick  # noqa: F401
from test_gpu_moe_kernels import Call, same
from test_gpu_moe_kernels import test_four_byte_alignment as four_byte_alignment
from test_gpu_moe_kernels import test_two_graphs_share_a_workspace as two_graphs_share_a_workspace
from test_gpu_moe_kernels import test_two_streams_at_once as two_streams_at_once

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


def whole(fmt, K):
    return K if fits(fmt, K) else -(-K // 256) * 256


def reach(g, fmt, kernel, down, T, top, E, N, K):  # noqa: F811
    """K as the format takes it, once the call of that shape runs the kernel (Q6_K has no tile of 64 rows)."""
    K = whole(fmt, K)
    if fmt == synth.Q6_K and kernel == 64:
        kernel = 128
    assert g.qmv_moe_rows(fmt, down, T, top, E, N, K) == kernel
    return K


# Q6_K's int8 sub-scales over their whole range where a wave takes 16 columns: 4 and 16 rows of an expert, items found
# in the kernel (up to 64 pairs) and planned; of one slot the product itself is compared, bit for bit
@pytest.mark.parametrize("kernel,down,T,top,E,N,K", [
    (4, 0, 2, 2, 3, 20, 8192 + 256), (16, 0, 9, 3, 4, 19, 8192 + 256), (16, 0, 70, 2, 4, 35, 512),
    (4, 1, 2, 17, 20, 50, 512), (4, 1, 3, 1, 2, 21, 16384 + 256), (16, 1, 9, 1, 2, 18, 16384 + 256),
    (16, 1, 150, 1, 8, 37, 768), (16, 1, 40, 4, 8, 35, 512), (128, 1, 200, 1, 2, 37, 768), (128, 0, 75, 2, 2, 37, 768)])
@pytest.mark.parametrize("s_range", [(-128, 127), (-66, 66), (127, 127), (-128, -128)])
def test_q6_k_scales_by_kernel(g, kernel, down, T, top, E, N, K, s_range):  # noqa: F811
    reach(g, synth.Q6_K, kernel, down, T, top, E, N, K)
    (check_down if down else check_gateup)(g, synth.Q6_K, T, top, E, N, K, "any", s_range=s_range)


# Tiles of 64 and 128 rows: a single block, three, an odd number; one weight row to a part of the second tile; rows that
# fill a tile, pass it by one and leave most of it empty
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel,T,top,E,N,K", [
    (64, 150, 1, 1, 33, 32), (64, 97, 2, 2, 17, 96), (64, 129, 1, 1, 1, 32), (64, 192, 1, 1, 63, 288),
    (64, 131, 3, 3, 65, 64), (128, 257, 1, 1, 17, 96), (128, 256, 1, 1, 33, 32), (128, 300, 2, 2, 1, 96),
    (128, 385, 1, 1, 63, 288), (128, 260, 2, 2, 129, 64)])
@pytest.mark.parametrize("kind", ["any", "none"])
def test_small_products_of_many_rows(g, fmt, kernel, T, top, E, N, K, kind):  # noqa: F811
    for down, t, s in ((0, T, top), (1, T, top), (1, T * top, 1)):
        k = reach(g, fmt, kernel, down, t, s, E, N, K)
        (check_down if down else check_gateup)(g, fmt, t, s, E, N, k, kind, staged=kind == "any")


# The same of up to 16 rows an item
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kernel,down,T,top,E,N,K", [
    (16, 0, 70, 2, 5, 33, 32), (16, 0, 70, 2, 5, 1, 96), (16, 0, 45, 3, 9, 17, 896), (16, 0, 17, 8, 20, 7, 512),
    (16, 0, 65, 2, 3, 65, 288), (16, 1, 70, 2, 5, 33, 32), (16, 1, 70, 2, 5, 1, 96), (16, 1, 45, 3, 9, 17, 896),
    (16, 1, 5, 17, 20, 7, 512), (16, 1, 140, 1, 5, 65, 288), (16, 1, 150, 1, 9, 11, 8192 + 64),
    (4, 1, 1, 17, 20, 33, 32), (4, 1, 4, 32, 40, 1, 96), (4, 1, 3, 20, 24, 17, 896), (4, 1, 2, 17, 3, 65, 288)])
@pytest.mark.parametrize("kind", ["one", "none"])
def test_small_products_of_few_rows(g, fmt, kernel, down, T, top, E, N, K, kind):  # noqa: F811
    K = reach(g, fmt, kernel, down, T, top, E, N, K)
    (check_down if down else check_gateup)(g, fmt, T, top, E, N, K, kind, staged=kind == "one")


def subnormal(fmt, blobs, N, rng):
    """The blobs with fp16 scales below 2^-14, of a third of their rows normal ones."""
    import gguf_quantized_matvec_amd as lib
    block, size = lib.BLOCK[fmt]
    at = size - 2 if fmt == synth.Q6_K else 0
    out = [b.copy() for b in blobs]
    for b in out:
        v = b.reshape(N, -1, size)
        bits = rng.integers(1, 0x400, v.shape[:2]).astype("<u2")
        bits[::3] |= 0x3800
        v[:, :, at:at + 2] = bits.view(np.uint8).reshape(*v.shape[:2], 2)
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [2e-5, 1e-6, 1e6])
@pytest.mark.parametrize("kernel,down,T,top,E,N,K", [
    (1, 0, 2, 2, 4, 32, 512), (4, 0, 3, 2, 3, 32, 8192 + 256), (16, 0, 9, 3, 4, 32, 8192 + 256), (16, 0, 70, 2, 4, 32, 512),
    (64, 0, 100, 2, 2, 32, 512), (128, 0, 260, 1, 1, 32, 512), (1, 1, 4, 1, 4, 32, 512), (4, 1, 3, 1, 2, 32, 16384 + 256),
    (16, 1, 9, 1, 2, 32, 16384 + 256), (16, 1, 150, 1, 4, 32, 512), (64, 1, 200, 1, 2, 32, 512), (128, 1, 260, 1, 1, 32, 512)])
def test_scales_that_are_subnormal_by_kernel(g, fmt, size, kernel, down, T, top, E, N, K):  # noqa: F811
    """fp16 scales below 2^-14 of weights and activations: as in the documented order, bit for bit."""
    reach(g, fmt, kernel, down, T, top, E, N, K)
    rng = np.random.default_rng(4)
    x = (synth.activations(T, K, 3) * np.float32(size)).astype(np.float32)
    blobs = subnormal(fmt, expert_blobs(fmt, E, N, K, 1), N, rng)
    idx, w, xd = pick(rng, T, top, E, "any"), dev(np.concatenate(blobs)), dev(x)
    if down:      # fma(1, product, +0): the product itself, but for its zero's sign
        y = g.moe_down(fmt, w, N, K, dev(idx), torch.ones(T, 1, device="cuda"), h=xd.view(T, 1, K)).cpu().numpy()
        assert_bitwise(y, moe_ref.product(fmt, blobs, N, K, x, idx[:, 0]) + np.float32(0), "y")
    else:
        h = g.moe_gateup_swiglu(fmt, w, w, N, K, dev(idx), x=xd).cpu().numpy()
        assert_bitwise(h, moe_ref.gateup(fmt, blobs, blobs, N, K, x, idx), "h")


# The rows kernel that finds its items among the numbers itself (up to 64 pairs), in both products
FEW = [(4, 2, 17, 20, 36, 8192 + 256), (16, 9, 7, 8, 36, 8192 + 256)]


def few(g, kernel, T, top, E, N, K):  # noqa: F811
    assert T * top <= 64
    for down in (0, 1):
        reach(g, synth.Q5_0, kernel, down, T, top, E, N, K)


@pytest.mark.parametrize("kernel,T,top,E,N,K", FEW)
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_items_found_with_four_byte_alignment(g, kernel, T, top, E, N, K, shift):  # noqa: F811
    few(g, kernel, T, top, E, N, K)
    four_byte_alignment(g, kernel, T, top, E, N, K, shift)


@pytest.mark.parametrize("kernel,T,top,E,N,K", FEW)
def test_items_found_on_two_streams(g, kernel, T, top, E, N, K):  # noqa: F811
    few(g, kernel, T, top, E, N, K)
    two_streams_at_once(g, kernel, T, top, E, N, K)


@pytest.mark.parametrize("kernel,T,top,E,N,K", FEW)
def test_items_found_in_two_graphs(g, kernel, T, top, E, N, K):  # noqa: F811
    """Replayed with other numbers: all of one expert, none, any, different ones."""
    few(g, kernel, T, top, E, N, K)
    two_graphs_share_a_workspace(g, kernel, T, top, E, N, K)


@pytest.mark.parametrize("kernel,T,top,E,N,K", FEW + [(1, 6, 4, 16, 36, 256), (128, 260, 2, 2, 36, 256)])
def test_buffers_that_touch(g, kernel, T, top, E, N, K):  # noqa: F811
    """Every buffer directly behind another: none overlaps, so the calls are taken, with the results of buffers apart."""
    a, b = Call(g, T, top, E, N, K), Call(g, T, top, E, N, K)
    b.work = b.work[:0].new_empty(-(-b.work.numel() // 16) * 16)
    names = ["out", "x", "work", "idx", "y", "h", "weight"]
    sizes = [getattr(b, n).numel() * getattr(b, n).element_size() for n in names]
    assert all(s % 16 == 0 for s in sizes[:2])                       # so that the workspace is aligned where it stands
    buffer, at = torch.empty(sum(sizes), dtype=torch.uint8, device="cuda"), 0
    for n, size in zip(names, sizes):
        old = getattr(b, n)
        new = buffer[at:at + size].view(old.dtype).view(old.shape)
        new.copy_(old)
        setattr(b, n, new)
        at += size
    a.run()
    b.run()
    same(b.results(), a.results())
    i, w = g.moe_route(buffer[:4 * 8 * 4].view(torch.float32).view(4, 8), 2, idx=buffer[128:160].view(torch.int32).view(4, 2),
                       weight=buffer[160:192].view(torch.float32).view(4, 2))
    assert i.data_ptr() + 32 == w.data_ptr()
