"""CPU tests of the operators around the products: sizes and refusals (every
check runs on the host before anything is enqueued)."""
import ctypes
import os
import subprocess
import sys

import pytest

import gguf_quantized_matvec_amd as g

pytestmark = pytest.mark.skipif(not os.path.exists(g.LIB_PATH), reason="libqmv.so not built")

P = 1 << 20  # a 16-byte aligned non-NULL address; never dereferenced
SHAPE, PTR = -2, -3


@pytest.mark.parametrize("args,code", [
    ((P, P, P, 1e-5, 0, 64, P, None, P), SHAPE),              # rows
    ((P, P, P, 1e-5, (1 << 24) + 1, 64, P, None, P), SHAPE),
    ((P, P, P, 1e-5, 1, 48, P, None, P), SHAPE),              # K
    ((P, P, P, 1e-5, 1, 0, P, None, P), SHAPE),
    ((P, P, P, 1e-5, 1, (1 << 20) + 32, P, None, P), SHAPE),
    ((P, P, P, -1.0, 1, 64, P, None, P), SHAPE),              # eps
    ((P, P, P, float("nan"), 1, 64, P, None, P), SHAPE),
    ((None, P, P, 1e-5, 1, 64, P, None, P), PTR),
    ((P, P, None, 1e-5, 1, 64, P, None, P), PTR),
    ((P, P, P, 1e-5, 1, 64, P, None, None), PTR),
    ((P, P, P, 1e-5, 1, 64, P, None, P + 8), PTR),            # xq 16-byte aligned
    ((P + 2, P, P, 1e-5, 1, 64, P, None, P), PTR),
    ((P, P + 1, P, 1e-5, 1, 64, P, None, P), PTR),
    ((P, P, P, 1e-5, 1, 64, P + 2, None, P), PTR),
    ((P, P, P, 1e-5, 1, 64, P, P + 2, P), PTR),
    ((P, P, P, 1e-5, 1, 64, None, None, P), PTR),             # res without h
    ((P, None, P, 1e-5, 1, 64, P, None, P), PTR),             # h without res
    ((P, P, P, 1e-5, 1, 64, P, P, P), PTR),                   # y over another buffer
])
def test_norm_refusals(args, code):
    assert g.lib().qmv_add_rmsnorm_q8_0(*args, None) == code


def test_norm_q8k_needs_whole_superblocks():
    assert g.lib().qmv_add_rmsnorm_q8_k(P, P, P, 1e-5, 1, 896, P, None, P, None) == SHAPE
    assert g.lib().qmv_add_rmsnorm_q8_k(P, P, P, 1e-5, 0, 256, P, None, P, None) == SHAPE


def test_kv_bytes():
    # 36 bytes per 32 elements of key and value, one token, one head
    assert g.qmv_kv_bytes(1, 16, 1, 32) == 16 * 36
    assert g.qmv_kv_bytes(5, 64, 8, 128) == 5 * 8 * 64 * 144
    assert g.qmv_kv_bytes((1 << 31) - 1, 1024, 1024, 256) == ((1 << 31) - 1) * 1024 * 1024 * 288
    for bad in [(0, 16, 1, 32), (1, 8, 1, 32), (1, 48, 1, 32), (1, 2048, 1, 32), (1, 16, 0, 32),
                (1, 16, 1025, 32), (1, 16, 1, 48), (1, 16, 1, 0), (1, 16, 1, 288), (1 << 31, 16, 1, 32)]:
        assert g.qmv_kv_bytes(*bad) == 0


def kv(**k):
    d = dict(pages=P, n_pages=4, page_tokens=16, kv_heads=2, head_dim=64)
    d.update(k)
    return g.KvStruct(*(d[n] for n, _ in g.KvStruct._fields_))


def seqs(**k):
    d = dict(table=P, table_stride=2, lens=P, q_start=None, B=3, T=3, max_len=32)
    d.update(k)
    return g.KvBatchStruct(*(d[n] for n, _ in g.KvBatchStruct._fields_))


BAD = [
    (kv(n_pages=0), seqs(), SHAPE), (kv(page_tokens=8), seqs(), SHAPE),
    (kv(page_tokens=24), seqs(), SHAPE), (kv(kv_heads=0), seqs(), SHAPE),
    (kv(head_dim=48), seqs(), SHAPE), (kv(head_dim=512), seqs(), SHAPE),
    (kv(), seqs(B=0, T=0), SHAPE), (kv(), seqs(T=4), SHAPE),           # one row a sequence
    (kv(), seqs(q_start=P, T=0), SHAPE), (kv(), seqs(q_start=P, T=(1 << 20) + 1), SHAPE),
    (kv(), seqs(table_stride=0), SHAPE), (kv(), seqs(max_len=0), SHAPE),
    (kv(), seqs(max_len=33), SHAPE),                                   # more than the table names
    (kv(page_tokens=1024), seqs(table_stride=1 << 22, max_len=(1 << 30) + 1), SHAPE),
    (kv(pages=None), seqs(), PTR), (kv(pages=P + 8), seqs(), PTR),
    (kv(), seqs(table=None), PTR), (kv(), seqs(lens=None), PTR), (kv(), seqs(lens=P + 2), PTR),
    (kv(), seqs(q_start=P + 1), PTR),
]


@pytest.mark.parametrize("c,s,code", BAD)
def test_cache_and_batch_refusals(c, s, code):
    L = g.lib()
    assert L.qmv_kv_append(c, s, P, 256, 4, P, 128, P, 128, P, 64, 0, P, None) == code
    assert L.qmv_kv_read(c, s, P, P, None) == code
    assert L.qmv_kv_attention(c, s, P, 256, 4, 0.1, 0, P, 2 * P, None) == code


def test_cache_without_structures():
    L = g.lib()
    assert L.qmv_kv_read(None, seqs(), P, P, None) == PTR
    assert L.qmv_kv_read(kv(), None, P, P, None) == PTR
    assert L.qmv_kv_read(kv(), seqs(), None, P, None) == PTR
    assert L.qmv_kv_read(kv(), seqs(), P, P + 2, None) == PTR


@pytest.mark.parametrize("args,code", [
    ((P, 256, 3, P, 128, P, 128, P, 64, 0, P), SHAPE),     # q_heads no multiple of kv_heads
    ((P, 256, 0, P, 128, P, 128, P, 64, 0, P), SHAPE),
    ((P, 2 ** 18, 1026, P, 128, P, 128, P, 64, 0, P), SHAPE),
    ((P, 255, 4, P, 128, P, 128, P, 64, 0, P), SHAPE),     # strides shorter than a row
    ((P, 256, 4, P, 127, P, 128, P, 64, 0, P), SHAPE),
    ((P, 256, 4, P, 128, P, 127, P, 64, 0, P), SHAPE),
    ((P, 256, 4, P, 128, P, 128, P, 66, 0, P), SHAPE),     # rot
    ((P, 256, 4, P, 128, P, 128, P, 31, 0, P), SHAPE),
    ((P, 256, 4, P, 128, P, 128, P, -2, 0, P), SHAPE),
    ((P, 256, 4, P, 128, P, 128, None, 64, 0, P), PTR),    # freq
    ((P, 256, 4, P, 128, P, 128, P + 4, 64, 0, P), PTR),
    ((None, 256, 4, P, 128, P, 128, P, 64, 0, P), PTR),
    ((P, 256, 4, None, 128, P, 128, P, 64, 0, P), PTR),
    ((P, 256, 4, P, 128, P + 2, 128, P, 64, 0, P), PTR),
    ((P, 256, 4, P, 128, P, 128, P, 64, 0, None), PTR),
    ((P, 300, 4, P, 128, P, 128, P, 64, 0, P), PTR),       # in place with another row length
])
def test_append_refusals(args, code):
    assert g.lib().qmv_kv_append(kv(), seqs(), *args, None) == code


@pytest.mark.parametrize("args,code", [
    ((P, 256, 3, 0.1, 0, 2 * P, 3 * P), SHAPE),
    ((P, 252, 4, 0.1, 0, 2 * P, 3 * P), SHAPE),
    ((P, 258, 4, 0.1, 0, 2 * P, 3 * P), SHAPE),            # a stride that breaks the alignment
    ((P, 256, 4, 0.0, 0, 2 * P, 3 * P), SHAPE),
    ((P, 256, 4, float("nan"), 0, 2 * P, 3 * P), SHAPE),
    ((P, 256, 4, float("inf"), 0, 2 * P, 3 * P), SHAPE),
    ((P, 256, 4, 0.1, -1, 2 * P, 3 * P), SHAPE),
    ((P + 4, 256, 4, 0.1, 0, 2 * P, 3 * P), PTR),
    ((P, 256, 4, 0.1, 0, 2 * P + 8, 3 * P), PTR),
    ((P, 256, 4, 0.1, 0, P, 3 * P), PTR),                  # out over q
    ((P, 256, 4, 0.1, 0, 2 * P, None), PTR),
    ((P, 256, 4, 0.1, 0, 2 * P, 3 * P + 4), PTR),
])
def test_attention_refusals(args, code):
    assert g.lib().qmv_kv_attention(kv(), seqs(), *args, None) == code


def test_attention_workspace():
    f = g.qmv_kv_attention_bytes
    for bad in [(0, 1, 4, 2, 64, 9), (1, 0, 4, 2, 64, 9), (1, 1, 3, 2, 64, 9), (1, 1, 4, 2, 48, 9),
                (1, 1, 4, 2, 64, 0), (1, 1, 4, 2, 64, (1 << 30) + 1), ((1 << 20) + 1, 1, 4, 2, 64, 9)]:
        assert f(*bad) == 0
    last = 0
    for n in (1, 100, 511, 512, 513, 4096, 70000, 1 << 20):
        assert f(1, 1, 32, 8, 128, n) >= max(last, 16)
        last = f(1, 1, 32, 8, 128, n)
    for t in (1, 2, 7, 16, 100, 511, 512, 513, 4096, 1 << 20):
        assert f(t, t, 32, 8, 128, 4096) >= 16 and f(t, 1, 32, 8, 128, 4096) >= 16
    # few rows of a long context: the workspace holds parts; many rows: nothing to hold
    assert f(1, 1, 32, 8, 128, 4096) > 32 * 128 * 4 * 2 and f(1 << 20, 1 << 20, 32, 8, 128, 4096) == 16


def test_helpers_refuse_on_the_host():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        g.add_rmsnorm(x, torch.zeros(64), 1e-5)                # not on a device
    with pytest.raises(ValueError):
        g.add_rmsnorm(x, torch.zeros(32), 1e-5)
    with pytest.raises(ValueError):
        g.add_rmsnorm(x, torch.zeros(64), 1e-5, res=torch.zeros(1, 64))
    with pytest.raises(ValueError):
        g.add_rmsnorm(x, torch.zeros(64), 1e-5, h=torch.zeros(2, 64))
    with pytest.raises(ValueError):
        g.KVCache(torch.zeros(16, dtype=torch.uint8), 24, 1, 32)
    with pytest.raises(TypeError):
        g.KVCache(torch.zeros(16 * 36, dtype=torch.uint8), 16, 1, 32)
    with pytest.raises(ValueError):
        g.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                  torch.zeros(2, dtype=torch.int32), T=2, max_len=5)
    assert ctypes.sizeof(g.KvStruct) == 32 and ctypes.sizeof(g.KvBatchStruct) == 56


@pytest.mark.parametrize("h,y", [(P, None), (2 * P, P)])
def test_norm_refuses_outputs_over_the_weights(h, y):
    assert g.lib().qmv_add_rmsnorm_q8_0(3 * P, 4 * P, P, 1e-5, 1, 64, h, y, 5 * P, None) == PTR


@pytest.mark.parametrize("out", [2 * P, 3 * P])
def test_append_refuses_an_output_over_k_or_v(out):
    args = (P, 256, 4, 2 * P, 128, 3 * P, 128, 4 * P, 64, 0, out)
    assert g.lib().qmv_kv_append(kv(), seqs(), *args, None) == PTR


@pytest.mark.parametrize("T,B,q_heads,kv_heads", [
    (1 << 20, 1 << 20, 32, 32), (1 << 20, 1, 128, 128), (1 << 17, 1 << 17, 1024, 1024),
    (1 << 14, 1 << 14, 1024, 1024)])
def test_attention_refuses_more_tiles_than_a_grid_holds(T, B, q_heads, kv_heads):
    one = T == B
    few = 100 if one else 1
    for t, b, refused in ((T, B, True), (100, few, False)):
        n = g.qmv_kv_attention_bytes(t, b, q_heads, kv_heads, 32, 32)
        assert (n == 0) == refused
    s = seqs(B=B, T=T, q_start=None if one else P)
    assert g.lib().qmv_kv_attention(kv(kv_heads=kv_heads, head_dim=32), s, P, 32 * q_heads, q_heads, 0.1, 0,
                                    2 * P, 3 * P, None) == SHAPE


def test_new_pages_need_a_number():
    for n in (None, 0, -1):
        with pytest.raises(ValueError):
            g.KVCache(None, 16, 1, 32, n_pages=n)


def test_attention_rows_of_invalid_shapes():
    f = g.qmv_kv_attention_rows
    for bad in [(0, 1, True, 4, 2, 64, 9), (1, 0, True, 4, 2, 64, 9), (1, 1, True, 3, 2, 64, 9), (1, 1, True, 4, 2, 48, 9),
                (1, 1, True, 4, 2, 64, 0), (2, 1, False, 4, 2, 64, 9), (1 << 20, 1 << 20, True, 32, 32, 64, 9)]:
        assert f(*bad) == 0
    assert f(1, 1, False, 4, 2, 64, 9) == 8


def test_the_choice_of_an_attention_kernel():
    """Few rows a key/value head: 8 rows a workgroup, never for heads beyond 128 elements."""
    rows = g.qmv_kv_attention_rows
    assert rows(1, 1, False, 32, 8, 128, 100) == 8 and rows(1, 1, False, 32, 2, 128, 100) == 16
    assert rows(1, 1, False, 32, 8, 160, 100) == 16 and rows(1 << 14, 1, True, 32, 8, 256, 1 << 14) == 16
    assert rows(64, 64, True, 8, 1, 64, 100) == 8 and rows(65, 64, True, 8, 1, 64, 100) == 16
    assert rows(2048, 1, True, 32, 8, 128, 2048) == 64 and rows(1024, 4, True, 32, 8, 128, 4096) == 16


def test_importing_the_package_does_not_import_torch():
    """The ctypes layer has no need of torch, and works where torch is missing or broken."""
    code = ("import sys; sys.modules['torch'] = None; import gguf_quantized_matvec_amd as g; "
            "assert sys.modules['torch'] is None; print(g.qmv_kv_bytes(1, 16, 1, 32))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == str(16 * 36), r.stderr
    code = "import sys, gguf_quantized_matvec_amd; assert 'torch' not in sys.modules"
    assert subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(
        os.path.abspath(__file__)))).returncode == 0
