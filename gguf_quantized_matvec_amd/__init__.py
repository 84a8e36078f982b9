"""Python binding of libqmv.so (include/qmv.h): the same entry points, argument
marshalling only.  Every step of the multiply runs in the HIP kernels.

Raw pointers and sizes go straight through; the torch-tensor helpers below
only turn tensors into (pointer, stream) and check shapes/dtypes.  There is no
CPU fallback: if the library is missing or the device is not gfx950 the calls
raise.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmv.so")

Q4_0, Q4_1, Q5_0, Q5_1, Q8_0, Q8_1, Q4_K, Q6_K = 2, 3, 6, 7, 8, 9, 12, 14
TYPES = {"Q4_0": Q4_0, "Q4_1": Q4_1, "Q5_0": Q5_0, "Q5_1": Q5_1, "Q8_0": Q8_0, "Q8_1": Q8_1,
         "Q4_K": Q4_K, "Q6_K": Q6_K}
BLOCK = {Q8_0: (32, 34), Q4_0: (32, 18), Q5_0: (32, 22), Q4_1: (32, 20), Q5_1: (32, 24),
         Q8_1: (32, 36), Q4_K: (256, 144), Q6_K: (256, 210)}
EXPORTS = ("qmv_act_bytes", "quantize_act_q8_0", "qmv_launch", "qmv_launch_group", "qmm_launch",
           "qmv_partials_launch", "qmm_partials_launch", "qmv_launch_noalloc", "qmv_gateup_act_bytes",
           "qmv_launch_gateup_swiglu", "qmv_launch_gateup_swiglu_q8", "qmv_act_bytes_q8k", "quantize_act_q8_k", "qmv_launch_q8k",
           "qmv_launch_gateup_swiglu_q8k", "qmv_launch_group_q8k", "qmm_launch_q8k", "qmv_partials_q8k_launch", "qmv_prepared_bytes", "qmv_prepare",
           "qmm_launch_q8k_prepared", "qmm_partials_q8k_prepared_launch", "qmv_add_rmsnorm_q8_0", "qmv_add_rmsnorm_q8_k",
           "qmv_kv_bytes", "qmv_kv_append", "qmv_kv_read", "qmv_kv_attention_bytes", "qmv_kv_attention_rows", "qmv_kv_attention",
           "qmv_moe_route", "qmv_moe_gateup_bytes", "qmv_moe_gateup_swiglu", "qmv_moe_down_bytes", "qmv_moe_down",
           "qmv_moe_rows", "qmv_strerror")
MAX_BATCH = 16
MAX_GROUP = 8
MOE_SCORES = {"softmax": 0, "sigmoid": 1}


class Gemv(ctypes.Structure):
    """struct qmv_gemv: one GEMV of qmv_launch_group (pointers as integers)."""
    _fields_ = [("w", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class KvStruct(ctypes.Structure):
    """struct qmv_kv: a layer's paged 4-bit cache (pointer as integer)."""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_tokens", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class KvBatchStruct(ctypes.Structure):
    """struct qmv_kv_batch: the sequences of one call (pointers as integers)."""
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("B", ctypes.c_int64),
                ("T", ctypes.c_int64), ("max_len", ctypes.c_int64)]


class QmvError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (status {code})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmv.so (built in-tree by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m gguf_quantized_matvec_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.qmv_act_bytes.argtypes = [I64, I64]
        L.qmv_act_bytes.restype = ctypes.c_size_t
        L.quantize_act_q8_0.argtypes = [P, P, I64, I64, P]
        L.qmv_launch.argtypes = [I, P, I64, I64, P, I64, P, P, P]
        L.qmm_launch.argtypes = [I, P, I64, I64, P, I64, P, P, P]
        L.qmv_launch_group.argtypes = [I, I64, ctypes.POINTER(Gemv), I, P]
        L.qmv_partials_launch.argtypes = [I, P, I64, I64, P, I64, P, P]
        L.qmv_launch_noalloc.argtypes = [I, P, I64, I64, P, I64, P, P]
        L.qmm_partials_launch.argtypes = [I, P, I64, I64, P, I64, P, P]
        L.qmv_act_bytes_q8k.argtypes = [I64, I64]
        L.qmv_act_bytes_q8k.restype = ctypes.c_size_t
        L.quantize_act_q8_k.argtypes = [P, P, I64, I64, P]
        L.qmv_launch_q8k.argtypes = [I, P, I64, I64, P, I64, P, P, P]
        L.qmm_launch_q8k.argtypes = [I, P, I64, I64, P, I64, P, P, P]
        L.qmv_partials_q8k_launch.argtypes = [I, P, I64, I64, P, I64, P, P]
        L.qmv_prepared_bytes.argtypes = [I, I64, I64]
        L.qmv_prepared_bytes.restype = ctypes.c_size_t
        L.qmv_prepare.argtypes = [I, P, I64, I64, P, P]
        L.qmm_launch_q8k_prepared.argtypes = [I, P, I64, I64, P, I64, P, P, P]
        L.qmm_partials_q8k_prepared_launch.argtypes = [I, P, I64, I64, P, I64, P, P]
        L.qmv_gateup_act_bytes.argtypes = [I64, I64, I64]
        L.qmv_gateup_act_bytes.restype = ctypes.c_size_t
        L.qmv_launch_gateup_swiglu.argtypes = [I, P, P, I64, I64, P, I64, P, P, P]
        L.qmv_launch_gateup_swiglu_q8.argtypes = [I, P, P, I64, I64, P, I64, P, P, P, P]
        L.qmv_launch_gateup_swiglu_q8k.argtypes = [I, P, P, I64, I64, P, I64, P, P, P]
        L.qmv_launch_group_q8k.argtypes = [I, I64, ctypes.POINTER(Gemv), I, P]
        F, KV, KB = ctypes.c_float, ctypes.POINTER(KvStruct), ctypes.POINTER(KvBatchStruct)
        for f in ("qmv_add_rmsnorm_q8_0", "qmv_add_rmsnorm_q8_k"):
            getattr(L, f).argtypes = [P, P, P, F, I64, I64, P, P, P, P]
        L.qmv_kv_bytes.argtypes = [I64, I, I, I]
        L.qmv_kv_bytes.restype = ctypes.c_size_t
        L.qmv_kv_append.argtypes = [KV, KB, P, I64, I, P, I64, P, I64, P, I, I, P, P]
        L.qmv_kv_read.argtypes = [KV, KB, P, P, P]
        L.qmv_kv_attention_bytes.argtypes = [I64, I64, I, I, I, I64]
        L.qmv_kv_attention_bytes.restype = ctypes.c_size_t
        L.qmv_kv_attention_rows.argtypes = [I64, I64, I, I, I, I, I64]
        L.qmv_kv_attention.argtypes = [KV, KB, P, I64, I, F, I64, P, P, P]
        L.qmv_moe_route.argtypes = [P, I64, I64, I, P, I, I, I, I, I, F, P, P, P]
        for f in ("qmv_moe_gateup_bytes", "qmv_moe_down_bytes"):
            getattr(L, f).argtypes = [I64, I, I64, I64, I64]
            getattr(L, f).restype = ctypes.c_size_t
        L.qmv_moe_gateup_swiglu.argtypes = [I, P, P, I64, I64, I64, P, I64, I, P, P, P, P, P]
        L.qmv_moe_down.argtypes = [I, P, I64, I64, I64, P, P, I64, I, P, P, P, P, P]
        L.qmv_moe_rows.argtypes = [I, I, I64, I, I64, I64, I64]
        for f in ("quantize_act_q8_0", "qmv_launch", "qmv_launch_group", "qmm_launch",
                  "qmv_partials_launch", "qmm_partials_launch", "qmv_launch_noalloc",
                  "qmv_launch_gateup_swiglu", "qmv_launch_gateup_swiglu_q8", "quantize_act_q8_k", "qmv_launch_q8k",
                  "qmv_launch_gateup_swiglu_q8k", "qmv_launch_group_q8k", "qmm_launch_q8k", "qmv_partials_q8k_launch", "qmv_prepare",
                  "qmm_launch_q8k_prepared", "qmm_partials_q8k_prepared_launch", "qmv_add_rmsnorm_q8_0",
                  "qmv_add_rmsnorm_q8_k", "qmv_kv_append", "qmv_kv_read", "qmv_kv_attention_rows",
                  "qmv_kv_attention", "qmv_moe_route", "qmv_moe_gateup_swiglu", "qmv_moe_down",
                  "qmv_moe_rows"):
            getattr(L, f).restype = I
        L.qmv_strerror.argtypes = [I]
        L.qmv_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().qmv_strerror(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise QmvError(rc, what)


# ---------------------------------------------------------------- raw C-ABI --

def qmv_act_bytes(rows: int, K: int) -> int:
    return int(lib().qmv_act_bytes(rows, K))


def quantize_act_q8_0(x, xq: int, rows: int, K: int, stream: int = 0) -> None:
    _check(lib().quantize_act_q8_0(x, xq, rows, K, stream), "quantize_act_q8_0")


def qmv_launch(type: int, w: int, N: int, K: int, x, B: int, xq: int, y: int,
               stream: int = 0) -> None:
    _check(lib().qmv_launch(type, w, N, K, x, B, xq, y, stream), "qmv_launch")


def qmv_launch_group(type: int, B: int, gemvs, stream: int = 0) -> None:
    """gemvs: a sequence of Gemv (or of (w, N, K, x, xq, y) tuples)."""
    arr = (Gemv * len(gemvs))(*[gv if isinstance(gv, Gemv) else Gemv(*gv) for gv in gemvs])
    _check(lib().qmv_launch_group(type, B, arr, len(gemvs), stream), "qmv_launch_group")


def qmv_launch_group_q8k(type: int, B: int, gemvs, stream: int = 0) -> None:
    """gemvs: a sequence of Gemv (or of (w, N, K, x, xq, y) tuples), Q8_K path."""
    arr = (Gemv * len(gemvs))(*[gv if isinstance(gv, Gemv) else Gemv(*gv) for gv in gemvs])
    _check(lib().qmv_launch_group_q8k(type, B, arr, len(gemvs), stream), "qmv_launch_group_q8k")


def qmm_launch(type: int, w: int, N: int, K: int, x, M: int, xq: int, y: int,
               stream: int = 0) -> None:
    _check(lib().qmm_launch(type, w, N, K, x, M, xq, y, stream), "qmm_launch")


def qmv_partials_launch(type: int, w: int, N: int, K: int, xq: int, B: int, P: int,
                        stream: int = 0) -> None:
    _check(lib().qmv_partials_launch(type, w, N, K, xq, B, P, stream), "qmv_partials_launch")


def qmm_partials_launch(type: int, w: int, N: int, K: int, xq: int, M: int, P: int,
                        stream: int = 0) -> None:
    _check(lib().qmm_partials_launch(type, w, N, K, xq, M, P, stream), "qmm_partials_launch")


def qmv_launch_noalloc(type: int, w: int, N: int, K: int, x: int, B: int, y: int,
                       stream: int = 0) -> None:
    _check(lib().qmv_launch_noalloc(type, w, N, K, x, B, y, stream), "qmv_launch_noalloc")


def qmv_gateup_act_bytes(B: int, N: int, K: int) -> int:
    return int(lib().qmv_gateup_act_bytes(B, N, K))


def qmv_launch_gateup_swiglu(type: int, w_gate: int, w_up: int, N: int, K: int, x, B: int,
                             xq: int, h: int, stream: int = 0) -> None:
    _check(lib().qmv_launch_gateup_swiglu(type, w_gate, w_up, N, K, x, B, xq, h, stream),
           "qmv_launch_gateup_swiglu")


def qmv_launch_gateup_swiglu_q8(type: int, w_gate: int, w_up: int, N: int, K: int, x, B: int,
                                xq: int, h: int, hq: int, stream: int = 0) -> None:
    _check(lib().qmv_launch_gateup_swiglu_q8(type, w_gate, w_up, N, K, x, B, xq, h, hq, stream),
           "qmv_launch_gateup_swiglu_q8")


def qmv_launch_gateup_swiglu_q8k(type: int, w_gate: int, w_up: int, N: int, K: int, x, B: int,
                                 xq: int, h: int, stream: int = 0) -> None:
    _check(lib().qmv_launch_gateup_swiglu_q8k(type, w_gate, w_up, N, K, x, B, xq, h, stream),
           "qmv_launch_gateup_swiglu_q8k")


def qmv_act_bytes_q8k(rows: int, K: int) -> int:
    return int(lib().qmv_act_bytes_q8k(rows, K))


def quantize_act_q8_k(x, xq: int, rows: int, K: int, stream: int = 0) -> None:
    _check(lib().quantize_act_q8_k(x, xq, rows, K, stream), "quantize_act_q8_k")


def qmv_launch_q8k(type: int, w: int, N: int, K: int, x, B: int, xq: int, y: int,
                   stream: int = 0) -> None:
    _check(lib().qmv_launch_q8k(type, w, N, K, x, B, xq, y, stream), "qmv_launch_q8k")


def qmm_launch_q8k(type: int, w: int, N: int, K: int, x, M: int, xq: int, y: int,
                   stream: int = 0) -> None:
    _check(lib().qmm_launch_q8k(type, w, N, K, x, M, xq, y, stream), "qmm_launch_q8k")


def qmv_partials_q8k_launch(type: int, w: int, N: int, K: int, xq: int, M: int, P: int,
                            stream: int = 0) -> None:
    _check(lib().qmv_partials_q8k_launch(type, w, N, K, xq, M, P, stream),
           "qmv_partials_q8k_launch")


def qmv_prepared_bytes(type: int, N: int, K: int) -> int:
    return int(lib().qmv_prepared_bytes(type, N, K))


def qmv_prepare(type: int, w: int, N: int, K: int, wp: int, stream: int = 0) -> None:
    _check(lib().qmv_prepare(type, w, N, K, wp, stream), "qmv_prepare")


def qmm_launch_q8k_prepared(type: int, wp: int, N: int, K: int, x, M: int, xq: int, y: int,
                            stream: int = 0) -> None:
    _check(lib().qmm_launch_q8k_prepared(type, wp, N, K, x, M, xq, y, stream),
           "qmm_launch_q8k_prepared")


def qmm_partials_q8k_prepared_launch(type: int, wp: int, N: int, K: int, xq: int, M: int,
                                     P: int, stream: int = 0) -> None:
    _check(lib().qmm_partials_q8k_prepared_launch(type, wp, N, K, xq, M, P, stream),
           "qmm_partials_q8k_prepared_launch")


def qmv_add_rmsnorm_q8_0(x: int, res, w: int, eps: float, rows: int, K: int, h, y, xq: int,
                         stream: int = 0) -> None:
    _check(lib().qmv_add_rmsnorm_q8_0(x, res, w, eps, rows, K, h, y, xq, stream),
           "qmv_add_rmsnorm_q8_0")


def qmv_add_rmsnorm_q8_k(x: int, res, w: int, eps: float, rows: int, K: int, h, y, xq: int,
                         stream: int = 0) -> None:
    _check(lib().qmv_add_rmsnorm_q8_k(x, res, w, eps, rows, K, h, y, xq, stream),
           "qmv_add_rmsnorm_q8_k")


def qmv_kv_bytes(n_pages: int, page_tokens: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().qmv_kv_bytes(n_pages, page_tokens, kv_heads, head_dim))


def qmv_kv_append(kv: KvStruct, seqs: KvBatchStruct, q: int, q_stride: int, q_heads: int, k: int,
                  k_stride: int, v: int, v_stride: int, freq, rot: int, halves: int, q_out: int,
                  stream: int = 0) -> None:
    _check(lib().qmv_kv_append(kv, seqs, q, q_stride, q_heads, k, k_stride, v, v_stride, freq, rot,
                               halves, q_out, stream), "qmv_kv_append")


def qmv_kv_read(kv: KvStruct, seqs: KvBatchStruct, k: int, v: int, stream: int = 0) -> None:
    _check(lib().qmv_kv_read(kv, seqs, k, v, stream), "qmv_kv_read")


def qmv_kv_attention_bytes(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int,
                           max_len: int) -> int:
    return int(lib().qmv_kv_attention_bytes(T, B, q_heads, kv_heads, head_dim, max_len))


def qmv_kv_attention_rows(T: int, B: int, starts: bool, q_heads: int, kv_heads: int, head_dim: int,
                          max_len: int) -> int:
    return int(lib().qmv_kv_attention_rows(T, B, int(starts), q_heads, kv_heads, head_dim, max_len))


def qmv_kv_attention(kv: KvStruct, seqs: KvBatchStruct, q: int, q_stride: int, q_heads: int,
                     scale: float, window: int, out: int, work: int, stream: int = 0) -> None:
    _check(lib().qmv_kv_attention(kv, seqs, q, q_stride, q_heads, scale, window, out, work, stream),
           "qmv_kv_attention")


def qmv_moe_route(logits: int, T: int, E: int, score: int, bias, groups: int, top_groups: int,
                  group_top: int, top: int, renorm: int, scale: float, idx: int, weight: int,
                  stream: int = 0) -> None:
    _check(lib().qmv_moe_route(logits, T, E, score, bias, groups, top_groups, group_top, top, renorm,
                               scale, idx, weight, stream), "qmv_moe_route")


def qmv_moe_gateup_bytes(T: int, top: int, E: int, N: int, K: int) -> int:
    return int(lib().qmv_moe_gateup_bytes(T, top, E, N, K))


def qmv_moe_gateup_swiglu(type: int, w_gate: int, w_up: int, E: int, N: int, K: int, idx: int, T: int,
                          top: int, x, xq, h: int, work: int, stream: int = 0) -> None:
    _check(lib().qmv_moe_gateup_swiglu(type, w_gate, w_up, E, N, K, idx, T, top, x, xq, h, work,
                                       stream), "qmv_moe_gateup_swiglu")


def qmv_moe_down_bytes(T: int, top: int, E: int, N: int, K: int) -> int:
    return int(lib().qmv_moe_down_bytes(T, top, E, N, K))


def qmv_moe_down(type: int, w: int, E: int, N: int, K: int, idx: int, weight: int, T: int, top: int,
                 h, hq, y: int, work: int, stream: int = 0) -> None:
    _check(lib().qmv_moe_down(type, w, E, N, K, idx, weight, T, top, h, hq, y, work, stream),
           "qmv_moe_down")


def qmv_moe_rows(type: int, down: bool, T: int, top: int, E: int, N: int, K: int) -> int:
    return int(lib().qmv_moe_rows(type, int(down), T, top, E, N, K))


def qmv_strerror(code: int) -> str:
    return strerror(code)


# ------------------------------------------------------------ torch helpers --

def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dev(t, dtype, what):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def row_bytes(type: int, K: int) -> int:
    qk, nbytes = BLOCK[type]
    return (K // qk) * nbytes


def act_buffer(rows: int, K: int, device="cuda"):
    """Allocate an activation scratch tensor of qmv_act_bytes(rows, K) bytes."""
    import torch
    n = qmv_act_bytes(rows, K)
    if n == 0:
        raise ValueError(f"bad activation shape rows={rows} K={K}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def quantize(x, xq=None, stream=None, rows=None, K=None):
    """x: f32 [rows, K] device tensor -> xq scratch (Q8_0 blocks first).
    x None: re-stage the Q8_0 blocks already in xq (rows, K given)."""
    import torch
    if x is not None:
        rows, K = x.shape
    if xq is None:
        xq = act_buffer(rows, K, x.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    quantize_act_q8_0(xp, _dev(xq, torch.uint8, "xq"), rows, K, _stream(stream))
    return xq


def matvec(type: int, w, N: int, K: int, x=None, xq=None, B=None, y=None, stream=None):
    """Decode GEMV: y [B, N] f32 = x [B, K] @ W^T, B <= 16 (x None: reuse xq)."""
    import torch
    if x is not None:
        B = x.shape[0]
    if xq is None:
        xq = act_buffer(B, K, w.device)
    if y is None:
        y = torch.empty(B, N, dtype=torch.float32, device=w.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmv_launch(type, _dev(w, torch.uint8, "w"), N, K, xp, B, _dev(xq, torch.uint8, "xq"),
               _dev(y, torch.float32, "y"), _stream(stream))
    return y


def matvec_group(type: int, items, stream=None):
    """Grouped decode GEMVs: items are dicts with w, N, K and x (f32 [B, K])
    or xq (staged), optional xq / y.  Returns the list of y [B, N]."""
    import torch
    B = None
    descs, ys = [], []
    for it in items:
        x, xq = it.get("x"), it.get("xq")
        b = x.shape[0] if x is not None else it["B"]
        if B is None:
            B = b
        elif b != B:
            raise ValueError("all GEMVs of a group take the same number of rows")
        w = it["w"]
        y = it.get("y")
        if y is None:
            y = torch.empty(B, it["N"], dtype=torch.float32, device=w.device)
        xp = _dev(x, torch.float32, "x") if x is not None else None
        qp = _dev(xq, torch.uint8, "xq") if xq is not None else None
        descs.append(Gemv(_dev(w, torch.uint8, "w"), it["N"], it["K"], xp, qp,
                          _dev(y, torch.float32, "y")))
        ys.append(y)
    qmv_launch_group(type, B, descs, _stream(stream))
    return ys


def gateup_swiglu(type: int, w_gate, w_up, N: int, K: int, x=None, xq=None, B=None, h=None,
                  stream=None):
    """h [B, N] f32 = silu(x @ Wg^T) * (x @ Wu^T) (x None: use the staged xq)."""
    import torch
    if x is not None:
        B = x.shape[0]
    if xq is None:
        n = qmv_gateup_act_bytes(B, N, K)
        if n == 0:
            raise ValueError(f"bad shape B={B} N={N} K={K}")
        xq = torch.empty(n, dtype=torch.uint8, device=w_gate.device)
    if h is None:
        h = torch.empty(B, N, dtype=torch.float32, device=w_gate.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmv_launch_gateup_swiglu(type, _dev(w_gate, torch.uint8, "w_gate"),
                             _dev(w_up, torch.uint8, "w_up"), N, K, xp, B,
                             _dev(xq, torch.uint8, "xq"), _dev(h, torch.float32, "h"),
                             _stream(stream))
    return h


def gateup_swiglu_q8(type: int, w_gate, w_up, N: int, K: int, x=None, xq=None, B=None, h=None,
                     hq=None, stream=None):
    """(h [B, N] f32, hq) with hq the Q8_0 scratch of h for the down GEMV."""
    import torch
    if x is not None:
        B = x.shape[0]
    if xq is None:
        n = qmv_gateup_act_bytes(B, N, K)
        if n == 0:
            raise ValueError(f"bad shape B={B} N={N} K={K}")
        xq = torch.empty(n, dtype=torch.uint8, device=w_gate.device)
    if h is None:
        h = torch.empty(B, N, dtype=torch.float32, device=w_gate.device)
    if hq is None:
        hq = act_buffer(B, N, w_gate.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmv_launch_gateup_swiglu_q8(type, _dev(w_gate, torch.uint8, "w_gate"),
                                _dev(w_up, torch.uint8, "w_up"), N, K, xp, B,
                                _dev(xq, torch.uint8, "xq"), _dev(h, torch.float32, "h"),
                                _dev(hq, torch.uint8, "hq"), _stream(stream))
    return h, hq


def matmul(type: int, w, N: int, K: int, x=None, xq=None, M=None, y=None, stream=None):
    """Prefill GEMM: y [M, N] f32 = x [M, K] @ W^T."""
    import torch
    if x is not None:
        M = x.shape[0]
    if xq is None:
        xq = act_buffer(M, K, w.device)
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=w.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmm_launch(type, _dev(w, torch.uint8, "w"), N, K, xp, M, _dev(xq, torch.uint8, "xq"),
               _dev(y, torch.float32, "y"), _stream(stream))
    return y


def partials(type: int, w, N: int, K: int, xq, B: int, P=None, stream=None, gemm=False):
    """Test hook: int32 per-block partials [B, N, K/32] (Q4_K, Q4_1, Q5_1: [B, N, K/32, 2])
    of the kernel that qmv_launch (gemm: qmm_launch) runs for B rows."""
    import torch
    shape = (B, N, K // 32, 2) if type in (Q4_K, Q4_1, Q5_1) else (B, N, K // 32)
    if P is None:
        P = torch.empty(shape, dtype=torch.int32, device=w.device)
    fn = qmm_partials_launch if gemm else qmv_partials_launch
    fn(type, _dev(w, torch.uint8, "w"), N, K, _dev(xq, torch.uint8, "xq"), B,
       _dev(P, torch.int32, "P"), _stream(stream))
    return P


# ------------------------------------------- K-quants x Q8_K activations --

def quantize_q8k(x, xq=None, stream=None, rows=None, K=None):
    """x: f32 [rows, K] (K % 256 == 0) -> Q8_K scratch (blocks first); x None:
    rebuild the staging from the Q8_K blocks already in xq."""
    import torch
    if x is not None:
        rows, K = x.shape
    if xq is None:
        n = qmv_act_bytes_q8k(rows, K)
        if n == 0:
            raise ValueError(f"bad shape rows={rows} K={K}")
        xq = torch.empty(n, dtype=torch.uint8, device=x.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    quantize_act_q8_k(xp, _dev(xq, torch.uint8, "xq"), rows, K, _stream(stream))
    return xq


def matmul_q8k(type: int, w, N: int, K: int, x=None, xq=None, M=None, y=None, stream=None):
    """y [M, N] f32 = x [M, K] @ W^T on the Q8_K path (any M; x None: staged xq)."""
    import torch
    if x is not None:
        M = x.shape[0]
    if xq is None:
        xq = torch.empty(qmv_act_bytes_q8k(M, K), dtype=torch.uint8, device=w.device)
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=w.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmm_launch_q8k(type, _dev(w, torch.uint8, "w"), N, K, xp, M, _dev(xq, torch.uint8, "xq"),
                   _dev(y, torch.float32, "y"), _stream(stream))
    return y


def gateup_swiglu_q8k(type: int, w_gate, w_up, N: int, K: int, x=None, xq=None, B=None, h=None,
                      stream=None):
    """h [B, N] f32 = silu(x Wg^T) * (x Wu^T) on the Q8_K path (x None: staged xq)."""
    import torch
    if x is not None:
        B = x.shape[0]
    if xq is None:
        xq = torch.empty(qmv_act_bytes_q8k(B, K), dtype=torch.uint8, device=w_gate.device)
    if h is None:
        h = torch.empty(B, N, dtype=torch.float32, device=w_gate.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmv_launch_gateup_swiglu_q8k(type, _dev(w_gate, torch.uint8, "w_gate"),
                                 _dev(w_up, torch.uint8, "w_up"), N, K, xp, B,
                                 _dev(xq, torch.uint8, "xq"), _dev(h, torch.float32, "h"),
                                 _stream(stream))
    return h


def partials_q8k(type: int, w, N: int, K: int, xq, M: int, P=None, stream=None):
    """Superblock partials of the Q8_K path: Q4_K [M, N, K/256, 2], Q6_K [M, N, K/256]."""
    import torch
    shape = (M, N, K // 256, 2) if type == Q4_K else (M, N, K // 256)
    if P is None:
        P = torch.empty(shape, dtype=torch.int32, device=w.device)
    qmv_partials_q8k_launch(type, _dev(w, torch.uint8, "w"), N, K, _dev(xq, torch.uint8, "xq"), M,
                            _dev(P, torch.int32, "P"), _stream(stream))
    return P


def prepare(type: int, w, N: int, K: int, wp=None, stream=None):
    """The load-time repack of a Q4_K / Q6_K blob for the Q8_K prefill GEMM."""
    import torch
    n = qmv_prepared_bytes(type, N, K)
    if n == 0:
        raise ValueError(f"no repacked layout for type {type} N={N} K={K}")
    if wp is None:
        wp = torch.empty(n, dtype=torch.uint8, device=w.device)
    qmv_prepare(type, _dev(w, torch.uint8, "w"), N, K, _dev(wp, torch.uint8, "wp"), _stream(stream))
    return wp


def matmul_q8k_prepared(type: int, wp, N: int, K: int, x=None, xq=None, M=None, y=None,
                        stream=None):
    """y [M, N] f32 = x [M, K] @ W^T from repacked weights (x None: staged xq)."""
    import torch
    if x is not None:
        M = x.shape[0]
    if xq is None:
        xq = torch.empty(qmv_act_bytes_q8k(M, K), dtype=torch.uint8, device=wp.device)
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=wp.device)
    xp = _dev(x, torch.float32, "x") if x is not None else None
    qmm_launch_q8k_prepared(type, _dev(wp, torch.uint8, "wp"), N, K, xp, M,
                            _dev(xq, torch.uint8, "xq"), _dev(y, torch.float32, "y"),
                            _stream(stream))
    return y


def partials_q8k_prepared(type: int, wp, N: int, K: int, xq, M: int, P=None, stream=None):
    import torch
    shape = (M, N, K // 256, 2) if type == Q4_K else (M, N, K // 256)
    if P is None:
        P = torch.empty(shape, dtype=torch.int32, device=wp.device)
    qmm_partials_q8k_prepared_launch(type, _dev(wp, torch.uint8, "wp"), N, K,
                                     _dev(xq, torch.uint8, "xq"), M, _dev(P, torch.int32, "P"),
                                     _stream(stream))
    return P


# ------------------------------- norm into 8 bits, the paged 4-bit cache --

class _On:
    """The device and stream of a call on tensors of `device`: makes that
    device current for the launch, allocates on the call's stream, and gives
    the stream's handle.  stream: None (the device's current one), a torch
    stream, or a handle."""

    def __init__(self, device, stream):
        import torch
        self._guards = []
        if torch.cuda.current_device() != device.index:
            self._guards.append(torch.cuda.device(device))
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device)
            self.handle = stream.cuda_stream
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _on_device(device, stream, call):
    """call(handle) on a device and stream; the common case, the current stream
    of the current device, without a context (these calls take microseconds)."""
    import torch
    if stream is None and torch.cuda.current_device() == device.index:
        return call((_raw_stream or _find_raw_stream())(device.index))
    with _On(device, stream) as handle:
        return call(handle)


# device index -> the handle of its current stream; looked up by the first call,
# since importing this package does not import torch
_raw_stream = None


def _find_raw_stream():
    import torch
    global _raw_stream
    # the handle without a Stream object around it, where torch gives it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream


def _on(t, dtype, what, device):
    """The address of a contiguous tensor of a type on a device."""
    if t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    _dev(t, dtype, what)
    raise ValueError(f"{what} must be on {device}, got {t.device}")


def _new(t, like, dtype, what, shape=None):
    """(t, its address); if t is None a new tensor on like's device, of like's shape and type or
    of the given ones."""
    import torch
    if t is not None:
        return t, _on(t, dtype, what, like.device)
    if shape is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        t = like.new_empty(shape, dtype=dtype)
    return t, t.data_ptr()


def _add_rmsnorm(q8k, x, w, eps, res, h, y, xq, stream):
    import torch
    f32 = torch.float32
    if x.dim() != 2 or w.shape != x.shape[1:]:
        raise ValueError(f"x must be [rows, K] and w [K], got {tuple(x.shape)} and {tuple(w.shape)}")
    for t, what in ((res, "res"), (h, "h"), (y, "y")):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{what} must have x's shape {tuple(x.shape)}, got {tuple(t.shape)}")
    if h is not None and res is None:
        raise ValueError("h receives x + res: it goes with res")
    rows, K = x.shape
    xp = _dev(x, f32, "x")
    dev = x.device
    n = qmv_act_bytes_q8k(rows, K) if q8k else qmv_act_bytes(rows, K)
    if n == 0:
        raise ValueError(f"bad shape rows={rows} K={K}")
    if xq is not None and xq.numel() < n:
        raise ValueError(f"xq must hold {n} bytes, got {xq.numel()}")
    rp, wp = None if res is None else _on(res, f32, "res", dev), _on(w, f32, "w", dev)
    yp = None if y is None else _on(y, f32, "y", dev)

    def call(s):
        q, qp = _new(xq, x, torch.uint8, "xq", n)
        out, hp = (None, None) if res is None else _new(h, x, f32, "h")
        (qmv_add_rmsnorm_q8_k if q8k else qmv_add_rmsnorm_q8_0)(
            xp, rp, wp, eps, rows, K, hp, yp, qp, s)
        return out, q

    return _on_device(dev, stream, call)


def add_rmsnorm(x, w, eps, res=None, h=None, y=None, xq=None, stream=None):
    """(h, xq): h = x + res (None without res; h may be x or res), and the
    Q8_0 scratch of RMS norm(h) * w for matvec / matmul with x None.  x, res
    f32 [rows, K], w f32 [K]; y, if given, receives the norm's f32 values."""
    return _add_rmsnorm(False, x, w, eps, res, h, y, xq, stream)


def add_rmsnorm_q8k(x, w, eps, res=None, h=None, y=None, xq=None, stream=None):
    """add_rmsnorm with the Q8_K scratch (K % 256 == 0), for the Q8_K path."""
    return _add_rmsnorm(True, x, w, eps, res, h, y, xq, stream)


class KVCache:
    """A layer's keys and values in 4 bits: pages, a uint8 device tensor of
    whole pages (None: n_pages new ones), as qmv_kv describes them."""

    def __init__(self, pages, page_tokens: int, kv_heads: int, head_dim: int, n_pages=None,
                 device="cuda"):
        import torch
        one = qmv_kv_bytes(1, page_tokens, kv_heads, head_dim)
        if one == 0:
            raise ValueError(f"bad cache shape page_tokens={page_tokens} kv_heads={kv_heads} "
                             f"head_dim={head_dim}")
        if pages is None:
            if n_pages is None or n_pages < 1:
                raise ValueError(f"give pages, or n_pages for new ones, got n_pages={n_pages}")
            pages = torch.empty(one * n_pages, dtype=torch.uint8, device=device)
        ptr = _dev(pages, torch.uint8, "pages")
        if pages.numel() == 0 or pages.numel() % one:
            raise ValueError(f"pages must be whole pages of {one} bytes, got {pages.numel()} bytes")
        self.pages, self.kv_heads, self.head_dim = pages, kv_heads, head_dim
        self.page_tokens = page_tokens
        self.c = KvStruct(ptr, pages.numel() // one, page_tokens, kv_heads, head_dim)


class KVBatch:
    """The sequences of a call: table int32 [B, pages], lens int32 [B] (with the
    call's own tokens), q_start int32 [B + 1] or None (one row a sequence), T
    rows in all, max_len a bound of the lengths (None: what the table holds,
    for a cache of page_tokens)."""

    def __init__(self, table, lens, q_start=None, T=None, max_len=None, page_tokens=None):
        import torch
        i32 = torch.int32
        if table.dim() != 2 or lens.shape != table.shape[:1]:
            raise ValueError(f"table must be [B, pages] and lens [B], got {tuple(table.shape)} and "
                             f"{tuple(lens.shape)}")
        B, stride = table.shape
        if q_start is not None and q_start.shape != (B + 1,):
            raise ValueError(f"q_start must be [{B + 1}], got {tuple(q_start.shape)}")
        if T is None:
            if q_start is not None:
                raise ValueError("T, the number of rows, goes with q_start")
            T = B
        if max_len is None:
            if page_tokens is None:
                raise ValueError("give max_len, or page_tokens for all that the table can name")
            max_len = stride * page_tokens
        dev = table.device
        self.c = KvBatchStruct(_dev(table, i32, "table"), stride, _on(lens, i32, "lens", dev),
                               None if q_start is None else _on(q_start, i32, "q_start", dev),
                               B, T, max_len)
        self.table, self.lens, self.q_start = table, lens, q_start
        self.B, self.T, self.max_len = B, T, max_len


def _rows(t, T, width, what, device):
    """(address, row stride) of T rows of `width` f32 with adjacent elements."""
    import torch
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    if t.dtype is not torch.float32:
        raise TypeError(f"{what} must be torch.float32, got {t.dtype}")
    if t.shape != (T, width) or t.stride(1) != 1:
        raise ValueError(f"{what} must be [{T}, {width}] with adjacent elements, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if T > 1 else width


def _heads(q, cache, what="q"):
    if q.dim() != 2 or q.shape[1] % cache.head_dim:
        raise ValueError(f"{what} must be [T, heads * {cache.head_dim}], got {tuple(q.shape)}")
    return q.shape[1] // cache.head_dim


def _here(cache, batch):
    dev = cache.pages.device
    if batch.table.device != dev:
        raise ValueError(f"table must be on {dev}, got {batch.table.device}")
    return dev


def kv_append(cache: KVCache, batch: KVBatch, q, k, v, freq=None, halves: bool = False, q_out=None,
              stream=None):
    """Rotates q [T, q_heads * D] and k [T, kv_heads * D] by their positions
    (freq f64 [rot / 2], None: no rotation) and appends k and v to the cache.
    Returns the rotated q (q_out, or a new tensor, whose skipped rows are
    not written)."""
    import torch
    dev, T = _here(cache, batch), batch.T
    heads, width = _heads(q, cache), cache.kv_heads * cache.head_dim
    qp, qs = _rows(q, T, q.shape[1], "q", dev)
    kp, ks = _rows(k, T, width, "k", dev)
    vp, vs = _rows(v, T, width, "v", dev)
    if q_out is not None and q_out.shape != q.shape:
        raise ValueError(f"q_out must have q's shape {tuple(q.shape)}, got {tuple(q_out.shape)}")
    rot, fp = 0, None
    if freq is not None:
        rot, fp = 2 * freq.numel(), _on(freq, torch.float64, "freq", dev)

    def call(s):
        out, op = _new(q_out, q, torch.float32, "q_out")
        qmv_kv_append(cache.c, batch.c, qp, qs, heads, kp, ks, vp, vs, fp, rot, int(halves), op, s)
        return out

    return _on_device(dev, stream, call)


def kv_read(cache: KVCache, batch: KVBatch, k=None, v=None, stream=None):
    """(k, v) [T, kv_heads * D] f32: the values held for the rows' tokens."""
    import torch
    dev = _here(cache, batch)
    shape = (batch.T, cache.kv_heads * cache.head_dim)
    for t, what in ((k, "k"), (v, "v")):
        if t is not None and t.shape != shape:
            raise ValueError(f"{what} must be {shape}, got {tuple(t.shape)}")

    def call(s):
        ko, kp = _new(k, cache.pages, torch.float32, "k", shape)
        vo, vp = _new(v, ko, torch.float32, "v")
        qmv_kv_read(cache.c, batch.c, kp, vp, s)
        return ko, vo

    return _on_device(dev, stream, call)


def kv_attention(cache: KVCache, batch: KVBatch, q, scale: float, window: int = 0, out=None,
                 work=None, stream=None):
    """out [T, q_heads * D] f32: causal attention of the rows q over the cache
    (window: only the last `window` positions; 0: all)."""
    import torch
    dev, T = _here(cache, batch), batch.T
    heads = _heads(q, cache)
    qp, qs = _rows(q, T, q.shape[1], "q", dev)
    if out is not None and out.shape != q.shape:
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    n = qmv_kv_attention_bytes(T, batch.B, heads, cache.kv_heads, cache.head_dim, batch.max_len)
    if work is not None and work.numel() < n:
        raise ValueError(f"work must hold {n} bytes, got {work.numel()}")

    def call(s):
        o, op = _new(out, q, torch.float32, "out")
        ws, wp = _new(work, q, torch.uint8, "work", n)
        qmv_kv_attention(cache.c, batch.c, qp, qs, heads, scale, window, op, wp, s)
        return o

    return _on_device(dev, stream, call)


# ------------------------------------------------------ mixture of experts --

def moe_route(logits, top: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_top: int = 1, renorm: bool = True, scale: float = 1.0, idx=None, weight=None,
              stream=None):
    """(idx int32, weight f32), both [T, top]: the experts that the tokens of logits [T, E] go to and
    their weights, as qmv_moe_route describes them (a slot without an expert: -1 and 0)."""
    import torch
    f32 = torch.float32
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got {tuple(logits.shape)}")
    if score not in MOE_SCORES:
        raise ValueError(f"score must be one of {sorted(MOE_SCORES)}, got {score!r}")
    T, E = logits.shape
    lp = _dev(logits, f32, "logits")
    dev = logits.device
    bp = None
    if bias is not None:
        if bias.shape != (E,):
            raise ValueError(f"bias must be [{E}], got {tuple(bias.shape)}")
        bp = _on(bias, f32, "bias", dev)
    for t, what in ((idx, "idx"), (weight, "weight")):
        if t is not None and t.shape != (T, top):
            raise ValueError(f"{what} must be [{T}, {top}], got {tuple(t.shape)}")

    def call(s):
        i, ip = _new(idx, logits, torch.int32, "idx", (T, top))
        w, wp = _new(weight, logits, f32, "weight", (T, top))
        qmv_moe_route(lp, T, E, MOE_SCORES[score], bp, groups, top_groups, group_top, top, int(renorm),
                      scale, ip, wp, s)
        return i, w

    return _on_device(dev, stream, call)


def _experts(type, w, N, K, what):
    """(address, number) of the matrices of an expert tensor."""
    import torch
    if type not in BLOCK:
        raise QmvError(-1, what)
    if N < 1 or K < 1 or K % BLOCK[type][0]:
        raise QmvError(-2, what)
    p = _dev(w, torch.uint8, what)
    one = N * row_bytes(type, K)
    if w.numel() == 0 or w.numel() % one:
        raise ValueError(f"{what} must be whole {N} x {K} matrices of {one} bytes, got {w.numel()} bytes")
    return p, w.numel() // one


def _pairs(idx, dev):
    import torch
    if idx.dim() != 2:
        raise ValueError(f"idx must be [T, top], got {tuple(idx.shape)}")
    return (_on(idx, torch.int32, "idx", dev), *idx.shape)


def _rows_or_blocks(x, xq, rows, K, what, dev):
    """Addresses of f32 rows or of their Q8_0 blocks, one of the two None."""
    import torch
    if (x is None) == (xq is None):
        raise ValueError(f"give {what} or {what}q, one of them")
    if x is not None:
        if x.numel() != rows * K or x.shape[-1] != K:
            raise ValueError(f"{what} must hold {rows} rows of {K}, got {tuple(x.shape)}")
        return _on(x, torch.float32, what, dev), None
    if xq.numel() < rows * (K // 32) * 34:
        raise ValueError(f"{what}q must hold {rows * (K // 32) * 34} bytes, got {xq.numel()}")
    return None, _on(xq, torch.uint8, what + "q", dev)


def _moe_work(work, n):
    if n == 0:
        raise ValueError("bad shape of a mixture of experts: see the limits in qmv.h")
    if work is not None and work.numel() < n:
        raise ValueError(f"work must hold {n} bytes, got {work.numel()}")


def moe_gateup_swiglu(type: int, w_gate, w_up, N: int, K: int, idx, x=None, xq=None, h=None, work=None,
                      stream=None):
    """h [T, top, N] f32 = silu(Wg[e] x) * (Wu[e] x) for the experts e of idx int32 [T, top]: w_gate
    and w_up hold E matrices N x K each; x f32 [T, K], or xq with the rows' Q8_0 blocks."""
    import torch
    gp, E = _experts(type, w_gate, N, K, "w_gate")
    dev = w_gate.device
    if w_up.numel() != w_gate.numel():
        raise ValueError(f"w_up must hold {w_gate.numel()} bytes as w_gate does, got {w_up.numel()}")
    up = _on(w_up, torch.uint8, "w_up", dev)
    ip, T, top = _pairs(idx, dev)
    xp, qp = _rows_or_blocks(x, xq, T, K, "x", dev)
    if h is not None and h.numel() != T * top * N:
        raise ValueError(f"h must hold {T * top} rows of {N}, got {tuple(h.shape)}")
    n = qmv_moe_gateup_bytes(T, top, E, N, K)
    _moe_work(work, n)

    def call(s):
        out, hp = _new(h, w_gate, torch.float32, "h", (T, top, N))
        ws, wp = _new(work, w_gate, torch.uint8, "work", n)
        qmv_moe_gateup_swiglu(type, gp, up, E, N, K, ip, T, top, xp, qp, hp, wp, s)
        return out

    return _on_device(dev, stream, call)


def moe_down(type: int, w, N: int, K: int, idx, weight, h=None, hq=None, y=None, work=None, stream=None):
    """y [T, N] f32 = sum over the slots of weight * (W[e] h) for the experts e of idx int32 [T, top]:
    w holds E matrices N x K; weight f32 [T, top]; h f32 [T, top, K], or hq with the rows' Q8_0 blocks."""
    import torch
    wp, E = _experts(type, w, N, K, "w")
    dev = w.device
    ip, T, top = _pairs(idx, dev)
    if weight.shape != idx.shape:
        raise ValueError(f"weight must have idx's shape {tuple(idx.shape)}, got {tuple(weight.shape)}")
    sp = _on(weight, torch.float32, "weight", dev)
    hp, qp = _rows_or_blocks(h, hq, T * top, K, "h", dev)
    if y is not None and y.shape != (T, N):
        raise ValueError(f"y must be [{T}, {N}], got {tuple(y.shape)}")
    n = qmv_moe_down_bytes(T, top, E, N, K)
    _moe_work(work, n)

    def call(s):
        out, yp = _new(y, w, torch.float32, "y", (T, N))
        ws, kp = _new(work, w, torch.uint8, "work", n)
        qmv_moe_down(type, wp, E, N, K, ip, sp, T, top, hp, qp, yp, kp, s)
        return out

    return _on_device(dev, stream, call)
