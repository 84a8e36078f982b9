// C-ABI of the operators around the quantised products (declared in
// include/qmv.h): argument checks on the host, a device check, and dispatch.
// As in qmv_api.cpp nothing is allocated or synchronised, and a refused call
// has no effect.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmv.h"
#include "qmv_device.h"
#include "qmv_step.h"

using qmv::aligned;
using qmv::check_device;
using qmv::launched;

namespace {

int add_rmsnorm(const float* x, const float* res, const float* w, float eps, int64_t rows,
                int64_t K, float* h, float* y, void* xq, void* stream, bool q8k) {
    if (rows < 1 || rows > QMV_MAX_M || K < 32 || K > QMV_MAX_K || K % (q8k ? 256 : 32))
        return QMV_EINVAL_SHAPE;
    if (!(eps >= 0.0f && eps <= 1.0f)) return QMV_EINVAL_SHAPE;
    if (!x || !w || !xq || !aligned(xq, 16) || !aligned(x, 4) || !aligned(w, 4))
        return QMV_EINVAL_PTR;
    // the sum is handed on exactly when something is added
    if ((res != nullptr) != (h != nullptr)) return QMV_EINVAL_PTR;
    if (!aligned(res, 4) || !aligned(h, 4) || !aligned(y, 4)) return QMV_EINVAL_PTR;
    if (y && (y == x || y == res || y == h || y == w)) return QMV_EINVAL_PTR;
    if (h == w) return QMV_EINVAL_PTR;
    const int rc = check_device();
    if (rc) return rc;
    return launched(qmv::launch_add_rmsnorm(x, res, w, eps, rows, K, h, y,
                                            static_cast<uint8_t*>(xq), q8k,
                                            static_cast<hipStream_t>(stream)));
}

bool cache_shape_ok(int64_t n_pages, int page_tokens, int kv_heads, int head_dim) {
    return n_pages >= 1 && n_pages <= INT32_MAX && page_tokens >= 16 && page_tokens <= 1024 &&
           (page_tokens & (page_tokens - 1)) == 0 && kv_heads >= 1 && kv_heads <= QMV_KV_MAX_HEADS &&
           head_dim >= 32 && head_dim <= 256 && head_dim % 32 == 0;
}

// Checks a cache and the sequences of a call and gives them as the kernels
// take them.
int kv_args(const qmv_kv* kv, const qmv_kv_batch* s, qmv::KvArgs* a) {
    if (!kv || !s) return QMV_EINVAL_PTR;
    if (!cache_shape_ok(kv->n_pages, kv->page_tokens, kv->kv_heads, kv->head_dim))
        return QMV_EINVAL_SHAPE;
    if (s->B < 1 || s->B > QMV_KV_MAX_ROWS || s->T < 1 || s->T > QMV_KV_MAX_ROWS ||
        s->table_stride < 1 || s->table_stride > INT32_MAX)
        return QMV_EINVAL_SHAPE;
    if (!s->q_start && s->T != s->B) return QMV_EINVAL_SHAPE;
    if (s->max_len < 1 || s->max_len > QMV_KV_MAX_LEN ||
        s->max_len > s->table_stride * kv->page_tokens)
        return QMV_EINVAL_SHAPE;
    if (!kv->pages || !aligned(kv->pages, 16)) return QMV_EINVAL_PTR;
    if (!s->table || !s->lens || !aligned(s->table, 4) || !aligned(s->lens, 4) ||
        !aligned(s->q_start, 4))
        return QMV_EINVAL_PTR;
    int log2p = 4;
    while ((1 << log2p) < kv->page_tokens) log2p++;
    const int nb = kv->head_dim / 32;
    *a = qmv::KvArgs{static_cast<uint8_t*>(kv->pages), kv->n_pages, s->table, s->table_stride,
                     s->lens, s->q_start, (int32_t)s->B, (int32_t)s->T, (int32_t)s->max_len,
                     log2p, kv->kv_heads, nb, (int64_t)(36 * nb) << log2p};
    return QMV_OK;
}

bool q_heads_ok(int q_heads, int kv_heads) {
    return q_heads >= kv_heads && q_heads <= QMV_KV_MAX_HEADS && q_heads % kv_heads == 0;
}

// The workgroups of an attention, one per row tile and key/value head (8 rows or more a tile, one
// tile more per sequence): a grid of 256 threads each holds fewer than 2^24.
bool tiles_ok(int64_t T, int64_t B, int64_t q_heads, int64_t kv_heads) {
    return T * q_heads / 8 + B * kv_heads < (1 << 24);
}

bool attention_shape_ok(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim,
                        int64_t max_len) {
    return cache_shape_ok(1, 16, kv_heads, head_dim) && q_heads_ok(q_heads, kv_heads) && B >= 1 &&
           B <= QMV_KV_MAX_ROWS && T >= 1 && T <= QMV_KV_MAX_ROWS && max_len >= 1 &&
           max_len <= QMV_KV_MAX_LEN && tiles_ok(T, B, q_heads, kv_heads);
}

}  // namespace

extern "C" {

int qmv_add_rmsnorm_q8_0(const float* x, const float* res, const float* w, float eps, int64_t rows,
                         int64_t K, float* h, float* y, void* xq, void* stream) {
    return add_rmsnorm(x, res, w, eps, rows, K, h, y, xq, stream, false);
}

int qmv_add_rmsnorm_q8_k(const float* x, const float* res, const float* w, float eps, int64_t rows,
                         int64_t K, float* h, float* y, void* xq, void* stream) {
    return add_rmsnorm(x, res, w, eps, rows, K, h, y, xq, stream, true);
}

size_t qmv_kv_bytes(int64_t n_pages, int page_tokens, int kv_heads, int head_dim) {
    if (!cache_shape_ok(n_pages, page_tokens, kv_heads, head_dim)) return 0;
    return (size_t)n_pages * kv_heads * page_tokens * (36 * (head_dim / 32));
}

int qmv_kv_append(const qmv_kv* kv, const qmv_kv_batch* seqs, const float* q, int64_t q_stride,
                  int q_heads, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                  const double* freq, int rot, int halves, float* q_out, void* stream) {
    qmv::AppendArgs a;
    int rc = kv_args(kv, seqs, &a.kv);
    if (rc) return rc;
    const int64_t D = kv->head_dim, qd = q_heads * D, kd = kv->kv_heads * D;
    if (!q_heads_ok(q_heads, kv->kv_heads) || rot < 0 || rot > D || rot % 2 || q_stride < qd ||
        k_stride < kd || v_stride < kd)
        return QMV_EINVAL_SHAPE;
    if (!q || !k || !v || !q_out || (rot && !freq) || !aligned(q, 4) || !aligned(k, 4) ||
        !aligned(v, 4) || !aligned(q_out, 4) || !aligned(freq, 8))
        return QMV_EINVAL_PTR;
    if (q_out == q && q_stride != qd) return QMV_EINVAL_PTR;  // in place: the same rows
    if (q_out == k || q_out == v) return QMV_EINVAL_PTR;
    if ((rc = check_device())) return rc;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.freq = freq;
    a.rot = rot;
    a.halves = halves != 0;
    a.Hq = q_heads;
    a.q_out = q_out;
    return launched(qmv::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

int qmv_kv_read(const qmv_kv* kv, const qmv_kv_batch* seqs, float* k, float* v, void* stream) {
    qmv::KvArgs a;
    int rc = kv_args(kv, seqs, &a);
    if (rc) return rc;
    if (!k || !v || !aligned(k, 4) || !aligned(v, 4)) return QMV_EINVAL_PTR;
    if ((rc = check_device())) return rc;
    return launched(qmv::launch_kv_read(a, k, v, static_cast<hipStream_t>(stream)));
}

size_t qmv_kv_attention_bytes(int64_t T, int64_t B, int q_heads, int kv_heads, int head_dim,
                              int64_t max_len) {
    if (!attention_shape_ok(T, B, q_heads, kv_heads, head_dim, max_len)) return 0;
    return (size_t)qmv::kv_attention_bytes(T, B, q_heads, kv_heads, head_dim / 32, max_len);
}

int qmv_kv_attention_rows(int64_t T, int64_t B, int starts, int q_heads, int kv_heads,
                          int head_dim, int64_t max_len) {
    if (!attention_shape_ok(T, B, q_heads, kv_heads, head_dim, max_len) || (!starts && T != B))
        return 0;
    return qmv::kv_attention_rows(T, B, starts != 0, q_heads, kv_heads, head_dim / 32, max_len);
}

int qmv_kv_attention(const qmv_kv* kv, const qmv_kv_batch* seqs, const float* q, int64_t q_stride,
                     int q_heads, float scale, int64_t window, float* out, void* work,
                     void* stream) {
    qmv::AttnArgs a;
    int rc = kv_args(kv, seqs, &a.kv);
    if (rc) return rc;
    if (!q_heads_ok(q_heads, kv->kv_heads) || q_stride < (int64_t)q_heads * kv->head_dim ||
        q_stride % 4 || window < 0 || !(scale > 0.0f && scale <= 1e6f) ||
        !tiles_ok(seqs->T, seqs->B, q_heads, kv->kv_heads))
        return QMV_EINVAL_SHAPE;
    if (!q || !out || !work || !aligned(q, 16) || !aligned(out, 16) || !aligned(work, 16) ||
        out == q)
        return QMV_EINVAL_PTR;
    if ((rc = check_device())) return rc;
    a.q = q;
    a.q_stride = q_stride;
    a.Hq = q_heads;
    a.scale = scale;
    a.window = window >= seqs->max_len ? 0 : (int32_t)window;  // longer than any sequence: none
    a.out = out;
    a.work = static_cast<float*>(work);
    return launched(qmv::launch_kv_attention(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
