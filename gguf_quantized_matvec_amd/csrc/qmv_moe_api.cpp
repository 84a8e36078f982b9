// C-ABI of the mixture-of-experts operators (declared in include/qmv.h):
// argument checks on the host, a device check, and dispatch.  As in qmv_api.cpp
// nothing is allocated or synchronised, and a refused call has no effect.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/qmv.h"
#include "qmv_device.h"
#include "qmv_moe.h"

using qmv::aligned;
using qmv::check_device;
using qmv::launched;

namespace {

bool pairs_ok(int64_t T, int64_t E, int top) {
    return T >= 1 && T <= QMV_MOE_MAX_PAIRS && top >= 1 && top <= QMV_MOE_MAX_TOP &&
           T * top <= QMV_MOE_MAX_PAIRS && E >= 1 && E <= QMV_MOE_MAX_EXPERTS;
}

// rows: of activations
bool shape_ok(int64_t N, int64_t K, int64_t rows) {
    return N >= 1 && N <= QMV_MAX_M && K >= 32 && K <= QMV_MAX_K && K % 32 == 0 &&
           rows * K < ((int64_t)1 << 33);
}

int check_type(int type, int64_t K) {
    switch (type) {
    case QMV_Q8_0:
    case QMV_Q4_0:
    case QMV_Q5_0:
    case QMV_Q4_1:
    case QMV_Q5_1:
    case QMV_Q8_1: return QMV_OK;
    case QMV_Q4_K:
    case QMV_Q6_K: return K % 256 ? QMV_EINVAL_SHAPE : QMV_OK;
    }
    return QMV_EINVAL_TYPE;
}

// A buffer of a call; p NULL: one that the call does not have.
struct Buffer {
    const void* p;
    int64_t bytes;
};
// Whether the outputs (the first `outs` of them) overlap each other or an input.
template <int N> bool overlap(const Buffer (&b)[N], int outs) {
    for (int i = 0; i < outs; i++)
        for (int j = i + 1; j < N; j++) {
            const uintptr_t u = reinterpret_cast<uintptr_t>(b[i].p), v = reinterpret_cast<uintptr_t>(b[j].p);
            if (u && v && (u < v ? v - u < (uint64_t)b[i].bytes : u - v < (uint64_t)b[j].bytes)) return true;
        }
    return false;
}
int64_t blocks_bytes(int64_t rows, int64_t K) { return rows * (K / 32) * 34; }

}  // namespace

extern "C" {

int qmv_moe_route(const float* logits, int64_t T, int64_t E, int score, const float* bias,
                  int groups, int top_groups, int group_top, int top, int renorm, float scale,
                  int32_t* idx, float* weight, void* stream) {
    if (!pairs_ok(T, E, top) || (score != QMV_MOE_SOFTMAX && score != QMV_MOE_SIGMOID))
        return QMV_EINVAL_SHAPE;
    if (groups < 1 || groups > 64 || E % groups || top_groups < 1 || top_groups > groups ||
        group_top < 1 || group_top > 2 || top > top_groups * (E / groups))
        return QMV_EINVAL_SHAPE;
    if (!isfinite(scale)) return QMV_EINVAL_SHAPE;
    if (!logits || !idx || !weight || !aligned(logits, 4) || !aligned(bias, 4) ||
        !aligned(idx, 4) || !aligned(weight, 4))
        return QMV_EINVAL_PTR;
    if (overlap({{idx, T * top * 4}, {weight, T * top * 4}, {logits, T * E * 4}, {bias, E * 4}}, 2))
        return QMV_EINVAL_PTR;
    const int rc = check_device();
    if (rc) return rc;
    const qmv::RouteArgs a{logits, bias, (int32_t)T, (int32_t)E, groups, top_groups, group_top, top,
                           score == QMV_MOE_SIGMOID, renorm != 0, scale, idx, weight};
    return launched(qmv::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

size_t qmv_moe_gateup_bytes(int64_t T, int top, int64_t E, int64_t N, int64_t K) {
    if (!pairs_ok(T, E, top) || !shape_ok(N, K, T)) return 0;
    return (size_t)qmv::moe_work_bytes(T * top, top, top, E, K);
}

int qmv_moe_gateup_swiglu(int type, const void* w_gate, const void* w_up, int64_t E, int64_t N,
                          int64_t K, const int32_t* idx, int64_t T, int top, const float* x,
                          const void* xq, float* h, void* work, void* stream) {
    int rc = check_type(type, K);
    if (rc) return rc;
    if (!pairs_ok(T, E, top) || !shape_ok(N, K, T)) return QMV_EINVAL_SHAPE;
    if (!w_gate || !w_up || !aligned(w_gate, 16) || !aligned(w_up, 16)) return QMV_EINVAL_PTR;
    if ((x != nullptr) == (xq != nullptr) || !aligned(x, 4) || !aligned(xq, 16))
        return QMV_EINVAL_PTR;
    if (!idx || !h || !work || !aligned(idx, 4) || !aligned(h, 4) || !aligned(work, 16))
        return QMV_EINVAL_PTR;
    const int64_t w_bytes = E * N * qmv::row_bytes(type, K);
    if (overlap({{h, T * top * N * 4}, {work, (int64_t)qmv_moe_gateup_bytes(T, top, E, N, K)},
                 {x, T * K * 4}, {xq, blocks_bytes(T, K)}, {idx, T * top * 4},
                 {w_gate, w_bytes}, {w_up, w_bytes}}, 2))
        return QMV_EINVAL_PTR;
    if ((rc = check_device())) return rc;
    const qmv::MoeArgs a{type, static_cast<const uint8_t*>(w_gate),
                         static_cast<const uint8_t*>(w_up), E, N, K, idx, T * top, top, top, x,
                         static_cast<const uint8_t*>(xq), static_cast<uint8_t*>(work), h};
    return launched(qmv::launch_moe_product(a, static_cast<hipStream_t>(stream)));
}

size_t qmv_moe_down_bytes(int64_t T, int top, int64_t E, int64_t N, int64_t K) {
    if (!pairs_ok(T, E, top) || !shape_ok(N, K, T * top)) return 0;
    return (size_t)(qmv::moe_work_bytes(T * top, top, 1, E, K) + qmv::align256(T * top * N * 4));
}

int qmv_moe_down(int type, const void* w, int64_t E, int64_t N, int64_t K, const int32_t* idx,
                 const float* weight, int64_t T, int top, const float* h, const void* hq, float* y,
                 void* work, void* stream) {
    int rc = check_type(type, K);
    if (rc) return rc;
    if (!pairs_ok(T, E, top) || !shape_ok(N, K, T * top)) return QMV_EINVAL_SHAPE;
    if (!w || !aligned(w, 16)) return QMV_EINVAL_PTR;
    if ((h != nullptr) == (hq != nullptr) || !aligned(h, 4) || !aligned(hq, 16))
        return QMV_EINVAL_PTR;
    if (!idx || !weight || !y || !work || !aligned(idx, 4) || !aligned(weight, 4) ||
        !aligned(y, 4) || !aligned(work, 16))
        return QMV_EINVAL_PTR;
    if (overlap({{y, T * N * 4}, {work, (int64_t)qmv_moe_down_bytes(T, top, E, N, K)},
                 {h, T * top * K * 4}, {hq, blocks_bytes(T * top, K)}, {idx, T * top * 4},
                 {weight, T * top * 4}, {w, E * N * qmv::row_bytes(type, K)}}, 2))
        return QMV_EINVAL_PTR;
    if ((rc = check_device())) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* wk = static_cast<uint8_t*>(work);
    float* yp = reinterpret_cast<float*>(wk + qmv::moe_work_bytes(T * top, top, 1, E, K));
    const qmv::MoeArgs a{type, static_cast<const uint8_t*>(w), nullptr, E, N, K, idx, T * top, top,
                         1, h, static_cast<const uint8_t*>(hq), wk, yp};
    return launched(qmv::launch_moe_down(a, weight, y, s));
}

int qmv_moe_rows(int type, int down, int64_t T, int top, int64_t E, int64_t N, int64_t K) {
    if (check_type(type, K) || !pairs_ok(T, E, top) || !shape_ok(N, K, down ? T * top : T)) return 0;
    qmv::MoeArgs a{};
    static const uint8_t some = 0;
    a.type = type;
    a.w = &some;
    a.w2 = down ? nullptr : &some;
    a.E = E;
    a.N = N;
    a.K = K;
    a.P = T * top;
    a.top = top;
    a.per = down ? 1 : top;
    return qmv::moe_gemv_fits(a) ? 1 : qmv::moe_rows(a);
}

}  // extern "C"
