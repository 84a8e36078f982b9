// Device helpers shared by the kernels of the paged 4-bit cache.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_step.h"

namespace qmv {
namespace {

__device__ __forceinline__ float half_value(uint16_t h) {
    _Float16 f;
    __builtin_memcpy(&f, &h, 2);
    return (float)f;
}

// Element e (0..7) of a K word sits in nibble K_NIB(e): 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ int k_nibble(int e) { return (e >> 1) | ((e & 1) << 2); }

// A sequence as a call sees it: rows [q0, q0 + n) at positions len - n ... .
struct Seq {
    int q0, n, len;
};

// Lengths and starts come from device memory and are not trusted: a length is
// cut to what the table can name and to max_len, a run of rows to the T rows
// of the call.
__device__ __forceinline__ Seq seq_of(const KvArgs& kv, int b) {
    Seq s;
    s.q0 = kv.q_start ? kv.q_start[b] : b;
    const int end = kv.q_start ? kv.q_start[b + 1] : b + 1;
    if (s.q0 < 0 || end < s.q0 || end > kv.T) s.q0 = s.n = 0;
    else s.n = end - s.q0;
    const int64_t most = kv.table_stride << kv.log2p;
    int len = kv.lens[b];
    if (len > kv.max_len) len = kv.max_len;
    if ((int64_t)len > most) len = (int)most;
    s.len = len < 0 ? 0 : len;
    return s;
}

// The sequence of row t: the last b with start[b] <= t, by the whole wave 64
// starts at a time.  Uniform over the wave; -1 if there is none.
__device__ __forceinline__ int seq_of_row(const KvArgs& kv, int t) {
    if (!kv.q_start) return t < kv.B ? t : -1;
    const int lane = threadIdx.x & 63;
    int below = 0;
    for (int b0 = 0; b0 <= kv.B; b0 += 64) {
        const int b = b0 + lane;
        const unsigned long long m = __ballot(b <= kv.B && kv.q_start[b] <= t);
        below += __popcll(m);
        if (m != ~0ull) break;
    }
    return below >= 1 && below <= kv.B ? below - 1 : -1;
}

// The page that holds position p of sequence b, or -1 if the table names none.
__device__ __forceinline__ int page_of(const KvArgs& kv, int b, int p) {
    const int pg = kv.table[(int64_t)b * kv.table_stride + (p >> kv.log2p)];
    return pg >= 0 && (int64_t)pg < kv.n_pages ? pg : -1;
}

__device__ __forceinline__ uint8_t* head_of(const KvArgs& kv, int page, int head) {
    return kv.pages + ((int64_t)page * kv.Hkv + head) * kv.head_bytes;
}

}  // namespace
}  // namespace qmv
