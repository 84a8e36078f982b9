// Internal declarations of the operators around the quantised products (the
// residual add with RMS norm, the paged 4-bit key/value cache): shared by
// their C-ABI layer (qmv_step_api.cpp) and kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {

// Residual add and RMS norm into a staged activation scratch (qmv_norm.hip):
// q8k selects the Q8_K layout, else Q8_0 with the staging staging_for() gives.
int launch_add_rmsnorm(const float* x, const float* res, const float* w, float eps, int64_t rows,
                       int64_t K, float* h, float* y, uint8_t* xq, bool q8k, hipStream_t s);

// The paged cache and the sequences of one call, as the kernels take them.
// A page holds 1 << log2p tokens; head h of page p is the (p * Hkv + h)-th
// block of head_bytes: K codes, V codes, K scales, V scales.
struct KvArgs {
    uint8_t* pages;
    int64_t n_pages;
    const int32_t* table;     // [B][table_stride] page of each run of 1 << log2p positions
    int64_t table_stride;
    const int32_t* lens;      // [B] tokens of each sequence, the call's own among them
    const int32_t* q_start;   // [B + 1] first row of each sequence, or NULL: one row each
    int32_t B, T, max_len;
    int32_t log2p, Hkv, nb;   // nb = head_dim / 32
    int64_t head_bytes;       // (36 nb) << log2p
};

struct AppendArgs {
    KvArgs kv;
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // in floats
    const double* freq;                    // [rot / 2] radians per position
    int32_t rot, halves, Hq;
    float* q_out;                          // [T][Hq * D]
};

struct AttnArgs {
    KvArgs kv;
    const float* q;
    int64_t q_stride;
    int32_t Hq;
    float scale;
    int32_t window;   // 0: none
    float* out;       // [T][Hq * D]
    float* work;
};

int launch_kv_append(const AppendArgs& a, hipStream_t s);
int launch_kv_read(const KvArgs& kv, float* k, float* v, hipStream_t s);
// Bytes of work that launch_kv_attention uses for these arguments.
int64_t kv_attention_bytes(int64_t T, int64_t B, int Hq, int Hkv, int nb, int64_t max_len);
// Rows of a workgroup in such a call (starts: it has q_start).
int kv_attention_rows(int64_t T, int64_t B, bool starts, int Hq, int Hkv, int nb, int64_t max_len);
int launch_kv_attention(const AttnArgs& a, hipStream_t s);

}  // namespace qmv
