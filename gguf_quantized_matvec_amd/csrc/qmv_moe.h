// Internal declarations of the mixture-of-experts operators, shared by their
// C-ABI layer (qmv_moe_api.cpp) and kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmv.h"
#include "qmv_internal.h"

namespace qmv {

struct RouteArgs {
    const float* logits;   // [T][E]
    const float* bias;     // [E], or NULL
    int32_t T, E, groups, top_groups, group_top, top;
    bool sigmoid, renorm;
    float scale;
    int32_t* idx;          // [T][top]
    float* weight;         // [T][top]
};
int launch_moe_route(const RouteArgs& a, hipStream_t s);

// Pairs up to which every workgroup finds its rows among the numbers itself
// (one wave holds a pair a lane); beyond, a launch before it sorts them.
constexpr int MOE_SCAN = 64;

// One product of the experts that a call's pairs (token, slot) name.  Pair p
// takes activation row p / per (per = top: a token's row for all its slots;
// per = 1: a row a pair) and leaves its result in row p of y.
struct MoeArgs {
    int type;
    const uint8_t *w, *w2;  // E matrices N x K; w2 (a gate/up pair: h = silu(w x) (w2 x)) or NULL
    int64_t E, N, K;
    const int32_t* idx;     // [P]; a number outside 0..E-1: no expert
    int64_t P;
    int32_t top, per;
    const float* x;         // [P / per][K], quantised first, or NULL:
    const uint8_t* xq;      // the Q8_0 blocks of those rows
    uint8_t* work;          // moe_work(...) bytes
    float* y;               // [P][N]; a gate/up pair's rows without an expert become 0, others are left alone
};

// Rows of an expert in one item, at most, which also names the kernel: 4 where
// no expert has more when a token's experts differ, else 16 (matrix products of
// 16 columns, qmv_moe_rows.hip), or 64 or 128 a tile of the GEMM
// (qmv_moe_gemm.hip), by the pairs an expert has on average.  Measured with 16,
// 64 and 128, in us:
//   pairs an expert                          48            96           192             384
//   gate/up Q4_K, 8 of 14336 x 4096      403 443 569   704 731 686  1338 1210 1162  2631 2259 1963
//   gate/up Q4_0, 64 of 1024 x 2048      106 114 152   187 178 198   350  295  299
//   down Q5_0, 16 of 896 x 4864           65  92 123    86  96 127   145  129  139   264  188  196
//   down Q6_K, 8 of 4096 x 14336         321  -  305   534  -  597   979   -   760  1873   -  1228
// (Q6_K has no tile of 64, whose decoding it would not share enough, and costs
// the matrix products of 16 columns two dots a block.)  One rule for all but
// Q6_K costs the others' types where they part: at 96 pairs 64 gains for Q4_0
// and loses 4 % to 16 rows (7 % to 128) for Q4_K and 12 % for Q5_0, at 192 it
// loses 4 % to 128 for Q4_K.
inline int moe_rows(int type, int64_t P, int top, int64_t E) {
    if (type == QMV_Q6_K) {
        if (P >= 48 * E) return 128;
    } else {
        if (P >= 256 * E) return 128;
        if (P >= 96 * E) return 64;
    }
    return P / top <= 4 ? 4 : 16;
}
// Items of P pairs, at most: every item but an expert's last is full.
inline int64_t moe_most_items(int64_t P, int64_t E, int rows) {
    const int64_t kinds = P < E + 1 ? P : E + 1;
    return kinds + (P - kinds) / rows;
}

// A row of activations as k_moe_gemv reads it: C = ceil(K / 256) chunks of 272
// bytes (256 codes and 16 bytes, so that lanes on different chunks differ in
// their banks), 8 C scales and, for formats with a minimum, 8 C scales times
// code sums.
inline __host__ __device__ int moe_gemv_row(int64_t K, bool min) {
    const int C = (int)((K / 32 + 7) / 8);
    return (C * 272 + 8 * C * 4 * (min ? 2 : 1) + 15) & ~15;
}

// Workspace of a product: the activations, then the plan.
//   blocks the Q8_0 blocks of x; for a single token its rows as above; for the
//          GEMM the codes as f16 [rows][K],
//   da     [rows][K / 32] fp16 scales, and
//   ca     [rows][K / 32] f32 scale times the block's code sum
//   items  [most items][4] int32  expert (E: rows without one), its first place in `order`, its
//                                 rows, its first item
//   order  [P] int32              the pairs, those of one expert side by side, ascending
//   count  int32                  items
struct MoeWork {
    int64_t blocks, da, ca, items, order, count, total;
};
inline MoeWork moe_work(int type, int64_t P, int top, int per, int64_t E, int64_t K) {
    const int R = moe_rows(type, P, top, E);
    const int64_t rows = P / per, nb = K / 32;
    MoeWork w;
    w.blocks = 0;
    w.da = R >= 64 ? align256(rows * K * 2) : align256(rows * (nb * 34 + 512) + 2 * rows * nb * 4);
    w.ca = w.da + (R >= 64 ? align256(rows * nb * 2) : 0);
    w.items = w.ca + (R >= 64 ? align256(rows * nb * 4) : 0);
    w.order = w.items + align256(moe_most_items(P, E, R) * 16);
    w.count = w.order + align256(P * 4);
    w.total = w.count + 256;
    return w;
}
inline MoeWork moe_work(const MoeArgs& a) { return moe_work(a.type, a.P, a.top, a.per, a.E, a.K); }
inline int moe_rows(const MoeArgs& a) { return moe_rows(a.type, a.P, a.top, a.E); }
// Bytes that are enough for every type (Q6_K alone has its own items).
inline int64_t moe_work_bytes(int64_t P, int top, int per, int64_t E, int64_t K) {
    const int64_t six = moe_work(QMV_Q6_K, P, top, per, E, K).total;
    const int64_t others = moe_work(QMV_Q4_0, P, top, per, E, K).total;
    return six > others ? six : others;
}

// The products into a.y, by the kernel that fits.
int launch_moe_product(const MoeArgs& a, hipStream_t s);
// y[t][n] = sum over slots j with an expert of weight[t][j] * product[t * top + j][n],
// s = fma(weight, product, s) from +0 in ascending j; a.y: room for the products.
int launch_moe_down(const MoeArgs& a, const float* weight, float* y, hipStream_t s);

// Many rows of an expert, after the preparation (qmv_moe_gemm.hip).
int launch_moe_gemm(const MoeArgs& a, hipStream_t s);

// Single tokens (qmv_moe_gemv.hip): whether the kernel takes the call, whether
// it quantises x itself, and the product (a gate/up pair) or the weighted sum
// into y.  rows: the activations quantised (moe_gemv_row), or NULL: a.x or a.xq.
bool moe_gemv_fits(const MoeArgs& a);
bool moe_gemv_quantises(const MoeArgs& a);
int launch_moe_gemv(const MoeArgs& a, const uint8_t* rows, const float* weight, float* y,
                    hipStream_t s);

}  // namespace qmv
