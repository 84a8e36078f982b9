// Internal declarations of the mixture-of-experts operators, shared by their
// C-ABI layer (qmv_moe_api.cpp) and kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// Workspace of a product: [0, blocks) the Q8_0 blocks of x, then the plan:
//   items  [most items][4] int32  expert (E: rows without one), first place in `order`, rows, 0
//   order  [P] int32              the pairs, those of one expert side by side, ascending
//   count  int32                  items
struct MoeWork {
    int64_t blocks, items, order, count, total;
};
// Rows of an expert in one item, at most: as many as it can have when a
// token's experts differ, up to the 16 of a matrix instruction.
inline int moe_rows(int64_t P, int top) {
    const int64_t T = P / top;
    return T <= 4 ? 4 : T <= 8 ? 8 : 16;
}
// Items of P pairs, at most: every item but an expert's last is full.
inline int64_t moe_most_items(int64_t P, int64_t E, int rows) {
    const int64_t kinds = P < E + 1 ? P : E + 1;
    return kinds + (P - kinds) / rows;
}
inline MoeWork moe_work(int64_t P, int top, int per, int64_t E, int64_t K) {
    MoeWork w;
    w.blocks = 0;
    w.items = align256(P / per * (K / 32) * 34);
    w.order = w.items + align256(moe_most_items(P, E, moe_rows(P, top)) * 16);
    w.count = w.order + align256(P * 4);
    w.total = w.count + 256;
    return w;
}
int launch_moe_product(const MoeArgs& a, hipStream_t s);

// y[t][n] = sum over slots j with an expert of weight[t][j] * yp[t * top + j][n],
// s = fma(weight, yp, s) from +0 in ascending j.
int launch_moe_combine(const float* yp, const int32_t* idx, const float* weight, int64_t T,
                       int top, int64_t E, int64_t N, float* y, hipStream_t s);

}  // namespace qmv
