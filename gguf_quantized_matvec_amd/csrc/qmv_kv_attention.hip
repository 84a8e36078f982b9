// Causal attention over the paged 4-bit cache on gfx950.
//
// Per row (a query token's head) and visible position t, with the keys and
// values held as d * (code - 8) per 32 elements:
//   s[t] = scale * sum_b dk[t][b] * sum_i q_i (k_i - 8)
//   out  = sum_t softmax(s)[t] sum_b dv[t][b] (v - 8)
//
// Both products run on the matrix cores (v_mfma_f32_16x16x32_f16, one 32-block
// per instruction) with the codes as exact f16 operands and the other side
// split into two f16 parts (22 bits), so the result has the accuracy of an
// f32 computation:
// - a code becomes an f16 operand by setting the exponent above its nibble
//   (1024 + code for nibbles at bits 0..3 of a half, 64 + code at bits 4..7)
//   and one packed addition of -1032 or -72: nine instructions for 8 codes, all
//   exact.  (The nibbles taken as f16 subnormals would need five, but MFMA
//   keeps no more bits of a product with a subnormal than of one with its leading
//   bit in place: 2^-18 instead of 2^-24 was left.)
// - scores come out transposed (positions down, rows across: K q^T), so that a
//   lane's results are the operand of the second product (V^T P^T) as they
//   stand: no lane exchange, no LDS round trip;
// - the fp16 block scales multiply the f32 block sums (keys) and the weights
//   before their split (values), v_fma_mix taking the halves as they are.
//
// Work split.  A wave takes 16 R rows that share a key/value head and SUB
// positions at a time: all scores first, one maximum, then the values; the
// WAVES waves of a workgroup take consecutive runs of SUB positions, and their
// results are joined in LDS into a segment of SEG positions.  Segments are
// joined in ascending order, by the workgroup itself or, when there are few
// rows, by k_attn_join from the workspace.  Segments start at multiples of SEG
// and every step depends on the row's own query and positions alone, so a row's
// bits do not depend on the batch, on the prompt's chunking or on the split.
//
// Weights are held relative to a reference r: p = 2^(s log2e - r), where r
// makes the largest p[t] * max_b |dv[t][b]| about 2^14, the top of f16's range:
// what is split then keeps 22 bits down to 2^-17 of the largest term, whatever
// the size of the values.
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_kv_device.h"

namespace qmv {
namespace {

constexpr int SUB = 128;           // positions a wave takes at a time
constexpr int TILES = SUB / 16;
constexpr int WAVES = 4;
constexpr int SEG = SUB * WAVES;   // positions of a segment
constexpr float NO_KEY = -1e30f;   // reference of a row that has seen no position

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

template <int N> struct Words { uint32_t w[N]; };
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {  // 4-byte aligned
    return *reinterpret_cast<const Words<N>*>(p);
}

__device__ __forceinline__ f4 mfma(half8 a, half8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ half8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint4 v = make_uint4(a, b, c, d);
    half8 h;
    __builtin_memcpy(&h, &v, 16);
    return h;
}

// code - 8 of the nibbles at bits 0..3 (low) or 4..7 (high) of both halves.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t plus(uint32_t w, float c) {
    half2v h;
    __builtin_memcpy(&h, &w, 4);
    h = h + (half2v){(_Float16)c, (_Float16)c};
    __builtin_memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
    return plus((w & 0x000F000Fu) | 0x64006400u, -1032.0f);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
    return plus((w & 0x00F000F0u) | 0x54005400u, -72.0f);
}

__device__ __forceinline__ _Float16 half_of(uint32_t w, int i) {
    const uint16_t b = (uint16_t)(i ? w >> 16 : w);
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return h;
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The launch: `tiles` row tiles of 16 R rows (per key/value head), `splits`
// workgroups each of `per` segments; splits > 1: segment results go to work.
struct Plan {
    int32_t tiles, splits, per, segs, R;
};

// A segment's result of one row in the workspace: O [D], then (for all rows)
// reference and sum.
__device__ __forceinline__ float* part_o(const AttnArgs& a, int64_t row, int segs, int seg) {
    return a.work + (row * segs + seg) * (int64_t)(32 * a.kv.nb);
}
__device__ __forceinline__ float* part_rl(const AttnArgs& a, int64_t row, int segs, int seg) {
    return a.work + (int64_t)a.kv.T * a.Hq * segs * (32 * a.kv.nb) + (row * segs + seg) * 2;
}

// Joining a later part (reference r, nothing if NO_KEY) to an earlier state R:
// the factors of the state and of the part, and the new reference.
struct Join {
    float a, b;
};
__device__ __forceinline__ Join join(float& R, float r) {
    const float n = fmaxf(R, r);
    const Join j{exp2_raw(R - n), exp2_raw(r - n)};
    R = n;
    return j;
}
__device__ __forceinline__ float joined(float o, float part, Join j) { return o * j.a + part * j.b; }

__device__ __forceinline__ float result(float o, float l) { return l == 0.0f ? 0.0f : o / l; }

template <int NB, int R>
__global__ __launch_bounds__(64 * WAVES) void k_attn(AttnArgs a, Plan plan) {
    const KvArgs& kv = a.kv;
    constexpr int D = 32 * NB;
    constexpr int NBP = NB < 4 ? NB : 4;  // blocks joined at a time
    constexpr int LD = 32 * NBP + 4;
    __shared__ __align__(16) uint32_t s_dk[WAVES][SUB * NB / 2];
    __shared__ __align__(16) uint32_t s_dv[WAVES][SUB * NB / 2];
    __shared__ __align__(16) float s_ev[WAVES][SUB];
    __shared__ __align__(16) float s_o[WAVES][16 * LD];
    __shared__ float s_r[WAVES][16 * R], s_l[WAVES][16 * R];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.Hq / kv.Hkv;
    const int head = blockIdx.x % kv.Hkv;
    int at = blockIdx.x / kv.Hkv;
    const int split = at % plan.splits;
    const int tile = plan.tiles - 1 - at / plan.splits;  // long rows first

    // the tile's sequence and rows
    int b, first;
    if (!kv.q_start) {
        const int per = (G + 16 * R - 1) / (16 * R);
        b = tile / per;
        first = (tile - b * per) * 16 * R;
        if (b >= kv.B) return;
    } else {
        // sequence b owns the tiles from (start[b] * G) / (16 R) + b on
        int below = 0;
        for (int b0 = 0; b0 < kv.B; b0 += 64) {
            const int i = b0 + lane;
            bool le = false;
            if (i < kv.B) le = (int64_t)kv.q_start[i] * G / (16 * R) + i <= tile;
            const unsigned long long m = __ballot(le);
            below += __popcll(m);
            if (m != ~0ull) break;
        }
        if (below == 0) return;
        b = uniform(below - 1);
        const int64_t f = (tile - ((int64_t)kv.q_start[b] * G / (16 * R) + b)) * 16 * R;
        if (f < 0 || f > INT32_MAX) return;
        first = (int)f;
    }
    const Seq s = seq_of(kv, b);
    const int64_t rows64 = (int64_t)s.n * G;
    if (first >= rows64) return;
    const int rows = (int)rows64;
    const int last = first + 16 * R < rows ? first + 16 * R - 1 : rows - 1;
    const int pos_lo = s.len - s.n + first / G, pos_hi = s.len - s.n + last / G;
    const int t_end = pos_hi + 1;
    const int t_begin = a.window && pos_lo + 1 > a.window ? pos_lo + 1 - a.window : 0;

    int seg0 = t_begin / SEG, seg1 = t_end > 0 ? (t_end + SEG - 1) / SEG : 0;
    if (plan.splits > 1) {
        const int lo = split * plan.per, hi = lo + plan.per;
        seg0 = seg0 > lo ? seg0 : lo;
        seg1 = seg1 < hi ? seg1 : hi;
        if (seg0 >= seg1) return;
    }

    // q as two f16 parts: lane (n, g) holds elements 32b + 8g ... + 7 of row n
    half8 qh[R][NB], ql[R][NB];
    float factor[R];
    int pos[R];
    const float to_log2 = a.scale * 1.44269504f;
#pragma unroll
    for (int rt = 0; rt < R; rt++) {
        const int rr = first + 16 * rt + n;
        const bool valid = rr < rows;
        const int j = valid ? rr / G : 0, hg = valid ? rr - j * G : 0;
        pos[rt] = valid ? s.len - s.n + j : -1;
        const float* qp = a.q + (int64_t)(s.q0 + j) * a.q_stride + (int64_t)(head * G + hg) * D + 8 * g;
        float x[NB][8];
        float big = 0.0f;
#pragma unroll
        for (int bb = 0; bb < NB; bb++) {
            float4 u = make_float4(0, 0, 0, 0), v = u;
            if (valid) {
                u = *reinterpret_cast<const float4*>(qp + 32 * bb);
                v = *reinterpret_cast<const float4*>(qp + 32 * bb + 4);
            }
            const float t[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; e++) {
                x[bb][e] = t[e] * to_log2;
                big = fmaxf(big, fabsf(x[bb][e]));
            }
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        int ex = (int)((__float_as_uint(big) >> 23) & 255) - 126;  // big < 2^ex
        ex = ex < -100 ? -100 : ex;
        const float up = ldexpf(1.0f, 15 - ex);
        factor[rt] = ldexpf(1.0f, ex - 15);
#pragma unroll
        for (int bb = 0; bb < NB; bb++) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float y = x[bb][e] * up;
                qh[rt][bb][e] = (_Float16)y;
                ql[rt][bb][e] = (_Float16)(y - (float)qh[rt][bb][e]);
            }
        }
    }

    const int page_tokens = 1 << kv.log2p;
    const int64_t codes = (int64_t)(16 * NB) << kv.log2p;
    const int32_t* table = kv.table + (int64_t)b * kv.table_stride;

    // the joined state: thread (row tid / 16, part tid % 16) of each row tile
    // holds 2 NBP elements of every NBP blocks
    const int jr = tid >> 4, jp = tid & 15;
    float O[R][2 * NB], L[R], RR[R];
#pragma unroll
    for (int rt = 0; rt < R; rt++) {
        L[rt] = 0.0f;
        RR[rt] = NO_KEY;
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) O[rt][i] = 0.0f;
    }

    for (int seg = seg0; seg < seg1; seg++) {
        const int t0 = seg * SEG + wave * SUB;
        const bool work = t0 < t_end && t0 + SUB > t_begin;
        f4 o[R][2 * NB];
        float r[R], l[R];
#pragma unroll
        for (int rt = 0; rt < R; rt++) {
            r[rt] = NO_KEY;
            l[rt] = 0.0f;
        }
        if (work) {
            // pages of the wave's tiles of 16 positions
            int pg = -1;
            if (lane < TILES && t0 + 16 * lane < s.len) {
                const int p = table[(t0 + 16 * lane) >> kv.log2p];
                if (p >= 0 && (int64_t)p < kv.n_pages) pg = p;
            }
            const uint32_t there = (uint32_t)__ballot(pg >= 0);  // tiles that have a page
            pg = pg < 0 ? 0 : pg;  // loads of the others read page 0 and are not used
            const bool masked = t0 + SUB > pos_lo + 1 || (a.window && t0 <= pos_hi - a.window) ||
                                there != (1u << TILES) - 1;
            // scales: lane i of 8 per tile takes two positions
            {
                const int u = lane >> 3, t = t0 + 16 * u + 2 * (lane & 7);
                const uint8_t* hd = head_of(kv, __shfl(pg, u), head) + 2 * codes +
                                    (int64_t)(t & (page_tokens - 1)) * 2 * NB;
                Words<NB> dk = load_words<NB>(hd);
                Words<NB> dv = load_words<NB>(hd + ((int64_t)(2 * NB) << kv.log2p));
                const int live = ((there >> u) & 1) ? s.len - t : 0;  // positions behind the last: scale 0
                uint32_t top[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < NB; i++) {
                    uint32_t keep = 0;
                    if (live > (2 * i) / NB) keep |= 0xFFFFu;
                    if (live > (2 * i + 1) / NB) keep |= 0xFFFF0000u;
                    dk.w[i] &= keep;
                    dv.w[i] &= keep;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t m = (h ? dv.w[i] >> 16 : dv.w[i]) & 0x7FFFu;
                        const int tok = (2 * i + h) / NB;
                        top[tok] = m > top[tok] ? m : top[tok];
                    }
                }
                // max_b |dv| < 2^ev; a position with an infinite or NaN scale gets ev = inf, which
                // turns the reference of a row that sees it infinite and its result NaN, and
                // scales of 0, so that the rows that do not see it have no 0 * NaN
                const bool bad[2] = {top[0] >= 0x7C00u, top[1] >= 0x7C00u};
#pragma unroll
                for (int i = 0; i < NB; i++) {
                    if (bad[(2 * i) / NB]) dv.w[i] &= 0xFFFF0000u;
                    if (bad[(2 * i + 1) / NB]) dv.w[i] &= 0x0000FFFFu;
                    s_dk[wave][lane * NB + i] = dk.w[i];
                    s_dv[wave][lane * NB + i] = dv.w[i];
                }
#pragma unroll
                for (int i = 0; i < 2; i++)
                    s_ev[wave][2 * lane + i] = bad[i] ? INFINITY : (float)((int)(top[i] >> 10) - 14);
            }
            // lane u of TILES: where tile u's K codes begin (its V codes, 16 positions of the
            // same size, are `codes` further)
            const int64_t at_k = ((int64_t)pg * kv.Hkv + head) * kv.head_bytes +
                                 (int64_t)((t0 + 16 * lane) & (page_tokens - 1)) * (16 * NB);
            const uint32_t at_lo = (uint32_t)at_k, at_hi = (uint32_t)(at_k >> 32);
            const auto tile_codes = [&](int u) {
                const uint64_t at = (uint32_t)__builtin_amdgcn_readlane(at_lo, u) |
                                    (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_hi, u) << 32;
                return kv.pages + at;
            };
            Words<NB> kw[TILES];
#pragma unroll
            for (int u = 0; u < TILES; u++)
                kw[u] = load_words<NB>(tile_codes(u) + n * (16 * NB) + g * (4 * NB));
            wave_sync();

            // scores: sc[rt][u][i] of position t0 + 16u + 4g + i, row n
            f4 sc[R][TILES];
#pragma unroll
            for (int u = 0; u < TILES; u++) {
                half8 ko[NB];
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    const uint32_t w = kw[u].w[bb], v = w >> 8;
                    ko[bb] = operand(low_codes(w), high_codes(w), low_codes(v), high_codes(v));
                }
                const Words<2 * NB> d = *reinterpret_cast<const Words<2 * NB>*>(
                    &s_dk[wave][(16 * u + 4 * g) * NB / 2]);
#pragma unroll
                for (int rt = 0; rt < R; rt++) {
                    f4 z = {0, 0, 0, 0};
#pragma unroll
                    for (int bb = 0; bb < NB; bb++) {
                        f4 acc = {0, 0, 0, 0};
                        acc = mfma(ko[bb], ql[rt][bb], acc);
                        acc = mfma(ko[bb], qh[rt][bb], acc);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            z[i] = __builtin_fmaf(
                                (float)half_of(d.w[(i * NB + bb) >> 1], (i * NB + bb) & 1), acc[i],
                                z[i]);
                    }
                    sc[rt][u] = z;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            Words<NB> vw[TILES];
#pragma unroll
            for (int u = 0; u < TILES; u++)
                vw[u] = load_words<NB>(tile_codes(u) + codes + lane * (4 * NB));

            // weights
            if (masked) {
#pragma unroll
                for (int rt = 0; rt < R; rt++) {
                    // a position 16u + i is seen in (rel - window, rel]
                    const int rel = pos[rt] - t0 - 4 * g;
                    const int from = a.window ? rel - a.window : -(1 << 30);
#pragma unroll
                    for (int u = 0; u < TILES; u++) {
                        const int hi = (there >> u) & 1 ? rel : -(1 << 30);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            sc[rt][u][i] = 16 * u + i <= hi && 16 * u + i > from ? sc[rt][u][i] : -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int rt = 0; rt < R; rt++) {
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < TILES; u++) {
                    const f4 e = *reinterpret_cast<const f4*>(&s_ev[wave][16 * u + 4 * g]);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        top = fmaxf(top, __builtin_fmaf(sc[rt][u][i], factor[rt], e[i]));
                }
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float ref = top > -INFINITY ? top - 14.0f : 0.0f;
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < TILES; u++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        sc[rt][u][i] = exp2_raw(__builtin_fmaf(sc[rt][u][i], factor[rt], -ref));
                        sum += sc[rt][u][i];
                    }
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                l[rt] = sum;
                // no maximum: nothing seen, or NaN scores, whose sum is NaN and stays
                r[rt] = top == -INFINITY && sum == 0.0f ? NO_KEY : ref;
#pragma unroll
                for (int i = 0; i < 2 * NB; i++) o[rt][i] = f4{0, 0, 0, 0};
            }

            // values, 32 positions at a time
#pragma unroll
            for (int q = 0; q < TILES / 2; q++) {
                const Words<2 * NB> d0 = *reinterpret_cast<const Words<2 * NB>*>(
                    &s_dv[wave][(32 * q + 4 * g) * NB / 2]);
                const Words<2 * NB> d1 = *reinterpret_cast<const Words<2 * NB>*>(
                    &s_dv[wave][(32 * q + 16 + 4 * g) * NB / 2]);
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    const uint32_t w0 = vw[2 * q].w[bb], w1 = vw[2 * q + 1].w[bb];
                    const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
                    const half8 even = operand(low_codes(w0), low_codes(v0), low_codes(w1), low_codes(v1));
                    const half8 odd = operand(high_codes(w0), high_codes(v0), high_codes(w1), high_codes(v1));
#pragma unroll
                    for (int rt = 0; rt < R; rt++) {
                        half8 ph, pl;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            // the order of the code words: positions 0, 2, 1, 3 of each tile
                            const int i = ((j & 1) << 1) | ((j >> 1) & 1), u = 2 * q + (j >> 2);
                            const float dd = (float)half_of((j < 4 ? d0 : d1).w[(i * NB + bb) >> 1],
                                                            (i * NB + bb) & 1);
                            ph[j] = (_Float16)(sc[rt][u][i] * dd);
                            pl[j] = (_Float16)__builtin_fmaf(sc[rt][u][i], dd, -(float)ph[j]);
                        }
                        o[rt][2 * bb] = mfma(even, pl, o[rt][2 * bb]);
                        o[rt][2 * bb + 1] = mfma(odd, pl, o[rt][2 * bb + 1]);
                        o[rt][2 * bb] = mfma(even, ph, o[rt][2 * bb]);
                        o[rt][2 * bb + 1] = mfma(odd, ph, o[rt][2 * bb + 1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }

        // join the waves' parts of the segment, then the segment to the state
#pragma unroll
        for (int rt = 0; rt < R; rt++) {
            if (g == 0) {
                s_r[wave][16 * rt + n] = r[rt];
                s_l[wave][16 * rt + n] = l[rt];
            }
            float f[WAVES], sr = NO_KEY, sl = 0.0f;
            Join jn{1.0f, 0.0f};
#pragma unroll
            for (int b0 = 0; b0 < NB; b0 += NBP) {
                const int nbp = NB - b0 < NBP ? NB - b0 : NBP;
                if (work) {
#pragma unroll
                    for (int bb = 0; bb < nbp; bb++) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            v[2 * i] = o[rt][2 * (b0 + bb)][i];
                            v[2 * i + 1] = o[rt][2 * (b0 + bb) + 1][i];
                        }
                        float* to = &s_o[wave][n * LD + 32 * bb + 8 * g];
                        *reinterpret_cast<f4*>(to) = f4{v[0], v[1], v[2], v[3]};
                        *reinterpret_cast<f4*>(to + 4) = f4{v[4], v[5], v[6], v[7]};
                    }
                }
                __syncthreads();
                if (b0 == 0) {
#pragma unroll
                    for (int w = 0; w < WAVES; w++) {
                        f[w] = s_r[w][16 * rt + jr];
                        sr = fmaxf(sr, f[w]);
                    }
#pragma unroll
                    for (int w = 0; w < WAVES; w++) {
                        const bool has = f[w] != NO_KEY;
                        f[w] = has ? exp2_raw(f[w] - sr) : -1.0f;  // -1: nothing there
                        if (has) sl = __builtin_fmaf(f[w], s_l[w][16 * rt + jr], sl);
                    }
                    if (plan.splits == 1 && sr != NO_KEY) {
                        jn = join(RR[rt], sr);
                        L[rt] = joined(L[rt], sl, jn);
                    }
                }
                const int per = 2 * nbp;
                float v[2 * NBP];
#pragma unroll
                for (int i = 0; i < 2 * NBP; i++) v[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; w++)
                    if (f[w] >= 0.0f || f[w] != f[w]) {
#pragma unroll
                        for (int i = 0; i < per; i++)
                            v[i] = __builtin_fmaf(f[w], s_o[w][jr * LD + jp * per + i], v[i]);
                    }
                if (plan.splits == 1) {
                    if (sr != NO_KEY) {
#pragma unroll
                        for (int i = 0; i < per; i++)
                            O[rt][2 * b0 + i] = joined(O[rt][2 * b0 + i], v[i], jn);
                    }
                } else {
                    const int rr = first + 16 * rt + jr;
                    if (rr < rows) {
                        const int64_t row =
                            (int64_t)(s.q0 + rr / G) * a.Hq + head * G + rr % G;
                        float* to = part_o(a, row, plan.segs, seg) + 32 * b0 + jp * per;
#pragma unroll
                        for (int i = 0; i < per; i++) to[i] = v[i];
                        if (b0 == 0 && jp == 0) {
                            float* rl = part_rl(a, row, plan.segs, seg);
                            rl[0] = sr;
                            rl[1] = sl;
                        }
                    }
                }
                __syncthreads();
            }
        }
    }
    if (plan.splits > 1) return;
#pragma unroll
    for (int rt = 0; rt < R; rt++) {
        const int rr = first + 16 * rt + jr;
        if (rr >= rows) continue;
        float* out = a.out + ((int64_t)(s.q0 + rr / G) * a.Hq + head * G + rr % G) * D;
#pragma unroll
        for (int b0 = 0; b0 < NB; b0 += NBP) {
            const int per = 2 * (NB - b0 < NBP ? NB - b0 : NBP);
#pragma unroll
            for (int i = 0; i < per; i++)
                out[32 * b0 + jp * per + i] = result(O[rt][2 * b0 + i], L[rt]);
        }
    }
}

// Joins the segments of a row in ascending order, as k_attn does when it has
// them all: one workgroup per row and query head, one element a thread.  The
// references' running maxima come from a scan over 64 segments at a time.
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int segs) {
    const KvArgs& kv = a.kv;
    const int t = blockIdx.x / a.Hq, lane = threadIdx.x & 63;
    const int D = 32 * kv.nb, e = threadIdx.x;
    const int b = seq_of_row(kv, t);
    if (b < 0) return;
    const Seq s = seq_of(kv, b);
    if (t < s.q0 || t >= s.q0 + s.n) return;
    const int pos = s.len - s.n + (t - s.q0);
    const int64_t row = blockIdx.x;
    const int lo = a.window && pos + 1 > a.window ? (pos + 1 - a.window) / SEG : 0;
    const int hi = pos < 0 ? lo : pos / SEG + 1;
    const float* po = part_o(a, row, segs, 0) + (e < D ? e : 0);
    const float* rl = part_rl(a, row, segs, 0);
    float O = 0.0f, L = 0.0f, R = NO_KEY;
    for (int c0 = lo; c0 < hi; c0 += 64) {
        const int c = c0 + lane;
        const float r = c < hi ? rl[2 * (int64_t)c] : NO_KEY;
        const float l = c < hi ? rl[2 * (int64_t)c + 1] : 0.0f;
        float top = fmaxf(R, r);  // maximum up to and with segment c
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float v = __shfl_up(top, o);
            if (lane >= o) top = fmaxf(top, v);
        }
        float before = __shfl_up(top, 1);
        if (lane == 0) before = R;
        R = before;
        const Join j = join(R, r);
        R = __shfl(top, 63);
        const int m = hi - c0 < 64 ? hi - c0 : 64;
        for (int i = 0; i < m; i++) {
            const float rc = __shfl(r, i);
            if (rc == NO_KEY) continue;
            const Join k{__shfl(j.a, i), __shfl(j.b, i)};
            O = joined(O, po[(int64_t)(c0 + i) * D], k);
            L = joined(L, __shfl(l, i), k);
        }
    }
    if (e < D) a.out[row * D + e] = result(O, L);
}

// one: a row each (no starts).
Plan plan_of(bool one, int64_t T, int64_t B, int Hq, int Hkv, int nb, int64_t max_len) {
    const int64_t G = Hq / Hkv;
    Plan p;
    p.R = 1;
    const int64_t tr = 16 * p.R;
    p.tiles = (int32_t)(one ? B * ((G + tr - 1) / tr) : T * G / tr + B);
    p.segs = (int32_t)((max_len + SEG - 1) / SEG);
    const int64_t want = 1024, groups = (int64_t)p.tiles * Hkv;
    int64_t splits = groups >= want / 2 ? 1 : (want + groups - 1) / groups;
    if (splits > p.segs) splits = p.segs;
    p.per = (int32_t)((p.segs + splits - 1) / splits);
    p.splits = (p.segs + p.per - 1) / p.per;
    return p;
}

template <int NB>
void launch_nb(const AttnArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.tiles * p.splits * a.kv.Hkv));
    hipLaunchKernelGGL((k_attn<NB, 1>), grid, dim3(64 * WAVES), 0, s, a, p);
}

}  // namespace

int64_t kv_attention_bytes(int64_t T, int64_t B, int Hq, int Hkv, int nb, int64_t max_len) {
    // a call with T == B may name its rows by starts or not
    const Plan p = plan_of(false, T, B, Hq, Hkv, nb, max_len);
    const bool split = p.splits > 1 || (T == B && plan_of(true, T, B, Hq, Hkv, nb, max_len).splits > 1);
    return split ? T * Hq * p.segs * (32 * nb + 2) * 4 : 16;
}

int launch_kv_attention(const AttnArgs& a, hipStream_t s) {
    const Plan p = plan_of(!a.kv.q_start, a.kv.T, a.kv.B, a.Hq, a.kv.Hkv, a.kv.nb, a.kv.max_len);
    switch (a.kv.nb) {
    case 1: launch_nb<1>(a, p, s); break;
    case 2: launch_nb<2>(a, p, s); break;
    case 3: launch_nb<3>(a, p, s); break;
    case 4: launch_nb<4>(a, p, s); break;
    case 5: launch_nb<5>(a, p, s); break;
    case 6: launch_nb<6>(a, p, s); break;
    case 7: launch_nb<7>(a, p, s); break;
    default: launch_nb<8>(a, p, s); break;
    }
    int rc = (int)hipGetLastError();
    if (rc || p.splits == 1) return rc;
    const unsigned block = (unsigned)((32 * a.kv.nb + 63) / 64 * 64);
    hipLaunchKernelGGL(k_attn_join, dim3((unsigned)((int64_t)a.kv.T * a.Hq)), dim3(block), 0, s, a,
                       p.segs);
    return (int)hipGetLastError();
}

}  // namespace qmv
