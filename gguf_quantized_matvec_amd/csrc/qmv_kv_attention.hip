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
// Work split.  A wave takes 16 (or 8) rows that share a key/value head and SUB
// positions at a time: all scores first, one maximum, then the values; the
// WAVES waves of a workgroup take consecutive runs of SUB positions, and their
// results are joined in LDS into a segment of SEG positions.  Segments are
// joined in ascending order, by the workgroup itself or, when there are few
// rows, by k_attn_join from the workspace.  Segments start at multiples of SEG
// and every step depends on the row's own query and positions alone, so a row's
// bits do not depend on the batch, on the prompt's chunking or on the split.
//
// Weights.  With max_b |dv[t][b]| < 2^e[t], a weight is held as p[t] =
// 2^(s[t] log2e + e[t] - r), where r makes the largest of a run 2^14, and its
// scales as dv 2^-e: the products, which are split into two f16 numbers, then
// fill f16's range from the top, keep 22 bits down to 2^-17 of the largest term
// and are off by 2^-39 of it below, whatever the size of the values.  The sum
// of the weights is that of p 2^-e, in f32.  Blocks far below the largest of
// their position: exact_sums.
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qmv_kv_device.h"
#include "qmv_lanes.h"

namespace qmv {
namespace {

constexpr int WAVES = 4;
// Positions a wave takes at a time: 128, or for heads beyond 128 elements 64, so
// that their codes, scores and sums fit the 256 registers of two waves per
// SIMD.  And of a segment.
constexpr int sub_of(int nb) { return nb <= 4 ? 128 : 64; }
constexpr int seg_of(int nb) { return WAVES * sub_of(nb); }
// Reference of a row that has seen no position: below every score (their size stays under 2^127), so
// that joining a part to it never takes it for the larger.
constexpr float NO_KEY = -3.402823466e38f;

// A block of values whose scale is this far below the largest of its position has its sums done
// apart (exact_sums).
constexpr float SMALL = 1.0f / 256;
constexpr uint16_t SMALL_BITS = (15 - 8) << 10;  // as f16

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfloat8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

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
// The constants come from registers that the compiler cannot see through, so
// that mask and exponent are one v_and_or_b32 (which takes no literals).
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
struct Unpack {
    uint32_t low_mask = 0x000F000Fu, low_exp = 0x64006400u;    // 1024 + code
    uint32_t high_mask = 0x00F000F0u, high_exp = 0x54005400u;  // 64 + code
    __device__ __forceinline__ Unpack() {
        asm("" : "+s"(low_mask), "+v"(low_exp), "+s"(high_mask), "+v"(high_exp));
    }
    __device__ __forceinline__ static uint32_t plus(uint32_t w, float c) {
        half2v h;
        __builtin_memcpy(&h, &w, 4);
        h = h + (half2v){(_Float16)c, (_Float16)c};
        __builtin_memcpy(&w, &h, 4);
        return w;
    }
    __device__ __forceinline__ uint32_t low(uint32_t w) const {
        return plus((w & low_mask) | low_exp, -1032.0f);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w) const {
        return plus((w & high_mask) | high_exp, -72.0f);
    }
};

__device__ __forceinline__ uint32_t half_bits(uint32_t w, int i) { return i ? w >> 16 : w & 0xFFFFu; }

__device__ __forceinline__ _Float16 half_of(uint32_t w, int i) {
    const uint16_t b = (uint16_t)(i ? w >> 16 : w);
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return h;
}

__device__ __forceinline__ half2v halves(uint32_t w) {
    half2v h;
    __builtin_memcpy(&h, &w, 4);
    return h;
}
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ ushort2v ushorts(uint32_t w) {
    ushort2v h;
    __builtin_memcpy(&h, &w, 4);
    return h;
}
__device__ __forceinline__ uint32_t word(half2v h) {
    uint32_t w;
    __builtin_memcpy(&w, &h, 4);
    return w;
}

// A number as the sum of two f16 numbers, two at a time.
struct Split {
    half2v h, l;
};
__device__ __forceinline__ Split two_parts(float a, float b) {
    Split s;
    s.h = __builtin_convertvector(f2{a, b}, half2v);
    s.l = __builtin_convertvector(f2{a - (float)s.h[0], b - (float)s.h[1]}, half2v);
    return s;
}
// s d, split again: what the rounded product of the first part leaves is exact in the f16 fma,
// the second part's product joins it.  Three packed instructions for two numbers (v_fma_mixlo_f16
// and v_fma_mixhi_f16 do two in four, at half the rate).
__device__ __forceinline__ Split times(Split s, half2v d) {
    Split r;
    r.h = s.h * d;
    r.l = __builtin_elementwise_fma(s.l, d, __builtin_elementwise_fma(s.h, d, -r.h));
    return r;
}

// LDS by byte offset: one register holds a lane's offset and every read adds a
// constant to it.  (Left to itself the compiler keeps an address for every read
// of an unrolled loop, some fifty registers.)
__device__ __forceinline__ uint32_t lds_at(const void* p) {
    uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
    asm("" : "+v"(at));
    return at;
}
template <class T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *(__attribute__((address_space(3))) const T*)(uintptr_t)at;
}

// The value of lane n ^ 8 among 16.
__device__ __forceinline__ float across8(float x) { return dpp<DPP_ROR8>(x); }

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The sums of values over a run for one block, from weights times scales with all their 24 bits, and
// whether the lane's row takes them.  The products' two f16 parts lose what lies 2^-39 below the
// largest product of all blocks, which is much of a block whose scales are far below the others':
// a row that sees a SMALL scale of the block takes these sums instead, three bf16 numbers a weight,
// which have f32's range.  (Where it sees none, a block keeps what is 2^-30 of its own largest
// product.)  The choice depends on what the row sees alone, so its bits still do.
//
// Few models need it, if any, so it is made for few registers rather than for speed: everything is
// loaded and the scores are computed once more, in the same steps (parts(b): the rows' two parts).
// Calls that do not need it take as long as without it, in k_attn_wide 3 % longer; calls that need it
// for one block of every position 2.3 to 2.9 times as long (32 sequences of 301..8191: 133 us for 57).
struct Exact {
    f4 sum[2];  // even elements, odd elements
    bool taken;
};
// The upper halves of two numbers' bits: bf16 numbers.
__device__ __forceinline__ uint32_t upper(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ uint32_t as_bf16(uint32_t w) {  // of two small whole f16 numbers
    return upper((float)half_of(w, 0), (float)half_of(w, 1));
}
// At the end of a branch that few runs take, so that behind it the others wait for their own loads
// only (4 % of k_attn_wide).
__device__ __forceinline__ void all_arrived() { __builtin_amdgcn_s_waitcnt(0); }

template <int NB, class F>
__device__ __forceinline__ Exact exact_sums(const AttnArgs& a, const Unpack& unpack,
                                            const int32_t* table, int len, int head, int t0, int bb,
                                            float factor, float ref, int pos, int lane, F&& parts) {
    constexpr int TILES = sub_of(NB) / 16;
    const KvArgs& kv = a.kv;
    Exact r = {};
    bool small = false;
    asm volatile("" : "+v"(lane));  // (nothing of this before the loop of the runs)
    const int n = lane & 15, g = lane >> 4;
#pragma nounroll
    for (int t = t0; t < t0 + 16 * TILES; t += 16) {  // a tile in half of a product, zeros in the other
        int page = t < len ? table[t >> kv.log2p] : -1;
        const bool ok = page >= 0 && (int64_t)page < kv.n_pages;
        page = ok ? page : 0;
        const uint8_t* hd = head_of(kv, page, head);
        const int off = t & ((1 << kv.log2p) - 1);
        const int64_t codes = (int64_t)(16 * NB) << kv.log2p, scales = (int64_t)(2 * NB) << kv.log2p;
        const Words<NB> kw = load_words<NB>(hd + (off + n) * (16 * NB) + g * (4 * NB));
        const uint8_t* sc = hd + 2 * codes + (off + 4 * g) * (2 * NB);
        const Words<2 * NB> dk = load_words<2 * NB>(sc);
        f4 z = {0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < NB; b++) {
            half8 qh, ql;
            parts(b, qh, ql);
            const uint32_t w = kw.w[b], v = w >> 8;
            const half8 ko = operand(unpack.low(w), unpack.high(w), unpack.low(v), unpack.high(v));
            const f4 acc = mfma(ko, qh, mfma(ko, ql, f4{0, 0, 0, 0}));
#pragma unroll
            for (int i = 0; i < 4; i++)
                z[i] = __builtin_fmaf((float)half_of(dk.w[(i * NB + b) >> 1], (i * NB + b) & 1), acc[i],
                                      z[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
        const Words<2 * NB> dv = load_words<2 * NB>(sc + scales);
        const uint16_t* dvb = reinterpret_cast<const uint16_t*>(sc + scales) + bb;
        const uint32_t vw =
            *reinterpret_cast<const uint32_t*>(hd + codes + off * (16 * NB) + lane * (4 * NB) + 4 * bb);
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const uint32_t m = half_bits(dv.w[(i * NB + b) >> 1], (i * NB + b) & 1) & 0x7FFFu;
                top = m > top ? m : top;
            }
            const int e = (int)(top >> 10) - 14, at = t + 4 * g + i;
            const bool bad = top >= 0x7C00u;
            const float down = bad ? 0.0f : __uint_as_float((uint32_t)(127 - e) << 23);
            const float d = bad ? 0.0f : half_value(dvb[i * NB]);
            const bool seen = ok && at <= pos && (!a.window || at > pos - a.window);
            const float s = __builtin_fmaf(z[i], factor, bad ? INFINITY : (float)e);
            const float p = seen ? exp2_raw(s - ref) : 0.0f;
            small |= p > 0.0f && fabsf(d) * down < SMALL;
            x[i] = p * down * d;
            __builtin_amdgcn_sched_barrier(0);
        }
        const uint4 ev = make_uint4(as_bf16(unpack.low(vw)), as_bf16(unpack.low(vw >> 8)), 0, 0);
        const uint4 od = make_uint4(as_bf16(unpack.high(vw)), as_bf16(unpack.high(vw >> 8)), 0, 0);
#pragma unroll
        for (int m = 0; m < 3; m++) {  // 8 bits each, cut off so that what is left is exact
            const uint4 part = make_uint4(upper(x[0], x[2]), upper(x[1], x[3]), 0, 0);
            bfloat8 e, o, w;
            __builtin_memcpy(&e, &ev, 16);
            __builtin_memcpy(&o, &od, 16);
            __builtin_memcpy(&w, &part, 16);
            r.sum[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e, w, r.sum[0], 0, 0, 0);
            r.sum[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o, w, r.sum[1], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] -= __uint_as_float(__float_as_uint(x[i]) & 0xFFFF0000u);
        }
    }
    r.taken = (__ballot(small) >> n) & 0x0001000100010001ull;
    return r;
}

// The launch: `tiles` row tiles (per key/value head), `splits` workgroups each
// of `per` segments; splits > 1: segment results go to work.
struct Plan {
    int32_t tiles, splits, per, segs;
    bool pack, wide;
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
__device__ __forceinline__ float joined(float o, float part, Join j) {
    return __builtin_fmaf(o, j.a, part * j.b);
}

// The reference of a run of scores whose largest is top: the weights relative to it reach 2^14.  From
// 2^25 on 14 may be no multiple of top's step, and the difference rounded to 16, whose weight is
// beyond f16: top itself then, with weights up to 1 (scores there are steps of 4 or more apart).
__device__ __forceinline__ float reference(float top) {
    const float r = top > -INFINITY ? top - 14.0f : 0.0f;
    return top - r > 15.0f ? top : r;
}

__device__ __forceinline__ float result(float o, float l) { return l == 0.0f ? 0.0f : o / l; }

// The sequence b and its first row of row tile `tile` of ROWS rows; false if
// there is none.
template <int ROWS>
__device__ __forceinline__ bool locate(const KvArgs& kv, int G, int tile, int lane, int& b, int& first) {
    if (!kv.q_start) {
        const int per = (G + ROWS - 1) / ROWS;
        b = tile / per;
        first = (tile - b * per) * ROWS;
        return b < kv.B;
    }
    // sequence b owns the tiles from start[b] * G / ROWS + b on
    int below = 0;
    for (int b0 = 0; b0 < kv.B; b0 += 64) {
        const int i = b0 + lane;
        bool le = false;
        if (i < kv.B) le = (int64_t)kv.q_start[i] * G / ROWS + i <= tile;
        const unsigned long long m = __ballot(le);
        below += __popcll(m);
        if (m != ~0ull) break;
    }
    if (below == 0) return false;
    b = uniform(below - 1);
    const int64_t f = (tile - ((int64_t)kv.q_start[b] * G / ROWS + b)) * ROWS;
    if (f < 0 || f > INT32_MAX) return false;
    first = (int)f;
    return true;
}

// Row rr of a sequence's rows as two f16 parts (lane group g holds elements
// 32b + 8g ... + 7), scaled so that its largest element is just below 2^15; what
// brings a product with it to base-2 scores (factor), and its position (-1 for
// rows past the last).  meanwhile() runs between the loads and their use.
template <int NB, class F>
__device__ __forceinline__ void prepare_q(const AttnArgs& a, const Seq& s, int head, int G, int rr,
                                          int rows, int g, half8 (&qh)[NB], half8 (&ql)[NB],
                                          float& factor, int& pos, F&& meanwhile) {
    constexpr int D = 32 * NB;
    const bool valid = rr < rows;
    const int j = valid ? rr / G : 0, hg = valid ? rr - j * G : 0;
    pos = valid ? s.len - s.n + j : -1;
    const float* qp = a.q + (int64_t)(s.q0 + j) * a.q_stride + (int64_t)(head * G + hg) * D + 8 * g;
    const float to_log2 = a.scale * 1.44269504f;
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
        for (int e = 0; e < 8; e++) x[bb][e] = t[e] * to_log2;
    }
    meanwhile();
#pragma unroll
    for (int bb = 0; bb < NB; bb++)
#pragma unroll
        for (int e = 0; e < 8; e++) big = fmaxf(big, fabsf(x[bb][e]));
    big = max_rows(big);
    int ex = (int)((__float_as_uint(big) >> 23) & 255) - 126;  // big < 2^ex
    ex = ex < -100 ? -100 : ex;
    const float up = ldexpf(1.0f, 15 - ex);
    factor = ldexpf(1.0f, ex - 15);
#pragma unroll
    for (int bb = 0; bb < NB; bb++) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float y = x[bb][e] * up;
            qh[bb][e] = (_Float16)y;
            ql[bb][e] = (_Float16)(y - (float)qh[bb][e]);
        }
    }
}

// Block scales of two positions (2 lane and 2 lane + 1 of a run) into LDS, by
// block; `live` of them lie before the sequence's end, the others get 0.
template <int NB>
__device__ __forceinline__ void keep_live(Words<NB>& d, int live) {
#pragma unroll
    for (int i = 0; i < NB; i++) {
        uint32_t keep = 0;
        if (live > (2 * i) / NB) keep |= 0xFFFFu;
        if (live > (2 * i + 1) / NB) keep |= 0xFFFF0000u;
        d.w[i] &= keep;
    }
}
template <int NB>
__device__ __forceinline__ void stage_key_scales(Words<NB> dk, int live, int lane,
                                                 uint32_t (*to)[sub_of(NB) / 2]) {
    keep_live<NB>(dk, live);
#pragma unroll
    for (int i = 0; i < NB; i++) {
        const half2v d = halves(__builtin_amdgcn_perm(
            dk.w[(NB + i) >> 1], dk.w[i >> 1],
            ((NB + i) & 1 ? 0x07060000u : 0x05040000u) | (i & 1 ? 0x0302u : 0x0100u)));
        // an infinite scale becomes NaN, as it would times a code of 8 (times the block's sum it would
        // be a score of -inf as well, a key of no weight)
        to[i][lane] = word(__builtin_elementwise_fma(d, half2v{0, 0}, d));
    }
}
// The exponent that bounds the largest scale of a position's values, max_b |dv|
// < 2^ev.  A position with an infinite or NaN scale gets ev = inf, which turns
// the reference of a row that sees it infinite and its result NaN, and scales of
// 0, so that the rows that do not see it have no 0 * NaN.
struct Sizes {
    int e[2];
    bool bad[2];
    __device__ __forceinline__ float down(int i) const {  // 2^-e
        return bad[i] ? 0.0f : __uint_as_float((uint32_t)(127 - e[i]) << 23);
    }
};
template <int NB>
__device__ __forceinline__ Sizes sizes_of(const Words<NB>& dv) {
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2 * NB; i++) {
        const uint32_t m = half_bits(dv.w[i >> 1], i & 1) & 0x7FFFu;
        top[i / NB] = m > top[i / NB] ? m : top[i / NB];
    }
    Sizes z;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        z.e[i] = (int)(top[i] >> 10) - 14;
        z.bad[i] = top[i] >= 0x7C00u;
    }
    return z;
}
template <int NB>
__device__ __forceinline__ void stage_value_sizes(Words<NB> dv, int live, int lane, float* ev) {
    keep_live<NB>(dv, live);
    const Sizes z = sizes_of<NB>(dv);
#pragma unroll
    for (int i = 0; i < 2; i++) ev[2 * lane + i] = z.bad[i] ? INFINITY : (float)z.e[i];
}
// The values' scales as dv 2^-ev, below 1, and 2^-ev.  True if a scale of the lane's live positions
// is SMALL beside the largest of its position.
template <int NB>
__device__ __forceinline__ bool stage_value_scales(Words<NB> dv, int live, int lane,
                                                   uint32_t (*to)[sub_of(NB) / 2], float* down) {
    keep_live<NB>(dv, live);
    const Sizes z = sizes_of<NB>(dv);
    // bytes 0..3 are the lane's own, 4..7 the other's: even lanes take both low halves
    const uint32_t pick = lane & 1 ? 0x03020706u : 0x05040100u;
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        f[i] = z.down(i);
        down[2 * lane + i] = f[i];
    }
    ushort2v least = {0x7FFF, 0x7FFF};
#pragma unroll
    for (int i = 0; i < NB; i++) {
        half2v v = {half_of(dv.w[i >> 1], i & 1), half_of(dv.w[(NB + i) >> 1], (NB + i) & 1)};
        v[0] = z.bad[0] ? (_Float16)0.0f : (_Float16)((float)v[0] * f[0]);
        v[1] = z.bad[1] ? (_Float16)0.0f : (_Float16)((float)v[1] * f[1]);
        // the lanes of positions 0, 1 and 2, 3 exchange to words of positions 0, 2 and 1, 3, the
        // order of the code words
        const uint32_t own = word(v);
        least = __builtin_elementwise_min(least, ushorts(own & 0x7FFF7FFFu));
        to[i][lane] = __builtin_amdgcn_perm(dpp_bits<DPP_XOR1>(own), own, pick);
    }
    return (live > 0 && !z.bad[0] && least[0] < SMALL_BITS) ||
           (live > 1 && !z.bad[1] && least[1] < SMALL_BITS);
}
// The blocks (bits) of a run in which some position's scale is SMALL and some other's is not 0, from the
// scales of two positions a lane; `live` 0 for lanes without any.
template <int NB>
__device__ __forceinline__ uint32_t blocks_apart(Words<NB> dv, int live) {
    keep_live<NB>(dv, live);
    const Sizes z = sizes_of<NB>(dv);
    uint32_t blocks = 0;
#pragma unroll
    for (int i = 0; i < NB; i++) {
        const float v[2] = {fabsf((float)half_of(dv.w[i >> 1], i & 1)),
                            fabsf((float)half_of(dv.w[(NB + i) >> 1], (NB + i) & 1))};
        bool small = false, some = false;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            small |= live > j && !z.bad[j] && v[j] * z.down(j) < SMALL;
            some |= !z.bad[j] && v[j] > 0.0f;
        }
        if (__ballot(small) && __ballot(some)) blocks |= 1u << i;
    }
    return blocks;
}

// PACK: at most 8 rows share a key/value head in the tile.  The 16 columns of
// a product then hold them twice, and each half of the columns keeps its own
// positions: the tiles of 16 positions of even number in columns 0..7, those of
// odd number in columns 8..15.  Scores, weights and their split are so done for
// two tiles at a time.  The values' sums run over the even
// tiles, move across, and go on over the odd tiles, which is the order of the
// sums in every variant.
//
// What bounds it: with few rows the loads' latency and the VALU, 58 % busy (131072 positions, 46 us
// with the join), with many the VALU (about 1670 instructions a wave and run, a third of them
// unpacking, beside 128 matrix instructions: 77 % busy on four chunks of 256 tokens, 142 us).  So three
// waves a SIMD: the rows' two parts, the same for the four waves, wait in LDS, and a wave's sums take
// the place of its scales (32 sequences of 301..8191: 57 us with the join, an eighth more with the rows
// in registers and two waves).  With 16 rows and 128 elements ten registers are spilled, nearly all
// before the loop of the runs.
template <int NB, bool PACK>
__global__ __launch_bounds__(64 * WAVES, NB <= 4 ? 3 : 2) void k_attn(AttnArgs a, Plan plan) {
    const KvArgs& kv = a.kv;
    constexpr int D = 32 * NB, SUB = sub_of(NB), SEG = seg_of(NB), TILES = SUB / 16;
    constexpr int ROWS = PACK ? 8 : 16;           // rows of a tile
    constexpr int SLOTS = PACK ? TILES / 2 : TILES;  // tiles of positions a column sees
    constexpr int NBP = NB < 4 ? NB : 4;          // blocks joined at a time
    constexpr int LD = 32 * NBP + 4;
    constexpr int PER_ROW = 64 * WAVES / ROWS;    // threads that join a row
    // A wave's own part: the scales of its run ([block][position], fp16), which nobody else reads,
    // and in their place, once it is done with them, its sums of the run for all to join.
    struct Scales {
        uint32_t dk[NB][SUB / 2], dv[NB][SUB / 2];
        float ev[SUB], down[SUB];
    };
    union Own {
        Scales s;
        float o[ROWS * LD];
    };
    __shared__ __align__(16) Own s_own[WAVES];
    __shared__ __align__(16) float s_r[ROWS][WAVES], s_l[ROWS][WAVES];
    __shared__ __align__(16) uint4 s_q[2 * NB][64];  // the rows' two parts, the same for every wave

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & (ROWS - 1), par = PACK ? (lane >> 3) & 1 : 0, g = lane >> 4;
    const int G = a.Hq / kv.Hkv;
    const int head = blockIdx.x % kv.Hkv;
    int at = blockIdx.x / kv.Hkv;
    const int split = at % plan.splits;
    const int tile = plan.tiles - 1 - at / plan.splits;  // long rows first

    int b, first;
    if (!locate<ROWS>(kv, G, tile, lane, b, first)) return;
    const Seq s = seq_of(kv, b);
    const int64_t rows64 = (int64_t)s.n * G;
    if (first >= rows64) return;
    const int rows = (int)rows64;
    const int last = first + ROWS < rows ? first + ROWS - 1 : rows - 1;
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

    // What a wave holds ahead of a run of SUB positions: the pages of its tiles (lane u of
    // TILES: where tile u's K codes begin; its V codes, 16 positions of the same size, are `codes`
    // further), the K codes, and the scales of two positions a lane.
    const int page_tokens = 1 << kv.log2p;
    const int64_t codes = (int64_t)(16 * NB) << kv.log2p;
    const int32_t* table = kv.table + (int64_t)b * kv.table_stride;
    int pg = -1;
    uint32_t there = 0, at_lo = 0, at_hi = 0;
    Words<NB> cw[TILES], dk, dv;  // codes: keys, then values, then the next run's keys
    const auto works = [&](int seg) {
        const int t0 = seg * SEG + wave * SUB;
        return seg < seg1 && t0 < t_end && t0 + SUB > t_begin;
    };
    const auto fetch_pages = [&](int seg) {
        const int t = seg * SEG + wave * SUB + 16 * lane;
        pg = -1;
        if (works(seg) && lane < TILES && t < s.len) pg = table[t >> kv.log2p];
    };
    const auto tile_codes = [&](int u) {
        const uint64_t at = (uint32_t)__builtin_amdgcn_readlane(at_lo, u) |
                            (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_hi, u) << 32;
        return kv.pages + at;
    };
    // The scales, and where the codes are, then the keys of a run.  Both without a branch, whose
    // other side would keep a second copy of all the registers: where there is no next run, the
    // lanes read one address of page 0.
    uint32_t lane_k = 0;
    const auto fetch_scales = [&](int seg) {
        const int t0 = seg * SEG + wave * SUB;
        const bool ok = pg >= 0 && (int64_t)pg < kv.n_pages;
        there = (uint32_t)__ballot(ok);  // tiles that have a page
        const int p = ok ? pg : 0;       // the others read page 0, which is not used
        const int64_t at_k = ((int64_t)p * kv.Hkv + head) * kv.head_bytes +
                             (int64_t)((t0 + 16 * lane) & (page_tokens - 1)) * (16 * NB);
        at_lo = (uint32_t)at_k;
        at_hi = (uint32_t)(at_k >> 32);
        const int u = lane >> 3, t = t0 + 16 * u + 2 * (lane & 7);
        const uint8_t* hd = head_of(kv, __shfl(p, u), head) + 2 * codes +
                            (int64_t)(t & (page_tokens - 1)) * 2 * NB;
        dk = load_words<NB>(hd);
        dv = load_words<NB>(hd + ((int64_t)(2 * NB) << kv.log2p));
        lane_k = works(seg) ? (lane & 15) * (16 * NB) + g * (4 * NB) : 0;
    };
    // (an offset that is seen to be 32 bits wide where it is used stays beside the tile's address, which
    // all lanes share, in the load; otherwise every load adds the two first)
    const auto fetch_keys = [&] {
        uint32_t off = lane_k;
        asm("" : "+v"(off));
#pragma unroll
        for (int u = 0; u < TILES; u++) cw[u] = load_words<NB>(tile_codes(u) + off);
    };
    fetch_pages(seg0);

    float factor;
    int pos;
    {
        half8 qh[NB], ql[NB];
        prepare_q<NB>(a, s, head, G, first + n, rows, g, qh, ql, factor, pos, [&] {
            fetch_scales(seg0);
            fetch_keys();
            fetch_pages(seg0 + 1);
        });
#pragma unroll
        for (int bb = 0; bb < NB; bb++)
            if ((bb & (WAVES - 1)) == wave) {
                __builtin_memcpy(&s_q[2 * bb][lane], &qh[bb], 16);
                __builtin_memcpy(&s_q[2 * bb + 1][lane], &ql[bb], 16);
            }
    }
    __syncthreads();

    // the joined state: thread (row tid / PER_ROW, part tid % PER_ROW) holds its share of every
    // NBP blocks
    const int jr = tid / PER_ROW, jp = tid % PER_ROW;
    constexpr int SHARE = 32 * NB / PER_ROW;
    float O[SHARE], L = 0.0f, RR = NO_KEY;
#pragma unroll
    for (int i = 0; i < SHARE; i++) O[i] = 0.0f;
    const auto row_of = [&](int i) {  // row i of the tile among all rows of the call
        return (int64_t)(s.q0 + (first + i) / G) * a.Hq + head * G + (first + i) % G;
    };
    const Unpack unpack;
    const uint32_t q_at = lds_at(&s_q[0][lane]);
    const uint32_t dk_at = lds_at(&s_own[wave].s.dk[0][8 * par + 2 * g]);
    const uint32_t dv_at = lds_at(&s_own[wave].s.dv[0][8 * par + 2 * g]);
    const uint32_t ev_at = lds_at(&s_own[wave].s.ev[16 * par + 4 * g]);
    const uint32_t down_at = lds_at(&s_own[wave].s.down[16 * par + 4 * g]);

    for (int seg = seg0; seg < seg1; seg++) {
        const int t0 = seg * SEG + wave * SUB;
        const bool work = works(seg);
        f4 o[2 * NB];
        float r = NO_KEY, l = 0.0f;
        if (work) {
            const bool masked = t0 + SUB > pos_lo + 1 || (a.window && t0 <= pos_hi - a.window) ||
                                there != (1u << TILES) - 1;
            const uint32_t here = there;
            const int mine = t0 + 16 * (lane >> 3) + 2 * (lane & 7);
            const int live = ((here >> (lane >> 3)) & 1) ? s.len - mine : 0;
            bool small = false;
            if (TILES == 8 || lane < 8 * TILES) {
                stage_key_scales<NB>(dk, live, lane, s_own[wave].s.dk);
                stage_value_sizes<NB>(dv, live, lane, s_own[wave].s.ev);
                small = stage_value_scales<NB>(dv, live, lane, s_own[wave].s.dv, s_own[wave].s.down);
            }
            uint32_t apart = 0;
            if (__ballot(small)) apart = blocks_apart<NB>(dv, live);
            apart = uniform(apart);
            wave_sync();

            // scores: sc[U][i] of row n at position t0 + 16 u + 4g + i, u the slot's tile
            // (the rows' parts and the block scales of a lane's four positions are read from LDS one
            // step ahead of use, here and below: the scheduler left to itself waits for each)
            f4 sc[SLOTS];
            const auto scales = [&](uint32_t from, int U, int bb) {
                return lds_read<u2>(from + 4 * (bb * (SUB / 2) + 8 * (PACK ? 2 * U : U)));
            };
            half8 qhn, qln;
            u2 dn[2];
            const auto ahead = [&](int P, int bb) {
                qhn = lds_read<half8>(q_at + 2048 * bb);
                qln = lds_read<half8>(q_at + 2048 * bb + 1024);
                dn[0] = scales(dk_at, PACK ? P : 2 * P, bb);
                if constexpr (!PACK) dn[1] = scales(dk_at, 2 * P + 1, bb);
            };
            ahead(0, 0);
#pragma unroll
            for (int P = 0; P < TILES / 2; P++) {
                f4 z[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                f4 accp[2];  // a step's results are used in the next one, behind its products
                u2 dp[2];
                const auto take = [&] {
#pragma unroll
                    for (int h = 0; h < (PACK ? 1 : 2); h++)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            z[h][i] = __builtin_fmaf((float)half_of(dp[h][i >> 1], i & 1),
                                                     PACK && par ? accp[1][i] : accp[h][i], z[h][i]);
                };
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    const half8 qh = qhn, ql = qln;
                    const u2 d[2] = {dn[0], dn[1]};
                    if (bb + 1 < NB) ahead(P, bb + 1);
                    else if (P + 1 < TILES / 2) ahead(P + 1, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    half8 ko[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t w = cw[2 * P + h].w[bb], v = w >> 8;
                        ko[h] = operand(unpack.low(w), unpack.high(w), unpack.low(v), unpack.high(v));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    f4 acc[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) acc[h] = mfma(ko[h], ql, f4{0, 0, 0, 0});
#pragma unroll
                    for (int h = 0; h < 2; h++) acc[h] = mfma(ko[h], qh, acc[h]);
                    if (bb) take();
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        accp[h] = acc[h];
                        dp[h] = d[h];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                take();
                // in base 2, relative to the size of the position's values
#pragma unroll
                for (int h = 0; h < (PACK ? 1 : 2); h++) {
                    const f4 e = lds_read<f4>(ev_at + 4 * 16 * (2 * P + h));
                    const int U = PACK ? P : 2 * P + h;
#pragma unroll
                    for (int i = 0; i < 4; i++) sc[U][i] = __builtin_fmaf(z[h][i], factor, e[i]);
                }
            }
            // the values' codes take the keys' registers and arrive during the softmax
            uint32_t lane_v = lane * (4 * NB);
            asm("" : "+v"(lane_v));
#pragma unroll
            for (int u = 0; u < TILES; u++)
                cw[u] = load_words<NB>(tile_codes(u) + codes + lane_v);

            // weights
            if (masked) {
                // a position is seen in (rel - window, rel]
                const int rel = pos - t0 - 4 * g - 16 * par;
                const int from = a.window ? rel - a.window : -(1 << 30);
#pragma unroll
                for (int U = 0; U < SLOTS; U++) {
                    const int off = PACK ? 32 * U : 16 * U;
                    const int hi = (here >> (PACK ? 2 * U + par : U)) & 1 ? rel : -(1 << 30);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        sc[U][i] = off + i <= hi && off + i > from ? sc[U][i] : -INFINITY;
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int U = 0; U < SLOTS; U++)
#pragma unroll
                for (int i = 0; i < 4; i++) top = fmaxf(top, sc[U][i]);
            if constexpr (PACK) top = fmaxf(top, across8(top));
            top = max_rows(top);
            const float ref = reference(top);
            float sum[2] = {0.0f, 0.0f};  // over the even and the odd tiles
            Split p[SLOTS][2];            // positions 0, 2 and 1, 3
#pragma unroll
            for (int U = 0; U < SLOTS; U++) {
                const f4 down = lds_read<f4>(down_at + 4 * 16 * (PACK ? 2 * U : U));
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    sc[U][i] = exp2_raw(sc[U][i] - ref);
                    float& l2 = sum[PACK ? 0 : U & 1];
                    l2 = __builtin_fmaf(sc[U][i], down[i], l2);
                }
                p[U][0] = two_parts(sc[U][0], sc[U][2]);
                p[U][1] = two_parts(sc[U][1], sc[U][3]);
            }
            l = sum[0] + (PACK ? across8(sum[0]) : sum[1]);
            l = sum_rows(l);
            // no maximum: nothing seen, or NaN scores, whose sum is NaN and stays
            r = top == -INFINITY && l == 0.0f ? NO_KEY : ref;

            // Values, two tiles of one parity (32 positions) at a product: the weights of slots
            // U0, U1 times the block's scales.
            const auto split_weights = [&](int U0, int U1, u2 d0, u2 d1, half8& ph,
                                           half8& pl) {
                const Split a0 = times(p[U0][0], halves(d0[0])), a1 = times(p[U0][1], halves(d0[1]));
                const Split a2 = times(p[U1][0], halves(d1[0])), a3 = times(p[U1][1], halves(d1[1]));
                ph = operand(word(a0.h), word(a1.h), word(a2.h), word(a3.h));
                pl = operand(word(a0.l), word(a1.l), word(a2.l), word(a3.l));
            };
            const auto add_values = [&](int u0, int u1, int bb, half8 ph, half8 pl, bool fresh) {
                const uint32_t w0 = cw[u0].w[bb], w1 = cw[u1].w[bb];
                const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
                const half8 even =
                    operand(unpack.low(w0), unpack.low(v0), unpack.low(w1), unpack.low(v1));
                const half8 odd =
                    operand(unpack.high(w0), unpack.high(v0), unpack.high(w1), unpack.high(v1));
                const f4 zero = {0, 0, 0, 0};
                o[2 * bb] = mfma(even, pl, fresh ? zero : o[2 * bb]);
                o[2 * bb + 1] = mfma(odd, pl, fresh ? zero : o[2 * bb + 1]);
                o[2 * bb] = mfma(even, ph, o[2 * bb]);
                o[2 * bb + 1] = mfma(odd, ph, o[2 * bb + 1]);
            };
            if constexpr (PACK) {
                constexpr int Q = TILES / 4;
                u2 dn[SLOTS];
#pragma unroll
                for (int U = 0; U < SLOTS; U++) dn[U] = scales(dv_at, U, 0);
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    half8 ph[Q], pl[Q];
                    u2 dc[SLOTS];
#pragma unroll
                    for (int U = 0; U < SLOTS; U++) dc[U] = dn[U];
                    if (bb + 1 < NB) {
#pragma unroll
                        for (int U = 0; U < SLOTS; U++) dn[U] = scales(dv_at, U, bb + 1);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int q = 0; q < Q; q++) {
                        split_weights(2 * q, 2 * q + 1, dc[2 * q], dc[2 * q + 1], ph[q], pl[q]);
                        add_values(4 * q, 4 * q + 2, bb, ph[q], pl[q], q == 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        o[2 * bb][i] = across8(o[2 * bb][i]);
                        o[2 * bb + 1][i] = across8(o[2 * bb + 1][i]);
                    }
#pragma unroll
                    for (int q = 0; q < Q; q++)
                        add_values(4 * q + 1, 4 * q + 3, bb, ph[q], pl[q], false);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                // tiles u and u + 2, even before odd
                const auto tile_of = [&](int q) { return 4 * (q % (TILES / 4)) + q / (TILES / 4); };
                u2 n0 = scales(dv_at, tile_of(0), 0), n1 = scales(dv_at, tile_of(0) + 2, 0);
#pragma unroll
                for (int q = 0; q < TILES / 2; q++) {
                    const int u = tile_of(q);
#pragma unroll
                    for (int bb = 0; bb < NB; bb++) {
                        const u2 d0 = n0, d1 = n1;
                        if (bb + 1 < NB || q + 1 < TILES / 2) {
                            const int un = bb + 1 < NB ? u : tile_of(q + 1), bn = bb + 1 < NB ? bb + 1 : 0;
                            n0 = scales(dv_at, un, bn);
                            n1 = scales(dv_at, un + 2, bn);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        half8 ph, pl;
                        split_weights(u, u + 2, d0, d1, ph, pl);
                        add_values(u, u + 2, bb, ph, pl, q == 0);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
#pragma nounroll
            for (; apart; apart &= apart - 1) {
                const int bb = __builtin_ctz(apart);
                const Exact x = exact_sums<NB>(a, unpack, table, s.len, head, t0, bb, factor, ref, pos, lane,
                                               [&](int b, half8& qh, half8& ql) {
                                                   qh = lds_read<half8>(q_at + 2048 * b);
                                                   ql = lds_read<half8>(q_at + 2048 * b + 1024);
                                               });
#pragma unroll
                for (int i = 0; i < 2 * NB; i++)
                    if (x.taken && bb == i / 2) o[i] = x.sum[i & 1];
                all_arrived();
            }
        }
        fetch_scales(seg + 1);
        fetch_keys();
        fetch_pages(seg + 2);

        // join the waves' parts of the segment, then the segment to the state
        wave_sync();  // the sums take the place of the scales
        if (lane < ROWS) {
            s_r[n][wave] = r;
            s_l[n][wave] = l;
        }
        f4 rw, lw;
        Join jw[WAVES], jn{1.0f, 0.0f};
#pragma unroll
        for (int b0 = 0; b0 < NB; b0 += NBP) {
            const int nbp = NB - b0 < NBP ? NB - b0 : NBP;
            if (work && (!PACK || par)) {
#pragma unroll
                for (int bb = 0; bb < nbp; bb++) {
                    const f4 x = o[2 * (b0 + bb)], y = o[2 * (b0 + bb) + 1];
                    float* to = &s_own[wave].o[n * LD + 32 * bb + 8 * g];
                    *reinterpret_cast<f4*>(to) = f4{x[0], y[0], x[1], y[1]};
                    *reinterpret_cast<f4*>(to + 4) = f4{x[2], y[2], x[3], y[3]};
                }
            }
            __syncthreads();
            // without branches, so that all reads are in flight at once; a run without keys for the
            // row has the factors 1 and 0 or 1, and -0 in the place of its sums adds nothing at all
            const int per = 32 * nbp / PER_ROW, o0 = 32 * b0 / PER_ROW;
            float part[WAVES][32 * NBP / PER_ROW], v[32 * NBP / PER_ROW];
            if (b0 == 0) {
                rw = *reinterpret_cast<const f4*>(s_r[jr]);
                lw = *reinterpret_cast<const f4*>(s_l[jr]);
            }
#pragma unroll
            for (int w = 0; w < WAVES; w++)
#pragma unroll
                for (int i = 0; i < per; i++) part[w][i] = s_own[w].o[jr * LD + jp * per + i];
            __builtin_amdgcn_sched_barrier(0);
            if (b0 == 0) {
                float sr = NO_KEY, sl = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; w++) {
                    jw[w] = join(sr, rw[w]);
                    sl = joined(sl, lw[w], jw[w]);
                }
                if (plan.splits == 1) {
                    jn = join(RR, sr);
                    L = joined(L, sl, jn);
                } else if (jp == 0 && first + jr < rows) {
                    float* rl = part_rl(a, row_of(jr), plan.segs, seg);
                    rl[0] = sr;
                    rl[1] = sl;
                }
            }
#pragma unroll
            for (int i = 0; i < per; i++) v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; w++)
#pragma unroll
                for (int i = 0; i < per; i++)
                    v[i] = joined(v[i], rw[w] != NO_KEY ? part[w][i] : -0.0f, jw[w]);
            if (plan.splits == 1) {
#pragma unroll
                for (int i = 0; i < per; i++) O[o0 + i] = joined(O[o0 + i], v[i], jn);
            } else if (first + jr < rows) {
                float* to = part_o(a, row_of(jr), plan.segs, seg) + 32 * b0 + jp * per;
#pragma unroll
                for (int i = 0; i < per; i++) to[i] = v[i];
            }
            __syncthreads();
        }
    }
    if (plan.splits > 1 || first + jr >= rows) return;
    float* out = a.out + row_of(jr) * D;
#pragma unroll
    for (int b0 = 0; b0 < NB; b0 += NBP) {
        const int per = 32 * (NB - b0 < NBP ? NB - b0 : NBP) / PER_ROW, o0 = 32 * b0 / PER_ROW;
#pragma unroll
        for (int i = 0; i < per; i++) out[32 * b0 + jp * per + i] = result(O[o0 + i], L);
    }
}

// Many rows: 64 of them a workgroup, 16 a wave, over the same positions.  The
// waves unpack a run of SUB positions together, a quarter each, into LDS in
// operand order, and each takes all of it from there: 144 instructions of
// unpacking a wave and run instead of 576, against 64 LDS reads.  Keys (and what the
// scores need) are replaced while values are worked on, and values while scores
// are, from words loaded a run ahead; two barriers a run.  Every wave joins its
// runs to segments and its segments to its state itself, in the steps of k_attn.
// 256 registers, so two waves a SIMD: VALU 59 %, LDS 32 %, matrix cores 23 % busy.
template <int NB>
__global__ __launch_bounds__(64 * WAVES, 2) void k_attn_wide(AttnArgs a, Plan plan) {
    static_assert(sub_of(NB) == 128 && WAVES == 4, "a wave unpacks two tiles of keys and a pair of values");
    const KvArgs& kv = a.kv;
    constexpr int D = 32 * NB, SUB = 128, TILES = 8, ROWS = 64;
    extern __shared__ __align__(16) uint8_t lds[];
    uint4 (*s_k)[64] = reinterpret_cast<uint4 (*)[64]>(lds);                 // [TILES * NB][lane]
    uint4 (*s_v)[64] = s_k + TILES * NB;                                     // [pair * NB * 2][lane]
    uint32_t (*s_dk)[SUB / 2] = reinterpret_cast<uint32_t (*)[SUB / 2]>(s_v + TILES * NB);
    uint32_t (*s_dv)[SUB / 2] = s_dk + NB;
    float* s_ev = reinterpret_cast<float*>(s_dv + NB);
    float* s_down = s_ev + SUB;
    uint32_t* s_apart = reinterpret_cast<uint32_t*>(s_down + SUB);  // blocks, of the values in LDS

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int G = a.Hq / kv.Hkv;
    const int head = blockIdx.x % kv.Hkv;
    const int tile = plan.tiles - 1 - blockIdx.x / kv.Hkv;  // long rows first
    int b, first;
    if (!locate<ROWS>(kv, G, tile, lane, b, first)) return;
    const Seq s = seq_of(kv, b);
    const int64_t rows64 = (int64_t)s.n * G;
    if (first >= rows64) return;
    const int rows = (int)rows64;
    // positions that the workgroup's rows see, and this wave's
    const auto pos_of = [&](int rr) { return s.len - s.n + (rr < rows ? rr : rows - 1) / G; };
    const auto begin_of = [&](int p) { return a.window && p + 1 > a.window ? p + 1 - a.window : 0; };
    const int t_end = pos_of(first + ROWS - 1) + 1, t_begin = begin_of(pos_of(first));
    const int row0 = first + 16 * wave;
    const bool mine = row0 < rows;
    const int pos_lo = pos_of(row0), pos_hi = pos_of(row0 + 15);
    const int w_end = mine ? pos_hi + 1 : 0, w_begin = begin_of(pos_lo);
    const int sub0 = t_begin / SUB, sub1 = t_end > 0 ? (t_end + SUB - 1) / SUB : 0;

    const int page_tokens = 1 << kv.log2p;
    const int64_t codes = (int64_t)(16 * NB) << kv.log2p;
    const int32_t* table = kv.table + (int64_t)b * kv.table_stride;
    const Unpack unpack;
    int pg = -1;
    uint32_t there = 0;
    Words<NB> kw[2], vw[2], dd;
    const auto tile_of = [](int q) { return 4 * (q & 1) + (q >> 1); };  // of a pair: this and two on
    const auto fetch_pages = [&](int sub) {
        const int t = sub * SUB + 16 * lane;
        pg = -1;
        if (sub < sub1 && lane < TILES && t < s.len) pg = table[t >> kv.log2p];
    };
    // the wave's share: tiles 2w, 2w + 1 of keys, pair w of values, wave 0 the keys' and wave 1 the
    // values' scales; fetch_keys notes which tiles have a page and where all of them lie
    uint32_t at_lo = 0, at_hi = 0;
    const auto tile_codes = [&](int u) {
        return kv.pages + ((uint32_t)__builtin_amdgcn_readlane(at_lo, u) |
                           (uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_hi, u) << 32);
    };
    const auto fetch_keys = [&](int sub) {
        const int t0 = sub * SUB;
        const bool ok = pg >= 0 && (int64_t)pg < kv.n_pages;
        there = (uint32_t)__ballot(ok);
        const int p = ok ? pg : 0;  // tiles without a page read page 0, which is not used
        const int64_t at = ((int64_t)p * kv.Hkv + head) * kv.head_bytes +
                           (int64_t)((t0 + 16 * lane) & (page_tokens - 1)) * (16 * NB);
        at_lo = (uint32_t)at;
        at_hi = (uint32_t)(at >> 32);
#pragma unroll
        for (int i = 0; i < 2; i++)
            kw[i] = load_words<NB>(tile_codes(2 * wave + i) + n * (16 * NB) + g * (4 * NB));
        if (wave < 2) {
            const int u = lane >> 3, t = t0 + 16 * u + 2 * (lane & 7);
            dd = load_words<NB>(head_of(kv, __shfl(p, u), head) + 2 * codes +
                                ((int64_t)(wave ? 2 * NB : 0) << kv.log2p) +
                                (int64_t)(t & (page_tokens - 1)) * 2 * NB);
        }
    };
    const auto fetch_values = [&] {
        const int u = tile_of(wave);
#pragma unroll
        for (int i = 0; i < 2; i++)
            vw[i] = load_words<NB>(tile_codes(u + 2 * i) + codes + lane * (4 * NB));
    };
    const auto live_of = [&](int sub, uint32_t have) {
        const int u = lane >> 3, t = sub * SUB + 16 * u + 2 * (lane & 7);
        return ((have >> u) & 1) ? s.len - t : 0;
    };
    const auto stage_keys = [&](int sub, uint32_t have) {
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int bb = 0; bb < NB; bb++) {
                const uint32_t w = kw[i].w[bb], v = w >> 8;
                s_k[(2 * wave + i) * NB + bb][lane] =
                    make_uint4(unpack.low(w), unpack.high(w), unpack.low(v), unpack.high(v));
            }
        if (wave == 0) stage_key_scales<NB>(dd, live_of(sub, have), lane, s_dk);
        if (wave == 1) stage_value_sizes<NB>(dd, live_of(sub, have), lane, s_ev);
    };
    const auto stage_values = [&](int sub, uint32_t have) {
#pragma unroll
        for (int bb = 0; bb < NB; bb++) {
            const uint32_t w0 = vw[0].w[bb], w1 = vw[1].w[bb], v0 = w0 >> 8, v1 = w1 >> 8;
            uint4 (*to)[64] = s_v + (wave * NB + bb) * 2;
            to[0][lane] = make_uint4(unpack.low(w0), unpack.low(v0), unpack.low(w1), unpack.low(v1));
            to[1][lane] = make_uint4(unpack.high(w0), unpack.high(v0), unpack.high(w1), unpack.high(v1));
        }
        if (wave == 1) {
            const int live = live_of(sub, have);
            uint32_t apart = 0;
            if (__ballot(stage_value_scales<NB>(dd, live, lane, s_dv, s_down)))
                apart = blocks_apart<NB>(dd, live);
            if (lane == 0) *s_apart = apart;
        }
    };
    const uint32_t k_at = lds_at(&s_k[0][lane]), v_at = lds_at(&s_v[0][lane]);
    const uint32_t dk_at = lds_at(&s_dk[0][2 * g]), dv_at = lds_at(&s_dv[0][2 * g]);
    const uint32_t ev_at = lds_at(s_ev + 4 * g), down_at = lds_at(s_down + 4 * g);

    fetch_pages(sub0);
    half8 qh[NB], ql[NB];
    float factor;
    int pos;
    prepare_q<NB>(a, s, head, G, row0 + n, rows, g, qh, ql, factor, pos, [&] {
        if (sub0 < sub1) {
            fetch_keys(sub0);
            fetch_values();
        }
        fetch_pages(sub0 + 1);
    });
    if (sub0 < sub1) {
        stage_keys(sub0, there);
        stage_values(sub0, there);
    }
    __syncthreads();

    // The segment's state: row n of the wave, elements 32b + 8g + 2i (first of a pair of f4) and + 1.
    // The state over whole segments would take as many registers again: its sums wait in the
    // row's place in out between segments.
    const int rr = row0 + n;
    float* out = a.out + 8 * g;
    if (rr < rows) out += ((int64_t)(s.q0 + rr / G) * a.Hq + head * G + rr % G) * D;
    f4 os[2 * NB];
    float R = NO_KEY, L = 0.0f, rs = NO_KEY, ls = 0.0f;
    bool begun = false;
#pragma unroll
    for (int i = 0; i < 2 * NB; i++) os[i] = f4{0, 0, 0, 0};
    if (sub0 >= sub1 && rr < rows) {  // rows that see no position
#pragma unroll
        for (int i = 0; i < 2 * NB; i++) *reinterpret_cast<f4*>(out + 32 * (i / 2) + 4 * (i & 1)) = os[i];
    }

    for (int sub = sub0; sub < sub1; sub++) {
        const int t0 = sub * SUB;
        const bool work = t0 < w_end && t0 + SUB > w_begin;
        const bool masked = t0 + SUB > pos_lo + 1 || (a.window && t0 <= pos_hi - a.window) || there != 0xFF;
        const uint32_t here = there;
        const bool more = sub + 1 < sub1;
        f4 sc[TILES];
        if (work) {
            // operands and scales are read one step ahead
            half8 kn[NB];
            u2 dn[NB];
            const auto ahead = [&](int u) {
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    kn[bb] = lds_read<half8>(k_at + 1024 * (u * NB + bb));
                    dn[bb] = lds_read<u2>(dk_at + 4 * (bb * (SUB / 2) + 8 * u));
                }
            };
            ahead(0);
#pragma unroll
            for (int u = 0; u < TILES; u++) {
                half8 ko[NB];
                u2 d[NB];
#pragma unroll
                for (int bb = 0; bb < NB; bb++) {
                    ko[bb] = kn[bb];
                    d[bb] = dn[bb];
                }
                const f4 e = lds_read<f4>(ev_at + 64 * u);
                if (u + 1 < TILES) ahead(u + 1);
                __builtin_amdgcn_sched_barrier(0);
                f4 acc[NB], z = {0, 0, 0, 0};
#pragma unroll
                for (int bb = 0; bb < NB; bb++) acc[bb] = mfma(ko[bb], ql[bb], f4{0, 0, 0, 0});
#pragma unroll
                for (int bb = 0; bb < NB; bb++) acc[bb] = mfma(ko[bb], qh[bb], acc[bb]);
#pragma unroll
                for (int bb = 0; bb < NB; bb++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        z[i] = __builtin_fmaf((float)half_of(d[bb][i >> 1], i & 1), acc[bb][i], z[i]);
#pragma unroll
                for (int i = 0; i < 4; i++) sc[u][i] = __builtin_fmaf(z[i], factor, e[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the next run's keys arrive during the softmax, its values while these are worked on
        if (more) fetch_keys(sub + 1);
        __syncthreads();  // every wave is done with the keys
        Split p[TILES][2];  // weights of positions 0, 2 and 1, 3 of each four
        Join js{1.0f, 0.0f};
        uint32_t apart = *s_apart;
        float ref = 0.0f;
        if (work) {
            if (masked) {
                const int rel = pos - t0 - 4 * g;
                const int from = a.window ? rel - a.window : -(1 << 30);
#pragma unroll
                for (int u = 0; u < TILES; u++) {
                    const int hi = (here >> u) & 1 ? rel : -(1 << 30);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        sc[u][i] = 16 * u + i <= hi && 16 * u + i > from ? sc[u][i] : -INFINITY;
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < TILES; u++)
#pragma unroll
                for (int i = 0; i < 4; i++) top = fmaxf(top, sc[u][i]);
            top = max_rows(top);
            ref = reference(top);
            float sum[2] = {0.0f, 0.0f};  // over the even and the odd tiles
#pragma unroll
            for (int u = 0; u < TILES; u++) {
                const f4 down = lds_read<f4>(down_at + 64 * u);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    sc[u][i] = exp2_raw(sc[u][i] - ref);
                    sum[u & 1] = __builtin_fmaf(sc[u][i], down[i], sum[u & 1]);
                }
                p[u][0] = two_parts(sc[u][0], sc[u][2]);
                p[u][1] = two_parts(sc[u][1], sc[u][3]);
                if (u & 1) __builtin_amdgcn_sched_barrier(0);
            }
            const float l = sum_rows(sum[0] + sum[1]);
            const float r = top == -INFINITY && l == 0.0f ? NO_KEY : ref;
            js = join(rs, r);
            ls = joined(ls, l, js);
        }
        if (more) {
            stage_keys(sub + 1, there);
            fetch_values();
        }
        fetch_pages(sub + 2);
        if (work) {
            half8 en, on;  // the next step's operands and scales
            u2 n0, n1;
            const auto next = [&](int bb, int q) {
                const int u = tile_of(q);
                en = lds_read<half8>(v_at + 1024 * ((q * NB + bb) * 2));
                on = lds_read<half8>(v_at + 1024 * ((q * NB + bb) * 2 + 1));
                n0 = lds_read<u2>(dv_at + 4 * (bb * (SUB / 2) + 8 * u));
                n1 = lds_read<u2>(dv_at + 4 * (bb * (SUB / 2) + 8 * u + 16));
            };
            // (the segment's state, to which exact sums are joined below, waits in memory, as the
            // registers are full; the compiler must not see through it and keep it in them)
            float before[8 * NB];
            apart = uniform(apart);
            if (apart) {
                float* to = before;
                asm volatile("" : "+v"(to));
#pragma unroll
                for (int i = 0; i < 8 * NB; i++) to[i] = os[i >> 2][i & 3];
                asm volatile("" : : "v"(to) : "memory");
                all_arrived();
            }
            next(0, 0);
#pragma unroll
            for (int bb = 0; bb < NB; bb++) {
                f4 o0 = {0, 0, 0, 0}, o1 = o0;
#pragma unroll
                for (int q = 0; q < TILES / 2; q++) {
                    const int u = tile_of(q);
                    const half8 even = en, odd = on;
                    const u2 d0 = n0, d1 = n1;
                    if (q + 1 < TILES / 2) next(bb, q + 1);
                    else if (bb + 1 < NB) next(bb + 1, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    const Split a0 = times(p[u][0], halves(d0[0])), a1 = times(p[u][1], halves(d0[1]));
                    const Split a2 = times(p[u + 2][0], halves(d1[0]));
                    const Split a3 = times(p[u + 2][1], halves(d1[1]));
                    const half8 ph = operand(word(a0.h), word(a1.h), word(a2.h), word(a3.h));
                    const half8 pl = operand(word(a0.l), word(a1.l), word(a2.l), word(a3.l));
                    o0 = mfma(even, pl, o0);
                    o1 = mfma(odd, pl, o1);
                    o0 = mfma(even, ph, o0);
                    o1 = mfma(odd, ph, o1);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    os[2 * bb][i] = joined(os[2 * bb][i], o0[i], js);
                    os[2 * bb + 1][i] = joined(os[2 * bb + 1][i], o1[i], js);
                }
            }
#pragma nounroll
            for (; apart; apart &= apart - 1) {
                const int bb = __builtin_ctz(apart);
                const float* from = before;
                asm volatile("" : "+v"(from) : : "memory");
                const Exact x = exact_sums<NB>(a, unpack, table, s.len, head, t0, bb, factor, ref, pos, lane,
                                               [&](int b, half8& h, half8& l) {
                                                   h = qh[b];
                                                   l = ql[b];
                                               });
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float y = joined(from[8 * bb + i], x.sum[i >> 2][i & 3], js);
#pragma unroll
                    for (int b = 0; b < NB; b++)
                        if (x.taken && bb == b) os[2 * b + (i >> 2)][i & 3] = y;
                }
                all_arrived();
            }
        }
        __syncthreads();  // every wave is done with the values
        if (more) stage_values(sub + 1, there);
        if ((sub & (WAVES - 1)) == WAVES - 1 || !more) {  // the segment is complete
            const Join jn = join(R, rs);
            L = joined(L, ls, jn);
            if (rr < rows) {
#pragma unroll
                for (int i = 0; i < 2 * NB; i++) {
                    f4* at = reinterpret_cast<f4*>(out + 32 * (i / 2) + 4 * (i & 1));
                    f4 x = {0, 0, 0, 0};
                    if (begun) x = *at;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float part = os[(i & ~1) + (e & 1)][2 * (i & 1) + (e >> 1)];
                        x[e] = joined(x[e], part, jn);
                        if (!more) x[e] = result(x[e], L);
                    }
                    *at = x;
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * NB; i++) os[i] = f4{0, 0, 0, 0};
            begun = true;
            rs = NO_KEY;
            ls = 0.0f;
        }
    }
}

template <int NB> constexpr int wide_lds() { return 2 * 8 * NB * 1024 + 2 * NB * 256 + 2 * 512 + 16; }

// Joins the segments of a row in ascending order, as k_attn does when it has
// them all: one workgroup per row, query head and W elements (all, or 32 where
// rows are few and segments many), one element a thread and the sum of the
// weights in one more.  Only a multiplication and an addition a segment stand
// in the chain: the references' running maxima come from a scan, and every
// part is multiplied by its factor on its way to LDS, LOT segments at a time,
// from where the chain takes four at a read.
template <int W>  // below 256
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int segs) {
    const KvArgs& kv = a.kv;
    constexpr int LOT = 8192 / W / 4 * 4 < 256 ? 8192 / W / 4 * 4 : 256;  // segments
    constexpr int LD = LOT + 4, HELD = (LOT * W / 4 + 255) / 256;
    __shared__ __align__(16) float s_x[(W + 1) * LD];  // part * b: [element, then the sum][segment]
    __shared__ __align__(16) float s_a[LD];
    __shared__ float s_b[LD], s_top[4];
    const int t = blockIdx.x / a.Hq, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int D = 32 * kv.nb;
    const int b = seq_of_row(kv, t);
    if (b < 0) return;
    const Seq s = seq_of(kv, b);
    if (t < s.q0 || t >= s.q0 + s.n) return;
    const int pos = s.len - s.n + (t - s.q0), SEG = seg_of(kv.nb);
    const int64_t row = blockIdx.x;
    const int lo = a.window && pos + 1 > a.window ? (pos + 1 - a.window) / SEG : 0;
    const int hi = pos < 0 ? lo : pos / SEG + 1;
    const float* po = part_o(a, row, segs, 0) + W * blockIdx.y;
    const float* rl = part_rl(a, row, segs, 0);
    float4 v[HELD];
    float r = NO_KEY, l = 0.0f;  // of segment c0 + tid
    const auto fetch = [&](int c0) {
        const int m = hi - c0 < LOT ? hi - c0 : LOT;
#pragma unroll
        for (int i = 0; i < HELD; i++) {
            const int at = tid + 256 * i, c = at / (W / 4), e = at % (W / 4);
            v[i] = make_float4(0, 0, 0, 0);
            if (c < m) v[i] = *reinterpret_cast<const float4*>(po + (int64_t)(c0 + c) * D + 4 * e);
        }
        const bool has = tid < m;
        r = has ? rl[2 * (int64_t)(c0 + tid)] : NO_KEY;
        l = has ? rl[2 * (int64_t)(c0 + tid) + 1] : 0.0f;
    };
    float O = 0.0f, R = NO_KEY;
    if (lo < hi) fetch(lo);
    for (int c0 = lo; c0 < hi; c0 += LOT) {
        const int m = hi - c0 < LOT ? hi - c0 : LOT;
        float top = r;  // maximum up to and with the thread's segment: in its wave, then in all
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float x = __shfl_up(top, o);
            if (lane >= o) top = fmaxf(top, x);
        }
        if (lane == 63) s_top[wave] = top;
        __syncthreads();
        float before = R;
        for (int w = 0; w < wave; w++) before = fmaxf(before, s_top[w]);
        const float up = __shfl_up(top, 1);
        if (lane) before = fmaxf(before, up);
        R = fmaxf(R, fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])));
        const Join j = join(before, r);
        if (tid < LOT) {  // segments past the last: a = 1, part 0
            const bool has = tid < m && r != NO_KEY;
            s_a[tid] = has ? j.a : 1.0f;
            s_b[tid] = has ? j.b : -1.0f;
            s_x[W * LD + tid] = has ? l * j.b : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < HELD; i++) {
            const int at = tid + 256 * i, c = at / (W / 4), e = at % (W / 4);
            if (c < LOT && c < m + 3) {  // the chain reads up to the next multiple of 4
                const float f = s_b[c];
                const bool has = !(f < 0.0f);  // (nothing was written for a segment without keys)
                float* to = &s_x[4 * e * LD + c];
                to[0] = has ? v[i].x * f : 0.0f;
                to[LD] = has ? v[i].y * f : 0.0f;
                to[2 * LD] = has ? v[i].z * f : 0.0f;
                to[3 * LD] = has ? v[i].w * f : 0.0f;
            }
        }
        __syncthreads();
        if (c0 + LOT < hi) fetch(c0 + LOT);
        if (tid <= W) {
#pragma unroll 4
            for (int i = 0; i < m; i += 4) {
                const f4 k = *reinterpret_cast<const f4*>(&s_a[i]);
                const f4 x = *reinterpret_cast<const f4*>(&s_x[tid * LD + i]);
#pragma unroll
                for (int e = 0; e < 4; e++) O = __builtin_fmaf(O, k[e], x[e]);
            }
        }
        __syncthreads();
    }
    if (tid == W) s_b[0] = O;
    __syncthreads();
    if (tid < W) a.out[row * D + W * blockIdx.y + tid] = result(O, s_b[0]);
}

// one: a row each (no starts).
Plan plan_of(bool one, int64_t T, int64_t B, int Hq, int Hkv, int nb, int64_t max_len) {
    const int64_t G = Hq / Hkv;
    Plan p;
    // Packed tiles of 8 rows where the sequences of a call have that few per key/value head on
    // average; 64 rows a workgroup where that many fill them and there are four per CU, as long
    // and short ones have to even out; else tiles of 16.  32 heads on 8 of 128, 64 rows against 16: a
    // prompt of 2048 tokens (1032 workgroups of 64 rows) 129 against 155 us, two of 1024 132 against
    // 158; four chunks of 256 on prefixes of up to 3750 (536) 187 against 146, six (800) 232 against 208,
    // eight (1064) 280 against 276.  Prompts without prefixes gain earlier (1536 tokens, 776: 76 against
    // 100 us; 1024, 520: 50 against 58), which the numbers of rows do not tell from the chunks.
    p.pack = nb <= 4 && (one ? G <= 8 : T * G <= 8 * B);
    p.wide = nb <= 4 && !one && T * G >= 64 * B && (T * G / 64 + B) * Hkv >= 1024;
    const int64_t tr = p.wide ? 64 : p.pack ? 8 : 16;
    p.tiles = (int32_t)(one ? B * ((G + tr - 1) / tr) : T * G / tr + B);
    p.segs = (int32_t)((max_len + seg_of(nb) - 1) / seg_of(nb));
    // One sequence: two workgroups per CU, all of which run at once, each with several segments, so
    // that the loads ahead work and the prologue is paid once (131072 positions, 32 heads on 8: 46.7 us,
    // 47.2 with three per CU, 45.2 with four).  Several sequences differ in length: four times as many,
    // which even out (32 of 301..8191: 57 us, 67 with half as many, 71 with as many as for one).  From
    // 512 tiles on no split: 64 sequences of 301..8191 110 us, 121 split in four, 104 in eight; 96 134
    // without, 138 in three, 143 in six; 64 of 1..2000 31 without, 43 with; but 63 of 301..8191, which
    // are split in four, 119, in eight 102.
    // All that goes by max_len, the bound, as the lengths are not known here: 32 sequences of 301..8191
    // take 60 us with 8191 and 173 with 131072, where each head is one workgroup's.
    const int64_t groups = (int64_t)p.tiles * Hkv, want = B == 1 ? 512 : 2048;
    int64_t splits = groups >= 512 ? 1 : (want + groups - 1) / groups;
    if (splits > p.segs) splits = p.segs;
    p.per = (int32_t)((p.segs + splits - 1) / splits);
    p.splits = (p.segs + p.per - 1) / p.per;
    return p;
}

// Raise a kernel's dynamic-LDS limit, once per kernel and device.  Concurrent
// first calls may both set the attribute, which changes nothing; a failure is
// returned and tried again on the next call.
int raise_lds_limit(const void* kernel, std::atomic<int> (&state)[64]) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return (int)hipErrorInvalidDevice;
    std::atomic<int>* st = dev >= 0 && dev < 64 ? &state[dev] : nullptr;
    if (st && st->load(std::memory_order_acquire) == 1) return 0;
    const hipError_t rc =
        hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (rc != hipSuccess) return (int)rc;
    if (st) st->store(1, std::memory_order_release);
    return 0;
}

template <int NB>
int launch_nb(const AttnArgs& a, const Plan& p, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.tiles * p.splits * a.kv.Hkv)), block(64 * WAVES);
    if constexpr (NB <= 4) {
        if (p.wide) {
            static std::atomic<int> lds_state[64];
            const int rc = raise_lds_limit(reinterpret_cast<const void*>(&k_attn_wide<NB>), lds_state);
            if (rc) return rc;
            hipLaunchKernelGGL((k_attn_wide<NB>), grid, block, wide_lds<NB>(), s, a, p);
            return (int)hipGetLastError();
        }
        if (p.pack) {
            hipLaunchKernelGGL((k_attn<NB, true>), grid, block, 0, s, a, p);
            return (int)hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_attn<NB, false>), grid, block, 0, s, a, p);
    return (int)hipGetLastError();
}

}  // namespace

int64_t kv_attention_bytes(int64_t T, int64_t B, int Hq, int Hkv, int nb, int64_t max_len) {
    // a call with T == B may name its rows by starts or not
    const Plan p = plan_of(false, T, B, Hq, Hkv, nb, max_len);
    const bool split = p.splits > 1 || (T == B && plan_of(true, T, B, Hq, Hkv, nb, max_len).splits > 1);
    return split ? T * Hq * p.segs * (32 * nb + 2) * 4 : 16;
}

int kv_attention_rows(int64_t T, int64_t B, bool starts, int Hq, int Hkv, int nb, int64_t max_len) {
    const Plan p = plan_of(!starts, T, B, Hq, Hkv, nb, max_len);
    return p.wide ? 64 : p.pack ? 8 : 16;
}

int launch_kv_attention(const AttnArgs& a, hipStream_t s) {
    const Plan p = plan_of(!a.kv.q_start, a.kv.T, a.kv.B, a.Hq, a.kv.Hkv, a.kv.nb, a.kv.max_len);
    int rc;
    switch (a.kv.nb) {
    case 1: rc = launch_nb<1>(a, p, s); break;
    case 2: rc = launch_nb<2>(a, p, s); break;
    case 3: rc = launch_nb<3>(a, p, s); break;
    case 4: rc = launch_nb<4>(a, p, s); break;
    case 5: rc = launch_nb<5>(a, p, s); break;
    case 6: rc = launch_nb<6>(a, p, s); break;
    case 7: rc = launch_nb<7>(a, p, s); break;
    default: rc = launch_nb<8>(a, p, s); break;
    }
    if (rc || p.splits == 1) return rc;
    const int64_t joins = (int64_t)a.kv.T * a.Hq;
    const bool narrow = p.segs >= 64 && joins < 256;
    const dim3 grid((unsigned)joins, narrow ? (unsigned)a.kv.nb : a.kv.nb == 8 ? 2u : 1u);
    switch (narrow ? 1 : a.kv.nb) {
    case 1: hipLaunchKernelGGL(k_attn_join<32>, grid, dim3(256), 0, s, a, p.segs); break;
    case 2: hipLaunchKernelGGL(k_attn_join<64>, grid, dim3(256), 0, s, a, p.segs); break;
    case 3: hipLaunchKernelGGL(k_attn_join<96>, grid, dim3(256), 0, s, a, p.segs); break;
    case 4: hipLaunchKernelGGL(k_attn_join<128>, grid, dim3(256), 0, s, a, p.segs); break;
    case 5: hipLaunchKernelGGL(k_attn_join<160>, grid, dim3(256), 0, s, a, p.segs); break;
    case 6: hipLaunchKernelGGL(k_attn_join<192>, grid, dim3(256), 0, s, a, p.segs); break;
    case 7: hipLaunchKernelGGL(k_attn_join<224>, grid, dim3(256), 0, s, a, p.segs); break;
    default: hipLaunchKernelGGL(k_attn_join<128>, grid, dim3(256), 0, s, a, p.segs); break;
    }
    return (int)hipGetLastError();
}

}  // namespace qmv
