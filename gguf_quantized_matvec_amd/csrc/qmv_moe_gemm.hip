// Experts' products for many rows of an expert, for gfx950: the multiply of
// qmm_launch (GGUF block weights x Q8_0 activations) on f16 MFMA, with each
// tile's weights those of the expert that its rows name and its activation
// rows gathered.  Every pair's result is bit-identical to qmv_launch.
//
// f16 MFMA on small integers is exact: codes with the integer sub-scales
// folded in are exact f16 values, a block's sum stays below 2^24, and a rank-1
// MFMA of the fp16 scales gives every d_w d_a of a tile exactly in f32.  Then
// p = fma(I, d_w d_a, p) is the term that the documented order adds.
//
// The weights are the instruction's rows and the activations its columns, so a
// lane holds one activation row and 16 weight rows of a 32 x 32 tile: results
// leave four adjacent floats at a time, a gate's and an up's element meet in
// one lane, and a block's minimum term takes one activation scalar a lane.
//
// A workgroup of 4 waves owns 128 weight rows (of a gate/up pair 64 of each, in
// runs of 32) x 128 or 64 rows of an expert, a wave 64 x 64 or 64 x 32 of them;
// Q6_K, whose fetched bytes leave no registers for 64 x 64, has 8 waves of 64 x
// 32.  K is walked two blocks (8 waves: four) a step: the activations' f16
// codes go from memory to LDS directly, a thread decodes one weight block into
// LDS, both into the buffers of the next step, while the current ones are
// multiplied; one barrier a step.  74 KB (8 waves: 145) and 256 registers leave
// two waves a SIMD, of two workgroups, whose barriers do not meet.
//
// 64 x 64 a wave, because the operands come from LDS: 2 KB a tile of 32 x 32
// and block, 16 of the unit's cycles against 24 of its four matrix cores; 64 x
// 32 takes 24, 32 x 32 (16 waves) 32.  Measured at 2048 tokens, 2 of 8 experts
// of 2 x 14336 x 4096 (4096 x 14336): Q4_0 1823 (1091) us, with 64 x 32 2047
// (1159), with 32 x 32 2369; Q4_K 2488 (1499), 2649 (1499), 2687; Q8_0 2030,
// 2241, 2212; Q6_K down 1528 with 64 x 32, 1561 with 64 x 64, 2319 with 32 x 32
// (one run of the forms in turn; by card and inputs Q4_K's 2488 is 2490 to 2650.)
// That is 315 to 530 TFLOP/s.  Matrix cores 36 (Q4_0), 26 (Q4_K), 21 % (Q6_K) busy,
// vector units 56, 62, 41 %, LDS 30, 43, 24 %, a third of the waves' time waiting:
// of a tile's block 96 cycles of MFMA, but 16 fma of 4 cycles (32 with a
// minimum) and 15 to 20 operations of the decoding, which the tile's rows
// share.  Without the decoding 16 waves took 1550 instead of 2369 us.  Half of
// 8 waves decoding after they multiply instead of before gave 4 % for Q4_K and
// lost 4 % for Q6_K; operands read a block ahead lost 6 %; a raised priority
// while multiplying changed nothing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_moe.h"
#include "qmv_moe_device.h"

namespace qmv {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// The 16 values are computed here, not later where they are used.
__device__ __forceinline__ void pin16(float (&v)[16]) {
    asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]),
                      "+v"(v[8]), "+v"(v[9]), "+v"(v[10]), "+v"(v[11]), "+v"(v[12]), "+v"(v[13]), "+v"(v[14]),
                      "+v"(v[15]) : : "memory");
}

// ---------------------------------------------------------------- weights ----
// The bytes that decode one 32-element block of a row.
template <int FMT> struct Raw { uint32_t v[(block_bytes(FMT) + 3) / 4]; };
template <> struct Raw<T_Q4_K> { uint32_t hdr[4], q[8]; };           // d, dmin, scales; the block's 32 nibble bytes
template <> struct Raw<T_Q6_K> { uint32_t ql[8], qh[8], sub, d; };   // sub: the block's two sub-scales

// Block b of the row at `row`.
template <int FMT>
__device__ __forceinline__ void fetch(const uint8_t* row, int b, Raw<FMT>& r) {
    if constexpr (FMT == T_Q4_K) {
        const uint8_t* s = row + (int64_t)144 * (b >> 3);
        __builtin_memcpy(r.hdr, s, 16);
        __builtin_memcpy(r.q, s + 16 + 32 * ((b & 7) >> 1), 32);
    } else if constexpr (FMT == T_Q6_K) {
        const uint8_t* s = row + (int64_t)210 * (b >> 3);
        const int j = b & 7, h = j >> 2;
        __builtin_memcpy(r.ql, s + 64 * h + 32 * (j & 1), 32);
        __builtin_memcpy(r.qh, s + 128 + 32 * h, 32);
        r.sub = *reinterpret_cast<const uint16_t*>(s + 192 + 2 * j);   // not combined here: that would wait for them
        r.d = *reinterpret_cast<const uint16_t*>(s + 208);
    } else {
        __builtin_memcpy(r.v, row + (int64_t)b * block_bytes(FMT), block_bytes(FMT));
    }
}

__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }

// Bytes 0, 1 (2, 3) of c as the f16 pair 1024 + byte: the bits 0x6400 | byte.
__device__ __forceinline__ h2 lower(uint32_t c) { return as_h2(__builtin_amdgcn_perm(0x64646464u, c, 0x04010400u)); }
__device__ __forceinline__ h2 upper(uint32_t c) { return as_h2(__builtin_amdgcn_perm(0x64646464u, c, 0x04030402u)); }

// Four codes in the bytes of c -> two dwords of f16 (code - bias).
__device__ __forceinline__ void codes4(uint32_t c, float bias, uint32_t* o) {
    const _Float16 k = (_Float16)(1024.0f + bias);
    o[0] = as_u32(lower(c) - h2{k, k});
    o[1] = as_u32(upper(c) - h2{k, k});
}

struct Scale {
    uint32_t d;    // fp16 bits
    uint32_t x;    // the minimum's factor (f32 bits: p += x * ca); Q6_K: see below
};

// A Q6_K value s (q - 32) is an exact f16 value if it is even or at most 2048;
// odd ones beyond need an odd scale beyond 64.  Blocks with such a scale leave
// out the value's lowest bit (what is left is even and at most 4096), and bit
// e of Scale::x holds it for element e; the multiply adds those ones in
// products of their own, in steps that have any.
__device__ __forceinline__ bool unfit(const Raw<T_Q6_K>& r) {
    const int s0 = (int8_t)(r.sub & 0xFF), s1 = (int8_t)((r.sub >> 8) & 0xFF);
    return ((s0 & 1) && (s0 > 64 || s0 < -64)) || ((s1 & 1) && (s1 > 64 || s1 < -64));
}
// Bits i and i + 1 of w as the f16 pair of 0 or 1.
__device__ __forceinline__ uint32_t two_bits(uint32_t w, int i) {
    return __umul24((w >> i) & 1u, 0x3C00u) | (__umul24((w >> (i + 1)) & 1u, 0x3C00u) << 16);
}

// Block b as 32 f16 integers in element order, its sub-scale folded in.
template <int FMT>
__device__ __forceinline__ void decode(const Raw<FMT>& r, int b, uint32_t (&o)[16], Scale& s) {
    s.x = 0;
    if constexpr (FMT == T_Q8_0 || FMT == T_Q8_1) {
        s.d = r.v[0] & 0xFFFFu;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t q = FMT == T_Q8_1 ? r.v[i + 1]
                             : __builtin_amdgcn_alignbyte(i == 7 ? r.v[8] & 0xFFFFu : r.v[i + 1], r.v[i], 2);
            codes4(q ^ 0x80808080u, 128.0f, o + 2 * i);   // as 0..255
        }
    } else if constexpr (FMT == T_Q4_K) {
        const int j = b & 7;
        auto byte = [&](int i) -> int {
            const uint32_t d = i < 4 ? r.hdr[1] : i < 8 ? r.hdr[2] : r.hdr[3];
            return (int)((d >> (8 * (i & 3))) & 0xFFu);
        };
        int sc, mn;
        if (j < 4) {
            sc = byte(j) & 63;
            mn = byte(j + 4) & 63;
        } else {
            sc = (byte(j + 4) & 15) | ((byte(j - 4) >> 6) << 4);
            mn = (byte(j + 4) >> 4) | ((byte(j) >> 6) << 4);
        }
        s.d = r.hdr[0] & 0xFFFFu;
        s.x = __float_as_uint(-(half_bits(r.hdr[0] >> 16) * (float)mn));   // exact: 11 x 6 bits
        // (1024 + q) sc - 1024 sc in one rounding of the exact sc q
        const _Float16 f = (_Float16)(float)sc, k = (_Float16)(-1024.0f * (float)sc);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t c = (r.q[i] >> (4 * (j & 1))) & 0x0F0F0F0Fu;
            o[2 * i] = as_u32(__builtin_elementwise_fma(lower(c), h2{f, f}, h2{k, k}));
            o[2 * i + 1] = as_u32(__builtin_elementwise_fma(upper(c), h2{f, f}, h2{k, k}));
        }
    } else if constexpr (FMT == T_Q6_K) {
        const int kk = b & 3;
        const int s0 = (int8_t)(r.sub & 0xFF), s1 = (int8_t)((r.sub >> 8) & 0xFF);
        s.d = r.d;
        const _Float16 f0 = (_Float16)(float)s0, f1 = (_Float16)(float)s1;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t c = ((r.ql[i] >> (4 * (kk >> 1))) & 0x0F0F0F0Fu) |
                               (((r.qh[i] >> (2 * kk)) & 0x03030303u) << 4);
            codes4(c, 32.0f, o + 2 * i);
        }
        if (unfit(r)) {
            // the codes' lowest bits where the sub-scale is odd
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t c = r.ql[i] >> (4 * (kk >> 1));
                if ((i < 4 ? s0 : s1) & 1)
                    s.x |= ((c & 1u) | ((c >> 7) & 2u) | ((c >> 14) & 4u) | ((c >> 21) & 8u)) << (4 * i);
            }
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const _Float16 f = i < 8 ? f0 : f1;
                o[i] = as_u32(__builtin_elementwise_fma(as_h2(o[i]), h2{f, f}, -as_h2(two_bits(s.x, 2 * i))));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const _Float16 f = i < 8 ? f0 : f1;
                o[i] = as_u32(as_h2(o[i]) * h2{f, f});
            }
        }
    } else {
        // 16 bytes of nibbles: the low ones are elements 0..15, the high ones 16..31
        constexpr bool five = FMT == T_Q5_0 || FMT == T_Q5_1;
        constexpr int QS = FMT == T_Q4_0 ? 2 : FMT == T_Q4_1 ? 4 : FMT == T_Q5_0 ? 6 : 8;
        constexpr float bias = FMT == T_Q4_0 ? 8.0f : FMT == T_Q5_0 ? 16.0f : 0.0f;
        s.d = r.v[0] & 0xFFFFu;
        if constexpr (has_min<FMT>()) s.x = __float_as_uint(half_bits(r.v[0] >> 16));
        uint32_t h = 0;
        if constexpr (FMT == T_Q5_0) h = __builtin_amdgcn_alignbyte(r.v[1], r.v[0], 2);
        if constexpr (FMT == T_Q5_1) h = r.v[1];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint32_t q;
            if constexpr (QS % 4 == 0)
                q = r.v[QS / 4 + i];
            else
                q = __builtin_amdgcn_alignbyte(r.v[QS / 4 + i + 1], r.v[QS / 4 + i], 2);
            uint32_t lo = q & 0x0F0F0F0Fu, hi = (q >> 4) & 0x0F0F0F0Fu;
            if constexpr (five) {
                lo |= spread(h >> (4 * i)) << 4;
                hi |= spread(h >> (16 + 4 * i)) << 4;
            }
            codes4(lo, bias, o + 2 * i);
            codes4(hi, bias, o + 8 + 2 * i);
        }
    }
}

// ------------------------------------------------------------------- GEMM ----
constexpr int TN = 128;           // weight rows of a workgroup

struct GemmArgs {
    const uint8_t *w, *w2;
    int64_t N, K;
    int32_t E, per;
    const uint8_t* codes;          // [rows][K] f16
    const uint16_t* da;            // [rows][K / 32] fp16 bits
    const float* ca;               // [rows][K / 32] d_a times the block's code sum
    const int32_t *items, *order, *count;
    float* y;
    bool vec;                      // rows of y begin 16-byte aligned
    int64_t from;                  // the launch's first workgroup, a multiple of 8
};

// Where piece q of tile row r stands, rows of PR 16-byte pieces: pieces change
// places so that 16 consecutive rows' same piece (one pass of a 16-byte read)
// meets all banks.
template <int PR> __device__ __forceinline__ int slot(int r, int q) {
    return r * PR + (q ^ (PR == 16 ? r & 15 : (r >> 1) & 7));
}

template <int FMT, bool PAIR, int AT, int WM>
__global__ __launch_bounds__(128 * WM, 2) void k_moe_gemm(GemmArgs a) {
    constexpr int THREADS = 128 * WM;                 // 2 x WM waves
    constexpr int SB = WM;                            // blocks a step: a weight block a thread
    constexpr int PR = 4 * SB;                        // 16-byte pieces of a tile row in a step
    constexpr int TM = 32 * AT * WM;                  // rows of the expert in a tile
    constexpr int COLS = PAIR ? TN / 2 : TN;          // outputs of a row
    // the weights: piece q of row r at q WP + r, so that the pieces' places differ by
    // constants, and SB blocks of 16 / SB rows (one pass of a 16-byte write) meet all banks
    constexpr int WP = TN + 4 / SB;
    constexpr bool MIN = has_min<FMT>();
    // two objects a kind, not one of two halves: the compiler sees that reads
    // of one do not wait for the copy into the other
    __shared__ uint4 lw0[WP * PR], lw1[WP * PR], la0[TM * PR], la1[TM * PR];
    __shared__ uint32_t ws[2][SB][TN], as[2][SB][TM];
    __shared__ uint32_t wodd[2][SB][FMT == T_Q6_K ? TN : 4];
    __shared__ v4f wmin[2][SB][MIN ? TN / 4 : 1];
    __shared__ float ac[2][SB][MIN ? TM : 4];
    __shared__ int pairs[TM], flag[4];
    const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6);
    const int lr = lane & 31, kq = lane >> 5;
    const int wn = wv & 1, wa = wv >> 1;

    // the tile: compute die x (workgroups go to the dies in turn) takes a run of
    // them, in which an expert's rows advance fastest
    const int NT = (int)((a.N + COLS - 1) / COLS);
    const int64_t total = (int64_t)*a.count * NT;
    const int64_t x = blockIdx.x & 7, k = (a.from + blockIdx.x) >> 3, share = total >> 3, rest = total & 7;
    if (k >= share + (x < rest)) return;
    const int64_t L = x * share + (x < rest ? x : rest) + k;
    const int4 it = reinterpret_cast<const int4*>(a.items)[L / NT];
    const int e = uniform(it.x), start = uniform(it.y), cnt = uniform(it.z), first = uniform(it.w);
    const int64_t rem = L - (int64_t)first * NT;
    const int me = (cnt + TM - 1) / TM;
    const int m = (int)(rem % me);
    const int64_t n0 = rem / me * COLS, N = a.N, K = a.K;
    const int rows = min(TM, cnt - m * TM);
    for (int j = tid; j < TM; j += THREADS) pairs[j] = a.order[start + m * TM + min(j, rows - 1)];
    if (tid < 4) flag[tid] = 0;
    __syncthreads();
    if (e == a.E) {   // pairs without an expert
        if constexpr (PAIR) {
            const int width = (int)(N - n0 < COLS ? N - n0 : COLS);
            for (int i = tid; i < rows * width; i += THREADS) {
                const int j = i / width;
                a.y[pairs[j] * N + n0 + (i - j * width)] = 0.0f;
            }
        }
        return;
    }
    const int nb = (int)(K >> 5);
    const int H = (nb + SB - 1) / SB;                 // steps

    // this thread's weight row and block of each step, and activation row for the scales
    const int sr = tid / SB, sk = tid % SB;
    const uint8_t* wrow;
    {
        int64_t n = n0 + (PAIR ? 32 * (sr >> 6) + (sr & 31) : sr);
        if (n >= N) n = N - 1;
        const uint8_t* w = PAIR && (sr & 32) ? a.w2 : a.w;
        wrow = w + ((int64_t)e * N + n) * (K / block_elements(FMT) * block_bytes(FMT));
    }
    const bool scales = sr < TM;
    const int64_t srow = (int64_t)(pairs[scales ? sr : 0] / a.per) * nb;
    // activation pieces: an instruction fills 64 slots, 64 / PR tile rows; lane
    // l the slot l % PR of row l / PR
    constexpr int NA = TM * PR / THREADS, AR = 64 / PR;
    const uint8_t* asrc[NA];
#pragma unroll
    for (int i = 0; i < NA; i++) {
        const int r = AR * (NA * wv + i) + lane / PR;
        const int piece = slot<PR>(r, lane % PR) - r * PR;    // the exchange is its own inverse
        asrc[i] = a.codes + ((int64_t)(pairs[r] / a.per) * K + 8 * (piece & 3)) * 2;   // of block 0
    }
    auto issue_a = [&](int h, uint4* la) {
#pragma unroll
        for (int i = 0; i < NA; i++) {
            // block past the row's end: its last one again, times a weight scale
            // of 0 (the exchange of pieces takes two bits, of SB = 2 one, of a tile row's
            // number to the block's; of the i-th row they are i's lowest)
            const int b = min(SB * h + (((lane % PR) >> 2) ^ (i & (SB - 1))), nb - 1);
            const uint8_t* src = asrc[i] + (uint32_t)b * 64u;
            __builtin_amdgcn_global_load_lds(src, (lds_void*)(la + AR * (NA * wv + i) * PR), 16, 0, 0);
        }
    };
    struct {
        Raw<FMT> w;
        uint32_t da;
        float ca;
    } raw;
    auto fetch_step = [&](int h) {
        const int b = min(SB * h + sk, nb - 1);
        fetch<FMT>(wrow, b, raw.w);
        raw.da = a.da[srow + b];
        if constexpr (MIN) raw.ca = a.ca[srow + b];
    };
    // decodes the fetched block of step h into the buffers of parity P
    auto stage = [&](int h, auto par) {
        constexpr int PB = decltype(par)::value;
        uint4* lw = PB ? lw1 : lw0;
        uint32_t o[16];
        Scale s;
        const int b = SB * h + sk;
        decode<FMT>(raw.w, b, o, s);
        const bool have = b < nb;
#pragma unroll
        for (int q = 0; q < 4; q++)
            lw[(4 * sk + q) * WP + sr] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        ws[PB][sk][sr] = have ? s.d : 0u;
        if constexpr (MIN) reinterpret_cast<float*>(wmin[PB][sk])[sr] = have ? __uint_as_float(s.x) : 0.0f;
        if constexpr (FMT == T_Q6_K) {
            wodd[PB][sk][sr] = have ? s.x : 0u;
            if (have && s.x) flag[h & 3] = 1;
        }
        if (scales) {
            // 0 past the row's end here too: the block read in its place may have no finite scale
            as[PB][sk][sr] = have ? raw.da : 0u;
            if constexpr (MIN) ac[PB][sk][sr] = have ? raw.ca : 0.0f;
        }
    };

    // tile (i, j): weight rows 32 i and activation rows 32 j onward of the wave's
    float p[2][AT][16], y[2][AT][16];
    each<2>([&](auto i) {
        each<AT>([&](auto j) {
#pragma unroll
            for (int c = 0; c < 16; c++) p[i][j][c] = y[i][j][c] = 0.0f;
        });
    });
    const v16f zero16 = {};
    const uint32_t first_k = kq ? 0u : ~0u;   // of the rank-1 product only k = 0 counts (in both operands: 0 inf is not 0)
    const int wrow0 = 64 * wn + lr, arow = 32 * AT * wa + lr;

    uint32_t apiece = 16 * slot<PR>(arow, kq);        // where the lane's first piece stands

    // the product of the buffers of parity P; odd: a Q6_K step with values that left out a bit
    auto multiply = [&](auto par, bool odd) {
        constexpr int PB = decltype(par)::value;
        const uint4* lw = PB ? lw1 : lw0;
        const uint4* la = PB ? la1 : la0;
        asm volatile("" : "+v"(apiece));              // the pieces' places are computed here, not kept
        each<SB>([&](auto bk) {
            v8h Af[AT][2], Wf[2][2];
            each<AT>([&](auto j) {
                each<2>([&](auto hh) {
                    Af[j][hh] = __builtin_bit_cast(v8h, *(const uint4*)((const char*)la + (apiece ^ (16 * (4 * bk + 2 * hh))) +
                                                                        512 * PR * j));
                });
            });
            each<2>([&](auto i) {
                each<2>([&](auto hh) { Wf[i][hh] = __builtin_bit_cast(v8h, lw[(4 * bk + 2 * hh + kq) * WP + wrow0 + 32 * i]); });
            });
            each<2>([&](auto i) {
                const v4h Ws = __builtin_bit_cast(v4h, make_uint2(ws[PB][bk][wrow0 + 32 * i] & first_k, 0u));
                each<AT>([&](auto j) {
                    const v4h As = __builtin_bit_cast(v4h, make_uint2(as[PB][bk][arow + 32 * j] & first_k, 0u));
                    const float ca = MIN ? ac[PB][bk][MIN ? arow + 32 * j : 0] : 0.0f;
                    v16f I = __builtin_amdgcn_mfma_f32_32x32x16_f16(Wf[i][0], Af[j][0], zero16, 0, 0, 0);
                    const v16f S = __builtin_amdgcn_mfma_f32_32x32x8f16(Ws, As, zero16, 0, 0, 0);
                    I = __builtin_amdgcn_mfma_f32_32x32x16_f16(Wf[i][1], Af[j][1], I, 0, 0, 0);
                    if (FMT == T_Q6_K && odd) {   // what the weights' values left out
                        const uint32_t w = wodd[PB][bk][wrow0 + 32 * i] >> (8 * kq);
                        each<2>([&](auto hh) {
                            uint4 o;
                            o.x = two_bits(w, 16 * hh);
                            o.y = two_bits(w, 16 * hh + 2);
                            o.z = two_bits(w, 16 * hh + 4);
                            o.w = two_bits(w, 16 * hh + 6);
                            I = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, o), Af[j][hh], I, 0, 0, 0);
                        });
                    }
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        v4f fs = {};
                        // the minimums of the lane's g-th run of four weight rows
                        if constexpr (MIN) fs = wmin[PB][bk][MIN ? 16 * wn + 8 * i + 2 * g + kq : 0];
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            float& o = p[i][j][4 * g + c];
                            o = fmaf(I[4 * g + c], S[4 * g + c], o);
                            if constexpr (MIN) o = fmaf(fs[c], ca, o);
                        }
                    }
                    pin16(p[i][j]);
                    // one tile after another where registers are short (2048 tokens, down of
                    // 4096 x 14336: Q4_K 1574 -> 1523 us; Q4_0 1098 -> 1127)
                    if constexpr (FMT == T_Q4_K || FMT == T_Q6_K) __builtin_amdgcn_sched_barrier(0);
                });
            });
        });
    };
    auto step = [&](int h, auto par) {
        using Par = decltype(par);
        using Next = std::integral_constant<int, 1 - Par::value>;
        // the copies into LDS and the fetches of the next weights have arrived
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        bool odd = false;
        if constexpr (FMT == T_Q6_K) {
            odd = uniform(flag[h & 3]) != 0;
            if (tid == 0) flag[(h + 3) & 3] = 0;      // read a step ago, set again in two steps
        }
        if (h + 1 < H) {
            // the longest decoding starts after the copies (Q6_K 1606 -> 1561 us; others lose 1 %)
            if constexpr (FMT == T_Q6_K) issue_a(h + 1, Next::value ? la1 : la0);
            stage(h + 1, Next{});
            if constexpr (FMT != T_Q6_K) issue_a(h + 1, Next::value ? la1 : la0);
            if (h + 2 < H) fetch_step(h + 2);
        }
        multiply(par, odd);
        // the end of a chunk of 8 blocks (of SB = 4 every other step: par says which)
        if ((SB == 4 ? Par::value == 1 : (h & 3) == 3) || h + 1 == H) {
            each<2>([&](auto i) {
                each<AT>([&](auto j) {
#pragma unroll
                    for (int c = 0; c < 16; c++) {
                        y[i][j][c] = y[i][j][c] + p[i][j][c];
                        p[i][j][c] = 0.0f;
                    }
                });
            });
        }
    };

    fetch_step(0);
    stage(0, std::integral_constant<int, 0>{});
    issue_a(0, la0);
    if (H > 1) fetch_step(1);
    for (int h = 0; h < H; h += 2) {
        step(h, std::integral_constant<int, 0>{});
        if (h + 1 < H) step(h + 1, std::integral_constant<int, 1>{});
    }

    // lane: row arow + 32 j; element c of tile i: weight row 8 (c / 4) + 4 kq + c % 4
    each<AT>([&](auto j) {
        if (arow + 32 * j >= rows) return;
        float* out = a.y + pairs[arow + 32 * j] * N;
        each<PAIR ? 1 : 2>([&](auto i) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int64_t n = n0 + (PAIR ? 32 * wn : 64 * wn + 32 * i) + 8 * g + 4 * kq;
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; c++)
                    v[c] = PAIR ? swiglu(y[0][j][4 * g + c], y[1][j][4 * g + c]) : y[i][j][4 * g + c];
                if (a.vec && n + 4 <= N) {
                    *reinterpret_cast<float4*>(out + n) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        if (n + c < N) out[n + c] = v[c];
                }
            }
        });
    });
}

template <int FMT, bool PAIR, int AT, int WM>
int launch_at(const MoeArgs& m, GemmArgs& a, hipStream_t s) {
    constexpr int COLS = PAIR ? TN / 2 : TN;
    const int64_t tiles = moe_most_items(m.P, m.E, 32 * AT * WM) * ((m.N + COLS - 1) / COLS);
    // a grid's dimension ends below 2^32 threads
    constexpr int64_t MOST = ((int64_t)1 << 31) / (128 * WM);
    for (a.from = 0; a.from < tiles; a.from += MOST) {
        const int64_t n = tiles - a.from < MOST ? tiles - a.from : MOST;
        hipLaunchKernelGGL((k_moe_gemm<FMT, PAIR, AT, WM>), dim3((unsigned)((n + 7) / 8 * 8)),
                           dim3(128 * WM), 0, s, a);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    return 0;
}

template <int FMT> int launch_fmt(const MoeArgs& m, GemmArgs& a, hipStream_t s) {
    if constexpr (FMT == T_Q6_K) {
        return m.w2 ? launch_at<FMT, true, 1, 4>(m, a, s) : launch_at<FMT, false, 1, 4>(m, a, s);
    } else {
        if (moe_rows(m) == 64)
            return m.w2 ? launch_at<FMT, true, 1, 2>(m, a, s) : launch_at<FMT, false, 1, 2>(m, a, s);
        return m.w2 ? launch_at<FMT, true, 2, 2>(m, a, s) : launch_at<FMT, false, 2, 2>(m, a, s);
    }
}

}  // namespace

int launch_moe_gemm(const MoeArgs& m, hipStream_t s) {
    const MoeWork L = moe_work(m);
    GemmArgs a{};
    a.w = m.w;
    a.w2 = m.w2;
    a.N = m.N;
    a.K = m.K;
    a.E = (int32_t)m.E;
    a.per = m.per;
    a.codes = m.work + L.blocks;
    a.da = reinterpret_cast<const uint16_t*>(m.work + L.da);
    a.ca = reinterpret_cast<const float*>(m.work + L.ca);
    a.items = reinterpret_cast<const int32_t*>(m.work + L.items);
    a.order = reinterpret_cast<const int32_t*>(m.work + L.order);
    a.count = reinterpret_cast<const int32_t*>(m.work + L.count);
    a.y = m.y;
    a.vec = m.N % 4 == 0 && aligned16(m.y);
    switch (m.type) {
    case T_Q8_0: return launch_fmt<T_Q8_0>(m, a, s);
    case T_Q4_0: return launch_fmt<T_Q4_0>(m, a, s);
    case T_Q5_0: return launch_fmt<T_Q5_0>(m, a, s);
    case T_Q4_1: return launch_fmt<T_Q4_1>(m, a, s);
    case T_Q5_1: return launch_fmt<T_Q5_1>(m, a, s);
    case T_Q8_1: return launch_fmt<T_Q8_1>(m, a, s);
    case T_Q4_K: return launch_fmt<T_Q4_K>(m, a, s);
    case T_Q6_K: return launch_fmt<T_Q6_K>(m, a, s);
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace qmv
