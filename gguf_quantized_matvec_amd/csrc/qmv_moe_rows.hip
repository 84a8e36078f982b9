// Experts' products for up to 16 rows of an expert at a time, for gfx950: the
// multiply of qmv_launch (GGUF block weights x Q8_0 activations, integer block
// dots, one f32 term a 32-element block, chunks of 8 blocks added in ascending
// order; include/qmv.h), with the weights of the expert that each pair names.
// Every pair's result is bit-identical to qmv_launch on that expert's matrix.
//
// An item is up to R (4 or 16) pairs of one expert.  A workgroup of 8 waves
// takes an item and 8 / KS tiles of 16 weight rows; KS waves share a tile and
// take its 256-element chunks in turn.  A wave fetches the 16 rows' bytes of a
// chunk as 16-byte pieces into registers, two chunks ahead (the gate's and the
// up's of a pair), lays them into its slice of LDS, and lane (nn = l % 16,
// kg = l / 16) decodes its quarter of each of weight row nn's blocks into an
// operand of v_mfma_i32_16x16x32_i8.  Result element i of the lane is
// activation row 4 kg + i of the instruction; the item's row j stands at
// 4 (j % 4) + j / 4, so that up to 4 NI rows need the elements i < NI only (NI
// = 1, 2, 4, by the item's rows): few rows cost few f32 terms.  The item's
// activations lie in LDS, a segment of chunks at a time, shared by the 8 waves.
//
// Few rows are bound by the weights' bytes, more by the f32 term a block and row
// and the decoding, which only an item's rows share.  Measured (the product's
// launch alone): 32 tokens, 8 of 64 experts of 2 x 1024 x 2048 in Q4_0 34.4 us
// (4.4 TB/s); 16 tokens, 2 of 8 of 4096 x 14336 in Q4_K 70.9 to 73 (3.7 TB/s); 300
// tokens, 4 of 16 of 896 x 4864 in Q5_0 63.5 to 71 (by run; 147 to 165 TFLOP/s).
//
// Order inside a block does not matter (the integers are exact), so lane kg
// takes bytes 4kg .. 4kg+3 of a 16-byte nibble block, low and high nibbles,
// and the activations are laid out to match: no lane reads nibbles that it
// does not use.
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qmv_moe.h"
#include "qmv_moe_device.h"

namespace qmv {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// 16-byte pieces that cover a chunk at the worst alignment of its start.
template <int FMT> constexpr int pieces() {
    return (16 - std::gcd(Fmt<FMT>::BB, 16) + Fmt<FMT>::CB + 15) / 16;
}
// Blocks of 16 bytes of nibbles: element e < 16 the low one of byte e, e + 16 the high one.
template <int FMT> constexpr bool nibble_block() {
    return FMT == T_Q4_0 || FMT == T_Q4_1 || FMT == T_Q5_0 || FMT == T_Q5_1;
}
// Codes with an offset are formed as 16 (c - 8) and 8 (c - 16), whose int8
// bits are a shift and a flipped top bit away; the factor leaves with the
// activation scale, both exactly (powers of two).
template <int FMT> constexpr float scale_back() {
    return FMT == T_Q4_0 ? 1.0f / 16 : FMT == T_Q5_0 ? 1.0f / 8 : 1.0f;
}
// AL: every chunk starts 16-byte aligned and is whole (K a multiple of 256 and
// the chunk a multiple of 16 bytes).  LDS rows are an odd number of pieces
// long, so that 16 rows' same piece meets all banks.
template <int FMT> constexpr bool can_align() { return Fmt<FMT>::CB % 16 == 0; }
template <int FMT, bool AL> constexpr int row_pieces() { return AL ? Fmt<FMT>::CB / 16 : pieces<FMT>(); }
template <int FMT, bool AL> constexpr int row_stride() { return 16 * (row_pieces<FMT, AL>() | 1); }
template <int FMT, bool AL> constexpr int slice() { return 16 * row_stride<FMT, AL>(); }

constexpr int WAVES = 8;
constexpr int SEG = 16;
constexpr int ACT_STRIDE = 272;   // a row's 256 codes of a chunk, and 16 bytes so that rows differ in their banks

// ----------------------------------------------------------- preparation ----
// One launch before the product: workgroups 0 .. E sort the pairs (only beyond
// MOE_SCAN pairs), the others quantise x to Q8_0 blocks.
//
// Workgroup e counts all pairs by expert, writes those of expert e in
// ascending order to their place, and e's items: no workgroup waits for
// another.  Its waves each take a run of the pairs, count and then write.
struct PrepArgs {
    const float* x;      // or NULL: the blocks at xq
    const uint8_t* xq;
    uint8_t* blocks;     // Q8_0 blocks, or (gemm) f16 codes
    uint16_t* da;        // gemm: fp16 scales
    float* ca;           // gemm: scale times code sum
    int64_t nblocks;     // blocks to quantise (0: none)
    bool gemm;
    int32_t row;         // not 0: rows of `row` bytes as k_moe_gemv reads them, of
    int32_t nb;          // nb blocks, their scales times
    float back;          // this
    bool min;            // and scales times code sums
    const int32_t* idx;
    int32_t P, E, R;
    int32_t planners;    // E + 1, or 0
    int32_t* items;
    int32_t* order;
    int32_t* count;
    bool a16;            // x is 16-byte aligned
};
constexpr int PREP = 512;
constexpr int AHEAD = 8;     // numbers a lane has on the way (262144 pairs, 256 experts: 320 us with one, 109 with these)

__device__ __forceinline__ int key_of(int e, int E) { return (unsigned)e < (unsigned)E ? e : E; }

__global__ __launch_bounds__(PREP) void k_moe_prep(PrepArgs a) {
    __shared__ int hist[1025], seen[PREP / 64], sums[2][PREP / 64];
    const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6);
    if ((int)blockIdx.x < a.planners) {
        const int E = a.E, P = a.P, e = blockIdx.x;
        for (int i = tid; i <= E; i += PREP) hist[i] = 0;
        __syncthreads();
        const int run = ((P + PREP - 1) / PREP) * 64, lo = wv * run, hi = min(P, lo + run);
        // keys of pairs p + 64 u + lane, -1 behind the run; all loads before the first use
        auto keys = [&](int p, int (&k)[AHEAD]) {
#pragma unroll
            for (int u = 0; u < AHEAD; u++) k[u] = a.idx[min(p + 64 * u + lane, P - 1)];
#pragma unroll
            for (int u = 0; u < AHEAD; u++) k[u] = p + 64 * u + lane < hi ? key_of(k[u], E) : -1;
        };
        int mine = 0;
        for (int p = lo; p < hi; p += 64 * AHEAD) {
            int k[AHEAD];
            keys(p, k);
#pragma unroll
            for (int u = 0; u < AHEAD; u++) {
                if (k[u] >= 0) atomicAdd(&hist[k[u]], 1);
                mine += __popcll(__builtin_amdgcn_ballot_w64(k[u] == e));
            }
        }
        if (lane == 0) seen[wv] = mine;
        __syncthreads();
        // pairs and items of the experts below e (and, for the last, of all)
        int before = 0, base = 0;
        for (int i = tid; i < e; i += PREP) {
            before += hist[i];
            base += (hist[i] + a.R - 1) / a.R;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            before += __shfl_xor(before, o);
            base += __shfl_xor(base, o);
        }
        if (lane == 0) {
            sums[0][wv] = before;
            sums[1][wv] = base;
        }
        __syncthreads();
        int start = 0, item = 0, at = 0;
        for (int i = 0; i < PREP / 64; i++) {
            start += sums[0][i];
            item += sums[1][i];
            if (i < wv) at += seen[i];
        }
        const int n = hist[e], items = (n + a.R - 1) / a.R;
        at += start;
        for (int p = lo; p < hi; p += 64 * AHEAD) {
            int k[AHEAD];
            keys(p, k);
#pragma unroll
            for (int u = 0; u < AHEAD; u++) {
                const uint64_t m = __builtin_amdgcn_ballot_w64(k[u] == e);
                if (k[u] == e) a.order[at + __popcll(m & ((1ull << lane) - 1))] = p + 64 * u + lane;
                at += __popcll(m);
            }
        }
        for (int i = tid; i < items; i += PREP)
            reinterpret_cast<int4*>(a.items)[item + i] =
                make_int4(e, start, n, item);
        if (e == E && tid == 0) *a.count = item + items;
        return;
    }
    // eight lanes a block, four elements each
    const int64_t b = (int64_t)((int)blockIdx.x - a.planners) * (PREP / 8) + (tid >> 3);
    const int sub = tid & 7;
    const bool live = b < a.nblocks;
    uint32_t c = 0;
    _Float16 d16 = 0;
    if (a.x)
        d16 = quantise_block(a.x + b * 32 + 4 * sub, live, a.a16, c);
    else if (live)
        d16 = read_block(a.xq + b * 34, sub, c);
    uint16_t dbits;
    __builtin_memcpy(&dbits, &d16, 2);
    if (a.gemm || a.row) {
        const int S = block_sum(c);
        if (!live) return;
        if (a.row) {
            const int64_t r = b / a.nb;
            const int k = (int)(b - r * a.nb), C = (a.nb + 7) >> 3;
            uint8_t* to = a.blocks + r * a.row;
            *reinterpret_cast<uint32_t*>(to + (k >> 3) * 272 + (k & 7) * 32 + 4 * sub) = c;
            if (sub == 0) {
                float* da = reinterpret_cast<float*>(to + C * 272);
                da[k] = (float)d16 * a.back;
                if (a.min) da[8 * C + k] = (float)d16 * (float)S;
            }
            return;
        }
        _Float16 h[4];
#pragma unroll
        for (int i = 0; i < 4; i++) h[i] = (_Float16)(float)(int8_t)(c >> (8 * i));
        uint2 two;
        __builtin_memcpy(&two, h, 8);
        *reinterpret_cast<uint2*>(a.blocks + b * 64 + 8 * sub) = two;
        if (sub == 0) {
            a.da[b] = dbits;
            a.ca[b] = (float)d16 * (float)S;
        }
        return;
    }
    if (!live) return;
    uint16_t* out = reinterpret_cast<uint16_t*>(a.blocks + b * 34);
    out[1 + 2 * sub] = (uint16_t)c;
    out[2 + 2 * sub] = (uint16_t)(c >> 16);
    if (sub == 0) out[0] = dbits;
}

// --------------------------------------------------------------- product ----
struct RowsArgs {
    const uint8_t *w, *w2;
    int64_t N, K, wbytes;    // wbytes: of all experts
    int32_t E, P, per;
    const int32_t* idx;
    const uint8_t* blocks;   // Q8_0 blocks of the activation rows
    const int32_t *items, *order, *count;
    float* y;
    int32_t ks;              // waves that share a tile: 1, 2, 4, 8
    int32_t seg;             // chunks of activations in LDS at a time: SEG, or all if they are fewer
    int32_t item0;           // the launch's first item
    bool scan;               // the workgroups find their items among idx; else items, order, count
};

// A chunk's fields in LDS as aligned dwords: reads that do not lie on their own
// size's border take twice the time there.  Blocks of 18, 22, 34 and 210 bytes
// leave fields, and without AL the chunk itself, on any even byte: a field at
// byte O is read from the dwords around it and shifted down.
template <bool AL> struct Fields {
    const uint32_t *even, *odd;   // the dwords that hold bytes 0 and 2
    uint32_t se, so;              // where in them: 0 or 2
    const uint8_t* at;            // byte 0
    __device__ __forceinline__ explicit Fields(const uint8_t* rb) : at(rb) {
        if constexpr (AL) {
            even = odd = reinterpret_cast<const uint32_t*>(rb);
            se = 0;
            so = 2;
        } else {
            const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(rb) & 2u;
            even = reinterpret_cast<const uint32_t*>(rb - low);
            odd = reinterpret_cast<const uint32_t*>(rb + low);
            se = low;
            so = 2 - low;
        }
    }
    // N dwords at byte O + 4 l
    template <int O, int N> __device__ __forceinline__ void get(int l, uint32_t (&o)[N]) const {
        const uint32_t* p = (O % 4 ? odd + (O - 2) / 4 : even + O / 4) + l;
        if constexpr (AL && O % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N; i++) o[i] = p[i];
        } else {
            uint32_t v[N + 1];
#pragma unroll
            for (int i = 0; i <= N; i++) v[i] = p[i];
#pragma unroll
            for (int i = 0; i < N; i++) o[i] = __builtin_amdgcn_alignbyte(v[i + 1], v[i], O % 4 ? so : se);
        }
    }
    template <int O> __device__ __forceinline__ uint32_t half() const {
        return *reinterpret_cast<const uint16_t*>(at + O);
    }
};

// One chunk of the 16 weight rows at rb (this lane's row) against the item's
// rows: p[i] = the chunk's sum of row kg + 4 i, in the documented order.
// ac: this lane's row of the activation codes (of the matrix operand); da, ca:
// scales (times scale_back) and scale * code sum of block b's rows kg + 4 i at
// [b * R + i].  nbc: blocks of the chunk.
template <int FMT, int NI, int R, bool AL>
__device__ __forceinline__ void chunk_rows(const Fields<AL>& rb, const uint8_t* ac, const float* da,
                                           const float* ca, int nbc, int kg, float (&p)[NI]) {
    using F = Fmt<FMT>;
    const v4i zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NI; i++) p[i] = 0.0f;
    // the superblock's fields
    uint32_t q[4][2], qh[2][2];
    uint32_t sc[4] = {0, 0, 0, 0}, mn[2] = {0, 0};
    float dw = 0.0f, dmin = 0.0f;
    if constexpr (FMT == T_Q4_K) {
        uint32_t hdr[4];
        rb.template get<0, 4>(0, hdr);
        dw = half_bits(hdr[0] & 0xFFFFu);
        dmin = half_bits(hdr[0] >> 16);
        // 6-bit scales and minimums of sub-blocks 0..3, 4..7, one a byte
        sc[0] = hdr[1] & 0x3F3F3F3Fu;
        mn[0] = hdr[2] & 0x3F3F3F3Fu;
        sc[1] = (hdr[3] & 0x0F0F0F0Fu) | ((hdr[1] >> 2) & 0x30303030u);
        mn[1] = ((hdr[3] >> 4) & 0x0F0F0F0Fu) | ((hdr[2] >> 2) & 0x30303030u);
        each<4>([&](auto j) { rb.template get<16 + 32 * j, 2>(2 * kg, q[j]); });
    } else if constexpr (FMT == T_Q6_K) {
        each<4>([&](auto j) { rb.template get<32 * j, 2>(2 * kg, q[j]); });
        each<2>([&](auto j) { rb.template get<128 + 32 * j, 2>(2 * kg, qh[j]); });
        rb.template get<192, 4>(0, sc);
        dw = half_bits(rb.template half<208>());
    }
    auto wide = [](const uint32_t (&v)[2]) { return ((uint64_t)v[1] << 32) | v[0]; };
    each<8>([&](auto bc) {
        constexpr int b = bc;
        // a short chunk's missing blocks get scales of 0 (their activation
        // scales are staged as 0): no branch between the blocks, whose reads
        // and products overlap
        const long a = *reinterpret_cast<const long*>(ac + 32 * b);
        v4i I;
        float mw = 0.0f;   // the minimum's factor: p += mw * ca
        if constexpr (F::QK == 32) {
            constexpr int O = F::BB * b;
            const uint32_t dbits = rb.template half<O>();
            dw = half_bits(b < nbc ? dbits : 0u);
            uint32_t w[2];
            if constexpr (FMT == T_Q8_0 || FMT == T_Q8_1) {
                rb.template get<O + (FMT == T_Q8_0 ? 2 : 4), 2>(2 * kg, w);
            } else {
                constexpr int QS = FMT == T_Q4_0 ? 2 : FMT == T_Q4_1 ? 4 : FMT == T_Q5_0 ? 6 : 8;
                uint32_t one[1];
                rb.template get<O + QS, 1>(kg, one);
                const uint32_t v = one[0];
                if constexpr (FMT == T_Q4_0) {
                    w[0] = ((v << 4) & 0xF0F0F0F0u) ^ 0x80808080u;
                    w[1] = (v & 0xF0F0F0F0u) ^ 0x80808080u;
                } else if constexpr (FMT == T_Q4_1) {
                    w[0] = v & 0x0F0F0F0Fu;
                    w[1] = (v >> 4) & 0x0F0F0F0Fu;
                } else {
                    // fifth bits of elements 4kg .. 4kg+3 and 16 + 4kg ..
                    rb.template get<O + (FMT == T_Q5_0 ? 2 : 4), 1>(0, one);
                    const uint32_t h = one[0] >> (4 * kg);
                    const uint32_t l5 = spread(h), h5 = spread(h >> 16);
                    if constexpr (FMT == T_Q5_0) {
                        w[0] = (((v << 3) & 0x78787878u) | (l5 << 7)) ^ 0x80808080u;
                        w[1] = (((v >> 1) & 0x78787878u) | (h5 << 7)) ^ 0x80808080u;
                    } else {
                        w[0] = (v & 0x0F0F0F0Fu) | (l5 << 4);
                        w[1] = ((v >> 4) & 0x0F0F0F0Fu) | (h5 << 4);
                    }
                }
            }
            if constexpr (has_min<FMT>()) {
                const uint32_t mbits = rb.template half<O + 2>();
                mw = half_bits(b < nbc ? mbits : 0u);
            }
            I = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, (long)wide(w), zero, 0, 0, 0);
        } else if constexpr (FMT == T_Q4_K) {
            mw = -(dmin * (float)((mn[b >> 2] >> (8 * (b & 3))) & 0xFFu));
            const uint64_t raw = wide(q[b >> 1]) >> (4 * (b & 1));
            I = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, (long)(raw & 0x0F0F0F0F0F0F0F0Full), zero,
                                                     0, 0, 0);
#pragma unroll
            for (int i = 0; i < NI; i++) I[i] = __mul24((int)((sc[b >> 2] >> (8 * (b & 3))) & 0xFFu), I[i]);
        } else {
            constexpr int h = b >> 2, kq = b & 3;
            const uint64_t ql = wide(q[2 * h + (kq & 1)]) >> (kq & 2 ? 4 : 0);
            const uint64_t q6 = (ql & 0x0F0F0F0F0F0F0F0Full) |
                                (((wide(qh[h]) >> (2 * kq)) & 0x0303030303030303ull) << 4);
            // q6 - 32 bytewise: no borrow leaves a byte whose top bit is set before
            const uint64_t top = 0x8080808080808080ull;
            const uint64_t w = ((q6 | top) - 0x2020202020202020ull) ^ top;
            const uint32_t sw = sc[b >> 1] >> (16 * (b & 1));
            const int s0 = (int8_t)(sw & 0xFF), s1 = (int8_t)((sw >> 8) & 0xFF);
            // each half of the block has a scale of its own: two products, the other half's codes zero
            const long lo = kg < 2 ? (long)w : 0, hi = kg < 2 ? 0 : (long)w;
            const v4i I0 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, lo, zero, 0, 0, 0);
            const v4i I1 = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, hi, zero, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < NI; i++) I[i] = __mul24(s0, I0[i]) + __mul24(s1, I1[i]);
        }
        typedef float vec __attribute__((ext_vector_type(NI)));
        const vec dv = *reinterpret_cast<const vec*>(da + b * R);
        vec cv = dv;
        if constexpr (has_min<FMT>()) cv = *reinterpret_cast<const vec*>(ca + b * R);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            p[i] = fmaf((float)I[i], dw * dv[i], p[i]);
            if constexpr (has_min<FMT>()) p[i] = fmaf(mw, cv[i], p[i]);
        }
        // a few blocks at a time: the reads and products of more would run ahead
        // and not fit the registers
        if constexpr ((b + 1) % ((NI == 4 ? 2 : 4) / (AL ? 1 : 2)) == 0) {
            if constexpr (NI == 1) asm volatile("" : "+v"(p[0]) : : "memory");
            if constexpr (NI == 2) asm volatile("" : "+v"(p[0]), "+v"(p[1]) : : "memory");
            if constexpr (NI == 4) asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]) : : "memory");
        }
    });
}

template <int FMT, bool PAIR, int R, bool AL>
__global__ __launch_bounds__(64 * WAVES, 4) void k_moe_rows(RowsArgs a) {
    using F = Fmt<FMT>;
    constexpr int MATS = PAIR ? 2 : 1, NIM = R / 4;
    constexpr int PPS = row_pieces<FMT, AL>(), NP = (16 * PPS + 63) / 64;
    constexpr int STRIDE = row_stride<FMT, AL>(), SLICE = slice<FMT, AL>();
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* pairs = reinterpret_cast<int*>(smem);    // [16] the item's pairs
    const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6);
    const int nn = lane & 15, kg = lane >> 4;

    // the item: its expert and rows
    int e = -1, rows = 0;
    if (a.scan) {
        const int key = lane < a.P ? key_of(a.idx[lane], a.E) : -1;
        uint64_t left = __builtin_amdgcn_ballot_w64(lane < a.P);
        int item = a.item0 + (int)blockIdx.y;
        while (left) {
            const int k = __builtin_amdgcn_readlane(key, (int)__builtin_ctzll(left));
            const uint64_t m = __builtin_amdgcn_ballot_w64(key == k);
            const int n = __popcll(m), items = (n + R - 1) / R;
            if (item < items) {
                e = k;
                rows = min(R, n - item * R);
                const int rank = __popcll(m & ((1ull << lane) - 1)) - item * R;
                if (wv == 0 && key == k && rank >= 0 && rank < R) pairs[rank] = lane;
                break;
            }
            item -= items;
            left &= ~m;
        }
    } else {
        const int at = a.item0 + (int)blockIdx.y;
        const int4 it = reinterpret_cast<const int4*>(a.items)[at];   // read along with the count
        if (at >= *a.count) return;
        const int done = uniform((at - it.w) * R);    // the expert's rows in items before this one
        e = uniform(it.x);
        rows = min(R, uniform(it.z) - done);
        if (tid < rows) pairs[tid] = a.order[it.y + done + tid];
    }
    if (e < 0) return;
    const int64_t N = a.N, K = a.K;
    const int KS = a.ks, TW = WAVES / KS, ks = wv % KS, tw = wv / KS;
    const int nb = (int)(K >> 5), C = (nb + 7) >> 3;
    const int tiles = (int)((N + 15) >> 4);
    if (e == a.E) {   // pairs without an expert
        if constexpr (PAIR) {
            __syncthreads();
            const int64_t n0 = (int64_t)blockIdx.x * TW * 16;
            const int width = (int)(N - n0 < TW * 16 ? N - n0 : TW * 16);
            for (int i = tid; i < rows * width; i += 64 * WAVES) {
                const int j = i / width;
                a.y[pairs[j] * N + n0 + (i - j * width)] = 0.0f;
            }
        }
        return;
    }

    // this wave's tile; a wave past the last one works on it too and stores nothing
    const int tile_ = blockIdx.x * TW + tw;
    const bool mine = tile_ < tiles;
    const int64_t n0 = (int64_t)(mine ? tile_ : tiles - 1) * 16;
    const int64_t Rb = (K / F::QK) * F::BB;
    const int64_t tb = ((int64_t)e * N + n0) * Rb;
    const uint32_t a0 = (uint32_t)(tb & 15);
    const uint8_t* wt = a.w + (tb - a0);
    const uint8_t* wt2 = PAIR ? a.w2 + (tb - a0) : wt;
    const int64_t room = a.wbytes - (tb - a0) - 16;
    const uint32_t lim = (uint32_t)(room < 0x7fffffff ? room : 0x7fffffff);
    const bool tail = room < 16 * Rb + 16;          // pieces may reach past the last expert's end
    const int last_row = (int)(N - 1 - n0 < 15 ? N - 1 - n0 : 15);
    uint8_t* wl = smem + 64 + wv * SLICE;
    uint8_t* acts = smem + 64 + WAVES * SLICE;
    const int seg = a.seg;
    float* dbuf = reinterpret_cast<float*>(acts + seg * R * ACT_STRIDE);    // [seg][8][4][R / 4]: row kg + 4 i at [kg][i]
    float* cbuf = dbuf + seg * R * 8;                                       // the same, with a minimum
    float* pbuf = cbuf + (has_min<FMT>() ? seg * R * 8 : 0);                // [seg][TW][MATS][R][16], KS > 1

    // 16-byte pieces: lane l's k-th is piece 64 k + l of the tile's rows
    uint32_t rowoff[NP];
    uint32_t where[NP];    // its place in the slice | its number in the row << 16
#pragma unroll
    for (int k = 0; k < NP; k++) {
        const int p = min(64 * k + lane, 16 * PPS - 1);
        const int n = p / PPS;
        const int j = p - n * PPS;
        where[k] = (uint32_t)(n * STRIDE + 16 * j) | (uint32_t)j << 16;
        rowoff[k] = a0 + (uint32_t)min(n, last_row) * (uint32_t)Rb + (AL ? 16 * j : 0);
    }
    // not AL: a piece past the chunk's end is its last one again, one past the
    // blob's end is moved back (and staged bytewise)
    auto piece = [&](int k, int c) -> uint32_t {
        const uint32_t len = F::QK == 32 ? min(8, nb - 8 * c) * F::BB : F::CB;
        const uint32_t s = rowoff[k] + (uint32_t)c * F::CB;
        return min((s & ~15u) + 16 * (where[k] >> 16), (s + len - 1) & ~15u);
    };
    auto fetch = [&](const uint8_t* base, int c, v4u (&r)[NP]) {
        if constexpr (AL) {
            const uint8_t* at = base + (int64_t)c * F::CB;
#pragma unroll
            for (int k = 0; k < NP; k++) r[k] = *reinterpret_cast<const v4u*>(at + rowoff[k]);
        } else {
#pragma unroll
            for (int k = 0; k < NP; k++) __builtin_memcpy(&r[k], base + min(piece(k, c), lim), 16);
        }
    };
    auto stage = [&](int c, const v4u (&r)[NP]) {
#pragma unroll
        for (int k = 0; k < NP; k++)
            if (64 * k + lane < 16 * PPS)
                *reinterpret_cast<v4u*>(wl + (where[k] & 0xFFFFu)) = r[k];
        if (!AL && tail) {
            // pieces that were moved back: their bytes to where they belong
#pragma unroll
            for (int k = 0; k < NP; k++) {
                const uint32_t off = piece(k, c);
                const uint32_t s = rowoff[k] + (uint32_t)c * F::CB;
                if (off > lim) {
                    uint8_t* at = wl + (where[k] & 0xFFFFu) - 16 * (where[k] >> 16) + (lim - (s & ~15u));
                    uint16_t h[8];
                    __builtin_memcpy(h, &r[k], 16);
#pragma unroll
                    for (int i = 0; i < 8; i++) __builtin_memcpy(at + 2 * i, &h[i], 2);
                }
            }
        }
        wave_sync();
    };

    // the wave's steps: its chunks ks, ks + KS, ...; of a pair first the gate's, then the up's
    // and of a single matrix two of them by turns.  Every fetch is made, beyond
    // the end the last chunk's again: a fetch behind a branch would make each
    // wait for one set of registers wait for the other's too
    auto valid = [&](int c) { return min(c, C - 1); };
    // Long chunks that need address arithmetic leave registers for one set only.
    constexpr int TURN = PAIR ? 1 : 2;
    constexpr bool ONE = !AL && R == 16 && NP >= 4;
    v4u r0[NP], r1[NP];
    fetch(wt, ks, r0);
    if constexpr (!ONE) fetch(wt2, PAIR ? ks : valid(ks + KS), r1);

    float acc[MATS][NIM];
#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int i = 0; i < NIM; i++) acc[m][i] = 0.0f;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // KS > 1: this thread's outputs tid + 512 q
    const int outs = TW * MATS * R * 16;

    // this lane's activation row of the matrix operand, and where its scales begin
    const int arow = (nn >> 2) + ((nn & 3) < NIM ? 4 * (nn & 3) : 0);

    // the staged chunk c against the item's rows
    auto multiply = [&](int m, int c, int c0) {
        const int cs = c - c0;
        const uint32_t s = a0 + (uint32_t)min(nn, last_row) * (uint32_t)Rb + (uint32_t)c * F::CB;
        const uint8_t* rb = wl + nn * STRIDE + (AL ? 0 : s & 15);
        const uint8_t* ac = acts + (cs * R + arow) * ACT_STRIDE + 8 * kg;
        const float* da = dbuf + cs * R * 8 + kg * NIM;
        const float* ca = cbuf + cs * R * 8 + kg * NIM;
        float* o = pbuf + cs * outs + ((tw * MATS + m) * R + kg) * 16 + nn;
        const int nbc = F::QK == 32 && !AL ? min(8, nb - 8 * c) : 8;
        auto run = [&](auto ni) {
            constexpr int NI = decltype(ni)::value;
            float p[NI];
            chunk_rows<FMT, NI, R, AL>(Fields<AL>(rb), ac, da, ca, nbc, kg, p);
#pragma unroll
            for (int i = 0; i < NI; i++) {
                if (KS == 1)
                    acc[m][i] = acc[m][i] + p[i];
                else
                    o[64 * i] = p[i];
            }
        };
        if constexpr (NIM == 4) {
            if (rows > 8)
                run(std::integral_constant<int, 4>{});
            else if (rows > 4)
                run(std::integral_constant<int, 2>{});
            else
                run(std::integral_constant<int, 1>{});
        } else {
            run(std::integral_constant<int, 1>{});
        }
        wave_sync();
    };

    int c = ks;
    for (int c0 = 0; c0 < C; c0 += seg) {
        const int c1 = min(C, c0 + seg);
        __syncthreads();
        // the segment's activations: a thread a block
        {
            const int nbs = min(nb, 8 * c1) - 8 * c0, all = 8 * (c1 - c0);
            for (int i = tid; i < rows * all; i += 64 * WAVES) {
                const int j = i / all, b = i - j * all;
                const int at = b * R + (j & 3) * NIM + (j >> 2);
                if (b >= nbs) {   // the missing blocks of a short chunk
                    dbuf[at] = 0.0f;
                    if constexpr (has_min<FMT>()) cbuf[at] = 0.0f;
                    continue;
                }
                const int64_t row = pairs[j] / a.per;
                uint32_t v[9];
                __builtin_memcpy(v, a.blocks + (row * nb + 8 * c0 + b) * 34, 34);
                uint32_t q[8];
#pragma unroll
                for (int k = 0; k < 8; k++) q[k] = __builtin_amdgcn_alignbyte(k == 7 ? v[8] & 0xFFFFu : v[k + 1], v[k], 2);
                const float d = half_bits(v[0] & 0xFFFFu);
                uint4* to = reinterpret_cast<uint4*>(acts + ((b >> 3) * R + j) * ACT_STRIDE + 32 * (b & 7));
                if constexpr (nibble_block<FMT>()) {
                    to[0] = make_uint4(q[0], q[4], q[1], q[5]);
                    to[1] = make_uint4(q[2], q[6], q[3], q[7]);
                } else {
                    to[0] = make_uint4(q[0], q[1], q[2], q[3]);
                    to[1] = make_uint4(q[4], q[5], q[6], q[7]);
                }
                dbuf[at] = d * scale_back<FMT>();
                if constexpr (has_min<FMT>()) {
                    int S = 0;
#pragma unroll
                    for (int k = 0; k < 8; k++) S = __builtin_amdgcn_sdot4((int)q[k], 0x01010101, S, false);
                    cbuf[at] = d * (float)S;
                }
            }
        }
        __syncthreads();
        for (; c < c1; c += TURN * KS) {
            const int d = PAIR ? c : c + KS;
            stage(c, r0);
            if constexpr (ONE)
                fetch(wt2, valid(d), r0);
            else
                fetch(wt, valid(c + TURN * KS), r0);
            multiply(0, c, c0);
            if constexpr (ONE) {
                stage(valid(d), r0);
                fetch(wt, valid(c + TURN * KS), r0);
            } else {
                stage(valid(d), r1);
                fetch(wt2, valid(d + TURN * KS), r1);
            }
            if (PAIR || d < c1) multiply(MATS - 1, d, c0);   // the last segment may end between the two
        }
        if (KS > 1) {
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int o = tid + 64 * WAVES * q;
                if (o < outs && (o >> 4) % R < rows)
                    for (int cs = 0; cs < c1 - c0; cs++) sum[q] = sum[q] + pbuf[cs * outs + o];
            }
        }
    }

    if (KS == 1) {
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < NIM; i++) {
            const int j = kg + 4 * i;
            if (j < rows && nn <= last_row)
                a.y[pairs[j] * N + n0 + nn] = PAIR ? swiglu(acc[0][i], acc[MATS - 1][i]) : acc[0][i];
        }
        return;
    }
    // output o = ((tile, matrix) R + row) 16 + weight row
    if constexpr (PAIR) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int o = tid + 64 * WAVES * q;
            if (o < outs) pbuf[o] = sum[q];
        }
        __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const int o = tid + 64 * WAVES * q;
        if (o >= outs) break;
        const int n = o & 15, j = (o >> 4) % R, m = (o >> 4) / R;
        const int64_t col = ((int64_t)blockIdx.x * TW + m / MATS) * 16 + n;
        if (j < rows && col < N && (!PAIR || m % 2 == 0))
            a.y[pairs[j] * N + col] = PAIR ? swiglu(sum[q], pbuf[o + R * 16]) : sum[q];
    }
}

constexpr int64_t MOST_Y = 32768;

// Raise a kernel's dynamic-LDS limit to the full 160 KB, once per kernel and device.
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

template <int FMT, bool PAIR, int R, bool AL>
int launch_rows(const MoeArgs& m, RowsArgs& a, hipStream_t s) {
    using F = Fmt<FMT>;
    constexpr int MATS = PAIR ? 2 : 1;
    const int64_t tiles = (a.N + 15) / 16, C = ((a.K >> 5) + 7) / 8;
    a.wbytes = m.E * a.N * (a.K / F::QK) * F::BB;
    const int64_t items = moe_most_items(m.P, m.E, R);
    // waves that share a tile: enough waves to fill the chip
    int ks = 1;
    while (ks < 8 && 2 * ks <= C && tiles * items * ks < 4096) ks *= 2;
    a.ks = ks;
    const int TW = WAVES / ks;
    // a segment: as many chunks as leave a compute unit two workgroups, at
    // least two a wave (the fetches run two ahead); 16 of them take at most
    // 148 KB in any variant
    auto lds_of = [&](int seg) {
        return 64 + (size_t)WAVES * slice<FMT, AL>() +
               (size_t)seg * R * (ACT_STRIDE + 32 * (has_min<FMT>() ? 2 : 1)) +
               (ks > 1 ? (size_t)seg * TW * MATS * R * 64 : 0);
    };
    int seg = SEG;
    while (seg > 2 * ks && lds_of(seg) > 80 * 1024) seg /= 2;
    a.seg = (int32_t)(C < seg ? C : seg);
    const size_t lds = lds_of(a.seg);
    static std::atomic<int> state[64];
    const int rc = raise_lds_limit(reinterpret_cast<const void*>(&k_moe_rows<FMT, PAIR, R, AL>), state);
    if (rc) return rc;
    for (int64_t at = 0; at < items; at += MOST_Y) {   // a grid's second dimension ends at 65535
        a.item0 = (int32_t)at;
        hipLaunchKernelGGL((k_moe_rows<FMT, PAIR, R, AL>),
                           dim3((unsigned)((tiles + TW - 1) / TW),
                                (unsigned)(items - at < MOST_Y ? items - at : MOST_Y)),
                           dim3(64 * WAVES), lds, s, a);
        const int rc2 = (int)hipGetLastError();
        if (rc2) return rc2;
    }
    return 0;
}

template <int FMT, bool PAIR> int launch_fmt(const MoeArgs& m, RowsArgs& a, hipStream_t s) {
    const bool four = moe_rows(m) == 4;
    if constexpr (can_align<FMT>()) {
        if (m.K % 256 == 0)
            return four ? launch_rows<FMT, PAIR, 4, true>(m, a, s) : launch_rows<FMT, PAIR, 16, true>(m, a, s);
    }
    if constexpr (FMT != T_Q4_K)   // whose rows are always whole chunks
        return four ? launch_rows<FMT, PAIR, 4, false>(m, a, s) : launch_rows<FMT, PAIR, 16, false>(m, a, s);
    return (int)hipErrorInvalidValue;
}

template <int FMT> int launch_any(const MoeArgs& m, RowsArgs& a, hipStream_t s) {
    return m.w2 ? launch_fmt<FMT, true>(m, a, s) : launch_fmt<FMT, false>(m, a, s);
}

// ----------------------------------------------------------- combination ----
// y[t][n] = sum over the token's slots with an expert, ascending, of
// weight * yp: one fma each from +0.  V: outputs a thread.
template <int V>
__global__ __launch_bounds__(256) void k_moe_combine(const float* __restrict__ yp,
                                                     const int32_t* __restrict__ idx,
                                                     const float* __restrict__ weight, int64_t T,
                                                     int top, int E, int64_t N,
                                                     float* __restrict__ y) {
    const int64_t per = N / V;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * per;
         i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per, n = (i - t * per) * V;
        float s[V];
#pragma unroll
        for (int v = 0; v < V; v++) s[v] = 0.0f;
        for (int j = 0; j < top; j++) {
            const int64_t p = t * top + j;
            if ((unsigned)idx[p] >= (unsigned)E) continue;
            const float w = weight[p];
            if constexpr (V == 4) {
                const float4 f = *reinterpret_cast<const float4*>(yp + p * N + n);
                s[0] = fmaf(w, f.x, s[0]);
                s[1] = fmaf(w, f.y, s[1]);
                s[2] = fmaf(w, f.z, s[2]);
                s[3] = fmaf(w, f.w, s[3]);
            } else {
                s[0] = fmaf(w, yp[p * N + n], s[0]);
            }
        }
        if constexpr (V == 4)
            *reinterpret_cast<float4*>(y + t * N + n) = make_float4(s[0], s[1], s[2], s[3]);
        else
            y[t * N + n] = s[0];
    }
}

}  // namespace

static int launch_moe_combine(const float* yp, const int32_t* idx, const float* weight, int64_t T,
                       int top, int64_t E, int64_t N, float* y, hipStream_t s) {
    const bool four = N % 4 == 0 && aligned16(y);
    const int64_t blocks = ((four ? T * (N / 4) : T * N) + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
    if (four)
        hipLaunchKernelGGL(k_moe_combine<4>, grid, dim3(256), 0, s, yp, idx, weight, T, top, (int)E,
                           N, y);
    else
        hipLaunchKernelGGL(k_moe_combine<1>, grid, dim3(256), 0, s, yp, idx, weight, T, top, (int)E,
                           N, y);
    return (int)hipGetLastError();
}

// The launch before a product: the sorted pairs (plan) and the activations as
// the kernel takes them (f16 for the GEMM, rows for the GEMV, else Q8_0 blocks
// of x).
static int prepare(const MoeArgs& m, bool plan, bool gemm, bool gemv, hipStream_t s) {
    const MoeWork L = moe_work(m);
    PrepArgs p{};
    p.x = m.x;
    p.xq = m.xq;
    p.blocks = m.work + L.blocks;
    p.da = reinterpret_cast<uint16_t*>(m.work + L.da);
    p.ca = reinterpret_cast<float*>(m.work + L.ca);
    p.nblocks = m.x || gemm ? m.P / m.per * (m.K / 32) : 0;
    p.gemm = gemm;
    if (gemv) {
        p.min = type_has_min(m.type);
        p.row = moe_gemv_row(m.K, p.min);
        p.nb = (int32_t)(m.K / 32);
        p.back = gemv_scale_back(m.type);
    }
    p.idx = m.idx;
    p.P = (int32_t)m.P;
    p.E = (int32_t)m.E;
    p.R = moe_rows(m);
    p.planners = plan ? p.E + 1 : 0;
    p.items = reinterpret_cast<int32_t*>(m.work + L.items);
    p.order = reinterpret_cast<int32_t*>(m.work + L.order);
    p.count = reinterpret_cast<int32_t*>(m.work + L.count);
    p.a16 = aligned16(m.x);
    const int64_t grid = p.planners + (p.nblocks + PREP / 8 - 1) / (PREP / 8);
    if (grid == 0) return 0;
    hipLaunchKernelGGL(k_moe_prep, dim3((unsigned)grid), dim3(PREP), 0, s, p);
    return (int)hipGetLastError();
}

int launch_moe_product(const MoeArgs& m, hipStream_t s) {
    if (m.w2 && moe_gemv_fits(m)) return launch_moe_gemv(m, nullptr, nullptr, m.y, s);
    const MoeWork L = moe_work(m);
    const bool gemm = moe_rows(m) >= 64;
    const int rc = prepare(m, gemm || m.P > MOE_SCAN, gemm, false, s);
    if (rc) return rc;
    if (gemm) return launch_moe_gemm(m, s);
    RowsArgs a{};
    a.w = m.w;
    a.w2 = m.w2;
    a.N = m.N;
    a.K = m.K;
    a.E = (int32_t)m.E;
    a.P = (int32_t)m.P;
    a.per = m.per;
    a.idx = m.idx;
    a.blocks = m.x ? m.work + L.blocks : m.xq;
    a.items = reinterpret_cast<const int32_t*>(m.work + L.items);
    a.order = reinterpret_cast<const int32_t*>(m.work + L.order);
    a.count = reinterpret_cast<const int32_t*>(m.work + L.count);
    a.y = m.y;
    a.scan = m.P <= MOE_SCAN;
    switch (m.type) {
    case T_Q8_0: return launch_any<T_Q8_0>(m, a, s);
    case T_Q4_0: return launch_any<T_Q4_0>(m, a, s);
    case T_Q5_0: return launch_any<T_Q5_0>(m, a, s);
    case T_Q4_1: return launch_any<T_Q4_1>(m, a, s);
    case T_Q5_1: return launch_any<T_Q5_1>(m, a, s);
    case T_Q8_1: return launch_any<T_Q8_1>(m, a, s);
    case T_Q4_K: return launch_any<T_Q4_K>(m, a, s);
    case T_Q6_K: return launch_any<T_Q6_K>(m, a, s);
    }
    return (int)hipErrorInvalidValue;
}

int launch_moe_down(const MoeArgs& m, const float* weight, float* y, hipStream_t s) {
    if (moe_gemv_fits(m)) {
        const uint8_t* rows = nullptr;
        if (m.x && !moe_gemv_quantises(m)) {
            const int rc = prepare(m, false, false, true, s);
            if (rc) return rc;
            rows = m.work + moe_work(m).blocks;
        }
        return launch_moe_gemv(m, rows, weight, y, s);
    }
    const int rc = launch_moe_product(m, s);
    return rc ? rc : launch_moe_combine(m.y, m.idx, weight, m.P / m.top, m.top, m.E, m.N, y, s);
}

}  // namespace qmv
