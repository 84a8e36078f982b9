// Experts' products for single tokens and few of them, for gfx950: hardly any
// two pairs share an expert, so the multiply is a matrix-vector product a pair,
// bound by the bytes of the experts' weights.  Order and rounding are
// qmv_launch's (include/qmv.h); every pair's result is bit-identical to it.
//
// Every lane owns one 256-element chunk of one weight row: it streams the
// chunk's bytes into registers, forms the codes of a block as int8 and takes
// the block's integer with v_dot4_i32_i8 against the activations in LDS.  With
// one activation row that needs a third of the vector instructions of the
// matrix kernels (qmv_moe_rows.hip), whose instructions would be filled to a
// sixteenth.  C lanes a row for C chunks, floor(64 / C) rows a wave; the chunk
// sums are added in chunk order through LDS.
//
// Gate and up: a workgroup takes one pair; half of a wave's lane rows take
// gate rows, the other half the same up rows, which meet in LDS.  The
// workgroup quantises its token's x itself: one launch.
// Down: a wave takes one slot's expert and a workgroup all slots of a token for
// the same rows, whose weighted products it adds itself.
//
// Measured for one token, two experts: gate and up of 14336 x 4096 in Q4_K 28.9
// us (4.6 TB/s; a copy of 2 GiB reaches 4.9), by the kernel of 16 columns 48 for
// the call; down of 4096 x 14336 in Q6_K 24.2 us (4.0 TB/s) behind a launch of 4
// that quantises, the call 28.0 against 46.
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "qmv_moe.h"
#include "qmv_moe_device.h"

namespace qmv {
namespace {

// Chunks start 4-byte aligned always, or (blocks of 18, 22, 34, 210 bytes) only
// 2-byte aligned: then one dword more is loaded, from the 4-byte aligned address
// at or below the start, and the bytes are shifted down just before their use
// (16-byte loads at 2-byte alignment lose a quarter of the bandwidth).
template <int FMT> constexpr bool always4() { return Fmt<FMT>::BB % 4 == 0; }
template <int FMT> constexpr int dwords() { return (Fmt<FMT>::CB + 3) / 4 + (always4<FMT>() ? 0 : 1); }

constexpr int WAVES = 4;          // of a workgroup (gate and up), at least (down)
constexpr int MOST_SLOTS = 16;    // of a token, a wave each (down)
constexpr int ACT_STRIDE = 272;   // bytes of a chunk in a row of activations

// The dword (16 bits, byte) at byte O of the chunk's registers.
template <int O, int W> __device__ __forceinline__ uint32_t dw(const uint32_t (&r)[W]) {
    static_assert(O >= 0 && O + 4 <= 4 * W, "outside the chunk");
    if constexpr (O % 4 == 0)
        return r[O / 4];
    else
        return __builtin_amdgcn_alignbyte(r[O / 4 + 1], r[O / 4], O % 4);
}
template <int O, int W> __device__ __forceinline__ uint32_t half(const uint32_t (&r)[W]) {
    return (r[O / 4] >> (8 * (O % 4))) & 0xFFFFu;
}
template <int O, int W> __device__ __forceinline__ int byte(const uint32_t (&r)[W]) {
    return (int)((r[O / 4] >> (8 * (O % 4))) & 0xFFu);
}
__device__ __forceinline__ int dot4(uint32_t a, uint32_t b, int c) {
    return __builtin_amdgcn_sdot4((int)a, (int)b, c, false);
}

// The sum of one chunk in the documented order.  act: its 256 activation codes;
// da, ca: scale (times gemv_scale_back) and scale times code sum of its blocks; nbc:
// how many blocks it has (the others are computed and dropped: no branch).
template <int FMT>
__device__ __forceinline__ float dot_chunk(const uint32_t (&r)[dwords<FMT>()], const uint8_t* act,
                                           const float* da, const float* ca, int nbc) {
    using F = Fmt<FMT>;
    float p = 0.0f;
    float d = 0.0f, dmin = 0.0f;
    uint32_t sc[2] = {0, 0}, mn[2] = {0, 0};
    if constexpr (FMT == T_Q4_K) {
        d = half_bits(half<0>(r));
        dmin = half_bits(half<2>(r));
        // 6-bit scales and minimums of sub-blocks 0..3, 4..7, one a byte
        sc[0] = r[1] & 0x3F3F3F3Fu;
        mn[0] = r[2] & 0x3F3F3F3Fu;
        sc[1] = (r[3] & 0x0F0F0F0Fu) | ((r[1] >> 2) & 0x30303030u);
        mn[1] = ((r[3] >> 4) & 0x0F0F0F0Fu) | ((r[2] >> 2) & 0x30303030u);
    }
    if constexpr (FMT == T_Q6_K) d = half_bits(half<208>(r));
    each<8>([&](auto B) {
        constexpr int b = B;
        const uint4 lo = *reinterpret_cast<const uint4*>(act + 32 * b);
        const uint4 hi = *reinterpret_cast<const uint4*>(act + 32 * b + 16);
        const uint32_t a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t w[8];
        float mw = 0.0f;
        if constexpr (FMT == T_Q8_0 || FMT == T_Q8_1) {
            d = half_bits(half<F::BB * b>(r));
            each<8>([&](auto i) { w[i] = dw<F::BB * b + (FMT == T_Q8_0 ? 2 : 4) + 4 * i>(r); });
        } else if constexpr (FMT == T_Q4_K) {
            each<8>([&](auto i) {
                w[i] = (dw<16 + 32 * (b >> 1) + 4 * i>(r) >> (4 * (b & 1))) & 0x0F0F0F0Fu;
            });
            mw = -(dmin * (float)((mn[b >> 2] >> (8 * (b & 3))) & 0xFFu));
        } else if constexpr (FMT == T_Q6_K) {
            constexpr int h = b >> 2, k = b & 3;
            // 4 (q - 32): the six bits at the top of a byte, the sign flipped
            each<8>([&](auto i) {
                const uint32_t ql = dw<64 * h + 32 * (k & 1) + 4 * i>(r), qh = dw<128 + 32 * h + 4 * i>(r);
                const uint32_t l = k >> 1 ? (ql >> 2) & 0x3C3C3C3Cu : (ql << 2) & 0x3C3C3C3Cu;
                const uint32_t u = k == 3 ? qh & 0xC0C0C0C0u : (qh << (6 - 2 * k)) & 0xC0C0C0C0u;
                w[i] = (l | u) ^ 0x80808080u;
            });
        } else {
            constexpr int QS = FMT == T_Q4_0 ? 2 : FMT == T_Q4_1 ? 4 : FMT == T_Q5_0 ? 6 : 8;
            d = half_bits(half<F::BB * b>(r));
            if constexpr (has_min<FMT>()) mw = half_bits(half<F::BB * b + 2>(r));
            uint32_t h = 0;
            if constexpr (FMT == T_Q5_0) h = dw<F::BB * b + 2>(r);
            if constexpr (FMT == T_Q5_1) h = dw<F::BB * b + 4>(r);
            each<4>([&](auto i) {
                const uint32_t v = dw<F::BB * b + QS + 4 * i>(r);
                if constexpr (FMT == T_Q4_0) {
                    w[i] = ((v << 4) & 0xF0F0F0F0u) ^ 0x80808080u;
                    w[4 + i] = (v & 0xF0F0F0F0u) ^ 0x80808080u;
                } else if constexpr (FMT == T_Q4_1) {
                    w[i] = v & 0x0F0F0F0Fu;
                    w[4 + i] = (v >> 4) & 0x0F0F0F0Fu;
                } else if constexpr (FMT == T_Q5_0) {
                    w[i] = (((v << 3) & 0x78787878u) | (spread(h >> (4 * i)) << 7)) ^ 0x80808080u;
                    w[4 + i] = (((v >> 1) & 0x78787878u) | (spread(h >> (16 + 4 * i)) << 7)) ^ 0x80808080u;
                } else {
                    w[i] = (v & 0x0F0F0F0Fu) | (spread(h >> (4 * i)) << 4);
                    w[4 + i] = ((v >> 4) & 0x0F0F0F0Fu) | (spread(h >> (16 + 4 * i)) << 4);
                }
            });
        }
        int I = 0;
        if constexpr (FMT == T_Q6_K) {
            int D0 = 0, D1 = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) D0 = dot4(w[i], a[i], D0);
#pragma unroll
            for (int i = 4; i < 8; i++) D1 = dot4(w[i], a[i], D1);
            I = __mul24((int)(int8_t)byte<192 + 2 * b>(r), D0) + __mul24((int)(int8_t)byte<193 + 2 * b>(r), D1);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) I = dot4(w[i], a[i], I);
            if constexpr (FMT == T_Q4_K) I = __mul24((int)((sc[b >> 2] >> (8 * (b & 3))) & 0xFFu), I);
        }
        float t = fmaf((float)I, d * da[b], p);
        if constexpr (has_min<FMT>()) t = fmaf(mw, ca[b], t);
        p = F::QK == 256 || b < nbc ? t : p;
    });
    return p;
}

// One chunk's bytes at byte `off` of the blob into registers.  LEAN: whole
// 4-byte aligned chunks, so that the loads are not behind a branch and a wait
// for loads issued before them need not wait for them.
template <int FMT, bool LEAN>
__device__ __forceinline__ void load_chunk(const uint8_t* w, int64_t off, int64_t wbytes, bool on,
                                           uint32_t (&r)[dwords<FMT>()]) {
    constexpr int W = dwords<FMT>(), CB = Fmt<FMT>::CB;
    if constexpr (LEAN) {
        __builtin_memcpy(r, reinterpret_cast<const uint32_t*>(w + (on ? off : 0)), CB);
#pragma unroll
        for (int i = CB / 4; i < W; i++) r[i] = 0;
    } else {
        const int64_t off4 = off & ~int64_t(3);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(w + off4);
        const bool near_end = on && off4 + 4 * W > wbytes;
        if (!on) {
#pragma unroll
            for (int i = 0; i < W; i++) r[i] = 0;
        } else if (__builtin_amdgcn_ballot_w64(near_end) == 0) {
            __builtin_memcpy(r, p, 4 * W);
        } else {   // the blob's last chunks: dwords, then the final half of one
#pragma unroll
            for (int i = 0; i < W; i++) {
                const int64_t at = off4 + 4 * i;
                r[i] = at + 4 <= wbytes ? p[i]
                     : at + 2 <= wbytes ? (uint32_t)*reinterpret_cast<const uint16_t*>(w + at) : 0u;
            }
        }
    }
}
template <int FMT, bool LEAN>
__device__ __forceinline__ void realign(int64_t off, uint32_t (&r)[dwords<FMT>()]) {
    if constexpr (!LEAN && !always4<FMT>()) {
        const uint32_t sh = (uint32_t)(off & 3);   // 0 or 2
        if (__builtin_amdgcn_ballot_w64(sh != 0) != 0) {
#pragma unroll
            for (int i = 0; i + 1 < dwords<FMT>(); i++) r[i] = __builtin_amdgcn_alignbyte(r[i + 1], r[i], sh);
        }
    }
}
template <int FMT> constexpr bool can_lean() { return Fmt<FMT>::CB % 4 == 0; }

// Quantises 8 lanes' 4 elements each of a Q8_0 block (as the library's
// quantisers do) and lays the block into a row of activations.
template <int FMT>
__device__ __forceinline__ void put_block(uint8_t* act, int C, int b, int sub, uint32_t c, float d, int S) {
    *reinterpret_cast<uint32_t*>(act + (b >> 3) * ACT_STRIDE + (b & 7) * 32 + 4 * sub) = c;
    if (sub == 0) {
        float* da = reinterpret_cast<float*>(act + C * ACT_STRIDE);
        da[b] = d * gemv_scale_back(FMT);
        if constexpr (has_min<FMT>()) da[8 * C + b] = d * (float)S;
    }
}

struct GemvArgs {
    const uint8_t *w, *w2;
    int64_t N, K, wbytes;
    int32_t E, top;
    const int32_t* idx;
    const uint8_t* rows;     // the activations quantised (moe_gemv_row), or NULL:
    const float* x;          // to be quantised here, or NULL:
    const uint8_t* blocks;   // their Q8_0 blocks
    const float* weight;     // down
    float* y;
    bool a16;                // x is 16-byte aligned
};

// One row of activations into LDS: row `row` of a.x or a.blocks.
template <int FMT>
__device__ __forceinline__ void stage_row(const GemvArgs& a, int64_t row, uint8_t* act, int nb, int C) {
    const int tid = threadIdx.x, sub = tid & 7;
    for (int b0 = 0; b0 < nb; b0 += blockDim.x / 8) {
        const int b = b0 + (tid >> 3);
        const bool live = b < nb;
        uint32_t c = 0;
        float d = 0.0f;
        if (a.x)
            d = quantise_block(a.x + row * a.K + 32 * b + 4 * sub, live, a.a16, c);
        else if (live)
            d = read_block(a.blocks + (row * nb + b) * 34, sub, c);
        const int S = has_min<FMT>() ? block_sum(c) : 0;
        if (live) put_block<FMT>(act, C, b, sub, c, d, S);
    }
}

// PAIR: gate and up of pair blockIdx.y, a wave a unit of rows.  Else the down
// products of token blockIdx.y with the weighted sum, a wave a unit and slot.
template <int FMT, bool PAIR, bool LEAN>
__global__ __launch_bounds__(PAIR ? 64 * WAVES : 64 * MOST_SLOTS) void k_moe_gemv(GemvArgs a) {
    using F = Fmt<FMT>;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wv = uniform(tid >> 6), waves = blockDim.x >> 6;
    const int64_t N = a.N, K = a.K;
    const int nb = (int)(K >> 5), C = (nb + 7) >> 3, G = 64 / C, GP = PAIR ? G >> 1 : G;
    const int slots = PAIR ? 1 : a.top, slot = wv % slots, unit = wv / slots;
    const int lrow = lane / C, c = lane - lrow * C;
    const int64_t u = (int64_t)blockIdx.x * (waves / slots) + unit;
    const int64_t row = u * GP + (PAIR && lrow >= GP ? lrow - GP : lrow);
    const int64_t p = (int64_t)blockIdx.y * slots + slot;
    const int e = uniform(a.idx[p]);
    const bool there = (unsigned)e < (unsigned)a.E;     // a slot with an expert
    const bool on = there && lrow < (PAIR ? 2 * GP : G) && row < N;
    const int64_t R = K / F::QK * F::BB;
    const int64_t at = (e * N + row) * R + (int64_t)c * F::CB;
    const int rowb = moe_gemv_row(K, has_min<FMT>());
    uint8_t* act = smem + slot * rowb;
    float* sums = reinterpret_cast<float*>(smem + slots * rowb);    // [waves][64] chunk sums, then rows
    float* mine = sums + 64 * wv;

    if (PAIR && !there) {
        if (lane < GP && u * GP + lane < N) a.y[p * N + u * GP + lane] = 0.0f;
        return;
    }
    uint32_t r[dwords<FMT>()];
    if (!PAIR && a.rows) {
        // the slots' rows as they are, straight into LDS, on the way together
        // with the weights: the wait is for both
        const uint8_t* from = a.rows + (int64_t)blockIdx.y * slots * rowb;
        for (int i0 = 64 * wv; i0 < slots * rowb / 16; i0 += blockDim.x)
            if (i0 + lane < slots * rowb / 16)
                __builtin_amdgcn_global_load_lds(from + 16 * (i0 + lane), (lds_void*)(smem + 16 * i0), 16, 0, 0);
        load_chunk<FMT, LEAN>(a.w, at, a.wbytes, on, r);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    } else {
        load_chunk<FMT, LEAN>(PAIR && lrow >= GP ? a.w2 : a.w, at, a.wbytes, on, r);
        for (int j = 0; j < slots; j++)
            stage_row<FMT>(a, PAIR ? p / a.top : (int64_t)blockIdx.y * slots + j, smem + j * rowb, nb, C);
    }
    __syncthreads();
    float sum = 0.0f;
    if (on) {
        realign<FMT, LEAN>(at, r);
        const float* da = reinterpret_cast<const float*>(act + C * ACT_STRIDE) + 8 * c;
        sum = dot_chunk<FMT>(r, act + c * ACT_STRIDE, da, da + 8 * C, F::QK == 32 ? min(8, nb - 8 * c) : 8);
    }
    mine[lane] = sum;
    wave_sync();
    float y = 0.0f;
    if (lane < G)
        for (int k = 0; k < C; k++) y = y + mine[lane * C + k];
    wave_sync();
    if (lane < G) mine[lane] = y;
    if constexpr (PAIR) {
        wave_sync();
        if (lane < GP && u * GP + lane < N)
            a.y[p * N + u * GP + lane] = swiglu(mine[lane], mine[GP + lane]);
    } else {
        __syncthreads();
        if (slot == 0 && lane < G && u * G + lane < N) {
            float s = 0.0f;
            for (int j = 0; j < slots; j++) {
                const int64_t q = (int64_t)blockIdx.y * slots + j;
                if ((unsigned)a.idx[q] < (unsigned)a.E) s = fmaf(a.weight[q], sums[64 * (wv + j) + lane], s);
            }
            a.y[blockIdx.y * N + u * G + lane] = s;
        }
    }
}

// The launch of a call (K <= 8192 for a gate/up pair, 16384 for a down product).
struct Grid {
    int slots, units;   // of a workgroup: slots, and units of rows, a wave each
    int64_t x;          // workgroups side by side
    int threads() const { return 64 * slots * units; }
};
Grid grid_of(const MoeArgs& m) {
    const int C = (int)((m.K / 32 + 7) / 8), rows = m.w2 ? 64 / C >> 1 : 64 / C;   // of a unit
    const int waves = m.w2 ? WAVES : 8, slots = m.w2 ? 1 : m.top;
    const int units = slots < waves ? waves / slots : 1;
    const int64_t all = (m.N + rows - 1) / rows;
    return {slots, units, (all + units - 1) / units};
}

template <int FMT, bool PAIR, bool LEAN>
int launch_lean(const MoeArgs& m, GemvArgs& a, hipStream_t s) {
    using F = Fmt<FMT>;
    a.wbytes = m.E * m.N * (m.K / F::QK) * F::BB;
    const Grid g = grid_of(m);
    const size_t lds = (size_t)g.slots * moe_gemv_row(m.K, has_min<FMT>()) + g.slots * g.units * 256;
    hipLaunchKernelGGL((k_moe_gemv<FMT, PAIR, LEAN>), dim3((unsigned)g.x, (unsigned)(m.P / g.slots)),
                       dim3(g.threads()), lds, s, a);
    return (int)hipGetLastError();
}

template <int FMT> int launch_fmt(const MoeArgs& m, GemvArgs& a, hipStream_t s) {
    if constexpr (can_lean<FMT>()) {
        if (m.K % 256 == 0)
            return m.w2 ? launch_lean<FMT, true, true>(m, a, s) : launch_lean<FMT, false, true>(m, a, s);
    }
    return m.w2 ? launch_lean<FMT, true, false>(m, a, s) : launch_lean<FMT, false, false>(m, a, s);
}

}  // namespace

bool moe_gemv_fits(const MoeArgs& m) {
    // Every pair reads its expert's weights here, once a pair; there once an
    // expert, behind a second launch.  So by the bytes that repeated experts
    // would read again, as far as the experts of different tokens are
    // independent (E (1 - (1 - top / E)^T) of them).  Measured, here / there in
    // us, at repeated MB: 64 experts of 2 x 1024 x 2048 in Q4_0, 8 a token: 8
    // tokens (52 MB) 23.9 / 29.9, 12 (106 MB) 32.3 / 33.7, 16 41.2 / 33.9; 16 of
    // 4096 x 4096 in Q6_K, 2 a token: 4 tokens (20 MB) 25.8 / 27.7, 8 (76 MB)
    // 46.9 / 48.3, 12 67.0 / 53.1.  Matrices beyond 16 MB do not stay in the
    // caches between two readers: 8 of 2 x 14336 x 4096 in Q4_K, 2 a token: 1
    // token 28.9 / 31.9, 2 (33 MB) 56.2 / 54.4, 4 98.9 / 86.4.
    // How many rows an expert has does not matter beside that, up to the 128
    // pairs: one expert of 2 x 256 x 256 in Q4_0 and 128 tokens 4.2 / 12.3, of 2 x
    // 896 x 1024 and 32 tokens 7.1 / 9.5, of 1024 x 2048 in Q6_K and 32 tokens 12.2 /
    // 12.4; 16 experts of 896 x 1024 in Q4_K, 4 a token, 32 tokens 16.0 / 14.8, the
    // most that is lost (of 118 shapes of 16 to 128 pairs, 1 to 128 an expert).
    if (m.P > 128) return false;
    const double T = (double)(m.P / m.top), E = (double)m.E;
    const double experts = m.top < E ? E * (1.0 - pow(1.0 - m.top / E, T)) : E;
    const double matrix = (double)(m.w2 ? 2 : 1) * m.N * row_bytes(m.type, m.K);
    if (T > 1.0 && (matrix > 16e6 || (m.P - experts) * matrix > 60e6)) return false;
    if (m.w2) {
        if (m.K > 8192) return false;                   // two rows a wave at least
    } else if (m.K > 16384 || m.top > MOST_SLOTS ||
               m.top * (moe_gemv_row(m.K, type_has_min(m.type)) + 256) + 8 * 256 > 64 * 1024) {
        return false;
    }
    // a grid's dimension ends below 2^32 threads (down: 11 million rows and more)
    const Grid g = grid_of(m);
    return g.x * g.threads() < (int64_t)1 << 32;
}

bool moe_gemv_quantises(const MoeArgs& m) { return m.w2 != nullptr || m.K <= 2048; }

int launch_moe_gemv(const MoeArgs& m, const uint8_t* rows, const float* weight, float* y,
                    hipStream_t s) {
    GemvArgs a{};
    a.w = m.w;
    a.w2 = m.w2;
    a.N = m.N;
    a.K = m.K;
    a.E = (int32_t)m.E;
    a.top = m.top;
    a.idx = m.idx;
    a.rows = rows;
    a.x = m.x;
    a.blocks = m.xq;
    a.weight = weight;
    a.y = y;
    a.a16 = aligned16(m.x);
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
