// The paged 4-bit key/value cache on gfx950: appending rotated keys and
// values, and reading stored values back.
//
// A key or value head is held as Q4_0 values: per 32 elements an fp16 scale d
// and 4-bit codes, value d * (code - 8).  The bytes of a page are laid out for
// the loads of the attention kernel (qmv_kv_attention.hip) rather than as 18-byte GGUF blocks
// (nb = head_dim / 32 blocks a head; per page and head, in this order):
//   K codes  [token][g = 0..3][b][4]   nibble j of the 4 bytes is element
//                                      NIB(j) of 32b + 8g ..., so that a masked
//                                      word holds two adjacent elements in its
//                                      two halves
//   V codes  [token / 4][m = 0..15][b][token % 4]  low nibble element 32b + 2m,
//                                      high nibble 32b + 2m + 1
//   K scales [token][b] fp16, V scales [token][b] fp16
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_internal.h"
#include "qmv_kv_device.h"
#include "qmv_lanes.h"

namespace qmv {
namespace {

// --------------------------------------------------------------- append ----
// One workgroup: some heads of one row, 8 adjacent elements a thread, which are
// a K code word, or 4 V code bytes, once quantised; the 4 threads of a 32-block
// find its largest magnitude by lane exchange, so nothing goes through LDS but
// the row's sines and cosines.  The rotation runs in f64 from the angle to the
// result (an angle of a far position loses its low bits in f32, and a value next
// to a rounding border decides a 4-bit code), rounded once to f32.
//
// A thread needs its elements' partners: within its 8 when pairs are adjacent,
// 8 others when they are halves apart (HALVES), loaded a second time.  VEC:
// 16-byte loads and stores (aligned rows, partners in whole eights).
// Bound by its bytes: 4117 rows of 32 heads on 8 of 128 elements, 178 MB, take 43
// us (4.1 TB/s; a copy reaches 5.2), 45 and 55 with a row's heads on two and three
// workgroups; more waves a SIMD do not help.
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    if constexpr (VEC) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = p[e];
    }
}

// Q4_0 codes of the thread's 8 of a 32-block, and the block's scale (every lane
// of the 4 takes part).
__device__ __forceinline__ _Float16 quantise8(const float (&x)[8], int g, uint32_t (&code)[8]) {
    float big = -1.0f, top = 0.0f;
    int at = 0, bad = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        bad |= !__builtin_isfinite(x[e]);
        if (fabsf(x[e]) > big) {
            big = fabsf(x[e]);
            top = x[e];
            at = 8 * g + e;
        }
    }
    const auto meet = [&](float ob, float ot, int oa, int obad) {  // the first of the largest magnitude
        bad |= obad;
        if (ob > big || (ob == big && oa < at)) {
            big = ob;
            top = ot;
            at = oa;
        }
    };
    meet(dpp<DPP_XOR1>(big), dpp<DPP_XOR1>(top), dpp<DPP_XOR1>(at), dpp<DPP_XOR1>(bad));
    meet(dpp<DPP_XOR2>(big), dpp<DPP_XOR2>(top), dpp<DPP_XOR2>(at), dpp<DPP_XOR2>(bad));
    const float d = top / -8.0f;
    const float r = 1.0f / d, id = __builtin_isinf(r) ? 0.0f : r;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const int c = (int)(x[e] * id + 8.5f);
        code[e] = bad ? 8u : (uint32_t)(c > 15 ? 15 : c);
    }
    return bad ? (_Float16)__builtin_nanf("") : (_Float16)d;
}

template <bool VEC, bool HALVES>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a, int passes) {
    const KvArgs& kv = a.kv;
    __shared__ double turn[2][128];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int D = 32 * kv.nb, eights = 4 * kv.nb;  // of a head
    const int hp = 256 / eights, hu = tid / eights, w = tid - hu * eights;  // heads a pass
    const int units = a.Hq + 2 * kv.Hkv;
    const int half = a.rot >> 1;
    int apart = 0;
    if (HALVES && 8 * w < a.rot) apart = 8 * w < half ? half : -half;
    // a pass's elements and their partners, loaded a pass ahead, and the first before anything else
    float x[8], p[8];
    const auto fetch = [&](int pass) {
        const int u = ((int)blockIdx.y * passes + pass) * hp + hu;
        if (pass >= passes || hu >= hp || u >= units) return;
        const bool is_q = u < a.Hq, is_v = u >= a.Hq + kv.Hkv;
        const float* src = is_q ? a.q + (int64_t)t * a.q_stride + (int64_t)u * D
                         : is_v ? a.v + (int64_t)t * a.v_stride + (int64_t)(u - a.Hq - kv.Hkv) * D
                                : a.k + (int64_t)t * a.k_stride + (int64_t)(u - a.Hq) * D;
        load8<VEC>(src + 8 * w, x);
        if (HALVES && !is_v) {
            if constexpr (VEC) {
                load8<true>(src + 8 * w + apart, p);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int i = 8 * w + e;
                    p[e] = src[i >= a.rot ? i : i < half ? i + half : i - half];
                }
            }
        }
    };
    fetch(0);
    const int b = seq_of_row(kv, t);
    if (b < 0) return;
    const Seq s = seq_of(kv, b);
    const int pos = s.len - s.n + (t - s.q0);
    if (t < s.q0 || t >= s.q0 + s.n || pos < 0) return;  // uniform per workgroup
    if (tid < half) {
        double sn, cs;
        sincos((double)pos * a.freq[tid], &sn, &cs);
        turn[0][tid] = cs;
        turn[1][tid] = sn;
    }
    const int page = page_of(kv, b, pos);
    __syncthreads();
    const int bb = w >> 2, g = w & 3;
    // y[e] = x[e] c + partner[e] (-s or s); adjacent pairs share c and s
    constexpr int TURNS = HALVES ? 8 : 4;
    double c[TURNS], sn[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; k++) {
        const int i = 8 * w + (HALVES ? k : 2 * k);
        const int j = HALVES ? (i < half ? i : i - half) : i >> 1;
        const bool turned = i < a.rot;
        c[k] = turned ? turn[0][j] : 1.0;
        sn[k] = turned ? (HALVES && i < half ? -turn[1][j] : turn[1][j]) : 0.0;
    }
    const int off = pos & ((1 << kv.log2p) - 1);
    const int64_t page_codes = (int64_t)(16 * kv.nb) << kv.log2p;
    for (int pass = 0; pass < passes; pass++) {
        const int u = ((int)blockIdx.y * passes + pass) * hp + hu;
        const bool live = hu < hp && u < units;
        const bool is_q = u < a.Hq, is_v = u >= a.Hq + kv.Hkv;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const float q = HALVES ? p[e] : x[e ^ 1];
            const int k = HALVES ? e : e >> 1;
            const double s = HALVES || (e & 1) ? sn[k] : -sn[k];
            y[e] = is_v || 8 * w + e >= a.rot ? x[e] : (float)((double)x[e] * c[k] + (double)q * s);
        }
        fetch(pass + 1);
        if constexpr (HALVES) __syncthreads();  // q in place: partners are read before any is written
        if (live && is_q) {
            float* dst = a.q_out + ((int64_t)t * a.Hq + u) * D + 8 * w;
            if constexpr (VEC) {
                *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(dst + 4) = make_float4(y[4], y[5], y[6], y[7]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) dst[e] = y[e];
            }
        }
        if (live && !is_q && page >= 0) {  // the same for the 4 threads of a block
            uint32_t code[8];
            const _Float16 dh = quantise8(y, g, code);
            uint8_t* hd = head_of(kv, page, is_v ? u - a.Hq - kv.Hkv : u - a.Hq);
            if (is_v) {
                uint8_t* to = hd + page_codes + (int64_t)(off >> 2) * 64 * kv.nb + (off & 3);
#pragma unroll
                for (int m = 0; m < 4; m++)
                    to[((4 * g + m) * kv.nb + bb) * 4] = (uint8_t)(code[2 * m] | (code[2 * m + 1] << 4));
            } else {
                uint32_t word = 0;
#pragma unroll
                for (int e = 0; e < 8; e++) word |= code[e] << (4 * k_nibble(e));
                *reinterpret_cast<uint32_t*>(hd + (int64_t)off * 16 * kv.nb + (g * kv.nb + bb) * 4) = word;
            }
            if (g == 0) {
                _Float16* sc = reinterpret_cast<_Float16*>(hd + 2 * page_codes);
                if (is_v) sc += (int64_t)kv.nb << kv.log2p;
                sc[off * kv.nb + bb] = dh;
            }
        }
    }
}

// ----------------------------------------------------------------- read ----
// The stored values of every row's token; 8 elements of K and of V a thread.
__global__ __launch_bounds__(256) void k_kv_read(KvArgs kv, float* __restrict__ k,
                                                 float* __restrict__ v) {
    const int t = blockIdx.x;
    const int b = seq_of_row(kv, t);
    if (b < 0) return;
    const Seq s = seq_of(kv, b);
    const int pos = s.len - s.n + (t - s.q0);
    if (t < s.q0 || t >= s.q0 + s.n || pos < 0) return;
    const int page = page_of(kv, b, pos);
    if (page < 0) return;
    const int off = pos & ((1 << kv.log2p) - 1);
    const int64_t page_codes = (int64_t)(16 * kv.nb) << kv.log2p;
    const int per = 4 * kv.nb;  // groups of 8 elements of a head
    for (int i = blockIdx.y * 256 + threadIdx.x; i < kv.Hkv * per; i += 256 * gridDim.y) {
        const int head = i / per, e8 = i - head * per, bb = e8 >> 2, g = e8 & 3;
        const uint8_t* hd = head_of(kv, page, head);
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(hd + 2 * page_codes);
        const float dk = half_value(sc[off * kv.nb + bb]);
        const float dv = half_value(sc[((int64_t)kv.nb << kv.log2p) + off * kv.nb + bb]);
        const uint32_t w =
            *reinterpret_cast<const uint32_t*>(hd + (int64_t)off * 16 * kv.nb + (g * kv.nb + bb) * 4);
        const uint8_t* c = hd + page_codes + (int64_t)(off >> 2) * 64 * kv.nb + (off & 3);
        const int64_t o = ((int64_t)t * kv.Hkv + head) * 32 * kv.nb + 32 * bb + 8 * g;
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const int byte = c[((4 * g + m) * kv.nb + bb) * 4];
            k[o + 2 * m] = dk * (float)((int)((w >> (4 * k_nibble(2 * m))) & 15) - 8);
            k[o + 2 * m + 1] = dk * (float)((int)((w >> (4 * k_nibble(2 * m + 1))) & 15) - 8);
            v[o + 2 * m] = dv * (float)((byte & 15) - 8);
            v[o + 2 * m + 1] = dv * (float)((byte >> 4) - 8);
        }
    }
}

}  // namespace

int launch_kv_append(const AppendArgs& a, hipStream_t s) {
    const int units = a.Hq + 2 * a.kv.Hkv, hp = 256 / (4 * a.kv.nb);
    // few rows: one pass of heads a workgroup; many: all of a row's heads, its sines once
    const int all = (units + hp - 1) / hp;
    const int passes = (int64_t)a.kv.T * all >= 2048 ? all : 1;
    const bool vec = aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.q_out) &&
                     (a.q_stride | a.k_stride | a.v_stride) % 4 == 0 &&
                     (!a.halves || a.rot % 16 == 0);
    const dim3 grid((unsigned)a.kv.T, (unsigned)((all + passes - 1) / passes));
    const auto kernel = a.halves ? vec ? k_kv_append<true, true> : k_kv_append<false, true>
                                 : vec ? k_kv_append<true, false> : k_kv_append<false, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, passes);
    return (int)hipGetLastError();
}

int launch_kv_read(const KvArgs& kv, float* k, float* v, hipStream_t s) {
    const int per = kv.Hkv * 4 * kv.nb;
    hipLaunchKernelGGL(k_kv_read, dim3((unsigned)kv.T, (unsigned)((per + 255) / 256)), dim3(256), 0,
                       s, kv, k, v);
    return (int)hipGetLastError();
}

}  // namespace qmv
