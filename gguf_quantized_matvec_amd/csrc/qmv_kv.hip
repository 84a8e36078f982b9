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

#include "qmv_kv_device.h"

namespace qmv {
namespace {

// --------------------------------------------------------------- append ----
constexpr int HEADS = 8;  // heads (of q, k and v together) per workgroup

// One workgroup: HEADS heads of one row.  The rotation runs in f64 from the
// angle to the result (an angle of a far position loses its low bits in f32,
// and a value next to a rounding border decides a 4-bit code), rounded once
// to f32; rotated keys and the values are staged in LDS and quantised by 4
// lanes per 32-element block.
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
    const KvArgs& kv = a.kv;
    __shared__ double turn[2][128];
    extern __shared__ float stage[];  // [HEADS][D]
    const int t = blockIdx.x, tid = threadIdx.x;
    const int D = 32 * kv.nb;
    const int b = seq_of_row(kv, t);
    if (b < 0) return;
    const Seq s = seq_of(kv, b);
    const int pos = s.len - s.n + (t - s.q0);
    if (t < s.q0 || t >= s.q0 + s.n || pos < 0) return;  // uniform per workgroup
    const int half = a.rot >> 1;
    if (tid < half) {
        double sn, cs;
        sincos((double)pos * a.freq[tid], &sn, &cs);
        turn[0][tid] = cs;
        turn[1][tid] = sn;
    }
    __syncthreads();
    const int u0 = blockIdx.y * HEADS, units = a.Hq + 2 * kv.Hkv;
    const int heads = units - u0 < HEADS ? units - u0 : HEADS;
    const int pairs = D >> 1;
    for (int i = tid; i < heads * pairs; i += 256) {
        const int hu = i / pairs, j = i - hu * pairs, u = u0 + hu;
        const bool is_q = u < a.Hq, is_v = u >= a.Hq + kv.Hkv;
        const float* src = is_q ? a.q + (int64_t)t * a.q_stride + (int64_t)u * D
                         : is_v ? a.v + (int64_t)t * a.v_stride + (int64_t)(u - a.Hq - kv.Hkv) * D
                                : a.k + (int64_t)t * a.k_stride + (int64_t)(u - a.Hq) * D;
        float* dst = is_q ? a.q_out + ((int64_t)t * a.Hq + u) * D : stage + hu * D;
        int e0 = 2 * j, e1 = 2 * j + 1;
        if (a.halves && j < half) {
            e0 = j;
            e1 = j + half;
        }
        const float x0 = src[e0], x1 = src[e1];
        if (!is_v && j < half) {
            const double c = turn[0][j], n = turn[1][j];
            dst[e0] = (float)((double)x0 * c - (double)x1 * n);
            dst[e1] = (float)((double)x0 * n + (double)x1 * c);
        } else {
            dst[e0] = x0;
            dst[e1] = x1;
        }
    }
    __syncthreads();
    const int page = page_of(kv, b, pos);
    if (page < 0) return;
    const int off = pos & ((1 << kv.log2p) - 1), g = tid & 3;
    const int64_t page_codes = (int64_t)(16 * kv.nb) << kv.log2p;
    const int blocks = heads * kv.nb;  // 4 lanes each: every lane of a group agrees on `live`
    for (int i0 = 0; i0 < blocks; i0 += 64) {
        const int blk = i0 + (tid >> 2), hu = blk / kv.nb, bb = blk - hu * kv.nb, u = u0 + hu;
        const bool live = blk < blocks && u >= a.Hq;
        float x[8];
        float big = -1.0f, top = 0.0f;
        int at = 0, bad = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            x[e] = live ? stage[hu * D + 32 * bb + 8 * g + e] : 0.0f;
            bad |= !__builtin_isfinite(x[e]);
            if (fabsf(x[e]) > big) {
                big = fabsf(x[e]);
                top = x[e];
                at = 8 * g + e;
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {  // the first of the largest magnitude
            const float ob = __shfl_xor(big, o), ot = __shfl_xor(top, o);
            const int oa = __shfl_xor(at, o);
            bad |= __shfl_xor(bad, o);
            if (ob > big || (ob == big && oa < at)) {
                big = ob;
                top = ot;
                at = oa;
            }
        }
        if (!live) continue;
        const float d = top / -8.0f;
        const float r = 1.0f / d, id = __builtin_isinf(r) ? 0.0f : r;
        uint32_t code[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int c = (int)(x[e] * id + 8.5f);
            code[e] = bad ? 8u : (uint32_t)(c > 15 ? 15 : c);
        }
        const _Float16 dh = bad ? (_Float16)__builtin_nanf("") : (_Float16)d;
        const bool is_v = u >= a.Hq + kv.Hkv;
        uint8_t* hd = head_of(kv, page, is_v ? u - a.Hq - kv.Hkv : u - a.Hq);
        if (is_v) {
            uint8_t* c = hd + page_codes + (int64_t)(off >> 2) * 64 * kv.nb + (off & 3);
#pragma unroll
            for (int m = 0; m < 4; m++)
                c[((4 * g + m) * kv.nb + bb) * 4] = (uint8_t)(code[2 * m] | (code[2 * m + 1] << 4));
        } else {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) w |= code[e] << (4 * k_nibble(e));
            *reinterpret_cast<uint32_t*>(hd + (int64_t)off * 16 * kv.nb + (g * kv.nb + bb) * 4) = w;
        }
        if (g == 0) {
            _Float16* sc = reinterpret_cast<_Float16*>(hd + 2 * page_codes);
            if (is_v) sc += (int64_t)kv.nb << kv.log2p;
            sc[off * kv.nb + bb] = dh;
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
    const int units = a.Hq + 2 * a.kv.Hkv;
    hipLaunchKernelGGL(k_kv_append, dim3((unsigned)a.kv.T, (unsigned)((units + HEADS - 1) / HEADS)),
                       dim3(256), (size_t)HEADS * 32 * a.kv.nb * 4, s, a);
    return (int)hipGetLastError();
}

int launch_kv_read(const KvArgs& kv, float* k, float* v, hipStream_t s) {
    const int per = kv.Hkv * 4 * kv.nb;
    hipLaunchKernelGGL(k_kv_read, dim3((unsigned)kv.T, (unsigned)((per + 255) / 256)), dim3(256), 0,
                       s, kv, k, v);
    return (int)hipGetLastError();
}

}  // namespace qmv
