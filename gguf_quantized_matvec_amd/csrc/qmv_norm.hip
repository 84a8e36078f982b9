// Residual add, RMS norm and 8-bit quantisation in one pass on gfx950.
//
//   h = x + res (one f32 addition; h = x without res)
//   y_i = (float)(h_i * r * w_i),  r = 1 / sqrt(sum h^2 / K + eps)
//
// and y quantised exactly as quantize_act_q8_0 / quantize_act_q8_k quantise
// a row (the same public blocks and private staging), so that the products
// that follow take it with x = NULL.  The llama-family block runs this before
// its attention and its feed-forward projections.
//
// The sum of squares and the products up to y are in f64: the codes follow
// the formula rather than the order of a 32-bit sum, and the f64 rate of this
// chip is its f32 rate, so the pass stays bound by bytes.  The order of the
// sum is fixed: each 256-element chunk is summed by one wave (4 elements a
// lane in order, then a butterfly over the lanes), the chunks are added in
// ascending order.  It depends on K alone, so a row's bits do not depend on
// the rows beside it or on the workgroup that takes it.
//
// Built with -ffp-contract=off: every float operation is the one written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_internal.h"
#include "qmv_lanes.h"
#include "qmv_step.h"

namespace qmv {
namespace {

struct NormArgs {
    const float *x, *res, *w;
    float eps;
    int64_t rows, K;
    float *h, *y;
    uint8_t* xq;
    int64_t row0;  // the launch's first row
};

// id = 1/d, or 0 when 1/d is not finite (the block quantises to zero codes)
__device__ __forceinline__ float inv_scale(float d) {
    const float r = 1.0f / d;
    return __builtin_isinf(r) ? 0.0f : r;
}

__device__ __forceinline__ uint16_t half_bits(float x) {
    const _Float16 f = (_Float16)x;
    uint16_t h;
    __builtin_memcpy(&h, &f, 2);
    return h;
}

__device__ __forceinline__ float half_value(uint16_t h) {
    _Float16 f;
    __builtin_memcpy(&f, &h, 2);
    return (float)f;
}

__device__ __forceinline__ float4 load4(const float* p, bool a16) {
    if (a16) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}

__device__ __forceinline__ void store4(float* p, float4 v, bool a16) {
    if (a16) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

__device__ __forceinline__ float amax4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// The four codes round-half-away(v * id) as bytes, and their sum.
__device__ __forceinline__ uint32_t codes4(float4 v, float id, int& sum) {
    const int c0 = (int)roundf(v.x * id), c1 = (int)roundf(v.y * id);
    const int c2 = (int)roundf(v.z * id), c3 = (int)roundf(v.w * id);
    sum = c0 + c1 + c2 + c3;
    return ((uint32_t)c0 & 0xFFu) | (((uint32_t)c1 & 0xFFu) << 8) | (((uint32_t)c2 & 0xFFu) << 16) |
           ((uint32_t)c3 << 24);
}

// What a wave writes of a 256-element chunk of y, 4 elements v a lane (live:
// the lane's elements are inside the row).  MODE: the Staging bit of Q8_0, or
// 0 for Q8_K.
template <int MODE, class Layout>
__device__ __forceinline__ void quantise_chunk(float4 v, bool live, int lane, int64_t chunk,
                                               int64_t r, const NormArgs& a, const Layout& L) {
    float amax = amax4(v);
    if constexpr (MODE != 0) {  // one 32-block per 8 lanes
        amax = max8(amax);
        const float d = amax / 127.0f;
        int s4;
        const uint32_t c4 = codes4(v, inv_scale(d), s4);
        int s16 = s4 + dpp<DPP_XOR1>(s4);
        s16 += dpp<DPP_XOR2>(s16);            // the sum of this lane's 16-code half
        const int s16o = dpp<DPP_MIRROR8>(s16);  // the other half's
        const int sub = lane & 7;
        const int64_t b = chunk * 8 + (lane >> 3), bi = r * L.nb + b;
        const uint16_t hb = half_bits(d);
        const float dval = half_value(hb);
        const int S = s16 + s16o;
        if (!live) return;
        uint8_t* pub = a.xq + bi * 34;
        uint16_t* pc = reinterpret_cast<uint16_t*>(pub + 2 + 4 * sub);
        pc[0] = (uint16_t)(c4 & 0xFFFFu);
        pc[1] = (uint16_t)(c4 >> 16);
        if (sub == 0) *reinterpret_cast<uint16_t*>(pub) = hb;
        if constexpr (MODE == ST_ROW) {
            *reinterpret_cast<uint32_t*>(a.xq + L.rcodes + r * a.K + 32 * b + 4 * sub) = c4;
            if (sub == 0) {
                reinterpret_cast<float*>(a.xq + L.rda)[bi] = dval;
                reinterpret_cast<float*>(a.xq + L.rca)[bi] = dval * (float)S;
                reinterpret_cast<int32_t*>(a.xq + L.rs16)[bi] =
                    (int32_t)(((uint32_t)s16 & 0xFFFFu) | ((uint32_t)s16o << 16));
            }
        } else if constexpr (MODE == ST_MFMA) {
            const int64_t gb = (r >> 4) * L.nb + b;
            const int m = (int)(r & 15);
            *reinterpret_cast<uint32_t*>(a.xq + L.codes + gb * 512 + (m + 16 * (sub >> 1)) * 8 +
                                         4 * (sub & 1)) = c4;
            if (sub == 0) {
                reinterpret_cast<float*>(a.xq + L.da)[gb * 16 + m] = dval;
                reinterpret_cast<float*>(a.xq + L.ca)[gb * 16 + m] = dval * (float)S;
                reinterpret_cast<int32_t*>(a.xq + L.S)[gb * 16 + m] = S;
            }
        } else {  // ST_F16: code values are exact in f16
            uint32_t hw[2];
#pragma unroll
            for (int t = 0; t < 2; t++)
                hw[t] = (uint32_t)half_bits((float)(int8_t)(c4 >> (16 * t))) |
                        ((uint32_t)half_bits((float)(int8_t)(c4 >> (16 * t + 8))) << 16);
            *reinterpret_cast<uint2*>(a.xq + L.hcodes + (r * a.K + 32 * b + 4 * sub) * 2) =
                make_uint2(hw[0], hw[1]);
            if (sub == 0) {
                reinterpret_cast<uint16_t*>(a.xq + L.hda)[bi] = hb;
                reinterpret_cast<float*>(a.xq + L.rca)[bi] = dval * (float)S;
            }
        }
    } else {  // one superblock per wave; K % 256 == 0, so every lane is live
        amax = max64(amax);
        const float d = amax / 127.0f;
        int s4;
        const uint32_t c4 = codes4(v, inv_scale(d), s4);
        int s16 = s4 + dpp<DPP_XOR1>(s4);
        s16 += dpp<DPP_XOR2>(s16);
        const int s16o = dpp<DPP_MIRROR8>(s16);
        const int64_t task = r * L.nsb + chunk;
        uint8_t* pub = a.xq + task * 292;
        if (lane == 0) *reinterpret_cast<float*>(pub) = d;
        *reinterpret_cast<uint32_t*>(pub + 4 + 4 * lane) = c4;
        if ((lane & 3) == 0)
            *reinterpret_cast<int16_t*>(pub + 260 + 2 * (lane >> 2)) = (int16_t)s16;
        *reinterpret_cast<uint32_t*>(a.xq + L.rcodes + r * a.K + 256 * chunk + 4 * lane) = c4;
        const int j = lane >> 3;
        if ((lane & 7) == 0) {
            const int64_t bi = r * L.nb + 8 * chunk + j;
            reinterpret_cast<float*>(a.xq + L.rda)[bi] = d;
            reinterpret_cast<int32_t*>(a.xq + L.rs16)[bi] =
                (int32_t)(((uint32_t)s16 & 0xFFFFu) | ((uint32_t)s16o << 16));
            // the 32-code sum as two digits, S = 64 hi + lo
            const int S = s16 + s16o, at = 8 * (j >> 2) + (j & 3);
            const uint8_t lo = (uint8_t)(S & 63), hi = (uint8_t)((S >> 6) & 0xFF);
            uint8_t* sd = a.xq + L.rsd + task * 16 + at;
            sd[0] = lo;
            sd[4] = hi;
            if (L.gsd) {
                uint8_t* gs = a.xq + L.gsd + chunk * 256 + r * 16 + at;
                gs[0] = lo;
                gs[4] = hi;
            }
        }
        if (L.gcodes) {
            const int kg = (lane & 7) >> 1;
            *reinterpret_cast<uint32_t*>(a.xq + L.gcodes + chunk * 4096 + (j >> 1) * 1024 +
                                         (r + 16 * kg) * 16 + (j & 1) * 8 + 4 * (lane & 1)) = c4;
            if (lane == 0) reinterpret_cast<float*>(a.xq + L.gda)[chunk * 16 + r] = d;
        }
    }
}

// One workgroup per row; wave w takes the 256-element chunks w, w + waves,
// ..., V of them kept in registers (V = 0: any number, h read again for the
// second half).  With the ST_MFMA staging, workgroups past `rows` write the
// zero rows that fill its last group of 16.
template <int MODE, int V, class Layout>
__global__ __launch_bounds__(1024) void k_add_rmsnorm(NormArgs a, Layout L, int a16) {
    extern __shared__ double chunk_sum[];  // [ceil(K / 256)]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t r = a.row0 + blockIdx.x;
    const int chunks = (int)((a.K + 255) / 256);
    if constexpr (MODE == ST_MFMA) {
        if (r >= a.rows) {
            const int64_t g = r >> 4;
            const int m = (int)(r & 15);
            for (int64_t b = threadIdx.x; b < L.nb; b += blockDim.x) {
                const int64_t gb = g * L.nb + b;
#pragma unroll
                for (int kg = 0; kg < 4; kg++)
                    *reinterpret_cast<uint64_t*>(a.xq + L.codes + gb * 512 + (m + 16 * kg) * 8) = 0;
                reinterpret_cast<float*>(a.xq + L.da)[gb * 16 + m] = 0.0f;
                reinterpret_cast<float*>(a.xq + L.ca)[gb * 16 + m] = 0.0f;
                reinterpret_cast<int32_t*>(a.xq + L.S)[gb * 16 + m] = 0;
            }
            return;
        }
    }
    const float* xr = a.x + r * a.K;
    const float* rr = a.res ? a.res + r * a.K : nullptr;
    float* hr = a.h ? a.h + r * a.K : nullptr;
    float4 keep[V > 0 ? V : 1], weight[V > 0 ? V : 1];
    const int steps = V > 0 ? V : (chunks + waves - 1) / waves;
#pragma unroll
    for (int i = 0; i < (V > 0 ? V : 1); i++) keep[i] = weight[i] = make_float4(0, 0, 0, 0);
    const auto first = [&](int i, float4& v) {
        const int c = wave + i * waves;
        if (c >= chunks) return;  // uniform per wave
        const int64_t e = 256 * (int64_t)c + 4 * lane;
        v = make_float4(0, 0, 0, 0);
        if (e < a.K) {
            v = load4(xr + e, a16);
            if constexpr (V > 0) weight[i] = load4(a.w + e, a16);  // ahead of the sum
            if (rr) {
                v = add4(v, load4(rr + e, a16));
                store4(hr + e, v, a16);
            }
        }
        double s = (double)v.x * v.x + (double)v.y * v.y;
        s = s + (double)v.z * v.z;
        s = s + (double)v.w * v.w;
        s = sum64(s);
        if (lane == 0) chunk_sum[c] = s;
    };
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; i++) first(i, keep[i]);
    } else {
        for (int i = 0; i < steps; i++) first(i, keep[0]);
    }
    __syncthreads();
    double ss = 0.0;
    for (int c = 0; c < chunks; c++) ss += chunk_sum[c];
    const double rs = 1.0 / sqrt(ss / (double)a.K + (double)a.eps);
    const auto second = [&](int i, float4 v) {
        const int c = wave + i * waves;
        if (c >= chunks) return;  // uniform per wave
        const int64_t e = 256 * (int64_t)c + 4 * lane;
        const bool live = e < a.K;
        float4 y = make_float4(0, 0, 0, 0);
        if (live) {
            if constexpr (V == 0) v = load4(rr ? hr + e : xr + e, a16);
            const float4 w = V > 0 ? weight[V > 0 ? i : 0] : load4(a.w + e, a16);
            y.x = (float)(((double)v.x * rs) * (double)w.x);
            y.y = (float)(((double)v.y * rs) * (double)w.y);
            y.z = (float)(((double)v.z * rs) * (double)w.z);
            y.w = (float)(((double)v.w * rs) * (double)w.w);
            if (a.y) store4(a.y + r * a.K + e, y, a16);
        }
        quantise_chunk<MODE>(y, live, lane, c, r, a, L);
    };
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; i++) second(i, keep[i]);
    } else {
        for (int i = 0; i < steps; i++) second(i, keep[0]);
    }
}

template <int MODE, class Layout>
int launch_mode(NormArgs a, const Layout& L, int64_t grid, hipStream_t s) {
    const int chunks = (int)((a.K + 255) / 256);
    const int a16 = aligned16(a.x) && aligned16(a.w) && (!a.res || aligned16(a.res)) &&
                    (!a.h || aligned16(a.h)) && (!a.y || aligned16(a.y));
    const size_t lds = (size_t)chunks * 8;
    // Few rows: as many waves per row as there are chunks, for latency.  Many: two chunks a wave,
    // so that more rows share a CU and one's loads overlap another's sums (2048 rows of 4096: 31.7
    // us, 34.6 with one chunk a wave, 34.8 with four).
    int per = chunks <= 16 ? 1 : chunks <= 32 ? 2 : chunks <= 64 ? 4 : 0;
    if (a.rows >= 512 && per == 1 && chunks > 1) per = 2;
    const int waves = per ? (chunks + per - 1) / per : 16;
    constexpr int64_t SLICE = 1 << 21;  // a grid holds fewer than 2^32 threads
    for (a.row0 = 0; a.row0 < grid; a.row0 += SLICE) {
        const dim3 g((unsigned)(grid - a.row0 < SLICE ? grid - a.row0 : SLICE)), b(64 * waves);
        if (per == 1) hipLaunchKernelGGL((k_add_rmsnorm<MODE, 1, Layout>), g, b, lds, s, a, L, a16);
        else if (per == 2) hipLaunchKernelGGL((k_add_rmsnorm<MODE, 2, Layout>), g, b, lds, s, a, L, a16);
        else if (per == 4) hipLaunchKernelGGL((k_add_rmsnorm<MODE, 4, Layout>), g, b, lds, s, a, L, a16);
        else hipLaunchKernelGGL((k_add_rmsnorm<MODE, 0, Layout>), g, b, lds, s, a, L, a16);
        const int rc = (int)hipGetLastError();
        if (rc) return rc;
    }
    return 0;
}

}  // namespace

int launch_add_rmsnorm(const float* x, const float* res, const float* w, float eps, int64_t rows,
                       int64_t K, float* h, float* y, uint8_t* xq, bool q8k, hipStream_t s) {
    const NormArgs a{x, res, w, eps, rows, K, h, y, xq, 0};
    if (q8k) return launch_mode<0>(a, act_layout_q8k(rows, K), rows, s);
    const ActLayout L = act_layout(rows, K);
    switch (staging_for(rows, K)) {
    case ST_ROW: return launch_mode<ST_ROW>(a, L, rows, s);
    case ST_MFMA: return launch_mode<ST_MFMA>(a, L, 16 * L.G, s);
    default: return launch_mode<ST_F16>(a, L, rows, s);
    }
}

}  // namespace qmv
