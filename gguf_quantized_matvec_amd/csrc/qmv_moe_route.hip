// Routing of tokens to experts for gfx950: scores, a bias for balance, groups
// of experts, the best `top` of what is left, and their weights.
//
//   s_e  softmax or sigmoid of the token's logits (f64)
//   c_e  what experts are chosen by: fl(fl(s_e) + bias_e) in f32 (without a
//        bias fl(s_e)); for a softmax without a bias, whose groups go by their
//        largest member, the logit itself: the softmax keeps the logits' order
//        and rounding it would only make ties
//   w_e  scale * s_e / (renorm ? the chosen experts' sum of s : 1)
//
// The choice is a whole number next to a border, so s is computed in f64 and
// rounded once: two ways of computing it agree but for one value in 2^29.
//
// One wave a token, experts lane + 64 i in registers.  The top experts come
// from `top` rounds of a maximum over the wave; a softmax that is
// renormalised needs an exponential for the chosen experts only.  What bounds it
// is the chain of those rounds: 3.3 us for one token of 64 experts, 12.2 for 8192
// of 128 (390 GB/s), 8.3 for 64 of 256 in 8 groups with a sigmoid in f64; a call
// is 9 to 10 us of the host's time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmv_lanes.h"
#include "qmv_moe.h"

namespace qmv {
namespace {

constexpr float NONE = -__builtin_inff();   // the choice of an expert that is not available

__device__ __forceinline__ int min64(int x) {
    x = min(x, dpp<DPP_XOR1>(x));
    x = min(x, dpp<DPP_XOR2>(x));
    x = min(x, dpp<DPP_MIRROR8>(x));
    x = min(x, dpp<DPP_MIRROR16>(x));
    Two t = both16((uint32_t)x);
    x = min((int)t.a, (int)t.b);
    t = both32((uint32_t)x);
    return min((int)t.a, (int)t.b);
}

__device__ __forceinline__ float lane_float(float x, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

constexpr int WAVES = 4;

// V: experts a lane.
template <int V>
__global__ __launch_bounds__(64 * WAVES) void k_moe_route(RouteArgs a) {
    extern __shared__ float lds[];      // [WAVES][E] choices, only with groups
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * WAVES + wv;
    if (t >= a.T) return;               // waves work alone: no barrier below
    const int E = a.E;
    const float* row = a.logits + t * E;
    float logit[V], choice[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = lane + 64 * i;
        logit[i] = e < E ? row[e] : NONE;
        if (!(logit[i] > NONE)) logit[i] = NONE;   // NaN: not available
    }
    // softmax: exp(l - m), 1 for the largest also where that is infinite
    float m = NONE;
#pragma unroll
    for (int i = 0; i < V; i++) m = fmaxf(m, logit[i]);
    m = max64(m);
    auto part = [&](float l) -> double {
        return l == m ? 1.0 : exp((double)l - (double)m);
    };
    const bool by_logit = !a.sigmoid && !a.bias && (a.groups == 1 || a.group_top == 1);
    double total = 1.0;
    if (!a.sigmoid && !(by_logit && a.renorm)) {
        total = 0.0;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (logit[i] > NONE) total += part(logit[i]);
        total = sum64(total);
    }
    auto score = [&](float l) -> double {
        if (!a.sigmoid) return part(l) / total;
        // exp(-l) ends at 709.78; there the sigmoid is exp(l), a subnormal number
        const bool low = l < -709.0f;
        const double t = exp(low ? (double)l : -(double)l);
        return low ? t : 1.0 / (1.0 + t);
    };
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = lane + 64 * i;
        choice[i] = logit[i];
        if (!by_logit && logit[i] > NONE) {
            choice[i] = (float)score(logit[i]);
            if (a.bias) {
                const float b = a.bias[e];
                choice[i] = b > NONE ? choice[i] + b : NONE;
            }
        }
    }
    if (a.groups > 1) {
        // the choices meet in LDS; lane g ranks group g
        float* c = lds + wv * E;
        const int G = a.groups, size = E / G;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (lane + 64 * i < E) c[lane + 64 * i] = choice[i];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        float first = NONE, second = NONE;
        if (lane < G) {
            for (int j = 0; j < size; j++) {
                const float v = c[lane * size + j];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        }
        const float rank = a.group_top == 2 && second > NONE ? first + second : first;
        int before = 0;
        for (int g = 0; g < G; g++) {
            const float r = lane_float(rank, g);
            before += r > rank || (r == rank && g < lane);
        }
        const uint64_t stay = __builtin_amdgcn_ballot_w64(lane < G && before < a.top_groups);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int e = lane + 64 * i;
            if (e < E && !(stay >> (e / size) & 1)) choice[i] = NONE;
        }
    }
    // `top` rounds: the largest choice, of equals the lowest expert
    int mine = -1;          // lane j: the expert of slot j
    float mine_logit = NONE;
    for (int j = 0; j < a.top; j++) {
        float best = choice[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; i++)
            if (choice[i] > best) { best = choice[i]; at = i; }
        const float top = max64(best);
        if (!(top > NONE)) break;
        const int e = min64(best == top ? lane + 64 * at : INT32_MAX);
        const int owner = e & 63, slot = e >> 6;
        float l = logit[0];
#pragma unroll
        for (int i = 1; i < V; i++)
            if (slot == i) l = logit[i];
        l = lane_float(l, owner);
#pragma unroll
        for (int i = 0; i < V; i++)
            if (lane == owner && slot == i) choice[i] = NONE;
        if (lane == j) { mine = e; mine_logit = l; }
    }
    double w = mine >= 0 ? score(mine_logit) : 0.0;
    if (a.renorm) {
        const double sum = sum64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < a.top) {
        a.idx[t * a.top + lane] = mine;
        a.weight[t * a.top + lane] = (float)(w * (double)a.scale);
    }
}

template <int V> int launch_route(const RouteArgs& a, hipStream_t s) {
    const size_t lds = a.groups > 1 ? (size_t)WAVES * a.E * 4 : 0;
    hipLaunchKernelGGL(k_moe_route<V>, dim3((unsigned)((a.T + WAVES - 1) / WAVES)),
                       dim3(64 * WAVES), lds, s, a);
    return (int)hipGetLastError();
}

}  // namespace

int launch_moe_route(const RouteArgs& a, hipStream_t s) {
    if (a.E <= 64) return launch_route<1>(a, s);
    if (a.E <= 128) return launch_route<2>(a, s);
    if (a.E <= 256) return launch_route<4>(a, s);
    if (a.E <= 512) return launch_route<8>(a, s);
    return launch_route<16>(a, s);
}

}  // namespace qmv
