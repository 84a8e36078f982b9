// Device code that the experts' kernels share: what the bit-identity of their
// results rests on (the types' layouts, the Q8_0 quantisation, the SwiGLU) and
// a few helpers.
//
// Built with -ffp-contract=off: every float operation is the one written.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <numeric>
#include <type_traits>
#include <utility>

namespace qmv {
namespace {

constexpr int T_Q4_0 = 2, T_Q4_1 = 3, T_Q5_0 = 6, T_Q5_1 = 7, T_Q8_0 = 8, T_Q8_1 = 9,
              T_Q4_K = 12, T_Q6_K = 14;

// Elements and bytes of a block.
constexpr int block_elements(int type) { return type == T_Q4_K || type == T_Q6_K ? 256 : 32; }
constexpr int block_bytes(int type) {
    return type == T_Q8_0 ? 34 : type == T_Q4_0 ? 18 : type == T_Q5_0 ? 22 : type == T_Q4_1 ? 20
         : type == T_Q5_1 ? 24 : type == T_Q8_1 ? 36 : type == T_Q4_K ? 144 : 210;
}
// QK, BB: elements and bytes of a block; CB: bytes of a chunk of 256 elements.
template <int FMT> struct Fmt {
    static constexpr int QK = block_elements(FMT), BB = block_bytes(FMT), CB = 256 / QK * BB;
};
// The block term has a second part, a minimum times the activation codes' sum.
constexpr bool type_has_min(int type) { return type == T_Q4_K || type == T_Q4_1 || type == T_Q5_1; }
template <int FMT> constexpr bool has_min() { return type_has_min(FMT); }

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ float half_bits(uint32_t h) {
    const uint16_t u = (uint16_t)h;
    _Float16 f;
    __builtin_memcpy(&f, &u, 2);
    return (float)f;
}
template <class Fn, int... Is>
__device__ __forceinline__ void each_of(Fn&& f, std::integer_sequence<int, Is...>) {
    (f(std::integral_constant<int, Is>{}), ...);
}
// f(0), f(1), ... f(N - 1) with constants
template <int N, class Fn> __device__ __forceinline__ void each(Fn&& f) {
    each_of(f, std::make_integer_sequence<int, N>{});
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// silu(g) u in f64 as t = exp(-g), s = g / (1 + t), s u, rounded once.
__device__ __forceinline__ float swiglu(float g, float u) {
    const double gd = (double)g;
    const double s = gd / (1.0 + exp(-gd));
    return (float)(s * (double)u);
}
// Fifth bits: bit j of the nibble h at bit 0 of byte j.  h * 0x204081 holds
// copies of h at bits 0, 7, 14 and 21, without carries.
__device__ __forceinline__ uint32_t spread(uint32_t h) {
    return __umul24(h & 15u, 0x204081u) & 0x01010101u;
}

// A Q8_0 block of activations over 8 lanes, 4 elements each; all 8 call.
// quantise_block: the scale, and the lane's codes in c (0 before), from its
// elements at x (live false: from zeros), as quantize_act_q8_0 gives them.
// read_block: the same from the block, sub the lane's number among the 8.
__device__ __forceinline__ _Float16 quantise_block(const float* x, bool live, bool a16, uint32_t& c) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) {
        if (a16) {   // x is 16-byte aligned
            const float4 f = *reinterpret_cast<const float4*>(x);
            v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = x[i];
        }
    }
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    const float q = amax / 127.0f;
    const float r = 1.0f / q, id = __builtin_isinf(r) ? 0.0f : r;
#pragma unroll
    for (int i = 0; i < 4; i++) c |= ((uint32_t)(int)roundf(v[i] * id) & 0xFFu) << (8 * i);
    return (_Float16)q;
}
__device__ __forceinline__ _Float16 read_block(const uint8_t* block, int sub, uint32_t& c) {
    const uint16_t* in = reinterpret_cast<const uint16_t*>(block);
    c = (uint32_t)in[1 + 2 * sub] | ((uint32_t)in[2 + 2 * sub] << 16);
    _Float16 d;
    __builtin_memcpy(&d, in, 2);
    return d;
}
// The sum of the block's 32 codes.
__device__ __forceinline__ int block_sum(uint32_t c) {
    int S = __builtin_amdgcn_sdot4((int)c, 0x01010101, 0, false);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) S += __shfl_xor(S, o);
    return S;
}

// The matrix-vector kernel's codes with an offset are formed as a power of two
// times (code - offset), whose int8 bits are a shift and a flipped top bit away;
// the power leaves with the activation scale, exactly.
constexpr float gemv_scale_back(int type) {
    return type == T_Q4_0 ? 1.0f / 16 : type == T_Q5_0 ? 1.0f / 8 : type == T_Q6_K ? 1.0f / 4 : 1.0f;
}

}  // namespace
}  // namespace qmv
