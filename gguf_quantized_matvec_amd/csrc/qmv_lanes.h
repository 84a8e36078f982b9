// Reductions over the lanes of a wave without LDS: DPP within 16 lanes, the
// row swaps of gfx950 beyond.  Each step combines a lane's value with that of
// lane ^ 1, ^ 2, ^ 4, ...; from the third on the other value is fetched by a
// mirror or a swap, which is the same once the lanes of a group agree.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {
namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_bits(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false);
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E;          // quad permutations
constexpr int DPP_MIRROR8 = 0x141, DPP_MIRROR16 = 0x140;  // xor 4, xor 8 of agreeing lanes
constexpr int DPP_ROR8 = 0x128;                           // xor 8

template <int CTRL> __device__ __forceinline__ float dpp(float x) {
    return __uint_as_float(dpp_bits<CTRL>(__float_as_uint(x)));
}
template <int CTRL> __device__ __forceinline__ int dpp(int x) {
    return (int)dpp_bits<CTRL>((uint32_t)x);
}
template <int CTRL> __device__ __forceinline__ double dpp(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint64_t r = dpp_bits<CTRL>((uint32_t)b) | (uint64_t)dpp_bits<CTRL>((uint32_t)(b >> 32)) << 32;
    return __longlong_as_double((long long)r);
}

// The two values that the lanes of rows (or halves) xor 16 (32) hold.
struct Two {
    uint32_t a, b;
};
__device__ __forceinline__ Two both16(uint32_t x) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return Two{r[0], r[1]};
}
__device__ __forceinline__ Two both32(uint32_t x) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return Two{r[0], r[1]};
}

// Of values that agree within 16 lanes (or any lanes 16 and 32 apart): the sum
// and the maximum over lanes ^ 16, then ^ 32.
__device__ __forceinline__ float sum_rows(float x) {
    Two t = both16(__float_as_uint(x));
    x = __uint_as_float(t.a) + __uint_as_float(t.b);
    t = both32(__float_as_uint(x));
    return __uint_as_float(t.a) + __uint_as_float(t.b);
}
__device__ __forceinline__ float max_rows(float x) {
    Two t = both16(__float_as_uint(x));
    x = fmaxf(__uint_as_float(t.a), __uint_as_float(t.b));
    t = both32(__float_as_uint(x));
    return fmaxf(__uint_as_float(t.a), __uint_as_float(t.b));
}

__device__ __forceinline__ float max8(float x) {
    x = fmaxf(x, dpp<DPP_XOR1>(x));
    x = fmaxf(x, dpp<DPP_XOR2>(x));
    return fmaxf(x, dpp<DPP_MIRROR8>(x));
}
__device__ __forceinline__ float max64(float x) {
    x = max8(x);
    return max_rows(fmaxf(x, dpp<DPP_MIRROR16>(x)));
}
__device__ __forceinline__ double sum64(double x) {
    x += dpp<DPP_XOR1>(x);
    x += dpp<DPP_XOR2>(x);
    x += dpp<DPP_MIRROR8>(x);
    x += dpp<DPP_MIRROR16>(x);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint64_t b = (uint64_t)__double_as_longlong(x);
        const Two lo = i ? both32((uint32_t)b) : both16((uint32_t)b);
        const Two hi = i ? both32((uint32_t)(b >> 32)) : both16((uint32_t)(b >> 32));
        x = __longlong_as_double((long long)(lo.a | (uint64_t)hi.a << 32)) +
            __longlong_as_double((long long)(lo.b | (uint64_t)hi.b << 32));
    }
    return x;
}

}  // namespace
}  // namespace qmv
