// wave.h -- sums and maxima over the 64 lanes of a wave, by DPP (no LDS): four
// steps within rows of 16 lanes, then row 0 into 1 and 2 into 3, then row 1 into
// 2 and 3; lane 63 holds the result, which every lane gets through a scalar
// register.  The order is fixed, so sums are run-to-run identical.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxk {

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;            // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;  // lane i <-> 7 - i, 15 - i
constexpr int kDppBcast15 = 0x142, kDppBcast31 = 0x143;
constexpr int kDppShr1 = 0x111, kDppShr2 = 0x112, kDppShr4 = 0x114, kDppShr8 = 0x118;   // lane i <- i - n of its row

// v of the lane that CTRL names; `old` where ROWS (a mask of rows of 16) or CTRL
// leaves a lane out.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float old, float v)
{
    return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(old), __float_as_uint(v)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp(double old, double v)
{
    const uint64_t o = (uint64_t)__double_as_longlong(old), x = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = dpp<CTRL, ROWS>((uint32_t)o, (uint32_t)x);
    const uint32_t hi = dpp<CTRL, ROWS>((uint32_t)(o >> 32), (uint32_t)(x >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ float from_lane(float v, int lane)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double from_lane(double v, int lane)
{
    const uint64_t x = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <class T>
__device__ __forceinline__ T wave_sum(T v)
{
    v += dpp<kDppXor1>(T(0), v);
    v += dpp<kDppXor2>(T(0), v);
    v += dpp<kDppHalfMirror>(T(0), v);
    v += dpp<kDppMirror>(T(0), v);
    v += dpp<kDppBcast15, 0xA>(T(0), v);
    v += dpp<kDppBcast31, 0xC>(T(0), v);
    return from_lane(v, 63);
}

// Each lane's sum of the lanes up to it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    v += dpp<kDppShr1>(0u, v);
    v += dpp<kDppShr2>(0u, v);
    v += dpp<kDppShr4>(0u, v);
    v += dpp<kDppShr8>(0u, v);
    v += dpp<kDppBcast15, 0xA>(0u, v);
    return v + dpp<kDppBcast31, 0xC>(0u, v);
}

__device__ __forceinline__ float max_of(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return __builtin_fmax(a, b); }

// Of values without NaN.
template <class T>
__device__ __forceinline__ T wave_max(T v)
{
    v = max_of(v, dpp<kDppXor1>(v, v));
    v = max_of(v, dpp<kDppXor2>(v, v));
    v = max_of(v, dpp<kDppHalfMirror>(v, v));
    v = max_of(v, dpp<kDppMirror>(v, v));
    v = max_of(v, dpp<kDppBcast15, 0xA>(v, v));
    v = max_of(v, dpp<kDppBcast31, 0xC>(v, v));
    return from_lane(v, 63);
}

// The same over each row of 16 lanes, in every lane of it.
template <class T>
__device__ __forceinline__ T row_sum(T v)
{
    v += dpp<kDppXor1>(T(0), v);
    v += dpp<kDppXor2>(T(0), v);
    v += dpp<kDppHalfMirror>(T(0), v);
    v += dpp<kDppMirror>(T(0), v);
    return v;
}
template <class T>
__device__ __forceinline__ T row_max(T v)
{
    v = max_of(v, dpp<kDppXor1>(v, v));
    v = max_of(v, dpp<kDppXor2>(v, v));
    v = max_of(v, dpp<kDppHalfMirror>(v, v));
    v = max_of(v, dpp<kDppMirror>(v, v));
    return v;
}

// Of unsigned numbers (0 is neutral, which lets each step be one instruction).
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max_u32(v, dpp<kDppXor1>(0u, v));
    v = max_u32(v, dpp<kDppXor2>(0u, v));
    v = max_u32(v, dpp<kDppHalfMirror>(0u, v));
    return max_u32(v, dpp<kDppMirror>(0u, v));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max_u32(v, dpp<kDppXor1>(0u, v));
    v = max_u32(v, dpp<kDppXor2>(0u, v));
    v = max_u32(v, dpp<kDppHalfMirror>(0u, v));
    v = max_u32(v, dpp<kDppMirror>(0u, v));
    v = max_u32(v, dpp<kDppBcast15, 0xA>(0u, v));
    v = max_u32(v, dpp<kDppBcast31, 0xC>(0u, v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

}  // namespace mxk
