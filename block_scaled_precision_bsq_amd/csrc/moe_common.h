// Helpers shared by the router, dispatch and combine kernels (gfx950).
//
// Wave-wide reductions run on the data-parallel-primitive lane moves: four
// rotations within rows of 16, each one instruction with its operation, then
// the swaps of 16 and of 32 lanes.  Every lane ends with the result, in an
// order that is the same in every run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace bsq {

// One step of a row's rotation: op(x, x rotated by N lanes).  fmaxf would quiet
// its operands first, hence the instruction itself, with the two wait states
// between the write of x and its move.
template <int N>
__device__ __forceinline__ float ror_max_f32(float x) {
    float r;
    asm("s_nop 1\n\tv_max_f32_dpp %0, %1, %1 row_ror:%2 row_mask:0xf bank_mask:0xf" : "=v"(r) : "v"(x), "n"(N));
    return r;
}
template <int N>
__device__ __forceinline__ float ror_add_f32(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xF, 0xF, true));
}

// x of the lane 16 (32) away within each 32 (64), with the lane's own: {x, y} in
// either order.
struct Pair32 {
    uint32_t a, b;
};
__device__ __forceinline__ Pair32 swap16(uint32_t x) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return {r[0], r[1]};
}
__device__ __forceinline__ Pair32 swap32(uint32_t x) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return {r[0], r[1]};
}

// fmaxf of values that are no NaN (without the quieting that fmaxf adds).
__device__ __forceinline__ float max_num(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

__device__ __forceinline__ float wave_max_f32(float x) {
    x = ror_max_f32<1>(ror_max_f32<2>(ror_max_f32<4>(ror_max_f32<8>(x))));
    Pair32 p = swap16(__float_as_uint(x));
    x = max_num(__uint_as_float(p.a), __uint_as_float(p.b));
    p = swap32(__float_as_uint(x));
    return max_num(__uint_as_float(p.a), __uint_as_float(p.b));
}

// Sum of the lane's row of 16.
__device__ __forceinline__ float row_sum_f32(float x) {
    return ror_add_f32<1>(ror_add_f32<2>(ror_add_f32<4>(ror_add_f32<8>(x))));
}

__device__ __forceinline__ float wave_sum_f32(float x) {
    x = row_sum_f32(x);
    Pair32 p = swap16(__float_as_uint(x));
    x = __uint_as_float(p.a) + __uint_as_float(p.b);
    p = swap32(__float_as_uint(x));
    return __uint_as_float(p.a) + __uint_as_float(p.b);
}

// (By shifts and row broadcasts to lane 63, whose identity lets the compiler
// make each step one instruction: 8 instructions less than by rotations.)
__device__ __forceinline__ int wave_max_i32(int x) {
    constexpr int LOWEST = -0x7FFFFFFF - 1;
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x111, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x112, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x114, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x118, 0xF, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x142, 0xA, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(LOWEST, x, 0x143, 0xC, 0xF, false));
    return __builtin_amdgcn_readlane(x, 63);
}

// e^x for x <= 0 from the hardware's 2^y: x log2(e) in two binary32 parts, the
// second one applied to first order, so the error stays at about 2 ulps for
// any x; results below the normal range are 0.
__device__ __forceinline__ float exp_neg(float x) {
    x = max_num(x, -200.0f);  // (0 from -104 on; -inf has no remainder)
    const float y = x * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596e-8
    const float lo = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -y));
    const float r = __builtin_amdgcn_exp2f(y);
    return fmaf(r, lo * 0.693147182f, r);
}

// Inclusive prefix sum over the wave's lanes.
__device__ __forceinline__ int wave_scan_i32(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

__device__ __forceinline__ float bits_bf16(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t bf16_rne(float x) { return (uint16_t)pack_bf16x2(x, 0.0f); }

}  // namespace bsq
