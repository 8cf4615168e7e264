// Helpers shared by the router, dispatch and combine kernels (gfx950).
//
// Wave-wide reductions run on the data-parallel-primitive lane shifts (a
// shift within rows of 16, then row broadcasts): six VALU instructions whose
// order is fixed, so a sum is the same in every run.  The result is read from
// lane 63 into a scalar register.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace bsq {

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float old, float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), CTRL, ROWS, 0xF, false));
}

__device__ __forceinline__ float lane63(float x) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

__device__ __forceinline__ float wave_max_f32(float x) {
    x = fmaxf(x, dpp_f32<0x111, 0xF>(x, x));
    x = fmaxf(x, dpp_f32<0x112, 0xF>(x, x));
    x = fmaxf(x, dpp_f32<0x114, 0xF>(x, x));
    x = fmaxf(x, dpp_f32<0x118, 0xF>(x, x));
    x = fmaxf(x, dpp_f32<0x142, 0xA>(x, x));
    x = fmaxf(x, dpp_f32<0x143, 0xC>(x, x));
    return lane63(x);
}

__device__ __forceinline__ float wave_sum_f32(float x) {
    x += dpp_f32<0x111, 0xF>(0.0f, x);
    x += dpp_f32<0x112, 0xF>(0.0f, x);
    x += dpp_f32<0x114, 0xF>(0.0f, x);
    x += dpp_f32<0x118, 0xF>(0.0f, x);
    x += dpp_f32<0x142, 0xA>(0.0f, x);
    x += dpp_f32<0x143, 0xC>(0.0f, x);
    return lane63(x);
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
