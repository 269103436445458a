// Device pieces of inputs saved in 8 bits (mxint8_kernels.hip describes the format).
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"

namespace lora {

// The float 2^(s - 127) of a scale byte: s = 0 is the subnormal 2^-127, and s = 255
// a NaN (all the block's values then are).
__device__ __forceinline__ float i8_scale(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7FC00000u : max(s << 23, 0x00400000u));
}

// Four codes times their scale -> two words of bf16 pairs, exact.
__device__ __forceinline__ uint2 i8_expand4(uint32_t v, float unit) {
    const float a = (float)(int8_t)v, b = (float)(int8_t)(v >> 8), c = (float)(int8_t)(v >> 16), d = (float)((int32_t)v >> 24);
    return make_uint2(pack_bf16x2(a * unit, b * unit), pack_bf16x2(c * unit, d * unit));
}
__device__ __forceinline__ uint4 i8_expand(uint2 v, float unit) {
    const uint2 a = i8_expand4(v.x, unit), b = i8_expand4(v.y, unit);
    return make_uint4(a.x, a.y, b.x, b.y);
}

}  // namespace lora
