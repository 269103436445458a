// Device pieces that the products over an MXFP4 weight share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "device_common.hpp"

namespace lora {

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// The float 2^(s - 127) of a scale byte: s = 0 is the subnormal 2^-127, and
// s = 255 an infinity (the conversions then give NaN for every code).
__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(max(s << 23, 0x00400000u)); }

// Byte e of a dword of codes -> two bf16, exact; all four -> an MFMA operand.
__device__ __forceinline__ uint32_t mx_pair(uint32_t w, float scale, int e) {
    return __builtin_bit_cast(uint32_t, e == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)
                                        : e == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)
                                        : e == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)
                                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
}
__device__ __forceinline__ uint4 mx_frag(uint32_t w, float scale) {
    return make_uint4(mx_pair(w, scale, 0), mx_pair(w, scale, 1), mx_pair(w, scale, 2), mx_pair(w, scale, 3));
}

// Vector memory down to N loads in flight, and no LDS read in flight.
template <int N>
__device__ __forceinline__ void wait_vmcnt_lds() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

// dma16 with a scalar byte offset added to the address; a lane whose own
// offset is kOOB reads zeros whatever it is.
__device__ __forceinline__ void dma16_at(sgpr4_t desc, uint32_t voff, uint32_t soff, uint32_t lds_base) {
    uint32_t saved_m0;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %4\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved_m0)
        : "v"(voff), "s"(desc), "s"(soff), "s"(lds_base)
        : "memory");
}

// Work-groups of one XCD (id mod 8) take a contiguous run of `total` ids.
__device__ __forceinline__ int xcd_order(int id, int total) {
    const int xcd = id & 7, local = id >> 3, each = total >> 3, rem = total & 7;
    return xcd * each + min(xcd, rem) + local;
}

// Lets `fn` use `bytes` of dynamic LDS, once a device.
inline hipError_t allow_lds(const void *fn, size_t bytes, std::atomic<uint64_t> &done) {
    if (bytes <= 64 * 1024) return hipSuccess;
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    (void)hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    done.fetch_or(bit, std::memory_order_relaxed);
    return hipSuccess;
}

// Microseconds of expanding a weight of `values` and of the bf16 product over it,
// of m x out with a contraction of `depth`: two launches of 3 us, 2.53 bytes a
// value at 6 TB/s, and rounds of 256 256 x 256 tiles that take 1.4 us for 64 of
// the depth (1.1 where half of the CUs or fewer have one).  Measured, model in
// brackets: 1 x 4096 x 4096 85 (84), 2000 x 4096 x 4096 86 (84), 8192 x 4096 x 4096
// 201 (192), 16 x 4096 x 14336 (dX) 265 (277), 2000 x 8192 x 28672 (dX) 738 (732).
inline double expanded_us(int64_t m, int64_t out, int64_t depth, double values) {
    const int64_t tiles = ((m + 255) / 256) * ((out + 255) / 256);
    return 6.0 + values * 2.53 / 6e6 + (double)((tiles + 255) / 256 * ((depth + 63) / 64)) * (tiles <= 128 ? 1.1 : 1.4);
}

// Microseconds of `groups` work-groups, `slots` at a time, of which each takes `one`
// and all read the weight's packed bytes once at 6 TB/s between them.
inline double rounds_us(int64_t groups, int64_t slots, double one, double values) {
    const int64_t full = groups / slots, rest = groups % slots;
    const double each = values * 0.53 / 6e6 / (double)groups;
    return (double)full * std::max(one, each * (double)slots) + (rest > 0 ? std::max(one, each * (double)rest) : 0.0);
}

// `find`'s answers for the shapes a thread asked for last (a plan takes a few
// microseconds to find, a call asks twice, and a program's shapes come back).
template <class Plan, class Find>
Plan remembered(int64_t m, int64_t k, int64_t n, int64_t tag, Find find) {
    struct Known {
        int64_t m, k, n, tag;
        Plan plan;
    };
    thread_local Known known[64] = {};
    const uint64_t h = ((uint64_t)m * 0x9E3779B97F4A7C15ull) ^ ((uint64_t)k * 0xC2B2AE3D27D4EB4Full) ^
                       ((uint64_t)n * 0x165667B19E3779F9ull) ^ ((uint64_t)tag * 0x27D4EB2F165667C5ull);
    Known &e = known[(h >> 40) & 63];
    if (e.m != m || e.k != k || e.n != n || e.tag != tag || m == 0) e = Known{m, k, n, tag, find()};
    return e.plan;
}

}  // namespace lora
