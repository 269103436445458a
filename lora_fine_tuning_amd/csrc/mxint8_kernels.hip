// A layer's input saved in 8 bits for the backward (MXINT8): 8-bit integers in
// blocks of 32 along each row, one power-of-two scale byte per block.
//
//   X'[i][32b + j] = c * 2^(s - 127),  c in -127 .. 127
//
// With a the block's largest magnitude the scale is 2^e, e = floor(log2 a) - 6, so
// that a / 2^e lies in [64, 128), and c = x / 2^e rounded to the nearest (ties to
// even).  Every X' is exactly a bf16 (seven bits and a sign), so the backward's
// products over X' are those over a bf16 input; and since a bf16 has eight
// significant bits, a / 2^e is at most 127.5: no value is off by more than half a
// step, 2^(e - 1).
//
// Storage: codes (m, KB, 32) int8 and scales (m, KB) bytes, KB = 4 ceil(k / 128),
// so that rows are whole cache lines of codes and whole words of scales.  Padding
// holds zero codes and scale bytes of 127.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "launch.hpp"
#include "mxint8.hpp"

namespace lora {

namespace {

constexpr int kUnroll = 4;                       // pieces of 8 values a lane
constexpr int kWaveValues = 64 * 8 * kUnroll;    // of one row

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

struct I8Shape {
    int64_t m, k;
    int64_t kb;      // blocks of a row
    int64_t chunks;  // waves a row takes
};

// Value of `v` in the lane whose number differs in bit 0 (or 1), and in the lane
// 4 (or 8) further in the row of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;

// Two bf16 over 2^e, rounded to integers: the low byte of each result.  Adding
// 1.5 * 2^23 leaves the nearest integer (ties to even) in the low bits.
__device__ __forceinline__ void codes_of(uint32_t pair, float unit, uint32_t &lo, uint32_t &hi) {
    const float a = __builtin_amdgcn_fmed3f(__uint_as_float(pair << 16) * unit, -127.f, 127.f);
    const float b = __builtin_amdgcn_fmed3f(__uint_as_float(pair & 0xFFFF0000u) * unit, -127.f, 127.f);
    lo = __float_as_uint(a + 12582912.f);
    hi = __float_as_uint(b + 12582912.f);
}
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), cd = __builtin_amdgcn_perm(d, c, 0x0C0C0400u);
    return __builtin_amdgcn_perm(cd, ab, 0x05040100u);
}

// A wave takes 2048 values of a row, a lane 8 at a time (four lanes a block), all
// loads before the first use.  Bound by HBM: 2 bytes in, 1.03 out a value; 8192 x 14336
// 54 us after 512 MiB of reads (6.6 TB/s), 78 right after a kernel that wrote 235 MB, whose
// lines go back to memory beside it (4.6 TB/s); read back 56 us (6.4 TB/s, the codes partly
// out of the last cache).
__global__ __launch_bounds__(256) void mxint8_quantize_kernel(const uint16_t *X, I8Shape S, uint8_t *codes, uint8_t *scales) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = S.m * S.chunks;
    for (int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); w < waves;
         w += (int64_t)gridDim.x * 4) {
        const int64_t row = w / S.chunks, c0 = (w - row * S.chunks) * kWaveValues + lane * 8;
        const uint16_t *src = X + row * S.k;
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + 512 * u;
            v[u] = c < S.k ? *(const uint4 *)(src + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            // bf16 magnitudes order as their bit patterns
            u16x2_t top = __builtin_bit_cast(u16x2_t, v[u].x & 0x7FFF7FFFu);
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[u].y & 0x7FFF7FFFu));
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[u].z & 0x7FFF7FFFu));
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, v[u].w & 0x7FFF7FFFu));
            uint32_t b = max((uint32_t)top[0], (uint32_t)top[1]);
            b = max(b, dpp<kXor1>(b));
            b = max(b, dpp<kXor2>(b));
            // exponent field E: 2^(E - 127) <= a, so s = E - 6.  The clamp keeps every
            // X' a normal bf16 (values below 2^-121 become zero).
            uint32_t s = max(b >> 7, 13u) - 6u;
            if (b == 0u) s = 127u;
            const bool bad = b >= 0x7F80u;  // an infinity or NaN: the whole block becomes NaN
            const float unit = bad ? 0.f : __uint_as_float((254u - s) << 23);
            uint32_t q[8];
            codes_of(v[u].x, unit, q[0], q[1]);
            codes_of(v[u].y, unit, q[2], q[3]);
            codes_of(v[u].z, unit, q[4], q[5]);
            codes_of(v[u].w, unit, q[6], q[7]);
            uint2 out = make_uint2(low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7]));
            if (bad) out = make_uint2(0u, 0u), s = 255u;
            // four blocks' bytes in one word
            uint32_t word = s << (8 * ((lane >> 2) & 3));
            word |= dpp<kRor4>(word);
            word |= dpp<kRor8>(word);
            const int64_t c = c0 + 512 * u;
            if (c < S.kb * 32) {
                *(uint2 *)(codes + row * S.kb * 32 + c) = out;
                if ((lane & 15) == 0) *(uint32_t *)(scales + row * S.kb + (c >> 5)) = word;
            }
        }
    }
}

__global__ __launch_bounds__(256) void mxint8_dequantize_kernel(const uint8_t *codes, const uint8_t *scales, I8Shape S, uint16_t *X) {
    const int lane = threadIdx.x & 63;
    const int64_t waves = S.m * S.chunks;
    for (int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); w < waves;
         w += (int64_t)gridDim.x * 4) {
        const int64_t row = w / S.chunks, c0 = (w - row * S.chunks) * kWaveValues + lane * 8;
        uint2 v[kUnroll];
        uint32_t s[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + 512 * u;
            const bool live = c < S.k;
            v[u] = live ? *(const uint2 *)(codes + row * S.kb * 32 + c) : make_uint2(0u, 0u);
            s[u] = live ? scales[row * S.kb + (c >> 5)] : 127u;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t c = c0 + 512 * u;
            const float unit = i8_scale(s[u]);
            if (c < S.k) *(uint4 *)(X + row * S.k + c) = i8_expand(v[u], unit);
        }
    }
}

__global__ __launch_bounds__(256) void widen_rows_kernel(WidenRows P, int64_t s_items, int64_t a_items, int64_t items) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        if (i < s_items) {
            const int64_t y = i / (P.row / 4);
            const int c = (int)(i - y * (P.row / 4)) * 4;
            const float *src = P.S + y * P.r + c;
            ((float4 *)P.S_out)[i] = make_float4(c < P.r ? src[0] : 0.f, c + 1 < P.r ? src[1] : 0.f, c + 2 < P.r ? src[2] : 0.f,
                                                 c + 3 < P.r ? src[3] : 0.f);
        } else if (i < s_items + a_items) {
            const int64_t at = i - s_items, y = at / (P.row / 4);
            const int c = (int)(at - y * (P.row / 4)) * 4;
            const uint16_t *src = (const uint16_t *)P.A + y * P.r + c;
            const uint32_t v0 = c < P.r ? src[0] : 0u, v1 = c + 1 < P.r ? src[1] : 0u, v2 = c + 2 < P.r ? src[2] : 0u,
                           v3 = c + 3 < P.r ? src[3] : 0u;
            ((uint2 *)P.A_out)[at] = make_uint2(v0 | v1 << 16, v2 | v3 << 16);
        } else {
            const int64_t at = i - s_items - a_items, y = at / (P.keep_row / 4);
            const int c = (int)(at - y * (P.keep_row / 4)) * 4;
            const uint32_t *src = P.keep + y * P.kw + c;
            ((uint4 *)P.keep_out)[at] =
                make_uint4(c < P.kw ? src[0] : 0u, c + 1 < P.kw ? src[1] : 0u, c + 2 < P.kw ? src[2] : 0u, c + 3 < P.kw ? src[3] : 0u);
        }
    }
}

I8Shape i8_shape(int64_t m, int64_t k) { return I8Shape{m, k, i8_blocks(k), (i8_blocks(k) * 32 + kWaveValues - 1) / kWaveValues}; }

unsigned i8_grid(const I8Shape &s) { return (unsigned)std::min<int64_t>((s.m * s.chunks + 3) / 4, 1 << 20); }

}  // namespace

hipError_t launch_mxint8_quantize(const void *X, int64_t m, int64_t k, void *codes, void *scales, hipStream_t stream) {
    const I8Shape s = i8_shape(m, k);
    const int slot = prof_begin("mxint8_quantize", stream);
    hipLaunchKernelGGL(mxint8_quantize_kernel, dim3(i8_grid(s)), dim3(256), 0, stream, (const uint16_t *)X, s, (uint8_t *)codes,
                       (uint8_t *)scales);
    prof_end(slot, stream);
    return hipGetLastError();
}

hipError_t launch_mxint8_dequantize(const void *codes, const void *scales, int64_t m, int64_t k, void *X, hipStream_t stream) {
    const I8Shape s = i8_shape(m, k);
    const int slot = prof_begin("mxint8_dequantize", stream);
    hipLaunchKernelGGL(mxint8_dequantize_kernel, dim3(i8_grid(s)), dim3(256), 0, stream, (const uint8_t *)codes,
                       (const uint8_t *)scales, s, (uint16_t *)X);
    prof_end(slot, stream);
    return hipGetLastError();
}

hipError_t launch_widen_rows(const WidenRows &w, hipStream_t stream) {
    const int64_t s = w.S_out ? w.m * (w.row / 4) : 0, a = w.A_out ? w.k * (w.row / 4) : 0;
    const int64_t items = s + a + (w.keep_out ? w.m * (w.keep_row / 4) : 0);
    const int slot = prof_begin("widen_rows", stream);
    hipLaunchKernelGGL(widen_rows_kernel, dim3((unsigned)std::min<int64_t>((items + 255) / 256, 1 << 20)), dim3(256), 0, stream, w, s, a, items);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
