// Frozen weights held as 4-bit integers in groups of rows:
//
//   W'[i][j] = s (q - z),  q in 0 .. 15, one scale s and zero z for `group` rows of a column
//
// Storage (N16 = ceil(n / 16), K128 = ceil(k / 128)): codes [N16][K128][4][16][16]
// bytes; word d of the 16 bytes of (c, t, g, j) holds rows 128t + 32d + 8g .. +7 of
// column 16c + j, the even rows in its low four nibbles and the odd ones in its high
// four.  A wave's 16-byte load of one (c, t) is 1 KiB in a row; word d of lane (g, l)
// is then a matrix operand of the 32 rows 128t + 32d (lane l mod 16 a column, lane
// group g its K slots), and since nibble p and nibble p + 4 are neighbouring rows, a
// shift and a mask bring a pair of them to the two halves of a word.  All 32 rows of
// an MFMA are consecutive, so no group of 32 rows or more is ever split.
//
// scales [N16][G][16] words: the bits of s as a float whose last 8 bits are zero (16
// significant bits, which holds a bf16's or an fp16's scale exactly), and z in those
// 8.  G = 128 K128 / group for groups of 32 or 64 rows, else ceil(k / group).
// Padding columns and groups hold zeros, padding rows the code 0.
#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>

#include <algorithm>

#include "int4.hpp"
#include "launch.hpp"

namespace lora {

namespace {

// fp32 -> 16 significant bits, nearest even; infinities, values that round to one
// (0x7F7FFF80 and more) and NaN become NaN.
__device__ __forceinline__ uint32_t short_scale(float s) {
    constexpr uint32_t kExponent = 0x7F800000u;
    const uint32_t u = __float_as_uint(s), v = (u + 0x7Fu + ((u >> 8) & 1u)) & 0xFFFFFF00u;
    return (u & kExponent) == kExponent || (v & kExponent) == kExponent ? 0x7FC00000u : v;
}

// The same from a double (one rounding), for scales of at least 2^-120.
__device__ __forceinline__ uint32_t short_scale(double s) {
    uint64_t u = (uint64_t)__double_as_longlong(s);
    u += (1ull << 36) - 1 + ((u >> 37) & 1ull);
    u &= ~((1ull << 37) - 1);
    return __float_as_uint((float)__longlong_as_double((long long)u));
}

// Scale and zero of a group with the smallest value lo <= 0 and the largest hi >= 0.
__device__ __forceinline__ uint32_t group_scale(float lo, float hi, bool symmetric) {
    const float most = fmaxf(-lo, hi);
    if (!(most < __uint_as_float(0x7F800000u))) return 0x7FC00000u;
    const double span = symmetric ? (double)most / 7.0 : ((double)hi - (double)lo) / 15.0;
    const double s = span == 0.0 ? 1.0 : fmax(span, 0x1p-120);
    const uint32_t bits = short_scale(s);
    if (symmetric) return bits | 8u;
    return bits | (uint32_t)rint(-(double)lo / (double)__uint_as_float(bits));
}

// w / s to the nearest integer (ties to even), plus z, kept in 0 .. 15; inv = 1 / s.  A
// quotient that is no tie is at least 2^-21 of its size away from one (w has 8
// significant bits, s 16, the tie 5), so an error of two fp32 steps does no harm, and a
// step of refinement makes a tie exact.  Adding 1.5 * 2^23 rounds and leaves the integer
// in the low bits; z_bits is z less that sum's other bits.
__device__ __forceinline__ uint32_t group_code(float w, float s, float inv, int z_bits) {
    float h = w * inv;
    h = fmaf(fmaf(-h, s, w), inv, h);
    const int q = __float_as_int(h + 12582912.f) + z_bits;
    return (uint32_t)min(max(q, 0), 15);
}

// 8 codes of a column -> a stored word.
__device__ __forceinline__ uint32_t code_word(const uint32_t q[8]) {
    return q[0] | q[2] << 4 | q[4] << 8 | q[6] << 12 | q[1] << 16 | q[3] << 20 | q[5] << 24 | q[7] << 28;
}

// Value of `v` in the lane whose number differs in bit 0 or bit 1.
template <int BIT>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, BIT == 0 ? 0xB1 : 0x4E, 0xF, 0xF, true);
}
template <int BIT>
__device__ __forceinline__ float quad(float v) {
    return __uint_as_float(quad<BIT>(__float_as_uint(v)));
}

// A wave: 128 rows of 32 columns; lane 4 p + d has rows 32d .. 32d+31 of columns 2p and
// 2p+1 in registers, so that a group's scale (the quad's lanes together) and its codes
// take one read of W.  The quad turns its words so that each lane writes the 16 bytes of
// one g.  GIVEN: scales have been made (groups of more than 128 rows).  HBM-bound, 2
// bytes in and 0.5 out a value, with 12 instructions a value beside: 28672 x 8192
// 146 us (590 MB, 4.1 TB/s; with 128 rows of two columns a lane, which spilled, this
// and the unpacking took 652 us together, 266 now).
template <bool GIVEN>
__global__ __launch_bounds__(256) void int4_quantize_kernel(const uint16_t *W, I4Shape S, bool symmetric, uint8_t *codes,
                                                            uint32_t *scales) {
    const int lane = threadIdx.x & 63, d = lane & 3;
    const int64_t n32 = (S.n16 + 1) / 2, waves = S.k128 * n32;
    const int each = GIVEN ? 4 : (int)S.group / 32;  // blocks of 32 rows that share a scale (of the 4 here)
    for (int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); w < waves;
         w += (int64_t)gridDim.x * 4) {
        const int64_t t = w / n32, col = (w - t * n32) * 32 + (lane >> 2) * 2, row0 = t * 128 + 32 * d;
        const int rows = col < S.n ? (int)min((int64_t)32, max((int64_t)0, S.k - row0)) : 0;  // (a multiple of 8)
        const uint16_t *src = W + row0 * S.n + col;
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = i < rows ? *(const uint32_t *)(src + i * S.n) : 0u;
        const int64_t cg = col >> 4;
        if (cg >= S.n16) continue;  // (whole quads; an odd last group of columns)
        uint8_t *dst = codes + (((cg * S.k128 + t) * 4) * 16 + (col & 15)) * 16;
        uint32_t *sc = scales + (cg * S.groups + (GIVEN ? t * 128 / S.group : t * (4 / each) + d / each)) * 16 + (col & 15);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            auto value = [&](int i) { return __uint_as_float(c ? r[i] & 0xFFFF0000u : r[i] << 16); };
            uint32_t word;
            if constexpr (GIVEN) {
                word = sc[c];
            } else {
                float lo = 0.f, hi = 0.f;
                uint32_t top = 0u;  // magnitudes order as their bit patterns
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    lo = fminf(lo, value(i));
                    hi = fmaxf(hi, value(i));
                    top = max(top, __float_as_uint(value(i)) & 0x7FFFFFFFu);
                }
                if (each >= 2) lo = fminf(lo, quad<0>(lo)), hi = fmaxf(hi, quad<0>(hi)), top = max(top, quad<0>(top));
                if (each >= 4) lo = fminf(lo, quad<1>(lo)), hi = fmaxf(hi, quad<1>(hi)), top = max(top, quad<1>(top));
                word = top >= 0x7F800000u ? 0x7FC00000u : group_scale(lo, hi, symmetric);
                // (groups past k, and padding columns, hold zeros)
                if (d % each == 0) sc[c] = rows > 0 ? word : 0u;
            }
            const float s = __uint_as_float(word & 0xFFFFFF00u), inv = 1.f / s;
            const int z_bits = (int)(word & 0xFFu) - 0x4B400000;
            const bool nan = s != s;
            uint32_t out[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = group_code(value(8 * g + e), s, inv, z_bits);
                out[g] = nan || 8 * g >= rows ? 0u : code_word(q);
            }
            // the quad's 4 x 4 words turned: lane d gets word g = d of every lane, in lane order
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const uint32_t give = d & 1 ? out[g] : out[g + 1], got = quad<0>(give);
                out[g] = d & 1 ? got : out[g];
                out[g + 1] = d & 1 ? out[g + 1] : got;
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t give = d & 2 ? out[g] : out[g + 2], got = quad<1>(give);
                out[g] = d & 2 ? got : out[g];
                out[g + 2] = d & 2 ? out[g + 2] : got;
            }
            *(uint4 *)(dst + d * 256 + c * 16) = make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

// Scales of groups of more than 128 rows: a thread walks a group's rows of two columns.
__global__ __launch_bounds__(256) void int4_scales_kernel(const uint16_t *W, I4Shape S, bool symmetric, uint32_t *scales) {
    const int64_t nc = S.n16 * 8, items = S.groups * nc;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t gr = it / nc, col = (it - gr * nc) * 2;
        const int64_t end = min(S.k, (gr + 1) * S.group);
        float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f};
        bool bad[2] = {false, false};
        if (col < S.n) {
#pragma unroll 16
            for (int64_t i = gr * S.group; i < end; ++i) {
                const uint32_t x = *(const uint32_t *)(W + i * S.n + col);
                const float w[2] = {__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    lo[c] = fminf(lo[c], w[c]);
                    hi[c] = fmaxf(hi[c], w[c]);
                    bad[c] |= w[c] != w[c];
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
            scales[((col >> 4) * S.groups + gr) * 16 + (col & 15) + c] =
                col >= S.n ? 0u : bad[c] ? 0x7FC00000u : group_scale(lo[c], hi[c], symmetric);
    }
}

// Codes (k x n bytes, their low four bits) in the stored order.  One thread: 128
// rows of four columns, read four bytes a row.
__global__ __launch_bounds__(256) void int4_pack_kernel(const uint8_t *Q, I4Shape S, uint8_t *codes) {
    const int64_t nc = S.n16 * 4, items = S.k128 * nc;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t t = it / nc, col = (it - t * nc) * 4, row0 = t * 128;
        const int rows = col < S.n ? (int)min((int64_t)128, S.k - row0) : 0;
        const uint8_t *src = Q + row0 * S.n + col;
        uint32_t r[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) r[i] = i < rows ? *(const uint32_t *)(src + i * S.n) & 0x0F0F0F0Fu : 0u;
        uint8_t *dst = codes + ((((col >> 4) * S.k128 + t) * 4) * 16 + (col & 15)) * 16;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w4[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    uint32_t q[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[e] = (r[32 * d + 8 * g + e] >> (8 * c)) & 0xFu;
                    w4[d] = code_word(q);
                }
                *(uint4 *)(dst + g * 256 + c * 16) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
    }
}

// Scales (TYPE 0: fp32, 1: bf16, 2: fp16) and zeros (bytes; none: 8) in the stored order.
template <int TYPE>
__global__ __launch_bounds__(256) void int4_pack_scales_kernel(const void *scales_in, const uint8_t *zeros, I4Shape S, int64_t given,
                                                               uint32_t *scales) {
    const int64_t nc = S.n16 * 16, items = S.groups * nc;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t gr = it / nc, col = it - gr * nc;
        uint32_t word = 0u;
        if (col < S.n && gr < given) {
            const int64_t at = gr * S.n + col;
            float s;
            if constexpr (TYPE == 0) s = ((const float *)scales_in)[at];
            else if constexpr (TYPE == 1) s = bf16_to_f32(((const uint16_t *)scales_in)[at]);
            else s = __half2float(((const __half *)scales_in)[at]);
            word = short_scale(s) | (zeros != nullptr ? zeros[at] : 8u);
        }
        scales[((col >> 4) * S.groups + gr) * 16 + (col & 15)] = word;
    }
}

// W' in row-major bf16, each value rounded once (s and q - z have 16 and 8
// significant bits: the product before it is exact).  A thread takes the 16-byte
// pieces of eight columns, 32 rows in four runs of eight, and writes 16 bytes of each
// row.
__global__ __launch_bounds__(256) void int4_dequantize_kernel(const uint8_t *codes, const uint32_t *scales, I4Shape S, uint16_t *W) {
    const int64_t n8 = S.n / 8, items = S.k128 * 4 * n8;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t b = it / n8, c8 = it - b * n8, t = b >> 2;
        const int g = (int)(b & 3);
        const uint8_t *src = codes + ((((c8 >> 1) * S.k128 + t) * 4 + g) * 16 + (c8 & 1) * 8) * 16;
        uint4 q[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) q[c] = *(const uint4 *)(src + c * 16);
        uint16_t *dst = W + c8 * 8;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int64_t row0 = t * 128 + 32 * d + 8 * g;
            if (row0 >= S.k) continue;  // (k is a multiple of 8)
            const uint32_t *sc = scales + ((c8 >> 1) * S.groups + row0 / S.group) * 16 + (c8 & 1) * 8;
            float s[8], z[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                s[c] = __uint_as_float(sc[c] & 0xFFFFFF00u);
                z[c] = (float)(sc[c] & 0xFFu);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = 4 * (e / 2 + 4 * (e & 1));
                float v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t w = d == 0 ? q[c].x : d == 1 ? q[c].y : d == 2 ? q[c].z : q[c].w;
                    v[c] = s[c] * ((float)((w >> at) & 15u) - z[c]);
                }
                *(uint4 *)(dst + (row0 + e) * S.n) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
    }
}

unsigned i4_grid(int64_t items) { return (unsigned)std::min<int64_t>((items + 255) / 256, 1 << 20); }

}  // namespace

hipError_t launch_int4_quantize(const void *W, int64_t k, int64_t n, int64_t group, bool symmetric, void *codes, void *scales,
                                hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    const dim3 grid(i4_grid(s.k128 * ((s.n16 + 1) / 2) * 64));
    const int slot = prof_begin("int4_quantize", stream);
    if (group <= 128) {
        hipLaunchKernelGGL((int4_quantize_kernel<false>), grid, dim3(256), 0, stream, (const uint16_t *)W, s, symmetric,
                           (uint8_t *)codes, (uint32_t *)scales);
    } else {
        hipLaunchKernelGGL(int4_scales_kernel, dim3(i4_grid(s.groups * s.n16 * 8)), dim3(256), 0, stream, (const uint16_t *)W, s,
                           symmetric, (uint32_t *)scales);
        hipLaunchKernelGGL((int4_quantize_kernel<true>), grid, dim3(256), 0, stream, (const uint16_t *)W, s, symmetric,
                           (uint8_t *)codes, (uint32_t *)scales);
    }
    prof_end(slot, stream);
    return hipGetLastError();
}

hipError_t launch_int4_pack(const void *Q, const void *scales_in, int scale_type, const void *zeros, int64_t k, int64_t n, int64_t group,
                            void *codes, void *scales, hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    const int64_t given = (k + group - 1) / group;
    const dim3 grid(i4_grid(s.groups * s.n16 * 16));
    const int slot = prof_begin("int4_pack", stream);
    hipLaunchKernelGGL(int4_pack_kernel, dim3(i4_grid(s.k128 * s.n16 * 4)), dim3(256), 0, stream, (const uint8_t *)Q, s, (uint8_t *)codes);
    const uint8_t *z = (const uint8_t *)zeros;
    uint32_t *out = (uint32_t *)scales;
    if (scale_type == 0) hipLaunchKernelGGL((int4_pack_scales_kernel<0>), grid, dim3(256), 0, stream, scales_in, z, s, given, out);
    else if (scale_type == 1) hipLaunchKernelGGL((int4_pack_scales_kernel<1>), grid, dim3(256), 0, stream, scales_in, z, s, given, out);
    else hipLaunchKernelGGL((int4_pack_scales_kernel<2>), grid, dim3(256), 0, stream, scales_in, z, s, given, out);
    prof_end(slot, stream);
    return hipGetLastError();
}

hipError_t launch_int4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, int64_t group, void *W,
                                  hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    const int slot = prof_begin("int4_dequantize", stream);
    hipLaunchKernelGGL(int4_dequantize_kernel, dim3(i4_grid(s.k128 * 4 * (n / 8))), dim3(256), 0, stream, (const uint8_t *)codes,
                       (const uint32_t *)scales, s, (uint16_t *)W);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
