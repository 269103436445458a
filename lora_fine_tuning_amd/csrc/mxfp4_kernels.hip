// Frozen weights held in microscaled 4-bit floating point (MXFP4): e2m1 codes
// in blocks of 32 along k, one power-of-two scale byte per block.
//
//   W'[i][j] = c(i, j) * 2^(s - 127),  c in {0, 1/2, 1, 3/2, 2, 3, 4, 6, and negatives}
//
// Every W' is exactly a bf16, so a product over W' needs no rounding beyond
// that of a product over a bf16 weight.
//
// Storage (N16 = ceil(n / 16), KB = 4 ceil(k / 128)): codes [N16][KB][16][16]
// bytes and scales [N16][KB][16] bytes; the 16 bytes of (c, b, j) hold column
// 16c + j, rows 32b .. 32b+31, two rows a byte, the lower row in the low
// nibble.  One wave's 16-byte load of four consecutive blocks of a column
// group is 1 KiB in a row and hands lane (g, l) the 32 rows of block g of
// column l: eight consecutive rows are one dword, which four conversions turn
// into an MFMA operand (lane l % 16 a column, lane l / 16 a K slot group).
// Padding columns and rows hold zero codes, padding blocks the scale byte 127.
#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// Two bf16 over the scale, rounded to the nearest code (ties to the even one,
// magnitudes past 6 to 6), into byte B of `old`.
template <int B>
__device__ __forceinline__ uint32_t mx_code(uint32_t old, uint32_t pair, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, pair), scale, B);
}

struct MxShape {
    int64_t k, n;
    int64_t kb, n16;  // blocks of 32 rows (a multiple of 4), groups of 16 columns
};

// One thread: one block of 32 rows of two columns, whose maxima stay inside the
// thread.  Reads 4 bytes of each row and writes 32 bytes of codes; the lanes of a
// wave are neighbours in both.  HBM-bound: 2 bytes in and 0.53 out an element.
// 28672 x 8192, right after a pass that wrote 470 MB: 140 us with two columns a
// thread (4.3 TB/s), 153 with four, 166 with eight (whose stores touch 64 lines an
// instruction); after a pass that read, 108 us (5.5 TB/s).
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const uint16_t *W, MxShape S, uint8_t *codes,
                                                             uint8_t *scales) {
    const int64_t nc = S.n16 * 8, items = S.kb * nc;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t kb = it / nc, cc = it - kb * nc;
        const int64_t col = cc * 2, row0 = kb * 32;
        uint32_t r[32];
        const int rows = col < S.n ? (int)min((int64_t)32, max((int64_t)0, S.k - row0)) : 0;
        const uint16_t *src = W + row0 * S.n + col;
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = i < rows ? *(const uint32_t *)(src + i * S.n) : 0u;
        // bf16 magnitudes order as their bit patterns
        u16x2_t top = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, r[i] & 0x7FFF7FFFu));
        const int64_t at = ((col >> 4) * S.kb + kb) * 16 + (col & 15);
        uint32_t sb = 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            // With the exponent field E and 7 mantissa bits M of the largest
            // magnitude, s = E - 2, one more from M = 96 (1.75) on: the largest
            // over 2^(s-127) lies in [3.5, 7) and rounds to 4 or 6, so nothing is
            // clipped by more than the half step of that part of the grid.  The
            // clamps keep every W' a normal finite bf16.
            const uint32_t b = top[c];
            uint32_t s = (b + 32u) >> 7;
            s = s < 4u ? 2u : min(s - 2u, 252u);
            if (b == 0u) s = 127u;
            const bool bad = b >= 0x7F80u;  // an infinity or NaN: the whole block becomes NaN
            const float scale = __uint_as_float(s << 23);
            uint32_t q[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t sel = c ? 0x07060302u : 0x05040100u;
                uint32_t o = 0u;
                o = mx_code<0>(o, __builtin_amdgcn_perm(r[8 * d + 1], r[8 * d], sel), scale);
                o = mx_code<1>(o, __builtin_amdgcn_perm(r[8 * d + 3], r[8 * d + 2], sel), scale);
                o = mx_code<2>(o, __builtin_amdgcn_perm(r[8 * d + 5], r[8 * d + 4], sel), scale);
                o = mx_code<3>(o, __builtin_amdgcn_perm(r[8 * d + 7], r[8 * d + 6], sel), scale);
                q[d] = bad ? 0u : o;
            }
            *(uint4 *)(codes + (at + c) * 16) = make_uint4(q[0], q[1], q[2], q[3]);
            sb |= (bad ? 255u : s) << (8 * c);
        }
        *(uint16_t *)(scales + at) = (uint16_t)sb;
    }
}

// The inverse, to row-major bf16: one thread writes 16 bytes of each of its
// block's 32 rows (a wave 1 KiB of a row).  28672 x 8192: 102 us, 5.8 TB/s.
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint8_t *codes, const uint8_t *scales,
                                                               MxShape S, uint16_t *W) {
    const int64_t n8 = S.n / 8, items = ((S.k + 31) / 32) * n8;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t kb = it / n8, c8 = it - kb * n8, row0 = kb * 32;
        const int64_t at = ((c8 >> 1) * S.kb + kb) * 16 + (c8 & 1) * 8;
        const uint2 s2 = *(const uint2 *)(scales + at);
        uint4 q[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) q[c] = *(const uint4 *)(codes + (at + c) * 16);
        float sc[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) sc[c] = mx_scale(((c < 4 ? s2.x : s2.y) >> (8 * (c & 3))) & 255u);
        uint16_t *dst = W + row0 * S.n + c8 * 8;
        const int rows = (int)min((int64_t)32, S.k - row0);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            // rows 8d .. 8d+7: dword d of each column's codes
            uint32_t p[8][4];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t w = d == 0 ? q[c].x : d == 1 ? q[c].y : d == 2 ? q[c].z : q[c].w;
                p[c][0] = mx_pair(w, sc[c], 0);
                p[c][1] = mx_pair(w, sc[c], 1);
                p[c][2] = mx_pair(w, sc[c], 2);
                p[c][3] = mx_pair(w, sc[c], 3);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
                uint32_t o[4];
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    o[w] = __builtin_amdgcn_perm(p[2 * w + 1][e >> 1], p[2 * w][e >> 1], sel);
                if (8 * d + e < rows) *(uint4 *)(dst + (8 * d + e) * S.n) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

MxShape mx_shape(int64_t k, int64_t n) { return MxShape{k, n, mx_blocks(k), mx_groups(n)}; }

unsigned mx_grid(int64_t items) { return (unsigned)std::min<int64_t>((items + 255) / 256, 1 << 20); }

}  // namespace

hipError_t launch_mxfp4_quantize(const void *W, int64_t k, int64_t n, void *codes, void *scales, hipStream_t stream) {
    const MxShape s = mx_shape(k, n);
    const int slot = prof_begin("mxfp4_quantize", stream);
    hipLaunchKernelGGL(mxfp4_quantize_kernel, dim3(mx_grid(s.kb * s.n16 * 8)), dim3(256), 0, stream, (const uint16_t *)W, s, (uint8_t *)codes, (uint8_t *)scales);
    prof_end(slot, stream);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, void *W,
                                   hipStream_t stream) {
    const MxShape s = mx_shape(k, n);
    const int slot = prof_begin("mxfp4_dequantize", stream);
    hipLaunchKernelGGL(mxfp4_dequantize_kernel, dim3(mx_grid((k + 31) / 32 * (n / 8))), dim3(256), 0, stream,
                       (const uint8_t *)codes, (const uint8_t *)scales, s, (uint16_t *)W);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
