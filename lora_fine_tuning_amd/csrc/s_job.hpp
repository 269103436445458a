// S = keep.X A formed beside a product over a packed weight, by further work-groups of
// its launch; the launch that finishes the product adds the partial sums.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"

namespace lora {

constexpr int kSK = 1024;  // k of one partial sum of S

struct SJobParams {
    const uint16_t *X;
    int M, K, tiles_m;
    const uint16_t *A;
    int r;            // with segments: the largest rank
    float *spart;     // [SK][M][rs], rs = r rounded up to 4
    int rs, SK;
    uint32_t *keep;   // their dropout mask, M x ceil(K / 32) words, written here (nullptr: none)
    uint64_t seed, offset;
    uint32_t drop;    // threshold of the mask's 16-bit numbers
    // rows in segments with an adapter each (nullptr: one adapter)
    const lora_adapter *adapters;
    const int64_t *seg_off;
    const int32_t *seg_adapter;
    int num_adapters, nseg;
};

// One work-group's share of keep.X A: 1024 of k (split over its NW waves), up to
// 16 MB rows of one adapter and 16 RT ranks.  X's rows come straight from memory, A's as
// 16 ranks of 32 rows a load, turned through 1 KiB of LDS (the layer of 1 row, 4096 x 4096
// in 4 bits, rank 16: 9.2 us in a graph, 10.1 with 8 two-byte loads for an operand); every
// load of a wave before its first use; the waves are added in LDS in wave order.
// A lane's 8 elements of X are one counter of the dropout mask and one byte of
// keep, which the first rank tile's work-groups write.  `smem`: NW MB RT KiB.
template <int NW, int MB, int RT>
__device__ __forceinline__ void s_job(const SJobParams &P, int job, uint4 *smem) {
    constexpr int TM = 16 * MB;
    static_assert(MB * RT <= NW && kSK % (32 * NW) == 0, "a wave for each sum, whole steps of k");
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int ks = job % P.SK;
    int rest = job / P.SK, m0, mend = P.M, r = P.r;
    const uint16_t *A = P.A;
    uint32_t drop = P.drop;
    if (P.adapters != nullptr) {  // a segment's rows in tiles; most segments have fewer than the batch
        const int seg = rest % P.nseg;
        rest /= P.nseg;
        const int which = P.seg_adapter[seg];
        if (which < 0 || which >= P.num_adapters) return;
        const lora_adapter ad = P.adapters[which];
        if (ad.r < 1 || ad.r > P.r) return;
        // (clamped before anything is added: an offset may be any int64)
        m0 = (int)min(max((int64_t)0, P.seg_off[seg]), (int64_t)P.M) + rest % P.tiles_m * TM;
        mend = (int)min(max((int64_t)0, P.seg_off[seg + 1]), (int64_t)P.M);
        if (m0 >= mend) return;
        A = (const uint16_t *)ad.A;
        r = ad.r;
        drop = drop_threshold(ad.p);
    } else {
        m0 = rest % P.tiles_m * TM;
    }
    const int r0 = rest / P.tiles_m * 16 * RT;
    if (r0 >= r) return;  // (the count is rounded up)
    mend = min(mend, m0 + TM);
    const int k0 = ks * kSK + wave * (kSK / NW);
    // rows past the end read as zeros
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(P.X + (size_t)m0 * P.K, (uint64_t)(mend - m0) * P.K * 2u);
    f32x4_t acc[MB][RT];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int J = kSK / NW / 32;
    uint4 x[J][MB];
    uint4 h[J][RT];  // row lane / 2 of 32, ranks 8 (lane mod 2) .. +7 of 16
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int k = k0 + 32 * j + 8 * lg, ka = k0 + 32 * j + (lane >> 1);
#pragma unroll
        for (int a = 0; a < MB; ++a)
            x[j][a] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                          rX, k < P.K ? ((uint32_t)(16 * a + l16) * (uint32_t)P.K + (uint32_t)k) * 2u : kOOB, 0, 0));
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int rank = r0 + 16 * t + 8 * (lane & 1), left = r - rank;
            const uint16_t *src = A + (size_t)ka * r + rank;
            h[j][t] = make_uint4(0u, 0u, 0u, 0u);
            if (ka < P.K && left >= 8) {
                __builtin_memcpy(&h[j][t], src, 16);  // (A may be unaligned)
            } else if (ka < P.K && left > 0) {
                uint32_t q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = e < left ? src[e] : 0u;
                h[j][t] = make_uint4(pack2(q[0], q[1]), pack2(q[2], q[3]), pack2(q[4], q[5]), pack2(q[6], q[7]));
            }
        }
    }
    if (P.keep != nullptr) {
        uint32_t bytes[J][MB];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int a = 0; a < MB; ++a) bytes[j][a] = 0xFFu;
        if (drop > 0) {  // (one branch: the generators' chains interleave)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int a = 0; a < MB; ++a)
                    bytes[j][a] = keep_byte(P.offset + (uint64_t)(m0 + 16 * a + l16) * (uint64_t)P.K + (uint64_t)(k0 + 32 * j + 8 * lg),
                                            P.seed, drop);
        }
        const uint32_t row_bytes = (uint32_t)((P.K + 31) / 32) * 4u;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                const int k = k0 + 32 * j + 8 * lg, row = m0 + 16 * a + l16;
                const uint32_t byte = k < P.K ? bytes[j][a] : 0u;
                x[j][a] = apply_keep(x[j][a], byte);
                if (r0 == 0 && row < mend && (uint32_t)k / 8u < row_bytes)
                    ((uint8_t *)P.keep)[(size_t)row * row_bytes + k / 8] = (uint8_t)byte;
            }
    }
    // (a wave's LDS accesses are taken in order: one step's rows after the last's reads)
    lds_char *turn = (lds_char *)smem + wave * MB * RT * 1024;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < RT; ++t) *(uint4 *)(turn + t * 1024 + lane * 16) = h[j][t];
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const lds_char *at = turn + t * 1024 + (8 * lg + (l16 >> 2)) * 32 + (l16 & 3) * 8;
            const uint2 w0 = lds_read_tr4(at), w1 = lds_read_tr4(at + 128);
            const uint4 w = make_uint4(w0.x, w0.y, w1.x, w1.y);
#pragma unroll
            for (int a = 0; a < MB; ++a) acc[a][t] = mfma16x16x32(w, x[j][a], acc[a][t]);
        }
    }
    asm volatile("" ::: "memory");
    f32x4_t *red = (f32x4_t *)smem;
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int t = 0; t < RT; ++t) red[(wave * MB * RT + a * RT + t) * 64 + lane] = acc[a][t];
    __syncthreads();
    if (wave >= MB * RT) return;
    // wave w adds tile w of every wave: lane (g, l) has ranks 4g .. 4g+3 of row l
    f32x4_t sum = red[wave * 64 + lane];
#pragma unroll
    for (int c = 1; c < NW; ++c) sum += red[(c * MB * RT + wave) * 64 + lane];
    const int row = m0 + 16 * (wave / RT) + l16, rank = r0 + 16 * (wave % RT) + 4 * lg;
    if (row >= mend) return;
    if (rank < P.rs) *(f32x4_t *)(P.spart + ((size_t)ks * P.M + row) * P.rs + rank) = sum;  // (zeros past r)
}

}  // namespace lora
