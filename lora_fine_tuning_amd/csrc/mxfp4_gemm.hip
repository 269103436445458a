// Y = X W' for few and middling numbers of rows, W' in MXFP4 (mxfp4_kernels.hip
// describes the storage), with the LoRA term alpha S B added before the store.
//
// With few rows the weight's bytes bound the product, so it is read packed, a
// quarter of its bf16 bytes, and expanded in registers: one 16-byte LDS read
// hands lane (g, l) rows 32g .. 32g+31 of column l of a 128-deep step, and each
// of its four dwords becomes the MFMA operand of a 32-deep step by four
// conversions.  The MFMA's K order is free as long as both operands follow it:
// lane group g takes k = 128 t + 32 g + 8 j .. +7 in step j, and reads X's row
// chunk 4 g + j.
//
// A work-group covers 16 WM MB rows and 16 WN NB columns; its waves split the
// rows (WM), the columns (WN) and each stage's k (WK chunks of 128).  Stages of
// X, codes and scales come through an NS-deep LDS ring by direct-to-LDS loads,
// NS - 1 stages ahead.  X rows take 256 bytes a chunk with their 16-byte pieces
// XORed by the row, so 16 rows read at one piece fall on 16 different bank
// ranges.  Waves along k are added in LDS in wave order.  Where the tiles would
// leave CUs idle, work-groups split k further: each slice writes fp32 partial
// sums and a second launch adds them in slice order.
#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "launch.hpp"

namespace lora {

namespace {

// Vector memory down to N loads in flight, and no LDS read in flight.
template <int N>
__device__ __forceinline__ void wait_vmcnt_lds() {
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

struct MxGemmParams {
    const uint16_t *X;
    const uint8_t *codes, *scales;
    uint16_t *Y;   // KS == 1
    float *part;   // KS > 1: [KS][M][N]
    int M, N, K;
    int groups, blocks;  // N16, KB
    int tiles_m, tiles_n;
    int KS, per;         // slices of k, stages of a slice
    const float *S;      // LoRA: M x r fp32 (nullptr: none)
    const uint16_t *B;   // r x N
    int r;
    float alpha;
};

__device__ __forceinline__ float mx_scale(uint32_t s) {
    return __uint_as_float((s << 23) | ((s == 0u || s == 255u) ? 0x00400000u : 0u));
}

// Eight codes (one dword) -> an MFMA operand.
__device__ __forceinline__ uint4 mx_frag(uint32_t w, float scale) {
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3)));
}

template <int WM_, int WN_, int WK_, int MB_, int NB_, int XR_, int NS_>
struct MxTile {
    static constexpr int WM = WM_, WN = WN_, WK = WK_, MB = MB_, NB = NB_, XR = XR_, NS = NS_;
    static constexpr int NW = WM * WN * WK, TM = 16 * WM * MB, TN = 16 * WN * NB, KW = 128 * WK;
    static constexpr int G = WN * NB;                  // column groups
    static constexpr int XU = XR * WK / 4, WU = G * WK, SU = (G * WK + 15) / 16;  // 1 KiB loads of a stage
    static constexpr int UPW = (XU + WU + SU + NW - 1) / NW;                      // per wave
    static constexpr int XB = XU * 1024, WB = WU * 1024, STAGE = XB + WB + SU * 1024;
    static constexpr int SPARE = NS * STAGE;  // 1 KiB that surplus loads fill with zeros
    static constexpr int RED = (WK - 1) * WM * WN * MB * NB * 1024;
    static constexpr int LDS = SPARE + 1024 > RED ? SPARE + 1024 : RED;
    static_assert(XR * WK % 4 == 0 && LDS <= 160 * 1024, "tile does not fit");
};

template <class T>
__global__ __launch_bounds__(64 * T::NW) void mxfp4_gemm_kernel(MxGemmParams P) {
    constexpr int WN = T::WN, WK = T::WK, MB = T::MB, NB = T::NB, XR = T::XR, NS = T::NS, G = T::G;
    extern __shared__ uint4 mx_smem[];
    lds_char *smem = (lds_char *)mx_smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
    const int l16 = lane & 15, lg = lane >> 4;

    // Work-groups of one XCD (id mod 8) take a contiguous run of (slice, column
    // tile, row tile) with the row tiles innermost, so a weight tile is fetched
    // into one L2 once.
    const int total = P.tiles_m * P.tiles_n * P.KS;
    int id = blockIdx.x;
    {
        const int xcd = id & 7, local = id >> 3, each = total >> 3, rem = total & 7;
        id = xcd * each + min(xcd, rem) + local;
    }
    const int tm = id % P.tiles_m, tn = id / P.tiles_m % P.tiles_n, ks = id / (P.tiles_m * P.tiles_n);
    const int m0 = tm * T::TM, n0 = tn * T::TN, g0 = tn * G;
    const int k0 = ks * P.per * T::KW;
    const int nit = min(P.per, (P.K - k0 + T::KW - 1) / T::KW);  // >= 1: the host sizes the slices

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.K * 2u, group_bytes = (uint32_t)P.blocks * 256u;
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.K, (uint32_t)min(P.M - m0, T::TM) * row_bytes);
    const uint32_t ng = (uint32_t)min(P.groups - g0, G);
    const sgpr4_t dW = make_desc(P.codes + (size_t)g0 * group_bytes, ng * group_bytes);
    const sgpr4_t dS = make_desc(P.scales + (size_t)g0 * (group_bytes / 16), ng * (group_bytes / 16));

    // This wave's loads of a stage: byte offset in the source at stage 0, and
    // the k it stands for (a load past `lim` fills zeros).
    uint32_t off[T::UPW];
    int pos[T::UPW], lim[T::UPW];
#pragma unroll
    for (int i = 0; i < T::UPW; ++i) {
        const int u = wave + T::NW * i;
        off[i] = 0;
        pos[i] = 0;
        lim[i] = -1;
        if (u < T::XU) {
            const int c = u / (XR / 4), row = (u % (XR / 4)) * 4 + (lane >> 4);
            const int piece = (lane & 15) ^ (row & 15);
            pos[i] = k0 + 128 * c + 8 * piece;
            off[i] = (uint32_t)row * row_bytes + (uint32_t)pos[i] * 2u;
            lim[i] = m0 + row < P.M ? P.K : -1;
        } else if (u < T::XU + T::WU) {
            const int q = u - T::XU, c = q / G, g = q % G;
            pos[i] = k0 + 128 * c + 32 * lg;
            off[i] = (uint32_t)g * group_bytes + (uint32_t)(pos[i] / 32) * 256u + (uint32_t)l16 * 16u;
            lim[i] = g0 + g < P.groups ? P.blocks * 32 : -1;
        } else if (u < T::XU + T::WU + T::SU) {
            const int q = (u - T::XU - T::WU) * 16 + (lane >> 2), c = q / G, g = q % G;
            pos[i] = k0 + 128 * c + 32 * (lane & 3);
            off[i] = (uint32_t)g * (group_bytes / 16) + (uint32_t)(pos[i] / 32) * 16u;
            lim[i] = q < G * WK && g0 + g < P.groups ? P.blocks * 32 : -1;
        }
    }
    auto issue = [&](int it, int buf) {
        const uint32_t base = lds0 + (uint32_t)buf * T::STAGE;
        const int dk = it * T::KW;
#pragma unroll
        for (int i = 0; i < T::UPW; ++i) {
            const int u = wave + T::NW * i;
            const bool live = it < nit && pos[i] + dk < lim[i];
            const uint32_t step = u < T::XU ? 2u * T::KW : u < T::XU + T::WU ? 8u * T::KW : T::KW / 2u;
            const uint32_t o = live ? off[i] + (uint32_t)it * step : kOOB;
            const uint32_t dst = u < T::XU + T::WU + T::SU ? base + (uint32_t)u * 1024u : lds0 + T::SPARE;
            if (u < T::XU) dma16(dX, o, dst);
            else if (u < T::XU + T::WU) dma16(dW, o, dst);
            else dma16(dS, o, dst);
        }
    };

    f32x4_t acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    int xrow[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) xrow[a] = ((wm * MB + a) * 16 + l16) & (XR < 16 ? XR - 1 : -1);

#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s, s);
    int buf = 0;
    for (int it = 0; it < nit; ++it) {
        // this stage has landed, and this wave's reads of the last one are done
        wait_vmcnt_lds<T::UPW *(NS - 2)>();
        asm volatile("" ::: "memory");  // keep the LDS reads below the barrier
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // the buffer of stage it - 1, which every wave has read
        issue(it + NS - 1, buf == 0 ? NS - 1 : buf - 1);
        const lds_char *sx = smem + buf * T::STAGE + wk * XR * 256;
        const lds_char *sw = smem + buf * T::STAGE + T::XB + (wk * G + wn * NB) * 1024 + lane * 16;
        const lds_char *ss = smem + buf * T::STAGE + T::XB + T::WB + (wk * G + wn * NB) * 64 + lane;
        uint4 q[NB];
        float sc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            q[b] = *(const uint4 *)(sw + b * 1024);
            sc[b] = mx_scale(*(const uint8_t *)(ss + b * 64));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 x[MB];
#pragma unroll
            for (int a = 0; a < MB; ++a) x[a] = *(const uint4 *)(sx + xrow[a] * 256 + (((4 * lg + j) ^ (xrow[a] & 15)) << 4));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 w = mx_frag(j == 0 ? q[b].x : j == 1 ? q[b].y : j == 2 ? q[b].z : q[b].w, sc[b]);
#pragma unroll
                for (int a = 0; a < MB; ++a) acc[a][b] = mfma16x16x32(w, x[a], acc[a][b]);
            }
        }
        buf = buf == NS - 1 ? 0 : buf + 1;
    }
    wait_vmcnt<0>();  // (the last loads fill zeros: nothing may land in the space used below)

    if constexpr (WK > 1) {
        __syncthreads();
        float4 *red = (float4 *)mx_smem;
        const int w2 = wave / WK;
        if (wk > 0) {
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    red[(((wk - 1) * T::WM * WN + w2) * MB * NB + a * NB + b) * 64 + lane] =
                        __builtin_bit_cast(float4, acc[a][b]);
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int c = 0; c < WK - 1; ++c)
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[a][b] += __builtin_bit_cast(f32x4_t, red[((c * T::WM * WN + w2) * MB * NB + a * NB + b) * 64 + lane]);
    }

    // alpha S B: ranks 32 a step, alpha S split into bf16 hi + lo
    if (P.S != nullptr && ks == 0) {
        const __amdgpu_buffer_rsrc_t rS = make_rsrc(P.S + (size_t)m0 * P.r, (uint64_t)min(P.M - m0, T::TM) * P.r * 4u);
        const __amdgpu_buffer_rsrc_t rB = make_rsrc(P.B, (uint64_t)P.r * P.N * 2u);
        for (int r0 = 0; r0 < P.r; r0 += 32) {
            const int rb = r0 + 8 * lg;
            uint4 hi[MB], lo[MB];
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                const uint32_t row = (uint32_t)((wm * MB + a) * 16 + l16);  // past the last row: past the resource
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = P.alpha * __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                         rS, rb + e < P.r ? (row * (uint32_t)P.r + (uint32_t)(rb + e)) * 4u : kOOB, 0, 0));
                split_frag(v, hi[a], lo[a]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int col = n0 + (wn * NB + b) * 16 + l16;
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
                        rB, rb + e < P.r && col < P.N ? ((uint32_t)(rb + e) * (uint32_t)P.N + (uint32_t)col) * 2u : kOOB, 0, 0);
                const uint4 w = make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7]));
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    acc[a][b] = mfma16x16x32(w, hi[a], acc[a][b]);
                    acc[a][b] = mfma16x16x32(w, lo[a], acc[a][b]);
                }
            }
        }
    }

    // lane (g, l): columns 4g .. 4g+3 of a group, row l
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const int row = m0 + (wm * MB + a) * 16 + l16;
        if (row >= P.M) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int col = n0 + (wn * NB + b) * 16 + 4 * lg;
            if (col >= P.N) continue;
            if (P.KS == 1)
                *(uint2 *)(P.Y + (size_t)row * P.N + col) =
                    make_uint2(pack_bf16x2(acc[a][b][0], acc[a][b][1]), pack_bf16x2(acc[a][b][2], acc[a][b][3]));
            else
                *(f32x4_t *)(P.part + ((size_t)ks * P.M + row) * P.N + col) = acc[a][b];
        }
    }
}

// Y = the slices' sums in slice order, rounded; 8 columns a thread.
__global__ __launch_bounds__(256) void mxfp4_sum_kernel(const float *part, int KS, int64_t count, uint16_t *Y) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= count) return;
    float4 a = *(const float4 *)(part + at), b = *(const float4 *)(part + at + 4);
    for (int s = 1; s < KS; ++s) {
        const float4 c = *(const float4 *)(part + s * count + at), d = *(const float4 *)(part + s * count + at + 4);
        a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
        b.x += d.x, b.y += d.y, b.z += d.z, b.w += d.w;
    }
    *(uint4 *)(Y + at) = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                                    pack_bf16x2(b.z, b.w));
}

template <class T>
hipError_t launch_t(const MxGemmParams &P, hipStream_t stream) {
    if (T::LDS > 64 * 1024)
        (void)hipFuncSetAttribute((const void *)mxfp4_gemm_kernel<T>, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
    hipLaunchKernelGGL((mxfp4_gemm_kernel<T>), dim3((unsigned)(P.tiles_m * P.tiles_n * P.KS)), dim3(64 * T::NW), T::LDS,
                       stream, P);
    return hipGetLastError();
}

using Tile4 = MxTile<1, 1, 8, 1, 1, 4, 3>;      // up to 4 rows, 16 columns
using Tile16 = MxTile<1, 1, 8, 1, 1, 16, 3>;    // up to 16 rows, 16 columns
using Tile32 = MxTile<1, 2, 4, 2, 2, 32, 3>;    // up to 32 rows, 64 columns
using Tile64 = MxTile<1, 4, 2, 4, 2, 64, 3>;    // up to 64 rows, 128 columns
using Tile128 = MxTile<2, 4, 1, 4, 2, 128, 3>;  // 128 rows, 128 columns
using TileBig = MxTile<2, 4, 1, 4, 4, 128, 3>;  // 128 rows, 256 columns

}  // namespace

MxGemmPlan mx_gemm_plan(int64_t m, int64_t k, int64_t n, int want) {
    MxGemmPlan p{};
    if (m <= 0 || k > (1 << 20) || n > (1 << 27) || m > 16384) return p;
    const int64_t tiles64 = (m + 127) / 128 * ((n + 255) / 256);
    p.kind = m <= 4 ? 1 : m <= 16 ? 2 : m <= 32 ? 3 : m <= 64 ? 4 : tiles64 >= 128 ? 6 : 5;
    if (want) p.kind = want;
    static const int tm[] = {0, Tile4::TM, Tile16::TM, Tile32::TM, Tile64::TM, Tile128::TM, TileBig::TM};
    static const int tn[] = {0, Tile4::TN, Tile16::TN, Tile32::TN, Tile64::TN, Tile128::TN, TileBig::TN};
    static const int kw[] = {0, Tile4::KW, Tile16::KW, Tile32::KW, Tile64::KW, Tile128::KW, TileBig::KW};
    p.tiles_m = (int)((m + tm[p.kind] - 1) / tm[p.kind]);
    p.tiles_n = (int)((n + tn[p.kind] - 1) / tn[p.kind]);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, stages = (k + kw[p.kind] - 1) / kw[p.kind];
    int64_t KS = 1;
    if (tiles < 192) KS = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, stages / 4));
    p.per = (int)((stages + KS - 1) / KS);
    p.KS = (int)((stages + p.per - 1) / p.per);
    p.part_bytes = p.KS > 1 ? (size_t)p.KS * m * n * sizeof(float) : 0;
    return p;
}

hipError_t launch_mxfp4_gemm(const MxGemmPlan &pl, const void *X, const void *codes, const void *scales, int m, int k,
                             int n, const float *S, const void *B, int r, float alpha, void *Y, float *part,
                             hipStream_t stream) {
    MxGemmParams P{};
    P.X = (const uint16_t *)X;
    P.codes = (const uint8_t *)codes;
    P.scales = (const uint8_t *)scales;
    P.Y = (uint16_t *)Y;
    P.part = part;
    P.M = m;
    P.N = n;
    P.K = k;
    P.groups = (int)mx_groups(n);
    P.blocks = (int)mx_blocks(k);
    P.tiles_m = pl.tiles_m;
    P.tiles_n = pl.tiles_n;
    P.KS = pl.KS;
    P.per = pl.per;
    P.S = S;
    P.B = (const uint16_t *)B;
    P.r = r;
    P.alpha = alpha;
    int slot = prof_begin("mxfp4_gemm", stream);
    hipError_t e = hipErrorInvalidValue;
    switch (pl.kind) {
    case 1: e = launch_t<Tile4>(P, stream); break;
    case 2: e = launch_t<Tile16>(P, stream); break;
    case 3: e = launch_t<Tile32>(P, stream); break;
    case 4: e = launch_t<Tile64>(P, stream); break;
    case 5: e = launch_t<Tile128>(P, stream); break;
    case 6: e = launch_t<TileBig>(P, stream); break;
    }
    prof_end(slot, stream);
    if (e != hipSuccess || pl.KS == 1) return e;
    slot = prof_begin("mxfp4_sum", stream);
    const int64_t count = (int64_t)m * n;
    hipLaunchKernelGGL(mxfp4_sum_kernel, dim3((unsigned)((count / 8 + 255) / 256)), dim3(256), 0, stream, part, pl.KS, count,
                       (uint16_t *)Y);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
