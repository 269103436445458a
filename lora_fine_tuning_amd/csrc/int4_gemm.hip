// Y = X W' + alpha S B for up to 64 rows, W' = s (q - z) in 4-bit integers
// (int4_kernels.hip describes the storage).
//
// With few rows the weight's bytes bound the product.  It is read once, straight into
// registers: 16 bytes of lane (g, l) are rows 32d + 8g .. +7 of column l, d = 0 .. 3,
// of a block of 128 rows, and word d is the MFMA operand of the 32 rows 128t + 32d
// after a shift and an and-or for each two values: with 4 bits of q on mantissa bits
// 3 .. 6 of 0x4180, the bf16 reads 16 + q.  So
//
//   sum x s (q - z) = s (sum x (16 + q) - (16 + z) sum x)
//
// group by group, in fp32: the weight is never rounded, eight values take eight
// instructions, and sum x comes from an MFMA with a matrix of ones, whose result has
// it in every lane where the product's has its row.  (Rounding s (q - z) to bf16 in
// registers would take 23 instructions for eight values, as long as the bytes take.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "int4.hpp"
#include "launch.hpp"
#include "mxfp4.hpp"
#include "s_job.hpp"

namespace lora {

namespace {

struct I4Params : SJobParams {
    const uint4 *codes;
    const uint4 *scales;  // [N16][G][4] of four words
    uint16_t *Y;          // direct
    float *part;          // [KS][M][N] (nullptr: direct)
    int N, N16, K128, G;
    int each;             // blocks of 128 rows that share a scale (groups of 128 rows or more)
    int tiles_n, KS, per; // slices of k, blocks of 128 rows in one
    int jobs;
};

// Word d of 16 bytes of codes -> the MFMA operand of values 16 + q.
__device__ __forceinline__ uint4 i4_frag(uint32_t w, uint32_t mask) {
    constexpr uint32_t kBias = 0x41804180u;
    return make_uint4(((w << 3) & mask) | kBias, ((w >> 1) & mask) | kBias, ((w >> 5) & mask) | kBias, ((w >> 9) & mask) | kBias);
}

// A work-group takes 16 NB columns and a slice of k; its WK waves take every WK-th
// block of 128 rows of it, D blocks ahead, and are added in LDS in wave order.  STEPS:
// MFMA steps of 32 rows that share a scale (1, 2 or 4).
template <int MB_, int NB_, int WK_, int STEPS_>
struct I4Tile {
    static constexpr int MB = MB_, NB = NB_, WK = WK_, STEPS = STEPS_;
    static constexpr int TN = 16 * NB;
    static constexpr int RT = MB * 2 <= WK ? 2 : 1;
    static constexpr int RED = WK * MB * NB * 1024, JOB = WK * MB * RT * 1024;
    static constexpr int LDS = RED > JOB ? RED : JOB;
};

template <class T>
__global__ __launch_bounds__(64 * T::WK) void int4_gemm_kernel(I4Params P) {
    constexpr int MB = T::MB, NB = T::NB, WK = T::WK, STEPS = T::STEPS, GR = 4 / STEPS;
    extern __shared__ uint4 i4_smem[];
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int id = blockIdx.x;
    if (id < P.jobs) return s_job<WK, MB, T::RT>(P, id, i4_smem);
    id = xcd_order(id - P.jobs, P.tiles_n * P.KS);
    int tn = id, ks = 0;
    if (P.KS > 1) ks = id / P.tiles_n, tn = id - ks * P.tiles_n;
    const int c0 = tn * NB, t0 = ks * P.per, t1 = min(P.K128, t0 + P.per);

    // rows past the last and chunks past k read as zeros
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(P.X, (uint64_t)P.M * P.K * 2u);
    uint32_t xo[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) xo[a] = ((uint32_t)(16 * a + l16) * (uint32_t)P.K + 8u * lg) * 2u;
    const uint4 *wp[NB];
    const uint4 *sp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int c = min(c0 + b, P.N16 - 1);  // (a column group past the last is not stored)
        wp[b] = P.codes + (size_t)c * P.K128 * 64 + lane;
        sp[b] = P.scales + (size_t)c * P.G * 4 + lg;
    }
    const uint32_t mask = 0x00780078u;
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);

    struct Block {
        uint4 w[NB], sc[NB][GR], x[4][MB];
    };
    auto load = [&](Block &B, int t) {
        const bool live = t < t1;
        const int at = live ? t : t0;
#pragma unroll
        for (int b = 0; b < NB; ++b) B.w[b] = wp[b][(size_t)at * 64];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                const int k = 128 * at + 32 * j + 8 * lg;
                B.x[j][a] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                rX, live && k < P.K ? xo[a] + (uint32_t)(128 * at + 32 * j) * 2u : kOOB, 0, 0));
            }
        const int gr = STEPS < 4 ? at * GR : P.each == 1 ? at : at / P.each;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < GR; ++e) B.sc[b][e] = sp[b][(size_t)(gr + e) * 4];
    };
    f32x4_t total[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) total[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Block &B) {
#pragma unroll
        for (int e = 0; e < GR; ++e) {
            f32x4_t acc[MB][NB], sum[MB];
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                sum[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                const int j = e * STEPS + q;
#pragma unroll
                for (int a = 0; a < MB; ++a) sum[a] = mfma16x16x32(ones, B.x[j][a], sum[a]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint4 &v = B.w[b];
                    const uint4 w = i4_frag(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, mask);
#pragma unroll
                    for (int a = 0; a < MB; ++a) acc[a][b] = mfma16x16x32(w, B.x[j][a], acc[a][b]);
                }
            }
            // lane (g, l): columns 4g .. 4g+3 of row l
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t word[4] = {B.sc[b][e].x, B.sc[b][e].y, B.sc[b][e].z, B.sc[b][e].w};
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float s = __uint_as_float(word[v] & 0xFFFFFF00u), z = 16.f + (float)(word[v] & 0xFFu);
#pragma unroll
                    for (int a = 0; a < MB; ++a) total[a][b][v] = fmaf(s, fmaf(-z, sum[a][v], acc[a][b][v]), total[a][b][v]);
                }
            }
        }
    };
    Block A0, A1;
    int t = t0 + wave;
    load(A0, t);
    for (; t < t1; t += 2 * WK) {
        load(A1, t + WK);
        multiply(A0);
        load(A0, t + 2 * WK);
        if (t + WK < t1) multiply(A1);
    }

    // the waves' sums, in wave order
    f32x4_t *red = (f32x4_t *)i4_smem;
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[(wave * MB * NB + a * NB + b) * 64 + lane] = total[a][b];
    __syncthreads();
    for (int q = wave; q < MB * NB; q += WK) {
        const int a = q / NB, b = q % NB;
        f32x4_t v = red[q * 64 + lane];
#pragma unroll
        for (int c = 1; c < WK; ++c) v += red[(c * MB * NB + q) * 64 + lane];
        const int row = 16 * a + l16, col = (c0 + b) * 16 + 4 * lg;
        if (row >= P.M || col >= P.N) continue;
        if (P.part != nullptr)
            *(f32x4_t *)(P.part + ((size_t)ks * P.M + row) * P.N + col) = v;
        else
            *(uint2 *)(P.Y + (size_t)row * P.N + col) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
}

template <class T>
hipError_t launch_t(const I4Params &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void *)int4_gemm_kernel<T>, T::LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((int4_gemm_kernel<T>), dim3((unsigned)(P.tiles_n * P.KS + P.jobs)), dim3(64 * T::WK), T::LDS, stream, P);
    return hipGetLastError();
}

struct I4Kind {
    const char *name;  // in the timing pool
    hipError_t (*launch[3])(const I4Params &, hipStream_t);  // groups of 32, 64, 128 rows or more
    int tm, tn, ranks;  // rows and columns of a tile, ranks of one job of S
};
template <int MB, int NB, int WK>
constexpr I4Kind kind_of(const char *name) {
    return I4Kind{name, {launch_t<I4Tile<MB, NB, WK, 1>>, launch_t<I4Tile<MB, NB, WK, 2>>, launch_t<I4Tile<MB, NB, WK, 4>>}, 16 * MB, 16 * NB,
                  16 * I4Tile<MB, NB, WK, 4>::RT};
}
const I4Kind kKinds[] = {
    kind_of<1, 1, 8>("int4_gemm 16x16"),
    kind_of<2, 2, 8>("int4_gemm 32x32"),
    kind_of<4, 2, 8>("int4_gemm 64x32"),
};

}  // namespace

I4Plan int4_plan(int64_t m, int64_t k, int64_t n, int64_t group, int r, int nseg) {
    I4Plan p{};
    // (offsets into X stay below 2^31, and counts within an int)
    if (m <= 0 || m > kI4Rows || k > (1 << 20) || n > (1 << 24)) return p;
    p.kind = m <= 16 ? 1 : m <= 32 ? 2 : 3;
    const I4Kind &K = kKinds[p.kind - 1];
    p.tiles_n = (int)((n + K.tn - 1) / K.tn);
    p.KS = 1;
    p.per = (int)((k + 127) / 128);
    p.finish = r > 0;
    p.part_bytes = p.finish ? (size_t)p.KS * m * n * sizeof(float) : 0;
    if (r > 0) {
        const int64_t jobs = (k + kSK - 1) / kSK * ((r + K.ranks - 1) / K.ranks) * std::max(nseg, 1);
        if (nseg == 0 || jobs <= 1024) {
            p.SK = (int)((k + kSK - 1) / kSK);
            p.jobs = (int)((jobs + 7) / 8 * 8);
            p.spart_bytes = (size_t)p.SK * m * ((r + 3) / 4 * 4) * sizeof(float);
        }
    }
    (void)group;
    return p;
}

hipError_t launch_int4_gemm(const I4Plan &pl, const void *X, const void *codes, const void *scales, int64_t group, int m, int k, int n,
                            const AdapterSource &src, const MxDropout &drop, float *S, void *Y, float *part, float *spart,
                            hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    I4Params P{};
    P.X = (const uint16_t *)X;
    P.M = m;
    P.K = k;
    P.tiles_m = 1;
    P.A = (const uint16_t *)src.A;
    P.r = src.r;
    P.spart = spart;
    P.rs = (src.r + 3) / 4 * 4;
    P.SK = pl.SK;
    P.keep = drop.keep;
    P.seed = drop.seed;
    P.offset = drop.offset;
    P.drop = drop_threshold(src.p);
    P.adapters = src.table;
    P.seg_off = src.seg_off;
    P.seg_adapter = src.seg_adapter;
    P.num_adapters = src.num_adapters;
    P.nseg = src.num_segments;
    P.codes = (const uint4 *)codes;
    P.scales = (const uint4 *)scales;
    P.Y = (uint16_t *)Y;
    P.part = pl.finish ? part : nullptr;
    P.N = n;
    P.N16 = (int)s.n16;
    P.K128 = (int)s.k128;
    P.G = (int)s.groups;
    P.each = group < 128 ? 1 : (int)(group / 128);
    P.tiles_n = pl.tiles_n;
    P.KS = pl.KS;
    P.per = pl.per;
    P.jobs = pl.jobs;
    const I4Kind &K = kKinds[pl.kind - 1];
    const int slot = prof_begin(K.name, stream);
    const hipError_t e = K.launch[group == 32 ? 0 : group == 64 ? 1 : 2](P, stream);
    prof_end(slot, stream);
    if (e != hipSuccess || !pl.finish) return e;
    if (src.table != nullptr) return launch_mxfp4_join(true, part, pl.KS, m, n, S, src.r, pl.SK, spart, nullptr, src, Y, stream);
    return launch_mxfp4_finish(part, pl.KS, m, n, S, pl.SK, spart, src, Y, stream);
}

}  // namespace lora
