// Y = X W' + alpha S B for few and middling numbers of rows, W' = s (q - z) in 4-bit integers
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
#include <type_traits>

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
    const float *S;       // the epilogue's LoRA term: M x r fp32 (nullptr: none)
    const uint16_t *B;    // r x N
    float alpha;
    int s_wide;           // S may be read 16 bytes at a time
    int each;             // blocks of 128 rows that share a scale (groups of 128 rows or more),
    uint32_t each_inv;    // and floor(2^32 / each) + 1: block t's group is the product's high word
    int tiles_n, KS, per; // slices of k, blocks of 128 rows in one
    int jobs;
};

// Word d of 16 bytes of codes -> the MFMA operand of values 16 + q.  The constants are
// a vector and a scalar register, which the one instruction for and-or takes.
struct I4Bits {
    uint32_t mask, bias;
};
__device__ __forceinline__ I4Bits i4_bits() {
    I4Bits c;
    asm("v_mov_b32 %0, 0x00780078" : "=v"(c.mask));
    asm("s_mov_b32 %0, 0x41804180" : "=s"(c.bias));
    return c;
}
__device__ __forceinline__ uint4 i4_frag(uint32_t w, const I4Bits &c) {
    return make_uint4(((w << 3) & c.mask) | c.bias, ((w >> 1) & c.mask) | c.bias, ((w >> 5) & c.mask) | c.bias, ((w >> 9) & c.mask) | c.bias);
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
    const I4Bits bits = i4_bits();
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
        const int gr = STEPS < 4 ? at * GR : P.each == 1 ? at : (int)__umulhi((uint32_t)at, P.each_inv);
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
                    const uint4 w = i4_frag(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, bits);
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

// More rows: a work-group takes 16 WM MB rows and 16 WN NB columns, and X and the weight
// come through an LDS ring of two or three stages by direct-to-LDS loads, so that the WN
// waves beside each other share X and the WM waves the weight.  A stage is WK blocks of
// 128 rows of the weight, one for each of the WK waves along k.  X takes 256 bytes a row and block; piece 4j + g
// (16 bytes: what lane group g reads in step j) of row i sits at place (4j + g) ^ (i mod
// 16), which puts the 16 lanes that a 16-byte read serves together on different banks.
// The shapes for up to 64 rows (WM = 1) form S beside the product and leave alpha S B to
// the finishing launch; the others are given S and add alpha S B themselves, where k is
// not split.
template <int MB_, int NB_, int WM_, int WN_, int WK_, int STEPS_>
struct I4Ring {
    static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, WK = WK_, STEPS = STEPS_;
    static constexpr bool RIDE = WM == 1;
    static constexpr int NW = WM * WN * WK, G = WN * NB, TM = 16 * WM * MB, TN = 16 * G, GR = 4 / STEPS;
    static constexpr int XU = 4 * WM * MB * WK, WU = G * WK, SU = (G * WK * GR + 15) / 16;  // 1 KiB loads of a stage
    static constexpr int XPW = (XU + NW - 1) / NW, WPW = (WU + NW - 1) / NW, SPW = (SU + NW - 1) / NW, UPW = XPW + WPW + SPW;
    static constexpr int XB = XU * 1024, WB = WU * 1024, STAGE = XB + WB + SU * 1024;
    static constexpr int NS = 3 * STAGE + 1024 <= 160 * 1024 ? 3 : 2;  // stages of the ring
    static constexpr int SPARE = NS * STAGE;  // 1 KiB that surplus loads fill with zeros
    static constexpr int RT = MB * 2 <= NW ? 2 : 1;
    static constexpr int RED = WK > 1 ? WK * WN * MB * NB * 1024 : 0, JOB = RIDE ? NW * MB * RT * 1024 : 0;
    static constexpr int MOST = RED > JOB ? RED : JOB;
    static constexpr int LDS = SPARE + 1024 > MOST ? SPARE + 1024 : MOST;
    static_assert(NW % 4 == 0 && LDS <= 160 * 1024 && (RIDE || WK == 1), "tile does not fit");
};

template <class T>
__global__ __launch_bounds__(64 * T::NW) void int4_ring_kernel(I4Params P) {
    constexpr int MB = T::MB, NB = T::NB, WM = T::WM, WN = T::WN, WK = T::WK, STEPS = T::STEPS, GR = T::GR, NW = T::NW, G = T::G;
    constexpr int XT = 4 * WM * MB;  // units of X of a block
    extern __shared__ uint4 i4_smem[];
    lds_char *smem = (lds_char *)i4_smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
    int id = blockIdx.x;
    if constexpr (T::RIDE) {
        if (id < P.jobs) return s_job<NW, MB, T::RT>(P, id, i4_smem);
        id -= P.jobs;
    }
    // (row tiles innermost: a weight tile is fetched into one L2 once)
    id = xcd_order(id, P.tiles_m * P.tiles_n * P.KS);
    int tm = 0, tn = id, ks = 0;
    if (P.tiles_m > 1) tn = id / P.tiles_m, tm = id - tn * P.tiles_m;
    if (P.KS > 1) ks = tn / P.tiles_n, tn -= ks * P.tiles_n;
    const int m0 = tm * T::TM, rows = min(P.M - m0, T::TM);
    const int c0 = tn * G, t0 = ks * P.per, t1 = min(P.K128, t0 + P.per);
    const int nit = (t1 - t0 + WK - 1) / WK;

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.K * 2u, code_bytes = (uint32_t)P.K128 * 1024u, scale_bytes = (uint32_t)P.G * 64u;
    const uint32_t ng = (uint32_t)min(P.N16 - c0, G);
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.K, (uint32_t)rows * row_bytes);
    const sgpr4_t dW = make_desc((const char *)P.codes + (size_t)c0 * code_bytes, ng * code_bytes);
    const sgpr4_t dS = make_desc((const char *)P.scales + (size_t)c0 * scale_bytes, ng * scale_bytes);

    // This wave's loads of a stage.  Unit u of X: rows 4 (u mod XT) .. +3 of block
    // u / XT of the stage; of codes: column group u mod G, block u / G; of scales: 16
    // pieces q of 64 bytes, column group q mod G, block q / G / GR, group q / G mod GR of
    // the block.  xo, wo, so: byte offsets at stage 0 (kOOB: zeros); a lane's k of X is xk
    // in every unit of a wave (4 divides NW), counted from its block.
    const int xk = 8 * (l16 ^ ((4 * (wave & 3) + lg) & 15)), kend = min(P.K, 128 * t1);
    uint32_t xo[T::XPW], wo[T::WPW], so[T::SPW];
    int st[T::SPW];
#pragma unroll
    for (int i = 0; i < T::XPW; ++i) {
        const int u = wave + NW * i, row = u % XT * 4 + lg;
        xo[i] = u < T::XU && row < rows ? (uint32_t)row * row_bytes + (uint32_t)(128 * (t0 + u / XT) + xk) * 2u : kOOB;
    }
#pragma unroll
    for (int i = 0; i < T::WPW; ++i) {
        const int u = wave + NW * i, c = u % G;
        wo[i] = u < T::WU && c < (int)ng ? (uint32_t)c * code_bytes + (uint32_t)(t0 + u / G) * 1024u + (uint32_t)lane * 16u : kOOB;
    }
#pragma unroll
    for (int i = 0; i < T::SPW; ++i) {
        const int q = (wave + NW * i) * 16 + (lane >> 2), c = q % G;
        st[i] = t0 + q / G / GR;
        so[i] = q < G * WK * GR && c < (int)ng ? (uint32_t)c * scale_bytes + (uint32_t)(q / G % GR) * 64u + (uint32_t)(lane & 3) * 16u : kOOB;
    }
    auto issue_one = [&](int it, int buf, int i) {
        const uint32_t base = lds0 + (uint32_t)buf * T::STAGE + (uint32_t)wave * 1024u, spare = lds0 + T::SPARE;
        const int dt = it * WK;
        if (i < T::XPW) {
            const int u = wave + NW * i;
            dma16_at(dX, xk < kend - 128 * (t0 + dt + u / XT) ? xo[i] : kOOB, (uint32_t)dt * 256u,
                     T::XU % NW == 0 || u < T::XU ? base + (uint32_t)(NW * i) * 1024u : spare);
        } else if (i < T::XPW + T::WPW) {
            const int j = i - T::XPW, u = wave + NW * j;
            dma16_at(dW, t0 + dt + u / G < t1 ? wo[j] : kOOB, (uint32_t)dt * 1024u,
                     T::WU % NW == 0 || u < T::WU ? base + T::XB + (uint32_t)(NW * j) * 1024u : spare);
        } else {
            const int j = i - T::XPW - T::WPW, at = st[j] + dt;
            const uint32_t gr = STEPS < 4 ? (uint32_t)at * GR : P.each == 1 ? (uint32_t)at : __umulhi((uint32_t)at, P.each_inv);
            dma16_at(dS, at < t1 && so[j] != kOOB ? so[j] + gr * 64u : kOOB, 0u,
                     T::SU % NW == 0 || wave + NW * j < T::SU ? base + T::XB + T::WB + (uint32_t)(NW * j) * 1024u : spare);
        }
    };
    // A stage has landed (`later` ones may be in flight), and this wave's LDS reads
    // are done; after the barrier both hold for every wave.
    auto stage_ready = [&](auto later) {
        wait_vmcnt_lds<T::UPW * decltype(later)::value>();
        asm volatile("" ::: "memory");  // keep LDS reads and loads into LDS on their side of the barrier
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    f32x4_t total[MB][NB], acc[MB][NB], sum[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) total[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const I4Bits bits = i4_bits();
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);

    // x[j % 2] holds X's rows of step j, q the wave's codes of the stage
    uint4 x[2][MB], q[NB];
    auto read_x = [&](int buf, int j, int a) {
        x[j & 1][a] = *(const uint4 *)(smem + buf * T::STAGE + (wk * WM * MB + wm * MB + a) * 4096 + l16 * 256 + (((4 * j + lg) ^ l16) << 4));
    };
    auto read_w = [&](int buf) {
        const lds_char *sw = smem + buf * T::STAGE + T::XB + (wk * G + wn * NB) * 1024 + lane * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) q[b] = *(const uint4 *)(sw + b * 1024);
    };
    auto read_s = [&](int buf, int e, uint4 (&s4)[NB]) {
        const lds_char *ss = smem + buf * T::STAGE + T::XB + T::WB + ((wk * GR + e) * G + wn * NB) * 64 + lg * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) s4[b] = *(const uint4 *)(ss + b * 64);
    };
    auto dword = [](const uint4 &v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
    // Step j's MFMAs over the codes qc; the next step's X rows are read meanwhile, and
    // `side` does its work after each column group.
    auto step = [&](int j, const uint32_t (&qc)[NB], int xbuf, auto side) {
        const bool first = j % STEPS == 0;
        const f32x4_t zero = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 w = i4_frag(qc[b], bits);
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                if (b == 0) {
                    sum[a] = mfma16x16x32(ones, x[j & 1][a], first ? zero : sum[a]);
                    if (j < 3) read_x(xbuf, j + 1, a);
                }
                acc[a][b] = mfma16x16x32(w, x[j & 1][a], first ? zero : acc[a][b]);
            }
            side(b);
        }
    };
    // lane (g, l): columns 4g .. 4g+3 of row l
    auto close = [&](const uint4 (&s4)[NB]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t word[4] = {s4[b].x, s4[b].y, s4[b].z, s4[b].w};
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float s = __uint_as_float(word[v] & 0xFFFFFF00u), z = 16.f + (float)(word[v] & 0xFFu);
#pragma unroll
                for (int a = 0; a < MB; ++a) total[a][b][v] = fmaf(s, fmaf(-z, sum[a][v], acc[a][b][v]), total[a][b][v]);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < T::NS; ++s)
#pragma unroll
        for (int i = 0; i < T::UPW; ++i) issue_one(s, s, i);
    stage_ready(std::integral_constant<int, T::NS - 1>{});
    read_w(0);
#pragma unroll
    for (int a = 0; a < MB; ++a) read_x(0, 0, a);
    int buf = 0;
    for (int it = 0; it < nit; ++it) {
        uint32_t qc[NB];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int b = 0; b < NB; ++b) qc[b] = dword(q[b], j);
            step(j, qc, buf, [](int) {});
            if ((j + 1) % STEPS == 0) {
                uint4 s4[NB];
                read_s(buf, j / STEPS, s4);
                close(s4);
            }
        }
        // step 3's operands are in registers: this stage's buffer takes stage it + NS, and
        // the next stage's first operands are read while step 3 multiplies
        uint4 s4[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) qc[b] = q[b].w;
        read_s(buf, GR - 1, s4);
        const int next = buf == T::NS - 1 ? 0 : buf + 1, here = buf;
        stage_ready(std::integral_constant<int, T::NS - 2>{});
        read_w(next);
#pragma unroll
        for (int a = 0; a < MB; ++a) read_x(next, 0, a);
        constexpr int EACH = (T::UPW + NB - 1) / NB;
        step(3, qc, 0, [&](int b) {
#pragma unroll
            for (int e = 0; e < EACH; ++e)
                if (b * EACH + e < T::UPW) issue_one(it + T::NS, here, b * EACH + e);
        });
        close(s4);
        buf = next;
    }
    wait_vmcnt<0>();  // (the last loads fill zeros: nothing may land in the space used below)
    const auto store = [&](int row, int col, f32x4_t v) {  // lane (g, l): columns 4g .. 4g+3 of row l
        if (row >= rows || col >= P.N) return;
        if (P.part != nullptr)
            *(f32x4_t *)(P.part + ((size_t)ks * P.M + m0 + row) * P.N + col) = v;
        else
            *(uint2 *)(P.Y + (size_t)(m0 + row) * P.N + col) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    };
    if constexpr (WK > 1) {
        // the waves along k, in wave order
        __syncthreads();
        f32x4_t *red = (f32x4_t *)i4_smem;
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) red[((wk * WN + wn) * MB * NB + a * NB + b) * 64 + lane] = total[a][b];
        __syncthreads();
        for (int q = wave; q < WN * MB * NB; q += NW) {
            const int a = q / NB % MB, b = q % NB, n = q / (MB * NB);
            f32x4_t v = red[q * 64 + lane];
#pragma unroll
            for (int c = 1; c < WK; ++c) v += red[(c * WN * MB * NB + q) * 64 + lane];
            store(16 * a + l16, (c0 + n * NB + b) * 16 + 4 * lg, v);
        }
    } else {
        // alpha S B: ranks 32 a step, alpha S split into bf16 hi + lo
        if (!T::RIDE && P.S != nullptr) {
            const __amdgpu_buffer_rsrc_t rS = make_rsrc(P.S + (size_t)m0 * P.r, (uint64_t)rows * P.r * 4u);
            const __amdgpu_buffer_rsrc_t rB = make_rsrc(P.B, (uint64_t)P.r * P.N * 2u);
#pragma unroll 1
            for (int r0 = 0; r0 < P.r; r0 += 32) {
                const int rb = r0 + 8 * lg;
                uint4 hi[MB], lo[MB];
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    const uint32_t row = (uint32_t)((wm * MB + a) * 16 + l16);  // past the last row: past the resource
                    const uint32_t at = (row * (uint32_t)P.r + (uint32_t)rb) * 4u;
                    float v[8];
                    if (P.s_wide) {
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const f32x4_t s = __builtin_bit_cast(
                                f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rS, rb + e < P.r ? at + 4u * e : kOOB, 0, 0));
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[e + i] = P.alpha * s[i];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = P.alpha * __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                 rS, rb + e < P.r ? at + 4u * e : kOOB, 0, 0));
                    }
                    split_frag(v, hi[a], lo[a]);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int col = (c0 + wn * NB + b) * 16 + l16;
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
                            rB, rb + e < P.r && col < P.N ? ((uint32_t)(rb + e) * (uint32_t)P.N + (uint32_t)col) * 2u : kOOB, 0, 0);
                    const uint4 w = make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7]));
#pragma unroll
                    for (int a = 0; a < MB; ++a) {
                        total[a][b] = mfma16x16x32(w, hi[a], total[a][b]);
                        total[a][b] = mfma16x16x32(w, lo[a], total[a][b]);
                    }
                }
            }
        }
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) store((wm * MB + a) * 16 + l16, (c0 + wn * NB + b) * 16 + 4 * lg, total[a][b]);
    }
}

// S of a mixed batch of more than 64 rows, whose joining launch adds its partial sums: jobs
// of 64 rows and 32 ranks in a launch of their own (beside the product's tiles, which fill
// the CUs, they took longer).  100 x 4096 x 4096 of 4 segments 33 us with the bf16 layer's
// router and pass, 27 so, 1000 x 14336 x 4096 189 and 170; one adapter's pass is as fast.
constexpr int kSRows = 64, kSRanks = 32;
__global__ __launch_bounds__(512) void int4_s_kernel(SJobParams P) {
    extern __shared__ uint4 i4s_smem[];
    s_job<8, kSRows / 16, kSRanks / 16>(P, blockIdx.x, i4s_smem);
}

template <class T, bool RING>
hipError_t launch_t(const I4Params &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const dim3 grid((unsigned)(P.tiles_m * P.tiles_n * P.KS + P.jobs));
    if constexpr (RING) {
        const hipError_t e = allow_lds((const void *)int4_ring_kernel<T>, T::LDS, done);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((int4_ring_kernel<T>), grid, dim3(64 * T::NW), T::LDS, stream, P);
    } else {
        const hipError_t e = allow_lds((const void *)int4_gemm_kernel<T>, T::LDS, done);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((int4_gemm_kernel<T>), grid, dim3(64 * T::WK), T::LDS, stream, P);
    }
    return hipGetLastError();
}

// Tile shapes, and what a call with one costs.  `stage` and `row`: microseconds that a
// stage of WK blocks takes a work-group when `share` of them fill every CU, for groups
// of 32, 64 and 128 rows or more (a group is closed in fp32: a multiply-add for the zero
// and one for the scale), and what each row adds to it (the direct shapes read X once a
// wave).
using I4Launch = hipError_t (*)(const I4Params &, hipStream_t);
struct I4Kind {
    const char *name;  // in the timing pool
    I4Launch launch[3];  // groups of 32, 64, 128 rows or more (nullptr: not for these)
    int tm, tn, step, ranks;  // rows and columns of a tile, blocks of 128 rows of a stage, ranks of one job of S
    float stage[3], row;
    int share;
};
template <class T, bool RING, bool USED>
constexpr I4Launch launch_of() {
    if constexpr (USED) return launch_t<T, RING>;
    return nullptr;
}
// LEAST: the smallest groups that a shape is for (of smaller ones others are faster).
template <int MB, int NB, int WK, int LEAST>
constexpr I4Kind direct(const char *name, float s32, float s64, float s128, float row, int share) {
    using T = I4Tile<MB, NB, WK, 4>;
    return I4Kind{name, {launch_of<I4Tile<MB, NB, WK, 1>, false, LEAST <= 32>(), launch_of<I4Tile<MB, NB, WK, 2>, false, LEAST <= 64>(),
                         launch_t<T, false>}, 16 * MB, 16 * NB, WK, 16 * T::RT, {s32, s64, s128}, row, share};
}
template <int MB, int NB, int WM, int WN, int WK, int LEAST = 32>
constexpr I4Kind ring(const char *name, float s32, float s64, float s128, int share) {
    using T = I4Ring<MB, NB, WM, WN, WK, 4>;
    return I4Kind{name, {launch_of<I4Ring<MB, NB, WM, WN, WK, 1>, true, LEAST <= 32>(),
                         launch_of<I4Ring<MB, NB, WM, WN, WK, 2>, true, LEAST <= 64>(), launch_t<T, true>},
                  T::TM, T::TN, WK, T::RIDE ? 16 * T::RT : 0, {s32, s64, s128}, 0.f, share};
}
const I4Kind kKinds[] = {
    direct<1, 1, 8, 32>("int4_gemm 16x16", 1.75f, 1.20f, 0.80f, 0.07f, 2),
    direct<1, 2, 8, 64>("int4_gemm 16x32", 3.10f, 1.90f, 1.30f, 0.06f, 2),
    ring<1, 1, 1, 2, 4>("int4_ring 16x32", 1.04f, 0.78f, 0.67f, 2),
    ring<1, 2, 1, 4, 2>("int4_ring 16x128", 1.17f, 0.77f, 0.60f, 1),
    ring<2, 1, 1, 2, 4>("int4_ring 32x32", 0.98f, 0.70f, 0.65f, 1),
    ring<2, 2, 1, 2, 4>("int4_ring 32x64", 1.59f, 1.22f, 0.97f, 1),
    ring<3, 1, 1, 2, 4>("int4_ring 48x32", 1.20f, 1.15f, 1.05f, 1),
    ring<3, 2, 1, 2, 4>("int4_ring 48x64", 2.03f, 1.58f, 1.31f, 1),
    ring<4, 1, 1, 4, 2>("int4_ring 64x64", 1.30f, 1.05f, 0.95f, 1),
    ring<4, 2, 1, 4, 2>("int4_ring 64x128", 2.90f, 1.60f, 1.42f, 1),
    ring<4, 1, 2, 4, 1>("int4_ring 128x64", 1.33f, 1.05f, 0.95f, 1),
    ring<4, 2, 2, 4, 1>("int4_ring 128x128", 2.08f, 1.52f, 1.30f, 1),
    ring<8, 2, 2, 4, 1, 128>("int4_ring 256x128", 3.67f, 4.68f, 2.45f, 1),
};

}  // namespace

// The cheapest of the tile shapes, with k split as far as pays, and for more than 64 rows
// of expanding the weight for the bf16 product (kind 0), by a model of their times:
//   shape:  4.2 us, rounds of work-groups (stages x stage time each, with two more for
//           each 32 ranks that a tile of 128 rows or more adds itself, and at least their
//           share of the weight's bytes at 5.5 TB/s; 0.7 us between rounds); the
//           work-groups that form S 0.8 us, 7 where they keep some of the product's from
//           starting; a finishing launch 3.5 us, 0.25 a slice more, and its partial sums
//           at 5 TB/s (int4_finish at least 14 us a million outputs)
//   expand: expanded_us
//   S apart: a mixed batch's in partial sums 5 us, else by the bf16 layer's pass, 9 us, 14 for
//           a mixed batch, and X's bytes at 4 TB/s
// Measured in a graph, groups of 128, model in brackets: 1 x 4096 x 14336 9.8 us (9.9),
// 1 x 8192 x 28672 25.2 (26.9), 32 x 4096 x 14336 12.3 (11.6), 48 x 14336 x 4096 18.4
// (17.7), 64 x 4096 x 14336 19.9 (19.1), 33 x 28672 x 8192 44.3 (44.9), 100 x 4096 x 4096
// 18.1 (18.0; expanded 83), 256 x 4096 x 14336 46 (46; expanded 108), 1000 x 14336 x 4096
// 144 (150; expanded 269), 2000 x 4096 x 4096 83 (83; expanded 86), 2000 x 14336 x 4096
// expanded 274 (296).  More rows than fill one round of these shapes are left to the
// expansion: a work-group that unpacks for itself spends as long on that and on scaling as
// on its MFMAs (8192 x 4096 x 4096 344 us from 128 x 256 tiles, expanded 201), and neither
// closing a group behind the next one's MFMAs from two sets of accumulators nor a wave's
// priority moved that: the compiler spills.
static I4Plan find_plan(int64_t m, int64_t k, int64_t n, int64_t group, int r, int nseg) {
    I4Plan best{};
    // (offsets into X and a tile's codes stay below 2^31, and counts within an int)
    if (m <= 0 || m > (1 << 19) || k > kI4MaxK || n > kI4MaxN) return best;
    const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t k128 = cdiv(k, 128);
    const double bytes = (double)k * n * (0.5 + 4.0 / (double)std::min<int64_t>(group, 128));
    const double f1 = r > 0 ? (nseg > 0 ? 14.0 : 9.0) + (double)m * k * 2 / 4e6 : 0.0;
    double least = m <= kI4Rows ? 1e30 : expanded_us(m, n, k, (double)k * n) + f1;
    for (int kind = 1; kind <= (int)(sizeof(kKinds) / sizeof(kKinds[0])); ++kind) {
        const I4Kind &K = kKinds[kind - 1];
        const bool wide = K.ranks == 0;
        const int form = group == 32 ? 0 : group == 64 ? 1 : 2;
        const double stage = K.stage[form];
        if (K.launch[form] == nullptr || wide != (m > kI4Rows) || (!wide && m > K.tm) || (m <= 16 && K.tm > 16)) continue;
        I4Plan p{};
        p.kind = kind;
        p.tiles_m = (int)cdiv(m, K.tm);
        p.tiles_n = (int)cdiv(n, K.tn);
        const int64_t stages = cdiv(k128, K.step);
        const int64_t s_jobs = cdiv(k, kSK) * cdiv(m, kSRows) * cdiv(r, kSRanks) * std::max(nseg, 1);
        if (r > 0 && !wide) {
            const int64_t jobs = cdiv(k, kSK) * cdiv(r, K.ranks) * std::max(nseg, 1);
            if (nseg == 0 || jobs <= 1024) {
                p.SK = (int)cdiv(k, kSK);
                p.jobs = (int)cdiv(jobs, 8) * 8;
                p.spart_bytes = (size_t)p.SK * m * ((r + 3) / 4 * 4) * sizeof(float);
            }
        }
        for (int want = 1; want <= 16 && want <= stages; ++want) {
            const int64_t per = cdiv(stages, want);
            p.KS = (int)cdiv(stages, per);
            if (p.KS != want) continue;
            p.per = (int)(per * K.step);
            p.finish = p.KS > 1 || (r > 0 && (!wide || nseg > 0));
            p.part_bytes = p.finish ? (size_t)p.KS * m * n * sizeof(float) : 0;
            if (wide) {
                p.s_jobs = nseg > 0 && r > 0 && s_jobs <= 1024 ? (int)s_jobs : 0;
                p.SK = p.s_jobs > 0 ? (int)cdiv(k, kSK) : 0;
                p.spart_bytes = (size_t)p.SK * m * ((r + 3) / 4 * 4) * sizeof(float);
            }
            const int64_t groups = (int64_t)p.tiles_m * p.tiles_n * p.KS, slots = 256 * K.share;
            if (groups > (1 << 24)) continue;
            const double lora = wide && !p.finish ? 2.0 * (double)cdiv(r, 32) : 0.0;  // stages that the epilogue takes
            const double one = (double)per * (stage + K.row * (double)m) + lora * stage, each = bytes / 5.5e6 / (double)groups;
            const int64_t full = groups / slots, rest = groups % slots;
            double t = 4.2 + (double)full * std::max(one, each * (double)slots);
            // (a ring's stages take their time however few run, two work-groups of a CU share some of
            // it; the direct shapes' share of X's bytes shrinks)
            const double least_part = K.row > 0.f ? 0.45 : K.share > 1 ? 0.67 : 0.95;
            if (rest > 0) t += std::max(one * std::max(least_part, (double)rest / (double)slots), each * (double)rest);
            t += 0.7 * (double)(full + (rest > 0) - 1);
            if (p.jobs > 0) t += rest + p.jobs > slots ? 7.0 : 0.8;
            if (p.s_jobs > 0) t += 5.0 + 4.0 * (p.s_jobs / 512);
            else if (p.jobs == 0) t += f1;
            if (p.finish) {
                const double sums = 3.5 + (double)p.part_bytes * 2 / 5e6 + 0.25 * (p.KS - 1);
                t += wide && nseg == 0 ? std::max(sums, 14e-6 * (double)m * (double)n) : sums;
            }
            if (t < least) {
                least = t;
                best = p;
            }
        }
    }
    return best;
}

I4Plan int4_plan(int64_t m, int64_t k, int64_t n, int64_t group, int r, int nseg) {
    // (groups beyond the largest k are one and the same; r is at most 256)
    return remembered<I4Plan>(m, k, n, (int64_t)nseg << 32 | std::min<int64_t>(group, kI4MaxK) << 10 | r, [&] { return find_plan(m, k, n, group, r, nseg); });
}

hipError_t launch_int4_gemm(const I4Plan &pl, const void *X, const void *codes, const void *scales, int64_t group, int m, int k, int n,
                            const AdapterSource &src, const MxDropout &drop, float *S, void *Y, float *part, float *spart,
                            hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    I4Params P{};
    P.X = (const uint16_t *)X;
    P.M = m;
    P.K = k;
    P.tiles_m = pl.tiles_m;
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
    P.each = group < 128 ? 1 : (int)std::min<int64_t>(group / 128, s.k128);
    P.each_inv = P.each > 1 ? (uint32_t)((1ull << 32) / (uint32_t)P.each + 1) : 0u;
    P.tiles_n = pl.tiles_n;
    P.KS = pl.KS;
    P.per = pl.per;
    P.jobs = pl.jobs;
    if (!pl.finish && src.r > 0) {  // (the plan has S formed before)
        P.S = S;
        P.B = (const uint16_t *)src.B;
        P.alpha = src.alpha;
        P.s_wide = src.r % 4 == 0 && ((uintptr_t)S & 15) == 0;
    }
    if (pl.s_jobs > 0) {
        SJobParams Q = P;
        Q.tiles_m = (m + kSRows - 1) / kSRows;
        const int slot = prof_begin("int4_s", stream);
        hipLaunchKernelGGL(int4_s_kernel, dim3((unsigned)pl.s_jobs), dim3(512), 8 * (kSRows / 16) * (kSRanks / 16) * 1024, stream, Q);
        prof_end(slot, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const I4Kind &K = kKinds[pl.kind - 1];
    const int slot = prof_begin(K.name, stream);
    const hipError_t e = K.launch[group == 32 ? 0 : group == 64 ? 1 : 2](P, stream);
    prof_end(slot, stream);
    if (e != hipSuccess || !pl.finish) return e;
    // (int4_finish's work-groups of 32 columns pay where few rows leave CUs idle: 1000 x 4096 x 4096 of 4
    // segments 120 us with it, 76 with the join's of 128)
    if (m > kI4Rows && src.table != nullptr) return launch_mxfp4_join(true, part, pl.KS, m, n, S, src.r, pl.SK, spart, nullptr, src, Y, stream);
    return launch_int4_finish(part, pl.KS, m, n, S, pl.SK, spart, src, Y, stream);
}

}  // namespace lora
