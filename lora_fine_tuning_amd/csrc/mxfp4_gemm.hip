// Y = X W' + alpha S B for few and middling numbers of rows, W' in MXFP4
// (mxfp4_kernels.hip describes the storage).
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
// NS - 1 stages ahead.  X rows take 256 bytes a chunk; piece 4 g + j (16 bytes)
// of row i sits at place (4 j + g) ^ (i mod 16).  A 16-byte read serves lanes
// 0-3, 12-15 and 20-27 (and so on) together: with g in the low bits of the place
// those 16 lanes fall on 16 different bank ranges (with j there, on 8).  Waves
// along k are added in LDS in wave order.  Where the tiles would leave CUs idle,
// work-groups split k further: each slice writes fp32 partial sums and a finishing
// launch adds them in slice order.
//
// With the shapes for up to 64 rows the adapter rides along: keep and keep.X A
// are formed by further work-groups of the same launch (partial sums over 1024 of
// k each), and the finishing launch adds those, writes S and adds alpha S B.  F1
// took 9 to 14 us before the product.  A mixed batch's segments have such
// work-groups too, up to 1024 of them (every segment one for each row tile that it
// could fill, which most leave at once), and mxfp4_join.hip finishes.  With the
// shapes for more rows F1 forms S first, and they add alpha S B in their own
// epilogue, as rank-deep MFMA steps, where k is not split.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

struct MxGemmParams {
    const uint16_t *X;
    const uint8_t *codes, *scales;
    uint16_t *Y;   // KS == 1
    float *part;   // KS > 1: [KS][M][N]
    int M, N, K;
    int groups, blocks;  // N16, KB
    int tiles_m, tiles_n;
    int KS, per;         // slices of k, stages of a slice
    const float *S;      // the epilogue's LoRA term: M x r fp32 (nullptr: none)
    const uint16_t *B;   // r x N
    int r;
    float alpha;
    // partial sums of S = X A by further work-groups
    const uint16_t *A;
    float *spart;     // [SK][M][rs], rs = r rounded up to 4
    int rs, SK, jobs; // partial sums; work-groups that form them (a multiple of 8)
    uint32_t *keep;   // their dropout mask, M x ceil(K / 32) words, written here (nullptr: none)
    uint64_t seed, offset;
    uint32_t drop;    // threshold of the mask's 16-bit numbers
    // rows in segments with an adapter each (nullptr: one adapter); r is then the largest rank
    const lora_adapter *adapters;
    const int64_t *seg_off;
    const int32_t *seg_adapter;
    int num_adapters, nseg;
};

constexpr int kSK = 1024;  // k of one partial sum of S

template <int WM_, int WN_, int WK_, int MB_, int NB_, int XR_, int NS_>
struct MxTile {
    static constexpr int WM = WM_, WN = WN_, WK = WK_, MB = MB_, NB = NB_, XR = XR_, NS = NS_;
    static constexpr int NW = WM * WN * WK, TM = 16 * WM * MB, TN = 16 * WN * NB, KW = 128 * WK;
    static constexpr int G = WN * NB;                  // column groups
    static constexpr int XU = XR * WK / 4, WU = G * WK, SU = (G * WK + 15) / 16;  // 1 KiB loads of a stage
    static constexpr int XPW = (XU + NW - 1) / NW, WPW = (WU + NW - 1) / NW, UPW = XPW + WPW + 1;  // per wave
    static constexpr int XB = XU * 1024, WB = WU * 1024, STAGE = XB + WB + SU * 1024;
    static constexpr int SPARE = NS * STAGE;  // 1 KiB that surplus loads fill with zeros
    static constexpr int RED = (WK - 1) * WM * WN * MB * NB * 1024;
    static constexpr int LDS = SPARE + 1024 > RED ? SPARE + 1024 : RED;
    static constexpr int SHARE = 160 * 1024 / LDS < 3 ? 160 * 1024 / LDS : 3;  // work-groups that a CU holds
    // 16-rank tiles of a job of S (every operand of it is in registers at once: few
    // where SHARE work-groups have to fit a CU)
    static constexpr int RT = SHARE > 2 ? 1 : 2;
    static constexpr bool RIDE = WM == 1;  // the adapter's S rides along, a second launch adds alpha S B
    static_assert(SU <= NW && LDS <= 160 * 1024, "tile does not fit");
};

// One work-group's share of keep.X A: 1024 of k (128 a wave), up to TM rows of one
// adapter and 16 RT ranks.  X's rows and A's columns come straight from memory
// (8 two-byte loads make a 16-rank operand: A's rows are r values long), every
// load of a wave before its first use; the waves are added in LDS in wave order.
// A lane's 8 elements of X are one counter of the dropout mask and one byte of
// keep, which the first rank tile's work-groups write.
template <class T>
__device__ __forceinline__ void s_job(const MxGemmParams &P, int job, uint4 *smem) {
    constexpr int MB = T::MB, RT = T::RT;
    static_assert(T::NW == 8 && T::WM == 1 && MB * RT <= 8 && 8 * MB * RT * 1024 <= T::LDS, "no room for the partial sums");
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
        m0 = (int)min(max((int64_t)0, P.seg_off[seg]), (int64_t)P.M) + rest % P.tiles_m * T::TM;
        mend = (int)min(max((int64_t)0, P.seg_off[seg + 1]), (int64_t)P.M);
        if (m0 >= mend) return;
        A = (const uint16_t *)ad.A;
        r = ad.r;
        drop = drop_threshold(ad.p);
    } else {
        m0 = rest % P.tiles_m * T::TM;
    }
    const int r0 = rest / P.tiles_m * 16 * RT;
    if (r0 >= r) return;  // (the count is rounded up)
    mend = min(mend, m0 + T::TM);
    const int k0 = ks * kSK + wave * (kSK / 8);
    // rows past the end read as zeros; the host keeps A under 2 GiB
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(P.X + (size_t)m0 * P.K, (uint64_t)(mend - m0) * P.K * 2u);
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, (uint64_t)P.K * r * 2u);
    f32x4_t acc[MB][RT];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int J = kSK / 8 / 32;
    uint4 x[J][MB];
    uint32_t h[J][RT][8];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int k = k0 + 32 * j + 8 * lg;
#pragma unroll
        for (int a = 0; a < MB; ++a)
            x[j][a] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                          rX, k < P.K ? ((uint32_t)(16 * a + l16) * (uint32_t)P.K + (uint32_t)k) * 2u : kOOB, 0, 0));
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int rank = r0 + 16 * t + l16;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[j][t][e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
                    rA, rank < r && k < P.K ? ((uint32_t)(k + e) * (uint32_t)r + (uint32_t)rank) * 2u : kOOB, 0, 0);
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
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const uint32_t *q = h[j][t];
            const uint4 w = make_uint4(pack2(q[0], q[1]), pack2(q[2], q[3]), pack2(q[4], q[5]), pack2(q[6], q[7]));
#pragma unroll
            for (int a = 0; a < MB; ++a) acc[a][t] = mfma16x16x32(w, x[j][a], acc[a][t]);
        }
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
    for (int c = 1; c < 8; ++c) sum += red[(c * MB * RT + wave) * 64 + lane];
    const int row = m0 + 16 * (wave / RT) + l16, rank = r0 + 16 * (wave % RT) + 4 * lg;
    if (row >= mend) return;
    if (rank < P.rs) *(f32x4_t *)(P.spart + ((size_t)ks * P.M + row) * P.rs + rank) = sum;  // (zeros past r)
}

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
    if constexpr (T::RIDE) {
        if (id < P.jobs) return s_job<T>(P, id, mx_smem);
        id -= P.jobs;
    }
    id = xcd_order(id, total);
    int tm = 0, tn = id, ks = 0;  // (the divisions are skipped where there is nothing to divide)
    if (P.tiles_m > 1) tn = id / P.tiles_m, tm = id - tn * P.tiles_m;
    if (P.KS > 1) ks = tn / P.tiles_n, tn -= ks * P.tiles_n;
    const int m0 = tm * T::TM, n0 = tn * T::TN, g0 = tn * G;
    const int k0 = ks * P.per * T::KW;
    const int nit = min(P.per, (P.K - k0 + T::KW - 1) / T::KW);  // >= 1: the host sizes the slices

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.K * 2u, group_bytes = (uint32_t)P.blocks * 256u;
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.K, (uint32_t)min(P.M - m0, T::TM) * row_bytes);
    const uint32_t ng = (uint32_t)min(P.groups - g0, G);
    const sgpr4_t dW = make_desc(P.codes + (size_t)g0 * group_bytes, ng * group_bytes);
    const sgpr4_t dS = make_desc(P.scales + (size_t)g0 * (group_bytes / 16), ng * (group_bytes / 16));

    // This wave's loads of a stage: XPW of X, WPW of codes, one of scales; where a
    // kind has no load left for a wave, zeros into the spare space, so that every
    // wave counts the same loads.  xo, wo, so: byte offsets at stage 0 (kOOB: zeros);
    // xk, wk32, sk32: the k a lane reads in a wave's first chunk.
    const int xrow4 = lane >> 4;
    int xk;
    uint32_t xo[T::XPW], wo[T::WPW], so = kOOB;
    {
        const int place = (lane & 15) ^ ((4 * (wave % (XR < 16 ? XR / 4 : 4)) + xrow4) & 15);
        xk = k0 + 8 * ((place & 3) * 4 + (place >> 2));
    }
    const uint32_t xlane = (uint32_t)xrow4 * row_bytes + (uint32_t)xk * 2u;
    auto xchunk = [&](int i) { return (wave + T::NW * i) / (XR / 4); };
#pragma unroll
    for (int i = 0; i < T::XPW; ++i) {
        const int u = wave + T::NW * i, row = u % (XR / 4) * 4;
        xo[i] = u < T::XU && row + xrow4 < P.M - m0 ? xlane + (uint32_t)row * row_bytes + (uint32_t)xchunk(i) * 256u : kOOB;
    }
    const uint32_t wlane = (uint32_t)(k0 / 32) * 256u + (uint32_t)lane * 16u;
    auto wchunk = [&](int i) { return (wave + T::NW * i) / G; };
#pragma unroll
    for (int i = 0; i < T::WPW; ++i) {
        const int u = wave + T::NW * i, g = u % G;
        wo[i] = u < T::WU && g0 + g < P.groups ? wlane + (uint32_t)g * group_bytes + (uint32_t)wchunk(i) * 1024u : kOOB;
    }
    const int sq = wave * 16 + (lane >> 2), schunk = sq / G, sg = sq % G;
    if (sq < G * WK && g0 + sg < P.groups)
        so = (uint32_t)sg * (group_bytes / 16) + (uint32_t)(k0 / 32 + 4 * schunk + (lane & 3)) * 16u;
    // One load of stage `it` into buffer `buf`.  A stage that lies inside K whole
    // advances by the scalar offset alone; the last ones test each lane's k.
    const int nfull = min(nit, (P.K - k0) / T::KW), kpad = P.blocks * 32;
    auto issue_one = [&](int it, int buf, int i) {
        const uint32_t base = lds0 + (uint32_t)buf * T::STAGE + (uint32_t)wave * 1024u, spare = lds0 + T::SPARE;
        const int dk = it < nit ? it * T::KW : 0x20000000;  // past every limit
        const bool whole = it < nfull;
        if (i < T::XPW) {
            dma16_at(dX, whole || xk + 128 * xchunk(i) + dk < P.K ? xo[i] : kOOB, (uint32_t)dk * 2u,
                     T::XU % T::NW == 0 || wave + T::NW * i < T::XU ? base + T::NW * i * 1024u : spare);
        } else if (i < T::XPW + T::WPW) {
            const int j = i - T::XPW;
            dma16_at(dW, whole || k0 + 32 * lg + 128 * wchunk(j) + dk < kpad ? wo[j] : kOOB, (uint32_t)dk * 8u,
                     T::WU % T::NW == 0 || wave + T::NW * j < T::WU ? base + T::XB + T::NW * j * 1024u : spare);
        } else {
            dma16_at(dS, whole || k0 + 32 * (lane & 3) + 128 * schunk + dk < kpad ? so : kOOB, (uint32_t)dk / 2u,
                     wave < T::SU ? base + T::XB + T::WB : spare);
        }
    };
    auto issue = [&](int it, int buf) {
#pragma unroll
        for (int i = 0; i < T::UPW; ++i) issue_one(it, buf, i);
    };

    f32x4_t acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    int xrow[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) xrow[a] = ((wm * MB + a) * 16 + l16) & (XR < 16 ? XR - 1 : -1);

    // x[j % 2] holds X's rows of step j, q and sc the wave's codes and scales of
    // the stage, w the operand of the next column group.
    uint4 x[2][MB], q[NB];
    float sc[NB];
    uint32_t xplace[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        xplace[j] = (uint32_t)(wk * XR * 256 + xrow[0] * 256 + (((4 * j + lg) ^ (xrow[0] & 15)) << 4));
    auto read_x = [&](int buf, int j, int a) {  // (rows 16 apart share a place)
        x[j & 1][a] = *(const uint4 *)(smem + buf * T::STAGE + xplace[j] + a * 4096);
    };
    auto read_w = [&](int buf) {
        const lds_char *sw = smem + buf * T::STAGE + T::XB + (wk * G + wn * NB) * 1024 + lane * 16;
        const lds_char *ss = smem + buf * T::STAGE + T::XB + T::WB + (wk * G + wn * NB) * 64 + lane;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            q[b] = *(const uint4 *)(sw + b * 1024);
            sc[b] = mx_scale(*(const uint8_t *)(ss + b * 64));
        }
    };
    auto dword = [](const uint4 &v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
    // Step j's MFMAs, each followed by a share of the work that is due meanwhile:
    // the next group's conversions (codes `qc`, scale `c` of this step, or of step
    // j + 1's first group), the next step's X rows, and what `side` does.
    uint4 w;
    auto step = [&](int j, const uint32_t (&qc)[NB], const float (&c)[NB], uint32_t qnext, float cnext, int xbuf, auto side) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 now = w;
            const uint32_t src = b + 1 < NB ? qc[b + 1 < NB ? b + 1 : 0] : qnext;
            const float scale = b + 1 < NB ? c[b + 1 < NB ? b + 1 : 0] : cnext;
            uint32_t n[4];
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                acc[a][b] = mfma16x16x32(now, x[j & 1][a], acc[a][b]);
#pragma unroll
                for (int e = a * 4 / MB; e < (a + 1) * 4 / MB; ++e) n[e] = mx_pair(src, scale, e);
                if (b == 0 && j < 3) read_x(xbuf, j + 1, a);
                side(b * MB + a);
                __builtin_amdgcn_sched_barrier(0);
            }
            w = make_uint4(n[0], n[1], n[2], n[3]);
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

#pragma unroll 1
    for (int s = 0; s < NS; ++s) issue(s, s);
    stage_ready(std::integral_constant<int, NS - 1>{});
    read_w(0);
#pragma unroll
    for (int a = 0; a < MB; ++a) read_x(0, 0, a);
    int buf = 0;
    for (int it = 0; it < nit; ++it) {
        w = mx_frag(q[0].x, sc[0]);
        uint32_t qc[NB];
        float c[NB];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int b = 0; b < NB; ++b) qc[b] = dword(q[b], j);
            step(j, qc, sc, dword(q[0], j + 1), sc[0], buf, [](int) {});
        }
        // step 3's operands are in registers: this stage's buffer takes stage it + NS, and
        // the next stage's first operands are read while step 3 multiplies
#pragma unroll
        for (int b = 0; b < NB; ++b) qc[b] = q[b].w, c[b] = sc[b];
        const int next = buf == NS - 1 ? 0 : buf + 1, here = buf;
        stage_ready(std::integral_constant<int, NS - 2>{});
        read_w(next);
#pragma unroll
        for (int a = 0; a < MB; ++a) read_x(next, 0, a);
        constexpr int EACH = (T::UPW + MB * NB - 1) / (MB * NB);
        step(3, qc, c, 0u, 1.f, 0, [&](int i) {
#pragma unroll
            for (int e = 0; e < EACH; ++e)
                if (i * EACH + e < T::UPW) issue_one(it + NS, here, i * EACH + e);
        });
        buf = next;
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
#pragma unroll 1
        for (int c = 0; c < WK - 1; ++c)
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[a][b] += __builtin_bit_cast(f32x4_t, red[((c * T::WM * WN + w2) * MB * NB + a * NB + b) * 64 + lane]);
    }

    // alpha S B: ranks 32 a step, alpha S split into bf16 hi + lo
    if (!T::RIDE && P.S != nullptr) {
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

    // lane (g, l): columns 4g .. 4g+3 of a group, row l.  Rows past M and columns
    // past N are dropped by the buffer's bounds (the host keeps a tile's rows
    // under 2^31 bytes).
    const bool direct = P.part == nullptr;
    const int rows = min(P.M - m0, T::TM);
    const __amdgpu_buffer_rsrc_t rY =
        direct ? make_rsrc(P.Y + (size_t)m0 * P.N, (uint64_t)rows * P.N * 2u)
               : make_rsrc(P.part + ((size_t)ks * P.M + m0) * P.N, (uint64_t)rows * P.N * 4u);
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const uint32_t row = (uint32_t)((wm * MB + a) * 16 + l16);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int col = n0 + (wn * NB + b) * 16 + 4 * lg;
            const uint32_t at = row < (uint32_t)rows && col < P.N ? row * (uint32_t)P.N + (uint32_t)col : kOOB / 4;
            if (direct)
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2_t{pack_bf16x2(acc[a][b][0], acc[a][b][1]), pack_bf16x2(acc[a][b][2], acc[a][b][3])}, rY, at * 2u, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[a][b]), rY, at * 4u, 0, 0);
        }
    }
}

// Y = the k slices' partial sums in slice order, and alpha S B, rounded.  A
// work-group takes 16 rows of 128 columns, a wave 32 columns: the sums start the
// accumulators, then 32 ranks an MFMA step, alpha S split into bf16 hi + lo.  S
// (the sum of SK partials in order, or given) goes to LDS first, and the first
// column tile writes a summed S out.  (Adding the ranks with plain FMAs took twice
// the kernel's time at rank 64: one wave a SIMD, 20 instructions a rank.)
struct MxFinishParams {
    const float *part;
    int KS, M, N;
    const float *spart;  // [SK][M][rs] or, with SK == 0, S itself; r == 0: no adapter
    int SK, r, rs;
    const uint16_t *B;
    float alpha, undrop;  // undrop: 1 / (1 - p), the scale of a summed S
    float *S;
    uint16_t *Y;
};

constexpr int kFinishRanks = 64;  // ranks of B in LDS at a time

__global__ __launch_bounds__(256) void mxfp4_finish_kernel(MxFinishParams P) {
    __shared__ float sS[16][260];  // alpha S, zero past r (rows 16 bytes past a bank period)
    __shared__ uint4 sB[kFinishRanks * 16];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row0 = (int)blockIdx.y * 16, n0 = (int)blockIdx.x * 128;
    // B's first ranks are on their way while S and the product are summed: 16-byte
    // pieces, 16 a rank (B may be unaligned)
    uint4 b[kFinishRanks / 16];
    const int br = tid >> 4, bc = tid & 15;
    auto load_b = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kFinishRanks / 16; ++i) {
            b[i] = make_uint4(0u, 0u, 0u, 0u);
            const int r = r0 + 16 * i + br;
            if (r < P.r && n0 + 8 * bc < P.N) __builtin_memcpy(&b[i], P.B + (size_t)r * P.N + n0 + 8 * bc, 16);
        }
    };
    const int rpad = (P.r + 31) & ~31;
    if (P.r > 0) {
        load_b(0);
        const int row = row0 + br;  // 16 threads a row of S, 4 ranks at a time
#pragma unroll 1
        for (int r = 4 * bc; r < rpad; r += 64) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < P.M && r < P.r) {
                if (P.SK > 0) {
                    const float *ps = P.spart + (size_t)row * P.rs + r;
                    const size_t part = (size_t)P.M * P.rs;
#pragma unroll 1
                    for (int c = 0; c < P.SK; c += 8) {
                        float4 u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[e] = c + e < P.SK ? *(const float4 *)(ps + (c + e) * part) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v.x += u[e].x, v.y += u[e].y, v.z += u[e].z, v.w += u[e].w;
                    }
                    v.x *= P.undrop, v.y *= P.undrop, v.z *= P.undrop, v.w *= P.undrop;
                    if (blockIdx.x == 0) {
                        float *d = P.S + (size_t)row * P.r + r;
                        d[0] = v.x;
                        if (r + 1 < P.r) d[1] = v.y;
                        if (r + 2 < P.r) d[2] = v.z;
                        if (r + 3 < P.r) d[3] = v.w;
                    }
                } else {
                    const float *s = P.spart + (size_t)row * P.r + r;
                    v.x = s[0];
                    if (r + 1 < P.r) v.y = s[1];
                    if (r + 2 < P.r) v.z = s[2];
                    if (r + 3 < P.r) v.w = s[3];
                }
            }
            *(float4 *)&sS[br][r] = make_float4(P.alpha * v.x, P.alpha * v.y, P.alpha * v.z, P.alpha * v.w);
        }
    }
    // lane (g, l): row l, columns 4g .. 4g+3 of the wave's two 16-column tiles
    const int row = row0 + l16, col = n0 + 32 * wave + 4 * lg;
    f32x4_t acc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
    const bool live0 = row < P.M && col < P.N, live1 = row < P.M && col + 16 < P.N;
    const size_t slice = (size_t)P.M * P.N;
    const float *src = P.part + (size_t)row * P.N + col;
#pragma unroll 1
    for (int s = 0; s < P.KS; s += 4) {
        f32x4_t t[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e][0] = t[e][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (live0 && s + e < P.KS) t[e][0] = *(const f32x4_t *)(src + (s + e) * slice);
            if (live1 && s + e < P.KS) t[e][1] = *(const f32x4_t *)(src + (s + e) * slice + 16);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0] += t[e][0], acc[1] += t[e][1];
    }
    // B's pieces in 256-byte rows, piece c of rank k at c ^ place(k): the transposing
    // reads of ranks {0-3, 8-11} mod 16 by a half-wave then fall on different banks
    auto place = [](int k) { return (4 * (k & 3)) ^ (2 * ((k >> 3) & 1)); };
#pragma unroll 1
    for (int r0 = 0; r0 < P.r; r0 += kFinishRanks) {
        if (r0 > 0) __syncthreads();  // the last ranks have been read
#pragma unroll
        for (int i = 0; i < kFinishRanks / 16; ++i) sB[(16 * i + br) * 16 + (bc ^ place(16 * i + br))] = b[i];
        __syncthreads();
        if (r0 + kFinishRanks < P.r) load_b(r0 + kFinishRanks);
#pragma unroll 1
        for (int q = 0; q < kFinishRanks && r0 + q < P.r; q += 32) {
            float v[8];
            *(float4 *)&v[0] = *(const float4 *)&sS[l16][r0 + q + 8 * lg];
            *(float4 *)&v[4] = *(const float4 *)&sS[l16][r0 + q + 8 * lg + 4];
            uint4 hi, lo;
            split_frag(v, hi, lo);
            const int k = q + 8 * lg + (l16 >> 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int c = 4 * wave + 2 * t + ((l16 & 3) >> 1);
                const lds_char *p = (const lds_char *)sB + k * 256 + ((c ^ place(k)) << 4) + (l16 & 1) * 8;
                const uint2 w0 = lds_read_tr4(p), w1 = lds_read_tr4(p + 1024);
                const uint4 w = make_uint4(w0.x, w0.y, w1.x, w1.y);
                acc[t] = mfma16x16x32(w, hi, acc[t]);
                acc[t] = mfma16x16x32(w, lo, acc[t]);
            }
        }
    }
    uint16_t *dst = P.Y + (size_t)row * P.N + col;
    if (live0) *(uint2 *)dst = make_uint2(pack_bf16x2(acc[0][0], acc[0][1]), pack_bf16x2(acc[0][2], acc[0][3]));
    if (live1) *(uint2 *)(dst + 16) = make_uint2(pack_bf16x2(acc[1][0], acc[1][1]), pack_bf16x2(acc[1][2], acc[1][3]));
}

template <class T>
hipError_t launch_t(const MxGemmParams &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void *)mxfp4_gemm_kernel<T>, T::LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mxfp4_gemm_kernel<T>), dim3((unsigned)(P.tiles_m * P.tiles_n * P.KS + P.jobs)), dim3(64 * T::NW),
                       T::LDS, stream, P);
    return hipGetLastError();
}

// Tile shapes, and what a call with one costs.  `stage`: microseconds a stage
// takes a work-group when a full round of them runs (measured at k = 14336 and
// 28672, 2.4 GHz); `share`: work-groups that a CU holds.
struct MxKind {
    const char *name;  // in the timing pool
    hipError_t (*launch)(const MxGemmParams &, hipStream_t);
    int tm, tn, kw, ranks;  // rows and columns of a tile; ranks: of one job of S, 0 where S does not ride along
    float stage;
    int share;
};
template <class T>
constexpr MxKind kind_of(const char *name, float stage) {
    return MxKind{name, launch_t<T>, T::TM, T::TN, T::KW, T::RIDE ? 16 * T::RT : 0, stage, T::SHARE};
}
const MxKind kKinds[] = {
    kind_of<MxTile<1, 1, 8, 1, 1, 4, 3>>("mxfp4_gemm 4x16", 0.36f),
    kind_of<MxTile<1, 2, 4, 1, 1, 4, 3>>("mxfp4_gemm 4x32", 0.31f),
    kind_of<MxTile<1, 1, 8, 1, 1, 16, 3>>("mxfp4_gemm 16x16", 0.60f),
    kind_of<MxTile<1, 2, 4, 1, 2, 16, 3>>("mxfp4_gemm 16x64", 0.53f),
    kind_of<MxTile<1, 2, 4, 2, 1, 32, 3>>("mxfp4_gemm 32x32", 0.61f),
    kind_of<MxTile<1, 4, 2, 2, 2, 32, 3>>("mxfp4_gemm 32x128", 0.67f),
    kind_of<MxTile<1, 4, 2, 3, 2, 48, 3>>("mxfp4_gemm 48x128", 0.78f),
    kind_of<MxTile<1, 4, 2, 4, 2, 64, 3>>("mxfp4_gemm 64x128", 1.00f),
    kind_of<MxTile<2, 4, 1, 2, 4, 64, 3>>("mxfp4_gemm 64x256", 0.98f),
    kind_of<MxTile<2, 4, 1, 4, 4, 128, 3>>("mxfp4_gemm 128x256", 1.65f),
};

}  // namespace

// The cheapest of the tile shapes, each with k split as far as pays, and of
// expanding the weight for the bf16 product, by a model of their times:
//   shape:  3.5 us + rounds of work-groups (stages x stage time + 1 us each, at least
//           their share of the weight's bytes at 6 TB/s); a finishing launch 3.5 us
//           and its partial sums at 8 TB/s
//   expand: expanded_us
//   S apart: 9 us and X's bytes at 4 TB/s (its work-groups beside a shape's add to the rounds)
// Measured, model in brackets: 1 x 4096 x 4096 5.6 us (5.9), 48 x 14336 x 4096 16.5
// (16), 300 x 14336 x 4096 45 (48), 1000 x 4096 x 4096 35 (36), 2000 x 4096 x 4096 59
// (57; expanded 86), 8192 x 4096 x 4096 expanded 201 (192; packed 245).
static MxGemmPlan find_plan(int64_t m, int64_t k, int64_t n, int r, MxForm form, int nseg) {
    MxGemmPlan best{};
    // (a tile's offsets stay below 2^31 within these)
    if (m <= 0 || k > (1 << 20) || n > (1 << 21) || m > (1 << 19)) return best;
    const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const double weight = (double)k * n;
    const double f1 = r > 0 ? (form == kMxMixed ? 14.0 : 9.0) + (double)m * k * 2 / 4e6 : 0.0;
    double least = expanded_us(m, n, k, weight) + f1;
    for (int kind = 1; kind <= (int)(sizeof(kKinds) / sizeof(kKinds[0])); ++kind) {
        const MxKind &K = kKinds[kind - 1];
        if ((kind <= 2 && m > 4) || (kind <= 4 && m > 16)) continue;  // (4 rows in LDS; columns too narrow)
        MxGemmPlan p{};
        p.kind = kind;
        p.tiles_m = (int)cdiv(m, K.tm);
        p.tiles_n = (int)cdiv(n, K.tn);
        const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, stages = cdiv(k, K.kw);
        if (tiles > (1 << 20)) continue;
        // a mixed batch's segments take a job for every row tile that they could fill
        const int64_t jobs = K.ranks > 0 ? cdiv(k, kSK) * p.tiles_m * cdiv(r, K.ranks) * (form == kMxMixed ? nseg : 1) : 0;
        if (r > 0 && jobs > 0 && (form == kMxPlain || jobs <= 1024)) {
            p.SK = (int)cdiv(k, kSK);
            p.jobs = (int)cdiv(jobs, 8) * 8;
            p.spart_bytes = (size_t)p.SK * m * ((r + 3) / 4 * 4) * sizeof(float);
        }
        for (int want = 1; want <= 16 && want <= stages; ++want) {
            p.per = (int)cdiv(stages, want);
            p.KS = (int)cdiv(stages, p.per);
            if (p.KS != want) continue;
            p.finish = p.KS > 1 || (r > 0 && (K.ranks > 0 || form == kMxMixed));
            p.part_bytes = p.finish ? (size_t)p.KS * m * n * sizeof(float) : 0;
            const int64_t groups = tiles * p.KS + p.jobs, slots = 256 * K.share;
            double t = 3.5 + rounds_us(groups, slots, p.per * K.stage + 1.0, weight) + (p.jobs == 0 ? f1 : 0.0);
            if (p.finish) t += 3.5 + (double)p.part_bytes * 2 / 8e6;
            if (t < least) {
                least = t;
                best = p;
            }
        }
    }
    return best;
}

MxGemmPlan mx_gemm_plan(int64_t m, int64_t k, int64_t n, int r, MxForm form, int nseg) {
    return remembered<MxGemmPlan>(m, k, n, nseg * (1LL << 32) + 4 * r + (int)form,
                                  [&] { return find_plan(m, k, n, r, form, nseg); });
}

hipError_t launch_mxfp4_gemm(const MxGemmPlan &pl, const void *X, const void *codes, const void *scales, int m, int k,
                             int n, const AdapterSource &src, const MxDropout &drop, float *S, void *Y, float *part,
                             float *spart, hipStream_t stream) {
    const int r = src.r;
    MxGemmParams P{};
    P.X = (const uint16_t *)X;
    P.codes = (const uint8_t *)codes;
    P.scales = (const uint8_t *)scales;
    P.Y = (uint16_t *)Y;
    P.part = pl.finish ? part : nullptr;
    P.M = m;
    P.N = n;
    P.K = k;
    P.groups = (int)mx_groups(n);
    P.blocks = (int)mx_blocks(k);
    P.tiles_m = pl.tiles_m;
    P.tiles_n = pl.tiles_n;
    P.KS = pl.KS;
    P.per = pl.per;
    P.S = r > 0 && !pl.finish ? S : nullptr;
    P.A = (const uint16_t *)src.A;
    P.spart = spart;
    P.SK = pl.SK;
    P.rs = (r + 3) / 4 * 4;
    P.B = (const uint16_t *)src.B;
    P.r = r;
    P.alpha = src.alpha;
    P.jobs = pl.jobs;
    P.keep = drop.keep;
    P.seed = drop.seed;
    P.offset = drop.offset;
    P.drop = drop_threshold(src.p);
    P.adapters = src.table;
    P.seg_off = src.seg_off;
    P.seg_adapter = src.seg_adapter;
    P.num_adapters = src.num_adapters;
    P.nseg = src.num_segments;
    int slot = prof_begin(kKinds[pl.kind - 1].name, stream);
    const hipError_t e = kKinds[pl.kind - 1].launch(P, stream);
    prof_end(slot, stream);
    if (e != hipSuccess || !pl.finish) return e;
    if (src.table != nullptr)
        return launch_mxfp4_join(true, part, pl.KS, m, n, S, r, pl.SK, spart, nullptr, src, Y, stream);
    const MxFinishParams F{part, pl.KS, m, n, pl.SK > 0 ? spart : S, pl.SK, r, P.rs, (const uint16_t *)src.B, src.alpha, drop_scale(src.p), S,
                           (uint16_t *)Y};
    slot = prof_begin("mxfp4_finish", stream);
    hipLaunchKernelGGL(mxfp4_finish_kernel, dim3((unsigned)((n + 127) / 128), (unsigned)((m + 15) / 16)), dim3(256), 0, stream,
                       F);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
