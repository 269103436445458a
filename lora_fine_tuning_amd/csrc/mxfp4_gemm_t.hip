// dX = dY W'^T + s keep.(dS A^T) for few and middling numbers of rows, W' in
// MXFP4 (mxfp4_kernels.hip describes the storage).
//
// The contraction runs over n, across the columns that the codes are stored by,
// so the codes pass through LDS twice: as they are stored, by direct-to-LDS
// loads, and expanded to bf16.  A wave owns 32 columns of dX, one block of rows
// of W', so a lane expands whole blocks (16 bytes of codes, one scale): 64
// columns of W' at a time go to the wave's own 4 KiB as 64 rows of 32 bf16, and
// transposing reads give the MFMA operand, 8 n of one column of dX.  No other
// wave reads it, so the expansion needs no barrier.
//
// A work-group covers 16 WM MB rows and 128 columns of dX; its waves split the
// rows (WM), the columns (4) and each stage's n (WK chunks of 128).  dY's tile,
// the ring and the split of n over work-groups are as in the forward product;
// mxfp4_join.hip adds the slices and the adapters' term.
//
// Bound, at few rows, by the chain of a stage (codes out of LDS, converted, into
// LDS, out again): 1.1 us for 256 n of 16 rows, at 27 KB/us of codes a CU.  Half a
// stage's conversions while the other half's operands come back took 6 to 10%
// off.  Measured against expanding the weight for the bf16 product, in us: 1 x
// 4096 x 4096 10 (85), 16 x 4096 x 14336 17 (265), 128 x 4096 x 4096 19 (86), 512
// rows 32 (85).  For more rows the second kernel below shares the expanded blocks:
// 1000 rows 53 (56 with this one's 128-row tile), 2000 rows 75 (109).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

struct MxGemmTParams {
    const uint16_t *X;  // dY: M x N
    const uint8_t *codes, *scales;
    uint16_t *Y;  // dX: M x K, written here where part is NULL
    float *part;  // [KS][M][K]
    int M, N, K;
    int groups, blocks;  // N16, KB
    int tiles_m, tiles_k;
    int KS, per;  // slices of n, stages of a slice
};

template <int WM_, int WK_, int MB_, int XR_, int NS_>
struct MxTileT {
    static constexpr int WM = WM_, WN = 4, WK = WK_, MB = MB_, XR = XR_, NS = NS_;
    static constexpr int NW = WM * WN * WK, TM = 16 * WM * MB, TN = 128, NWD = 128 * WK;
    static constexpr int XU = XR * WK / 4, WU = 8 * WK;  // 1 KiB loads of a stage
    static constexpr int XPW = (XU + NW - 1) / NW, WPW = (WU + NW - 1) / NW, UPW = XPW + WPW + 1;
    static constexpr int XB = XU * 1024, WB = WU * 1024, STAGE = XB + WB + 1024;
    static constexpr int OWN = NS * STAGE, SPARE = OWN + NW * 4096;  // the waves' expanded blocks; surplus loads
    static constexpr int RED = (WK - 1) * WM * WN * MB * 2 * 1024;
    static constexpr int LDS = SPARE + 1024 > RED ? SPARE + 1024 : RED;
    static_assert(WK <= 2 && LDS <= 160 * 1024, "tile does not fit");
};

template <class T>
__global__ __launch_bounds__(64 * T::NW) void mxfp4_gemm_t_kernel(MxGemmTParams P) {
    constexpr int WN = T::WN, WK = T::WK, MB = T::MB, XR = T::XR, NS = T::NS;
    extern __shared__ uint4 mxt_smem[];
    lds_char *smem = (lds_char *)mxt_smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
    const int l16 = lane & 15, lg = lane >> 4;

    const int id = xcd_order(blockIdx.x, P.tiles_m * P.tiles_k * P.KS);
    int tm = 0, tk = id, ks = 0;  // (the divisions are skipped where there is nothing to divide)
    if (P.tiles_m > 1) tk = id / P.tiles_m, tm = id - tk * P.tiles_m;
    if (P.KS > 1) ks = tk / P.tiles_k, tk -= ks * P.tiles_k;
    const int m0 = tm * T::TM, c0 = tk * T::TN, kb0 = c0 / 32;
    const int n0 = ks * P.per * T::NWD;
    const int nit = min(P.per, (P.N - n0 + T::NWD - 1) / T::NWD);  // >= 1: the host sizes the slices

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.N * 2u, group_bytes = (uint32_t)P.blocks * 256u;
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.N, (uint32_t)min(P.M - m0, T::TM) * row_bytes);
    const sgpr4_t dW = make_desc(P.codes, (uint32_t)P.groups * group_bytes);
    const sgpr4_t dS = make_desc(P.scales, (uint32_t)P.groups * (group_bytes / 16));

    // This wave's loads of a stage (kOOB: zeros): XPW of dY, as the forward
    // product loads X; WPW of codes, a load 16 columns of four blocks; one of
    // scales, 16 such pieces of 64 bytes.
    const int xrow4 = lane >> 4;
    int xn;
    uint32_t xo[T::XPW], wo[T::WPW], so = kOOB;
    {
        const int place = (lane & 15) ^ ((4 * (wave % (XR < 16 ? XR / 4 : 4)) + xrow4) & 15);
        xn = n0 + 8 * ((place & 3) * 4 + (place >> 2));
    }
    auto xchunk = [&](int i) { return (wave + T::NW * i) / (XR / 4); };
#pragma unroll
    for (int i = 0; i < T::XPW; ++i) {
        const int u = wave + T::NW * i, row = u % (XR / 4) * 4 + xrow4;
        xo[i] = u < T::XU && row < P.M - m0 ? (uint32_t)row * row_bytes + (uint32_t)(xn + 128 * xchunk(i)) * 2u : kOOB;
    }
    const int g0 = n0 / 16;
#pragma unroll
    for (int i = 0; i < T::WPW; ++i) {
        const int u = wave + T::NW * i;
        wo[i] = u < T::WU && kb0 + lg < P.blocks
            ? (uint32_t)(g0 + u) * group_bytes + (uint32_t)(kb0 + lg) * 256u + (uint32_t)l16 * 16u : kOOB;
    }
    const int sg = lane >> 2;
    if (sg < T::WU && kb0 + (lane & 3) < P.blocks)
        so = (uint32_t)(g0 + sg) * (group_bytes / 16) + (uint32_t)(kb0 + (lane & 3)) * 16u;
    const int nfull = min(nit, (P.N - n0) / T::NWD);
    auto issue = [&](int it, int buf) {
        const uint32_t base = lds0 + (uint32_t)buf * T::STAGE + (uint32_t)wave * 1024u, spare = lds0 + T::SPARE;
        const int dn = it < nit ? it * T::NWD : 0x20000000;  // past every limit
        const bool whole = it < nfull;
        // (a dead stage adds nothing: its lanes read zeros)
        const uint32_t dg = it < nit ? (uint32_t)(it * T::WU) * group_bytes : 0u;
#pragma unroll
        for (int i = 0; i < T::XPW; ++i)
            dma16_at(dX, whole || xn + 128 * xchunk(i) + dn < P.N ? xo[i] : kOOB, (uint32_t)dn * 2u,
                     T::XU % T::NW == 0 || wave + T::NW * i < T::XU ? base + T::NW * i * 1024u : spare);
#pragma unroll
        for (int i = 0; i < T::WPW; ++i)
            dma16_at(dW, whole || 16 * (g0 + wave + T::NW * i) + dn < P.N ? wo[i] : kOOB, dg,
                     T::WU % T::NW == 0 || wave + T::NW * i < T::WU ? base + T::XB + T::NW * i * 1024u : spare);
        dma16_at(dS, whole || 16 * (g0 + sg) + dn < P.N ? so : kOOB, dg / 16u, wave == 0 ? base + T::XB + T::WB : spare);
    };

    f32x4_t acc[MB][2];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int t = 0; t < 2; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const int xrow = (wm * MB * 16 + l16) & (XR < 16 ? XR - 1 : -1);
    uint32_t xplace[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xplace[j] = (uint32_t)(wk * XR * 256 + xrow * 256 + (((4 * j + lg) ^ (xrow & 15)) << 4));
    // The expanded half: row p (lane p's block) 64 bytes, piece d (its 8 rows of
    // W' from 8d on) at d ^ turn(p).  Sixteen rows written at one piece, and the
    // rows {0-3, 16-19} that a half-wave's transposing read takes, fall on
    // different banks.  (Eight waves at once: 16 cycles a 1 KiB write, 2.3 a 512-byte
    // transposing read, the best of all turns; with (p >> 3) & 3, 32 cycles a write.)
    auto turn = [](int p) { return ((p >> 2) & 3) ^ ((p >> 3) & 2); };
    lds_char *own = smem + T::OWN + wave * 4096;
    uint32_t put[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) put[d] = (uint32_t)(lane * 64 + ((d ^ turn(lane)) << 4));
    // column tile 0, step 0 of the half, its first four rows; the second column
    // tile is at ^ 32, rows 4 on at + 256 ^ 16, step 1 at + 512 ^ 32
    const int p0 = 16 * lg + (l16 >> 2);
    const uint32_t get = (uint32_t)(p0 * 64 + ((((l16 & 3) >> 1) ^ turn(p0)) << 4) + (l16 & 1) * 8);

#pragma unroll 1
    for (int s = 0; s < NS - 1; ++s) issue(s, s);
    int buf = 0;
    for (int it = 0; it < nit; ++it) {
        // this stage has landed, and this wave's reads of the last one are done
        wait_vmcnt_lds<T::UPW *(NS - 2)>();
        asm volatile("" ::: "memory");  // keep LDS reads and loads into LDS on their side of the barrier
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const lds_char *sx = smem + buf * T::STAGE;
        const lds_char *sw = sx + T::XB + (wk * 8 + 2 * lg) * 1024 + wn * 256 + l16 * 16;
        const lds_char *ss = sx + T::XB + T::WB + (wk * 8 + 2 * lg) * 64 + wn * 16 + l16;
        // Half h: lane (g, l)'s block is column 32g + 16h + l of the chunk, and its
        // two steps take n = 32g + 16h + 8jj .. +7.  The second half is converted
        // while the first one's operands come back from LDS.
        uint32_t sb[2];
        uint4 q[2], x[2][2][MB], e[2][4], w[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            q[h] = *(const uint4 *)(sw + h * 1024);
            sb[h] = *(const uint8_t *)(ss + h * 64);
        }
        auto rows = [&](int h) {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int a = 0; a < MB; ++a) x[h][jj][a] = *(const uint4 *)(sx + xplace[2 * h + jj] + a * 4096);
        };
        rows(0);
        __builtin_amdgcn_sched_barrier(0);
        issue(it + NS - 1, buf == 0 ? NS - 1 : buf - 1);  // the buffer of stage it - 1
        auto expand = [&](int h) {
            const float sc = mx_scale(sb[h]);
            e[h][0] = mx_frag(q[h].x, sc), e[h][1] = mx_frag(q[h].y, sc);
            e[h][2] = mx_frag(q[h].z, sc), e[h][3] = mx_frag(q[h].w, sc);
        };
        auto turned = [&](int h) {
#pragma unroll
            for (int d = 0; d < 4; ++d) *(uint4 *)(own + put[d]) = e[h][d];
            asm volatile("" ::: "memory");  // other lanes' pieces are read below: LDS takes a wave's accesses in order
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t at = (get + 512 * jj) ^ (32 * (jj ^ t));
                    const uint2 w0 = lds_read_tr4(own + at), w1 = lds_read_tr4(own + ((at + 256) ^ 16));
                    w[jj][t] = make_uint4(w0.x, w0.y, w1.x, w1.y);
                }
            asm volatile("" ::: "memory");
        };
        auto products = [&](int h) {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int a = 0; a < MB; ++a) acc[a][t] = mfma16x16x32(w[jj][t], x[h][jj][a], acc[a][t]);
        };
        expand(0);
        turned(0);
        rows(1);
        __builtin_amdgcn_sched_barrier(0);
        expand(1);
        products(0);
        __builtin_amdgcn_sched_barrier(0);
        turned(1);
        products(1);
        buf = buf == NS - 1 ? 0 : buf + 1;
    }
    wait_vmcnt<0>();  // (the last loads fill zeros: nothing may land in the space used below)

    if constexpr (WK > 1) {
        __syncthreads();
        f32x4_t *red = (f32x4_t *)mxt_smem;
        const int w2 = wave / WK;
        if (wk > 0) {
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int t = 0; t < 2; ++t) red[(w2 * MB * 2 + a * 2 + t) * 64 + lane] = acc[a][t];
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[a][t] += red[(w2 * MB * 2 + a * 2 + t) * 64 + lane];
    }

    // lane (g, l): columns 4g .. 4g+3 of a tile, row l; rows past M and columns
    // past K are dropped by the buffer's bounds
    const bool direct = P.part == nullptr;
    const int rows = min(P.M - m0, T::TM);
    const __amdgpu_buffer_rsrc_t rY =
        direct ? make_rsrc(P.Y + (size_t)m0 * P.K, (uint64_t)rows * P.K * 2u)
               : make_rsrc(P.part + ((size_t)ks * P.M + m0) * P.K, (uint64_t)rows * P.K * 4u);
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const uint32_t row = (uint32_t)((wm * MB + a) * 16 + l16);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int col = c0 + 32 * wn + 16 * t + 4 * lg;
            const uint32_t at = row < (uint32_t)rows && col < P.K ? row * (uint32_t)P.K + (uint32_t)col : kOOB / 4;
            if (direct)
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2_t{pack_bf16x2(acc[a][t][0], acc[a][t][1]), pack_bf16x2(acc[a][t][2], acc[a][t][3])}, rY, at * 2u, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[a][t]), rY, at * 4u, 0, 0);
        }
    }
}

// The shape for many rows: 128 rows and 256 columns of dX, 2 x 4 waves of 64 x 64,
// 64 n a stage.  Each wave expands one block of rows of W' for the next stage, 4 KiB,
// into one of two buffers that all waves read, so a code is expanded once for 128
// rows and its operands are read by two waves.  One barrier a stage: it stands
// between the writes of a stage's W' and its reads, and the loads of X two stages and
// of codes three stages ahead.  Bound by LDS, of whose cycles a stage takes about
// 1900 (32 KiB written at 64 bytes a cycle, 25 KiB by the loads, 64 KiB of X and 64
// KiB of W' read), against 1024 of the MFMAs.  dX of 1000 x 4096 x 4096 53 us (56 with
// 128 x 128 tiles), 2000 x 4096 x 4096 75 (86 expanded), 1024 x 4096 x 14336 135
// (174; 271 expanded); 4096 x 4096 x 4096 154 (105 expanded).  A half's reads moved
// over the other half's MFMAs, with the second half carried into the next stage,
// gained nothing.
struct MxBigT {
    static constexpr int TM = 128, TN = 256, NWD = 64, NW = 8, MB = 4, NB = 4;
    static constexpr int XB = 16 * 1024, CB = 9 * 1024;  // X; codes and scales
    static constexpr int CODES = 3 * XB, WIDE = CODES + 3 * CB, SPARE = WIDE + 2 * 32 * 1024, LDS = SPARE + 1024;
    static_assert(LDS <= 160 * 1024, "tile does not fit");
};

__global__ __launch_bounds__(512) void mxfp4_gemm_big_t_kernel(MxGemmTParams P) {
    using T = MxBigT;
    constexpr int MB = T::MB, NB = T::NB;
    extern __shared__ uint4 mxb_smem[];
    lds_char *smem = (lds_char *)mxb_smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wn = wave & 3, wm = wave >> 2;

    const int id = xcd_order(blockIdx.x, P.tiles_m * P.tiles_k * P.KS);
    int tk = id / P.tiles_m;
    const int tm = id - tk * P.tiles_m, ks = tk / P.tiles_k;
    tk -= ks * P.tiles_k;
    const int m0 = tm * T::TM, c0 = tk * T::TN, kb0 = c0 / 32;
    const int n0 = ks * P.per * T::NWD, g0 = n0 / 16;
    const int nit = min(P.per, (P.N - n0 + T::NWD - 1) / T::NWD);  // >= 1: the host sizes the slices

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.N * 2u, group_bytes = (uint32_t)P.blocks * 256u;
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.N, (uint32_t)min(P.M - m0, T::TM) * row_bytes);
    const sgpr4_t dW = make_desc(P.codes, (uint32_t)P.groups * group_bytes);
    const sgpr4_t dS = make_desc(P.scales, (uint32_t)P.groups * (group_bytes / 16));

    // This wave's loads (kOOB: zeros): of X two, 8 rows of 128 bytes each, piece c (8 n)
    // of row i at c ^ (i mod 8); of codes one, four blocks of a column group; of scales
    // wave 0's 32 pieces, block by block of each group.
    const int xn = n0 + 8 * ((lane & 7) ^ (lane >> 3));
    uint32_t xo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * wave + 8 * i + (lane >> 3);
        xo[i] = row < P.M - m0 ? (uint32_t)row * row_bytes + (uint32_t)xn * 2u : kOOB;
    }
    const int wg = wave >> 1, wb = 4 * (wave & 1) + lg, sg = (lane & 31) >> 3;
    const uint32_t wo = kb0 + wb < P.blocks
        ? (uint32_t)(g0 + wg) * group_bytes + (uint32_t)(kb0 + wb) * 256u + (uint32_t)l16 * 16u : kOOB;
    const uint32_t so = lane < 32 && kb0 + (lane & 7) < P.blocks
        ? (uint32_t)(g0 + sg) * (group_bytes / 16) + (uint32_t)(kb0 + (lane & 7)) * 16u : kOOB;
    auto load_x = [&](int it) {
        const int dn = it < nit ? it * T::NWD : 0x20000000;  // past every limit
        const uint32_t base = lds0 + (uint32_t)(it % 3) * T::XB + (uint32_t)wave * 2048u;
        const bool in = xn + dn < P.N;
#pragma unroll
        for (int i = 0; i < 2; ++i) dma16_at(dX, in ? xo[i] : kOOB, (uint32_t)dn * 2u, base + 1024u * i);
    };
    auto load_w = [&](int it) {
        const int dn = it < nit ? it * T::NWD : 0x20000000;
        const uint32_t dg = it < nit ? (uint32_t)(it * 4) * group_bytes : 0u;
        const uint32_t base = lds0 + T::CODES + (uint32_t)(it % 3) * T::CB;
        dma16_at(dW, 16 * (g0 + wg) + dn < P.N ? wo : kOOB, dg, base + (uint32_t)wave * 1024u);
        dma16_at(dS, 16 * (g0 + sg) + dn < P.N ? so : kOOB, dg / 16u, wave == 0 ? base + 8192u : lds0 + T::SPARE);
    };

    // The expanded stage: block b's 64 rows of 64 bytes from b * 4096 on, piece d at
    // d ^ turn(row), as in the kernel above.
    auto turn = [](int p) { return ((p >> 2) & 3) ^ ((p >> 3) & 2); };
    uint32_t put[4], get[2];
#pragma unroll
    for (int d = 0; d < 4; ++d) put[d] = (uint32_t)(wave * 4096 + lane * 64 + ((d ^ turn(lane)) << 4));
    // step 0, a block's first column tile, rows 8 lg + (0 .. 3) and + (4 .. 7); the second
    // tile is at ^ 32, step 1 (32 rows on, of the same turn) at + 2048
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int p = 8 * lg + 4 * e + (l16 >> 2);
        get[e] = (uint32_t)(wn * 8192 + p * 64 + ((((l16 & 3) >> 1) ^ turn(p)) << 4) + (l16 & 1) * 8);
    }
    auto codes = [&](int it, uint4 &q, float &sc) {  // this wave's block of stage it, a lane a row
        const lds_char *from = smem + T::CODES + it % 3 * T::CB;
        q = *(const uint4 *)(from + (lg * 2 + (wave >> 2)) * 1024 + (wave & 3) * 256 + l16 * 16);
        sc = mx_scale(*(const uint8_t *)(from + 8192 + (lg * 8 + wave) * 16 + l16));
    };

    f32x4_t acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int t = 0; t < NB; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    load_w(0);
    load_x(0);
    load_w(1);
    load_x(1);
    load_w(2);
    wait_vmcnt_lds<8>();  // codes of stage 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    {
        uint4 q;
        float sc;
        codes(0, q, sc);
        const uint32_t part[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int d = 0; d < 4; ++d) *(uint4 *)(smem + T::WIDE + put[d]) = mx_frag(part[d], sc);
    }
    for (int it = 0; it < nit; ++it) {
        // X of this stage and the codes of the next have landed, this wave has written its block
        wait_vmcnt_lds<4>();
        asm volatile("" ::: "memory");  // keep LDS accesses and loads into LDS on their side of the barrier
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const lds_char *sx = smem + it % 3 * T::XB + (wm * 64 + l16) * 128;
        const lds_char *sw = smem + T::WIDE + (it & 1) * 32768;
        uint4 q, x[2][MB], w[2][NB];
        float sc;
        auto read = [&](int s) {
#pragma unroll
            for (int a = 0; a < MB; ++a) x[s][a] = *(const uint4 *)(sx + a * 2048 + (((4 * s + lg) ^ (l16 & 7)) << 4));
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                const uint32_t at = 4096 * (t >> 1) + 2048 * s, flip = 32 * (t & 1);
                const uint2 w0 = lds_read_tr4(sw + at + (get[0] ^ flip)), w1 = lds_read_tr4(sw + at + (get[1] ^ flip));
                w[s][t] = make_uint4(w0.x, w0.y, w1.x, w1.y);
            }
        };
        codes(it + 1, q, sc);
        read(0);
        __builtin_amdgcn_sched_barrier(0);
        load_x(it + 2);  // over stage it - 1's X
        load_w(it + 3);  // over this stage's codes
        read(1);
        __builtin_amdgcn_sched_barrier(0);
        // the next stage's block between this one's MFMAs
        lds_char *to = smem + T::WIDE + ((it + 1) & 1) * 32768;
        const uint32_t part[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < NB; ++t) {
#pragma unroll
                for (int a = 0; a < MB; ++a) acc[a][t] = mfma16x16x32(w[s][t], x[s][a], acc[a][t]);
                if (t & 1) *(uint4 *)(to + put[2 * s + (t >> 1)]) = mx_frag(part[2 * s + (t >> 1)], sc);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    wait_vmcnt<0>();  // (the last loads fill zeros)

    const bool direct = P.part == nullptr;
    const int rows = min(P.M - m0, T::TM);
    const __amdgpu_buffer_rsrc_t rY =
        direct ? make_rsrc(P.Y + (size_t)m0 * P.K, (uint64_t)rows * P.K * 2u)
               : make_rsrc(P.part + ((size_t)ks * P.M + m0) * P.K, (uint64_t)rows * P.K * 4u);
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const uint32_t row = (uint32_t)(wm * 64 + a * 16 + l16);
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const int col = c0 + 64 * wn + 16 * t + 4 * lg;
            const uint32_t at = row < (uint32_t)rows && col < P.K ? row * (uint32_t)P.K + (uint32_t)col : kOOB / 4;
            if (direct)
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2_t{pack_bf16x2(acc[a][t][0], acc[a][t][1]), pack_bf16x2(acc[a][t][2], acc[a][t][3])}, rY, at * 2u, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[a][t]), rY, at * 4u, 0, 0);
        }
    }
}

hipError_t launch_big(const MxGemmTParams &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void *)mxfp4_gemm_big_t_kernel, MxBigT::LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(mxfp4_gemm_big_t_kernel, dim3((unsigned)(P.tiles_m * P.tiles_k * P.KS)), dim3(512), MxBigT::LDS, stream,
                       P);
    return hipGetLastError();
}

template <class T>
hipError_t launch_tt(const MxGemmTParams &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void *)mxfp4_gemm_t_kernel<T>, T::LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((mxfp4_gemm_t_kernel<T>), dim3((unsigned)(P.tiles_m * P.tiles_k * P.KS)), dim3(64 * T::NW), T::LDS,
                       stream, P);
    return hipGetLastError();
}

struct MxKindT {
    const char *name;  // in the timing pool
    hipError_t (*launch)(const MxGemmTParams &, hipStream_t);
    int tm, tn, nwd;
    float stage;  // microseconds a stage takes a work-group when a full round of them runs
};
template <class T>
constexpr MxKindT kind_t(const char *name, float stage) {
    return MxKindT{name, launch_tt<T>, T::TM, T::TN, T::NWD, stage};
}
const MxKindT kKindsT[] = {
    kind_t<MxTileT<1, 2, 1, 16, 3>>("mxfp4_gemm_t 16x128", 1.13f),
    kind_t<MxTileT<1, 2, 2, 32, 3>>("mxfp4_gemm_t 32x128", 1.27f),
    kind_t<MxTileT<1, 2, 3, 48, 3>>("mxfp4_gemm_t 48x128", 1.45f),
    kind_t<MxTileT<1, 2, 4, 64, 2>>("mxfp4_gemm_t 64x128", 1.70f),
    kind_t<MxTileT<2, 1, 4, 128, 2>>("mxfp4_gemm_t 128x128", 1.60f),
    MxKindT{"mxfp4_gemm_t 128x256", launch_big, MxBigT::TM, MxBigT::TN, MxBigT::NWD, 1.06f},
};

}  // namespace

// The cheapest of the tile shapes and of expanding the weight, by the forward
// product's model (which says 10, 16, 17, 32, 50 and 72 us for the packed shapes
// measured above, and 84 us for up to 2000 rows of 4096 x 4096 expanded).  The
// 128 x 256 tile is taken from 71 rows of 4096 x 14336 on and from 519 of 4096 x 4096,
// and, for a microsecond, for few rows of a short contraction.
static MxGemmTPlan find_plan(int64_t m, int64_t k, int64_t n, int r) {
    MxGemmTPlan best{};
    if (m <= 0 || k > (1 << 20) || n > (1 << 20) || m > (1 << 19) || mx_groups(n) * mx_blocks(k) * 256 >= (1LL << 31))
        return best;
    const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const double weight = (double)k * n;
    double least = expanded_us(m, k, n, weight) + (r > 0 ? 8.0 : 0.0);
    for (int kind = 1; kind <= (int)(sizeof(kKindsT) / sizeof(kKindsT[0])); ++kind) {
        const MxKindT &K = kKindsT[kind - 1];
        MxGemmTPlan p{};
        p.kind = kind;
        p.tiles_m = (int)cdiv(m, K.tm);
        p.tiles_k = (int)cdiv(k, K.tn);
        const int64_t tiles = (int64_t)p.tiles_m * p.tiles_k, stages = cdiv(n, K.nwd);
        if (tiles > (1 << 20)) continue;
        for (int want = 1; want <= 16 && want <= stages; ++want) {
            p.per = (int)cdiv(stages, want);
            p.KS = (int)cdiv(stages, p.per);
            if (p.KS != want) continue;
            p.finish = p.KS > 1 || r > 0;
            p.part_bytes = p.finish ? (size_t)p.KS * m * k * sizeof(float) : 0;
            double t = 3.5 + rounds_us(tiles * p.KS, 256, p.per * K.stage + 1.0, weight);
            if (p.finish) t += 3.5 + (double)p.part_bytes * 2 / 8e6;
            if (t < least) {
                least = t;
                best = p;
            }
        }
    }
    return best;
}

MxGemmTPlan mx_gemm_t_plan(int64_t m, int64_t k, int64_t n, int r) {
    return remembered<MxGemmTPlan>(m, k, n, r, [&] { return find_plan(m, k, n, r); });
}

hipError_t launch_mxfp4_gemm_t(const MxGemmTPlan &pl, const void *dY, const void *codes, const void *scales, int m, int k,
                               int n, void *dX, float *part, hipStream_t stream) {
    MxGemmTParams P{};
    P.X = (const uint16_t *)dY;
    P.codes = (const uint8_t *)codes;
    P.scales = (const uint8_t *)scales;
    P.Y = (uint16_t *)dX;
    P.part = pl.finish ? part : nullptr;
    P.M = m;
    P.N = n;
    P.K = k;
    P.groups = (int)mx_groups(n);
    P.blocks = (int)mx_blocks(k);
    P.tiles_m = pl.tiles_m;
    P.tiles_k = pl.tiles_k;
    P.KS = pl.KS;
    P.per = pl.per;
    const int slot = prof_begin(kKindsT[pl.kind - 1].name, stream);
    const hipError_t e = kKindsT[pl.kind - 1].launch(P, stream);
    prof_end(slot, stream);
    return e;
}

}  // namespace lora
