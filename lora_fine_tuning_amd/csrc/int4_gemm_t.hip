// dX = dY W'^T + s keep.(dS A^T) for few and middling numbers of rows, W' = s (q - z) in
// 4-bit integers (int4_kernels.hip describes the storage).
//
// The contraction runs over n, across the columns that the codes are stored by, and the
// scales change with every column, so W' is rounded to bf16 value by value, exactly as
// when it is expanded.  The plan is that of MXFP4's transposed product: codes through an
// LDS ring by direct-to-LDS loads; a wave owns 32 columns of dX, one block of 32 rows of W',
// and a lane expands whole blocks of a column (its four words of codes, one scale) into
// the wave's own 4 KiB, from which transposing reads give the MFMA operand, 8 n of one
// column of dX.  No other wave reads it, so the expansion needs no barrier.
//
// A work-group covers 16 WM MB rows and 128 columns of dX; its waves split the rows
// (WM), the columns (4) and each stage's n (WK chunks of 128).  mxfp4_join.hip adds the
// slices of n and the adapters' term.
//
// Bound by a stage's chain (codes out of LDS, 31 instructions for eight values, into LDS,
// out again): 1.85 us for 256 n of 16 rows, 2.05 for 128 n of 128 rows.  Measured against
// expanding the weight for the bf16 product, in us: 1 x 4096 x 4096 11 (95), 16 x 4096 x
// 14336 21 (270), 128 x 4096 x 4096 20 (96), 512 rows 39 (96), 1000 rows 70 (96).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "int4.hpp"
#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

struct I4TParams {
    const uint16_t *X;  // dY: M x N
    const uint8_t *codes;
    const uint32_t *scales;
    uint16_t *Y;  // dX: M x K, written here where part is NULL
    float *part;  // [KS][M][K]
    int M, N, K;
    int N16, K128, G, each;  // each: blocks of 128 rows that share a scale (groups of 128 rows or more)
    int tiles_m, tiles_k;
    int KS, per;  // slices of n, stages of a slice
};

// GR: groups of scales in 128 rows (1: groups of 128 rows or more).
template <int WM_, int WK_, int MB_, int XR_, int NS_, int GR_>
struct I4TileT {
    static constexpr int WM = WM_, WN = 4, WK = WK_, MB = MB_, XR = XR_, GR = GR_;
    static constexpr int NW = WM * WN * WK, TM = 16 * WM * MB, TN = 128, NWD = 128 * WK;
    static constexpr int XU = XR * WK / 4, WU = 8 * WK;  // 1 KiB loads of a stage
    static constexpr int XPW = (XU + NW - 1) / NW, WPW = (WU + NW - 1) / NW, UPW = XPW + WPW + 1;
    static constexpr int XB = XU * 1024, WB = WU * 1024, STAGE = XB + WB + GR * 1024;
    static constexpr int NS = NS_ * STAGE + NW * 4096 + 1024 <= 160 * 1024 ? NS_ : 2;  // stages of the ring
    static constexpr int OWN = NS * STAGE, SPARE = OWN + NW * 4096;  // the waves' expanded blocks; surplus loads
    static constexpr int RED = (WK - 1) * WM * WN * MB * 2 * 1024;
    static constexpr int LDS = SPARE + 1024 > RED ? SPARE + 1024 : RED;
    static_assert(WK <= 2 && GR <= NW && LDS <= 160 * 1024, "tile does not fit");
};

// A stored word -> eight rows of s (q - z) in bf16.  q - z and its product are exact in
// fp32 (8 and 24 bits), so each value is rounded once.
__device__ __forceinline__ uint4 i4_values(uint32_t w, float s, float z) {
    const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;  // rows 0 4 1 5 and 2 6 3 7
    const auto v = [&](uint32_t bytes, int i) { return s * ((float)((bytes >> (8 * i)) & 0xFFu) - z); };
    return make_uint4(pack_bf16x2(v(a, 0), v(a, 2)), pack_bf16x2(v(b, 0), v(b, 2)), pack_bf16x2(v(a, 1), v(a, 3)),
                      pack_bf16x2(v(b, 1), v(b, 3)));
}

template <class T>
__global__ __launch_bounds__(64 * T::NW) void int4_gemm_t_kernel(I4TParams P) {
    constexpr int WN = T::WN, WK = T::WK, MB = T::MB, XR = T::XR, NS = T::NS, GR = T::GR;
    extern __shared__ uint4 i4t_smem[];
    lds_char *smem = (lds_char *)i4t_smem;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
    const int l16 = lane & 15, lg = lane >> 4;

    const int id = xcd_order(blockIdx.x, P.tiles_m * P.tiles_k * P.KS);
    int tm = 0, tk = id, ks = 0;  // (the divisions are skipped where there is nothing to divide)
    if (P.tiles_m > 1) tk = id / P.tiles_m, tm = id - tk * P.tiles_m;
    if (P.KS > 1) ks = tk / P.tiles_k, tk -= ks * P.tiles_k;
    const int m0 = tm * T::TM, c0 = tk * T::TN;
    const int n0 = ks * P.per * T::NWD;
    const int nit = min(P.per, (P.N - n0 + T::NWD - 1) / T::NWD);  // >= 1: the host sizes the slices

    // the host keeps every offset below 2^31
    const uint32_t row_bytes = (uint32_t)P.N * 2u, group_bytes = (uint32_t)P.K128 * 1024u, scale_bytes = (uint32_t)P.G * 64u;
    const sgpr4_t dX = make_desc(P.X + (size_t)m0 * P.N, (uint32_t)min(P.M - m0, T::TM) * row_bytes);
    const sgpr4_t dW = make_desc(P.codes, (uint32_t)P.N16 * group_bytes);
    const sgpr4_t dS = make_desc(P.scales, (uint32_t)P.N16 * scale_bytes);

    // This wave's loads of a stage (kOOB: zeros): XPW of dY, as the forward product loads
    // X; WPW of codes, a load 128 rows of 16 columns; one of scales, 16 column groups'
    // 64 bytes of the wave's one of the GR groups of rows.
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
        wo[i] = u < T::WU ? (uint32_t)(g0 + u) * group_bytes + (uint32_t)tk * 1024u + (uint32_t)lane * 16u : kOOB;
    }
    const int sg = lane >> 2;
    if (sg < T::WU && wave < GR)
        so = (uint32_t)(g0 + sg) * scale_bytes + (uint32_t)(GR > 1 ? tk * GR + wave : tk / P.each) * 64u + (uint32_t)(lane & 3) * 16u;
    const int nfull = min(nit, (P.N - n0) / T::NWD);
    auto issue = [&](int it, int buf) {
        const uint32_t base = lds0 + (uint32_t)buf * T::STAGE + (uint32_t)wave * 1024u, spare = lds0 + T::SPARE;
        const int dn = it < nit ? it * T::NWD : 0x20000000;  // past every limit
        const bool whole = it < nfull;
        // (a dead stage adds nothing: its lanes read zeros)
        const uint32_t dc = it < nit ? (uint32_t)(it * T::WU) : 0u;
#pragma unroll
        for (int i = 0; i < T::XPW; ++i)
            dma16_at(dX, whole || xn + 128 * xchunk(i) + dn < P.N ? xo[i] : kOOB, (uint32_t)dn * 2u,
                     T::XU % T::NW == 0 || wave + T::NW * i < T::XU ? base + T::NW * i * 1024u : spare);
#pragma unroll
        for (int i = 0; i < T::WPW; ++i)
            dma16_at(dW, whole || 16 * (g0 + wave + T::NW * i) + dn < P.N ? wo[i] : kOOB, dc * group_bytes,
                     T::WU % T::NW == 0 || wave + T::NW * i < T::WU ? base + T::XB + T::NW * i * 1024u : spare);
        dma16_at(dS, so != kOOB && (whole || 16 * (g0 + sg) + dn < P.N) ? so : kOOB, dc * scale_bytes, wave < GR ? base + T::XB + T::WB : spare);
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
        const lds_char *sw = sx + T::XB + (wk * 8 + 2 * lg) * 1024 + l16 * 16 + wn * 4;
        const lds_char *ss = sx + T::XB + T::WB + wn * GR / 4 * 1024 + (wk * 8 + 2 * lg) * 64 + l16 * 4;
        // Half h: lane (g, l)'s block is column 32g + 16h + l of the chunk, and its
        // two steps take n = 32g + 16h + 8jj .. +7.  The second half is converted
        // while the first one's operands come back from LDS.
        uint32_t sb[2];
        uint32_t q[2][4];
        uint4 x[2][2][MB], e[2][4], w[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int g = 0; g < 4; ++g) q[h][g] = *(const uint32_t *)(sw + h * 1024 + g * 256);
            sb[h] = *(const uint32_t *)(ss + h * 64);
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
            const float s = __uint_as_float(sb[h] & 0xFFFFFF00u), z = (float)(sb[h] & 0xFFu);
#pragma unroll
            for (int g = 0; g < 4; ++g) e[h][g] = i4_values(q[h][g], s, z);
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
        f32x4_t *red = (f32x4_t *)i4t_smem;
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

template <class T>
hipError_t launch_t(const I4TParams &P, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void *)int4_gemm_t_kernel<T>, T::LDS, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((int4_gemm_t_kernel<T>), dim3((unsigned)(P.tiles_m * P.tiles_k * P.KS)), dim3(64 * T::NW), T::LDS, stream, P);
    return hipGetLastError();
}

struct I4KindT {
    const char *name;  // in the timing pool
    hipError_t (*launch[3])(const I4TParams &, hipStream_t);  // groups of 32, 64, 128 rows or more
    int tm, nwd;
    float stage;  // microseconds a stage takes a work-group when a full round of them runs
};
template <int WM, int WK, int MB, int XR, int NS>
constexpr I4KindT kind_t(const char *name, float stage) {
    using T = I4TileT<WM, WK, MB, XR, NS, 1>;
    return I4KindT{name, {launch_t<I4TileT<WM, WK, MB, XR, NS, 4>>, launch_t<I4TileT<WM, WK, MB, XR, NS, 2>>, launch_t<T>}, T::TM, T::NWD,
                   stage};
}
const I4KindT kKindsT[] = {
    kind_t<1, 2, 1, 16, 3>("int4_gemm_t 16x128", 1.85f),
    kind_t<1, 2, 2, 32, 3>("int4_gemm_t 32x128", 1.95f),
    kind_t<1, 2, 3, 48, 3>("int4_gemm_t 48x128", 2.10f),
    kind_t<1, 2, 4, 64, 2>("int4_gemm_t 64x128", 2.20f),
    kind_t<2, 1, 4, 128, 2>("int4_gemm_t 128x128", 2.05f),
};

}  // namespace

// The cheapest of the tile shapes, n split as far as pays, and of expanding the weight, by
// a model of their times: 3.5 us, rounds of work-groups (stages x stage time + 1 us each, at
// least their share of the weight's bytes); a joining launch 3.5 us and its partial sums at
// 8 TB/s.  Measured, model in brackets: 1 x 4096 x 4096 11.1 (11.7), 16 x 4096 x 14336 20.8
// (21.5), 64 x 4096 x 14336 25.6 (25.5), 512 x 4096 x 4096 39.4 (39.7), 1000 x 4096 x 4096
// 69.8 (70.1).
static I4TPlan find_plan(int64_t m, int64_t k, int64_t n, int64_t group, int r) {
    I4TPlan best{};
    const I4Shape s = i4_shape(k, n, group);
    // (every offset stays below 2^31)
    if (m <= 0 || m > (1 << 19) || k > (1 << 20) || n > (1 << 20) || s.n16 * s.k128 * 1024 >= (1LL << 31)) return best;
    const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const double weight = (double)k * n;
    double least = expanded_us(m, k, n, weight) + (r > 0 ? 8.0 : 0.0);
    for (int kind = 1; kind <= (int)(sizeof(kKindsT) / sizeof(kKindsT[0])); ++kind) {
        const I4KindT &K = kKindsT[kind - 1];
        I4TPlan p{};
        p.kind = kind;
        p.tiles_m = (int)cdiv(m, K.tm);
        p.tiles_k = (int)s.k128;
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

I4TPlan int4_t_plan(int64_t m, int64_t k, int64_t n, int64_t group, int r) {
    return remembered<I4TPlan>(m, k, n, (group << 10) ^ r, [&] { return find_plan(m, k, n, group, r); });
}

hipError_t launch_int4_gemm_t(const I4TPlan &pl, const void *dY, const void *codes, const void *scales, int64_t group, int m, int k, int n,
                              void *dX, float *part, hipStream_t stream) {
    const I4Shape s = i4_shape(k, n, group);
    I4TParams P{};
    P.X = (const uint16_t *)dY;
    P.codes = (const uint8_t *)codes;
    P.scales = (const uint32_t *)scales;
    P.Y = (uint16_t *)dX;
    P.part = pl.finish ? part : nullptr;
    P.M = m;
    P.N = n;
    P.K = k;
    P.N16 = (int)s.n16;
    P.K128 = (int)s.k128;
    P.G = (int)s.groups;
    P.each = group < 128 ? 1 : (int)std::min<int64_t>(group / 128, s.k128);
    P.tiles_m = pl.tiles_m;
    P.tiles_k = pl.tiles_k;
    P.KS = pl.KS;
    P.per = pl.per;
    const I4KindT &K = kKindsT[pl.kind - 1];
    const int slot = prof_begin(K.name, stream);
    const hipError_t e = K.launch[group == 32 ? 0 : group == 64 ? 1 : 2](P, stream);
    prof_end(slot, stream);
    return e;
}

}  // namespace lora
