// The second launch of the products over a weight of 4-bit integers: the partial sums of
// the contraction's slices and the adapters' term, rounded once.  (Mixed batches of more
// than 64 rows end in mxfp4_join.hip.)
//
//   Y = sum_s part_s + alpha S B             (S: M x RS, B: r x N)
//
// for one adapter or for segments of rows with an adapter each.  S is given, or it is
// the sum of the product's partial sums of keep.X A, and the first column tile writes it.
//
// Bound by latency: everything it reads is a few MiB out of L2.  So a work-group takes
// 16 rows of 32 columns only, and its waves share the work: a task is one MFMA step of 32
// ranks of one segment's adapter (16 rows have 16 segments with rows at most), and wave w
// takes every eighth task, and every eighth slice of the product.  The first wave reads
// the segment table with a lane for each segment and lists the tasks in LDS.  S of all 16
// rows goes to LDS next, eight of a thread's partial sums on their way at once, and the
// tasks' first B meanwhile; a task's B passes through 2 KiB of the wave's own LDS, the
// next task's on its way.  The waves are added in wave order.  A lane takes a task's sums where
// its row belongs to the segment only, so that an infinity in one adapter's matrix stays
// out of the others' rows; rows in no segment get the product alone.
// 4096 columns, 16 rows of 16 adapters (ranks 8 to 128, k 4096): 8.2 us (26 with each
// wave reading the segment table and 16 loads on their way, which spilled); 1 row of one
// adapter (rank 16, k 4096): 5.8 us.
#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

struct I4FinishParams {
    const float *part;  // [KS][M][N]
    int KS, M, N;
    float *S;  // M x RS
    int RS;
    int SK;  // > 0: S is the sum of spart's [SK][M][RS rounded up to 4], and written
    const float *spart;
    const uint16_t *B;
    int r;
    float alpha, undrop;
    const lora_adapter *adapters;
    const int64_t *seg_off;
    const int32_t *seg_adapter;
    int num_adapters, nseg;
    uint16_t *Y;
};

// A task: 32 ranks (from r0) of the adapter of rows lo .. hi - 1.
struct I4Task {
    int lo, hi, r, r0;
    const uint16_t *B;
};

constexpr int NW = 8, TPR = 4 * NW;  // waves, threads a row of S
constexpr int kTasks = 64 * 8;       // of 64 segments, of ranks up to 256

template <bool MULTI>
__global__ __launch_bounds__(64 * NW) void int4_finish_kernel(I4FinishParams P) {
    __shared__ float sS[16][260];   // the rows' scaled S (rows 16 bytes past a bank period)
    __shared__ uint4 sB[NW * 128];  // a wave's 32 ranks of 32 columns of B; at the end its sums
    __shared__ I4Task tasks[MULTI ? kTasks : 1];
    __shared__ float rows[MULTI ? 16 : 1][4];  // rank, alpha and 1 / (1 - p) of a row's adapter (rank 0: none)
    __shared__ int state[2];                   // the tasks of this table's 64 segments; whether they are the last
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row0 = (int)blockIdx.y * 16, row = row0 + l16, rend = min(row0 + 16, P.M);
    const int c0 = (int)blockIdx.x * 32, col = c0 + 4 * lg;
    const bool live0 = row < P.M && col < P.N, live1 = row < P.M && col + 16 < P.N;
    // lane (g, l): row l, columns 4g .. 4g+3 of two groups of 16
    f32x4_t total[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};

    // a task's B: rank 16 i + lane / 4, the columns' 16-byte piece lane mod 4
    auto fetch = [&](const I4Task &it, uint4 (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[i] = make_uint4(0u, 0u, 0u, 0u);
            const int k = it.r0 + 16 * i + (lane >> 2), c = c0 + 8 * (lane & 3);
            if (k < it.r && c < P.N) __builtin_memcpy(&f[i], it.B + (size_t)k * P.N + c, 16);  // (B may be unaligned)
        }
    };
    // The rows' S, TPR threads a row, 4 ranks at a time; r: the rank of this thread's row (0: no adapter)
    auto stage = [&](int r, float alpha, float undrop) {
        const int br = tid / TPR, mine = row0 + br;
        const int rs = (P.RS + 3) & ~3;
        const size_t part = (size_t)P.M * rs;
#pragma unroll 1
        for (int c = 4 * (tid % TPR); c < ((P.RS + 31) & ~31); c += 4 * TPR) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (c < r) {
                if (P.SK > 0) {
                    const float *ps = P.spart + (size_t)mine * rs + c;
                    f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int q = 0; q < P.SK; q += 8) {
                        f32x4_t u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) u[e] = *(const f32x4_t *)(ps + min(q + e, P.SK - 1) * part);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum += q + e < P.SK ? u[e] : f32x4_t{0.f, 0.f, 0.f, 0.f};
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = c + e < r ? undrop * sum[e] : 0.f;  // (past r nothing was written)
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = c + e < r ? P.S[(size_t)mine * P.RS + c + e] : 0.f;
                }
            }
            if (P.SK > 0 && blockIdx.x == 0 && r > 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < P.RS) P.S[(size_t)mine * P.RS + c + e] = v[e];
            }
            *(float4 *)&sS[br][c] = make_float4(alpha * v[0], alpha * v[1], alpha * v[2], alpha * v[3]);
        }
    };
    auto multiply = [&](const I4Task &it, const uint4 (&f)[2]) {
        const bool mine = row >= it.lo && row < it.hi;
        float v[8];
        *(float4 *)&v[0] = *(const float4 *)&sS[l16][it.r0 + 8 * lg];
        *(float4 *)&v[4] = *(const float4 *)&sS[l16][it.r0 + 8 * lg + 4];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mine ? v[e] : 0.f;
        uint4 hi, lo;
        split_frag(v, hi, lo);
        // rank k's 64 bytes, piece d at d ^ turn(k); the transposing reads give a lane 8
        // ranks of its column
        auto turn = [](int k) { return ((k >> 2) & 3) ^ ((k >> 3) & 2); };
        lds_char *own = (lds_char *)sB + wave * 2048;
        asm volatile("" ::: "memory");  // the last ranks' reads come first: LDS takes a wave's accesses in order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = 16 * i + (lane >> 2), d = lane & 3;
            *(uint4 *)(own + k * 64 + ((d ^ turn(k)) << 4)) = f[i];
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k = 8 * lg + (l16 >> 2), d = 2 * t + ((l16 & 3) >> 1);
            const uint2 w0 = lds_read_tr4(own + k * 64 + ((d ^ turn(k)) << 4) + (l16 & 1) * 8);
            const uint2 w1 = lds_read_tr4(own + (k + 4) * 64 + ((d ^ turn(k + 4)) << 4) + (l16 & 1) * 8);
            const uint4 a = make_uint4(w0.x, w0.y, w1.x, w1.y);
            f32x4_t low = mfma16x16x32(a, lo, f32x4_t{0.f, 0.f, 0.f, 0.f});
            low = mfma16x16x32(a, hi, low);
#pragma unroll
            for (int e = 0; e < 4; ++e) total[t][e] += mine ? low[e] : 0.f;
        }
    };
    // Tasks wave, wave + NW, ... of `count`, one fetched ahead, after S has been staged
    auto work = [&](int count, auto &&get, auto &&staged) {
        uint4 f[2], g[2];
        I4Task now{}, after{};
        if (wave < count) now = get(wave), fetch(now, f);
        staged();
        for (int i = wave; i < count; i += NW) {
            if (i + NW < count) after = get(i + NW), fetch(after, g);
            multiply(now, f);
            now = after;
            f[0] = g[0], f[1] = g[1];
        }
    };

    if constexpr (MULTI) {
        // the first segment that ends beyond this tile's first row (segments are in row order)
        int first = 0;
        if (P.nseg > 64) {
            for (int top = P.nseg; first < top;) {
                const int mid = (first + top) >> 1;
                if (P.seg_off[mid + 1] <= (int64_t)row0) first = mid + 1;
                else top = mid;
            }
        }
#pragma unroll 1
        for (; first < P.nseg; first += 64) {
            if (tid < 16) rows[tid][0] = 0.f;
            if (wave == 0) {
                const int s = first + lane;
                bool past = false;
                int lo = 0, hi = 0, r = 0;
                lora_adapter ad{};
                if (s < P.nseg) {
                    const int64_t o0 = P.seg_off[s], o1 = P.seg_off[s + 1];
                    const int which = P.seg_adapter[s];
                    // (clamped before they are narrowed: an offset may be any int64)
                    lo = (int)min(max((int64_t)row0, o0), (int64_t)rend);
                    hi = (int)min(max((int64_t)row0, o1), (int64_t)rend);
                    past = o0 >= (int64_t)rend;
                    if (which >= 0 && which < P.num_adapters && lo < hi) {
                        ad = P.adapters[which];
                        r = ad.r < 1 || ad.r > P.RS ? 0 : ad.r;
                    }
                }
                // the tasks before this lane's
                const int mine = (r + 31) >> 5;
                int upto = mine;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int other = __shfl_up(upto, d);
                    if (lane >= d) upto += other;
                }
                for (int c = 0; c < mine; ++c) tasks[upto - mine + c] = I4Task{lo, hi, r, 32 * c, (const uint16_t *)ad.B};
                if (r > 0)
                    for (int i = lo - row0; i < hi - row0; ++i) {
                        rows[i][0] = (float)r;
                        rows[i][1] = ad.alpha;
                        rows[i][2] = drop_scale(ad.p);
                    }
                const bool last = __any(past);
                if (lane == 63) state[0] = upto, state[1] = last;
            }
            __syncthreads();
            const int count = state[0], br = tid / TPR;
            const bool last = state[1] != 0;
            work(count, [&](int i) { return tasks[i]; },
                 [&]() {
                     stage((int)rows[br][0], rows[br][1], rows[br][2]);
                     __syncthreads();
                 });
            if (last) break;
            __syncthreads();  // (the next 64 segments' tasks)
        }
    } else if (P.r > 0) {
        work((P.r + 31) >> 5, [&](int i) { return I4Task{0, P.M, P.r, 32 * i, P.B}; },
             [&]() {
                 stage(row0 + tid / TPR < P.M ? P.r : 0, P.alpha, P.undrop);
                 __syncthreads();
             });
    }

    const size_t slice = (size_t)P.M * P.N;
    const float *src = P.part + (size_t)row * P.N + col;
    for (int s = wave; s < P.KS; s += NW) {
        if (live0) total[0] += *(const f32x4_t *)(src + s * slice);
        if (live1) total[1] += *(const f32x4_t *)(src + s * slice + 16);
    }
    __syncthreads();
    f32x4_t *red = (f32x4_t *)sB;
    red[(wave * 2 + 0) * 64 + lane] = total[0];
    red[(wave * 2 + 1) * 64 + lane] = total[1];
    __syncthreads();
    if (wave >= 2) return;
    f32x4_t v = red[wave * 64 + lane];
#pragma unroll
    for (int c = 1; c < NW; ++c) v += red[(c * 2 + wave) * 64 + lane];
    if (wave == 0 ? live0 : live1)
        *(uint2 *)(P.Y + (size_t)row * P.N + col + 16 * wave) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

}  // namespace

hipError_t launch_int4_finish(const float *part, int KS, int m, int n, float *S, int SK, const float *spart, const AdapterSource &src,
                              void *Y, hipStream_t stream) {
    I4FinishParams P{};
    P.part = part;
    P.KS = KS;
    P.M = m;
    P.N = n;
    P.S = S;
    P.RS = src.r;
    P.SK = SK;
    P.spart = spart;
    P.B = (const uint16_t *)src.B;
    P.r = src.r;
    P.alpha = src.alpha;
    P.undrop = drop_scale(src.p);
    P.adapters = src.table;
    P.seg_off = src.seg_off;
    P.seg_adapter = src.seg_adapter;
    P.num_adapters = src.num_adapters;
    P.nseg = src.num_segments;
    P.Y = (uint16_t *)Y;
    const dim3 grid((unsigned)((n + 31) / 32), (unsigned)((m + 15) / 16));
    const int slot = prof_begin("int4_finish", stream);
    if (src.table != nullptr) hipLaunchKernelGGL((int4_finish_kernel<true>), grid, dim3(64 * NW), 0, stream, P);
    else hipLaunchKernelGGL((int4_finish_kernel<false>), grid, dim3(64 * NW), 0, stream, P);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
