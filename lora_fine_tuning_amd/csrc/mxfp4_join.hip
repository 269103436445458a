// The second launch of the products over an MXFP4 weight, and over one of 4-bit integers
// of dX and of mixed batches of more than 64 rows: the partial sums of the contraction's
// slices in slice order, and the adapters' term, rounded once.
//
//   up:    Y  = sum_s part_s + alpha S B             (S: M x RS, B: r x N)
//   down:  dX = sum_s part_s + s keep.(dS A^T)       (A: N x r, s = 1 / (1 - p))
//
// for one adapter (down) or for segments of rows with an adapter each (both; one
// adapter's up form stands with its product).  Up, S is given, or it is summed here
// from the product's partial sums of keep.X A, and the first column tile writes it.
//
// A work-group takes 16 rows of 128 columns, a wave 32 columns (one word of keep a
// row).  Bound by latency: the partial sums are a few hundred KiB out of L2.  So a
// wave reads the segment table with a lane for each segment, S of all 16 rows goes
// to LDS at once, and while 32 ranks of an adapter (one MFMA step, the scaled S
// split into bf16 hi + lo) are multiplied, the next 32, or the next segment's, are
// on their way.  A lane adds an adapter's sums where its row belongs to the segment
// only, so that an infinity in one adapter's matrix stays out of the others' rows;
// rows in no segment get the product alone.  16 rows of 8 adapters (ranks 8 to 64),
// 4096 x 4096 forward: 34.5 us for the layer with the segments read and summed one
// after the other, 17.4 so.
#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace lora {

namespace {

struct MxJoinParams {
    const float *part;  // [KS][M][N]
    int KS, M, N;
    float *S;  // M x RS; r == 0 and no table: no adapter
    int RS;
    int SK;  // > 0: S is summed from spart and written
    const float *spart;
    const uint16_t *R;  // the adapter's B or A
    int r;
    float scale;
    const lora_adapter *adapters;
    const int64_t *seg_off;
    const int32_t *seg_adapter;
    int num_adapters, nseg;
    const uint32_t *keep;  // NULL: everything is kept
    int KW;
    uint16_t *Y;
};

// A segment (or the one adapter): its rows, and its adapter.
struct MxRun {
    int lo, hi, r;
    const uint16_t *R;
};

template <bool UP, bool MULTI>
__global__ __launch_bounds__(256) void mxfp4_join_kernel(MxJoinParams P) {
    __shared__ float sS[16][260];           // the rows' scaled S (rows 16 bytes past a bank period)
    __shared__ uint4 sB[UP ? 4 * 128 : 1];  // a wave's 32 ranks of 32 columns of B
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row0 = (int)blockIdx.y * 16, row = row0 + l16, rend = min(row0 + 16, P.M);
    const int c0 = (int)blockIdx.x * 128 + 32 * wave, col = c0 + 4 * lg;
    const bool live0 = row < P.M && col < P.N, live1 = row < P.M && col + 16 < P.N;
    f32x4_t total[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};

    // 32 ranks of an adapter's matrix for this wave's columns: UP rank k's pieces of
    // 16 bytes, rank 16 i + lane / 4 and piece lane mod 4; else 8 ranks of a column
    auto fetch = [&](const MxRun &it, int r0, uint4 (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[i] = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (UP) {
                const int k = r0 + 16 * i + (lane >> 2), c = c0 + 8 * (lane & 3);
                if (k < it.r && c < P.N) __builtin_memcpy(&f[i], it.R + (size_t)k * P.N + c, 16);  // (B may be unaligned)
            } else {
                const int k = c0 + 16 * i + l16, rb = r0 + 8 * lg, left = it.r - rb;
                const uint16_t *src = it.R + (size_t)k * it.r + rb;
                if (k < P.N && left >= 8) {
                    __builtin_memcpy(&f[i], src, 16);
                } else if (k < P.N && left > 0) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = e < left ? src[e] : 0u;
                    f[i] = make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7]));
                }
            }
        }
    };
    // The rows' S, 16 threads a row, 4 ranks at a time; r: the rank of this thread's row (0: no adapter)
    auto stage = [&](int r, float scale, float undrop) {
        const int br = tid >> 4, mine = row0 + br;
#pragma unroll 1
        for (int c = 4 * (tid & 15); c < ((P.RS + 31) & ~31); c += 64) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (c < r) {
                if (UP && P.SK > 0) {
                    const int rs = (P.RS + 3) & ~3;
                    const float *ps = P.spart + (size_t)mine * rs + c;
                    const size_t part = (size_t)P.M * rs;
                    f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int q = 0; q < P.SK; q += 8) {
                        f32x4_t u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[e] = q + e < P.SK ? *(const f32x4_t *)(ps + (q + e) * part) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum += u[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = c + e < r ? undrop * sum[e] : 0.f;  // (past r nothing was written)
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = c + e < r ? P.S[(size_t)mine * P.RS + c + e] : 0.f;
                }
            }
            if (UP && P.SK > 0 && blockIdx.x == 0 && r > 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < P.RS) P.S[(size_t)mine * P.RS + c + e] = v[e];
            }
            *(float4 *)&sS[br][c] = make_float4(scale * v[0], scale * v[1], scale * v[2], scale * v[3]);
        }
    };
    // The runs that `next` hands out, 32 ranks at a time
    auto multiply = [&](MxRun it, auto &&next) {
        f32x4_t low[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
        uint4 f[2];
        fetch(it, 0, f);
        __syncthreads();  // the rows' S is in place
        for (int r0 = 0;;) {
            uint4 a[2];
            if constexpr (UP) {
                // rank k's 64 bytes, piece d at d ^ turn(k); the transposing reads give
                // a lane 8 ranks of its column
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
                    a[t] = make_uint4(w0.x, w0.y, w1.x, w1.y);
                }
            } else {
                a[0] = f[0], a[1] = f[1];
            }
            MxRun after = it;
            int rnext = r0 + 32;
            bool more = true;
            if (rnext >= it.r) {
                rnext = 0;
                more = next(after);
            }
            if (more) fetch(after, rnext, f);
            const bool mine = row >= it.lo && row < it.hi;
            float v[8];
            *(float4 *)&v[0] = *(const float4 *)&sS[l16][r0 + 8 * lg];
            *(float4 *)&v[4] = *(const float4 *)&sS[l16][r0 + 8 * lg + 4];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mine ? v[e] : 0.f;
            uint4 hi, lo;
            split_frag(v, hi, lo);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                low[t] = mfma16x16x32(a[t], hi, low[t]);
                low[t] = mfma16x16x32(a[t], lo, low[t]);
            }
            if (rnext == 0) {  // the run's last ranks
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        total[t][e] = mine ? low[t][e] : total[t][e];
                        low[t][e] = 0.f;
                    }
            }
            if (!more) break;
            it = after;
            r0 = rnext;
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
        // a lane for each of 64 segments
#pragma unroll 1
        for (; first < P.nseg; first += 64) {
            const int s = first + lane;
            int lo = 0, hi = 0, r = 0;
            float scale = 0.f, undrop = 0.f;
            uint64_t R = 0;
            bool past = false;
            if (s < P.nseg) {
                const int64_t o0 = P.seg_off[s], o1 = P.seg_off[s + 1];
                lo = (int)min(max((int64_t)0, o0), (int64_t)P.M);
                hi = (int)min(max((int64_t)0, o1), (int64_t)P.M);
                past = o0 >= (int64_t)rend;
                const int which = P.seg_adapter[s];
                if (which >= 0 && which < P.num_adapters && lo < rend && hi > row0) {
                    const lora_adapter ad = P.adapters[which];
                    r = ad.r < 1 || ad.r > P.RS ? 0 : ad.r;
                    R = (uint64_t)(UP ? ad.B : ad.A);
                    undrop = drop_scale(ad.p);
                    scale = UP ? ad.alpha : undrop;
                }
            }
            const bool last = __any(past);
            uint64_t runs = __ballot(r > 0 && hi > lo);
            auto take = [&](MxRun &it) {
                if (runs == 0) return false;
                const int at = __builtin_ctzll(runs);
                runs &= runs - 1;
                it.lo = __builtin_amdgcn_readlane(lo, at);
                it.hi = __builtin_amdgcn_readlane(hi, at);
                it.r = __builtin_amdgcn_readlane(r, at);
                it.R = (const uint16_t *)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)R, at) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(R >> 32), at) << 32);
                return true;
            };
            // this thread's row of S: its segment's rank and scales
            int rr = 0;
            float rscale = 0.f, rundrop = 0.f;
            const int mine = row0 + (tid >> 4);
            for (uint64_t left = runs; left != 0; left &= left - 1) {
                const int at = __builtin_ctzll(left);
                if (mine >= __builtin_amdgcn_readlane(lo, at) && mine < __builtin_amdgcn_readlane(hi, at)) {
                    rr = __builtin_amdgcn_readlane(r, at);
                    rscale = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), at));
                    rundrop = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(undrop), at));
                }
            }
            MxRun it;
            if (take(it)) {  // (the same in every wave)
                stage(rr, rscale, rundrop);
                multiply(it, take);
                __syncthreads();  // (the next 64 segments' S)
            }
            if (last) break;
        }
    } else if (P.r > 0) {
        stage(row0 + (tid >> 4) < P.M ? P.r : 0, P.scale, 1.f);
        multiply(MxRun{0, P.M, P.r, P.R}, [](MxRun &) { return false; });
    }

    f32x4_t acc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
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
    const uint32_t word = !UP && P.keep != nullptr && live0 ? P.keep[(size_t)row * P.KW + (c0 >> 5)] : ~0u;
    uint16_t *dst = P.Y + (size_t)row * P.N + col;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = acc[t][e] + (UP || (word >> (16 * t + 4 * lg + e)) & 1u ? total[t][e] : 0.f);
        if (t == 0 ? live0 : live1) *(uint2 *)(dst + 16 * t) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
}

}  // namespace

hipError_t launch_mxfp4_join(bool up, const float *part, int KS, int m, int n, float *S, int RS, int SK,
                             const float *spart, const uint32_t *keep, const AdapterSource &src, void *Y, hipStream_t stream) {
    MxJoinParams P{};
    P.part = part;
    P.KS = KS;
    P.M = m;
    P.N = n;
    P.S = S;
    P.RS = RS;
    P.SK = SK;
    P.spart = spart;
    P.R = (const uint16_t *)(up ? src.B : src.A);
    P.r = up ? src.r : src.a_r;
    P.scale = up ? src.alpha : drop_scale(src.p);
    P.adapters = src.table;
    P.seg_off = src.seg_off;
    P.seg_adapter = src.seg_adapter;
    P.num_adapters = src.num_adapters;
    P.nseg = src.num_segments;
    P.keep = keep;
    P.KW = (n + 31) / 32;
    P.Y = (uint16_t *)Y;
    const bool multi = src.table != nullptr;
    const dim3 grid((unsigned)((n + 127) / 128), (unsigned)((m + 15) / 16));
    const int slot = prof_begin(up ? "mxfp4_join_up" : "mxfp4_join_down", stream);
    if (up) hipLaunchKernelGGL((mxfp4_join_kernel<true, true>), grid, dim3(256), 0, stream, P);
    else if (multi) hipLaunchKernelGGL((mxfp4_join_kernel<false, true>), grid, dim3(256), 0, stream, P);
    else hipLaunchKernelGGL((mxfp4_join_kernel<false, false>), grid, dim3(256), 0, stream, P);
    prof_end(slot, stream);
    return hipGetLastError();
}

}  // namespace lora
