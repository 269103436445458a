// The second launch of the products over an MXFP4 weight: the partial sums of
// the contraction's slices in slice order, and the adapters' term, rounded once.
//
//   up:    Y  = sum_s part_s + alpha S B             (S: M x RS, B: r x N)
//   down:  dX = sum_s part_s + s keep.(dS A^T)       (A: N x r, s = 1 / (1 - p))
//
// for one adapter (down) or for segments of rows with an adapter each (both; one
// adapter's up form stands with its product).  Up, S is given, or it is summed here
// from the product's partial sums of keep.X A, and the first column tile writes it.  A
// work-group takes 16 rows of 128 columns, a wave 32 columns (one word of keep a
// row); it meets the segments of its rows one after the other.  32 ranks are one
// MFMA step, the scaled S split into bf16 hi + lo.  A lane adds an adapter's sums
// where its row belongs to the segment only, so that an infinity in one
// adapter's matrix stays out of the others' rows; rows in no segment get the
// product alone.  Bound by the partial sums: a few hundred KiB out of L2.
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

template <bool UP, bool MULTI>
__global__ __launch_bounds__(256) void mxfp4_join_kernel(MxJoinParams P) {
    __shared__ uint4 sB[UP ? 4 * 128 : 1];  // a wave's 32 ranks of 32 columns of B
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row0 = (int)blockIdx.y * 16, row = row0 + l16, rend = min(row0 + 16, P.M);
    const int c0 = (int)blockIdx.x * 128 + 32 * wave, col = c0 + 4 * lg;
    const bool live0 = row < P.M && col < P.N, live1 = row < P.M && col + 16 < P.N;
    f32x4_t total[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};

    auto adapter = [&](const uint16_t *R, int r, float scale, float undrop, bool mine) {
        f32x4_t low[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
        for (int r0 = 0; r0 < r; r0 += 32) {
            const int rb = r0 + 8 * lg, left = r - rb;  // this lane's ranks rb .. rb+7
            float *s = P.S + (size_t)row * P.RS + rb;
            float v[8];
            if (UP && P.SK > 0) {
                const int rs = (P.RS + 3) & ~3;
                f32x4_t u[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
                const float *ps = P.spart + (size_t)row * rs + rb;
#pragma unroll 4
                for (int c = 0; c < P.SK; ++c) {
                    if (mine && left > 0) u[0] += *(const f32x4_t *)(ps + (size_t)c * P.M * rs);
                    if (mine && left > 4) u[1] += *(const f32x4_t *)(ps + (size_t)c * P.M * rs + 4);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = e < left ? undrop * u[e / 4][e % 4] : 0.f;  // (past the rank nothing was written)
                    if (mine && blockIdx.x == 0 && wave == 0 && rb + e < P.RS) s[e] = x;
                    v[e] = scale * x;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = mine && e < left ? scale * s[e] : 0.f;
            }
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
                    uint4 b = make_uint4(0u, 0u, 0u, 0u);
                    if (r0 + k < r && c0 + 8 * d < P.N) __builtin_memcpy(&b, R + (size_t)(r0 + k) * P.N + c0 + 8 * d, 16);
                    *(uint4 *)(own + k * 64 + ((d ^ turn(k)) << 4)) = b;
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
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    a[t] = make_uint4(0u, 0u, 0u, 0u);
                    const int k = c0 + 16 * t + l16;
                    const uint16_t *src = R + (size_t)k * r + rb;
                    if (k < P.N && left >= 8) {
                        __builtin_memcpy(&a[t], src, 16);  // (A may be unaligned)
                    } else if (k < P.N && left > 0) {
                        uint32_t h[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = e < left ? src[e] : 0u;
                        a[t] = make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7]));
                    }
                }
            }
            uint4 hi, lo;
            split_frag(v, hi, lo);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                low[t] = mfma16x16x32(a[t], hi, low[t]);
                low[t] = mfma16x16x32(a[t], lo, low[t]);
            }
        }
        if (UP && P.SK > 0 && blockIdx.x == 0 && wave == 0 && mine)  // S's columns past the rank's last 32
            for (int c = ((r + 31) & ~31) + lg; c < P.RS; c += 4) P.S[(size_t)row * P.RS + c] = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[t][e] = mine ? low[t][e] : total[t][e];
    };

    if constexpr (MULTI) {
        // the first segment that ends beyond this tile's first row (segments are in row order)
        int s = 0;
        for (int top = P.nseg; s < top;) {
            const int mid = (s + top) >> 1;
            if (P.seg_off[mid + 1] <= (int64_t)row0) s = mid + 1;
            else top = mid;
        }
        for (; s < P.nseg && P.seg_off[s] < (int64_t)rend; ++s) {
            const int lo = (int)max((int64_t)0, P.seg_off[s]), hi = (int)min(P.seg_off[s + 1], (int64_t)P.M);
            const int which = P.seg_adapter[s];
            if (which < 0 || which >= P.num_adapters || hi <= lo) continue;
            const lora_adapter ad = P.adapters[which];
            if (ad.r < 1 || ad.r > P.RS) continue;
            adapter((const uint16_t *)(UP ? ad.B : ad.A), ad.r, UP ? ad.alpha : drop_scale(ad.p),
                    drop_scale(ad.p), row >= lo && row < hi);
        }
    } else {
        adapter(P.R, P.r, P.scale, 1.f, row < P.M);
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
    P.r = src.r;
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
