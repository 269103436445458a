// AdamW over many tensors in one launch:
//
//   m = b1 m + (1 - b1) g            v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// with every sum in fp32.  The moments are fp32, or 8 bits a value: e4m3
// codes of m and of u = sqrt(v) with one fp32 scale (largest / 448) for each
// block of 256 values.  u rather than v, since it needs half the range and is
// what the update divides by.
//
// The new moments are rounded to codes at random, up with the probability
// that makes the expected value exact.  A step moves v by about (1 - b2) of
// itself, far below half a step of a 4-bit significand, so rounding to the
// nearest would never move it.  A second moment above zero keeps at least the
// smallest code: with m above zero and u at zero the next update would divide
// by eps alone.
//
// A work-group takes 4096 values of one tensor and finds the tensor in the
// launch's table (kernel arguments: nothing is copied or kept).  Streaming
// bytes bound it: 16-byte loads, a block's 256 values in 32 lanes so its
// maximum takes five lane exchanges and no LDS.
#include <hip/hip_runtime.h>

#include "adamw.hpp"
#include "device_common.hpp"
#include "launch.hpp"

namespace lora {

namespace {

constexpr int kChunk = 4096;  // values per work-group: 256 threads x 8 values x 2

struct AdamwKernelTensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    uint64_t offset;
};

constexpr int kPerLaunch = 48;
struct AdamwArgs {
    AdamwKernelTensor t[kPerLaunch];
    int32_t first[kPerLaunch];  // first chunk of each tensor
    uint64_t vec;               // bit i: every pointer of tensor i is aligned for 16-byte pieces
    int32_t count;
    float decay, lr, b1, a1, b2, a2, eps;  // decay = 1 - lr wd, a = 1 - b
    float rc1, rc2;             // 1 / (1 - b^t), where t is known on the host
    float ln_b1, ln_b2;
    const int64_t *step_dev;
    uint64_t seed, step;
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

constexpr float kTop = 448.f;           // largest e4m3
constexpr float kLeast = 0.001953125f;  // smallest e4m3, 2^-9
constexpr float kTiny = 7.888609e-31f;  // 2^-100

__device__ __forceinline__ float max32(float x) {  // over the 32 lanes of a block
    x = fmaxf(x, __shfl_xor(x, 1));
    x = fmaxf(x, __shfl_xor(x, 2));
    x = fmaxf(x, __shfl_xor(x, 4));
    x = fmaxf(x, __shfl_xor(x, 8));
    return fmaxf(x, __shfl_xor(x, 16));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// y in [0, 448] to floor(y / step + r / 65536) e4m3 steps.  From 2^-6 on a
// step is the float's mantissa past 3 bits, below it is 2^-9.
__device__ __forceinline__ float e4m3_at_random(float y, uint32_t r) {
    const float big = __uint_as_float((__float_as_uint(y) + (r << 4)) & 0xFFF00000u);
    const uint32_t fixed = (uint32_t)(fminf(y, 0.015625f) * 536870912.f);  // y / 2^-9 in 2^-20 parts
    const float small = (float)((fixed + (r << 4)) >> 20) * kLeast;
    return y >= 0.015625f ? big : small;
}

template <int BITS, bool MASTER, bool PBF, bool GBF>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs P) {
    int lo = 0, hi = P.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const AdamwKernelTensor T = P.t[lo];
    const bool vec = (P.vec >> lo) & 1;
    float rc1 = P.rc1, rc2 = P.rc2;
    uint64_t step = P.step;
    if (P.step_dev != nullptr) {
        step = (uint64_t)*P.step_dev;
        rc1 = 1.f / -expm1f((float)(int64_t)step * P.ln_b1);
        rc2 = 1.f / -expm1f((float)(int64_t)step * P.ln_b2);
    }
    const uint64_t key = P.seed + step * 0x9E3779B97F4A7C15ull;
    const int64_t chunk0 = (int64_t)((int)blockIdx.x - P.first[lo]) * kChunk;

#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int64_t e0 = chunk0 + half * (kChunk / 2) + (int)threadIdx.x * 8;
        const int live = (int)max((int64_t)0, min((int64_t)8, T.n - e0));  // may be 0: the lane still joins its block's maximum
        const bool wide = vec && live == 8;
        float g[8], w[8], m[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = w[i] = m[i] = v[i] = 0.f;
        auto load_f32 = [&](const float *src, float (&x)[8]) {
            if (wide) {
                const float4 a = ((const float4 *)(src + e0))[0], b = ((const float4 *)(src + e0))[1];
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) x[i] = src[e0 + i];
            }
        };
        auto load_bf16 = [&](const uint16_t *src, float (&x)[8]) {
            if (wide) {
                const uint4 a = *(const uint4 *)(src + e0);
                const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = __uint_as_float(q[i] << 16);
                    x[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) x[i] = bf16_to_f32(src[e0 + i]);
            }
        };
        auto load_codes = [&](const uint8_t *src, float scale, float (&x)[8]) {
            uint32_t q[2] = {0u, 0u};
            if (wide) {
                const uint2 a = *(const uint2 *)(src + e0);
                q[0] = a.x, q[1] = a.y;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) q[i >> 2] |= (uint32_t)src[e0 + i] << (8 * (i & 3));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
                const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
                x[4 * i] = a[0] * scale, x[4 * i + 1] = a[1] * scale;
                x[4 * i + 2] = b[0] * scale, x[4 * i + 3] = b[1] * scale;
            }
        };
        if constexpr (GBF) load_bf16((const uint16_t *)T.grad, g);
        else load_f32((const float *)T.grad, g);
        if constexpr (MASTER) load_f32(T.master, w);
        else if constexpr (PBF) load_bf16((const uint16_t *)T.param, w);
        else load_f32((const float *)T.param, w);
        if constexpr (BITS == 32) {
            load_f32((const float *)T.m, m);
            load_f32((const float *)T.v, v);
        } else {
            const int64_t blk = e0 >> 8;
            load_codes((const uint8_t *)T.m, live > 0 ? T.m_scale[blk] : 0.f, m);
            load_codes((const uint8_t *)T.v, live > 0 ? T.v_scale[blk] : 0.f, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = P.b1 * m[i] + P.a1 * g[i];
            v[i] = P.b2 * v[i] + P.a2 * (g[i] * g[i]);
            w[i] = w[i] * P.decay - P.lr * ((m[i] * rc1) / (sqrtf(v[i] * rc2) + P.eps));
        }
        auto store_f32 = [&](float *dst, const float (&x)[8]) {
            if (wide) {
                ((float4 *)(dst + e0))[0] = make_float4(x[0], x[1], x[2], x[3]);
                ((float4 *)(dst + e0))[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) dst[e0 + i] = x[i];
            }
        };
        if constexpr (MASTER) store_f32(T.master, w);
        if constexpr (PBF) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(w[2 * i], w[2 * i + 1]);
            uint16_t *dst = (uint16_t *)T.param;
            if (wide) {
                *(uint4 *)(dst + e0) = make_uint4(q[0], q[1], q[2], q[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) dst[e0 + i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
            }
        } else {
            store_f32((float *)T.param, w);
        }
        if constexpr (BITS == 32) {
            store_f32((float *)T.m, m);
            store_f32((float *)T.v, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = sqrtf(v[i]);
            // scales from the finite values; an infinity or a NaN is stored as NaN
            float tm = 0.f, tv = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                tm = fmaxf(tm, finite(m[i]) ? fabsf(m[i]) : 0.f);
                tv = fmaxf(tv, finite(v[i]) ? v[i] : 0.f);
            }
            tm = max32(tm);
            tv = max32(tv);
            tm = tm < kTiny ? 0.f : tm;
            tv = tv < kTiny ? 0.f : tv;
            const float im = tm > 0.f ? kTop / tm : 0.f, iv = tv > 0.f ? kTop / tv : 0.f;
            float cm[8], cv[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const PhiloxOut rnd = philox10((T.offset + (uint64_t)e0) / 4 + q, key);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 4 * q + j;
                    const float a = e4m3_at_random(fminf(fabsf(m[i]) * im, kTop), rnd.w[j] & 0xFFFFu);
                    float b = e4m3_at_random(fminf(v[i] * iv, kTop), rnd.w[j] >> 16);
                    if (b == 0.f && v[i] * iv > 0.f) b = kLeast;
                    cm[i] = finite(m[i]) ? __builtin_copysignf(a, m[i]) : __builtin_nanf("");
                    cv[i] = finite(v[i]) ? b : __builtin_nanf("");
                }
            }
            auto store_codes = [&](uint8_t *dst, const float (&c)[8]) {
                uint32_t q[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    int p = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
                    q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], p, true);
                }
                if (wide) {
                    *(uint2 *)(dst + e0) = make_uint2(q[0], q[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < live) dst[e0 + i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
                }
            };
            store_codes((uint8_t *)T.m, cm);
            store_codes((uint8_t *)T.v, cv);
            if ((threadIdx.x & 31) == 0 && live > 0) {
                T.m_scale[e0 >> 8] = tm / kTop;
                T.v_scale[e0 >> 8] = tv / kTop;
            }
        }
    }
}

using AdamwFn = void (*)(AdamwArgs);
template <int BITS>
AdamwFn pick(bool master, bool pbf, bool gbf) {
    if (master) return gbf ? adamw_kernel<BITS, true, true, true> : adamw_kernel<BITS, true, true, false>;
    if (pbf) return gbf ? adamw_kernel<BITS, false, true, true> : adamw_kernel<BITS, false, true, false>;
    return gbf ? adamw_kernel<BITS, false, false, true> : adamw_kernel<BITS, false, false, false>;
}

bool wide_ok(const lora_adamw_tensor &t, int bits) {
    const uintptr_t all = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.master;
    const uintptr_t moments = (uintptr_t)t.m | (uintptr_t)t.v;
    return all % 16 == 0 && moments % (bits == 8 ? 8 : 16) == 0;
}

}  // namespace

hipError_t launch_adamw(const lora_adamw_tensor *tensors, int32_t count, const AdamwPlan &pl, hipStream_t stream) {
    const AdamwFn fn = pl.bits == 8 ? pick<8>(pl.master, pl.param_bf16, pl.grad_bf16)
                                    : pick<32>(pl.master, pl.param_bf16, pl.grad_bf16);
    AdamwArgs a{};
    a.decay = (float)(1.0 - pl.lr * pl.weight_decay);
    a.lr = (float)pl.lr;
    a.b1 = (float)pl.beta1;
    a.a1 = (float)(1.0 - pl.beta1);
    a.b2 = (float)pl.beta2;
    a.a2 = (float)(1.0 - pl.beta2);
    a.eps = (float)pl.eps;
    a.rc1 = (float)pl.rc1;
    a.rc2 = (float)pl.rc2;
    a.ln_b1 = (float)pl.ln_b1;
    a.ln_b2 = (float)pl.ln_b2;
    a.step_dev = pl.step_dev;
    a.seed = pl.seed;
    a.step = (uint64_t)pl.step;
    int64_t chunks = 0;
    auto flush = [&]() -> hipError_t {
        if (a.count == 0) return hipSuccess;
        const int slot = prof_begin("adamw", stream);
        hipLaunchKernelGGL(fn, dim3((unsigned)chunks), dim3(256), 0, stream, a);
        prof_end(slot, stream);
        a.count = 0;
        a.vec = 0;
        chunks = 0;
        return hipGetLastError();
    };
    for (int32_t i = 0; i < count; ++i) {
        const lora_adamw_tensor &t = tensors[i];
        if (t.n == 0) continue;
        const int64_t c = (t.n + kChunk - 1) / kChunk;
        if (a.count == kPerLaunch || chunks + c > kAdamwMaxChunks) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        a.t[a.count] = AdamwKernelTensor{t.param, t.grad, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, t.offset};
        a.first[a.count] = (int32_t)chunks;
        if (wide_ok(t, pl.bits)) a.vec |= 1ull << a.count;
        ++a.count;
        chunks += c;
    }
    return flush();
}

}  // namespace lora
