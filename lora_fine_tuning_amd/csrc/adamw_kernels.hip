// AdamW over many tensors in one launch:
//
//   m = b1 m + (1 - b1) g            v = b2 v + (1 - b2) g^2
//   w = w - (lr wd w + lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
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
// A work-group takes 2048 values of one tensor and finds the tensor in the
// launch's table (kernel arguments: nothing is copied or kept).  A full chunk
// takes 8 values a lane: 16-byte loads, and a block's 256 values in 32 lanes, so
// its maximum takes five lane exchanges and no LDS.  A tensor's last, partial
// chunk takes a value a lane, a block the whole work-group: both forms are short,
// and none has a bounds check for each value of a vector.
#include <hip/hip_runtime.h>

#include <cmath>

#include "adamw.hpp"
#include "device_common.hpp"
#include "launch.hpp"

namespace lora {

namespace {

constexpr int kChunk = 2048;  // values per work-group: 256 threads x 8 values

struct AdamwKernelTensor {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    uint64_t offset;
};

// A tensor in a launch's arguments: its seven addresses and n in 48 bits each, so
// that 64 tensors fit (448 tensors: 7 launches, not 10 of 48; 185 -> 168 us).
struct AdamwRecord {
    uint32_t low[8], high[4];
    uint64_t offset;
};

constexpr int kPerLaunch = 64;
struct AdamwArgs {
    AdamwRecord t[kPerLaunch];
    int32_t first[kPerLaunch];  // first chunk of each tensor
    int32_t count;
    float lr_wd, lr, b1, a1, b2, a2, eps;  // lr_wd = lr wd, a = 1 - b
    float rc1, rc2;                        // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t), where t is known on the host
    float ln_b1, ln_b2;
    const int64_t *step_dev;
    uint64_t seed, step;
};
static_assert(sizeof(AdamwArgs) <= 4096 && kPerLaunch <= 64, "kernel arguments; a lane for each tensor");
static_assert(kAdamwMaxValues < (1LL << 48), "n in 48 bits");

AdamwRecord pack_record(const lora_adamw_tensor &t) {
    const uint64_t v[8] = {(uint64_t)t.param, (uint64_t)t.grad,    (uint64_t)t.master,  (uint64_t)t.m,
                           (uint64_t)t.v,     (uint64_t)t.m_scale, (uint64_t)t.v_scale, (uint64_t)t.n};
    AdamwRecord r{};
    for (int i = 0; i < 8; ++i) {
        r.low[i] = (uint32_t)v[i];
        r.high[i / 2] |= (uint32_t)((v[i] >> 32) & 0xFFFF) << (16 * (i & 1));
    }
    r.offset = t.offset;
    return r;
}

__device__ __forceinline__ AdamwKernelTensor unpack_record(const AdamwRecord &r) {
    auto value = [&](int i) { return (uint64_t)r.low[i] | (uint64_t)((r.high[i / 2] >> (16 * (i & 1))) & 0xFFFFu) << 32; };
    AdamwKernelTensor t;
    t.param = (void *)value(0);
    t.grad = (const void *)value(1);
    t.master = (float *)value(2);
    t.m = (void *)value(3);
    t.v = (void *)value(4);
    t.m_scale = (float *)value(5);
    t.v_scale = (float *)value(6);
    t.n = (int64_t)value(7);
    t.offset = r.offset;
    return t;
}

constexpr float kTop = 448.f;           // largest e4m3
constexpr float kTiny = 7.888609e-31f;  // 2^-100
constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

struct AdamwStep {
    float b1, a1, b2, a2, lr_wd, lr, eps, rc1, rc2;
    // One value: m, v and w after the step, and the new root of v.  v_sqrt and
    // v_rcp are within one unit in the last place; the update is the one place
    // that uses them.  Decay and update make one difference, subtracted from w in
    // one rounding: a factor 1 - lr wd in fp32 would round lr wd itself to a
    // multiple of 2^-24, for every value and step alike (1.4% too strong at 1e-6,
    // nothing at 2e-8).  (The median keeps an infinite w from becoming NaN.)
    __device__ __forceinline__ float operator()(float g, float &w, float &m, float &v) const {
        m = b1 * m + a1 * g;
        v = b2 * v + a2 * (g * g);
        const float u = __builtin_amdgcn_sqrtf(v);
        w -= __builtin_fmaf(lr_wd, __builtin_amdgcn_fmed3f(w, -kLargest, kLargest),
                            lr * ((m * rc1) * __builtin_amdgcn_rcpf(u * rc2 + eps)));
        return u;
    }
};

// x / scale (inv = 1 / scale) to one of its two e4m3 neighbours, the upper one in
// magnitude where the fraction of a step and r / 65536 make 1 or more, with r in
// the high half of `r16_high`.
__device__ __forceinline__ uint32_t e4m3_at_random(float x, float inv, uint32_t r16_high) {
    const float y = __builtin_copysignf(fminf(fabsf(x) * inv, kTop), x);
    return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y, (int)r16_high, 0, 0) & 255u;
}

template <int BITS, bool MASTER, bool PBF, bool GBF>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs P) {
    const int tid = threadIdx.x, lane = tid & 63;
    // the tensor whose chunks include this work-group's: a lane looks at each
    const int32_t mine = lane < P.count ? P.first[min(lane, kPerLaunch - 1)] : 0x7FFFFFFF;
    const int at = __builtin_popcountll(__ballot(mine <= (int)blockIdx.x)) - 1;
    const AdamwKernelTensor T = unpack_record(P.t[at]);
    const int64_t e0 = (int64_t)((int)blockIdx.x - P.first[at]) * kChunk;
    AdamwStep step{P.b1, P.a1, P.b2, P.a2, P.lr_wd, P.lr, P.eps, P.rc1, P.rc2};
    uint64_t t = P.step;
    if (P.step_dev != nullptr) {
        t = (uint64_t)*P.step_dev;
        step.rc1 = 1.f / -expm1f((float)(int64_t)t * P.ln_b1);
        step.rc2 = 1.f / sqrtf(-expm1f((float)(int64_t)t * P.ln_b2));
    }
    const uint64_t key = P.seed + t * 0x9E3779B97F4A7C15ull;

    if (e0 + kChunk <= T.n) {
        const int64_t e = e0 + tid * 8;
        float g[8], w[8], m[8], v[8];
        // (whole vectors at the alignment of their values)
        auto load_f32 = [&](const void *src, float (&x)[8]) { __builtin_memcpy(x, (const float *)src + e, 32); };
        auto store_f32 = [&](void *dst, const float (&x)[8]) { __builtin_memcpy((float *)dst + e, x, 32); };
        auto load_bf16 = [&](const void *src, float (&x)[8]) {
            uint32_t q[4];
            __builtin_memcpy(q, (const uint16_t *)src + e, 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(q[i] << 16);
                x[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
            }
        };
        uint32_t qm[2], qv[2];
        float sm = 0.f, sv = 0.f;
        if constexpr (BITS == 8) {
            __builtin_memcpy(qm, (const uint8_t *)T.m + e, 8);
            __builtin_memcpy(qv, (const uint8_t *)T.v + e, 8);
            sm = T.m_scale[e >> 8];
            sv = T.v_scale[e >> 8];
        } else {
            load_f32(T.m, m);
            load_f32(T.v, v);
        }
        if constexpr (GBF) load_bf16(T.grad, g);
        else load_f32(T.grad, g);
        if constexpr (MASTER) load_f32(T.master, w);
        else if constexpr (PBF) load_bf16(T.param, w);
        else load_f32(T.param, w);
        if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)qm[i], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)qm[i], true);
                const auto v0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)qv[i], false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)qv[i], true);
                m[4 * i] = m0[0] * sm, m[4 * i + 1] = m0[1] * sm, m[4 * i + 2] = m1[0] * sm, m[4 * i + 3] = m1[1] * sm;
                v[4 * i] = v0[0] * sv, v[4 * i + 1] = v0[1] * sv, v[4 * i + 2] = v1[0] * sv, v[4 * i + 3] = v1[1] * sv;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= v[i];
        }
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = step(g[i], w[i], m[i], v[i]);
        if constexpr (MASTER) store_f32(T.master, w);
        if constexpr (PBF) {
            const uint32_t q[4] = {pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]),
                                   pack_bf16x2(w[6], w[7])};
            __builtin_memcpy((uint16_t *)T.param + e, q, 16);
        } else {
            store_f32(T.param, w);
        }
        if constexpr (BITS == 32) {
            store_f32(T.m, m);
            store_f32(T.v, v);
        } else {
            float tm = 0.f, tv = 0.f, odd = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                tm = fmaxf(tm, fabsf(m[i]));
                tv = fmaxf(tv, u[i]);
                odd += (m[i] + u[i]) * 0.f;  // NaN if any of them is infinite or NaN
            }
            const bool strange = __any(odd != 0.f || odd != odd);
            if (strange) {  // scales from the finite values; the others are stored as NaN
                tm = tv = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    tm = fmaxf(tm, finite(m[i]) ? fabsf(m[i]) : 0.f);
                    tv = fmaxf(tv, finite(u[i]) ? u[i] : 0.f);
                }
            }
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                tm = fmaxf(tm, __shfl_xor(tm, d));
                tv = fmaxf(tv, __shfl_xor(tv, d));
            }
            tm = tm < kTiny ? 0.f : tm;
            tv = tv < kTiny ? 0.f : tv;
            const float im = tm > 0.f ? kTop / tm : 0.f, iv = tv > 0.f ? kTop / tv : 0.f;
            uint32_t cm[2] = {0u, 0u}, cv[2] = {0u, 0u};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const PhiloxOut rnd = philox10((T.offset + (uint64_t)e) / 4 + q, key);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 4 * q + j;
                    uint32_t a = e4m3_at_random(m[i], im, rnd.w[j] << 16);
                    uint32_t b = e4m3_at_random(u[i], iv, rnd.w[j] & 0xFFFF0000u);
                    if (u[i] * iv > 0.f) b = max(b, 1u);
                    if (strange) {
                        a = finite(m[i]) ? a : 0x7Fu;
                        b = finite(u[i]) ? b : 0x7Fu;
                    }
                    cm[q] |= a << (8 * j);
                    cv[q] |= b << (8 * j);
                }
            }
            __builtin_memcpy((uint8_t *)T.m + e, cm, 8);
            __builtin_memcpy((uint8_t *)T.v + e, cv, 8);
            if ((tid & 31) == 0) {
                T.m_scale[e >> 8] = tm / kTop;
                T.v_scale[e >> 8] = tv / kTop;
            }
        }
        return;
    }

    __shared__ float tops[2][8];
#pragma unroll 1
    for (int p = 0; p < kChunk / 256 && e0 + 256 * p < T.n; ++p) {
        const int64_t e = e0 + 256 * p + tid;
        const bool live = e < T.n;
        const int64_t i = live ? e : T.n - 1;  // (in bounds; its result is dropped)
        const float g = GBF ? bf16_to_f32(((const uint16_t *)T.grad)[i]) : ((const float *)T.grad)[i];
        float w = MASTER ? T.master[i] : PBF ? bf16_to_f32(((const uint16_t *)T.param)[i]) : ((const float *)T.param)[i];
        float m, v;
        if constexpr (BITS == 32) {
            m = ((const float *)T.m)[i];
            v = ((const float *)T.v)[i];
        } else {
            m = __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t *)T.m)[i], 0) * T.m_scale[i >> 8];
            v = __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t *)T.v)[i], 0) * T.v_scale[i >> 8];
            v *= v;
        }
        const float u = step(g, w, m, v);
        if constexpr (BITS == 8) {
            float tm = live && finite(m) ? fabsf(m) : 0.f, tv = live && finite(u) ? u : 0.f;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                tm = fmaxf(tm, __shfl_xor(tm, d));
                tv = fmaxf(tv, __shfl_xor(tv, d));
            }
            if (lane == 0) tops[p & 1][tid >> 6] = tm, tops[p & 1][4 + (tid >> 6)] = tv;
            __syncthreads();  // (every lane has read its moments and scales too)
            const float *o = tops[p & 1];
            tm = fmaxf(fmaxf(o[0], o[1]), fmaxf(o[2], o[3]));
            tv = fmaxf(fmaxf(o[4], o[5]), fmaxf(o[6], o[7]));
            tm = tm < kTiny ? 0.f : tm;
            tv = tv < kTiny ? 0.f : tv;
            const float im = tm > 0.f ? kTop / tm : 0.f, iv = tv > 0.f ? kTop / tv : 0.f;
            const uint64_t c = T.offset + (uint64_t)e;
            const PhiloxOut rnd = philox10(c / 4, key);
            const int j = (int)(c & 3);
            const uint32_t r = j == 0 ? rnd.w[0] : j == 1 ? rnd.w[1] : j == 2 ? rnd.w[2] : rnd.w[3];
            uint32_t a = e4m3_at_random(m, im, r << 16), b = e4m3_at_random(u, iv, r & 0xFFFF0000u);
            if (u * iv > 0.f) b = max(b, 1u);
            if (live) {
                ((uint8_t *)T.m)[e] = finite(m) ? (uint8_t)a : 0x7F;
                ((uint8_t *)T.v)[e] = finite(u) ? (uint8_t)b : 0x7F;
                if (tid == 0) {
                    T.m_scale[e >> 8] = tm / kTop;
                    T.v_scale[e >> 8] = tv / kTop;
                }
            }
        } else if (live) {
            ((float *)T.m)[e] = m;
            ((float *)T.v)[e] = v;
        }
        if (live) {
            if constexpr (MASTER) T.master[e] = w;
            if constexpr (PBF) ((uint16_t *)T.param)[e] = (uint16_t)(pack_bf16x2(w, 0.f) & 0xFFFFu);
            else ((float *)T.param)[e] = w;
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

}  // namespace

hipError_t launch_adamw(const lora_adamw_tensor *tensors, int32_t count, const AdamwPlan &pl, hipStream_t stream) {
    const AdamwFn fn = pl.bits == 8 ? pick<8>(pl.master, pl.param_bf16, pl.grad_bf16)
                                    : pick<32>(pl.master, pl.param_bf16, pl.grad_bf16);
    AdamwArgs a{};
    a.lr_wd = (float)(pl.lr * pl.weight_decay);
    a.lr = (float)pl.lr;
    a.b1 = (float)pl.beta1;
    a.a1 = (float)(1.0 - pl.beta1);
    a.b2 = (float)pl.beta2;
    a.a2 = (float)(1.0 - pl.beta2);
    a.eps = (float)pl.eps;
    a.rc1 = (float)pl.rc1;
    a.rc2 = (float)std::sqrt(pl.rc2);
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
        a.t[a.count] = pack_record(t);
        a.first[a.count] = (int32_t)chunks;
        ++a.count;
        chunks += c;
    }
    return flush();
}

}  // namespace lora
