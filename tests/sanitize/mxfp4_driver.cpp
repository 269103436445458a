// Host-only driver for the sanitizer build of the MXFP4 and AdamW entry points
// (argument checks, workspace queries, the plans of the products).  No call here
// reaches a kernel launch: every layer call fails validation or has nothing to
// do (the pointers are fake but aligned).  Exits non-zero on an unexpected
// status or a plan that does not cover its product.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "launch.hpp"
#include "lora_fused.h"

using namespace lora;

static int failures = 0;
#define EXPECT(call, want)                                                              \
    do {                                                                                \
        const lora_status _s = (call);                                                  \
        if (_s != (want)) {                                                             \
            std::fprintf(stderr, "%s:%d: %s -> %d, want %d (%s)\n", __FILE__, __LINE__, \
                         #call, (int)_s, (int)(want), lora_last_error_message());       \
            ++failures;                                                                 \
        }                                                                               \
    } while (0)
#define HOLDS(cond)                                                                                  \
    do {                                                                                             \
        if (!(cond)) {                                                                               \
            std::fprintf(stderr, "%s:%d: %s (m %lld k %lld n %lld r %d)\n", __FILE__, __LINE__, #cond, \
                         (long long)m, (long long)k, (long long)n, r);                               \
            ++failures;                                                                              \
        }                                                                                            \
    } while (0)

static void queries(int64_t m, int64_t k, int64_t n, int32_t r, int32_t adapters, int32_t segments) {
    (void)lora_mxfp4_codes_size(k, n);
    (void)lora_mxfp4_scales_size(k, n);
    (void)lora_mxfp4_frozen_fwd_workspace_size(m, k, n);
    (void)lora_mxfp4_frozen_bwd_workspace_size(m, k, n);
    const size_t sizes[] = {lora_mxfp4_linear_fwd_workspace_size(m, k, n, r), lora_mxfp4_linear_bwd_workspace_size(m, k, n, r),
                            multi_lora_mxfp4_fwd_workspace_size(m, k, n, r, adapters, segments),
                            multi_lora_mxfp4_bwd_workspace_size(m, k, n, r, adapters, segments)};
    if (r < 1 || r > 256)
        for (size_t s : sizes) HOLDS(s == 0);
    if (adapters < 0 || segments < 0)
        for (int i = 2; i < 4; ++i) HOLDS(sizes[i] == 0);
}

// A plan's tiles and slices cover the product, none is empty, and its scratch holds them.
static void plans(int64_t m, int64_t k, int64_t n, int r, int nseg) {
    const MxForm form = nseg > 0 ? kMxMixed : kMxPlain;
    const MxGemmPlan f = mx_gemm_plan(m, k, n, r, form, nseg);
    const int tms[] = {4, 4, 16, 16, 32, 32, 48, 64, 64, 128}, tns[] = {16, 32, 16, 64, 32, 128, 128, 128, 256, 256},
              kws[] = {1024, 512, 1024, 512, 512, 256, 256, 256, 128, 128};
    if (f.kind) {
        HOLDS(f.kind >= 1 && f.kind <= 10);
        const int64_t tm = tms[f.kind - 1], tn = tns[f.kind - 1], kw = kws[f.kind - 1];
        HOLDS(f.tiles_m * tm >= m && (f.tiles_m - 1) * tm < m);
        HOLDS(f.tiles_n * tn >= n && (f.tiles_n - 1) * tn < n);
        HOLDS(f.KS >= 1 && (int64_t)f.KS * f.per * kw >= k && (int64_t)(f.KS - 1) * f.per * kw < k);
        HOLDS(f.KS == 1 || f.finish);
        HOLDS(f.part_bytes == (f.finish ? (size_t)f.KS * m * n * 4 : 0));
        HOLDS((int64_t)f.tiles_m * f.tiles_n * f.KS + f.jobs < (1LL << 31) / 512);
        HOLDS(f.jobs % 8 == 0 && (f.jobs > 0) == (f.SK > 0) && (f.SK == 0 || (int64_t)f.SK * 1024 >= k));
    }
    const MxGemmTPlan b = mx_gemm_t_plan(m, k, n, r);
    if (b.kind) {
        HOLDS(b.kind >= 1 && b.kind <= 6);
        const int tmt[] = {16, 32, 48, 64, 128, 128}, tnt[] = {128, 128, 128, 128, 128, 256}, nwt[] = {256, 256, 256, 256, 128, 64};
        const int64_t tm = tmt[b.kind - 1], tn = tnt[b.kind - 1], nw = nwt[b.kind - 1];
        HOLDS(b.tiles_m * tm >= m && (b.tiles_m - 1) * tm < m);
        HOLDS(b.tiles_k * tn >= k && (b.tiles_k - 1) * tn < k);
        HOLDS(b.KS >= 1 && (int64_t)b.KS * b.per * nw >= n && (int64_t)(b.KS - 1) * b.per * nw < n);
        HOLDS(b.KS == 1 || b.finish);
        HOLDS(b.part_bytes == (b.finish ? (size_t)b.KS * m * k * 4 : 0));
        HOLDS((int64_t)b.tiles_m * b.tiles_k * b.KS < (1LL << 31) / 512);
    }
}

int main() {
    void *F = (void *)(uintptr_t)0x10000;  // aligned, never dereferenced
    float *Ff = (float *)F;
    uint32_t *Fu = (uint32_t *)F;
    const int64_t *F8 = (const int64_t *)F;
    const int32_t *F4 = (const int32_t *)F;
    const lora_adapter *Fa = (const lora_adapter *)F;
    const lora_status OK = LORA_OK, INV = LORA_ERR_INVALID_ARG, WS = LORA_ERR_WORKSPACE;
    const size_t big = (size_t)1 << 50;

    // ranks and counts outside their ranges, sizes at the ends of theirs
    const int64_t ends[] = {INT64_MIN, -1, 0, 1, 7, 8, 4096, (1 << 20) + 8, (1LL << 31) - 8, 1LL << 31, INT64_MAX};
    const int32_t few[] = {INT32_MIN, -1, 0, 1, 8, 256, 257, 1 << 29, INT32_MAX};
    for (int64_t m : ends)
        for (int64_t k : ends)
            for (int64_t n : ends) {
                // (the bf16 layer's queries take any rank, and sizes that no layer has: their plans are not asked here)
                const bool real = m < (1 << 20) && k <= (1 << 21) && n <= (1 << 21);
                for (int32_t r : few)
                    if (real || r < 1 || r > 256) queries(m, k, n, r, 8, 8);
                if (real) queries(m, k, n, 16, 0, INT32_MIN), queries(m, k, n, 16, -1, 8);
            }
    std::mt19937_64 rng(5);
    auto draw = [&](double top) { return (int64_t)std::exp2(std::uniform_real_distribution<double>(0, top)(rng)); };
    for (int i = 0; i < 20000; ++i) {
        const int64_t m = draw(i % 4 ? 13 : 21), k = std::max<int64_t>(8, draw(i % 5 ? 15 : 22) / 8 * 8),
                      n = std::max<int64_t>(8, draw(i % 5 ? 15 : 22) / 8 * 8);
        const int r = i % 3 ? (int)draw(8) : 0;
        plans(m, k, n, r, r > 0 && i % 2 ? (int)draw(10) : 0);
    }

    for (auto f : {0, 1}) {
        auto call = [&](void *W, int64_t k, int64_t n, void *c, void *s) {
            return f ? lora_mxfp4_dequantize(c, s, k, n, W, nullptr) : lora_mxfp4_quantize(W, k, n, c, s, nullptr);
        };
        EXPECT(call(nullptr, 64, 64, F, F), INV);
        EXPECT(call(F, 60, 64, F, F), INV);
        EXPECT(call(F, 64, INT64_MAX, F, F), INV);
        EXPECT(call(F, 64, 64, nullptr, F), INV);
        EXPECT(call(F, 1 << 30, 1 << 30, F, F), INV);
    }
    EXPECT(lora_mxfp4_frozen_fwd(F, F, F, 4, 60, 64, F, F, big, nullptr), INV);
    EXPECT(lora_mxfp4_frozen_fwd(F, F, F, INT64_MIN, 64, 64, F, F, big, nullptr), INV);
    EXPECT(lora_mxfp4_frozen_fwd(nullptr, F, F, 0, 64, 64, nullptr, nullptr, 0, nullptr), OK);
    EXPECT(lora_mxfp4_frozen_bwd(F, F, F, 4, 64, 64, nullptr, F, big, nullptr), INV);
    EXPECT(lora_mxfp4_frozen_bwd(nullptr, F, F, 0, 64, 64, nullptr, nullptr, 0, nullptr), OK);
    for (int32_t r : {INT32_MIN, 0, 257, INT32_MAX}) {
        EXPECT(lora_mxfp4_linear_fwd(F, F, F, F, F, 64, 64, 64, r, 1.f, 0.1f, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
        EXPECT(lora_mxfp4_linear_bwd(F, F, F, F, F, F, Ff, Fu, 64, 64, 64, r, 1.f, 0.1f, F, F, F, F, big, nullptr), INV);
        EXPECT(multi_lora_mxfp4_linear_fwd(F, F, F, Fa, 2, F8, F4, 1, 64, 64, 64, r, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
        EXPECT(multi_lora_mxfp4_linear_bwd(F, F, F, F, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, r, F, F, big, nullptr), INV);
    }
    EXPECT(lora_mxfp4_linear_fwd(F, F, F, F, F, 64, 64, 64, 8, 1.f, NAN, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(lora_mxfp4_linear_fwd(F, F, F, F, F, 64, 4096, 4096, 8, 1.f, 0.1f, 0, 0, F, Ff, Fu, F, 0, nullptr), WS);
    EXPECT(lora_mxfp4_linear_fwd(nullptr, F, F, F, F, 0, 64, 64, 8, 1.f, 0.1f, 0, 0, nullptr, nullptr, nullptr, nullptr, 0,
                                 nullptr), OK);
    EXPECT(lora_mxfp4_linear_bwd(F, F, F, F, F, F, Ff, Fu, 64, 64, 64, 8, 1.f, 0.1f, F, F, F, F, 0, nullptr), WS);
    EXPECT(multi_lora_mxfp4_linear_fwd(F, F, F, Fa, 2, F8, F4, INT32_MIN, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(multi_lora_mxfp4_linear_fwd(F, F, F, Fa, -1, F8, F4, 1, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(multi_lora_mxfp4_linear_fwd(F, F, F, Fa, 2, F8, F4, 1, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, 0, nullptr), WS);
    EXPECT(multi_lora_mxfp4_linear_bwd(F, F, F, F, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, 16, F, F, 0, nullptr), WS);

    auto adamw = [&](const lora_adamw_tensor *t, int32_t count, int bits, double lr, double b1, double eps, int64_t step) {
        return lora_adamw_step(t, count, 1, 1, bits, lr, b1, 0.999, eps, 0.01, step, nullptr, ~0ull, nullptr);
    };
    const lora_adamw_tensor good{F, F, nullptr, F, F, Ff, Ff, 0, 0};
    EXPECT(adamw(nullptr, 0, 8, 1e-3, 0.9, 1e-8, INT64_MAX), OK);
    EXPECT(adamw(nullptr, 1, 8, 1e-3, 0.9, 1e-8, 1), INV);
    EXPECT(adamw(nullptr, INT32_MIN, 8, 1e-3, 0.9, 1e-8, 1), INV);
    EXPECT(adamw(&good, 1, 8, 1e-3, 0.0, 0.0, 1), OK);
    EXPECT(adamw(&good, 1, 8, 1e-3, 0.9, 1e-8, INT64_MIN), INV);
    EXPECT(adamw(&good, 1, 9, 1e-3, 0.9, 1e-8, 1), INV);
    EXPECT(adamw(&good, 1, 8, INFINITY, 0.9, 1e-8, 1), INV);
    EXPECT(adamw(&good, 1, 8, 1e-3, 1.0, 1e-8, 1), INV);
    EXPECT(adamw(&good, 1, 8, 1e-3, 0.9, 1e-40, 1), INV);
    for (int64_t n : {INT64_MIN, (int64_t)-1, INT64_MAX}) {
        lora_adamw_tensor t = good;
        t.n = n;
        EXPECT(adamw(&t, 1, 32, 1e-3, 0.9, 1e-8, 1), INV);
    }
    std::vector<lora_adamw_tensor> many(300, good);
    EXPECT(adamw(many.data(), 300, 32, 1e-3, 0.9, 1e-8, 1), OK);
    many[299].n = 8;
    many[299].offset = 4;
    EXPECT(adamw(many.data(), 300, 32, 1e-3, 0.9, 1e-8, 1), INV);

    if (failures) return 1;
    std::puts("all checks passed");
    return 0;
}
