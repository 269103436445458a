// Host-only driver for the sanitizer build of the entry points over 4-bit integer
// weights and over inputs saved in 8 bits (argument checks, workspace queries, the plans
// of the products).  No call here reaches a kernel launch: every call fails validation
// or has nothing to do (the pointers are fake but aligned).  Exits non-zero on an
// unexpected status or a plan that does not cover its product.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

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
#define HOLDS(cond)                                                                                             \
    do {                                                                                                        \
        if (!(cond)) {                                                                                          \
            std::fprintf(stderr, "%s:%d: %s (m %lld k %lld n %lld group %lld r %d)\n", __FILE__, __LINE__, #cond, \
                         (long long)m, (long long)k, (long long)n, (long long)group, r);                        \
            ++failures;                                                                                         \
        }                                                                                                       \
    } while (0)

static void queries(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r, int32_t adapters, int32_t segments) {
    (void)lora_int4_codes_size(k, n);
    (void)lora_int4_scales_size(k, n, group);
    (void)lora_int4_frozen_fwd_workspace_size(m, k, n, group);
    (void)lora_int4_frozen_bwd_workspace_size(m, k, n, group);
    (void)lora_mxint8_codes_size(m, k);
    (void)lora_mxint8_scales_size(m, k);
    size_t sizes[] = {lora_int4_linear_fwd_workspace_size(m, k, n, group, r),
                      lora_int4_linear_bwd_workspace_size(m, k, n, group, r),
                      lora_mxint8_linear_bwd_workspace_size(2, group, m, k, n, r),
                      multi_lora_int4_fwd_workspace_size(m, k, n, group, r, adapters, segments),
                      multi_lora_int4_bwd_workspace_size(m, k, n, group, r, adapters, segments),
                      multi_lora_mxint8_bwd_workspace_size(2, group, m, k, n, r, adapters, segments)};
    for (int kind : {0, 1}) {
        (void)lora_mxint8_linear_bwd_workspace_size(kind, group, m, k, n, r);
        (void)multi_lora_mxint8_bwd_workspace_size(kind, group, m, k, n, r, adapters, segments);
    }
    if (r < 1 || r > 256)
        for (size_t s : sizes) HOLDS(s == 0);
    if (adapters < 0 || segments < 0)
        for (int i = 3; i < 6; ++i) HOLDS(sizes[i] == 0);
}

// A plan's tiles and slices cover the product, none is empty, and its scratch holds them.
static void plans(int64_t m, int64_t k, int64_t n, int64_t group, int r, int nseg) {
    const I4Plan p = int4_plan(m, k, n, group, r, nseg);
    HOLDS(p.kind > 0 || m > kI4Rows || k > (1 << 20) || n > (1 << 24));
    if (!p.kind) return;
    const int tms[] = {16, 16, 16, 16, 32, 32, 48, 48, 64, 64, 128, 128, 256},
              tns[] = {16, 32, 32, 128, 32, 64, 32, 64, 64, 128, 64, 128, 128}, steps[] = {8, 8, 4, 2, 4, 4, 4, 4, 2, 2, 1, 1, 1};
    HOLDS(p.kind <= 13);
    const int64_t tm = tms[p.kind - 1], tn = tns[p.kind - 1], k128 = (k + 127) / 128;
    HOLDS(p.tiles_m * tm >= m && (p.tiles_m - 1) * tm < m);
    HOLDS(p.tiles_m == 1 || tm >= 128);
    HOLDS(p.tiles_n * tn >= n && (p.tiles_n - 1) * tn < n);
    HOLDS(p.per % steps[p.kind - 1] == 0);
    HOLDS(p.KS >= 1 && (int64_t)p.KS * p.per >= k128 && (int64_t)(p.KS - 1) * p.per < k128);
    HOLDS(p.finish == (p.KS > 1 || (r > 0 && (tm < 128 || nseg > 0))));
    HOLDS(p.part_bytes == (p.finish ? (size_t)p.KS * m * n * 4 : 0));
    HOLDS((int64_t)p.tiles_m * p.tiles_n * p.KS + p.jobs < (1LL << 31) / 512);
    HOLDS(p.jobs % 8 == 0 && (p.jobs > 0 || p.s_jobs > 0) == (p.SK > 0) && (p.SK == 0 || (p.finish && (int64_t)p.SK * 1024 >= k)));
    HOLDS(p.s_jobs == 0 || (tm >= 128 && p.jobs == 0));
    HOLDS(p.spart_bytes == (size_t)p.SK * m * ((r + 3) / 4 * 4) * 4);
}

static void plans_t(int64_t m, int64_t k, int64_t n, int64_t group, int r) {
    const I4TPlan p = int4_t_plan(m, k, n, group, r);
    if (!p.kind) return;
    const int tms[] = {16, 32, 48, 64, 128}, nwds[] = {256, 256, 256, 256, 128};
    HOLDS(p.kind <= 5);
    const int64_t tm = tms[p.kind - 1], nwd = nwds[p.kind - 1];
    HOLDS(p.tiles_m * tm >= m && (p.tiles_m - 1) * tm < m);
    HOLDS((int64_t)p.tiles_k * 128 >= k && (int64_t)(p.tiles_k - 1) * 128 < k);
    HOLDS(p.KS >= 1 && (int64_t)p.KS * p.per * nwd >= n && (int64_t)(p.KS - 1) * p.per * nwd < n);
    HOLDS(p.finish == (p.KS > 1 || r > 0));
    HOLDS(p.part_bytes == (p.finish ? (size_t)p.KS * m * k * 4 : 0));
    HOLDS((int64_t)p.tiles_m * p.tiles_k * p.KS < (1LL << 31) / 512);
    HOLDS((n + 15) / 16 * ((k + 127) / 128) * 1024 < (1LL << 31));
}

int main() {
    void *F = (void *)(uintptr_t)0x10000;  // aligned, never dereferenced
    void *odd = (void *)(uintptr_t)0x10008;
    float *Ff = (float *)F;
    uint32_t *Fu = (uint32_t *)F;
    const int64_t *F8 = (const int64_t *)F;
    const int32_t *F4 = (const int32_t *)F;
    const lora_adapter *Fa = (const lora_adapter *)F;
    const lora_status OK = LORA_OK, INV = LORA_ERR_INVALID_ARG, WS = LORA_ERR_WORKSPACE;
    const size_t big = (size_t)1 << 50;

    // ranks, counts and groups outside their ranges, sizes at the ends of theirs
    const int64_t ends[] = {INT64_MIN, -1, 0, 1, 7, 8, 4096, (1 << 20) + 8, (1LL << 31) - 8, 1LL << 31, INT64_MAX};
    const int64_t groups[] = {INT64_MIN, -128, 0, 1, 32, 64, 96, 128, 1 << 20, 1LL << 31, INT64_MAX};
    const int32_t few[] = {INT32_MIN, -1, 0, 1, 8, 256, 257, INT32_MAX};
    for (int64_t m : ends)
        for (int64_t k : ends)
            for (int64_t n : ends)
                for (int64_t g : groups) {
                    // (the bf16 layer's queries take sizes that no layer has: their plans are not asked here)
                    const bool real = m < (1 << 20) && k <= (1 << 21) && n <= (1 << 21);
                    for (int32_t r : few)
                        if (real || r < 1 || r > 256) queries(m, k, n, g, r, 8, 8);
                    if (real) queries(m, k, n, g, 16, 0, INT32_MIN), queries(m, k, n, g, 16, -1, 8);
                }
    std::mt19937_64 rng(7);
    auto draw = [&](double top) { return (int64_t)std::exp2(std::uniform_real_distribution<double>(0, top)(rng)); };
    for (int i = 0; i < 20000; ++i) {
        const int64_t m = draw(i % 4 ? 11 : 20), k = std::max<int64_t>(8, draw(i % 5 ? 15 : 21) / 8 * 8),
                      n = std::max<int64_t>(8, draw(i % 5 ? 15 : 25) / 8 * 8);
        const int64_t group = i % 7 == 0 ? 32 : i % 7 == 1 ? 64 : 128 * (i % 7 == 2 ? draw(10) : 1);
        const int r = i % 3 ? (int)draw(8) : 0;
        plans(m, k, n, group, r, r > 0 && i % 2 ? (int)draw(10) : 0);
        plans_t(m, k, n, group, r);
    }

    // (a plan is remembered by all that it depends on: no group stands for segments)
    for (int64_t group : {(int64_t)128, ((int64_t)1 << 22) + 128})
        for (int nseg : {0, 1, 0}) plans(1000, 4096, 4096, group, 16, nseg);

    // packing
    for (int64_t g : {(int64_t)0, (int64_t)-32, (int64_t)16, (int64_t)96, (int64_t)200, INT64_MIN, INT64_MAX}) {
        EXPECT(lora_int4_quantize(F, 64, 64, g, 0, F, F, nullptr), INV);
        EXPECT(lora_int4_pack(F, F, 0, nullptr, 64, 64, g, F, F, nullptr), INV);
        EXPECT(lora_int4_dequantize(F, F, 64, 64, g, F, nullptr), INV);
        EXPECT(lora_int4_frozen_fwd(F, F, F, g, 4, 64, 64, F, F, big, nullptr), INV);
        EXPECT(lora_mxint8_linear_bwd(F, F, F, 2, F, F, g, F, F, Ff, Fu, 4, 64, 64, 8, 1.f, 0.f, F, F, F, F, big, nullptr), INV);
    }
    EXPECT(lora_int4_quantize(nullptr, 64, 64, 32, 0, F, F, nullptr), INV);
    EXPECT(lora_int4_quantize(F, 60, 64, 32, 0, F, F, nullptr), INV);
    EXPECT(lora_int4_quantize(F, 64, INT64_MAX, 32, 0, F, F, nullptr), INV);
    EXPECT(lora_int4_quantize(F, 1 << 30, 1 << 30, 32, 0, F, F, nullptr), INV);
    EXPECT(lora_int4_quantize(F, 64, 64, 32, 0, odd, F, nullptr), INV);
    for (int32_t t : {INT32_MIN, -1, 3, INT32_MAX}) EXPECT(lora_int4_pack(F, F, t, nullptr, 64, 64, 32, F, F, nullptr), INV);
    EXPECT(lora_int4_pack(nullptr, F, 0, nullptr, 64, 64, 32, F, F, nullptr), INV);
    EXPECT(lora_int4_pack(F, nullptr, 0, nullptr, 64, 64, 32, F, F, nullptr), INV);
    EXPECT(lora_mxint8_quantize(F, INT64_MIN, 64, F, F, nullptr), INV);
    EXPECT(lora_mxint8_quantize(F, 4, 60, F, F, nullptr), INV);
    EXPECT(lora_mxint8_quantize(nullptr, 4, 64, F, F, nullptr), INV);
    EXPECT(lora_mxint8_quantize(F, 4, 64, odd, F, nullptr), INV);
    EXPECT(lora_mxint8_quantize(nullptr, 0, 64, nullptr, nullptr, nullptr), OK);
    EXPECT(lora_mxint8_dequantize(F, F, INT64_MAX, 64, F, nullptr), INV);
    EXPECT(lora_mxint8_dequantize(nullptr, nullptr, 0, 64, nullptr, nullptr), OK);

    // the layers over a 4-bit weight
    EXPECT(lora_int4_frozen_fwd(F, F, F, 32, INT64_MIN, 64, 64, F, F, big, nullptr), INV);
    EXPECT(lora_int4_frozen_fwd(nullptr, F, F, 32, 0, 64, 64, nullptr, nullptr, 0, nullptr), OK);
    EXPECT(lora_int4_frozen_fwd(F, F, F, 32, 4000, 4096, 4096, F, F, 0, nullptr), WS);
    EXPECT(lora_int4_frozen_bwd(F, F, F, 32, 4, 64, 64, nullptr, F, big, nullptr), INV);
    EXPECT(lora_int4_frozen_bwd(F, F, F, 32, 4000, 4096, 4096, F, F, 0, nullptr), WS);
    EXPECT(lora_int4_frozen_bwd(nullptr, F, F, 32, 0, 64, 64, nullptr, nullptr, 0, nullptr), OK);
    for (int32_t r : {INT32_MIN, 0, 257, INT32_MAX}) {
        EXPECT(lora_int4_linear_fwd(F, F, F, 64, F, F, 64, 64, 64, r, 1.f, 0.1f, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
        EXPECT(lora_int4_linear_bwd(F, F, F, F, 64, F, F, Ff, Fu, 64, 64, 64, r, 1.f, 0.1f, F, F, F, F, big, nullptr), INV);
        EXPECT(multi_lora_int4_linear_fwd(F, F, F, 64, Fa, 2, F8, F4, 1, 64, 64, 64, r, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
        EXPECT(multi_lora_int4_linear_bwd(F, F, F, F, 64, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, r, F, F, big, nullptr), INV);
        EXPECT(multi_lora_mxint8_linear_bwd(F, F, F, 0, F, nullptr, 0, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, r, F, F, big, nullptr), INV);
    }
    EXPECT(lora_int4_linear_fwd(F, F, F, 64, F, F, 64, 64, 64, 8, 1.f, NAN, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(lora_int4_linear_fwd(F, F, F, 64, F, F, 64, 64, 64, 8, 1.f, 0.1f, 0, 0, F, Ff, nullptr, F, big, nullptr), INV);
    EXPECT(lora_int4_linear_fwd(F, F, F, 64, F, F, 64, 4096, 4096, 8, 1.f, 0.1f, 0, 0, F, Ff, Fu, F, 0, nullptr), WS);
    EXPECT(lora_int4_linear_fwd(nullptr, F, F, 64, F, F, 0, 64, 64, 8, 1.f, 0.1f, 0, 0, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
           OK);
    EXPECT(lora_int4_linear_bwd(F, F, F, F, 64, F, F, Ff, Fu, 64, 64, 64, 8, 1.f, 0.1f, F, F, F, F, 0, nullptr), WS);
    EXPECT(multi_lora_int4_linear_fwd(F, F, F, 64, Fa, 2, F8, F4, INT32_MIN, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(multi_lora_int4_linear_fwd(F, F, F, 64, Fa, -1, F8, F4, 1, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, big, nullptr), INV);
    EXPECT(multi_lora_int4_linear_fwd(F, F, F, 64, Fa, 2, F8, F4, 1, 64, 64, 64, 16, 0, 0, F, Ff, Fu, F, 0, nullptr), WS);
    EXPECT(multi_lora_int4_linear_bwd(F, F, F, F, 64, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, 16, F, F, 0, nullptr), WS);

    // the backward from a saved input
    for (int32_t kind : {INT32_MIN, -1, 3, INT32_MAX})
        EXPECT(lora_mxint8_linear_bwd(F, F, F, kind, F, F, 32, F, F, Ff, Fu, 4, 64, 64, 8, 1.f, 0.f, F, F, F, F, big, nullptr), INV);
    for (int32_t kind : {0, 1, 2}) {
        EXPECT(lora_mxint8_linear_bwd(F, F, F, kind, F, F, 32, F, F, Ff, Fu, 4, 64, 64, 8, 1.f, 0.1f, F, F, F, F, 0, nullptr), WS);
        EXPECT(lora_mxint8_linear_bwd(F, odd, F, kind, F, F, 32, F, F, Ff, Fu, 4, 64, 64, 8, 1.f, 0.1f, F, F, F, F, big, nullptr), INV);
        EXPECT(lora_mxint8_linear_bwd(F, F, F, kind, nullptr, F, 32, F, F, Ff, Fu, 4, 64, 64, 8, 1.f, 0.1f, F, F, F, F, big, nullptr),
               INV);
        EXPECT(lora_mxint8_linear_bwd(F, F, F, kind, F, F, 32, F, F, Ff, nullptr, 4, 64, 64, 8, 1.f, 0.1f, F, F, F, F, big, nullptr), INV);
        EXPECT(multi_lora_mxint8_linear_bwd(F, F, F, kind, F, F, 32, Fa, 2, F8, F4, 1, Ff, Fu, 64, 64, 64, 16, F, F, 0, nullptr), WS);
        EXPECT(multi_lora_mxint8_linear_bwd(F, F, F, kind, F, F, 32, Fa, 2, F8, F4, INT32_MIN, Ff, Fu, 64, 64, 64, 16, F, F, big, nullptr),
               INV);
    }

    if (failures) return std::fprintf(stderr, "%d failures\n", failures), 1;
    std::printf("all checks passed\n");
    return 0;
}
