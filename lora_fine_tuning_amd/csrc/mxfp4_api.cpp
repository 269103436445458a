// C-ABI entry points over a frozen weight held in MXFP4: packing, the frozen
// layer and the LoRA layer in both adapter forms.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_checks.hpp"
#include "launch.hpp"
#include "lora_fused.h"

using namespace lora;

static lora_status check_weight(int64_t k, int64_t n, const void *codes, const void *scales) {
    CHECK(check_shape(0, k, n));
    REQUIRE(k * n < (1LL << 46), "weight too large");
    REQ_PTR(codes, 16);
    REQ_PTR(scales, 16);
    return LORA_OK;
}

extern "C" size_t lora_mxfp4_codes_size(int64_t k, int64_t n) {
    if (k <= 0 || n <= 0 || k >= (1LL << 31) || n >= (1LL << 31)) return 0;
    return (size_t)mx_blocks(k) * (size_t)mx_groups(n) * 256;
}

extern "C" size_t lora_mxfp4_scales_size(int64_t k, int64_t n) { return lora_mxfp4_codes_size(k, n) / 16; }

extern "C" lora_status lora_mxfp4_quantize(const void *W, int64_t k, int64_t n, void *codes, void *scales,
                                           hipStream_t stream) {
    CHECK(check_weight(k, n, codes, scales));
    REQ_PTR(W, 16);
    HIPCHK(launch_mxfp4_quantize(W, k, n, codes, scales, stream), "MXFP4 quantise launch");
    return LORA_OK;
}

extern "C" lora_status lora_mxfp4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, void *W,
                                             hipStream_t stream) {
    CHECK(check_weight(k, n, codes, scales));
    REQ_PTR(W, 16);
    HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, W, stream), "MXFP4 dequantise launch");
    return LORA_OK;
}

// The expanded weight (none without rows) sits at the start of the workspace, the
// bf16 layer's own workspace after it.
static size_t expanded_bytes(int64_t m, int64_t k, int64_t n) { return m > 0 ? align_up((size_t)k * (size_t)n * 2) : 0; }

static bool sizes_ok(int64_t m, int64_t k, int64_t n) {
    return m >= 0 && k > 0 && n > 0 && m < (1LL << 31) && k < (1LL << 31) && n < (1LL << 31) && k * n < (1LL << 46);
}

// What the workspace queries take for a layer: ranks that a layer can have, counts
// that a plan can be sized by.
static bool ranks_ok(int32_t r, int32_t num_adapters, int32_t num_segments) {
    return r >= 1 && r <= 256 && num_adapters >= 0 && num_segments >= 0;
}

#define REQ_WORKSPACE(need)                                                                            \
    do {                                                                                               \
        if (workspace_bytes < (need))                                                                  \
            return host_fail(LORA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, (size_t)(need)); \
        if ((need) > 0) REQ_PTR(workspace, 16);                                                        \
    } while (0)

extern "C" size_t lora_mxfp4_frozen_fwd_workspace_size(int64_t m, int64_t k, int64_t n) {
    if (!sizes_ok(m, k, n) || m == 0) return 0;
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, 0, kMxPlain);
    return pl.kind ? pl.part_bytes : expanded_bytes(m, k, n);
}

extern "C" size_t lora_mxfp4_frozen_bwd_workspace_size(int64_t m, int64_t k, int64_t n) {
    if (!sizes_ok(m, k, n) || m == 0) return 0;
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, 0);
    return pl.kind ? pl.part_bytes : expanded_bytes(m, k, n);
}

extern "C" lora_status lora_mxfp4_frozen_fwd(const void *X, const void *codes, const void *scales, int64_t m,
                                             int64_t k, int64_t n, void *Y, void *workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_WORKSPACE(lora_mxfp4_frozen_fwd_workspace_size(m, k, n));
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, 0, kMxPlain);
    if (pl.kind) {
        HIPCHK(launch_mxfp4_gemm(pl, X, codes, scales, (int)m, (int)k, (int)n, AdapterSource{}, MxDropout{}, nullptr, Y,
                                 (float *)workspace, nullptr, stream), "MXFP4 product launch");
        return LORA_OK;
    }
    CHECK(check_fwd_tiles(m, k, n));
    HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return lora_frozen_fwd(X, workspace, m, k, n, Y, stream);
}

extern "C" lora_status lora_mxfp4_frozen_bwd(const void *dY, const void *codes, const void *scales, int64_t m,
                                             int64_t k, int64_t n, void *dX, void *workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(dY, 16);
    REQ_PTR(dX, 16);
    REQ_WORKSPACE(lora_mxfp4_frozen_bwd_workspace_size(m, k, n));
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, 0);
    if (pl.kind) {
        HIPCHK(launch_mxfp4_gemm_t(pl, dY, codes, scales, (int)m, (int)k, (int)n, dX, (float *)workspace, stream),
               "MXFP4 transposed product launch");
        if (pl.finish)
            HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, nullptr, 0, 0,
                                     nullptr, nullptr, AdapterSource{}, dX, stream), "MXFP4 sum launch");
        return LORA_OK;
    }
    CHECK(check_dx_tiles(m, k, n));
    HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return lora_frozen_bwd(dY, workspace, m, k, n, dX, stream);
}

extern "C" size_t lora_mxfp4_linear_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r) {
    if (!sizes_ok(m, k, n) || m == 0 || !ranks_ok(r, 0, 0)) return 0;
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, r, kMxPlain);
    if (!pl.kind) return expanded_bytes(m, k, n) + lora_linear_fwd_workspace_size(m, k, n, r);
    return align_up(pl.part_bytes) + std::max(pl.spart_bytes, lora_linear_fwd_workspace_size(m, k, n, r));
}

extern "C" size_t lora_mxfp4_linear_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r) {
    if (!sizes_ok(m, k, n) || !ranks_ok(r, 0, 0) || !bwd_k_ok(k)) return 0;
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, r);
    return (pl.kind ? align_up(pl.part_bytes) : expanded_bytes(m, k, n)) + lora_linear_bwd_workspace_size(m, k, n, r);
}

extern "C" lora_status lora_mxfp4_linear_fwd(const void *X, const void *codes, const void *scales, const void *A,
                                             const void *B, int64_t m, int64_t k, int64_t n, int32_t r,
                                             float alpha, float p, uint64_t seed, uint64_t offset, void *Y,
                                             float *S, uint32_t *keep_bits, void *workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    CHECK(check_rank(r));
    CHECK(check_p(p));
    CHECK(check_b_size(r, k, n));
    REQUIRE(offset % 8 == 0, "offset = %llu must be a multiple of 8", (unsigned long long)offset);
    REQ_PTR(A, 2);
    REQ_PTR(B, 2);
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_PTR(S, 4);
    REQUIRE(keep_bits != nullptr || p == 0.0f, "keep_bits may be NULL only when p == 0");
    REQUIRE(aligned(keep_bits, 4), "keep_bits must be 4-byte aligned");
    REQ_WORKSPACE(lora_mxfp4_linear_fwd_workspace_size(m, k, n, r));
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, r, kMxPlain);
    if (pl.kind) {
        char *rest = ws_at(workspace, align_up(pl.part_bytes));
        if (pl.SK == 0) CHECK(forward_s_only(X, A, m, k, r, p, seed, offset, S, keep_bits, rest, stream));
        HIPCHK(launch_mxfp4_gemm(pl, X, codes, scales, (int)m, (int)k, (int)n,
                                 single_source(A, B, nullptr, nullptr, r, alpha, p), MxDropout{seed, offset, keep_bits}, S,
                                 Y, (float *)workspace, (float *)rest, stream), "MXFP4 product launch");
        return LORA_OK;
    }
    const size_t w = expanded_bytes(m, k, n);
    CHECK(check_fwd_tiles(m, k, n));
    HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return lora_linear_fwd(X, workspace, A, B, m, k, n, r, alpha, p, seed, offset, Y, S, keep_bits,
                           ws_at(workspace, w), workspace_bytes - w, stream);
}

namespace lora {
lora_status mxfp4_linear_backward(const void *dY, const LayerInput &X, const void *codes, const void *scales, const AdapterSource &src,
                                  const float *S, const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n, void *dX, void *workspace,
                                  hipStream_t stream) {
    const int32_t r = src.r_cap;
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, r);
    if (pl.kind) {
        const float *dS = nullptr;
        CHECK(backward_low_rank_only(dY, X, src, S, keep_bits, m, k, n, r, ws_at(workspace, align_up(pl.part_bytes)), &dS, stream));
        if (dX != nullptr) {
            HIPCHK(launch_mxfp4_gemm_t(pl, dY, codes, scales, (int)m, (int)k, (int)n, nullptr, (float *)workspace, stream),
                   "MXFP4 transposed product launch");
            HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, (float *)dS, r, 0,
                                     nullptr, src.p == 0.0f ? nullptr : keep_bits, src, dX, stream), "MXFP4 sum launch");
        }
        return LORA_OK;
    }
    if (dX != nullptr) CHECK(check_dx_tiles(m, k, n));
    if (m > 0 && dX != nullptr)
        HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return linear_backward(dY, X, workspace, src, S, keep_bits, m, k, n, dX, ws_at(workspace, expanded_bytes(m, k, n)), stream);
}

lora_status multi_mxfp4_linear_backward(const void *dY, const LayerInput &X, const void *codes, const void *scales,
                                        const AdapterSource &src, const float *S, const uint32_t *keep_bits, int64_t m, int64_t k,
                                        int64_t n, void *dX, void *workspace, hipStream_t stream) {
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, src.r_cap);
    if (pl.kind) {
        const float *dS = nullptr;
        CHECK(multi_backward_low_rank_only(dY, X, src, S, keep_bits, m, k, n, ws_at(workspace, align_up(pl.part_bytes)), &dS, stream));
        if (dX != nullptr) {
            HIPCHK(launch_mxfp4_gemm_t(pl, dY, codes, scales, (int)m, (int)k, (int)n, nullptr, (float *)workspace, stream),
                   "MXFP4 transposed product launch");
            HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, (float *)dS, src.r_cap, 0,
                                     nullptr, keep_bits, src, dX, stream), "MXFP4 sum launch");
        }
        return LORA_OK;
    }
    if (dX != nullptr) CHECK(check_dx_tiles(m, k, n));
    if (m > 0 && dX != nullptr)
        HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return multi_linear_backward(dY, X, workspace, src, S, keep_bits, m, k, n, dX, ws_at(workspace, expanded_bytes(m, k, n)), stream);
}
}  // namespace lora

extern "C" lora_status lora_mxfp4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales,
                                             const void *A, const void *B, const float *S,
                                             const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n, int32_t r,
                                             float alpha, float p, void *dX, void *dA, void *dB, void *workspace,
                                             size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    CHECK(check_rank(r));
    CHECK(check_p(p));
    CHECK(check_b_size(r, k, n));
    CHECK(check_bwd_k(k));
    REQ_PTR(A, 2);
    REQ_PTR(B, 2);
    REQ_PTR(dA, 2);
    REQ_PTR(dB, 2);
    if (m > 0) {
        REQ_PTR(dY, 16);
        REQ_PTR(X, 16);
        REQ_PTR(S, 4);
        REQUIRE(dX == nullptr || aligned(dX, 16), "dX must be 16-byte aligned (or NULL: no input gradient)");
        REQUIRE(keep_bits != nullptr || p == 0.0f, "keep_bits may be NULL only when p == 0");
        REQUIRE(aligned(keep_bits, 4), "keep_bits must be 4-byte aligned");
    }
    REQ_WORKSPACE(lora_mxfp4_linear_bwd_workspace_size(m, k, n, r));
    return mxfp4_linear_backward(dY, X, codes, scales, single_source(A, B, dA, dB, r, alpha, p), S, keep_bits, m, k, n, dX, workspace,
                                 stream);
}

extern "C" size_t multi_lora_mxfp4_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                                      int32_t num_adapters, int32_t num_segments) {
    if (!sizes_ok(m, k, n) || m == 0 || !ranks_ok(r_max, num_adapters, num_segments)) return 0;
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, r_max, kMxMixed, num_segments);
    const size_t layer = multi_lora_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments);
    return pl.kind ? align_up(pl.part_bytes) + std::max(pl.spart_bytes, layer) : expanded_bytes(m, k, n) + layer;
}

extern "C" size_t multi_lora_mxfp4_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int32_t r_max,
                                                      int32_t num_adapters, int32_t num_segments) {
    if (!sizes_ok(m, k, n) || !ranks_ok(r_max, num_adapters, num_segments) || !bwd_k_ok(k)) return 0;
    const MxGemmTPlan pl = mx_gemm_t_plan(m, k, n, r_max);
    return (pl.kind ? align_up(pl.part_bytes) : expanded_bytes(m, k, n)) +
           multi_lora_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments);
}

extern "C" lora_status multi_lora_mxfp4_linear_fwd(const void *X, const void *codes, const void *scales,
                                                   const lora_adapter *adapters, int32_t num_adapters,
                                                   const int64_t *seg_off, const int32_t *seg_adapter,
                                                   int32_t num_segments, int64_t m, int64_t k, int64_t n,
                                                   int32_t r_max, uint64_t seed, uint64_t offset, void *Y,
                                                   float *S, uint32_t *keep_bits, void *workspace,
                                                   size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    // everything else is checked before the weight is expanded, by the call on no rows
    CHECK(multi_lora_linear_fwd(X, codes, adapters, num_adapters, seg_off, seg_adapter, num_segments, 0, k, n, r_max,
                                seed, offset, Y, S, keep_bits, workspace, workspace_bytes, stream));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_PTR(S, 4);
    REQ_PTR(keep_bits, 4);
    REQ_WORKSPACE(multi_lora_mxfp4_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments));
    const MxGemmPlan pl = mx_gemm_plan(m, k, n, r_max, kMxMixed, num_segments);
    if (pl.kind) {
        const AdapterSource src = multi_source(adapters, num_adapters, seg_off, seg_adapter, num_segments, r_max);
        char *rest = ws_at(workspace, align_up(pl.part_bytes));
        if (pl.SK == 0) CHECK(multi_forward_s_only(X, src, m, k, seed, offset, S, keep_bits, rest, stream));
        HIPCHK(launch_mxfp4_gemm(pl, X, codes, scales, (int)m, (int)k, (int)n, src, MxDropout{seed, offset, keep_bits}, S,
                                 Y, (float *)workspace, (float *)rest, stream), "MXFP4 product launch");
        return LORA_OK;
    }
    const size_t w = expanded_bytes(m, k, n);
    CHECK(check_fwd_tiles(m, k, n));
    HIPCHK(launch_mxfp4_dequantize(codes, scales, k, n, workspace, stream), "MXFP4 dequantise launch");
    return multi_lora_linear_fwd(X, workspace, adapters, num_adapters, seg_off, seg_adapter, num_segments, m, k, n,
                                 r_max, seed, offset, Y, S, keep_bits, ws_at(workspace, w), workspace_bytes - w,
                                 stream);
}

extern "C" lora_status multi_lora_mxfp4_linear_bwd(const void *dY, const void *X, const void *codes,
                                                   const void *scales, const lora_adapter *adapters,
                                                   int32_t num_adapters, const int64_t *seg_off,
                                                   const int32_t *seg_adapter, int32_t num_segments,
                                                   const float *S, const uint32_t *keep_bits, int64_t m, int64_t k,
                                                   int64_t n, int32_t r_max, void *dX, void *workspace,
                                                   size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, codes, scales));
    // (the forward on no rows makes the same checks of the adapter and segment tables, and enqueues nothing)
    CHECK(multi_lora_linear_fwd(X, codes, adapters, num_adapters, seg_off, seg_adapter, num_segments, 0, k, n, r_max,
                                0, 0, nullptr, nullptr, nullptr, workspace, workspace_bytes, stream));
    CHECK(check_bwd_k(k));
    if (m > 0) {
        REQ_PTR(dY, 16);
        REQ_PTR(X, 16);
        REQ_PTR(S, 4);
        REQ_PTR(keep_bits, 4);
        REQUIRE(dX == nullptr || aligned(dX, 16), "dX must be 16-byte aligned (or NULL: no input gradient)");
    }
    REQ_WORKSPACE(multi_lora_mxfp4_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments));
    return multi_mxfp4_linear_backward(dY, X, codes, scales,
                                       multi_source(adapters, num_adapters, seg_off, seg_adapter, num_segments, r_max), S, keep_bits, m,
                                       k, n, dX, workspace, stream);
}
