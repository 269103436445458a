// C-ABI entry points over a frozen weight of 4-bit integers in groups of rows:
// packing, the frozen layer and the LoRA layer in both adapter forms.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_checks.hpp"
#include "int4.hpp"
#include "launch.hpp"
#include "lora_fused.h"

using namespace lora;

static bool group_ok(int64_t group) { return group == 32 || group == 64 || (group > 0 && group % 128 == 0 && group < (1LL << 31)); }

static lora_status check_weight(int64_t k, int64_t n, int64_t group, const void *codes, const void *scales) {
    CHECK(check_shape(0, k, n));
    REQUIRE(k * n < (1LL << 46), "weight too large");
    REQUIRE(group_ok(group), "group = %lld must be 32, 64 or a multiple of 128", (long long)group);
    REQ_PTR(codes, 16);
    REQ_PTR(scales, 16);
    return LORA_OK;
}

static bool weight_ok(int64_t k, int64_t n, int64_t group) {
    return k > 0 && n > 0 && k < (1LL << 31) && n < (1LL << 31) && k * n < (1LL << 46) && group_ok(group);
}

extern "C" size_t lora_int4_codes_size(int64_t k, int64_t n) {
    if (!weight_ok(k, n, 128)) return 0;
    const I4Shape s = i4_shape(k, n, 128);
    return (size_t)s.k128 * (size_t)s.n16 * 1024;
}

extern "C" size_t lora_int4_scales_size(int64_t k, int64_t n, int64_t group) {
    if (!weight_ok(k, n, group)) return 0;
    const I4Shape s = i4_shape(k, n, group);
    return (size_t)s.groups * (size_t)s.n16 * 64;
}

extern "C" lora_status lora_int4_quantize(const void *W, int64_t k, int64_t n, int64_t group, int32_t symmetric, void *codes,
                                          void *scales, hipStream_t stream) {
    CHECK(check_weight(k, n, group, codes, scales));
    REQ_PTR(W, 16);
    HIPCHK(launch_int4_quantize(W, k, n, group, symmetric != 0, codes, scales, stream), "4-bit quantise launch");
    return LORA_OK;
}

extern "C" lora_status lora_int4_pack(const void *Q, const void *group_scales, int32_t scale_type, const void *zeros, int64_t k,
                                      int64_t n, int64_t group, void *codes, void *scales, hipStream_t stream) {
    CHECK(check_weight(k, n, group, codes, scales));
    REQUIRE(scale_type >= 0 && scale_type <= 2, "scale_type = %d must be 0 (fp32), 1 (bf16) or 2 (fp16)", scale_type);
    REQ_PTR(Q, 4);
    REQ_PTR(group_scales, 4);
    HIPCHK(launch_int4_pack(Q, group_scales, scale_type, zeros, k, n, group, codes, scales, stream), "4-bit pack launch");
    return LORA_OK;
}

extern "C" lora_status lora_int4_dequantize(const void *codes, const void *scales, int64_t k, int64_t n, int64_t group, void *W,
                                            hipStream_t stream) {
    CHECK(check_weight(k, n, group, codes, scales));
    REQ_PTR(W, 16);
    HIPCHK(launch_int4_dequantize(codes, scales, k, n, group, W, stream), "4-bit dequantise launch");
    return LORA_OK;
}

// The expanded weight (none without rows) sits at the start of the workspace, the
// bf16 layer's own workspace after it.
static size_t expanded_bytes(int64_t m, int64_t k, int64_t n) { return m > 0 ? align_up((size_t)k * (size_t)n * 2) : 0; }

static bool sizes_ok(int64_t m, int64_t k, int64_t n, int64_t group) { return m >= 0 && m < (1LL << 31) && weight_ok(k, n, group); }

#define REQ_WORKSPACE(need)                                                                            \
    do {                                                                                               \
        if (workspace_bytes < (need))                                                                  \
            return host_fail(LORA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, (size_t)(need)); \
        if ((need) > 0) REQ_PTR(workspace, 16);                                                        \
    } while (0)

#define EXPAND() HIPCHK(launch_int4_dequantize(codes, scales, k, n, group, workspace, stream), "4-bit dequantise launch")

extern "C" size_t lora_int4_frozen_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group) {
    if (!sizes_ok(m, k, n, group) || m == 0) return 0;
    const I4Plan pl = int4_plan(m, k, n, group, 0, 0);
    return pl.kind ? pl.part_bytes : expanded_bytes(m, k, n);
}

extern "C" size_t lora_int4_frozen_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group) {
    if (!sizes_ok(m, k, n, group) || m == 0) return 0;
    const I4TPlan pl = int4_t_plan(m, k, n, group, 0);
    return pl.kind ? pl.part_bytes : expanded_bytes(m, k, n);
}

extern "C" lora_status lora_int4_frozen_fwd(const void *X, const void *codes, const void *scales, int64_t group, int64_t m, int64_t k,
                                            int64_t n, void *Y, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_WORKSPACE(lora_int4_frozen_fwd_workspace_size(m, k, n, group));
    const I4Plan pl = int4_plan(m, k, n, group, 0, 0);
    if (pl.kind) {
        HIPCHK(launch_int4_gemm(pl, X, codes, scales, group, (int)m, (int)k, (int)n, AdapterSource{}, MxDropout{}, nullptr, Y,
                                (float *)workspace, nullptr, stream), "4-bit product launch");
        return LORA_OK;
    }
    CHECK(check_fwd_tiles(m, k, n));
    EXPAND();
    return lora_frozen_fwd(X, workspace, m, k, n, Y, stream);
}

extern "C" lora_status lora_int4_frozen_bwd(const void *dY, const void *codes, const void *scales, int64_t group, int64_t m, int64_t k,
                                            int64_t n, void *dX, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(dY, 16);
    REQ_PTR(dX, 16);
    REQ_WORKSPACE(lora_int4_frozen_bwd_workspace_size(m, k, n, group));
    const I4TPlan pl = int4_t_plan(m, k, n, group, 0);
    if (pl.kind) {
        HIPCHK(launch_int4_gemm_t(pl, dY, codes, scales, group, (int)m, (int)k, (int)n, dX, (float *)workspace, stream),
               "4-bit transposed product launch");
        if (pl.finish)
            HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, nullptr, 0, 0, nullptr, nullptr,
                                     AdapterSource{}, dX, stream), "4-bit sum launch");
        return LORA_OK;
    }
    CHECK(check_dx_tiles(m, k, n));
    EXPAND();
    return lora_frozen_bwd(dY, workspace, m, k, n, dX, stream);
}

extern "C" size_t lora_int4_linear_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r) {
    if (!sizes_ok(m, k, n, group) || m == 0 || r < 1 || r > 256) return 0;
    const I4Plan pl = int4_plan(m, k, n, group, r, 0);
    const size_t layer = lora_linear_fwd_workspace_size(m, k, n, r);
    return pl.kind ? align_up(pl.part_bytes) + std::max(pl.spart_bytes, layer) : expanded_bytes(m, k, n) + layer;
}

// What the layers' backward needs before the bf16 layer's own workspace.
static size_t weight_bytes(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r) {
    if (m == 0) return 0;
    const I4TPlan pl = int4_t_plan(m, k, n, group, r);
    return pl.kind ? align_up(pl.part_bytes) : expanded_bytes(m, k, n);
}

extern "C" size_t lora_int4_linear_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r) {
    if (!sizes_ok(m, k, n, group) || r < 1 || r > 256 || !bwd_k_ok(k)) return 0;
    return weight_bytes(m, k, n, group, r) + lora_linear_bwd_workspace_size(m, k, n, r);
}

extern "C" lora_status lora_int4_linear_fwd(const void *X, const void *codes, const void *scales, int64_t group, const void *A,
                                            const void *B, int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                                            uint64_t seed, uint64_t offset, void *Y, float *S, uint32_t *keep_bits, void *workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
    // everything else is checked before the weight is expanded, by the call on no rows
    CHECK(lora_linear_fwd(X, codes, A, B, 0, k, n, r, alpha, p, seed, offset, Y, S, keep_bits, workspace, workspace_bytes, stream));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_PTR(S, 4);
    REQUIRE(keep_bits != nullptr || p == 0.0f, "keep_bits may be NULL only when p == 0");
    REQUIRE(aligned(keep_bits, 4), "keep_bits must be 4-byte aligned");
    REQ_WORKSPACE(lora_int4_linear_fwd_workspace_size(m, k, n, group, r));
    const I4Plan pl = int4_plan(m, k, n, group, r, 0);
    if (pl.kind) {
        char *rest = ws_at(workspace, align_up(pl.part_bytes));
        if (pl.SK == 0) CHECK(forward_s_only(X, A, m, k, r, p, seed, offset, S, keep_bits, rest, stream));
        HIPCHK(launch_int4_gemm(pl, X, codes, scales, group, (int)m, (int)k, (int)n, single_source(A, B, nullptr, nullptr, r, alpha, p),
                                MxDropout{seed, offset, keep_bits}, S, Y, (float *)workspace, (float *)rest, stream),
               "4-bit product launch");
        return LORA_OK;
    }
    const size_t w = expanded_bytes(m, k, n);
    CHECK(check_fwd_tiles(m, k, n));
    EXPAND();
    return lora_linear_fwd(X, workspace, A, B, m, k, n, r, alpha, p, seed, offset, Y, S, keep_bits, ws_at(workspace, w),
                           workspace_bytes - w, stream);
}

namespace lora {
lora_status int4_linear_backward(const void *dY, const LayerInput &X, const void *codes, const void *scales, int64_t group,
                                 const AdapterSource &src, const float *S, const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n,
                                 void *dX, void *workspace, hipStream_t stream) {
    const I4TPlan pl = int4_t_plan(m, k, n, group, src.r_cap);
    char *rest = ws_at(workspace, weight_bytes(m, k, n, group, src.r_cap));
    if (pl.kind) {
        const float *dS = nullptr;
        CHECK(backward_low_rank_only(dY, X, src, S, keep_bits, m, k, n, src.r_cap, rest, &dS, stream));
        if (dX == nullptr) return LORA_OK;
        HIPCHK(launch_int4_gemm_t(pl, dY, codes, scales, group, (int)m, (int)k, (int)n, nullptr, (float *)workspace, stream),
               "4-bit transposed product launch");
        HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, (float *)dS, src.r_cap, 0, nullptr,
                                 src.p == 0.0f ? nullptr : keep_bits, src, dX, stream), "4-bit sum launch");
        return LORA_OK;
    }
    if (dX != nullptr) CHECK(check_dx_tiles(m, k, n));
    if (m > 0 && dX != nullptr) EXPAND();
    return linear_backward(dY, X, workspace, src, S, keep_bits, m, k, n, dX, rest, stream);
}

lora_status multi_int4_linear_backward(const void *dY, const LayerInput &X, const void *codes, const void *scales, int64_t group,
                                       const AdapterSource &src, const float *S, const uint32_t *keep_bits, int64_t m, int64_t k,
                                       int64_t n, void *dX, void *workspace, hipStream_t stream) {
    const I4TPlan pl = int4_t_plan(m, k, n, group, src.r_cap);
    char *rest = ws_at(workspace, weight_bytes(m, k, n, group, src.r_cap));
    if (pl.kind) {
        const float *dS = nullptr;
        CHECK(multi_backward_low_rank_only(dY, X, src, S, keep_bits, m, k, n, rest, &dS, stream));
        if (dX == nullptr) return LORA_OK;
        HIPCHK(launch_int4_gemm_t(pl, dY, codes, scales, group, (int)m, (int)k, (int)n, nullptr, (float *)workspace, stream),
               "4-bit transposed product launch");
        HIPCHK(launch_mxfp4_join(false, (const float *)workspace, pl.KS, (int)m, (int)k, (float *)dS, src.r_cap, 0, nullptr, keep_bits,
                                 src, dX, stream), "4-bit sum launch");
        return LORA_OK;
    }
    if (dX != nullptr) CHECK(check_dx_tiles(m, k, n));
    if (m > 0 && dX != nullptr) EXPAND();
    return multi_linear_backward(dY, X, workspace, src, S, keep_bits, m, k, n, dX, rest, stream);
}
}  // namespace lora

extern "C" lora_status lora_int4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales, int64_t group,
                                            const void *A, const void *B, const float *S, const uint32_t *keep_bits, int64_t m, int64_t k,
                                            int64_t n, int32_t r, float alpha, float p, void *dX, void *dA, void *dB, void *workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
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
    REQ_WORKSPACE(lora_int4_linear_bwd_workspace_size(m, k, n, group, r));
    return int4_linear_backward(dY, X, codes, scales, group, single_source(A, B, dA, dB, r, alpha, p), S, keep_bits, m, k, n, dX,
                                workspace, stream);
}

extern "C" size_t multi_lora_int4_fwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r_max, int32_t num_adapters,
                                                     int32_t num_segments) {
    if (!sizes_ok(m, k, n, group) || m == 0 || r_max < 1 || r_max > 256 || num_adapters < 0 || num_segments < 0) return 0;
    const I4Plan pl = int4_plan(m, k, n, group, r_max, num_segments);
    const size_t layer = multi_lora_fwd_workspace_size(m, k, n, r_max, num_adapters, num_segments);
    return pl.kind ? align_up(pl.part_bytes) + std::max(pl.spart_bytes, layer) : expanded_bytes(m, k, n) + layer;
}

extern "C" size_t multi_lora_int4_bwd_workspace_size(int64_t m, int64_t k, int64_t n, int64_t group, int32_t r_max, int32_t num_adapters,
                                                     int32_t num_segments) {
    if (!sizes_ok(m, k, n, group) || r_max < 1 || r_max > 256 || num_adapters < 0 || num_segments < 0 || !bwd_k_ok(k)) return 0;
    return weight_bytes(m, k, n, group, r_max) + multi_lora_bwd_workspace_size(m, k, n, r_max, num_adapters, num_segments);
}

extern "C" lora_status multi_lora_int4_linear_fwd(const void *X, const void *codes, const void *scales, int64_t group,
                                                  const lora_adapter *adapters, int32_t num_adapters, const int64_t *seg_off,
                                                  const int32_t *seg_adapter, int32_t num_segments, int64_t m, int64_t k, int64_t n,
                                                  int32_t r_max, uint64_t seed, uint64_t offset, void *Y, float *S, uint32_t *keep_bits,
                                                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
    CHECK(multi_lora_linear_fwd(X, codes, adapters, num_adapters, seg_off, seg_adapter, num_segments, 0, k, n, r_max, seed, offset, Y, S,
                                keep_bits, workspace, workspace_bytes, stream));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    REQ_PTR(Y, 16);
    REQ_PTR(S, 4);
    REQ_PTR(keep_bits, 4);
    REQ_WORKSPACE(multi_lora_int4_fwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments));
    const I4Plan pl = int4_plan(m, k, n, group, r_max, num_segments);
    if (pl.kind) {
        const AdapterSource src = multi_source(adapters, num_adapters, seg_off, seg_adapter, num_segments, r_max);
        char *rest = ws_at(workspace, align_up(pl.part_bytes));
        if (pl.SK == 0) CHECK(multi_forward_s_only(X, src, m, k, seed, offset, S, keep_bits, rest, stream));
        HIPCHK(launch_int4_gemm(pl, X, codes, scales, group, (int)m, (int)k, (int)n, src, MxDropout{seed, offset, keep_bits}, S, Y,
                                (float *)workspace, (float *)rest, stream), "4-bit product launch");
        return LORA_OK;
    }
    const size_t w = expanded_bytes(m, k, n);
    CHECK(check_fwd_tiles(m, k, n));
    EXPAND();
    return multi_lora_linear_fwd(X, workspace, adapters, num_adapters, seg_off, seg_adapter, num_segments, m, k, n, r_max, seed, offset, Y,
                                 S, keep_bits, ws_at(workspace, w), workspace_bytes - w, stream);
}

extern "C" lora_status multi_lora_int4_linear_bwd(const void *dY, const void *X, const void *codes, const void *scales, int64_t group,
                                                  const lora_adapter *adapters, int32_t num_adapters, const int64_t *seg_off,
                                                  const int32_t *seg_adapter, int32_t num_segments, const float *S,
                                                  const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n, int32_t r_max, void *dX,
                                                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(k, n, group, codes, scales));
    // (the forward on no rows makes the same checks of the adapter and segment tables, and enqueues nothing)
    CHECK(multi_lora_linear_fwd(X, codes, adapters, num_adapters, seg_off, seg_adapter, num_segments, 0, k, n, r_max, 0, 0, nullptr,
                                nullptr, nullptr, workspace, workspace_bytes, stream));
    CHECK(check_bwd_k(k));
    if (m > 0) {
        REQ_PTR(dY, 16);
        REQ_PTR(X, 16);
        REQ_PTR(S, 4);
        REQ_PTR(keep_bits, 4);
        REQUIRE(dX == nullptr || aligned(dX, 16), "dX must be 16-byte aligned (or NULL: no input gradient)");
    }
    REQ_WORKSPACE(multi_lora_int4_bwd_workspace_size(m, k, n, group, r_max, num_adapters, num_segments));
    return multi_int4_linear_backward(dY, X, codes, scales, group,
                                      multi_source(adapters, num_adapters, seg_off, seg_adapter, num_segments, r_max), S, keep_bits, m,
                                      k, n, dX, workspace, stream);
}
