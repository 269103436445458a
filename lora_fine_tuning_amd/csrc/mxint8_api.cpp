// C-ABI entry points for a layer's input saved in 8 bits (MXINT8), and the layer's
// backward from it in both adapter forms, over a frozen weight in any of its forms.
#include <hip/hip_runtime.h>

#include "api_checks.hpp"
#include "launch.hpp"
#include "lora_fused.h"

using namespace lora;

static lora_status check_input(int64_t m, int64_t k, const void *codes, const void *scales) {
    CHECK(check_shape(m, k, 8));
    if (m == 0) return LORA_OK;
    REQ_PTR(codes, 16);
    REQ_PTR(scales, 4);
    return LORA_OK;
}

extern "C" size_t lora_mxint8_codes_size(int64_t m, int64_t k) {
    if (m < 0 || k <= 0 || m >= (1LL << 31) || k >= (1LL << 31)) return 0;
    return (size_t)m * (size_t)i8_blocks(k) * 32;
}

extern "C" size_t lora_mxint8_scales_size(int64_t m, int64_t k) { return lora_mxint8_codes_size(m, k) / 32; }

extern "C" lora_status lora_mxint8_quantize(const void *X, int64_t m, int64_t k, void *codes, void *scales, hipStream_t stream) {
    CHECK(check_input(m, k, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    HIPCHK(launch_mxint8_quantize(X, m, k, codes, scales, stream), "MXINT8 quantise launch");
    return LORA_OK;
}

extern "C" lora_status lora_mxint8_dequantize(const void *codes, const void *scales, int64_t m, int64_t k, void *X, hipStream_t stream) {
    CHECK(check_input(m, k, codes, scales));
    if (m == 0) return LORA_OK;
    REQ_PTR(X, 16);
    HIPCHK(launch_mxint8_dequantize(codes, scales, m, k, X, stream), "MXINT8 dequantise launch");
    return LORA_OK;
}

// The dA pass reads the codes themselves where it takes all ranks at once, up to 128; for
// higher ranks the input is expanded to bf16 first.  The fast kernels of all passes read S,
// dS and A in pieces of 8 ranks, so a rank that is no multiple of 8 gets copies of S and, for
// dX, of one adapter's A with rows as long as that takes (333 x 1032 x 776, rank 5: 69 us with the
// input expanded and the general kernels, 60 so; 436 x 1328 x 2336, rank 113: 409 and 173).
// The dX product over a bf16 weight reads the mask 128 columns at a time, so where its
// rows are no multiple of that the mask is copied too (the product of 333 x 1032 x 776, rank 8:
// 37 us, 23 so; of 2325 x 2448 x 4320, mixed, 177 and 131).  All copies are one launch's, at
// the start of the workspace, the layer's own after them.
static int32_t row_of(int32_t r) { return (r + 7) / 8 * 8; }
struct InputPlan {
    bool expand, widen, mask, packed;  // packed: dX straight from a packed weight
    size_t s_at, a_at, keep_at, bytes;
};
static InputPlan input_plan(int32_t kind, int64_t group, int64_t m, int64_t k, int64_t n, int32_t r, bool multi) {
    InputPlan p{r > 128, row_of(r) != r, false, false, 0, 0, 0, 0};
    if (m == 0) return InputPlan{};
    const int64_t kw = (k + 31) / 32;
    p.packed = kind == LORA_WEIGHT_MXFP4 ? mx_gemm_t_plan(m, k, n, row_of(r)).kind != 0
                                         : kind == LORA_WEIGHT_INT4 && int4_t_plan(m, k, n, group, row_of(r)).kind != 0;
    p.mask = kw % 4 != 0 && !p.packed;
    if (p.expand) p.bytes = align_up((size_t)m * (size_t)k * 2);
    p.s_at = p.bytes;
    if (p.widen) p.bytes += align_up((size_t)m * (size_t)row_of(r) * 4);
    p.a_at = p.bytes;
    if (p.widen && !multi) p.bytes += align_up((size_t)k * (size_t)row_of(r) * 2);
    p.keep_at = p.bytes;
    if (p.mask) p.bytes += align_up((size_t)m * (size_t)((kw + 3) / 4 * 4) * 4);
    return p;
}

// The input, S, one adapter's A and the mask as the backward is to read them.
static lora_status prepare(const InputPlan &pl, const void *x_codes, const void *x_scales, int64_t m, int64_t k, int32_t r, LayerInput &X,
                           const float *&S, AdapterSource &src, const uint32_t *keep_bits, bool want_dX, void *workspace,
                           hipStream_t stream) {
    const bool multi = src.table != nullptr;
    src.r_cap = row_of(r);
    if (pl.expand) {
        HIPCHK(launch_mxint8_dequantize(x_codes, x_scales, m, k, workspace, stream), "MXINT8 dequantise launch");
        X = LayerInput(workspace);
    }
    WidenRows w{};
    w.m = m;
    w.k = k;
    w.r = r;
    w.row = row_of(r);
    w.kw = (int)((k + 31) / 32);
    w.keep_row = (w.kw + 3) / 4 * 4;
    w.S = S;
    w.A = src.A;
    w.keep = keep_bits;
    if (pl.widen) {
        w.S_out = (float *)ws_at(workspace, pl.s_at);
        S = w.S_out;
        if (!multi && want_dX) {  // (nothing else reads A)
            w.A_out = ws_at(workspace, pl.a_at);
            src.A = w.A_out;
            src.a_r = w.row;
        }
    }
    if (pl.mask && want_dX && (multi || src.p != 0.0f)) {
        w.keep_out = (uint32_t *)ws_at(workspace, pl.keep_at);
        X.keep = w.keep_out;
        X.keep_row = w.keep_row;
    }
    if (w.S_out || w.keep_out) HIPCHK(launch_widen_rows(w, stream), "copy launch");
    return LORA_OK;
}

static bool sizes_ok(int64_t m, int64_t k, int64_t n) {
    return m >= 0 && k > 0 && n > 0 && m < (1LL << 31) && k < (1LL << 31) && n < (1LL << 31) && m * k < (1LL << 46) && k * n < (1LL << 46);
}

static bool kind_ok(int32_t kind) { return kind == LORA_WEIGHT_BF16 || kind == LORA_WEIGHT_MXFP4 || kind == LORA_WEIGHT_INT4; }

static bool group_ok(int32_t kind, int64_t group) { return kind != LORA_WEIGHT_INT4 || lora_int4_scales_size(128, 8, group) > 0; }

static lora_status check_weight(int32_t kind, const void *W, const void *W_scales, int64_t group) {
    REQUIRE(kind_ok(kind), "weight kind %d is unknown", kind);
    REQ_PTR(W, 16);
    if (kind != LORA_WEIGHT_BF16) REQ_PTR(W_scales, 16);
    REQUIRE(group_ok(kind, group), "group = %lld must be 32, 64 or a multiple of 128",
            (long long)group);
    return LORA_OK;
}

// What both backward calls read and write a row at a time.
static lora_status check_rows(int64_t m, const void *dY, const float *S, const uint32_t *keep_bits, bool keep_needed, const void *dX) {
    if (m == 0) return LORA_OK;
    REQ_PTR(dY, 16);
    REQ_PTR(S, 4);
    REQUIRE(dX == nullptr || aligned(dX, 16), "dX must be 16-byte aligned (or NULL: no input gradient)");
    REQUIRE(keep_bits != nullptr || !keep_needed, "keep_bits may be NULL only for one adapter with p == 0");
    REQUIRE(aligned(keep_bits, 4), "keep_bits must be 4-byte aligned");
    return LORA_OK;
}

extern "C" size_t lora_mxint8_linear_bwd_workspace_size(int32_t kind, int64_t group, int64_t m, int64_t k, int64_t n, int32_t r) {
    if (!sizes_ok(m, k, n) || !kind_ok(kind) || !group_ok(kind, group) || r < 1 || r > 256 || !bwd_k_ok(k)) return 0;
    const size_t layer = kind == LORA_WEIGHT_BF16    ? lora_linear_bwd_workspace_size(m, k, n, row_of(r))
                         : kind == LORA_WEIGHT_MXFP4 ? lora_mxfp4_linear_bwd_workspace_size(m, k, n, row_of(r))
                                                     : lora_int4_linear_bwd_workspace_size(m, k, n, group, row_of(r));
    return input_plan(kind, group, m, k, n, r, false).bytes + layer;
}

extern "C" size_t multi_lora_mxint8_bwd_workspace_size(int32_t kind, int64_t group, int64_t m, int64_t k, int64_t n, int32_t r_max,
                                                       int32_t num_adapters, int32_t num_segments) {
    if (!sizes_ok(m, k, n) || !kind_ok(kind) || !group_ok(kind, group) || r_max < 1 || r_max > 256 || num_adapters < 1 || num_segments < 0 || !bwd_k_ok(k)) return 0;
    const size_t layer = kind == LORA_WEIGHT_BF16    ? multi_lora_bwd_workspace_size(m, k, n, row_of(r_max), num_adapters, num_segments)
                         : kind == LORA_WEIGHT_MXFP4 ? multi_lora_mxfp4_bwd_workspace_size(m, k, n, row_of(r_max), num_adapters, num_segments)
                                                     : multi_lora_int4_bwd_workspace_size(m, k, n, group, row_of(r_max), num_adapters, num_segments);
    return input_plan(kind, group, m, k, n, r_max, true).bytes + layer;
}

// The layer's backward over a weight of any form, after the checks.
static lora_status layer_backward(bool multi, int32_t kind, const void *W, const void *W_scales, int64_t group, const void *dY,
                                  const LayerInput &X, const AdapterSource &src, const float *S, const uint32_t *keep_bits, int64_t m,
                                  int64_t k, int64_t n, void *dX, void *workspace, hipStream_t stream) {
    if (kind == LORA_WEIGHT_MXFP4)
        return multi ? multi_mxfp4_linear_backward(dY, X, W, W_scales, src, S, keep_bits, m, k, n, dX, workspace, stream)
                     : mxfp4_linear_backward(dY, X, W, W_scales, src, S, keep_bits, m, k, n, dX, workspace, stream);
    if (kind == LORA_WEIGHT_INT4)
        return multi ? multi_int4_linear_backward(dY, X, W, W_scales, group, src, S, keep_bits, m, k, n, dX, workspace, stream)
                     : int4_linear_backward(dY, X, W, W_scales, group, src, S, keep_bits, m, k, n, dX, workspace, stream);
    return multi ? multi_linear_backward(dY, X, W, src, S, keep_bits, m, k, n, dX, workspace, stream)
                 : linear_backward(dY, X, W, src, S, keep_bits, m, k, n, dX, workspace, stream);
}

extern "C" lora_status lora_mxint8_linear_bwd(const void *dY, const void *x_codes, const void *x_scales, int32_t kind, const void *W,
                                              const void *W_scales, int64_t group, const void *A, const void *B, const float *S,
                                              const uint32_t *keep_bits, int64_t m, int64_t k, int64_t n, int32_t r, float alpha, float p,
                                              void *dX, void *dA, void *dB, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(kind, W, W_scales, group));
    CHECK(check_input(m, k, x_codes, x_scales));
    CHECK(check_rank(r));
    CHECK(check_p(p));
    CHECK(check_b_size(r, k, n));
    if (dX != nullptr) CHECK(check_b_size(row_of(r), k, 0));  // (the dX product reads A's copy, whose rows are longer)
    CHECK(check_bwd_k(k));
    REQ_PTR(A, 2);
    REQ_PTR(B, 2);
    REQ_PTR(dA, 2);
    REQ_PTR(dB, 2);
    CHECK(check_rows(m, dY, S, keep_bits, p != 0.0f, dX));
    const size_t need = lora_mxint8_linear_bwd_workspace_size(kind, group, m, k, n, r);
    if (workspace_bytes < need) return host_fail(LORA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need > 0) REQ_PTR(workspace, 16);
    LayerInput X(x_codes, x_scales);
    AdapterSource src = single_source(A, B, dA, dB, r, alpha, p);
    const InputPlan pl = input_plan(kind, group, m, k, n, r, false);
    if (dX != nullptr && !pl.packed) CHECK(check_dx_tiles(m, k, n));
    CHECK(prepare(pl, x_codes, x_scales, m, k, r, X, S, src, keep_bits, dX != nullptr, workspace, stream));
    return layer_backward(false, kind, W, W_scales, group, dY, X, src, S, keep_bits, m, k, n, dX, ws_at(workspace, pl.bytes), stream);
}

extern "C" lora_status multi_lora_mxint8_linear_bwd(const void *dY, const void *x_codes, const void *x_scales, int32_t kind, const void *W,
                                                    const void *W_scales, int64_t group, const lora_adapter *adapters,
                                                    int32_t num_adapters, const int64_t *seg_off, const int32_t *seg_adapter,
                                                    int32_t num_segments, const float *S, const uint32_t *keep_bits, int64_t m, int64_t k,
                                                    int64_t n, int32_t r_max, void *dX, void *workspace, size_t workspace_bytes,
                                                    hipStream_t stream) {
    CHECK(check_shape(m, k, n));
    CHECK(check_weight(kind, W, W_scales, group));
    CHECK(check_input(m, k, x_codes, x_scales));
    // (the forward on no rows makes the checks of the adapter and segment tables, and enqueues nothing)
    CHECK(multi_lora_linear_fwd(nullptr, W, adapters, num_adapters, seg_off, seg_adapter, num_segments, 0, k, n, r_max, 0, 0, nullptr,
                                nullptr, nullptr, nullptr, 0, stream));
    CHECK(check_bwd_k(k));
    CHECK(check_rows(m, dY, S, keep_bits, true, dX));
    const size_t need = multi_lora_mxint8_bwd_workspace_size(kind, group, m, k, n, r_max, num_adapters, num_segments);
    if (workspace_bytes < need) return host_fail(LORA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (need > 0) REQ_PTR(workspace, 16);
    LayerInput X(x_codes, x_scales);
    AdapterSource src = multi_source(adapters, num_adapters, seg_off, seg_adapter, num_segments, r_max);
    const InputPlan pl = input_plan(kind, group, m, k, n, r_max, true);
    if (dX != nullptr && !pl.packed) CHECK(check_dx_tiles(m, k, n));
    CHECK(prepare(pl, x_codes, x_scales, m, k, r_max, X, S, src, keep_bits, dX != nullptr, workspace, stream));
    return layer_backward(true, kind, W, W_scales, group, dY, X, src, S, keep_bits, m, k, n, dX, ws_at(workspace, pl.bytes), stream);
}
