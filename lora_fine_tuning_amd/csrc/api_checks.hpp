// Argument checks and workspace carving shared by the C-ABI translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "host_status.hpp"
#include "lora_fused.h"

namespace lora {

inline lora_status hip_fail(hipError_t e, const char *what) {
    return host_fail(LORA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

#define REQUIRE(cond, ...)                                        \
    do {                                                          \
        if (!(cond)) return host_fail(LORA_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

inline lora_status check_shape(int64_t m, int64_t k, int64_t n) {
    REQUIRE(m >= 0 && m < (1LL << 31), "m = %lld out of range [0, 2^31)", (long long)m);
    REQUIRE(k > 0 && k < (1LL << 31), "k = %lld out of range (0, 2^31)", (long long)k);
    REQUIRE(n > 0 && n < (1LL << 31), "n = %lld out of range (0, 2^31)", (long long)n);
    REQUIRE(k % 8 == 0, "k = %lld must be a multiple of 8", (long long)k);
    REQUIRE(n % 8 == 0, "n = %lld must be a multiple of 8", (long long)n);
    REQUIRE(m * k < (1LL << 46) && m * n < (1LL << 46), "tensor too large");
    return LORA_OK;
}

inline lora_status check_rank(int32_t r) {
    REQUIRE(r >= 1 && r <= 256, "rank r = %d must be in [1, 256]", r);
    return LORA_OK;
}

// The GEMM epilogues and the dS/dB kernel address B (r x n bf16) and A
// (k x r bf16) with 32-bit byte offsets.
inline lora_status check_b_size(int32_t r, int64_t k, int64_t n) {
    if ((int64_t)r * n * 2 >= (1LL << 31))
        return host_fail(LORA_ERR_UNSUPPORTED, "B of %d x %lld bf16 exceeds 2 GiB", r, (long long)n);
    if ((int64_t)r * k * 2 >= (1LL << 31))
        return host_fail(LORA_ERR_UNSUPPORTED, "A of %lld x %d bf16 exceeds 2 GiB", (long long)k, r);
    return LORA_OK;
}

// The backward's dA kernels take runs of 32 rows of X or more, whose bytes they address
// with 32 bits.
inline bool bwd_k_ok(int64_t k) { return k * 64 < (1LL << 31); }
inline lora_status check_bwd_k(int64_t k) {
    if (!bwd_k_ok(k)) return host_fail(LORA_ERR_UNSUPPORTED, "32 rows of X of k = %lld exceed 2 GiB", (long long)k);
    return LORA_OK;
}

// The bf16 GEMM's tiles address their rows with 32-bit byte offsets: 256 of the row side
// and of the output, and of W 64 (forward) or 256 (dX).
inline bool tile_ok(int64_t rows, int64_t tile, int64_t len) { return (rows < tile ? rows : tile) * len * 2 < (1LL << 31); }
inline lora_status check_fwd_tiles(int64_t m, int64_t k, int64_t n) {
    if (m > 0 && !(tile_ok(m, 256, k) && tile_ok(m, 256, n) && tile_ok(k, 64, n)))
        return host_fail(LORA_ERR_UNSUPPORTED, "256 rows of X or Y or 64 of W exceed 2 GiB (m = %lld, k = %lld, n = %lld)",
                         (long long)m, (long long)k, (long long)n);
    return LORA_OK;
}
inline lora_status check_dx_tiles(int64_t m, int64_t k, int64_t n) {
    if (m > 0 && !(tile_ok(m, 256, n) && tile_ok(m, 256, k) && tile_ok(k, 256, n)))
        return host_fail(LORA_ERR_UNSUPPORTED, "256 rows of dY, dX or W exceed 2 GiB (m = %lld, k = %lld, n = %lld)",
                         (long long)m, (long long)k, (long long)n);
    return LORA_OK;
}

inline lora_status check_p(float p) {
    REQUIRE(p >= 0.0f && p < 1.0f, "dropout p = %g must be in [0, 1)", (double)p);
    return LORA_OK;
}

#define CHECK(x)                          \
    do {                                  \
        lora_status _st = (x);            \
        if (_st != LORA_OK) return _st;   \
    } while (0)

#define REQ_PTR(p, align) \
    REQUIRE((p) != nullptr && aligned((p), (align)), #p " must be non-NULL and %d-byte aligned", (int)(align))

#define HIPCHK(call, what)                         \
    do {                                           \
        hipError_t _e = (call);                    \
        if (_e != hipSuccess) return hip_fail(_e, what); \
    } while (0)

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

struct Carve {
    size_t off = 0;
    size_t take(size_t bytes) {
        size_t o = off;
        off = align_up(off + bytes);
        return o;
    }
};
inline char *ws_at(void *ws, size_t off) { return (char *)ws + off; }

}  // namespace lora
