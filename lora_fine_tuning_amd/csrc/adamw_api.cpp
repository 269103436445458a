// C-ABI entry point of the optimizer step.
#include <hip/hip_runtime.h>

#include <cmath>

#include "adamw.hpp"
#include "api_checks.hpp"

using namespace lora;

extern "C" lora_status lora_adamw_step(const lora_adamw_tensor *tensors, int32_t count, int32_t param_bf16,
                                       int32_t grad_bf16, int32_t state_bits, double lr, double beta1,
                                       double beta2, double eps, double weight_decay, int64_t step,
                                       const int64_t *step_dev, uint64_t seed, hipStream_t stream) {
    REQUIRE(count >= 0, "count = %d must be >= 0", count);
    REQUIRE(count == 0 || tensors != nullptr, "tensors must be a non-NULL host array");
    REQUIRE(param_bf16 == 0 || param_bf16 == 1, "param_bf16 = %d must be 0 or 1", param_bf16);
    REQUIRE(grad_bf16 == 0 || grad_bf16 == 1, "grad_bf16 = %d must be 0 or 1", grad_bf16);
    REQUIRE(state_bits == 8 || state_bits == 32, "state_bits = %d must be 8 or 32", state_bits);
    REQUIRE(std::isfinite(lr) && std::isfinite(weight_decay), "lr = %g and weight_decay = %g must be finite",
            lr, weight_decay);
    REQUIRE(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1, "betas (%g, %g) must be in [0, 1)", beta1, beta2);
    REQUIRE(eps >= 0 && std::isfinite(eps), "eps = %g must be finite and >= 0", eps);
    // (the reciprocal takes a subnormal for zero: 0 / eps would be NaN where v is zero)
    REQUIRE(eps == 0 || eps >= 0x1p-126, "eps = %g must be 0 or at least 2^-126", eps);
    REQUIRE(step_dev != nullptr || step >= 1, "step = %lld must be >= 1", (long long)step);
    REQUIRE(aligned(step_dev, 8), "step_dev must be 8-byte aligned");
    bool master = false;
    for (int32_t i = 0, seen = 0; i < count; ++i) {
        const lora_adamw_tensor &t = tensors[i];
        REQUIRE(t.n >= 0 && t.n <= kAdamwMaxValues, "tensor %d: n = %lld out of range", i, (long long)t.n);
        if (t.n == 0) continue;
        const size_t pa = param_bf16 ? 2 : 4, ga = grad_bf16 ? 2 : 4, ma = state_bits == 8 ? 1 : 4;
        REQUIRE(t.param != nullptr && aligned(t.param, pa), "tensor %d: param must be non-NULL and aligned", i);
        REQUIRE(t.grad != nullptr && aligned(t.grad, ga), "tensor %d: grad must be non-NULL and aligned", i);
        REQUIRE(t.m != nullptr && aligned(t.m, ma) && t.v != nullptr && aligned(t.v, ma),
                "tensor %d: m and v must be non-NULL and aligned", i);
        if (state_bits == 8)
            REQUIRE(t.m_scale != nullptr && aligned(t.m_scale, 4) && t.v_scale != nullptr && aligned(t.v_scale, 4),
                    "tensor %d: 8-bit moments need m_scale and v_scale", i);
        REQUIRE(aligned(t.master, 4), "tensor %d: master must be 4-byte aligned", i);
        REQUIRE(t.offset % 8 == 0, "tensor %d: offset = %llu must be a multiple of 8", i,
                (unsigned long long)t.offset);
        const bool has = t.master != nullptr;
        REQUIRE(!has || param_bf16 == 1, "tensor %d: a master copy goes with a bf16 param", i);
        REQUIRE(seen == 0 || has == master, "tensor %d: either every tensor has a master copy or none", i);
        master = has;
        seen = 1;
    }
    AdamwPlan pl{};
    pl.bits = state_bits;
    pl.master = master;
    pl.param_bf16 = param_bf16 == 1;
    pl.grad_bf16 = grad_bf16 == 1;
    pl.lr = lr;
    pl.beta1 = beta1;
    pl.beta2 = beta2;
    pl.eps = eps;
    pl.weight_decay = weight_decay;
    pl.ln_b1 = std::log(beta1);
    pl.ln_b2 = std::log(beta2);
    if (step_dev == nullptr) {
        pl.rc1 = 1.0 / -std::expm1((double)step * pl.ln_b1);
        pl.rc2 = 1.0 / -std::expm1((double)step * pl.ln_b2);
    }
    pl.step_dev = step_dev;
    pl.step = step;
    pl.seed = seed;
    HIPCHK(launch_adamw(tensors, count, pl, stream), "AdamW launch");
    return LORA_OK;
}
