// Between the AdamW entry point (adamw_api.cpp) and its kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_fused.h"

namespace lora {

struct AdamwPlan {
    int bits;  // of the moments: 8 or 32
    bool master, param_bf16, grad_bf16;
    double lr, beta1, beta2, eps, weight_decay;
    double rc1, rc2;      // 1 / (1 - beta^step)
    double ln_b1, ln_b2;  // for a step read on the device
    const int64_t *step_dev;
    int64_t step;
    uint64_t seed;
};

// Work-groups of one launch (2^24 x 256 threads is the limit of a grid), and
// the values of the largest tensor.
constexpr int64_t kAdamwMaxChunks = (1 << 24) - 1;
constexpr int64_t kAdamwMaxValues = kAdamwMaxChunks * 2048;

hipError_t launch_adamw(const lora_adamw_tensor *tensors, int32_t count, const AdamwPlan &pl, hipStream_t stream);

}  // namespace lora
