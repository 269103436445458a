// Shapes of weights held as 4-bit integers (int4_kernels.hip describes the storage).
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"

namespace lora {

struct I4Shape {
    int64_t k, n;
    int64_t k128, n16;      // blocks of 128 rows, groups of 16 columns
    int64_t group, groups;  // rows that share a scale; scales of a column
};

inline I4Shape i4_shape(int64_t k, int64_t n, int64_t group) {
    const int64_t k128 = (k + 127) / 128;
    return I4Shape{k, n, k128, (n + 15) / 16, group, group < 128 ? k128 * 128 / group : (k + group - 1) / group};
}

}  // namespace lora
