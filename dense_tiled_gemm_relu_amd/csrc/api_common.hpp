// Host helpers shared by the C-ABI units.
#pragma once

#include <cstdint>

namespace gemm_relu_hip {

constexpr int kMaxDevices = 64;
constexpr int kNumCUs = 256;   // MI355X: 8 XCDs x 32 CUs
// The tiles count K in 32 bits and round it up to a step, of at most 128 elements.
constexpr int64_t kMaxK = INT32_MAX - 127;

// GEMM_RELU_OK where the current device is a gfx950 (cached per device).
int check_device();

inline bool overlaps(uintptr_t a, uint64_t na, uintptr_t b, uint64_t nb)
{
    if (na == 0 || nb == 0) return false;
    return a < b + nb && b < a + na;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace gemm_relu_hip
