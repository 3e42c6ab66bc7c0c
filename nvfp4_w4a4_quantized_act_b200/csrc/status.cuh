// status.cuh -- bits of the per-device status word that kernels latch
// (atomicOr) and nvfp4_get_status() reads and clears.
#pragma once

#include <cstdint>

namespace nvfp4 {

constexpr uint32_t kStatusTimeout = 1u;    // a bounded wait ran out
constexpr uint32_t kStatusNonFinite = 2u;  // an input held Inf or NaN, or a scale was not positive and finite
constexpr uint32_t kStatusBadIndex = 4u;   // a length, offset or page index was out of range

}  // namespace nvfp4
