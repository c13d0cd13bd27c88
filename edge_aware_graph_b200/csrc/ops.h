// What the operators around the block share (ops_*.cu).
#pragma once
#include <cmath>
#include "common.cuh"
#include "fast_common.cuh"

namespace eaga {
namespace ops {

using fast::sm_count;

inline bool bad_align16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace ops
}  // namespace eaga
