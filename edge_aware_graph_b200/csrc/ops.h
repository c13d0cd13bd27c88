// What the operators around the block share (ops_*.cu).
#pragma once
#include <cmath>
#include "common.cuh"
#include "fast_common.cuh"

namespace eaga {
namespace ops {

using fast::sm_count;
using fast::launch_pdl;

// First in the operators' kernels (all are launched with launch_pdl): nothing is read or written before the previous launch is
// done.  The next launch may become resident before this one is done, so that small kernels follow one another 1 to 2 us sooner:
// at once behind a few CTAs; behind more only when they are nearly done (before_next), since CTAs that are placed while these
// compute land unevenly on the SMs (an fp32 product of 160 CTAs took 43 us behind another instead of 16).
__device__ __forceinline__ void after_previous() {
    if (gridDim.x * gridDim.y <= 32) sm100::griddep_launch_dependents();
    sm100::griddep_wait();
}
__device__ __forceinline__ void before_next() { sm100::griddep_launch_dependents(); }

inline bool bad_align16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace ops
}  // namespace eaga
