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
// compute land unevenly on the SMs (an fp32 product of 160 CTAs took 43 us behind another instead of 16).  The first thread of a CTA
// that gets there signals for the CTA: in k_lin_tc without column sums that is a warp without work, at the start.
__device__ __forceinline__ void after_previous() {
    if (gridDim.x * gridDim.y <= 32) sm100::griddep_launch_dependents();
    sm100::griddep_wait();
}
__device__ __forceinline__ void before_next() { sm100::griddep_launch_dependents(); }

// ------------------------------------------------------------------ two fp32 values at once
// The elementwise kernels are bound by the instructions they issue as much as by
// memory; sm_100a adds, multiplies and fuses two fp32 values (each rounded as
// alone) in one instruction.
struct f2 {
    unsigned long long b;
};
__device__ __forceinline__ f2 pair(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float lo(f2 a) { return __uint_as_float((unsigned)a.b); }
__device__ __forceinline__ float hi(f2 a) { return __uint_as_float((unsigned)(a.b >> 32)); }
__device__ __forceinline__ f2 operator+(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}
__device__ __forceinline__ float across(f2 a) { return lo(a) + hi(a); }

inline bool bad_align16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace ops
}  // namespace eaga
