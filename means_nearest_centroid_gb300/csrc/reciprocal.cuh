// reciprocal.cuh -- 1 / y for routing's scores.
#pragma once

#include <cmath>

namespace kma {

// 1 / y correctly rounded for 1 <= y <= 2^125: one Newton step with fused
// multiply-adds from the hardware's approximation, which is within one ulp
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  It has the quotient's bits for all 2^23 significands
// (tests/reciprocal_check.cu compares them); a power of two only scales both.
__device__ __forceinline__ float reciprocal(float y)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return fmaf(r, fmaf(-y, r, 1.0f), r);
}

}  // namespace kma
