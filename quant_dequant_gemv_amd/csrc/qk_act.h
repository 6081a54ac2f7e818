// qk_act.h -- the logistic function in fp32, for kernels that run it once an
// element.
#pragma once

#include <hip/hip_runtime.h>

namespace qk {

// 1 / (1 + e^-z) within 6 x 2^-24 of itself (below 2^-126 of 1: as 2^-126).
// e^-z is 2^t (1 + d ln 2) with t + d = -z log2(e) in two fp32 parts; the
// reciprocal is refined once.  Eleven instructions, two of them quarter rate:
// expf and a rounded division are 25.
__device__ __forceinline__ float logistic(float z) {
    const float c = fminf(fmaxf(z, -87.f), 87.f);
    const float t = c * -0x1.715476p+0f;
    const float d = fmaf(c, -0x1.715476p+0f, -t) + c * -0x1.4ae0cp-26f;  // (log2 e less its fp32 value)
    float e = __builtin_amdgcn_exp2f(t);
    e = 1.f + fmaf(e, d * 0x1.62e43p-1f, e);
    const float r = __builtin_amdgcn_rcpf(e);
    return z != z ? z : fmaf(fmaf(-e, r, 1.f), r, r);
}
// z below -87 as -87: what a gate of -inf or of the lowest value leaves is 0 to 2^-119.
__device__ __forceinline__ float silu(float z) { return fmaxf(z, -87.f) * logistic(z); }

}  // namespace qk
