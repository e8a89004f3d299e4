// Correctly rounded square roots and quotients, two at a time, from the
// special-function unit's approximations.  The steps are Markstein's: correct
// an estimate by its remainder, which a fused multiply-add gives exactly.
// tests/native/rounding_check.cu compares them with the device's own rounded
// functions, square roots and reciprocals over every mantissa.
#pragma once

#include "rr_step.h"

namespace rr {

__device__ __forceinline__ float rsqrt_fast(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sqrt(v) rounded to nearest for v in [2^-100, 2^100]; nv = -v.  s = v * y with
// y ~ 1 / sqrt(v); s - (s^2 - v) * y / 2.
__device__ __forceinline__ float2 root2(float2 v, float2 nv)
{
    const float2 y = make_float2(rsqrt_fast(v.x), rsqrt_fast(v.y));
    const float2 s = mul2(v, y);
    return fma2(fma2(s, s, nv), mul2(y, both(-0.5f)), s);
}

// m / d rounded to nearest for d in [2^-100, 2^100] and m = 0 or |m| in [2^-100,
// 2^100] with a normal quotient below 2^127; nd = -d.  Nothing else is sound: the
// remainder of a smaller m underflows and leaves the quotient off by a unit in
// its last place, a smaller quotient is rounded twice, a larger one is NaN.
// y = 1 / d refined once, q = m * y, q + (m - d * q) * y.
__device__ __forceinline__ float2 quotient2(float2 m, float2 nd)
{
    float2 y = make_float2(rcp_fast(-nd.x), rcp_fast(-nd.y));
    y = fma2(y, fma2(nd, y, both(1.0f)), y);
    const float2 q = mul2(m, y);
    return fma2(fma2(nd, q, m), y, q);
}

}  // namespace rr
