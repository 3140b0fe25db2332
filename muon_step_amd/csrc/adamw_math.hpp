// Device arithmetic the AdamW kernels share.
#pragma once

#include "common.hpp"

namespace muon {

// Correctly rounded fp32 square root.  The hardware estimate v_sqrt_f32
// (within 1 ulp) is corrected by the signs of the exact FMA residuals
// x - s*pred(s) and x - s*succ(s): the true root lies below the midpoint
// (s + pred(s))/2 iff x <= s*pred(s), because no float x falls strictly between
// s*pred(s) and the square of that midpoint (Markstein's FMA-based square-root
// rounding; Muller et al., Handbook of Floating-Point Arithmetic, square-root
// chapter).  Inputs below 2^-96 are scaled by 2^32 so the residuals cannot
// underflow; zeros, infinities, NaN and negative inputs take the hardware result.
__device__ __forceinline__ float sqrt_rn(float x) {
    if (!(x > 0.0f) || x == __builtin_inff()) return __builtin_amdgcn_sqrtf(x);
    const bool tiny = x < 0x1p-96f;
    const float xs = tiny ? x * 0x1p32f : x;
    float s = __builtin_amdgcn_sqrtf(xs);
    for (int i = 0; i < 2; ++i) {
        const float dn = __uint_as_float(__float_as_uint(s) - 1u);
        const float up = __uint_as_float(__float_as_uint(s) + 1u);
        const float r_dn = __builtin_fmaf(-dn, s, xs);
        const float r_up = __builtin_fmaf(-up, s, xs);
        if (r_dn <= 0.0f) s = dn;
        else if (r_up > 0.0f) s = up;
    }
    return tiny ? s * 0x1p-16f : s;
}

}  // namespace muon
