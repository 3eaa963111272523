// mx_math.h -- gfx950 device arithmetic shared by the row operators and the
// fused GEMM epilogue.
#pragma once

#include <hip/hip_runtime.h>

namespace mx {

// 1 / (1 + exp(-x)).  exp(-x) = 2^(-x log2 e), the product in two parts so
// that its rounding does not grow with |x|; the hardware's exp2 and
// reciprocal are good to one unit in the last place.  Arguments above 64
// give 1 like 64 itself (an infinity would leave inf - inf in the low part);
// below -87 the result, under 2^-125, counts as 0.  A NaN argument may give
// a number: the callers multiply by the argument itself.
__device__ __forceinline__ float sigmoid(float x)
{
    constexpr float L = -1.44269502162933349609f, L_LO = -1.925963e-8f;   // L + L_LO = -log2 e
    constexpr float LN2 = 0.693147180559945f;
    const float c = __builtin_amdgcn_fmed3f(x, -88.f, 64.f);
    const float hi = c * L, lo = fmaf(c, L_LO, fmaf(c, L, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    const float sig = __builtin_amdgcn_rcpf(1.f + fmaf(e, lo * LN2, e));
    return x < -87.f ? 0.f : sig;
}

}  // namespace mx
