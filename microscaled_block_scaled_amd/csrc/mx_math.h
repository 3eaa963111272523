// mx_math.h -- gfx950 device arithmetic shared by the row operators and the
// fused GEMM epilogue.
#pragma once

#include <hip/hip_runtime.h>

namespace mx {

// 1 / (1 + exp(-x)).  exp(-x) = 2^(-x log2 e): the product's rounding error
// and the low part of log2 e are carried in `lo`, so that the error does not
// grow with |x|; the hardware's exp2 and reciprocal are good to one unit in
// the last place.  Arguments above 64 give 1 like 64 itself (an infinity
// would leave inf - inf in the low part); below -87.3 exp(-x) passes 2^126 and
// the result counts as 0.  A NaN argument may give a number: the callers
// multiply by the argument itself.
__device__ __forceinline__ float sigmoid(float x)
{
    constexpr float L = -1.44269502162933349609f, L_LO = -1.925963e-8f;   // L + L_LO = -log2 e
    constexpr float LN2 = 0.693147180559945f;
    const float c = fminf(x, 64.f);
    const float hi = c * L, lo = fmaf(c, L_LO, fmaf(c, L, -hi));
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(hi), fmaf(lo, LN2, 1.f), 1.f));
}

}  // namespace mx
