// mx_math.h -- gfx950 device arithmetic and ordering shared by the row
// operators, the expert routing and the fused GEMM epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Orders the wave's LDS accesses before this point against those after it,
// across its lanes (the hardware keeps them in order; this keeps the compiler
// to it).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Two BF16 values in one dword (low half: a), rounded to nearest even: one
// v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}

// 1 / (1 + exp(-x)).  exp(-x) = 2^(-x log2 e): the product's rounding error
// and the low part of log2 e are carried in `lo`, so that the error does not
// grow with |x|; the hardware's exp2 and reciprocal are good to one unit in
// the last place.  Arguments beyond -128 and 64 are taken as those (an
// infinity would leave inf - inf in the low part): the results there are 0 and
// 1, as from -87.3 on, where exp(-x) passes 2^126 and its reciprocal is
// flushed.  A NaN argument may give a number: the callers multiply by the
// argument itself.
__device__ __forceinline__ float sigmoid(float x)
{
    constexpr float L = -1.44269502162933349609f, L_LO = -1.925963e-8f;   // L + L_LO = -log2 e
    constexpr float LN2 = 0.693147180559945f;
    const float c = __builtin_amdgcn_fmed3f(x, -128.f, 64.f);
    const float hi = c * L, lo = fmaf(c, L_LO, fmaf(c, L, -hi));
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(hi), fmaf(lo, LN2, 1.f), 1.f));
}

}  // namespace mx
