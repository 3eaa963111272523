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

// -log2 e in two parts.  exp(-x) is 2^(hi + lo): the product with the first
// part, and in `lo` its rounding error and the second, so that no digits are
// lost as |x| grows.
constexpr float kMinusLog2e = -1.44269502162933349609f, kMinusLog2eLow = -1.925963e-8f;
constexpr float kLn2 = 0.693147180559945f;

// 1 / (1 + exp(-x)); the hardware's exp2 and reciprocal are good to one unit in
// the last place.  Arguments beyond -128 and 64 are taken as those (an infinity
// would leave inf - inf in the low part).  Below -87.3 the reciprocal is
// subnormal, which the hardware flushes to 0: sigmoid_tail is for there.  A NaN
// argument may give a number: the callers multiply by the argument itself.
__device__ __forceinline__ float sigmoid(float x)
{
    const float c = __builtin_amdgcn_fmed3f(x, -128.f, 64.f);
    const float hi = c * kMinusLog2e;
    const float lo = fmaf(c, kMinusLog2eLow, fmaf(c, kMinusLog2e, -hi));
    return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(hi), fmaf(lo, kLn2, 1.f), 1.f));
}

// The sigmoid below kSigmoidTail, where it is exp(x) and leaves FP32's normal
// range at -87.3 while a product with it may not (gate -88, up 3e30: -1.6e-6):
// its value times 2^126, for the caller to multiply by kTailScale last, or
// into another factor.  It is 0 below 2^-252 (x < -174.6).
constexpr float kSigmoidTail = -87.f, kTailScale = 0x1p-126f;
__device__ __forceinline__ float sigmoid_tail(float x)
{
#pragma clang fp contract(off)                   // hi + 126 is of the rounded hi, and exact
    const float c = fmaxf(x, -256.f);
    const float hi = c * -kMinusLog2e;
    const float lo = fmaf(c, -kMinusLog2eLow, fmaf(c, -kMinusLog2e, -hi));
    return __builtin_amdgcn_exp2f(hi + 126.f) * fmaf(lo, kLn2, 1.f);
}

// Whether any of N values in any lane of the wave is below a negative bound:
// one integer maximum a value, since the patterns of negative values order by
// magnitude (a NaN with its sign set counts too).  For a whole wave, and not
// expected, so that the code it leads to is laid out of the way.
template <int N>
__device__ __forceinline__ bool any_below(const float (&v)[N], float bound)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]));
    return __builtin_expect(__ballot(m > __float_as_uint(bound)) != 0, 0);
}

}  // namespace mx
