// mx_epilogue.h -- gfx950 device code of the fused GEMM epilogue: what a
// product's FP32 sums become on their way to C,
//   C = residual + act(A * B^T + bias),
// in FP32, rounded once to the output type.  The sums are still in registers
// or LDS when it runs, so it costs the bytes of bias and residual and no
// pass over C of its own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_decode.h"
#include "mx_kernels.h"
#include "mx_math.h"

namespace mx {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };   // MX_ACT_*

struct Epilogue {
    static constexpr bool fused = true;
    const void *bias;            // N values, null: none
    const void *residual;        // rows of the output's type, pitch ldr, null: none
    int64_t ldr;
    int bias_bf16, act;
};

// erf(x) by the compiler's own FP32 function (a few units in the last place).
__device__ __forceinline__ float act_apply(float v, int act)
{
    switch (act) {
    case ACT_RELU: return v > 0.f ? v : v != v ? v : 0.f;
    case ACT_SILU: return v * sigmoid(v);
    case ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.707106781f));
    // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (v + 0.044715 v^3)
    case ACT_GELU_TANH: return v * sigmoid(1.59576912f * v * fmaf(0.044715f * v, v, 1.f));
    default: return v;
    }
}

// Bias of column n (n < N).
template <typename EP>
__device__ __forceinline__ float bias_at(const EP &ep, int n)
{
    if (!ep.bias) return 0.f;
    return ep.bias_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)ep.bias)[n] << 16)
                        : ((const float *)ep.bias)[n];
}

// Residual at (m, n).
template <int OUT>
__device__ __forceinline__ float residual_at(const Epilogue &ep, int64_t m, int n)
{
    if (!ep.residual) return 0.f;
    const int64_t at = m * ep.ldr + n;
    return OUT == OF32 ? ((const float *)ep.residual)[at]
                       : __uint_as_float((uint32_t)((const uint16_t *)ep.residual)[at] << 16);
}

// C at (m, n) from its sum v.
template <int OUT, typename EP>
__device__ __forceinline__ float epilogue_at(const EP &ep, float v, int64_t m, int n)
{
    return act_apply(v + bias_at(ep, n), ep.act) + residual_at<OUT>(ep, m, n);
}

// The tile kernel's epilogue of one 32-row band of a wave's sub-tile: sums
// (bias added) in the wave's LDS at `stage`, WTN columns, row pitch PITCH
// bytes.  First the activation, in place and in a loop that is not unrolled
// (one copy of its code); then all residual loads of the band together, so
// that their latency is paid once, and the 16-byte stores.  The thread that
// stores an element of C is the one that has read its residual, so C may be
// the residual itself.
template <int OUT, int WTN, int PITCH, typename EP>
__device__ __forceinline__ void fused_band(const EP &ep, uint8_t *stage, void *C, int row0,
                                           int col0, int M, int N, int lane)
{
    constexpr int OS = OUT == OF32 ? 4 : 2, VE = 16 / OS;
    constexpr int CPR = WTN / VE, NIT = (32 * CPR + 63) / 64;   // chunks per row, per lane
    if (ep.act != ACT_NONE) {
        constexpr int QPR = WTN / 4;                            // float4 per row
#pragma unroll 1
        for (int t = lane; t < 32 * QPR; t += 64) {
            v4f *p = (v4f *)(stage + (t / QPR) * PITCH + (t % QPR) * 16);
            v4f v = *p;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = act_apply(v[q], ep.act);
            *p = v;
        }
    }
    const bool vec_c = ((int64_t)N * OS) % 16 == 0, vec_r = (ep.ldr * OS) % 16 == 0;
    typedef typename std::conditional<OUT == OF32, float, uint16_t>::type otype;
    v4i res[NIT];
    if (ep.residual) {
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int t = it * 64 + lane;
            const int row = row0 + t / CPR, col = col0 + t % CPR * VE;
            res[it] = v4i{0, 0, 0, 0};
            if (t >= 32 * CPR || row >= M || col >= N) continue;
            const otype *p = (const otype *)ep.residual + row * ep.ldr + col;
            if (vec_r && col + VE <= N) {
                res[it] = *(const v4i *)p;
            } else {
#pragma unroll
                for (int q = 0; q < VE; ++q) {
                    if (col + q >= N) break;
                    if constexpr (OUT == OF32) res[it][q] = __float_as_int(p[q]);
                    else res[it][q / 2] |= (int)((uint32_t)p[q] << (16 * (q & 1)));
                }
            }
        }
    }
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
        const int t = it * 64 + lane;
        const int r = t / CPR, ch = t % CPR;
        const int row = row0 + r, col = col0 + ch * VE;
        if (t >= 32 * CPR || row >= M || col >= N) continue;
        const float *src = (const float *)(stage + r * PITCH) + ch * VE;
        float v[VE];
#pragma unroll
        for (int q = 0; q < VE; q += 4) *(v4f *)(v + q) = *(const v4f *)(src + q);
        if (ep.residual) {
#pragma unroll
            for (int q = 0; q < VE; ++q)
                v[q] += OUT == OF32 ? __int_as_float(res[it][q])
                                    : __uint_as_float((q & 1) ? (uint32_t)res[it][q / 2] & 0xffff0000u
                                                              : (uint32_t)res[it][q / 2] << 16);
        }
        v4i w;
        if constexpr (OUT == OF32) {
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = __float_as_int(v[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = (int)bf16_pair(v[2 * q], v[2 * q + 1]);
        }
        otype *dst = (otype *)C + (int64_t)row * N + col;
        if (vec_c) {                                            // N % VE == 0: whole chunks
            *(v4i *)dst = w;
        } else {
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                if (col + q >= N) break;
                if constexpr (OUT == OF32) dst[q] = v[q];
                else dst[q] = (uint16_t)((uint32_t)w[q / 2] >> (16 * (q & 1)));
            }
        }
    }
}

// splitk_reduce with the epilogue: C[i] from the sum over slices, in slice
// order, of W[s * plane + i]; n_cols is C's row length.  mn < 2^31.
template <int OUT>
__global__ void __launch_bounds__(256)
splitk_fused(const float *__restrict__ W, void *C, int mn, int n_cols, int64_t plane, int slices,
             Epilogue ep)
{
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= mn) return;
    v4f acc = *(const v4f *)(W + i);
    for (int s = 1; s < slices; ++s) acc += *(const v4f *)(W + s * plane + i);
    const int n = min(4, mn - i);
    int m = (int)((uint32_t)i / (uint32_t)n_cols), c = i - m * n_cols;
    for (int q = 0; q < n; ++q) {
        const float v = epilogue_at<OUT>(ep, acc[q], m, c);
        if (OUT == OF32) ((float *)C)[i + q] = v;
        else ((uint16_t *)C)[i + q] = f32_to_bf16(v);
        if (++c == n_cols) { c = 0; ++m; }
    }
}

// The decode kernel with the epilogue.
template <int FA, int FB, int OUT, int WA>
__global__ void __launch_bounds__(kDecodeWaves * 64)
fused_decode(const uint8_t *__restrict__ A, const uint8_t *__restrict__ As,
             const uint8_t *__restrict__ B, const uint8_t *__restrict__ Bs, void *C, int M, int N,
             int K, Epilogue ep)
{
    decode_body<FA, FB, OUT, WA>(A, As, B, Bs, C, M, N, K, ep);
}

}  // namespace mx
