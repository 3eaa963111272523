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
    static constexpr bool fused = true, stream_b = false;
    const void *bias;            // N values, null: none
    const void *residual;        // rows of the output's type, pitch ldr, null: none
    int64_t ldr;
    int bias_bf16, act;
};

// The standard normal distribution's upper tail for a >= 0: exp(-a^2 / 2)
// times a polynomial in t = 1 / (1 + 0.29 a) (the form Hastings used for the
// error integral), fitted to exp(a^2 / 2) times the tail on [0, 5.5] by
// iteratively reweighted least squares: relative error 1.1e-8 in exact
// arithmetic, absolute error 1.5e-7 in FP32.  One branch-free path, a third of
// the instructions of a general erf.
__device__ __forceinline__ float normal_tail(float a)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(0.29f, a, 1.f));
    float s = 0.039472931656970515f;
    s = fmaf(s, t, -0.19295293815400552f);
    s = fmaf(s, t, 0.3049042611311115f);
    s = fmaf(s, t, -0.1477244668201993f);
    s = fmaf(s, t, 0.18146478893171267f);
    s = fmaf(s, t, 0.07963898545118427f);
    s = fmaf(s, t, 0.11977550288692076f);
    s = fmaf(s, t, 0.11542094019023019f);
    return s * t * __builtin_amdgcn_exp2f(a * a * -0.721347520f);      // -log2(e) / 2
}

__device__ __forceinline__ float act_apply(float v, int act)
{
    switch (act) {
    case ACT_RELU: return v > 0.f ? v : v != v ? v : 0.f;
    case ACT_SILU: return v * sigmoid(v);
    case ACT_GELU: {
        const float q = normal_tail(fabsf(v));
        return v * (v > 0.f ? 1.f - q : q);
    }
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

// U consecutive values of C's type at p (p aligned to them).
template <int OUT, int U>
__device__ __forceinline__ void read_c(const void *p, float (&v)[U])
{
    if constexpr (OUT == OF32) {
        if constexpr (U == 4) *(v4f *)v = *(const v4f *)p;
        else v[0] = *(const float *)p;
    } else if constexpr (U == 1) {
        v[0] = __uint_as_float((uint32_t)*(const uint16_t *)p << 16);
    } else {
        uint32_t w[U / 2];
        if constexpr (U == 8) *(v4i *)w = *(const v4i *)p;
        else w[0] = *(const uint32_t *)p;
#pragma unroll
        for (int i = 0; i < U / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <int OUT, int U>
__device__ __forceinline__ void write_c(void *p, const float (&v)[U])
{
    if constexpr (OUT == OF32) {
        if constexpr (U == 4) *(v4f *)p = *(const v4f *)v;
        else *(float *)p = v[0];
    } else if constexpr (U == 1) {
        *(uint16_t *)p = f32_to_bf16(v[0]);
    } else {
        uint32_t w[U / 2];
#pragma unroll
        for (int i = 0; i < U / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        if constexpr (U == 8) *(v4i *)p = *(const v4i *)w;
        else *(uint32_t *)p = w[0];
    }
}

// A band's residual and stores, U values at a time: consecutive lanes take
// consecutive units of a row, eight rounds of the wave's residual loads
// before their stores, so that their latency is paid once per eight.  (C may
// be the residual: an element's only reader is the thread that stores it.)
template <int OUT, int WTN, int PITCH, int U>
__device__ __forceinline__ void store_band(const Epilogue &ep, const uint8_t *stage, void *C,
                                           int row0, int col0, int M, int N, int lane)
{
    typedef typename std::conditional<OUT == OF32, float, uint16_t>::type otype;
    constexpr int UPR = WTN / U, NIT = (32 * UPR + 63) / 64;    // units per row, rounds
    constexpr int NB = NIT < 8 ? NIT : 8;
#pragma unroll 1
    for (int b = 0; b < NIT; b += NB) {
        float res[NB][U];
        if (ep.residual) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int t = (b + i) * 64 + lane, row = row0 + t / UPR, col = col0 + t % UPR * U;
                if (t < 32 * UPR && row < M && col < N)
                    read_c<OUT, U>((const otype *)ep.residual + row * ep.ldr + col, res[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int t = (b + i) * 64 + lane, r = t / UPR, c = t % UPR * U;
            if (t >= 32 * UPR || row0 + r >= M || col0 + c >= N) continue;
            const float *src = (const float *)(stage + r * PITCH) + c;
            float v[U];
            if constexpr (U >= 4) {
#pragma unroll
                for (int q = 0; q < U; q += 4) *(v4f *)(v + q) = *(const v4f *)(src + q);
            } else {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] = src[q];
            }
            if (ep.residual) {
#pragma unroll
                for (int q = 0; q < U; ++q) v[q] += res[i][q];
            }
            write_c<OUT, U>((otype *)C + (int64_t)(row0 + r) * N + col0 + c, v);
        }
    }
}

// The tile kernel's epilogue of one 32-row band of a wave's sub-tile: sums
// (bias added) in the wave's LDS at `stage`, WTN columns, row pitch PITCH
// bytes.  First the activation, in place and in a loop that is not unrolled
// (one copy of its code), then residual and stores in the widest units that
// divide the rows of C and of the residual: 16 bytes, 4 bytes, or single
// values.
template <int OUT, int WTN, int PITCH, typename EP>
__device__ __forceinline__ void fused_band(const EP &ep, uint8_t *stage, void *C, int row0,
                                           int col0, int M, int N, int lane)
{
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
    constexpr int OS = OUT == OF32 ? 4 : 2;
    const int64_t rows = (ep.residual ? ep.ldr : 0) | N;        // both pitches' low bits
    if (rows * OS % 16 == 0) store_band<OUT, WTN, PITCH, 16 / OS>(ep, stage, C, row0, col0, M, N, lane);
    else if (OS == 4 || rows % 2 == 0)
        store_band<OUT, WTN, PITCH, 4 / OS>(ep, stage, C, row0, col0, M, N, lane);
    else store_band<OUT, WTN, PITCH, 1>(ep, stage, C, row0, col0, M, N, lane);
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
