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
    static constexpr bool fused = true, stream_b = false, order_all = true;
    typedef void *C_ptr;
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

// 2 sqrt(2 / pi) (v + 0.044715 v^3)
__device__ __forceinline__ float tanh_argument(float v)
{
    return 1.59576912f * v * fmaf(0.044715f * v, v, 1.f);
}

// An activation for values that are not in the tail.
template <int ACT>
__device__ __forceinline__ float act_of(float v)
{
    if constexpr (ACT == ACT_RELU) return v > 0.f ? v : v != v ? v : 0.f;
    if constexpr (ACT == ACT_SILU) return v * sigmoid(v);
    if constexpr (ACT == ACT_GELU) {
        const float q = normal_tail(fabsf(v));
        return v * (v > 0.f ? 1.f - q : q);
    }
    // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
    if constexpr (ACT == ACT_GELU_TANH) return v * sigmoid(tanh_argument(v));
    return v;
}

// And for any value.
template <int ACT>
__device__ __forceinline__ float act_any(float v)
{
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU_TANH) {
        const float w = ACT == ACT_SILU ? v : tanh_argument(v);
        if (w < kSigmoidTail) return v * sigmoid_tail(w) * kTailScale;
    }
    return act_of<ACT>(v);
}

__device__ __forceinline__ float act_apply(float v, int act)
{
    switch (act) {
    case ACT_RELU: return act_any<ACT_RELU>(v);
    case ACT_SILU: return act_any<ACT_SILU>(v);
    case ACT_GELU: return act_any<ACT_GELU>(v);
    case ACT_GELU_TANH: return act_any<ACT_GELU_TANH>(v);
    default: return v;
    }
}

// The values below which the activation's sigmoid is in its tail: by the
// argument itself, or by the cubic, which is -85.0 at -9.9 (and -87.3 at
// -10.0); no values for the others.
__device__ __forceinline__ float act_tail(int act)
{
    return act == ACT_SILU ? kSigmoidTail : act == ACT_GELU_TANH ? -9.9f : -__builtin_inff();
}

template <int ACT>
__device__ __forceinline__ void act_16(v4f (&v)[4])
{
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[u][q] = act_of<ACT>(v[u][q]);
}
__device__ __forceinline__ void act_apply16(v4f (&v)[4], int act)
{
    switch (act) {
    case ACT_RELU: act_16<ACT_RELU>(v); break;
    case ACT_SILU: act_16<ACT_SILU>(v); break;
    case ACT_GELU: act_16<ACT_GELU>(v); break;
    case ACT_GELU_TANH: act_16<ACT_GELU_TANH>(v); break;
    default: break;
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

// U values of C's type as they are in memory: 16, 4 or 2 bytes.
template <int BYTES> struct c_unit;
template <> struct c_unit<16> { typedef v4i t; };
template <> struct c_unit<4> { typedef uint32_t t; };
template <> struct c_unit<2> { typedef uint16_t t; };

template <int OUT, int U, typename T>
__device__ __forceinline__ void add_unit(const T &r, float (&v)[U])
{
    if constexpr (U == 1) {
        v[0] += __uint_as_float(OUT == OF32 ? (uint32_t)r : (uint32_t)r << 16);
    } else {
        uint32_t w[sizeof(T) / 4];
        __builtin_memcpy(w, &r, sizeof(T));
#pragma unroll
        for (int i = 0; i < U; ++i)
            v[i] += __uint_as_float(OUT == OF32 ? w[i] : (i & 1) ? w[i / 2] & 0xffff0000u
                                                                  : w[i / 2] << 16);
    }
}
template <int OUT, int U, typename T>
__device__ __forceinline__ T make_unit(const float (&v)[U])
{
    T r;
    if constexpr (OUT == OF32) {
        __builtin_memcpy(&r, v, sizeof(T));
    } else if constexpr (U == 1) {
        r = f32_to_bf16(v[0]);
    } else {
        uint32_t w[U / 2];
#pragma unroll
        for (int i = 0; i < U / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        __builtin_memcpy(&r, w, sizeof(T));
    }
    return r;
}

constexpr int gcd_of(int a, int b) { return b ? gcd_of(b, a % b) : a; }
// The largest divisor of n that is at most `most`.
constexpr int part_of(int n, int most)
{
    int d = n < most ? n : most;
    while (n % d) --d;
    return d;
}

// The tile kernel's epilogue for a wave's FM bands of 32 rows and WTN
// columns, U values at a time.  stage_band writes a band's sums (bias added)
// to the wave's LDS.  L lanes take consecutive units of a row, 64 / L rows at
// once, SEG times across the row, so that a lane's column and its row within
// a turn do not change from turn to turn (dividing a running index by 96
// columns cost more than the stores on the 192-column tile).
//
// The residual is read ahead, up to 8 or 16 units a lane: all bands' before
// the first is staged, or a band's first part before its activation and each
// further part before its stores, so its latency is met seldom; one load per
// store and wait for it cost 10 us on 293 x 3443 x 2688.  The band's LDS is the
// wave's own, and the hardware keeps a wave's LDS accesses in order, so its
// lanes hand values to each other without a barrier; the wave fences, which
// cost no instruction, keep the compiler to that order.  (C may be the
// residual: an element's only reader is the thread that stores it.)
// 2048 x 8192 x 28672 E2M1 with bias, GELU and residual takes 245 us, the
// product alone 232.
template <int OUT, int WTN, int PITCH, int FM, int U, typename Stage>
__device__ __forceinline__ void fused_rows(const Epilogue &ep, Stage stage_band, uint8_t *stage,
                                           void *C, int row0, int col0, int M, int N, int lane)
{
    typedef typename std::conditional<OUT == OF32, float, uint16_t>::type otype;
    typedef typename c_unit<U * sizeof(otype)>::t T;
    constexpr int UPR = WTN / U, NIT = UPR / 2;                 // units per row, per lane and band
    constexpr int L = gcd_of(UPR, 64), SEG = UPR / L, RPT = 64 / L;   // RPT: rows per turn
    constexpr int MOST = sizeof(T) == 16 ? 8 : 16;              // units read ahead
    constexpr bool AHEAD = FM * NIT <= MOST;
    constexpr int NB = part_of(NIT / SEG, MOST / SEG > 0 ? MOST / SEG : 1) * SEG;
    static_assert(NIT % SEG == 0 && NIT % NB == 0 && NB % SEG == 0, "whole turns and parts");
    const int lrow = lane / L, lcol = lane % L * U;
    T res[AHEAD ? FM : 1][NB];
    auto load = [&](int band, int first, T (&r)[NB]) {
        const int row = row0 + band * 32 + first / SEG * RPT + lrow;
        const otype *p = (const otype *)ep.residual + row * ep.ldr + col0 + lcol;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int dr = i / SEG * RPT, dc = i % SEG * L * U;
            r[i] = T{};
            if (row + dr < M && col0 + lcol + dc < N) r[i] = *(const T *)(p + dr * ep.ldr + dc);
        }
    };
    if (AHEAD && ep.residual) {
#pragma unroll
        for (int b = 0; b < FM; ++b) load(b, 0, res[AHEAD ? b : 0]);
    }
    static_for<FM>([&](auto bc) {
        constexpr int b = decltype(bc)::value;
        stage_band(bc);
        wave_fence();                        // staged by other lanes than read it
        if (!AHEAD && ep.residual) load(b, 0, res[0]);
        if (ep.act != ACT_NONE) {
            // in place, 16 values a lane and turn: enough independent chains
            // to keep the wave busy, one copy of the code per band
            constexpr int QPR = WTN / 4;                        // float4 per row
            static_assert(QPR % 8 == 0, "whole turns");
            const float tail = act_tail(ep.act);
#pragma unroll 1
            for (int t0 = lane; t0 < 32 * QPR; t0 += 256) {
                v4f v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = t0 + u * 64;
                    v[u] = *(const v4f *)(stage + (t / QPR) * PITCH + (t % QPR) * 16);
                }
                float all[16];
                __builtin_memcpy(all, v, sizeof(all));
                if (any_below(all, tail)) {          // seldom: value by value, in little code
#pragma unroll 1
                    for (int e = 0; e < 16; ++e) {
                        const int t = t0 + (e >> 2) * 64;
                        float *x = (float *)(stage + (t / QPR) * PITCH + (t % QPR) * 16) + (e & 3);
                        *x = act_apply(*x, ep.act);
                    }
                    continue;
                }
                act_apply16(v, ep.act);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = t0 + u * 64;
                    *(v4f *)(stage + (t / QPR) * PITCH + (t % QPR) * 16) = v[u];
                }
            }
            wave_fence();                    // so are the activated values
        }
#pragma unroll 1
        for (int first = 0; first < NIT; first += NB) {
            if (first && ep.residual) load(b, first, res[AHEAD ? b : 0]);
            const int r0 = first / SEG * RPT + lrow, row = row0 + b * 32 + r0;
            const float *src = (const float *)(stage + r0 * PITCH) + lcol;
            otype *dst = (otype *)C + (int64_t)row * N + col0 + lcol;
            // all values first, then all stores: a wait between a store and the
            // next value would be for the store itself
            T(&out)[NB] = res[AHEAD ? b : 0];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int dr = i / SEG * RPT, dc = i % SEG * L * U;
                const float *s = (const float *)((const uint8_t *)src + dr * PITCH) + dc;
                float v[U];
                if constexpr (U >= 4) {
#pragma unroll
                    for (int q = 0; q < U; q += 4) *(v4f *)(v + q) = *(const v4f *)(s + q);
                } else {
#pragma unroll
                    for (int q = 0; q < U; ++q) v[q] = s[q];
                }
                if (ep.residual) add_unit<OUT, U>(out[i], v);
                out[i] = make_unit<OUT, U, T>(v);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int dr = i / SEG * RPT, dc = i % SEG * L * U;
                if (row + dr < M && col0 + lcol + dc < N) *(T *)(dst + (int64_t)dr * N + dc) = out[i];
            }
        }
        wave_fence();                        // all lanes have read before the next band
    });
}

// In the widest units that divide the rows of C and of the residual: 16
// bytes, 4 bytes, or single values.
template <int OUT, int WTN, int PITCH, int FM, typename EP, typename Stage>
__device__ __forceinline__ void fused_store(const EP &ep, Stage stage_band, uint8_t *stage,
                                            void *C, int row0, int col0, int M, int N, int lane)
{
    constexpr int OS = OUT == OF32 ? 4 : 2;
    const int64_t pitch = (ep.residual ? ep.ldr : 0) | N;       // both pitches' low bits
    if (pitch * OS % 16 == 0)
        fused_rows<OUT, WTN, PITCH, FM, 16 / OS>(ep, stage_band, stage, C, row0, col0, M, N, lane);
    else if (OS == 4 || pitch % 2 == 0)
        fused_rows<OUT, WTN, PITCH, FM, 4 / OS>(ep, stage_band, stage, C, row0, col0, M, N, lane);
    else
        fused_rows<OUT, WTN, PITCH, FM, 1>(ep, stage_band, stage, C, row0, col0, M, N, lane);
}

// splitk_reduce with the epilogue: C[i] from the sum over slices, in slice
// order, of W[s * plane + i]; n_cols is C's row length, mn < 2^30.  A thread
// takes 4 consecutive values; where all rows (C's and the residual's) are
// multiples of 4 values they lie in one row and are read and stored together.
template <int OUT>
__global__ void __launch_bounds__(256)
splitk_fused(const float *__restrict__ W, void *C, int mn, int n_cols, int64_t plane, int slices,
             Epilogue ep)
{
    typedef typename std::conditional<OUT == OF32, v4f, uint2>::type T;
    typedef typename std::conditional<OUT == OF32, float, uint16_t>::type otype;
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= mn) return;
    int m = (int)((uint32_t)i / (uint32_t)n_cols), c = i - m * n_cols;
    const bool whole = (((ep.residual ? ep.ldr : 0) | n_cols) & 3) == 0;
    T r{};
    if (whole && ep.residual) r = *(const T *)((const otype *)ep.residual + m * ep.ldr + c);
    v4f acc = *(const v4f *)(W + i);
    for (int s = 1; s < slices; ++s) acc += *(const v4f *)(W + s * plane + i);
    if (whole) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = act_apply(acc[q] + bias_at(ep, c + q), ep.act);
        if (ep.residual) add_unit<OUT, 4>(r, v);
        *(T *)((otype *)C + i) = make_unit<OUT, 4, T>(v);
        return;
    }
    for (int q = 0; q < min(4, mn - i); ++q) {
        const float v = epilogue_at<OUT>(ep, acc[q], m, c);
        if (OUT == OF32) ((float *)C)[i + q] = v;
        else ((uint16_t *)C)[i + q] = f32_to_bf16(v);
        if (++c == n_cols) { c = 0; ++m; }
    }
}

// The decode kernel with the epilogue.  Bound by the weights: 8 x 8192 x 28672
// E4M3 x E2M1 with bias and residual 26 us a call, 4.9 TB/s.  That is one
// column group a workgroup; with several the rings run empty after each (the
// bias's and residual's loads, see mx_decode.h) and the last round is partial:
// 20 x 12326 x 10368 E2M1 27.4 us, 26.4 without either, for 68 MB.
template <int FA, int FB, int OUT, int WA>
__global__ void __launch_bounds__(kDecodeWaves * 64)
fused_decode(const uint8_t *__restrict__ A, const uint8_t *__restrict__ As,
             const uint8_t *__restrict__ B, const uint8_t *__restrict__ Bs, void *C, int M, int N,
             int K, Epilogue ep)
{
    decode_body<FA, FB, OUT, WA>(A, As, B, Bs, C, M, N, K, ep);
}

}  // namespace mx
