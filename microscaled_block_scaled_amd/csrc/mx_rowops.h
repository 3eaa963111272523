// mx_rowops.h -- gfx950 device code of the row operators that stand between
// two MX GEMMs: root-mean-square norm with the residual's addition and an MX
// output, its gradient, and the gated activation silu(gate) * up with an MX
// output, and its gradient.
//
// All of them read each input once and write each output once, so memory
// bounds them; the arithmetic is kept short enough to hide behind it.  A
// thread handles chunks of 8 consecutive values: 16 bytes of BF16 or two
// times 16 bytes of FP32 per load, 8 bytes of 8-bit elements per store.  Four
// consecutive lanes share a block of 32 values, whose largest magnitude is a
// maximum over those lanes (group_max).  All sums, statistics and gradients
// are FP32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_kernels.h"
#include "mx_math.h"
#include "mx_quant.h"
#include "mx_quant6.h"

namespace mx {

// 8 consecutive values as loaded: 4 (BF16) or 8 (FP32) dwords.
template <int IN> struct raw8 { v4i q[IN == IN_F32 ? 2 : 1]; };

template <int IN>
__device__ __forceinline__ raw8<IN> load8(const void *p, int64_t at)
{
    raw8<IN> r;
    if constexpr (IN == IN_F32) {
        r.q[0] = *(const v4i *)((const float *)p + at);
        r.q[1] = *(const v4i *)((const float *)p + at + 4);
    } else {
        r.q[0] = *(const v4i *)((const uint16_t *)p + at);
    }
    return r;
}

template <int IN>
__device__ __forceinline__ void unpack8(const raw8<IN> &r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IN == IN_F32) {
            v[i] = __int_as_float(r.q[0][i]);
            v[4 + i] = __int_as_float(r.q[1][i]);
        } else {
            v[2 * i] = __uint_as_float((uint32_t)r.q[0][i] << 16);
            v[2 * i + 1] = __uint_as_float((uint32_t)r.q[0][i] & 0xffff0000u);
        }
    }
}

// Round to the rows' type (BF16: to nearest even).
template <int IN>
__device__ __forceinline__ raw8<IN> pack8(const float (&v)[8])
{
    raw8<IN> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IN == IN_F32) {
            r.q[0][i] = __float_as_int(v[i]);
            r.q[1][i] = __float_as_int(v[4 + i]);
        } else {
            r.q[0][i] = (int)((uint32_t)f32_to_bf16(v[2 * i]) |
                              ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16));
        }
    }
    return r;
}

template <int IN>
__device__ __forceinline__ void store8(void *p, int64_t at, const raw8<IN> &r)
{
    if constexpr (IN == IN_F32) {
        *(v4i *)((float *)p + at) = r.q[0];
        *(v4i *)((float *)p + at + 4) = r.q[1];
    } else {
        *(v4i *)((uint16_t *)p + at) = r.q[0];
    }
}

// Bytes of 8 elements in MX format F.
template <int F> struct mx8 {
    static constexpr int bytes = F == FP4 ? 4 : is_fp6<F>::value ? 6 : 8;
    static constexpr int emax = (F == FP4 || F == F6E2) ? 2 : F == FP8 ? 8 : F == BF8 ? 15 : 4;
};

// MX elements and scale byte of 8 values of a block whose other values are
// in the other lanes of the lane's group of four, by the conversion rule of
// quantize_kernel: the same bytes for the same FP32 values.  q addresses the
// lane's own elements; `first` marks the group's first lane, which stores the
// block's scale byte.  The magnitudes are compared as sign-cleared bit
// patterns (those of finite values order as their magnitudes; a NaN or an
// infinity is at least the infinity pattern, which then stands for it).
template <int F>
__device__ __forceinline__ void quantize8(const float (&v)[8], uint8_t *q, uint8_t *s, bool first)
{
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mb = max(mb, __float_as_uint(v[i]) & 0x7fffffffu);
    const float amax = group_max<4>(__uint_as_float(min(mb, 0x7f800000u)));
    const bool bad = amax == __builtin_inff();
    int e = 0;
    if (bad) e = 255;
    else if (amax > 0.f) e = min(254, max(0, floor_log2(amax) - mx8<F>::emax + 127));
    if (first) *s = (uint8_t)e;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = bad ? 0.f : ldexpf(v[i], 127 - e);
    if constexpr (F == FP4) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= e2m1_pair(y[2 * i], y[2 * i + 1]) << (8 * i);
        *(uint32_t *)q = w;
    } else if constexpr (is_fp6<F>::value) {
        uint64_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (uint64_t)fp6_code<F>(y[i]) << (6 * i);
#pragma unroll
        for (int i = 0; i < 3; ++i) ((uint16_t *)q)[i] = (uint16_t)(w >> (16 * i));
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = F == BF8 ? e5m2_pair(y[4 * i], y[4 * i + 1]) |
                                  (e5m2_pair(y[4 * i + 2], y[4 * i + 3]) << 16)
                            : e4m3_pair(y[4 * i], y[4 * i + 1]) |
                                  (e4m3_pair(y[4 * i + 2], y[4 * i + 3]) << 16);
        *(uint2 *)q = make_uint2(w[0], w[1]);
    }
}

// Sum over the wave, by halving distance; every lane gets it.
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sum over the workgroup in a fixed order (each wave's, then the waves in
// order); every thread gets it.  `part` is a float of LDS per wave that no
// thread is still reading: two of them in turn need no other barrier.
__device__ __forceinline__ float block_sum(float v, float *part)
{
    v = wave_sum(v);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = part[0];
    for (int w = 1; w < waves; ++w) t += part[w];
    return t;
}

// 8 weights as loaded, FP32 or BF16 by a uniform flag.
__device__ __forceinline__ raw8<IN_F32> load_weight(const void *w, int col, int bf16)
{
    raw8<IN_F32> r;
    if (bf16) r.q[0] = load8<IN_BF16>(w, col).q[0];
    else r = load8<IN_F32>(w, col);
    return r;
}
__device__ __forceinline__ void unpack_weight(const raw8<IN_F32> &r, int bf16, float (&v)[8])
{
    if (bf16) unpack8<IN_BF16>(raw8<IN_BF16>{{r.q[0]}}, v);
    else unpack8<IN_F32>(r, v);
}

// What the norm reads and writes (pitches in elements of the rows' type; y,
// rstd and q may be null: not wanted; r null: no residual).
struct NormArgs {
    const void *x, *r, *w;
    void *h, *y;
    uint8_t *q, *s;
    float *rstd;
    int64_t rows, ldx, ldr;
    int width, w_bf16;
    float eps;
};

// h = x + r rounded to the rows' type; rstd = 1 / sqrt(mean(h^2) + eps);
// y = h * rstd * w; (q, s) = MX(y) from the unrounded y.  The statistic is of
// the rounded h, which is what the next layer and the gradient read.
//
// One workgroup per row, the row in registers (C chunks of 8 per thread,
// chunk c of thread t holding values 8 (c T + t) .., T threads), so the row is
// read once for both the sum and the norm.  The weights are loaded before the
// sum is known, beside the row itself.
template <int IN, int F, int MAXT, int C>
__global__ void __launch_bounds__(MAXT)
norm_quantize(NormArgs a)
{
    __shared__ float part[2][MAXT / 64];
    const int tid = threadIdx.x, T = blockDim.x;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        raw8<IN> hv[C], rv[C];
        raw8<IN_F32> wv[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * T + tid) * 8;
            if (col >= a.width) continue;
            hv[c] = load8<IN>(a.x, row * a.ldx + col);
            if (a.r) rv[c] = load8<IN>(a.r, row * a.ldr + col);
            wv[c] = load_weight(a.w, col, a.w_bf16);
        }
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * T + tid) * 8;
            if (col >= a.width) continue;
            float h[8];
            if (a.r) {
                float r[8];
                unpack8<IN>(hv[c], h);
                unpack8<IN>(rv[c], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += r[i];
                hv[c] = pack8<IN>(h);
                store8<IN>(a.h, row * a.width + col, hv[c]);
            }
            unpack8<IN>(hv[c], h);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[i], h[i], sum);
        }
        sum = block_sum(sum, part[flip]);
        const float rstd = 1.f / sqrtf(sum / (float)a.width + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * T + tid) * 8;
            if (col >= a.width) continue;
            float h[8], w[8], y[8];
            unpack8<IN>(hv[c], h);
            unpack_weight(wv[c], a.w_bf16, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
            const int64_t at = row * a.width + col;
            if (a.y) store8<IN>(a.y, at, pack8<IN>(y));
            if (a.q) quantize8<F>(y, a.q + at / 8 * mx8<F>::bytes, a.s + at / 32, (tid & 3) == 0);
        }
    }
}

// Gradient of the norm's unquantized y (the MX rounding passes gradients
// through unchanged), with xhat = h * rstd:
//   dx = rstd * (dy * w - xhat * mean(dy * w * xhat)) + dh,
//   dw = sum over rows of dy * xhat.
// dx is the gradient of x and of the residual alike; dh is what reaches h
// from the rest of the graph (null: nothing).
struct NormGradArgs {
    const void *dy, *h, *w, *dh;
    const float *rstd;
    void *dx;
    float *part;                 // gridDim.x x width partial dw sums (null: no dw)
    int64_t rows, lddy, ldh, lddh;
    int width, w_bf16;
};

// Workgroup b takes rows b, b + gridDim.x, ...; a thread keeps its columns'
// weights and dw sums in registers over all of them.  The next row's loads
// are issued before the current row's sum is joined over the workgroup, so
// memory stays busy across the barrier.
template <int IN, int MAXT, int C>
__global__ void __launch_bounds__(MAXT)
norm_grad(NormGradArgs a)
{
    __shared__ float part[2][MAXT / 64];
    const int tid = threadIdx.x, T = blockDim.x;
    float dw[C][8] = {};
    raw8<IN_F32> wv[C];
    raw8<IN> gv[C], hv[C], dv[C];
    float rs = 0.f;
    auto load_row = [&](int64_t row) {
        rs = a.rstd[row];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * T + tid) * 8;
            if (col >= a.width) continue;
            gv[c] = load8<IN>(a.dy, row * a.lddy + col);
            hv[c] = load8<IN>(a.h, row * a.ldh + col);
            if (a.dh) dv[c] = load8<IN>(a.dh, row * a.lddh + col);
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * T + tid) * 8;
        if (col < a.width) wv[c] = load_weight(a.w, col, a.w_bf16);
    }
    if (blockIdx.x < a.rows) load_row(blockIdx.x);
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        const float rstd = rs;
        float dot = 0.f;
        raw8<IN> g0[C], h0[C], d0[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            g0[c] = gv[c], h0[c] = hv[c], d0[c] = dv[c];
            if ((c * T + tid) * 8 >= a.width) continue;
            float g[8], h[8], w[8];
            unpack8<IN>(gv[c], g);
            unpack8<IN>(hv[c], h);
            unpack_weight(wv[c], a.w_bf16, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = h[i] * rstd;
                dot = fmaf(g[i] * w[i], xhat, dot);
                dw[c][i] = fmaf(g[i], xhat, dw[c][i]);
            }
        }
        if (row + gridDim.x < a.rows) load_row(row + gridDim.x);
        const float mean = block_sum(dot, part[flip]) / (float)a.width;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * T + tid) * 8;
            if (col >= a.width) continue;
            float g[8], h[8], w[8], d[8] = {};
            unpack8<IN>(g0[c], g);
            unpack8<IN>(h0[c], h);
            unpack_weight(wv[c], a.w_bf16, w);
            if (a.dh) unpack8<IN>(d0[c], d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = fmaf(fmaf(-(h[i] * rstd), mean, g[i] * w[i]), rstd, d[i]);
            store8<IN>(a.dx, row * a.width + col, pack8<IN>(d));
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * T + tid) * 8;
        if (col >= a.width) continue;
        store8<IN_F32>(a.part, (int64_t)blockIdx.x * a.width + col, pack8<IN_F32>(dw[c]));
    }
}

// dw[j] = sum over the n partial rows of part[.][j], in a fixed order: 32
// columns per workgroup, 32 threads down the rows by 8 threads of 4 columns.
__global__ void __launch_bounds__(256)
column_sum(const float *__restrict__ part, float *__restrict__ dw, int n, int width)
{
    __shared__ v4f sums[32][8];
    const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
    const int col = blockIdx.x * 32 + cx * 4;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int r = ry; r < n; r += 32) acc += *(const v4f *)(part + (int64_t)r * width + col);
    sums[ry][cx] = acc;
    __syncthreads();
    if (ry) return;
    for (int r = 1; r < 32; ++r) acc += sums[r][cx];
    *(v4f *)(dw + col) = acc;
}

// y = silu(gate) * up -> MX, gate and up the two halves of a row of 2 * width
// values.  A thread takes one chunk; the workgroups walk (row, 2048 columns)
// items in order.
struct GluArgs {
    const void *gu;
    uint8_t *q, *s;
    int64_t rows, ld, items;
    int width, per_row;          // per_row: workgroup items in a row
};

template <int IN, int F>
__global__ void __launch_bounds__(256)
swiglu_quantize(GluArgs a)
{
    for (int64_t it = blockIdx.x; it < a.items; it += gridDim.x) {
        const int64_t row = it / a.per_row;
        const int col = (int)(it - row * a.per_row) * 2048 + threadIdx.x * 8;
        if (col >= a.width) continue;
        const raw8<IN> gr = load8<IN>(a.gu, row * a.ld + col);
        const raw8<IN> ur = load8<IN>(a.gu, row * a.ld + a.width + col);
        float g[8], u[8], y[8];
        unpack8<IN>(gr, g);
        unpack8<IN>(ur, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = g[i] * sigmoid(g[i]) * u[i];
        const int64_t at = row * a.width + col;
        quantize8<F>(y, a.q + at / 8 * mx8<F>::bytes, a.s + at / 32, (threadIdx.x & 3) == 0);
    }
}

// Gradient of y = silu(gate) * up (the MX rounding passes it through):
//   d_up = dy * gate * sig, d_gate = dy * up * sig * (1 + gate * (1 - sig)).
struct GluGradArgs {
    const void *dy, *gu;
    void *dgu;
    int64_t rows, lddy, ld, items;
    int width, per_row;
};

template <int IN>
__global__ void __launch_bounds__(256)
swiglu_grad(GluGradArgs a)
{
    for (int64_t it = blockIdx.x; it < a.items; it += gridDim.x) {
        const int64_t row = it / a.per_row;
        const int col = (int)(it - row * a.per_row) * 2048 + threadIdx.x * 8;
        if (col >= a.width) continue;
        const raw8<IN> gr = load8<IN>(a.gu, row * a.ld + col);
        const raw8<IN> ur = load8<IN>(a.gu, row * a.ld + a.width + col);
        const raw8<IN> yr = load8<IN>(a.dy, row * a.lddy + col);
        float g[8], u[8], d[8];
        unpack8<IN>(gr, g);
        unpack8<IN>(ur, u);
        unpack8<IN>(yr, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float sig = sigmoid(g[i]), t = d[i] * sig;
            const float du = t * g[i];
            g[i] = t * u[i] * fmaf(g[i], 1.f - sig, 1.f);
            u[i] = du;
        }
        void *const out = a.dgu;
        store8<IN>(out, row * 2 * a.width + col, pack8<IN>(g));
        store8<IN>(out, row * 2 * a.width + a.width + col, pack8<IN>(u));
    }
}

}  // namespace mx
