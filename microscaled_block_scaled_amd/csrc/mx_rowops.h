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

template <int IN, bool NT = false>
__device__ __forceinline__ raw8<IN> load8(const void *p, int64_t at)
{
    const v4i *q = IN == IN_F32 ? (const v4i *)((const float *)p + at)
                                : (const v4i *)((const uint16_t *)p + at);
    raw8<IN> r;
#pragma unroll
    for (int i = 0; i < (IN == IN_F32 ? 2 : 1); ++i)
        r.q[i] = NT ? __builtin_nontemporal_load(q + i) : q[i];
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
            r.q[0][i] = (int)bf16_pair(v[2 * i], v[2 * i + 1]);
        }
    }
    return r;
}

// Outputs are stored with the nontemporal hint: they are written once and
// next read by another kernel.  (Measured: norm of 16384 x 8192 BF16 168 ->
// 159 us, of 4096 x 4096 24 -> 20 us.)
template <int IN>
__device__ __forceinline__ void store8(void *p, int64_t at, const raw8<IN> &r)
{
    v4i *q = IN == IN_F32 ? (v4i *)((float *)p + at) : (v4i *)((uint16_t *)p + at);
#pragma unroll
    for (int i = 0; i < (IN == IN_F32 ? 2 : 1); ++i) __builtin_nontemporal_store(r.q[i], q + i);
}

// Bytes of 8 elements in MX format F.
template <int F> struct mx8 {
    static constexpr int bytes = F == FP4 ? 4 : is_fp6<F>::value ? 6 : 8;
    static constexpr int emax = (F == FP4 || F == F6E2) ? 2 : F == FP8 ? 8 : F == BF8 ? 15 : 4;
};

// Conversions to 8-bit floats saturate instead of overflowing to NaN or an
// infinity while bit 23 of the wave's MODE register is set.  It does the same
// to BF16 conversions, which are to round to infinities as usual, so it is
// only set around the 8-bit ones.
__device__ __forceinline__ void saturate_fp8(bool on)
{
    if (on) __builtin_amdgcn_s_setreg(1 | (23 << 6), 1);
    else __builtin_amdgcn_s_setreg(1 | (23 << 6), 0);
}

// To the compiler a conversion is pure: nothing in it says that it depends on
// MODE, so nothing keeps it on its side of saturate_fp8.  One of its operands
// and its result pass through empty volatile asm, which costs no instruction
// and stays in order with the register writes: what is computed from a held
// value comes after, what is held was computed before.  (The 8-bit conversions
// hold their scale: holding the values took registers, and 6 % of a norm of
// FP32 rows of 32768 that is short of them.)
template <typename T>
__device__ __forceinline__ void hold(T &v)
{
    asm volatile("" : "+v"(v));
}

// pack8 in a kernel that also converts to format F: outside of the windows
// that 8-bit formats have.
template <int IN, int F>
__device__ __forceinline__ raw8<IN> pack8_beside(float (&v)[8])
{
    constexpr bool HELD = IN == IN_BF16 && (F == FP8 || F == BF8);
    if constexpr (HELD)
#pragma unroll
        for (int i = 0; i < 8; i += 2) hold(v[i]);
    raw8<IN> r = pack8<IN>(v);
    if constexpr (HELD) hold(r.q[0]);
    return r;
}

// MX elements and scale byte of 8 values of a block whose other values are
// in the other lanes of the lane's group of four, by the conversion rule of
// quantize_kernel: the same bytes for the same FP32 values.  q addresses the
// lane's own elements; `first` marks the group's first lane, which stores the
// block's scale byte.
//
// In fewer operations than there, since here the arithmetic counts:
//   * the magnitudes are compared as sign-cleared bit patterns, which order as
//     they do, a NaN or an infinity at or above the infinity pattern;
//   * floor(log2 amax) + 127 is the largest one's exponent field, for a
//     subnormal or zero amax 0 (the scale byte is then 0 either way);
//   * the scaled conversions divide by 2^(byte - 127), given as the FP32
//     pattern byte << 23 (0 stands for 2^-127), round to nearest even and
//     saturate: equal to scaling, clamping and converting for every byte and
//     all values a block can hold (checked against the rule on the device
//     over all exponents, midpoints and values next to overflow).
template <int F>
__device__ __forceinline__ void quantize8(const float (&v)[8], uint8_t *q, uint8_t *s, bool first)
{
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mb = max(mb, __float_as_uint(v[i]) & 0x7fffffffu);
    mb = max(mb, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mb, 0xB1, 0xF, 0xF, false));
    mb = max(mb, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mb, 0x4E, 0xF, 0xF, false));
    const int field = (int)(mb >> 23);
    const bool bad = field == 255;
    const int e = bad ? 255 : max(field - mx8<F>::emax, 0);
    if (first) __builtin_nontemporal_store((uint8_t)e, s);
    const float scale = __int_as_float(e << 23);
    if constexpr (F == FP4) {
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
        __builtin_nontemporal_store(bad ? 0u : w, (uint32_t *)q);
    } else if constexpr (is_fp6<F>::value) {
        uint64_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (uint64_t)fp6_code<F>(ldexpf(v[i], 127 - e)) << (6 * i);
#pragma unroll
        for (int i = 0; i < 3; ++i) ((uint16_t *)q)[i] = bad ? 0 : (uint16_t)(w >> (16 * i));
    } else {
        typedef short s16x2 __attribute__((vector_size(4)));
        s16x2 w[2] = {};
        float by = scale;
        saturate_fp8(true);
        hold(by);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (F == BF8) {
                w[i] = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w[i], v[4 * i], v[4 * i + 1], by, false);
                w[i] = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w[i], v[4 * i + 2], v[4 * i + 3], by, true);
            } else {
                w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w[i], v[4 * i], v[4 * i + 1], by, false);
                w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w[i], v[4 * i + 2], v[4 * i + 3], by, true);
            }
        }
        hold(w[0]);
        hold(w[1]);
        saturate_fp8(false);
        const uint64_t both = (uint64_t)__builtin_bit_cast(uint32_t, w[0]) |
                              ((uint64_t)__builtin_bit_cast(uint32_t, w[1]) << 32);
        __builtin_nontemporal_store(bad ? 0 : both, (uint64_t *)q);
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

// 1 / sqrt(x) for x >= 0, rounded once: the hardware's root r and one Newton
// step r + r / 2 (1 - x r^2), whose residual is formed to twice FP32's width
// by two fused products.  (1 / sqrtf rounds twice, an error that a whole row
// of the norm shares.)  The hardware's root takes no subnormals, so small x is
// scaled by a square; 0 and infinity keep its infinity and 0.
__device__ __forceinline__ float root_reciprocal(float x)
{
    const bool small = x < 0x1p-100f;
    const float s = small ? x * 0x1p64f : x;
    const float r = __builtin_amdgcn_rsqf(s);
    const float h = s * r, l = fmaf(s, r, -h);             // h + l = s r
    const float e = fmaf(-l, r, fmaf(-h, r, 1.f));         // 1 - s r^2
    const float y = s > 0.f && s < __builtin_inff() ? fmaf(0.5f * r, e, r) : r;
    return small ? y * 0x1p32f : y;
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
// read once for both the sum and the norm.  Beyond 16384 values (FP32) or
// 32768 the 128 registers of 1024 threads do not hold all of it and some are
// spilled: 1024 x 32768 FP32 112 us, 3.9 TB/s of what it must move, 1024 x
// 65536 BF16 182 us, 2.6 TB/s.  The weights are loaded before the sum is known,
// beside the row itself.  Bound by HBM: 16384 x 8192 BF16 to
// E4M3 with residual 156 us a call, 6.0 TB/s of what it must move.
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
                hv[c] = pack8_beside<IN, F>(h);
                store8<IN>(a.h, row * a.width + col, hv[c]);
            }
            unpack8<IN>(hv[c], h);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[i], h[i], sum);
        }
        sum = block_sum(sum, part[flip]);
        const float rstd = root_reciprocal(sum / (float)a.width + a.eps);
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
            if (a.y) store8<IN>(a.y, at, pack8_beside<IN, F>(y));
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
// memory stays busy across the barrier.  4001 x 5120 BF16: 31 us, 5.5 TB/s of
// HBM, and 5 us for column_sum.  Beyond 8192 values a thread has 4 or 8 chunks
// and its dw sums, weights and two rows pass the registers: with the spills
// 2048 x 16384 takes 66 us in BF16 and 250 in FP32 (4096 x 8192, the same
// bytes, 52 and 105), 512 x 65536 BF16 443.
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
            gv[c] = load8<IN, true>(a.dy, row * a.lddy + col);
            hv[c] = load8<IN, true>(a.h, row * a.ldh + col);
            if (a.dh) dv[c] = load8<IN, true>(a.dh, row * a.lddh + col);
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
        float *p = a.part + (int64_t)blockIdx.x * a.width + col;   // read again at once
        *(v4f *)p = v4f{dw[c][0], dw[c][1], dw[c][2], dw[c][3]};
        *(v4f *)(p + 4) = v4f{dw[c][4], dw[c][5], dw[c][6], dw[c][7]};
    }
}

// The gradient for few rows in one launch: workgroups 0 .. rows - 1 take a
// row's dx each, the others 32 columns of dw each, straight from dy and h
// (dw needs no row sum): 8 threads of 4 columns by blockDim / 8 threads down
// the rows, joined by halves.
template <int IN>
__device__ __forceinline__ v4f load4(const void *p, int64_t at)
{
    if constexpr (IN == IN_F32) return *(const v4f *)((const float *)p + at);
    const uint2 r = *(const uint2 *)((const uint16_t *)p + at);
    return v4f{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
               __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u)};
}

template <int IN, int MAXT, int C>
__global__ void __launch_bounds__(MAXT)
norm_grad_few(NormGradArgs a, float *dw)
{
    __shared__ float part[MAXT / 64];
    __shared__ v4f sums[MAXT / 8][8];
    const int tid = threadIdx.x, T = blockDim.x;
    if (blockIdx.x >= a.rows) {
        const int cx = tid & 7, ry = tid >> 3, n = T >> 3;
        const int col = ((int)(blockIdx.x - a.rows) * 8 + cx) * 4;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int r = ry; r < (int)a.rows; r += n) {
            const v4f g = load4<IN>(a.dy, r * a.lddy + col), h = load4<IN>(a.h, r * a.ldh + col);
            const float rstd = a.rstd[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(g[i], h[i] * rstd, acc[i]);
        }
        sums[ry][cx] = acc;
        __syncthreads();
        for (int m = n; m > 1;) {
            const int half = (m + 1) >> 1;
            if (ry + half < m) sums[ry][cx] += sums[ry + half][cx];
            __syncthreads();
            m = half;
        }
        if (ry == 0) *(v4f *)(dw + col) = sums[0][cx];
        return;
    }
    const int64_t row = blockIdx.x;
    const float rstd = a.rstd[row];
    float gw[C][8], xhat[C][8], dot = 0.f;
    raw8<IN> dv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * T + tid) * 8;
        if (col >= a.width) continue;
        float w[8];
        unpack8<IN>(load8<IN>(a.dy, row * a.lddy + col), gw[c]);
        unpack8<IN>(load8<IN>(a.h, row * a.ldh + col), xhat[c]);
        unpack_weight(load_weight(a.w, col, a.w_bf16), a.w_bf16, w);
        if (a.dh) dv[c] = load8<IN>(a.dh, row * a.lddh + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            gw[c][i] *= w[i];
            xhat[c][i] *= rstd;
            dot = fmaf(gw[c][i], xhat[c][i], dot);
        }
    }
    const float mean = block_sum(dot, part) / (float)a.width;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * T + tid) * 8;
        if (col >= a.width) continue;
        float d[8] = {};
        if (a.dh) unpack8<IN>(dv[c], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(fmaf(-xhat[c][i], mean, gw[c][i]), rstd, d[i]);
        store8<IN>(a.dx, row * a.width + col, pack8<IN>(d));
    }
}

// dw[j] = sum over the n partial rows of part[.][j], in a fixed order: 32
// columns per workgroup, 8 threads of 4 columns by 128 threads down the rows,
// joined by halves.  256 rows of 5120: 4.6 us, 1.1 TB/s, a launch too short to
// reach HBM's rate.
__global__ void __launch_bounds__(1024)
column_sum(const float *__restrict__ part, float *__restrict__ dw, int n, int width)
{
    __shared__ v4f sums[128][8];
    const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
    const int col = blockIdx.x * 32 + cx * 4;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int r = ry; r < n; r += 128) acc += *(const v4f *)(part + (int64_t)r * width + col);
    sums[ry][cx] = acc;
    __syncthreads();
#pragma unroll
    for (int half = 64; half; half >>= 1) {
        if (ry < half) sums[ry][cx] += sums[ry + half][cx];
        __syncthreads();
    }
    if (ry == 0) *(v4f *)(dw + col) = sums[0][cx];
}

// y = silu(gate) * up -> MX, gate and up the two halves of a row of 2 * width
// values.  A thread takes one chunk of columns (workgroup x of the row) in
// the rows blockIdx.y, blockIdx.y + gridDim.y, ...  A wave with a gate in the
// sigmoid's tail writes its chunks again with those values (an FP32 gradient of
// 999 x 25600 took 95.5 us so, 97 with the choice ahead of its stores, 100 with
// stores on both sides of it).  Bound by HBM: 2048 x 28672
// BF16 to E4M3 50 us a call, 5.9 TB/s, with 20 VALU instructions a value.
struct GluArgs {
    const void *gu;
    uint8_t *q, *s;
    int64_t rows, ld;
    int width;
};

template <int IN, int F>
__global__ void __launch_bounds__(256)
swiglu_quantize(GluArgs a)
{
    const int col = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (col >= a.width) return;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const raw8<IN> gr = load8<IN>(a.gu, row * a.ld + col);
        const raw8<IN> ur = load8<IN>(a.gu, row * a.ld + a.width + col);
        float g[8], u[8];
        unpack8<IN>(gr, g);
        unpack8<IN>(ur, u);
        auto glu = [&](auto tail) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = g[i] * sigmoid(g[i]) * u[i];
                if (decltype(tail)::value && g[i] < kSigmoidTail)
                    y[i] = g[i] * sigmoid_tail(g[i]) * (kTailScale * u[i]);
            }
            const int64_t at = row * a.width + col;
            quantize8<F>(y, a.q + at / 8 * mx8<F>::bytes, a.s + at / 32, (threadIdx.x & 3) == 0);
        };
        glu(std::false_type{});
        if (any_below(g, kSigmoidTail)) glu(std::true_type{});
    }
}

// Gradient of y = silu(gate) * up (the MX rounding passes it through):
//   d_up = dy * gate * sig, d_gate = dy * up * sig * (1 + gate * (1 - sig)).
// Bound by HBM: 1999 x 25600 BF16 79 us a call, 6.5 TB/s.
struct GluGradArgs {
    const void *dy, *gu;
    void *dgu;
    int64_t rows, lddy, ld;
    int width;
};

template <int IN>
__global__ void __launch_bounds__(256)
swiglu_grad(GluGradArgs a)
{
    const int col = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (col >= a.width) return;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const raw8<IN> gr = load8<IN, true>(a.gu, row * a.ld + col);
        const raw8<IN> ur = load8<IN, true>(a.gu, row * a.ld + a.width + col);
        const raw8<IN> yr = load8<IN, true>(a.dy, row * a.lddy + col);
        float g[8], u[8], d[8];
        unpack8<IN>(gr, g);
        unpack8<IN>(ur, u);
        unpack8<IN>(yr, d);
        auto grad = [&](auto tail) {
            float dg[8], du[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float sig = sigmoid(g[i]), t = d[i] * sig;
                du[i] = t * g[i];
                dg[i] = t * u[i] * fmaf(g[i], 1.f - sig, 1.f);
                if (decltype(tail)::value && g[i] < kSigmoidTail) {
                    const float f = d[i] * sigmoid_tail(g[i]);
                    du[i] = f * (kTailScale * g[i]);
                    dg[i] = f * (kTailScale * u[i]) * (g[i] + 1.f);
                }
            }
            store8<IN>(a.dgu, row * 2 * a.width + col, pack8<IN>(dg));
            store8<IN>(a.dgu, row * 2 * a.width + a.width + col, pack8<IN>(du));
        };
        grad(std::false_type{});
        if (any_below(g, kSigmoidTail)) grad(std::true_type{});
    }
}

}  // namespace mx
