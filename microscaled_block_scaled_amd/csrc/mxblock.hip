// mxblock.hip -- host side of the row operators and the expert routing of
// include/mxgemm.h: argument checks (all before any HIP call) and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "mxgemm.h"
#include "mx_host.h"
#include "mx_moe.h"
#include "mx_rowops.h"

using namespace mxhost;

namespace {

bool is_fmt(int fmt) { return fmt >= MX_FMT_E2M1 && fmt <= MX_FMT_E3M2; }
bool is_dtype(int t) { return t == MX_IN_FP32 || t == MX_IN_BF16; }
int64_t size_of(int t) { return t == MX_IN_FP32 ? 4 : 2; }

// rows x width of a row operator: width a multiple of 32 (one scale block),
// at most MX_ROW_MAX_WIDTH; zero rows are allowed.
bool row_shape(int64_t rows, int64_t width)
{
    return rows >= 0 && rows <= MX_MAX_DIM && width >= 32 && width % 32 == 0 &&
           width <= MX_ROW_MAX_WIDTH;
}

// A pitch in elements of `size` bytes: whole rows, each 16-byte aligned.
bool pitch_shape(int64_t ld, int64_t width) { return ld >= width && ld <= MX_MAX_DIM; }
bool pitch_aligned(int64_t ld, int64_t size) { return ld * size % 16 == 0; }

// Grid of a kernel whose workgroups walk `items` grid-stride: enough to fill
// the GPU many times over, and few enough for a 32-bit count of threads.
unsigned stride_grid(int64_t items) { return (unsigned)std::min<int64_t>(items, 1 << 20); }

// The y extent of a grid whose workgroups walk rows with its stride.
unsigned rows_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 65535); }

// `waves` waves per row or token, in workgroups of at most 8.
struct WaveGrid { dim3 grid, block; };
WaveGrid wave_grid(int64_t waves, int64_t rows)
{
    const int64_t wgs = cdiv(waves, 8);
    return {dim3((unsigned)wgs, rows_grid(rows)), dim3((unsigned)(cdiv(waves, wgs) * 64))};
}

int launched() { return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

// Calls f(IN, F) with the rows' type and the MX format as integral constants.
template <typename Fn>
void with_fmt(int dtype, int fmt, Fn f)
{
    auto in = [&](auto fc) {
        if (dtype == MX_IN_FP32) f(std::integral_constant<int, mx::IN_F32>{}, fc);
        else f(std::integral_constant<int, mx::IN_BF16>{}, fc);
    };
    switch (fmt) {
    case MX_FMT_E2M1: in(std::integral_constant<int, mx::FP4>{}); break;
    case MX_FMT_E4M3: in(std::integral_constant<int, mx::FP8>{}); break;
    case MX_FMT_E5M2: in(std::integral_constant<int, mx::BF8>{}); break;
    case MX_FMT_E2M3: in(std::integral_constant<int, mx::F6E2>{}); break;
    default: in(std::integral_constant<int, mx::F6E3>{}); break;
    }
}

// Calls f(MAXT, C, threads): chunks of 8 values per thread, the threads of a
// row's workgroup, and the most threads of that kernel.  Rows of up to 8192
// values take FIRST chunks per thread; longer rows what 512 or 1024 threads
// need, with registers spilled as the kernels say.
template <int FIRST, typename Fn>
void with_row(int64_t width, Fn f)
{
    const int64_t chunks = width / 8;
    auto go = [&](auto t, auto c) { f(t, c, (int)(cdiv(chunks, 64 * c()) * 64)); };
#define MX_ROW(T_, C_) go(std::integral_constant<int, T_>{}, std::integral_constant<int, C_>{})
    if (chunks <= 1024) MX_ROW(1024 / FIRST, FIRST);
    else if (chunks <= 2048) MX_ROW(512, 4);
    else if (chunks <= 4096) MX_ROW(1024, 4);
    else MX_ROW(1024, 8);
#undef MX_ROW
}

// Workgroups of the norm's gradient: each keeps partial dw sums over its
// rows, which are written and read once more, so one per CU.  (Two per CU:
// 8192 x 4096 BF16 53.7 us against 50.5, four 59.0.)
int64_t norm_grad_groups(int64_t rows) { return std::min<int64_t>(rows, kCUs); }

// Up to this many rows of at most 8192 values the gradient with dw is one
// launch without partial sums (norm_grad_few), which reads dy and h twice.
// (A call on 64 x 4096 BF16 7.6 us, with partial sums 11.0; 256 x 8192 7.7 and
// 12.6; 512 x 4096 8.0 and 10.4; 1024 x 4096 14.1 and 12.9.)
constexpr int64_t kGradFew = 512;
bool grad_few(int64_t rows, int64_t width) { return rows > 0 && rows <= kGradFew && width <= 8192; }

// Pairs per workgroup of the sort: all of them up to kSortOne, else a 256th
// part in whole 1024-pair steps of the workgroup, 2048 at least.  (One
// workgroup and launch: 1024 pairs 6.3 us a call, two launches 9.6; 4096
// pairs 8.4 and 9.6; 8192 pairs 13.4 and 9.6.)
constexpr int64_t kSortOne = 4096;
int64_t sort_chunk(int64_t n)
{
    if (n <= kSortOne) return cdiv(n, mx::kSortThreads) * mx::kSortThreads;
    return std::max<int64_t>(2048, cdiv(cdiv(n, kCUs), mx::kSortThreads) * mx::kSortThreads);
}

bool moe_shape(int64_t tokens, int64_t top)
{
    return tokens >= 0 && top >= 1 && top <= MX_MOE_MAX_TOP && tokens <= MX_MAX_DIM &&
           tokens * top <= MX_MAX_DIM;
}

}  // namespace

extern "C" int mx_rmsnorm_quantize(int fmt, int dtype, int w_dtype, int64_t rows, int64_t width,
                                   const void *X, int64_t ldx, const void *R, int64_t ldr,
                                   const void *W, float eps, void *H, void *Y, void *Q,
                                   void *Q_scale, float *rstd, void *stream)
{
    if (Q && !is_fmt(fmt)) return MX_ERR_FORMAT;
    if (!is_dtype(dtype) || !is_dtype(w_dtype)) return MX_ERR_IN_DTYPE;
    if (!row_shape(rows, width) || !pitch_shape(ldx, width) || (R && !pitch_shape(ldr, width)))
        return MX_ERR_ROW_SHAPE;
    if (!(eps >= 0.f)) return MX_ERR_ROW_SHAPE;
    if (rows == 0) return MX_OK;
    if (!X || !W || (R && !H) || (!Q && !Y) || (Q && !Q_scale)) return MX_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(X, 16) || !aligned(R, 16) || !aligned(W, 16) || !aligned(H, 16) ||
        !aligned(Y, 16) || !aligned(Q, 8) || !aligned(rstd, 4) || !pitch_aligned(ldx, es) ||
        (R && !pitch_aligned(ldr, es)))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    const mx::NormArgs a{X, R, W, H, Y, (uint8_t *)Q, (uint8_t *)Q_scale, rstd, rows, ldx, ldr,
                         (int)width, w_dtype == MX_IN_BF16, eps};
    with_fmt(dtype, Q ? fmt : MX_FMT_E4M3, [&](auto in, auto f) {
        // two chunks per thread: 4096 x 8192 BF16 44 us, with one 46; 8 x 8192
        // 4.3 us, with one 4.4
        with_row<2>(width, [&](auto t, auto c, int threads) {
            hipLaunchKernelGGL((mx::norm_quantize<in(), f(), t(), c()>), dim3(stride_grid(rows)),
                               dim3(threads), 0, (hipStream_t)stream, a);
        });
    });
    return launched();
}

extern "C" int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t width)
{
    if (!row_shape(rows, width)) return MX_ERR_ROW_SHAPE;
    return grad_few(rows, width) ? 0 : norm_grad_groups(rows) * width * 4;
}

extern "C" int mx_rmsnorm_backward(int dtype, int w_dtype, int64_t rows, int64_t width,
                                   const void *dY, int64_t lddy, const void *H, int64_t ldh,
                                   const float *rstd, const void *W, const void *dH,
                                   int64_t lddh, void *dX, float *dW, void *workspace,
                                   int64_t workspace_bytes, void *stream)
{
    if (!is_dtype(dtype) || !is_dtype(w_dtype)) return MX_ERR_IN_DTYPE;
    if (!row_shape(rows, width) || !pitch_shape(lddy, width) || !pitch_shape(ldh, width) ||
        (dH && !pitch_shape(lddh, width)))
        return MX_ERR_ROW_SHAPE;
    if (rows == 0 && !dW) return MX_OK;
    const int64_t need = dW ? mx_rmsnorm_backward_workspace(rows, width) : 0;
    if ((rows && (!dY || !H || !rstd || !W || !dX)) || (need && !workspace)) return MX_ERR_NULL;
    if (workspace_bytes < need) return MX_ERR_WORKSPACE;
    const int64_t es = size_of(dtype);
    if (!aligned(dY, 16) || !aligned(H, 16) || !aligned(W, 16) || !aligned(dH, 16) ||
        !aligned(dX, 16) || !aligned(dW, 16) || !aligned(workspace, 16) || !aligned(rstd, 4) ||
        !pitch_aligned(lddy, es) || !pitch_aligned(ldh, es) || (dH && !pitch_aligned(lddh, es)))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    hipStream_t s = (hipStream_t)stream;
    const int64_t groups = norm_grad_groups(rows);
    const mx::NormGradArgs a{dY, H, W, dH, rstd, dX, dW ? (float *)workspace : nullptr, rows,
                             lddy, ldh, lddh, (int)width, w_dtype == MX_IN_BF16};
    if (dW && grad_few(rows, width)) {
        with_row<1>(width, [&](auto t, auto c, int threads) {
            const dim3 grid((unsigned)(rows + width / 32));
            if constexpr (c() <= 1) {
                if (dtype == MX_IN_FP32)
                    hipLaunchKernelGGL((mx::norm_grad_few<mx::IN_F32, t(), c()>), grid,
                                       dim3(threads), 0, s, a, dW);
                else
                    hipLaunchKernelGGL((mx::norm_grad_few<mx::IN_BF16, t(), c()>), grid,
                                       dim3(threads), 0, s, a, dW);
            }
        });
        return launched();
    }
    if (groups)
        // one chunk per thread, and with it the next row's loads in flight:
        // 8192 x 4096 BF16 50 us, with two 52
        with_row<1>(width, [&](auto t, auto c, int threads) {
            if (dtype == MX_IN_FP32)
                hipLaunchKernelGGL((mx::norm_grad<mx::IN_F32, t(), c()>), dim3((unsigned)groups),
                                   dim3(threads), 0, s, a);
            else
                hipLaunchKernelGGL((mx::norm_grad<mx::IN_BF16, t(), c()>), dim3((unsigned)groups),
                                   dim3(threads), 0, s, a);
        });
    if (dW)
        hipLaunchKernelGGL(mx::column_sum, dim3((unsigned)(width / 32)), dim3(1024), 0, s,
                           (const float *)workspace, dW, (int)groups, (int)width);
    return launched();
}

extern "C" int mx_swiglu_quantize(int fmt, int dtype, int64_t rows, int64_t width,
                                  const void *GU, int64_t ld, void *Q, void *Q_scale,
                                  void *stream)
{
    if (!is_fmt(fmt)) return MX_ERR_FORMAT;
    if (!is_dtype(dtype)) return MX_ERR_IN_DTYPE;
    if (!row_shape(rows, width) || !pitch_shape(ld, 2 * width)) return MX_ERR_ROW_SHAPE;
    if (rows == 0) return MX_OK;
    if (!GU || !Q || !Q_scale) return MX_ERR_NULL;
    if (!aligned(GU, 16) || !aligned(Q, 8) || !pitch_aligned(ld, size_of(dtype)))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    const mx::GluArgs a{GU, (uint8_t *)Q, (uint8_t *)Q_scale, rows, ld, (int)width};
    const dim3 grid((unsigned)cdiv(width, 2048), rows_grid(rows));
    with_fmt(dtype, fmt, [&](auto in, auto f) {
        hipLaunchKernelGGL((mx::swiglu_quantize<in(), f()>), grid, dim3(256), 0, (hipStream_t)stream, a);
    });
    return launched();
}

extern "C" int mx_swiglu_backward(int dtype, int64_t rows, int64_t width, const void *dY,
                                  int64_t lddy, const void *GU, int64_t ld, void *dGU,
                                  void *stream)
{
    if (!is_dtype(dtype)) return MX_ERR_IN_DTYPE;
    if (!row_shape(rows, width) || !pitch_shape(lddy, width) || !pitch_shape(ld, 2 * width))
        return MX_ERR_ROW_SHAPE;
    if (rows == 0) return MX_OK;
    if (!dY || !GU || !dGU) return MX_ERR_NULL;
    if (!aligned(dY, 16) || !aligned(GU, 16) || !aligned(dGU, 16) ||
        !pitch_aligned(lddy, size_of(dtype)) || !pitch_aligned(ld, size_of(dtype)))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    const mx::GluGradArgs a{dY, GU, dGU, rows, lddy, ld, (int)width};
    const dim3 grid((unsigned)cdiv(width, 2048), rows_grid(rows));
    if (dtype == MX_IN_FP32)
        hipLaunchKernelGGL(mx::swiglu_grad<mx::IN_F32>, grid, dim3(256), 0,
                           (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL(mx::swiglu_grad<mx::IN_BF16>, grid, dim3(256), 0,
                           (hipStream_t)stream, a);
    return launched();
}

extern "C" int64_t mx_moe_sort_workspace(int64_t tokens, int64_t top, int64_t experts)
{
    if (!moe_shape(tokens, top) || experts < 1 || experts > MX_MAX_GROUPS)
        return MX_ERR_ROW_SHAPE;
    const int64_t n = tokens * top;
    return n <= kSortOne ? 0 : cdiv(n, sort_chunk(n)) * (experts + 1) * 4;
}

extern "C" int mx_moe_sort(int id_bytes, int64_t tokens, int64_t top, int64_t experts,
                           const void *ids, int64_t *group_rows, int32_t *row_of,
                           void *workspace, int64_t workspace_bytes, void *stream)
{
    if (id_bytes != 4 && id_bytes != 8) return MX_ERR_IN_DTYPE;
    const int64_t need = mx_moe_sort_workspace(tokens, top, experts);
    if (need < 0) return (int)need;
    if (!group_rows || (tokens && (!ids || !row_of)) || (need && !workspace)) return MX_ERR_NULL;
    if (workspace_bytes < need) return MX_ERR_WORKSPACE;
    if (!aligned(ids, id_bytes) || !aligned(group_rows, 8) || !aligned(row_of, 4) ||
        !aligned(workspace, 4))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    hipStream_t s = (hipStream_t)stream;
    const int64_t n = tokens * top;
    const mx::SortArgs a{ids, group_rows, row_of, (int32_t *)workspace, n, sort_chunk(n),
                         (int)experts, id_bytes == 8};
    if (n <= kSortOne) {
        hipLaunchKernelGGL(mx::moe_sort<false>, dim3(1), dim3(mx::kSortThreads), 0, s, a);
    } else {
        const dim3 grid((unsigned)cdiv(n, a.chunk));
        hipLaunchKernelGGL(mx::moe_count, grid, dim3(mx::kSortThreads), 0, s, a);
        hipLaunchKernelGGL(mx::moe_sort<true>, grid, dim3(mx::kSortThreads), 0, s, a);
    }
    return launched();
}

extern "C" int mx_moe_gather(int64_t tokens, int64_t top, const int32_t *row_of,
                             const void *X, int64_t row_bytes, int64_t ldx,
                             const void *X_scale, int64_t scale_bytes, int64_t lds,
                             void *XS, void *XS_scale, void *stream)
{
    if (!moe_shape(tokens, top) || row_bytes < 1 || row_bytes > MX_MAX_K || ldx < row_bytes ||
        ldx > MX_MAX_DIM)
        return MX_ERR_ROW_SHAPE;
    if (X_scale && (scale_bytes < 1 || scale_bytes > MX_MAX_K || lds < scale_bytes ||
                    lds > MX_MAX_DIM))
        return MX_ERR_ROW_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!row_of || !X || !XS || (X_scale && !XS_scale)) return MX_ERR_NULL;
    if (!aligned(row_of, 4)) return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    // Copy units: 16, 4 or 1 bytes, the largest that divides every address.
    auto unit_of = [](const void *p, const void *q, int64_t bytes, int64_t ld) {
        const uintptr_t all = (uintptr_t)p | (uintptr_t)q | (uintptr_t)bytes | (uintptr_t)ld;
        return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
    };
    const int u = unit_of(X, XS, row_bytes, ldx);
    const int us = X_scale ? unit_of(X_scale, XS_scale, scale_bytes, lds) : u;
    const int row_segs = (int)cdiv(row_bytes, 64 * u);
    const int segs = row_segs + (X_scale ? (int)cdiv(scale_bytes, 64 * us) : 0);
    const mx::GatherArgs a{(const uint8_t *)X, (const uint8_t *)X_scale, (uint8_t *)XS,
                           (uint8_t *)XS_scale, row_of, tokens, tokens * top, ldx, lds,
                           (int)top, (int)row_bytes, (int)scale_bytes, row_segs, segs};
    const WaveGrid g = wave_grid(segs, tokens);
    hipStream_t s = (hipStream_t)stream;
#define MX_GATHER(U_, US_)                                                                 \
    if (u == U_ && us == US_)                                                              \
        hipLaunchKernelGGL((mx::moe_gather<U_, US_>), g.grid, g.block, 0, s, a);
    MX_GATHER(16, 16) MX_GATHER(16, 4) MX_GATHER(16, 1)
    MX_GATHER(4, 16) MX_GATHER(4, 4) MX_GATHER(4, 1)
    MX_GATHER(1, 16) MX_GATHER(1, 4) MX_GATHER(1, 1)
#undef MX_GATHER
    return launched();
}

extern "C" int mx_moe_combine(int dtype, int64_t tokens, int64_t top, int64_t width,
                              const int32_t *row_of, const void *Y, int64_t y_rows, int64_t ldy,
                              const float *weights, const void *R, int64_t ldr, void *out,
                              void *stream)
{
    if (!is_dtype(dtype)) return MX_ERR_IN_DTYPE;
    if (!moe_shape(tokens, top) || width < 8 || width % 8 != 0 || width > MX_MAX_K ||
        y_rows < 0 || y_rows > MX_MAX_DIM || !pitch_shape(ldy, width) ||
        (R && !pitch_shape(ldr, width)))
        return MX_ERR_ROW_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!row_of || (y_rows && !Y) || !out) return MX_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(row_of, 4) || !aligned(Y, 16) || !aligned(weights, 4) || !aligned(R, 16) ||
        !aligned(out, 16) || !pitch_aligned(ldy, es) || !pitch_aligned(width, es) ||
        (R && !pitch_aligned(ldr, es)))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    const mx::CombineArgs a{Y, R, weights, row_of, out, tokens, y_rows, ldy, ldr,
                            (int)top, (int)width};
    const WaveGrid g = wave_grid(cdiv(width, 512), tokens);
    if (dtype == MX_IN_FP32)
        hipLaunchKernelGGL(mx::moe_combine<mx::IN_F32>, g.grid, g.block, 0, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL(mx::moe_combine<mx::IN_BF16>, g.grid, g.block, 0, (hipStream_t)stream, a);
    return launched();
}

extern "C" int mx_moe_combine_backward(int dtype, int64_t tokens, int64_t top, int64_t width,
                                       const int32_t *row_of, const void *dOut, int64_t lddo,
                                       const void *Y, int64_t y_rows, int64_t ldy,
                                       const float *weights, void *dY, float *dweights,
                                       void *stream)
{
    if (!is_dtype(dtype)) return MX_ERR_IN_DTYPE;
    if (!moe_shape(tokens, top) || width < 8 || width % 8 != 0 || width > MX_MAX_K ||
        y_rows < 0 || y_rows > tokens * top || !pitch_shape(ldy, width) ||
        !pitch_shape(lddo, width))
        return MX_ERR_ROW_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!row_of || !dOut || (y_rows && (!Y || !dY)) || !weights || !dweights) return MX_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(row_of, 4) || !aligned(Y, 16) || !aligned(weights, 4) || !aligned(dOut, 16) ||
        !aligned(dY, 16) || !aligned(dweights, 4) || !pitch_aligned(ldy, es) ||
        !pitch_aligned(width, es) || !pitch_aligned(lddo, es))
        return MX_ERR_ALIGN;
    int dev = -1;
    const int rc = device_ready(&dev);
    if (rc != MX_OK) return rc;
    (void)hipGetLastError();
    const mx::CombineGradArgs a{dOut, Y, weights, row_of, dY, dweights, tokens, y_rows,
                                lddo, ldy, (int)top, (int)width};
    const WaveGrid g = wave_grid(top, tokens);
    if (dtype == MX_IN_FP32)
        hipLaunchKernelGGL(mx::moe_combine_grad<mx::IN_F32>, g.grid, g.block, 0,
                           (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL(mx::moe_combine_grad<mx::IN_BF16>, g.grid, g.block, 0,
                           (hipStream_t)stream, a);
    return launched();
}
