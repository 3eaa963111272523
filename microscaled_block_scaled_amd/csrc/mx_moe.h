// mx_moe.h -- gfx950 device code of expert routing around the grouped GEMM:
// (token, choice) pairs sorted by expert, token rows gathered into expert
// order, expert rows combined back with weights, and the gradient of the
// combination.
//
// Pair i = token * top + choice.  The sort is stable: an expert's rows are in
// the order of their pairs, so nothing depends on timing.  row_of[i] is pair
// i's row in expert order; a pair whose id is no expert (a padding token, a
// dropped choice) comes after all experts, at row r, and has row_of = -1 - r.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_math.h"
#include "mx_rowops.h"

namespace mx {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBins = kMaxGroups + 1;       // the experts, and no expert
constexpr int kSortParts = kSortThreads / 256;  // threads that share a bin's counts

struct SortArgs {
    const void *ids;
    int64_t *group_rows;
    int32_t *row_of;
    int32_t *counts;             // chunks x bins: pairs of each bin in each chunk
    int64_t n, chunk;            // pairs, and pairs per workgroup (a multiple of kSortThreads)
    int experts, id64;
};

// Bin of pair i (i < n): its expert, or `experts` for none.
__device__ __forceinline__ int sort_bin(const SortArgs &a, int64_t i)
{
    const int64_t id = a.id64 ? ((const int64_t *)a.ids)[i] : (int64_t)((const int32_t *)a.ids)[i];
    return id >= 0 && id < a.experts ? (int)id : a.experts;
}

// The lanes of the wave that hold the same bin as this lane (dead lanes
// match nobody): one ballot per bit of the bin number.
__device__ __forceinline__ uint64_t same_bin(int bin, bool live, int bits)
{
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (bin >> b) & 1;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

// Adds this wave's share of the workgroup's chunk, a run of chunk / 16
// consecutive pairs, to its row of per-wave bin counts in LDS.
__device__ __forceinline__ void sort_count(const SortArgs &a, int (*cnt)[kSortBins + 1], int bits)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSortWaves * (kSortBins + 1); i += kSortThreads)
        ((int *)cnt)[i] = 0;
    __syncthreads();
    const int64_t per = a.chunk / kSortWaves;
    const int64_t lo = blockIdx.x * a.chunk + wave * per, hi = min(lo + per, a.n);
    for (int64_t i = lo + lane; i - lane < hi; i += 64) {
        const bool live = i < hi;
        const int bin = live ? sort_bin(a, i) : 0;
        const uint64_t m = same_bin(bin, live, bits);
        if (live && (m & ((1ull << lane) - 1)) == 0) cnt[wave][bin] += __popcll(m);
        wave_fence();
    }
    __syncthreads();
}

// First of two launches for many pairs: the bin counts of each chunk.  131072
// pairs of 256 experts: 4.7 us, and 7.6 us for the sort after it.
__global__ void __launch_bounds__(kSortThreads)
moe_count(SortArgs a)
{
    __shared__ int cnt[kSortWaves][kSortBins + 1];
    sort_count(a, cnt, 32 - __clz(a.experts));
    const int bins = a.experts + 1;
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        int t = 0;
        for (int w = 0; w < kSortWaves; ++w) t += cnt[w][b];
        a.counts[(int64_t)blockIdx.x * bins + b] = t;
    }
}

// A counting sort: the first row of every (bin, chunk, wave) is the number
// of pairs before it in that order; each wave then walks its run of pairs,
// 64 at a time, and a pair's row is its wave's next row of the bin plus the
// earlier lanes of the same bin.  MANY: one workgroup per chunk, the other
// chunks' counts from moe_count; otherwise the one workgroup has them all.
template <bool MANY>
__global__ void __launch_bounds__(kSortThreads)
moe_sort(SortArgs a)
{
    __shared__ int cnt[kSortWaves][kSortBins + 1];
    __shared__ int sums[2][kSortParts][kSortBins];           // in all, in earlier chunks
    __shared__ int wave_total[kSortThreads / 64];
    const int bits = 32 - __clz(a.experts), bins = a.experts + 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    sort_count(a, cnt, bits);
    // Each bin's pairs: kSortParts threads per bin take every kSortParts-th
    // chunk (or wave), so that few loads follow one another.
    {
        const int part = tid / 256;
        for (int b = tid % 256; b < bins; b += 256) {
            int total = 0, before = 0;
            if constexpr (MANY) {
#pragma unroll 16
                for (int c = part; c < (int)gridDim.x; c += kSortParts) {
                    const int v = a.counts[(int64_t)c * bins + b];
                    total += v;
                    before += c < (int)blockIdx.x ? v : 0;
                }
            } else {
                for (int w = part; w < kSortWaves; w += kSortParts) total += cnt[w][b];
            }
            sums[0][part][b] = total;
            sums[1][part][b] = before;
        }
    }
    __syncthreads();
    int before = 0, total = 0;
    if (tid < bins) {
#pragma unroll
        for (int p = 0; p < kSortParts; ++p) {
            total += sums[0][p][tid];
            before += sums[1][p][tid];
        }
        if (blockIdx.x == 0 && tid < a.experts) a.group_rows[tid] = total;
    }
    // first row of each bin: sums over the earlier bins, a wave at a time
    int upto = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    if (tid < bins) {
        int at = upto - total + before;
        for (int w = 0; w < wave; ++w) at += wave_total[w];
        for (int w = 0; w < kSortWaves; ++w) {
            const int v = cnt[w][tid];
            cnt[w][tid] = at;
            at += v;
        }
    }
    __syncthreads();
    const int64_t per = a.chunk / kSortWaves;
    const int64_t lo = blockIdx.x * a.chunk + wave * per, hi = min(lo + per, a.n);
    for (int64_t i = lo + lane; i - lane < hi; i += 64) {
        const bool live = i < hi;
        const int bin = live ? sort_bin(a, i) : 0;
        const uint64_t m = same_bin(bin, live, bits);
        const int ahead = __popcll(m & ((1ull << lane) - 1));
        const int row = live ? cnt[wave][bin] + ahead : 0;
        // every lane has read its bin's next row before its first lane moves it
        wave_fence();
        if (live && ahead == 0) cnt[wave][bin] += __popcll(m);
        wave_fence();
        if (live) a.row_of[i] = bin == a.experts ? -1 - row : row;
    }
}

// Rows of x (row_bytes each, and scale_bytes of scales) copied to the rows of
// their pairs; rows of pairs without an expert are filled with zeros.  Each
// token row is read once and written `top` times.  A wave takes 64 units of
// U bytes of a token's row (wave `seg` of the row's waves, the scales' after
// the row's), for the tokens blockIdx.y, blockIdx.y + gridDim.y, ...
struct GatherArgs {
    const uint8_t *x, *s;
    uint8_t *xs, *ss;
    const int32_t *row_of;
    int64_t tokens, n, ldx, lds;                 // n: pairs; pitches in bytes
    int top, row_bytes, scale_bytes;
    int row_segs, segs;                          // waves per token: rows, and rows + scales
};

template <int U> struct unit;
template <> struct unit<16> { typedef v4i t; };
template <> struct unit<4> { typedef int t; };
template <> struct unit<1> { typedef uint8_t t; };

template <int U>
__device__ __forceinline__ void gather_seg(const uint8_t *src, uint8_t *dst, int bytes, int at,
                                           const int32_t *row_of, int top, int64_t n)
{
    typedef typename unit<U>::t T;
    if (at >= bytes) return;
    const T v = *(const T *)(src + at);
    for (int j = 0; j < top; ++j) {
        const int r = row_of[j];
        const int64_t to = r < 0 ? -1 - (int64_t)r : r;
        if (to >= n) continue;
        __builtin_nontemporal_store(r < 0 ? T{} : v, (T *)(dst + to * bytes + at));
    }
}

// This wave's number among all waves along x.
__device__ __forceinline__ int wave_x()
{
    return blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// Bound by the writes to HBM: 16384 tokens to 8 rows of 4096 bytes each 108
// us, 5.1 TB/s written.
template <int U, int US>
__global__ void __launch_bounds__(512)
moe_gather(GatherArgs a)
{
    const int lane = threadIdx.x & 63, seg = wave_x();
    if (seg >= a.segs) return;
    for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
        const int32_t *row_of = a.row_of + t * a.top;
        if (seg < a.row_segs)
            gather_seg<U>(a.x + t * a.ldx, a.xs, a.row_bytes, (seg * 64 + lane) * U, row_of,
                          a.top, a.n);
        else
            gather_seg<US>(a.s + t * a.lds, a.ss, a.scale_bytes,
                           ((seg - a.row_segs) * 64 + lane) * US, row_of, a.top, a.n);
    }
}

// out[t] = r[t] + sum over choices j, in order, of w[t][j] * y[row_of[t][j]];
// pairs without an expert add nothing and nothing of theirs is read.  Without
// weights each counts 1, which is the gradient of the gather.  A wave takes
// 512 columns, four choices' loads at a time.  Bound by HBM: 8192 tokens of 4
// BF16 rows of 4096 with residual 68 us a call, 5.9 TB/s.
struct CombineArgs {
    const void *y, *r;
    const float *w;
    const int32_t *row_of;
    void *out;
    int64_t tokens, rows, ldy, ldr;              // rows of y; pitches in elements
    int top, width;
};

template <int IN>
__global__ void __launch_bounds__(512)
moe_combine(CombineArgs a)
{
    const int col = (wave_x() * 64 + (threadIdx.x & 63)) * 8;
    if (col >= a.width) return;
    for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
        const int32_t *row_of = a.row_of + t * a.top;
        const float *w = a.w ? a.w + t * a.top : nullptr;
        raw8<IN> rv;
        if (a.r) rv = load8<IN, true>(a.r, t * a.ldr + col);
        float acc[8] = {};
        for (int j0 = 0; j0 < a.top; j0 += 4) {
            raw8<IN> yv[4];
            bool live[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j0 + j < a.top ? row_of[j0 + j] : -1;
                live[j] = r >= 0 && r < a.rows;
                if (live[j]) yv[j] = load8<IN, true>(a.y, r * a.ldy + col);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!live[j]) continue;
                const float wj = w ? w[j0 + j] : 1.f;
                float v[8];
                unpack8<IN>(yv[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(v[i], wj, acc[i]);
            }
        }
        if (a.r) {
            float v[8];
            unpack8<IN>(rv, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
        }
        store8<IN>(a.out, t * a.width + col, pack8<IN>(acc));
    }
}

// Gradient of the combination: dy[row_of[t][j]] = w[t][j] * dout[t] (zeros in
// the rows of pairs without an expert) and dw[t][j] = <dout[t], y[row]> (0
// without an expert).  A wave takes one choice of a token, whole rows; the
// waves of a workgroup share the token's dout row through the caches.  Bound
// by HBM: 4095 tokens of 4 BF16 rows of 4096 56 us a call, 5.4 TB/s.
struct CombineGradArgs {
    const void *dout, *y;
    const float *w;
    const int32_t *row_of;
    void *dy;
    float *dw;
    int64_t tokens, rows, lddo, ldy;
    int top, width;
};

template <int IN>
__global__ void __launch_bounds__(512)
moe_combine_grad(CombineGradArgs a)
{
    const int lane = threadIdx.x & 63, j = wave_x();
    if (j >= a.top) return;
    for (int64_t t = blockIdx.y; t < a.tokens; t += gridDim.y) {
        const int64_t i = t * a.top + j;
        const int r = a.row_of[i];
        const int64_t to = r < 0 ? -1 - (int64_t)r : r;
        float dot = 0.f;
        if (to >= a.rows) {
            // a row that y leaves out: no expert
        } else if (r < 0) {
            for (int col = lane * 8; col < a.width; col += 512)
                store8<IN>(a.dy, to * a.width + col, raw8<IN>{});
        } else {
            const float w = a.w[i];
#pragma unroll 2
            for (int col = lane * 8; col < a.width; col += 512) {
                float d[8], v[8];
                unpack8<IN>(load8<IN>(a.dout, t * a.lddo + col), d);
                unpack8<IN>(load8<IN, true>(a.y, to * a.ldy + col), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot = fmaf(d[e], v[e], dot);
                    d[e] *= w;
                }
                store8<IN>(a.dy, to * a.width + col, pack8<IN>(d));
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) a.dw[i] = dot;
    }
}

}  // namespace mx
