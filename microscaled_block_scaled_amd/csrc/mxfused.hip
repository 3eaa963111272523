// mxfused.hip -- launches of the GEMM kernels with the fused epilogue
// (mx_epilogue.h) for the format pairs that mx_gemm_fused takes, in a
// translation unit of their own so that the library builds in parallel.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mx_epilogue.h"
#include "mx_launch.h"

namespace mxhost {

namespace {

template <int FA, int FB, int OUT, int BM, int BN, int WGM, int WGN, int S>
void go_cfg(const void *A, const void *As, const void *B, const void *Bs, void *C, int64_t M,
            int64_t N, int64_t K, int split, float *W, const mx::Epilogue &ep, hipStream_t s)
{
    const int tiles_m = (int)cdiv(M, BM), tiles_n = (int)cdiv(N, BN);
    const int gm = 4;
    const dim3 grid((unsigned)(tiles_m * tiles_n * split)), block(WGM * WGN * 64);
    const uint8_t *a = (const uint8_t *)A, *as = (const uint8_t *)As;
    const uint8_t *b = (const uint8_t *)B, *bs = (const uint8_t *)Bs;
    if (split == 1) {
        hipLaunchKernelGGL((mx::tile_kernel<FA, FB, OUT, BM, BN, WGM, WGN, S, mx::NoGroups,
                                            mx::Epilogue>),
                           grid, block, 0, s, a, as, b, bs, C, (int)M, (int)N, (int)K, tiles_m,
                           tiles_n, gm, (int)K, (int64_t)0, mx::NoGroups{}, ep);
        return;
    }
    // the slices' sums as they are, then the epilogue where they are added
    const int64_t plane = plane_of(M, N);
    hipLaunchKernelGGL((mx::tile_kernel<FA, FB, mx::OF32, BM, BN, WGM, WGN, S, mx::NoGroups,
                                        mx::PlainSums>),
                       grid, block, 0, s, a, as, b, bs, (void *)W, (int)M, (int)N, (int)K,
                       tiles_m, tiles_n, gm, (int)slice_k(K, split), plane, mx::NoGroups{},
                       mx::PlainSums{});
    hipLaunchKernelGGL((mx::splitk_fused<OUT>), dim3((unsigned)cdiv(M * N, 1024)), dim3(256), 0,
                       s, (const float *)W, C, (int)(M * N), (int)N, plane, split, ep);
}

// The tiles of the fused GEMMs: {BM, BN, waves along M, waves along N}, and
// the cost of one tile of theirs in units of a 64 x 64 tile's.  The small
// tiles are for the many products of a block that the 256-row tiles cannot
// spread over the GPU (2944 columns and 257 rows: 46 workgroups of 256 x 128).
struct FusedTile { int bm, bn, wgm, wgn; double cost; };
constexpr FusedTile kFusedTiles[] = {
    {256, 256, 4, 2, 6.0}, {256, 192, 4, 2, 5.3}, {256, 128, 4, 2, 3.9},
    {128, 128, 4, 2, 2.4}, {128, 64, 2, 2, 1.6}, {64, 64, 2, 2, 1.0},
};

template <int FA, int FB, int OUT>
bool go_tile(const mx_plan_t &p, const void *A, const void *As, const void *B, const void *Bs,
             void *C, int64_t M, int64_t N, int64_t K, float *W, const mx::Epilogue &ep,
             hipStream_t s)
{
    // The smallest tile takes the deepest ring that lets two workgroups share
    // a CU: 4 slabs, or 3 where the scale period allows no more (E2M1).
    constexpr int S64 = FA == mx::FP4 ? 3 : 4;
#define MX_CFG(BM_, BN_, WM_, WN_, S_)                                                     \
    if (p.tile_m == BM_ && p.tile_n == BN_) {                                              \
        go_cfg<FA, FB, OUT, BM_, BN_, WM_, WN_, S_>(A, As, B, Bs, C, M, N, K, p.split_k,   \
                                                    W, ep, s);                             \
        return true;                                                                       \
    }
    MX_CFG(256, 256, 4, 2, 2)
    MX_CFG(256, 192, 4, 2, 2)
    MX_CFG(256, 128, 4, 2, 3)
    MX_CFG(128, 128, 4, 2, 3)
    MX_CFG(128, 64, 2, 2, 3)
    MX_CFG(64, 64, 2, 2, S64)
#undef MX_CFG
    return false;
}

template <int FA, int FB, int OUT, int WA>
void go_decode(const void *A, const void *As, const void *B, const void *Bs, void *C, int64_t M,
               int64_t N, int64_t K, const mx::Epilogue &ep, hipStream_t s)
{
    const dim3 grid((unsigned)std::min<int64_t>(cdiv(N, MX_DECODE_TILE), kCUs));
    hipLaunchKernelGGL((mx::fused_decode<FA, FB, OUT, WA>), grid, dim3(mx::kDecodeWaves * 64), 0,
                       s, (const uint8_t *)A, (const uint8_t *)As, (const uint8_t *)B,
                       (const uint8_t *)Bs, C, (int)M, (int)N, (int)K, ep);
}

template <int FA, int FB, int OUT>
bool go(const mx_plan_t &p, const void *A, const void *As, const void *B, const void *Bs,
        void *C, int64_t M, int64_t N, int64_t K, float *W, const mx::Epilogue &ep,
        hipStream_t s)
{
    if constexpr (FA != mx::B16) {
        if (p.variant == MX_VARIANT_DECODE) {
            // A rows staged as in launch_decode
            if constexpr (FB == mx::FP4 && FA != mx::FP4) {
                if (M <= 8) go_decode<FA, FB, OUT, 8>(A, As, B, Bs, C, M, N, K, ep, s);
                else if (M <= 16) go_decode<FA, FB, OUT, 16>(A, As, B, Bs, C, M, N, K, ep, s);
                else go_decode<FA, FB, OUT, 32>(A, As, B, Bs, C, M, N, K, ep, s);
            } else {
                go_decode<FA, FB, OUT, 0>(A, As, B, Bs, C, M, N, K, ep, s);
            }
            return true;
        }
    }
    return go_tile<FA, FB, OUT>(p, A, As, B, Bs, C, M, N, K, W, ep, s);
}

}  // namespace

bool fused_pair(int fmt_a, int fmt_b)
{
    return (fmt_a == MX_FMT_E2M1 && fmt_b == MX_FMT_E2M1) ||
           (fmt_a == MX_FMT_E4M3 && fmt_b == MX_FMT_E4M3) ||
           (fmt_a == MX_FMT_E4M3 && fmt_b == MX_FMT_E2M1) ||
           (fmt_a == kFmtBF16 && fmt_b == kFmtBF16);
}

// The tile and split with the least estimated time.  A CU works through its
// share of the tiles, so the tiles cost ceil(tiles / CUs) * cost per K-value,
// and splitting K adds a second kernel and a round trip of the planes.  The
// costs per tile and the two constants were fitted to times of all tiles and
// splits over 75 shapes (M 20 .. 2048, N 1000 .. 28672, K 1024 .. 28672, each
// with bias and residual, operands rotating) in E4M3, E2M1, E4M3 x E2M1 and
// BF16 on MI355X: the choice takes 1.02 times the best tile and split's time
// (geometric mean; worst 1.28), the unfused plan's choice 1.55 times (worst
// 3.1).  In E4M3 293 x 3443 x 2688 takes 13 us against 26, 453 x 1628 x 1664
// 7.8 against 18.6.
void fused_plan(int fmt_a, int fmt_b, int64_t M, int64_t N, int64_t K, int max_split,
                mx_plan_t *p)
{
    // microseconds of a 64 x 64 tile per 128 K-values
    const double unit = fmt_a == kFmtBF16 ? 0.45 : fmt_a == MX_FMT_E2M1 ? 0.16
                      : fmt_b == MX_FMT_E2M1 ? 0.20 : 0.25;
    double best = -1.0;
    memset(p, 0, sizeof(*p));
    for (const FusedTile &c : kFusedTiles) {
        const int64_t tiles = cdiv(M, c.bm) * cdiv(N, c.bn);
        for (int req = 1; req <= max_split; req *= 2) {
            const int64_t k = slice_k(K, req);
            const int split = req == 1 ? 1 : (int)cdiv(K, k);
            // slices of at least 1024 K, planes and grid within 32-bit indices
            if (req > 1 && (split < 2 || k < 1024 || M * N >= ((int64_t)1 << 30))) break;
            double t = (double)cdiv(tiles * split, kCUs) * c.cost * unit *
                       (double)(split > 1 ? k : K) / 128.0;
            if (split > 1) t += 3.5 + 2.3e-6 * (double)(M * N * split);
            // a launch has less than 2^32 threads, and 2^24 tiles of 64 columns
            // (N = 2^30) have that many: such a grid only where all are
            if (tiles * split * c.wgm * c.wgn * 64 >= (int64_t)1 << 32) t *= 1e9;
            if (best >= 0.0 && t >= best) continue;
            best = t;
            p->variant = MX_VARIANT_TILE;
            p->tile_m = c.bm;
            p->tile_n = c.bn;
            p->split_k = split;
            p->threads = c.wgm * c.wgn * 64;
            p->workgroups = tiles * split;
            p->workspace_bytes = split > 1 ? split * plane_of(M, N) * 4 : 0;
        }
    }
}

bool launch_fused(int fmt_a, int fmt_b, const mx_plan_t &p, int out_dtype, const void *A,
                  const void *As, const void *B, const void *Bs, void *C, int64_t M, int64_t N,
                  int64_t K, float *W, const mx::Epilogue &ep, hipStream_t s)
{
    const bool f32 = out_dtype == MX_OUT_FP32;
#define MX_GO(FA_, FB_)                                                                    \
    return f32 ? go<FA_, FB_, mx::OF32>(p, A, As, B, Bs, C, M, N, K, W, ep, s)             \
               : go<FA_, FB_, mx::OBF16>(p, A, As, B, Bs, C, M, N, K, W, ep, s);
    if (fmt_a == kFmtBF16) MX_GO(mx::B16, mx::B16)
    if (fmt_a == MX_FMT_E2M1) MX_GO(mx::FP4, mx::FP4)
    if (fmt_b == MX_FMT_E2M1) MX_GO(mx::FP8, mx::FP4)
    MX_GO(mx::FP8, mx::FP8)
#undef MX_GO
}

}  // namespace mxhost
