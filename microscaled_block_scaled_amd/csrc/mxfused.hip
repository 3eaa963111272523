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
    hipLaunchKernelGGL((mx::tile_kernel<FA, FB, mx::OF32, BM, BN, WGM, WGN, S>), grid, block, 0,
                       s, a, as, b, bs, (void *)W, (int)M, (int)N, (int)K, tiles_m, tiles_n, gm,
                       (int)slice_k(K, split), plane);
    hipLaunchKernelGGL((mx::splitk_fused<OUT>), dim3((unsigned)cdiv(M * N, 1024)), dim3(256), 0,
                       s, (const float *)W, C, (int)(M * N), (int)N, plane, split, ep);
}

template <int FA, int FB, int OUT>
bool go_tile(const mx_plan_t &p, const void *A, const void *As, const void *B, const void *Bs,
             void *C, int64_t M, int64_t N, int64_t K, float *W, const mx::Epilogue &ep,
             hipStream_t s)
{
#define MX_CFG(BM_, BN_, WM_, WN_, S_)                                                     \
    if (p.tile_m == BM_ && p.tile_n == BN_ && p.threads == WM_ * WN_ * 64) {              \
        go_cfg<FA, FB, OUT, BM_, BN_, WM_, WN_, S_>(A, As, B, Bs, C, M, N, K, p.split_k,   \
                                                    W, ep, s);                             \
        return true;                                                                       \
    }
    MX_CFG(256, 256, 4, 2, 2)
    MX_CFG(256, 192, 4, 2, 2)
    MX_CFG(256, 160, 4, 1, 2)
    MX_CFG(256, 128, 4, 2, 3)
    MX_CFG(128, 128, 2, 2, 3)
    MX_CFG(64, 256, 1, 8, 3)
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
