// Host checks of the row, routing and epilogue operators under the
// sanitizers, without a device (tests/test_sanitize_block_cpu.py): their
// argument checks, plans and workspace sizes over shapes up to the ABI's
// limits, and valid calls, which end at the missing device.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "mxgemm.h"

#define CHECK(x)                                                       \
    do {                                                               \
        if (!(x)) {                                                    \
            std::printf("line %d: %s\n", __LINE__, #x);                \
            std::exit(1);                                              \
        }                                                              \
    } while (0)

int main()
{
    // an address that no call looks at, aligned for every argument
    void *const p = reinterpret_cast<void *>(static_cast<uintptr_t>(1) << 20);
    float *const f = static_cast<float *>(p);
    int32_t *const i32 = static_cast<int32_t *>(p);
    int64_t *const i64 = static_cast<int64_t *>(p);
    const int64_t big = INT64_MAX, huge = (int64_t)1 << 30;
    const int none = MX_ERR_NO_DEVICE;

    for (int64_t rows : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)511, huge, huge + 1, big})
        for (int64_t width : {(int64_t)-32, (int64_t)0, (int64_t)32, (int64_t)48, (int64_t)8192,
                              (int64_t)65536, (int64_t)65568, big}) {
            const bool ok = rows >= 0 && rows <= huge && width >= 32 && width % 32 == 0 && width <= 65536;
            const int64_t ws = mx_rmsnorm_backward_workspace(rows, width);
            CHECK(ok ? ws >= 0 && ws <= 65536 * 4 * 1024 : ws == MX_ERR_ROW_SHAPE);
            const int want = !ok ? MX_ERR_ROW_SHAPE : rows ? none : MX_OK;
            for (int fmt = 1; fmt <= 5; ++fmt)
                for (int dt = 1; dt <= 2; ++dt) {
                    CHECK(mx_rmsnorm_quantize(fmt, dt, 1, rows, width, p, width, p, width, p, 1e-6f, p,
                                              p, p, p, f, nullptr) == want);
                    CHECK(mx_swiglu_quantize(fmt, dt, rows, width, p, ok ? 2 * width : 0, p, p,
                                             nullptr) == want);
                }
            CHECK(mx_rmsnorm_backward(1, 2, rows, width, p, width, p, width, f, p, p, width, p, f, p,
                                      big, nullptr) == (ok ? none : MX_ERR_ROW_SHAPE));
            CHECK(mx_swiglu_backward(2, rows, width, p, width, p, ok ? 2 * width : 0, p, nullptr) == want);
        }
    // pitches up to the limits of 64 bits
    for (int64_t ld : {(int64_t)-1, (int64_t)0, (int64_t)63, big}) {
        CHECK(mx_rmsnorm_quantize(2, 1, 1, 4, 64, p, ld, nullptr, 0, p, 0.f, p, p, p, p, f, nullptr) ==
              MX_ERR_ROW_SHAPE);
        CHECK(mx_moe_combine(2, 4, 2, 64, i32, p, 8, ld, f, nullptr, 0, p, nullptr) == MX_ERR_ROW_SHAPE);
        CHECK(mx_moe_gather(4, 2, i32, p, 64, ld, nullptr, 0, 0, p, nullptr, nullptr) == MX_ERR_ROW_SHAPE);
    }
    for (int64_t tokens : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)100000, huge, huge + 1, big})
        for (int64_t top : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)8, (int64_t)64, (int64_t)65, big}) {
            const bool ok = tokens >= 0 && tokens <= huge && top >= 1 && top <= 64 && tokens * top <= huge;
            for (int64_t experts : {(int64_t)0, (int64_t)1, (int64_t)256, (int64_t)257, big}) {
                const bool fine = ok && experts >= 1 && experts <= 256;
                const int64_t ws = mx_moe_sort_workspace(tokens, top, experts);
                CHECK(fine ? ws >= 0 && ws <= 257 * 257 * 4 : ws == MX_ERR_ROW_SHAPE);
                CHECK(mx_moe_sort(8, tokens, top, experts, p, i64, i32, p, big, nullptr) ==
                      (fine ? none : MX_ERR_ROW_SHAPE));
            }
            const int want = !ok ? MX_ERR_ROW_SHAPE : tokens ? none : MX_OK;
            CHECK(mx_moe_gather(tokens, top, i32, p, 1, 1, p, 1, 1, p, p, nullptr) == want);
            CHECK(mx_moe_gather(tokens, top, i32, p, MX_MAX_K, huge, nullptr, 0, 0, p, nullptr, nullptr) == want);
            CHECK(mx_moe_combine(1, tokens, top, MX_MAX_K, i32, p, huge, huge, f, p, huge, p, nullptr) == want);
            CHECK(mx_moe_combine_backward(2, tokens, top, 8, i32, p, 8, p, 0, 8, f, p, f, nullptr) == want);
        }
    mx_plan_t plan;
    for (int64_t M : {(int64_t)0, (int64_t)1, (int64_t)32, (int64_t)300, huge, huge + 1, big})
        for (int64_t N : {(int64_t)0, (int64_t)1, (int64_t)4099, huge, big})
            for (int64_t K : {(int64_t)0, (int64_t)128, (int64_t)4096, (int64_t)MX_MAX_K, big}) {
                for (int fa = 0; fa <= 6; ++fa)
                    for (int fb = 0; fb <= 6; ++fb) {
                        const int rc = mx_gemm_fused_plan(fa, fb, M, N, K, MX_OUT_BF16, &plan);
                        if (rc == MX_OK) CHECK(plan.workgroups > 0 && plan.workspace_bytes >= 0);
                        const int call = mx_gemm_fused(fa, fb, M, N, K, p, p, p, p, p, MX_IN_FP32,
                                                       MX_ACT_GELU, p, N, p, MX_OUT_BF16, p, big,
                                                       nullptr);
                        CHECK(rc == MX_OK ? call == none : call == rc);
                    }
                const int rc = mx_gemm_bf16_fused_plan(M, N, K, MX_OUT_FP32, &plan);
                const int call = mx_gemm_bf16_fused(M, N, K, p, p, nullptr, 0, MX_ACT_NONE, nullptr, 0,
                                                    p, MX_OUT_FP32, nullptr, 0, nullptr);
                CHECK(rc == MX_OK ? call == none : call == rc);
            }
    for (int code : {MX_ERR_ROW_SHAPE, MX_ERR_WORKSPACE, MX_ERR_ACT}) CHECK(mx_strerror(code)[0] != 'u' || code == MX_ERR_ACT);
    std::printf("block checks passed\n");
    return 0;
}
