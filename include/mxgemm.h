/*
 * mxgemm.h -- C ABI of the MI355X (gfx950) MX block-scaled NT GEMM, its
 * grouped (mixture-of-experts) form, MX quantization, and a dense BF16 GEMM
 * on the same kernels.
 *
 * The operation (FlyDSL summary pages, section "API compatibility is not
 * universal input coverage"; AI-compiler digest 2026-10-22, item 1
 * "Accelerating PyTorch on AMD GPUs with FlyDSL": MXFP8 / MXFP4 scaled GEMM,
 * BlockWise1x32, E8M0 scale, FP32 accumulation, K a multiple of 128):
 *
 *   C[m][n] = sum_b 2^(sA[m][b] + sB[n][b] - 254)
 *                   * sum_{j<32} A[m][32b+j] * B[n][32b+j]
 *
 * for m < M, n < N, b < K/32, with A and B holding MXFP4 (E2M1) or MXFP8
 * (E4M3) elements and sA, sB their E8M0 scale bytes.  Products and sums are
 * accumulated in FP32; C is written as FP32 or as BF16 (round to nearest
 * even).  The element and scale encodings are those of the OCP Microscaling
 * (MX) v1.0 specification.
 *
 * Memory layout (all dense, row-major, device memory owned by the caller):
 *   A        M x K   elements, K-contiguous.  E4M3: M x K bytes, element k in
 *            byte k.  E2M1: M x K/2 bytes, element 2i in the low nibble of
 *            byte i, element 2i+1 in the high nibble.
 *   B        N x K   elements, K-contiguous, same encoding as A ("NT": C is
 *            A times B transposed).
 *   A_scale  M x K/32 bytes; byte [m][b] scales K-values 32b .. 32b+31 of row m.
 *   B_scale  N x K/32 bytes; likewise for B.
 *   C        M x N  float or bfloat16 (uint16 bit pattern), row pitch N.
 * There are no stride arguments: callers with other layouts must copy.
 *
 * Errors.  Every argument check runs before any HIP call; a failed check
 * returns a negative MX_ERR_* code and touches nothing.  Launch failures are
 * reported as MX_ERR_LAUNCH.  No function aborts or throws.
 *
 * Asynchrony.  mx_gemm enqueues its kernels on `stream` (a hipStream_t;
 * NULL means the device's null stream) and returns without synchronising:
 * C is ready when the stream reaches that point.  Inputs must stay alive and
 * unmodified until then.  C must not overlap any input.  Results are
 * bit-for-bit deterministic for a given (M, N, K, formats, device).
 *
 * Thread safety.  Calls may be made concurrently from several host threads
 * and streams.  The library keeps read-only per-device state, set up once per
 * device on first use, and, for split-K calls (see mx_plan_t), one workspace
 * per (device, stream handle).  Lifetime of a workspace: it is allocated on
 * that stream with hipMallocAsync the first time a call there needs one,
 * replaced (freed and reallocated on the stream) when a call needs more, and
 * otherwise held, at the largest size a call on that stream has needed,
 * until the process exits -- destroying the stream does not free it.  Calls
 * on one stream are ordered by the stream; calls on different streams use
 * different workspaces; split-K calls on one stream from several host threads
 * are serialised while they are enqueued.  One precondition follows: a
 * stream must have finished its split-K calls (hipStreamSynchronize) before
 * it is destroyed, because a stream created later may receive the same
 * handle and would then share that workspace with the still-running calls.
 */
#ifndef MXGEMM_H
#define MXGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element formats: MXFP4 = E2M1; MXFP8 = E4M3, or its other OCP encoding
 * E5M2 (wider range: 2^-16 .. 57344, with infinities and NaNs); MXFP6 =
 * E2M3 (largest 7.5) or E3M2 (largest 28), no infinities or NaNs.  E5M2 is
 * accepted, like the FP6 formats, by mx_gemm, mx_gemm_tile, mx_gemm_mixed
 * (paired with any format), the grouped GEMMs (any pair) and mx_quantize.
 * FP6 rows are K*3/4 bytes: a little-endian bit string with element k in
 * bits 6k .. 6k+5 (bit b is bit b % 8 of byte b / 8), four elements in
 * three bytes (OCP MX v1.0 fixes the element encoding; this packing is this
 * library's). */
enum { MX_FMT_E2M1 = 1, MX_FMT_E4M3 = 2, MX_FMT_E5M2 = 3, MX_FMT_E2M3 = 4, MX_FMT_E3M2 = 5 };

/* Output element types. */
enum { MX_OUT_FP32 = 1, MX_OUT_BF16 = 2 };

/* Return codes. */
enum {
    MX_OK = 0,
    MX_ERR_FORMAT = -1,     /* unknown format, or one this call does not take */
    MX_ERR_OUT_DTYPE = -2,  /* out_dtype is not MX_OUT_FP32 / MX_OUT_BF16     */
    MX_ERR_SHAPE = -3,      /* M < 1, N < 1, K < 128, K % 128 != 0, M or N
                               above MX_MAX_DIM, K above MX_MAX_K, or more
                               than 2^31 - 1 workgroups of tiles needed        */
    MX_ERR_NULL = -4,       /* a required pointer is NULL                     */
    MX_ERR_ALIGN = -5,      /* A, B or C not 16-byte aligned, or a scale
                               array not 4-byte aligned                        */
    MX_ERR_NO_DEVICE = -6,  /* no HIP device is visible                       */
    MX_ERR_ARCH = -7,       /* the current device is not gfx950               */
    MX_ERR_ALLOC = -8,      /* split-K workspace allocation failed            */
    MX_ERR_LAUNCH = -9,     /* a kernel launch failed                         */
    MX_ERR_IN_DTYPE = -10,  /* in_dtype is not MX_IN_FP32 / MX_IN_BF16       */
    MX_ERR_SCRATCH = -11,   /* mx_gemm_noalloc: the problem's split-K workspace
                               exceeds MX_NOALLOC_SCRATCH_BYTES               */
    MX_ERR_ROW_SHAPE = -12, /* a size or pitch a row, routing or epilogue
                               operator does not take                         */
    MX_ERR_WORKSPACE = -13, /* the caller's workspace is too small             */
    MX_ERR_ACT = -14        /* act is not an MX_ACT_* code                     */
};

/* Input element types of mx_quantize. */
enum { MX_IN_FP32 = 1, MX_IN_BF16 = 2 };

/* Largest M or N accepted (keeps every tile index in 32 bits). */
#define MX_MAX_DIM ((int64_t)1 << 30)
/* Largest K accepted (keeps a tile's per-lane copy offsets, up to 256 rows of
 * one operand, within 32 bits). */
#define MX_MAX_K ((int64_t)1 << 24)

/*
 * C = A * B^T with MX block scaling, enqueued on `stream`.
 *   fmt        any MX_FMT_* code (A and B share the format; mx_gemm_mixed
 *              takes one per operand)
 *   M, N, K    sizes; K a multiple of 128, at most MX_MAX_K
 *   A, B       packed elements (layout above), 16-byte aligned device pointers
 *   A_scale,
 *   B_scale    E8M0 scale bytes (layout above), 4-byte aligned
 *   C          output, 16-byte aligned; float if out_dtype == MX_OUT_FP32,
 *              bfloat16 bits if MX_OUT_BF16
 *   stream     hipStream_t, or NULL
 * Returns MX_OK or a negative MX_ERR_* code.
 */
int mx_gemm(int fmt, int64_t M, int64_t N, int64_t K,
            const void *A, const void *A_scale,
            const void *B, const void *B_scale,
            void *C, int out_dtype, void *stream);

/* Static, NUL-terminated description of a return code. */
const char *mx_strerror(int code);

/*
 * Kernel variants a plan can choose.
 * MX_VARIANT_TILE: the tiled kernel, in which each workgroup computes one
 *   tile_m x tile_n tile of C, staging A and B through LDS.  Small M uses a
 *   128- or 64-row tile.  When the tiles cannot fill the GPU and K is long,
 *   each workgroup takes one of split_k K-slices and writes FP32 partial
 *   results to a workspace that a second kernel adds in slice order
 *   (workspace_bytes of the stream's workspace, see "Thread safety" above;
 *   mx_gemm_noalloc uses a fixed scratch instead).
 * MX_VARIANT_DECODE: the decode kernel, for M <= MX_DECODE_TILE rows with
 *   both operands E2M1, E4M3 or E5M2 and K >= 512.  C is cut into groups
 *   of MX_DECODE_TILE columns (all M rows); workgroups = min(groups, 256),
 *   at most one per CU, and workgroup b computes groups b, b + workgroups,
 *   ...; its four waves take four K-ranges of whole 512-K periods and add
 *   their partial sums in LDS in a fixed order.  tile_m = tile_n =
 *   MX_DECODE_TILE, split_k = 1, no workspace.  The plan takes it where it streams B faster than the tiled
 *   kernel; mx_gemm_tile and mx_gemm_mixed run it when asked for the tile
 *   (MX_DECODE_TILE, MX_DECODE_TILE).
 */
enum { MX_VARIANT_TILE = 1, MX_VARIANT_DECODE = 2 };
#define MX_DECODE_TILE 32

/* How mx_gemm would run a problem (filled by mx_gemm_plan). */
typedef struct {
    int variant;            /* MX_VARIANT_*                                   */
    int tile_m, tile_n;     /* output tile of one workgroup                   */
    int split_k;            /* K slices per output tile (1 = none); they are
                               added in a fixed order, never with atomics       */
    int threads;            /* threads per workgroup                          */
    int lds_bytes;          /* dynamic LDS per workgroup                      */
    int64_t workgroups;     /* workgroups in the main launch                  */
    int64_t workspace_bytes;/* split-K workspace the call uses (0 = none)     */
} mx_plan_t;

/*
 * Fill *plan with the launch mx_gemm would make for these arguments.  Pure
 * host logic: it makes no HIP call and does not need a device.  Returns
 * MX_OK, or the same argument error mx_gemm would return.
 */
int mx_gemm_plan(int fmt, int64_t M, int64_t N, int64_t K, int out_dtype,
                 mx_plan_t *plan);

/*
 * mx_gemm for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, plan, kernels, errors and results (bit for bit) as mx_gemm;
 * the only difference is where a split-K call keeps its FP32 partial planes.
 * Instead of allocating them, it uses a fixed scratch array in device memory
 * of MX_NOALLOC_SCRATCH_BYTES, one per device, which the library holds from
 * its first call on that device until the process ends.  It calls no
 * allocator at all (no hipMalloc, hipMallocAsync, hipFree or library routine
 * that allocates).
 *   Returns MX_ERR_SCRATCH, before any HIP call, when the plan's
 *   workspace_bytes (mx_gemm_plan) exceeds MX_NOALLOC_SCRATCH_BYTES: e.g.
 *   M = 256, N = 8192, K = 28672 (4 K-slices) needs exactly 32 MiB and runs;
 *   M = 512, N = 6144, K = 28672 (4 slices of 12 MiB) is refused.  Problems
 *   the plan does not split need no scratch and have no limit.
 * Every call on one device shares that device's scratch, and it keeps what
 * the last call wrote (each split-K call writes every element it reads, so
 * nothing needs clearing): two calls that overlap in time on one device --
 * on different streams, or from different host threads without stream
 * ordering between them -- race on it and may return wrong results.
 */
#define MX_NOALLOC_SCRATCH_BYTES ((int64_t)32 << 20)
int mx_gemm_noalloc(int fmt, int64_t M, int64_t N, int64_t K,
                    const void *A, const void *A_scale,
                    const void *B, const void *B_scale,
                    void *C, int out_dtype, void *stream);

/*
 * Test hook: the next `count` calls of mx_gemm and its variants that need a
 * split-K workspace fail as if obtaining it had failed: they return
 * MX_ERR_ALLOC and launch nothing.  count <= 0 clears it.  For exercising
 * the MX_ERR_ALLOC path only.
 */
void mx_debug_fail_allocations(int count);

/*
 * The output tile shapes the library has kernels for.  Writes up to
 * max_pairs (tile_m, tile_n) pairs to pairs[2i], pairs[2i+1] (pairs may be
 * NULL) and returns how many shapes there are.  Host logic only.
 */
int mx_tile_shapes(int *pairs, int max_pairs);

/*
 * mx_gemm on the tile kernel with the output tile (and K split) chosen by the
 * caller instead of the plan: (tile_m, tile_n) must be one of the shapes
 * mx_tile_shapes lists, and split_k is 0 (the plan's choice) or 1 ..
 * MX_MAX_SPLIT_K (K is then cut into that many slices of whole 512-K
 * periods, or fewer when K is short); otherwise MX_ERR_SHAPE.  The tile
 * (MX_DECODE_TILE, MX_DECODE_TILE) runs the decode kernel (MX_VARIANT_DECODE)
 * instead: it needs fmt E2M1, E4M3 or E5M2, M <= MX_DECODE_TILE, K >= 512 and
 * split_k 0 or 1, else MX_ERR_SHAPE.  Everything else -- arguments, layouts,
 * errors, results -- is as for mx_gemm.  It exists so that every kernel
 * configuration can be exercised (and timed) on any problem size.
 */
#define MX_MAX_SPLIT_K 8
int mx_gemm_tile(int fmt, int64_t M, int64_t N, int64_t K,
                 const void *A, const void *A_scale,
                 const void *B, const void *B_scale,
                 void *C, int out_dtype, int tile_m, int tile_n, int split_k,
                 void *stream);

/*
 * MX quantization, the step that produces mx_gemm's operands: X (rows x K,
 * FP32 or BF16, K-contiguous) -> Q and Q_scale in the layouts described
 * above for A and A_scale.  The rule is the OCP Microscaling v1.0
 * conversion (the FlyDSL article times its scaled GEMMs from operands
 * already in this form, section "Performance numbers need their
 * baselines"); per block of 32 consecutive values x along K:
 *   X = floor(log2 max|x|) - emax      (emax = 2 for E2M1, 8 for E4M3,
 *                                       15 for E5M2, 2 for E2M3, 4 for E3M2)
 *   scale byte = X + 127, clamped to [0, 254]; 0 for an all-zero block
 *   element    = x * 2^(127 - scale byte) rounded to the nearest element
 *                value (ties to the code with an even last bit), magnitudes
 *                above 6 (E2M1) / 448 (E4M3) / 57344 (E5M2) / 7.5 (E2M3) /
 *                28 (E3M2) saturating,
 *                sign kept
 *   a block holding a NaN or an infinity: scale byte 255, element codes 0.
 *   fmt        any MX_FMT_* code
 *   in_dtype   MX_IN_FP32 or MX_IN_BF16
 *   rows, K    rows >= 1, K >= 32, K % 32 == 0, both <= MX_MAX_DIM
 *   X          device pointer, 16-byte aligned
 *   Q          device pointer, 8-byte aligned: rows x K bytes (E4M3, E5M2)
 *              or rows x K/2 bytes (E2M1, element 2i in the low nibble)
 *              or rows x 3K/4 bytes (E2M3, E3M2, the FP6 bit string)
 *   Q_scale    device pointer: rows x K/32 bytes
 *   stream     hipStream_t, or NULL
 * Returns MX_OK or a negative MX_ERR_* code; errors and asynchrony as for
 * mx_gemm.  Outputs must not overlap X.
 */
int mx_quantize(int fmt, int in_dtype, int64_t rows, int64_t K,
                const void *X, void *Q, void *Q_scale, void *stream);

/*
 * MX GEMM with A and B in different element formats: fmt_a for A, fmt_b for
 * B, each any MX_FMT_* code, in any pair (A E4M3 with B E2M1 is the usual
 * "W4A8" serving layout; E4M3 with E5M2 pairs the two MXFP8 encodings; FP6
 * pairs with the 4- and 8-bit formats and with the other FP6 format).  The
 * block dot product is the one of mx_gemm with
 * each operand decoded in its own format (the OCP MX v1.0 dot product does
 * not require equal formats; the pages' "broader low precision" outlook, and
 * gfx950's scaled MFMA takes a format per operand).  A is M x K in fmt_a's
 * layout (K, K/2 or 3K/4 bytes per row), B is N x K in fmt_b's; scales, C, the
 * output types, alignment, errors and asynchrony as for mx_gemm.
 * tile_m = tile_n = 0 takes the plan's tile (the plan depends on M, N and K,
 * and on whether both formats are E2M1, E4M3 or E5M2, which the decode
 * kernel needs: mx_gemm_plan with either format describes it when both are,
 * and with an FP6 format when one is); otherwise (tile_m, tile_n) must be
 * one of mx_tile_shapes, or the decode tile under mx_gemm_tile's conditions.
 * split_k as for mx_gemm_tile (0: the plan's).  With fmt_a == fmt_b the
 * result equals mx_gemm's / mx_gemm_tile's bit for bit.
 */
int mx_gemm_mixed(int fmt_a, int fmt_b, int64_t M, int64_t N, int64_t K,
                  const void *A, const void *A_scale,
                  const void *B, const void *B_scale,
                  void *C, int out_dtype, int tile_m, int tile_n, int split_k,
                  void *stream);

/*
 * Dense BF16 NT GEMM, C = A * B^T with no scales:
 *   C[m][n] = sum_{k<K} A[m][k] * B[n][k]
 * accumulated in FP32 -- the FlyDSL article's second GEMM workload (dense
 * BF16 GEMMs, section "Performance numbers need their baselines").  It runs
 * on the same tile kernels as mx_gemm, on gfx950's BF16 matrix instruction.
 *   M, N, K    M, N >= 1 and <= MX_MAX_DIM; K >= 16, K % 16 == 0,
 *              K <= MX_MAX_K_BF16
 *   A          M x K bfloat16 values (16-bit patterns), K-contiguous, row
 *              pitch K; 16-byte aligned device pointer
 *   B          N x K bfloat16 values, likewise ("NT": C is A times B
 *              transposed)
 *   C          output, 16-byte aligned; float if out_dtype == MX_OUT_FP32,
 *              bfloat16 bits (round to nearest even) if MX_OUT_BF16
 *   tile_m, tile_n, split_k  as for mx_gemm_mixed: 0, 0, 0 takes the plan's
 *              choice (mx_gemm_bf16_plan describes it), otherwise one of
 *              mx_tile_shapes and 0 .. MX_MAX_SPLIT_K slices of whole 512-K
 *              periods
 *   stream     hipStream_t, or NULL
 * Returns MX_OK or a negative MX_ERR_* code.  Errors, asynchrony, the
 * split-K workspace and determinism are as for mx_gemm; C must not overlap
 * A or B.
 */
#define MX_MAX_K_BF16 ((int64_t)1 << 23)
int mx_gemm_bf16(int64_t M, int64_t N, int64_t K, const void *A, const void *B,
                 void *C, int out_dtype, int tile_m, int tile_n, int split_k,
                 void *stream);

/*
 * The launch mx_gemm_bf16 would make with tile and split 0.  Host logic only:
 * no HIP call, no device needed.  Returns MX_OK or mx_gemm_bf16's argument
 * error (MX_ERR_NULL for a NULL plan).
 */
int mx_gemm_bf16_plan(int64_t M, int64_t N, int64_t K, int out_dtype, mx_plan_t *plan);

/* Largest number of groups of mx_gemm_grouped. */
#define MX_MAX_GROUPS 256

/*
 * Grouped MX GEMM, as in a mixture-of-experts layer (the FlyDSL article's
 * grouped-GEMM cases, section "Performance numbers need their baselines":
 * uniform groups, changing projection sizes, uneven expert loads): group g
 * multiplies its group_rows[g] rows of A by its own N x K weight B_g,
 *   C_g = A_g * B_g^T  for g = 0 .. groups-1,
 * each exactly as mx_gemm would.
 *   groups       1 .. MX_MAX_GROUPS
 *   group_rows   HOST array of `groups` row counts, each >= 0 (0 allowed)
 *   A, A_scale   the groups' rows stacked in group order: (sum of
 *                group_rows) rows, laid out as mx_gemm's A / A_scale
 *   B, B_scale   the groups' weights stacked: groups * N rows, laid out as
 *                mx_gemm's B / B_scale (weight g is rows g*N .. g*N+N-1)
 *   C            (sum of group_rows) x N, rows in the order of A's rows
 * N, K, formats, alignment, errors and asynchrony as for mx_gemm (checked
 * with M = the total row count); groups * N must not exceed MX_MAX_DIM.
 * With no rows at all it returns MX_OK at once: nothing is launched and no
 * pointer is looked at.  No workspace is used.
 */
int mx_gemm_grouped(int fmt, int64_t groups, const int64_t *group_rows,
                    int64_t N, int64_t K, const void *A, const void *A_scale,
                    const void *B, const void *B_scale, void *C, int out_dtype,
                    void *stream);

/*
 * mx_gemm_grouped with the weights in their own format: A (and A_scale) in
 * fmt_a, every B_g (and B_scale) in fmt_b: the pairs mx_gemm_mixed takes
 * (any two MX formats; E4M3
 * activations with E2M1 expert weights is the usual serving layout of a
 * mixture-of-experts layer; the block dot product is mx_gemm_mixed's).
 * A's rows are as long as fmt_a says, B's as fmt_b says; everything
 * else as for mx_gemm_grouped, whose plan (mx_gemm_grouped_plan with fmt_a)
 * describes the launch.  With fmt_a == fmt_b it is mx_gemm_grouped.
 */
int mx_gemm_grouped_mixed(int fmt_a, int fmt_b, int64_t groups, const int64_t *group_rows,
                          int64_t N, int64_t K, const void *A, const void *A_scale,
                          const void *B, const void *B_scale, void *C, int out_dtype,
                          void *stream);

/*
 * How mx_gemm_grouped would run a problem: one tile shape for all groups
 * (split_k is always 1, workspace_bytes 0; workgroups is the total number of
 * tiles over the groups, 0 when there are no rows).  Host logic only: no
 * HIP call, no device needed.  Returns MX_OK or mx_gemm_grouped's argument
 * error (MX_ERR_NULL also for a NULL plan).
 */
int mx_gemm_grouped_plan(int fmt, int64_t groups, const int64_t *group_rows,
                         int64_t N, int64_t K, int out_dtype, mx_plan_t *plan);

/*
 * Grouped dense BF16 GEMM (the FlyDSL article's grouped-GEMM cases, section
 * "Performance numbers need their baselines", with the dense BF16 GEMM's
 * element type): group g multiplies its group_rows[g] rows of A by its own
 * N x K weight B_g with no scales,
 *   C_g = A_g * B_g^T  for g = 0 .. groups-1,
 * each exactly as mx_gemm_bf16 would (with its plan's tile and no K split).
 *   groups       1 .. MX_MAX_GROUPS
 *   group_rows   HOST array of `groups` row counts, each >= 0
 *   A            (sum of group_rows) x K bfloat16 values, K-contiguous
 *   B            groups * N rows of K bfloat16 values (weight g is rows
 *                g*N .. g*N+N-1)
 *   C            (sum of group_rows) x N, rows in the order of A's rows
 * K, the output types, alignment (16 bytes for A, B and C), errors and
 * asynchrony as for mx_gemm_bf16; groups * N must not exceed MX_MAX_DIM.
 * With no rows at all it returns MX_OK at once.  No workspace is used.
 */
int mx_gemm_grouped_bf16(int64_t groups, const int64_t *group_rows, int64_t N, int64_t K,
                         const void *A, const void *B, void *C, int out_dtype, void *stream);

/*
 * How mx_gemm_grouped_bf16 would run a problem (as mx_gemm_grouped_plan
 * does for MX formats).  Host logic only.
 */
int mx_gemm_grouped_bf16_plan(int64_t groups, const int64_t *group_rows, int64_t N,
                              int64_t K, int out_dtype, mx_plan_t *plan);

/* Launch shape of mx_mfma_ceiling: the tile kernel's (one 512-thread
 * workgroup per compute unit of the MI355X). */
#define MX_CEILING_WORKGROUPS 256
#define MX_CEILING_THREADS 512

/*
 * Measurement, not part of the GEMM: the rate at which the current device
 * sustains the block-scaled matrix instruction with no memory traffic, to
 * set a GEMM's measured rate against (the datasheet peak assumes the top
 * clock, which the power limit may not allow).  Every wave of
 * MX_CEILING_WORKGROUPS x MX_CEILING_THREADS threads keeps a 2 x 4 grid of
 * 32x32 FP32 accumulators and runs `steps` K-steps of 8 instructions (K 64
 * each, 2*32*32*64 FLOPs each) on register-resident operands: two operand
 * sets alternating step by step, hashed ("random_data" non-zero; E4M3 NaN
 * codes replaced) or constant.  Total FLOPs =
 * MX_CEILING_WORKGROUPS * MX_CEILING_THREADS / 64 * steps * 8 * 131072.
 *   fmt     MX_FMT_E2M1 or MX_FMT_E4M3 (both operands)
 *   steps   even, 2 .. 2^30
 *   out     device memory for MX_CEILING_WORKGROUPS * MX_CEILING_THREADS
 *           floats, 4-byte aligned; receives each lane's accumulator sum (a
 *           value with no meaning, written so that no work is dead code)
 * Returns MX_OK or MX_ERR_FORMAT / MX_ERR_SHAPE / MX_ERR_NULL / MX_ERR_ALIGN
 * / a device error; asynchronous on `stream` like mx_gemm.
 */
int mx_mfma_ceiling(int fmt, int64_t steps, int random_data, float *out, void *stream);

/* Launch shape of mx_hbm_read_ceiling: two 256-thread workgroups per CU. */
#define MX_HBM_CEILING_WORKGROUPS 512
#define MX_HBM_CEILING_THREADS 256

/*
 * Measurement only, not part of the GEMM: reads `bytes` of device memory at
 * src once, as a plain streaming kernel does.  The buffer is cut into
 * MX_HBM_CEILING_WORKGROUPS contiguous ranges of ceil(bytes/16 /
 * MX_HBM_CEILING_WORKGROUPS) 16-byte chunks (the last ones shorter or
 * empty); thread t of workgroup w folds with XOR the chunks t, t + 256, ...
 * of range w, and writes its fold to out[256 w + t] (out holds
 * MX_HBM_CEILING_WORKGROUPS * MX_HBM_CEILING_THREADS 32-bit words,
 * caller-owned device memory).  Loads carry the nontemporal hint.  Timing
 * it over a buffer larger than the last-level cache gives the rate at which
 * this device actually delivers HBM data to the CUs, the practical bound of
 * the memory-bound GEMM shapes (the FlyDSL article, "Performance numbers need
 * their baselines": a rate means little without its baseline).  bytes is a
 * positive multiple of 16; src is 16-byte aligned, out 4-byte aligned.
 * Enqueued on `stream`, asynchronous.  Returns MX_OK, MX_ERR_NULL,
 * MX_ERR_SHAPE, MX_ERR_ALIGN, a device error or MX_ERR_LAUNCH.
 */
int mx_hbm_read_ceiling(const void *src, int64_t bytes, uint32_t *out, void *stream);

/*
 * -------------------------------------------------------------------------
 * The operators between two products of a transformer block: row operators
 * (norm, gated activation) whose outputs are MX operands, expert routing
 * around mx_gemm_grouped, and products with a fused epilogue.
 *
 * Common to them:
 *   - dtype is MX_IN_FP32 or MX_IN_BF16, the type of the rows they read and
 *     write; sums, statistics and weights are FP32, and each output is
 *     rounded once (to nearest even), from FP32;
 *   - ld* arguments are row pitches in elements (in bytes for
 *     mx_moe_gather), at least the row's length; outputs are dense;
 *   - rows of floating values start 16-byte aligned (pointer and pitch);
 *   - zero rows or tokens are allowed: nothing is launched and no pointer is
 *     looked at (a dW or group_rows that is asked for is still written);
 *   - errors, asynchrony and determinism are as for mx_gemm.  An output
 *     overlaps no input unless it says otherwise.  They allocate nothing and
 *     can be captured in a graph; where a workspace is needed it is the
 *     caller's, used on `stream` until the call's work is done there.
 */

/* Longest row of a row operator. */
#define MX_ROW_MAX_WIDTH 65536

/*
 * Residual addition, root-mean-square norm and MX quantization in one pass:
 *   H = X + R (rounded to dtype),  rstd = 1 / sqrt(mean_j H_j^2 + eps),
 *   Y_j = H_j * rstd * W_j,        (Q, Q_scale) = MX(Y), from the unrounded Y.
 *   fmt        any MX_FMT_* code (not looked at without Q)
 *   w_dtype    MX_IN_FP32 or MX_IN_BF16, the type of W (width values)
 *   width      a multiple of 32, at most MX_ROW_MAX_WIDTH
 *   R          NULL: no residual, H = X
 *   H          rows x width, written only with R (may be X or R itself when
 *              that is dense)
 *   Y          rows x width in dtype, or NULL
 *   Q, Q_scale mx_quantize's layout (Q 8-byte aligned), or NULL; Y and Q may
 *              not both be NULL
 *   rstd       rows floats for mx_rmsnorm_backward, or NULL
 *   eps        at least 0
 * A NaN in a row gives NaNs in its Y and blocks of scale 255 with zero codes,
 * as mx_quantize does for such blocks.  The sum of squares is FP32: a row
 * with an infinity, or whose squares pass FP32's range, has rstd 0 (its
 * infinities become NaNs, the rest zeros).
 */
int mx_rmsnorm_quantize(int fmt, int dtype, int w_dtype, int64_t rows, int64_t width,
                        const void *X, int64_t ldx, const void *R, int64_t ldr, const void *W,
                        float eps, void *H, void *Y, void *Q, void *Q_scale, float *rstd,
                        void *stream);

/*
 * Gradient of mx_rmsnorm_quantize; the MX rounding passes gradients through
 * unchanged.  With xhat = H * rstd:
 *   dX = rstd * (dY * W - xhat * mean_j(dY * W * xhat)) + dH
 *   dW = sum over rows of dY * xhat   (FP32; NULL: not wanted)
 * dX, rows x width in dtype, is the gradient of X and of R alike.  dH (or
 * NULL) is the gradient that reaches H from its other uses.
 *   workspace  mx_rmsnorm_backward_workspace(rows, width) bytes, 16-byte
 *              aligned; only used for dW
 */
int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t width);
int mx_rmsnorm_backward(int dtype, int w_dtype, int64_t rows, int64_t width, const void *dY,
                        int64_t lddy, const void *H, int64_t ldh, const float *rstd,
                        const void *W, const void *dH, int64_t lddh, void *dX, float *dW,
                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Gated activation and MX quantization: GU holds rows of 2 * width values,
 * gate then up (the output of a fused gate/up product), and
 *   (Q, Q_scale) = MX(gate * sigmoid(gate) * up).
 * width as for mx_rmsnorm_quantize; ld >= 2 * width.  The sigmoid keeps its
 * precision down to 2^-252, so that a far negative gate and a large up give
 * their product; below that it is 0.
 */
int mx_swiglu_quantize(int fmt, int dtype, int64_t rows, int64_t width, const void *GU,
                       int64_t ld, void *Q, void *Q_scale, void *stream);

/*
 * Its gradient (the MX rounding passes through): with s = sigmoid(gate),
 *   d_up = dY * gate * s,  d_gate = dY * up * s * (1 + gate * (1 - s)),
 * written as dense rows of 2 * width values, d_gate then d_up.  dGU may be GU
 * itself when that is dense.
 */
int mx_swiglu_backward(int dtype, int64_t rows, int64_t width, const void *dY, int64_t lddy,
                       const void *GU, int64_t ld, void *dGU, void *stream);

/* Most choices per token. */
#define MX_MOE_MAX_TOP 64

/*
 * Sorts tokens by expert: ids is tokens x top (dense; id_bytes 4 or 8 for
 * 32- or 64-bit signed integers), the experts each token goes to.  The sort
 * is stable in the order of ids.
 *   group_rows device array of `experts` counts: the rows of each expert
 *              (what mx_gemm_grouped takes, once copied to the host)
 *   row_of     tokens x top: the row of each (token, choice) in expert order.
 *              An id outside 0 .. experts - 1 (a padding token, a dropped
 *              choice) is no expert: its pair comes after all experts', at
 *              some row r, and row_of holds -1 - r.
 *   experts    1 .. MX_MAX_GROUPS; tokens * top at most MX_MAX_DIM
 *   workspace  mx_moe_sort_workspace(tokens, top, experts) bytes (may be 0),
 *              4-byte aligned
 */
int64_t mx_moe_sort_workspace(int64_t tokens, int64_t top, int64_t experts);
int mx_moe_sort(int id_bytes, int64_t tokens, int64_t top, int64_t experts, const void *ids,
                int64_t *group_rows, int32_t *row_of, void *workspace, int64_t workspace_bytes,
                void *stream);

/*
 * Copies token rows into expert order: row t of X (row_bytes bytes, pitch
 * ldx bytes) goes to row row_of[t][j] of XS for every choice j, and likewise
 * its scale_bytes of scales from X_scale to XS_scale (X_scale NULL: none, as
 * for BF16 rows).  XS and XS_scale have tokens * top dense rows; rows of
 * pairs without an expert, which come last, are zeros.  Any byte layout and
 * alignment is taken; 16-byte aligned rows are fastest.  Its gradient is
 * mx_moe_combine without weights.
 */
int mx_moe_gather(int64_t tokens, int64_t top, const int32_t *row_of, const void *X,
                  int64_t row_bytes, int64_t ldx, const void *X_scale, int64_t scale_bytes,
                  int64_t lds, void *XS, void *XS_scale, void *stream);

/*
 * out[t] = R[t] + sum over choices j, in order, of weights[t][j] *
 * Y[row_of[t][j]], skipping pairs without an expert (nothing of theirs is
 * read).  A token with none gets R[t], or zeros.
 *   width      the rows' length, a multiple of 8
 *   Y          y_rows x width; rows at or past y_rows count as no expert
 *   weights    tokens x top floats, or NULL: all 1
 *   R          tokens x width, or NULL: nothing is added
 *   out        tokens x width (may be R itself when that is dense)
 */
int mx_moe_combine(int dtype, int64_t tokens, int64_t top, int64_t width, const int32_t *row_of,
                   const void *Y, int64_t y_rows, int64_t ldy, const float *weights,
                   const void *R, int64_t ldr, void *out, void *stream);

/*
 * Its gradient (R's is dOut itself):
 *   dY[row_of[t][j]] = weights[t][j] * dOut[t], zeros in the rows of pairs
 *   without an expert (y_rows, at most tokens * top, covers the rows that are
 *   wanted); dweights[t][j] = sum over columns of dOut[t] * Y[row_of[t][j]],
 *   0 without an expert.
 */
int mx_moe_combine_backward(int dtype, int64_t tokens, int64_t top, int64_t width,
                            const int32_t *row_of, const void *dOut, int64_t lddo,
                            const void *Y, int64_t y_rows, int64_t ldy, const float *weights,
                            void *dY, float *dweights, void *stream);

/* Activations of a fused epilogue: none, max(x, 0), x * sigmoid(x), and GELU
 * by erf or by its tanh form (sigmoids as for mx_swiglu_quantize). */
enum { MX_ACT_NONE = 0, MX_ACT_RELU = 1, MX_ACT_SILU = 2, MX_ACT_GELU = 3, MX_ACT_GELU_TANH = 4 };

/*
 * C = residual + act(A * B^T + bias): mx_gemm_mixed's product with bias,
 * activation and residual applied to the FP32 sums before C's one rounding.
 *   fmt_a,
 *   fmt_b      E2M1 with E2M1, E4M3 with E4M3, or E4M3 with E2M1;
 *              MX_ERR_FORMAT otherwise
 *   bias       N values in bias_dtype (MX_IN_FP32 or MX_IN_BF16), or NULL
 *   act        MX_ACT_*
 *   residual   M x N in C's type with pitch ldr, 16-byte aligned, or NULL;
 *              may be C itself (with ldr == N)
 *   workspace  the plan's workspace_bytes (mx_gemm_fused_plan; often 0),
 *              16-byte aligned; with less, or NULL, K is not split
 * Everything else as for mx_gemm.
 */
int mx_gemm_fused(int fmt_a, int fmt_b, int64_t M, int64_t N, int64_t K, const void *A,
                  const void *A_scale, const void *B, const void *B_scale, const void *bias,
                  int bias_dtype, int act, const void *residual, int64_t ldr, void *C,
                  int out_dtype, void *workspace, int64_t workspace_bytes, void *stream);

/* The same on mx_gemm_bf16's operands. */
int mx_gemm_bf16_fused(int64_t M, int64_t N, int64_t K, const void *A, const void *B,
                       const void *bias, int bias_dtype, int act, const void *residual,
                       int64_t ldr, void *C, int out_dtype, void *workspace,
                       int64_t workspace_bytes, void *stream);

/*
 * The launch they would make: the decode kernel or a tile (128 x 64 and
 * 64 x 64 among them, so that products of a few hundred rows fill the GPU)
 * and a K split.  Host logic only; returns MX_OK or their argument error
 * (MX_ERR_NULL for a NULL plan).
 */
int mx_gemm_fused_plan(int fmt_a, int fmt_b, int64_t M, int64_t N, int64_t K, int out_dtype,
                       mx_plan_t *plan);
int mx_gemm_bf16_fused_plan(int64_t M, int64_t N, int64_t K, int out_dtype, mx_plan_t *plan);

#ifdef __cplusplus
}
#endif

#endif /* MXGEMM_H */
