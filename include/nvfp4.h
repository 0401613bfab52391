/*
 * nvfp4.h -- C ABI of libnvfp4, the MI355X (gfx950) NVFP4 weight-only
 * projection GEMV of batched LLM decode.
 *
 * The operation (Atlas PR #266, PR description "What it does"): for n
 * concurrent decode tokens, one projection computes
 *
 *     Y[t][r] = gscale * sum_k X[t][k] * e2m1(code[r][k]) * e4m3(scale[r][k/16])
 *
 * for t < n, r < N.  The page's point is that a tile of tokens shares one read
 * of the weight matrix instead of one read per token; its greedy tiling into
 * 3-token tiles is available as an explicit schedule (nvfp4_gemv_sched),
 * while the default launch reads the weight once for all n <= 16 tokens.
 *
 * Number formats: the pages name NVFP4 without defining its bits.  Codes are
 * OCP FP4 E2M1 (sign bit 3, magnitudes {0,.5,1,1.5,2,3,4,6}), block scales OCP
 * FP8 E4M3FN (bias 7, max 448, 0x7F/0xFF NaN), one scale per 16 consecutive k
 * of a row, and one fp32 tensor multiplier gscale.  X and Y are bf16 bit
 * patterns, accumulation is fp32, Y is rounded to nearest even.
 *
 * Conventions for every entry point:
 *   - all array pointers are DEVICE pointers of the current device (the
 *     one hipSetDevice selected), where every launch runs; calls are
 *     asynchronous on `stream` (a hipStream_t of that device; NULL is its
 *     default stream);
 *   - the caller allocates and owns every buffer; the GEMV entry points
 *     allocate nothing, cache no pointer and never synchronise;
 *   - arguments are validated on the host before any HIP call; a failed
 *     validation returns a status and launches nothing;
 *   - no exception crosses the ABI; nvfp4_strerror names every status.
 *
 * Layouts:
 *   canonical codes  [N][K/2] u8: element (r,k) in byte r*K/2 + k/2, low
 *                    nibble for even k, high nibble for odd k;
 *   canonical scales [N][K/16] u8: one E4M3 byte per 16 consecutive k;
 *   packed (device)  layout written by nvfp4_pack and read by the GEMV
 *                    entry points: rows padded to a multiple of 16 and K to
 *                    a multiple of 128 with zero codes, stored as 16-row x
 *                    128-column tiles whose 1 KiB of codes is one 16-byte
 *                    load per lane of a 64-lane wavefront; its byte sizes
 *                    are nvfp4_packed_codes_bytes / nvfp4_packed_scales_bytes;
 *   X [n][K] bf16 row-major (token-major), Y [n][N] bf16 row-major.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_NULL = 1,      /* a required pointer is NULL                      */
    NVFP4_ERR_RANGE = 2,     /* n outside [1,16], N or K not positive, bad rows */
    NVFP4_ERR_ALIGN = 3,     /* a pointer is not aligned as documented          */
    NVFP4_ERR_SHAPE = 4,     /* K not a multiple of 16, or a size limit         */
    NVFP4_ERR_SCHEDULE = 5,  /* an explicit tile schedule is invalid            */
    NVFP4_ERR_LAUNCH = 6,    /* the HIP runtime rejected a launch               */
    NVFP4_ERR_DEVICE = 7,    /* the current device is not a gfx950 GPU          */
    NVFP4_ERR_WORKSPACE = 8, /* a required workspace is NULL or too small       */
    NVFP4_ERR_SCRATCH = 9,   /* beyond the fixed scratch of nvfp4_gemv_ws_static */
    NVFP4_ERR_OVERLAP = 10   /* an output overlaps another argument             */
} nvfp4_status;

/* Largest number of tokens one launch covers (the decode batch of the pages:
 * up to 16 concurrent sequences, Atlas PR #266 A/B table, C = 1..16). */
#define NVFP4_MAX_TOKENS 16

/* Byte sizes of the packed device layout for an N x K weight: the weight in
 * the order the GEMV kernels load it, built once at load time.  The pages
 * trace their fast path to exactly this: the wide kernel ran fast only on a
 * weight copy laid out for it, and the fix they propose is to emit that copy
 * when the weight is (re)quantised (Atlas PR #266 automated review page,
 * "Tiebreaker" comment and the "Complete picture" follow-up).  Rows are padded
 * to 16 and K to 128, so the sizes are ceil(N/16)*16 * ceil(K/128)*128 / 2
 * bytes of codes and a sixteenth of that count of scale bytes, computed in
 * 64-bit arithmetic.  0 if N <= 0 or K <= 0 or K % 16 != 0. */
size_t nvfp4_packed_codes_bytes(int N, int K);
size_t nvfp4_packed_scales_bytes(int N, int K);

/* Quantise an fp32 weight W [N][K] (device, row-major, finite values) to the
 * canonical NVFP4 layout with the recipe: gscale = fp32(amax / (6*448));
 * per 16-block scale = E4M3 round-to-nearest-even of amax_block/(6*gscale),
 * saturating at 448; code = sign(w) | E2M1 round-to-nearest-even of
 * |w| / (scale*gscale) (magnitude 0 when that product is 0).
 * tensor_scale: device float[2]; [0] receives gscale, [1] the tensor amax.
 * codes: [N][K/2], scales: [N][K/16] (canonical).  Requires K % 16 == 0,
 * W 16-byte aligned.  Errors: NULL, RANGE, SHAPE, ALIGN, LAUNCH. */
int nvfp4_quantize(const float *W, int N, int K, uint8_t *codes, uint8_t *scales,
                   float *tensor_scale, void *stream);

/* Input element types of nvfp4_quantize_packed. */
#define NVFP4_DTYPE_F32 0
#define NVFP4_DTYPE_BF16 1

/* The same recipe as nvfp4_quantize, writing the packed device layout
 * directly (no canonical copy, no nvfp4_pack pass): the pages' runtime
 * requantisation, whose fix emits the layout the GEMV reads during the
 * requant (Atlas PR #266 review and follow-up on the transposed copy).  W is
 * [N][K] row-major, fp32 (dtype NVFP4_DTYPE_F32, finite) or bf16 bit patterns
 * (NVFP4_DTYPE_BF16, widened to fp32 exactly, so the result is the fp32
 * recipe on the widened values), 16-byte aligned.  codes_packed /
 * scales_packed: device buffers of nvfp4_packed_*_bytes(N, K), 16-byte
 * aligned, byte-identical to nvfp4_pack(nvfp4_quantize(W)) including the zero
 * padding.  tensor_scale: device float[2] = {gscale, amax}.  Errors: NULL,
 * RANGE (N, K, dtype), SHAPE (K % 16), ALIGN, DEVICE, LAUNCH. */
int nvfp4_quantize_packed(const void *W, int dtype, int N, int K, uint8_t *codes_packed,
                          uint8_t *scales_packed, float *tensor_scale, void *stream);

/* Reorder canonical codes/scales (device) into the packed device layout
 * (device buffers of nvfp4_packed_*_bytes; the padding is written as zeros):
 * the one-time layout step the pages ask for, the weight copy the fast kernel
 * reads, made once at load instead of on every call (Atlas PR #266 automated
 * review page, "Tiebreaker" comment: the wide GEMM's fast path needs such a
 * copy, and emitting it at load is named as the fix).  A pure byte gather
 * (nibble order unchanged), so packing loses nothing.  Errors: NULL, RANGE,
 * SHAPE, ALIGN (packed buffers must be 16-byte aligned), LAUNCH, DEVICE. */
int nvfp4_pack(const uint8_t *codes, const uint8_t *scales, int N, int K,
               uint8_t *codes_packed, uint8_t *scales_packed, void *stream);

/* Y[n][N] = X[n][K] . dequant(W)^T for 1 <= n <= 16 tokens: one projection
 * of n concurrent decode tokens that reads the weight once for all of them
 * (Atlas PR #266 conversation page, PR description "What it does": a tile of
 * tokens shares one read of the projection weight instead of one read per
 * token).  Here the tile is the whole batch of up to 16 tokens.
 * Wq / Wscale: packed layout (nvfp4_pack), 16-byte aligned.
 * X: bf16 [n][K], 16-byte aligned.  Y: bf16 [n][N], 2-byte aligned.
 * Each token's result is bit-identical to the same token computed alone
 * (n = 1) and under any schedule of nvfp4_gemv_sched.  Any N >= 1 and any
 * K % 16 == 0 up to 262144; K beyond 8192 runs in several K-chunk passes
 * inside the one launch.  Errors: NULL, RANGE, SHAPE (K % 16, K > 262144, or
 * a workgroup's share of the weight beyond 2 GiB), ALIGN, LAUNCH, DEVICE. */
int nvfp4_gemv(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
               const uint16_t *X, uint16_t *Y, int n, int N, int K, void *stream);

/* nvfp4_gemv with the K dimension cut into ks parts, for long-K projections
 * such as a dense FFN's down projection (the dense-FFN decode paths of the
 * spark_model::layers page's FfnComponent dispatch).  One launch computes the
 * fp32 partial of each (K part, 16-row group) unit into `workspace`
 * ([ks][n][N] fp32, DEVICE, 16-byte aligned, at least
 * nvfp4_gemv_workspace_bytes(n, N, K, ks) bytes, owned by the caller); a
 * second launch on the same stream adds the parts in part
 * order, scales by gscale and rounds to bf16.  The parts fill the chip where
 * N alone has fewer 16-row groups than there are compute units and cut the
 * share of X each compute unit loads.  ks = 0 takes nvfp4_gemv_kparts(N, K);
 * ks = 1 is exactly nvfp4_gemv (no workspace needed, none touched).  The sum
 * order depends only on (N, K, ks), so each token's result is bit-identical
 * to the same token alone (n = 1) at the same ks; across different ks the
 * rounding order differs (all within the documented fp32 error bound).
 * Calls that share a workspace on different streams race.  Errors: as
 * nvfp4_gemv; RANGE (ks < 0 or ks > 64), SHAPE (with T = ceil(K/128) and
 * tp = ceil(T/ks) tiles per part: a part would be empty, ks > T or
 * (ks-1)*tp >= T, or longer than one pass, ks > 1 and tp > 64),
 * WORKSPACE (ks > 1 and workspace NULL or too small), ALIGN (workspace). */
int nvfp4_gemv_ws(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
                  const uint16_t *X, uint16_t *Y, int n, int N, int K, int ks,
                  void *workspace, size_t workspace_bytes, void *stream);

/* nvfp4_gemv_ws for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, kernels and results (bit for bit) as nvfp4_gemv_ws, except
 * that the fp32 partials go to a fixed scratch array inside the library
 * instead of a caller workspace: nvfp4_gemv_static_scratch_bytes() bytes
 * (8 MiB) of device memory per GPU the library runs on, held until the
 * process ends.  Its address on a device is looked up on the first call with
 * ks > 1 on that device (make that first call outside graph capture); no call
 * allocates or frees anything.  Every element the reduction reads is written
 * earlier in the same call, so nothing needs clearing between calls.  All
 * calls on one GPU share the array: calls that overlap on one GPU (other
 * streams, other threads) race and give wrong results; calls ordered on one
 * stream are safe.  Errors: as nvfp4_gemv_ws (no WORKSPACE), SCRATCH when
 * ks * n * N * 4 bytes exceed the scratch (checked before any HIP call),
 * DEVICE if the scratch address cannot be looked up. */
int nvfp4_gemv_ws_static(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
                         const uint16_t *X, uint16_t *Y, int n, int N, int K, int ks,
                         void *stream);

/* Bytes of the fixed scratch nvfp4_gemv_ws_static uses (8 MiB).  Pure host
 * function. */
size_t nvfp4_gemv_static_scratch_bytes(void);

/* K parts nvfp4_gemv_ws takes for ks = 0, from the shape alone: 1 while K <=
 * 8192 (one pass of the 8 waves' X slices); beyond, the part count that
 * minimises (rounds of 16-row groups per compute unit of MI355X's 256) x
 * (128-column tiles per part) with every part within one pass, the fewest on
 * a tie (4 for 5120 x 17408).  Pure host function; returns ks >= 1 or a
 * negative status (-RANGE, -SHAPE). */
int nvfp4_gemv_kparts(int N, int K);

/* Bytes of workspace nvfp4_gemv_ws needs for (n, N, K, ks): ks * n * N * 4
 * for ks > 1 (ks = 0: nvfp4_gemv_kparts), 0 for ks = 1 and for invalid
 * arguments.  Pure host function. */
size_t nvfp4_gemv_workspace_bytes(int n, int N, int K, int ks);

/* Fused QKV projection (Atlas PR #266, PR description, multi_seq/qkv.rs
 * bullet: one fused weight whose q, k and v rows land at fixed offsets of a
 * per-sequence buffer).  W has N = rows[0]+rows[1]+rows[2] rows: rows
 * [0,rows[0]) are q, the next rows[1] are k, the last rows[2] are v.  Token t's
 * q/k/v outputs are written straight to Y + t*ldy + out_off[p] + j (j < rows[p])
 * with no scratch buffer and no device-to-device copy.  The three output
 * ranges must not overlap and must fit in ldy (ldy >= out_off[p] + rows[p]).
 * rows / out_off are HOST arrays read during the call.  Same bit-identity
 * guarantees as nvfp4_gemv; results equal the three slices of nvfp4_gemv on
 * the same weight bit for bit.  Errors: as nvfp4_gemv, RANGE for bad
 * rows/out_off/ldy. */
int nvfp4_gemv_qkv(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
                   const uint16_t *X, uint16_t *Y, int n, int K,
                   const int32_t rows[3], const int64_t out_off[3], int64_t ldy,
                   void *stream);

/* nvfp4_gemv under an explicit token-tile schedule: tile_widths (HOST array
 * of ntiles entries, each in [1,16], summing to n) splits the n tokens into
 * consecutive tiles, each one launch that reads the whole weight once.  This
 * is how the pages' greedy [3,3,...,2|1] tiling (Atlas PR #266 description)
 * is reproduced for comparison.  Errors: as nvfp4_gemv, SCHEDULE for a bad
 * schedule (never a silent fallback). */
int nvfp4_gemv_sched(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
                     const uint16_t *X, uint16_t *Y, int n, int N, int K,
                     const uint8_t *tile_widths, int ntiles, void *stream);

/* The dispatcher's schedule for (n, N, K): writes the tile widths nvfp4_gemv
 * uses into widths (HOST, capacity max_tiles) and returns their count, or a
 * negative status (RANGE, SHAPE for a shape nvfp4_gemv refuses, SCHEDULE for
 * no room).  Pure host function. */
int nvfp4_schedule(int n, int N, int K, uint8_t *widths, int max_tiles);

/* The pages' greedy schedule (Atlas PR #266 description): as many tiles of
 * `width` tokens as fit, then one tile with the remaining tokens; with width 3
 * a batch of 8 tokens takes 3 weight reads.  Returns the tile count or a
 * negative status.  Pure host function. */
int nvfp4_schedule_greedy(int n, int width, uint8_t *widths, int max_tiles);

/* Launch geometry the library uses for (n, N, K): workgroups, waves per
 * workgroup and 128-column tiles per wave.  Pure host function; returns a
 * status. */
int nvfp4_launch_geometry(int n, int N, int K, int *workgroups, int *waves,
                          int *tiles_per_wave);

/* The GEMV kernel a call launches for (n, N, K) with ks K parts (ks = 1:
 * nvfp4_gemv, nvfp4_gemv_qkv and every tile of nvfp4_gemv_sched; ks = 0: the
 * part count nvfp4_gemv_ws takes, nvfp4_gemv_kparts(N, K); ks > 1: that many
 * parts of nvfp4_gemv_ws).  The kernel is specialised on five values, which
 * variant (HOST int[5]) receives: [0] 128-column tiles of each wave's K-slice
 * in one pass (1 .. 8), [1] groups of four tokens carried, ceil(n/4), [2] 1 if
 * every wave owns exactly [0] tiles of every pass (no column predication),
 * [3] K-chunk passes inside the launch (1 = one pass), [4] K parts.  Lets a
 * caller, and the tests, know which specialisation serves a shape (the tile
 * schedule and its variants are the dispatch the PR description describes,
 * here picked from the shape).  Pure host function; returns a status (RANGE,
 * SHAPE as nvfp4_gemv_ws would). */
int nvfp4_gemv_variant(int n, int N, int K, int ks, int *variant);

/* Largest token count of one nvfp4_gemm call. */
#define NVFP4_MAX_GEMM_TOKENS (1 << 20)

/* Prefill / many-token form of the same operation (the step after decode as
 * n grows: the spark_model::layers page's W4A16 tile GEMMs for prefill, with
 * tile shapes picked by an occupancy rule):
 *     Y[t][r] = gscale * sum_k X[t][k] * e2m1(code[r][k]) * e4m3(scale[r][k/16])
 * for any 1 <= n <= NVFP4_MAX_GEMM_TOKENS.  Same packed weight (nvfp4_pack),
 * X bf16 [n][K] and Y bf16 [n][N] (row-major, contiguous) as nvfp4_gemv.
 * The weight is dequantised exactly to bf16 once per token tile (32, 64 or
 * 128 tokens) and multiplied with MFMA, fp32 accumulation over all of K.
 * Each token's result is bit-identical whatever n and its place in the batch
 * (the sum over K runs in one fixed order), but it is a different rounding
 * order from nvfp4_gemv's (both within the documented fp32 error bound).
 * For n <= 16 nvfp4_gemv is the faster call: it splits K over the waves of a
 * workgroup and keeps many more weight bytes in flight (on MI355X, 14336 x
 * 5120 fused QKV at n = 16: about 10 us against 18.5 us; nvfp4_gemm takes
 * 18.4 - 18.7 us at any n <= 16, where it runs the 32-token tile).
 * Errors: NULL, RANGE (n, N, K), SHAPE (K % 16, K > 262144), ALIGN (Wq,
 * Wscale, X 16-byte; Y 2-byte), DEVICE, LAUNCH. */
int nvfp4_gemm(const uint8_t *Wq, const uint8_t *Wscale, float gscale,
               const uint16_t *X, uint16_t *Y, int n, int N, int K, void *stream);

/* Tile shape and grid nvfp4_gemm uses for (n, N, K) on MI355X: weight rows
 * and tokens per workgroup, workgroups along rows and along tokens.  Tokens:
 * the smallest of 32 / 64 / 128 holding n.  Rows: 256 (8 waves) when that grid
 * gives at least half of the 256 compute units a workgroup (also with 64-token
 * tiles instead of two or more 128-token tiles where only they get there),
 * else 64 (4 waves, or 8 waves sharing the row groups' tokens when there is
 * one 128-token tile).
 * Pure host function; returns a status. */
int nvfp4_gemm_geometry(int n, int N, int K, int *rows_per_workgroup,
                        int *tokens_per_workgroup, int *grid_x, int *grid_y);

/* ---- fused operators ------------------------------------------------------
 *
 * The projection with its epilogue, the gated feed-forward block and the
 * product the other way through the weight, with the gradients of a frozen
 * NVFP4 weight (to the activations, the biases and the residual).  Conventions
 * as above, and for all of them:
 *   - matrices are row-major with a row stride in elements (>= the columns);
 *     X rows are 16-byte aligned (stride a multiple of 8, at most 2^22);
 *   - n = 0 is a valid call that launches nothing (but zeroes bias gradients);
 *   - sums, biases, activations and products are fp32, rounded once when
 *     stored;
 *   - outputs may not overlap other arguments (OVERLAP), except that the
 *     residual may be the output itself (same address, stride and type).
 *     Matrices with one stride in bytes may be neighbouring columns of one
 *     buffer; with different strides their spans, first to last element, lie
 *     apart;
 *   - a call may run in K parts: fp32 partial sums in a workspace the caller
 *     owns (16-byte aligned, at least the bytes its _workspace_bytes function
 *     names, 0 for most sizes), added in part order by a second launch.  Calls
 *     that share a workspace must be ordered (one stream); graphs captured with
 *     one must not run at the same time;
 *   - the order of every sum depends on the sizes (n, N, K) alone, so results do
 *     not vary from run to run; nvfp4_linear and nvfp4_gated take one order for
 *     all n <= 16 of an (N, K), so a token's result does not depend on the batch
 *     there (the gradients' products have no such form). */

/* Activations: z; max(z, 0); z / (1 + exp(-z)); z Phi(z) (erf form);
 * 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))). */
#define NVFP4_ACT_NONE 0
#define NVFP4_ACT_RELU 1
#define NVFP4_ACT_SILU 2
#define NVFP4_ACT_GELU 3
#define NVFP4_ACT_GELU_TANH 4

typedef struct nvfp4_epilogue {
    const void *bias;        /* [N], added before the activation (gated: of the gate), or NULL */
    const void *up_bias;     /* gated only: [F], of the up projection, or NULL */
    const void *residual;    /* linear only: [n][ldr], added after the activation, or NULL */
    float *preact;           /* receives the pre-activations for the backward pass, or NULL:
                                [n][ldp], ldp a multiple of 8, 16-byte aligned; linear: N columns;
                                gated: nvfp4_gated_rows(F) columns in the gated weight's row order
                                (columns of rows that do not exist are left as they were) */
    int64_t ldr, ldp;
    int32_t activation;      /* NVFP4_ACT_* */
    int32_t bias_dtype;      /* of bias and up_bias: NVFP4_DTYPE_* */
    int32_t residual_dtype;
    int32_t out_dtype;       /* of Y or H */
} nvfp4_epilogue;

/* Y = act(gscale X dequant(W)^T + bias) + residual for any n up to
 * NVFP4_MAX_GEMM_TOKENS and N up to 2^30, Wq / Wscale packed (nvfp4_pack).  Up
 * to 16 tokens run the decode product (K parts beyond K = 8192), more a
 * token-tiled product (K parts where its tiles alone would leave compute units
 * idle).
 * Errors: NULL, RANGE (n, N, K, strides, activation, types; up_bias set),
 * SHAPE (K % 16, K > 262144, strides), ALIGN, OVERLAP, WORKSPACE, DEVICE,
 * LAUNCH. */
int nvfp4_linear(const uint8_t *Wq, const uint8_t *Wscale, float gscale, const uint16_t *X, int64_t ldx,
                 void *Y, int64_t ldy, int n, int N, int K, const nvfp4_epilogue *epilogue,
                 void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_linear_workspace_bytes(int n, int N, int K);

/* The tile the fused operators take for n > 16 tokens on a packed weight of
 * `rows` rows and K contracted columns (gated: nvfp4_gated_rows(F) rows; the
 * gradients: the weight's K as rows, its rows up to a multiple of 8 as K):
 * weight rows and tokens of a workgroup, K groups inside it, K parts of the
 * launch (with more than one, fp32 partial sums and a second launch).  Pure
 * host function; returns a status (RANGE, SHAPE). */
int nvfp4_fused_geometry(int n, int rows, int K, int *rows_per_workgroup, int *tokens_per_workgroup,
                         int *k_groups, int *k_parts);

/* Rows of the packed weight of a gated block with F outputs: its 16-row groups
 * alternate gate, up, so gate row r is row (r / 16) * 32 + r % 16 and up row r
 * lies 16 further; F is padded to 16.  0 if F < 1. */
size_t nvfp4_gated_rows(int F);

/* The gated weight from the packed gate and up weights (F x K each): codes /
 * scales receive nvfp4_packed_*_bytes(nvfp4_gated_rows(F), K) bytes.  Once, at
 * load time.  Errors: NULL, RANGE, SHAPE, ALIGN (16), OVERLAP, DEVICE, LAUNCH. */
int nvfp4_pack_gated(const uint8_t *gate_codes, const uint8_t *gate_scales, const uint8_t *up_codes,
                     const uint8_t *up_scales, int F, int K, uint8_t *codes, uint8_t *scales, void *stream);

/* H = act(gate_gscale X Wg^T + bias) * (up_gscale X Wu^T + up_bias): both
 * projections, the activation and the product in one launch on the gated
 * weight of nvfp4_pack_gated.  n, workspace and errors as nvfp4_linear
 * (residual set: RANGE). */
int nvfp4_gated(const uint8_t *Wq, const uint8_t *Wscale, float gate_gscale, float up_gscale,
                const uint16_t *X, int64_t ldx, void *H, int64_t ldh, int n, int F, int K,
                const nvfp4_epilogue *epilogue, void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_gated_workspace_bytes(int n, int F, int K);

/* The transposed copy of a packed weight, which the gradients read: tiles of
 * 16 columns x 128 rows (rows padded with zero codes), codes in the lane order
 * of the packed layout, and beside each tile the scales of its 128 rows.
 * Another 9/16 byte a weight, made once, kept only where gradients are wanted. */
size_t nvfp4_transposed_codes_bytes(int N, int K);
size_t nvfp4_transposed_scales_bytes(int N, int K);
int nvfp4_pack_transposed(const uint8_t *codes_packed, const uint8_t *scales_packed, int N, int K,
                          uint8_t *codes_t, uint8_t *scales_t, void *stream);

/* The gradients of nvfp4_linear: with dZ = dY * act'(Z),
 *     dX = gscale dZ . dequant(W)   bf16 [n][ldx], on the transposed copy (NULL: not wanted,
 *                                   nor then the copy), dZ rounded to bf16 for the product;
 *     dbias = column sums of dZ     unrounded, in a fixed order (NULL: not wanted).
 * The residual's gradient is dY itself.  dY: bf16 or fp32, any stride and
 * element alignment; preact: as nvfp4_linear stored it (NULL with
 * NVFP4_ACT_NONE).  With no activation and no dbias this is the product the
 * other way through the weight, the input gradient of any projection of this
 * library.  Workspace (16-byte aligned): nvfp4_linear_backward_workspace_bytes
 * with dx and dbias as they are wanted, copy = 0 only if dZ is dY as it stands:
 * no activation, bf16, N a multiple of 8, dY 16-byte aligned, ldy a multiple of
 * 8 and at most 2^22.  Errors: NULL, RANGE, SHAPE (K % 16, K > 262144, strides,
 * N beyond 2^22), ALIGN, OVERLAP, WORKSPACE, DEVICE, LAUNCH. */
int nvfp4_linear_backward(const uint8_t *codes_t, const uint8_t *scales_t, float gscale, const void *dY,
                          int dy_dtype, int64_t ldy, const float *preact, int64_t ldp, int activation,
                          uint16_t *dX, int64_t ldx, void *dbias, int bias_dtype, int n, int N, int K,
                          void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_linear_backward_workspace_bytes(int n, int N, int K, int dx, int dbias, int copy);

/* The gradients of nvfp4_gated, on the transposed copy of the gated weight
 * (nvfp4_pack_transposed with N = nvfp4_gated_rows(F)): with dG = dH * U *
 * act'(G) and dU = dH * act(G), dX = gate_gscale dG . Wg + up_gscale dU . Wu in
 * one product (the scaled dG and dU rounded to bf16 for it), dgate_bias and
 * dup_bias the column sums of dG and dU.  Arguments and errors as
 * nvfp4_linear_backward. */
int nvfp4_gated_backward(const uint8_t *codes_t, const uint8_t *scales_t, float gate_gscale, float up_gscale,
                         const void *dH, int dh_dtype, int64_t ldh, const float *preact, int64_t ldp,
                         int activation, uint16_t *dX, int64_t ldx, void *dgate_bias, void *dup_bias,
                         int bias_dtype, int n, int F, int K, void *workspace, size_t workspace_bytes,
                         void *stream);
size_t nvfp4_gated_backward_workspace_bytes(int n, int F, int K, int dx, int dbias);

/* ---- expert layer -----------------------------------------------------------
 *
 * A router from logits to each token's experts and their weights, and the whole
 * layer of gated NVFP4 experts that reads them, with gradients (the experts are
 * frozen: gradients go to the activations, the weights and the logits).
 * Conventions as for the fused operators above. */

#define NVFP4_SCORE_SOFTMAX 0
#define NVFP4_SCORE_SIGMOID 1

/* The k experts of each token with the largest scores, largest first, ties to
 * the lowest index, and their weights:
 *     p = softmax(logits) or sigmoid(logits);   chosen by p + bias (bias NULL: by p);
 *     weights = scale p  or, with normalize, scale p / (sum of the chosen p).
 * logits: [n][ldl] fp32 or bf16; bias: [E] fp32, of the choice alone; weights
 * [n][k] fp32 and experts [n][k], contiguous.  E up to 1024, k up to 32 and E.
 * A logit of -infinity masks an expert: it is never chosen, and slots for which
 * no expert is left have expert -1 and weight 0.  A NaN logit counts as the
 * largest (with a softmax and a bias every score of its row is NaN: the experts
 * are then the first ones that are not masked) and makes the weights that
 * depend on it NaN.  Scores that are compared with a bias are 64-bit.
 * Errors: NULL, RANGE, ALIGN, OVERLAP, DEVICE, LAUNCH. */
int nvfp4_moe_route(const void *logits, int dtype, int64_t ldl, const float *bias, int n, int E, int k,
                    int scoring, int normalize, float scale, float *weights, int32_t *experts, void *stream);

/* dlogits [n][ldd] (every element of a row's E; the logits' type) from dweights
 * [n][k], with the experts that nvfp4_moe_route chose; the choice and its bias
 * have no gradient.  Experts outside [0, E) are skipped. */
int nvfp4_moe_route_backward(const void *logits, int dtype, int64_t ldl, const int32_t *experts,
                             const float *dweights, int n, int E, int k, int scoring, int normalize, float scale,
                             void *dlogits, int64_t ldd, void *stream);

/* E experts of one shape, each part of the E experts in turn in one buffer
 * (16-byte aligned): gated weights (nvfp4_pack_gated, F outputs, K columns) and
 * packed down weights (K rows, F columns), or for nvfp4_moe_backward the
 * transposed copies of both (nvfp4_pack_transposed).  F and K are multiples of
 * 16 up to 262144, E up to 1024.  gscale: DEVICE fp32 [3][E], the tensor scales
 * of the gate, up and down weights. */
typedef struct nvfp4_experts {
    const uint8_t *gate_up_codes, *gate_up_scales;
    const uint8_t *down_codes, *down_scales;
    const float *gscale;
    int32_t E, F, K;
} nvfp4_experts;

/* Y[t] = sum over s < k of weights[t][s] FFN(experts[t][s], X[t]) + residual[t],
 *     FFN(e, x) = (act(gate_e x Wg_e^T) * (up_e x Wu_e^T)) (down_e Wd_e)^T,
 * for n = 0 .. NVFP4_MAX_GEMM_TOKENS tokens.  experts int32 and weights fp32
 * [n][k], contiguous, k up to 32; an expert outside [0, E) is no expert (its
 * weight is not read into the sum), so a row may be empty; the same expert twice
 * counts twice.  X rows as nvfp4_linear's, ldx at most 2^18.  epilogue: activation,
 * residual (it may be Y itself), out_dtype, and preact: fp32 [n k][ldp >= 2 F]
 * receives the pre-activations for nvfp4_moe_backward, its rows in the order of
 * the experts within each part (below; rows of slots without an expert are left as
 * they were); biases NULL.  h = act() * (), an operand of the matrix instructions,
 * is held to 16 significant bits in the form for up to 16 tokens; in the other to 11
 * where Y is bf16, whose own rounding is to 8, and to 22 where Y is fp32, down to
 * 2^-24 of its row's largest value; all sums are fp32.
 * Up to 16 tokens (K up to 8192, no preact) take two launches, and a token's
 * result does not depend on the others there; more are sorted by expert, in parts
 * of 2^16 / k tokens (fewer where K is above about 16000 k).  Workspace:
 * nvfp4_moe_workspace_bytes, 16-byte aligned, with preact 1 where it is given.
 * Errors: NULL, RANGE, SHAPE, ALIGN, OVERLAP, WORKSPACE, DEVICE, LAUNCH. */
int nvfp4_moe(const nvfp4_experts *w, const uint16_t *X, int64_t ldx, const int32_t *experts,
              const float *weights, int n, int k, void *Y, int64_t ldy, const nvfp4_epilogue *epilogue,
              void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_moe_workspace_bytes(int n, int k, int E, int F, int K, int preact);

/* The tile of the grouped products for more than 16 tokens (or with preact):
 * weight rows and tokens of a workgroup.  Pure host function; returns a status
 * (NULL, RANGE, SHAPE). */
int nvfp4_moe_geometry(int n, int k, int E, int F, int K, int *rows_per_workgroup, int *tokens_per_workgroup);

/* Outputs of a workgroup in the down projection of up to 16 tokens on a device of
 * so many compute units (any number: K / outputs workgroups).  Pure host function;
 * returns a status (NULL, RANGE, SHAPE: K not a multiple of 16 up to 8192). */
int nvfp4_moe_decode_geometry(int K, int compute_units, int *outputs_per_workgroup);

/* The gradients of nvfp4_moe, on the transposed copies: dX bf16 [n][ldx] (NULL:
 * not wanted) and dweights fp32 [n][k] (NULL: not wanted; 0 where there is no
 * expert).  dY fp32 or bf16 [n][ldy], ldy at most 2^18; fp32 enters the products
 * with 16 significant bits.  The gradients of the pre-activations are held to 11
 * bits, as h of a bf16 result (dX, which they are summed to, is one).
 * preact as nvfp4_moe stored it.  The residual's gradient is dY itself.
 * Workspace: nvfp4_moe_backward_workspace_bytes with dx as it is wanted, copy =
 * 0 only if dY is bf16, 16-byte aligned and ldy a multiple of 8. */
int nvfp4_moe_backward(const nvfp4_experts *wt, const void *dY, int dy_dtype, int64_t ldy,
                       const int32_t *experts, const float *weights, const float *preact, int64_t ldp,
                       int activation, int n, int k, uint16_t *dX, int64_t ldx, float *dweights, void *workspace,
                       size_t workspace_bytes, void *stream);
size_t nvfp4_moe_backward_workspace_bytes(int n, int k, int E, int F, int K, int dx, int copy);

/* ---- 8-bit projection --------------------------------------------------------
 *
 * For layers that do not stand four bits: weight and activations in 8-bit
 * integers, one fp32 scale for each weight row (channel) and each token.  Sums
 * are exact 32-bit integers, so a result depends on its own row and token alone.
 * Conventions as for the fused operators above.  K: a multiple of 16 up to
 * 131056 (128 * 128 * K stays below 2^31). */

/* The packed layout of codes [N][K]: 16-row x 64-column tiles in the lane order
 * of the matrix instructions, rows padded to 16 and columns to 128 with zeros. */
size_t nvfp4_int8_packed_bytes(int N, int K);
int nvfp4_int8_pack(const int8_t *codes, int N, int K, int8_t *packed, void *stream);

/* Rows of X (bf16 or fp32 [n][ldx]) to 8 bits: scale = amax / 127 and
 * q = 127 x / amax rounded to the nearest integer, halves to the even one (for
 * bf16 exactly; fp32 after one rounding of each operation), amax the row's largest
 * magnitude.  A row of zeros has scale 0; a row that holds a NaN or an infinity
 * scale NaN and q 0.  K is any multiple of 16 here.  X and q rows are 16-byte
 * aligned.  Errors: NULL, RANGE, SHAPE (K % 16), ALIGN, OVERLAP, DEVICE, LAUNCH. */
int nvfp4_int8_quantize(const void *X, int dtype, int64_t ldx, int n, int K, int8_t *q, int64_t ldq,
                        float *scale, void *stream);

/* Y[t][r] = act(xscale[t] wscale[r] sum_k Xq[t][k] Wq[r][k] + bias[r]) + residual[t][r]
 * for n = 0 .. NVFP4_MAX_GEMM_TOKENS.  Wq packed.  xscale [n] with X int8
 * [n][ldx]; or xscale NULL with X bf16 [n][ldx], which is then quantised as by
 * nvfp4_int8_quantize.  X rows are 16-byte aligned, ldx at most
 * 2^22.  epilogue: bias, activation, residual (it may be Y itself), out_dtype;
 * up_bias and preact NULL (a quantised product has no derivative).  Workspace:
 * nvfp4_int8_linear_workspace_bytes (0 for some calls), quantize = 1 where xscale is
 * NULL; 16-byte aligned.
 * Errors: NULL, RANGE, SHAPE, ALIGN, OVERLAP, WORKSPACE, DEVICE, LAUNCH. */
int nvfp4_int8_linear(const int8_t *Wq, const float *wscale, const void *X, int64_t ldx, const float *xscale,
                      void *Y, int64_t ldy, int n, int N, int K, const nvfp4_epilogue *epilogue,
                      void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_int8_linear_workspace_bytes(int n, int N, int K, int quantize);

/* The tile of nvfp4_int8_linear for n > 16 tokens, as nvfp4_fused_geometry gives
 * it.  Pure host function; returns a status (NULL, RANGE, SHAPE). */
int nvfp4_int8_geometry(int n, int N, int K, int *rows_per_workgroup, int *tokens_per_workgroup, int *k_groups,
                        int *k_parts);

/* Human-readable name of a status code (static storage). */
const char *nvfp4_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
