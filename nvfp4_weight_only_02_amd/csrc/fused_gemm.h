// Launch of the many-token fused product (fused_gemm.hip).
#ifndef NVFP4_FUSED_GEMM_H
#define NVFP4_FUSED_GEMM_H

#include "internal.h"

struct nvfp4_fused_gemm_args {
    int mode;                     // 0 linear, 1 gated, 2 transposed weight
    const uint8_t *codes, *scales;
    const uint16_t *X;            // bf16 [n][ldx], 16-byte aligned rows
    long long ldx;
    int n, K;                     // K: columns contracted
    int row_groups;               // of 16 rows (gated: gate and up ones together)
    float *partial;               // of a plan with several K parts: [ks][n][16 * row_groups]
    nvfp4_epi_params epi;
};

// Tile shape and K parts of a call, from its sizes alone.
struct nvfp4_fused_gemm_plan {
    int tile, ks, tp;             // tp: 128-column tiles a part
};

NVFP4_HIDDEN nvfp4_fused_gemm_plan nvfp4_plan_fused_gemm(int n, int row_groups, int K);
NVFP4_HIDDEN void nvfp4_fused_gemm_tile(int tile, int *rows, int *tokens, int *k_groups);

NVFP4_HIDDEN int nvfp4_launch_fused_gemm(const nvfp4_fused_gemm_args &a, const nvfp4_fused_gemm_plan &plan,
                                         hipStream_t stream);

#endif  // NVFP4_FUSED_GEMM_H
