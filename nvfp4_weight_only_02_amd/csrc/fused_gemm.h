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
    nvfp4_epi_params epi;
};

NVFP4_HIDDEN int nvfp4_launch_fused_gemm(const nvfp4_fused_gemm_args &a, hipStream_t stream);

#endif  // NVFP4_FUSED_GEMM_H
