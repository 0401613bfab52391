// What the translation units of the 8-bit projection share.
#ifndef NVFP4_INT8_H
#define NVFP4_INT8_H

#include "internal.h"

// Packed weight: tiles of 16 rows x 64 columns, 1 KiB each, whose lane (i, g)
// holds columns 16 g .. 16 g + 15 of row i; rows padded to 16 and columns to 128
// with zeros; [row group][tile].
struct nvfp4_int8_args {
    const int8_t *codes;
    const float *wscale;          // [N]
    const int8_t *X;              // [n][ldx], 16-byte aligned rows
    long long ldx;
    const float *xscale;          // [n]
    int n, N, K;
    int32_t *partial;             // of a plan with several K parts: [ks][n][16 row groups]
    nvfp4_epi_params epi;
};

struct nvfp4_int8_plan {
    int tile, ks, tp;             // K parts of tp 64-column steps
};
NVFP4_HIDDEN nvfp4_int8_plan nvfp4_plan_int8(int n, int row_groups, int K);
NVFP4_HIDDEN void nvfp4_int8_tile(int tile, int *rows, int *tokens, int *k_groups);
NVFP4_HIDDEN int nvfp4_launch_int8_gemm(const nvfp4_int8_args &a, const nvfp4_int8_plan &plan, hipStream_t stream);

#endif  // NVFP4_INT8_H
