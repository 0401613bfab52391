// What the translation units of the expert layer share.
#ifndef NVFP4_MOE_H
#define NVFP4_MOE_H

#include "fused_gemm.h"

// Pairs of a token and an expert, in the experts' order (moe.hip, nvfp4_moe_sort_kernel).
struct nvfp4_moe_order {
    const int *tile;     // [1 + 2 tiles]: token tiles in use, then expert and first row of each
    const int *offset;   // [E + 1]
    const int *pair;     // [rows]: the pair at each row
};

struct nvfp4_moe_gemm_args {
    int mode;                     // 1 gated, 2 transposed, 0 linear, as nvfp4_fused_gemm_args
    bool gather;                  // X's rows are the tokens; else the rows in the experts' order, in
                                  // fp16 with exponents (store_block)
    const uint8_t *codes, *scales;
    long long cstride, sstride;   // bytes of an expert's
    const uint16_t *X;
    const int *xexp;              // of X, and of the rows of mode 1's output
    int *hexp;
    int nexp;                     // of a row
    uint16_t *hrest;              // as GroupedGemmParams
    int rest;
    long long ldx;
    int xrows, k;                 // rows of X (gather), experts of a token
    int rows, E;                  // at most so many rows
    int tile_tokens;              // of a tile (nvfp4_moe_tile_tokens)
    int K, row_groups;            // of an expert's weight
    const float *gscale, *up_gscale;
    nvfp4_moe_order order;
    nvfp4_epi_params epi;
};

// The tile of the grouped products, from the layer's sizes: its tokens (32 or 64) and
// weight rows; and the most tiles that `rows` rows of E experts can take.
NVFP4_HIDDEN int nvfp4_moe_tile_tokens(int rows, int E, int F);
NVFP4_HIDDEN int nvfp4_moe_tile_rows(int rows, int E, int tokens);
NVFP4_HIDDEN long long nvfp4_moe_max_tiles(int rows, int E, int tokens);
NVFP4_HIDDEN int nvfp4_launch_moe_gemm(const nvfp4_moe_gemm_args &a, hipStream_t stream);

// The layer for a few tokens (moe_few.hip).
struct nvfp4_moe_few_args {
    const uint8_t *gu_codes, *gu_scales, *d_codes, *d_scales;
    const float *gscale;          // [3][E]: gate, up, down
    const uint16_t *X;
    const int *experts;
    const float *weights;
    uint16_t *h;                  // nvfp4_moe_few_bytes
    int ldx, n, k, E, F, K, act;
    nvfp4_epi_params epi;         // residual and output
};
NVFP4_HIDDEN bool nvfp4_moe_is_few(int n, int K);
NVFP4_HIDDEN size_t nvfp4_moe_few_bytes(int n, int k, int F);
NVFP4_HIDDEN int nvfp4_launch_moe_few(const nvfp4_moe_few_args &a, hipStream_t stream);

#endif  // NVFP4_MOE_H
