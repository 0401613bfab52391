// Host functions shared by the translation units of libnvfp4 (not exported).
#ifndef NVFP4_INTERNAL_H
#define NVFP4_INTERNAL_H

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#define NVFP4_HIDDEN __attribute__((visibility("hidden")))

struct nvfp4_gemv_geometry {
    int workgroups, mt, kc;
    int ks, tp, wpp;   // K parts, tiles per part, workgroups per part
    bool exact;
};

// Compute units of the current device; NVFP4_ERR_DEVICE if it is no gfx950 GPU.
NVFP4_HIDDEN int nvfp4_device_cus(int *cus);
// Launch shape of the decode product (geometry_for in nvfp4.hip).
NVFP4_HIDDEN bool nvfp4_gemv_geometry_for(int N, int K, int cus, int ks, nvfp4_gemv_geometry *geo);

// What the fused operators do with a finished sum (epilogue.h).
struct nvfp4_epi_params {
    const void *bias, *up_bias;   // [N] (gated: of the gate and of the up rows), or null
    const void *residual;         // [n][ldr], or null
    float *preact;                // [n][ldp], or null
    void *out;                    // [n][ldo]
    int ldr, ldp, ldo;
    float gscale, up_gscale;
    int N;                        // outputs a token (gated: F)
    int flags;                    // the activation and kEpi* (one register of the kernels)
};

enum {
    kEpiAct = 7,
    kEpiBiasF32 = 8,
    kEpiResidualF32 = 16,
    kEpiOutF32 = 32,
    kEpiVec = 64                  // rows 4j .. 4j+3 of a token may be moved as one vector
};

struct nvfp4_fused_gemv_args {
    const uint8_t *codes, *scales;
    const uint16_t *X;
    int ldx, n, K;
    int rows;       // rows of the packed weight (gated: gate and up row groups in turn)
    int units;      // row groups, in pairs where gated
    int ks;         // K parts; > 1: fp32 partials [ks][n][rows] go to `partials`
    float *partials;
    nvfp4_epi_params epi;
};

// One decode launch; `mode`'s kernels live in a translation unit each.
NVFP4_HIDDEN int nvfp4_launch_fused_gemv_linear(const nvfp4_fused_gemv_args &a, hipStream_t stream);
NVFP4_HIDDEN int nvfp4_launch_fused_gemv_gated(const nvfp4_fused_gemv_args &a, hipStream_t stream);
NVFP4_HIDDEN int nvfp4_launch_fused_gemv_partial(const nvfp4_fused_gemv_args &a, hipStream_t stream);

#endif  // NVFP4_INTERNAL_H
