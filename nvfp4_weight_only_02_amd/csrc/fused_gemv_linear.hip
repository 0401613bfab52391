// The linear form of the decode product with a fused epilogue (fused_gemv.inc).
#include "fused_gemv.inc"

int nvfp4_launch_fused_gemv_linear(const nvfp4_fused_gemv_args &a, hipStream_t stream)
{
    return launch_fused_gemv<0>(a, stream);
}
