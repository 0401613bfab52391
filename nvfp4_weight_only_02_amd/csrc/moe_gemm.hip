// Products of rows grouped by expert with the experts' NVFP4 weights: the
// many-token form of the expert layer and its gradients.
#include "fused_gemm_kernel.h"
#include "moe.h"

namespace {

template <int RG, int TB, int RW, int KG>
int launch_grouped(GroupedGemmParams p, const nvfp4_moe_gemm_args &a, hipStream_t stream)
{
    p.tiles_x = (p.RG + RW * RG - 1) / (RW * RG);
    p.tiles_y = (int)nvfp4_moe_max_tiles(a.rows, a.E, a.tile_tokens);
    const long long total = (long long)p.tiles_x * p.tiles_y;
    if (total > INT32_MAX || (long long)p.T * RG * 1024 > INT32_MAX)
        return NVFP4_ERR_SHAPE;   // a wave's codes must stay within a 32-bit buffer offset
    // (the XCDs' shares differ by one workgroup at most: 8 more cover every share)
    const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * RW * KG);
    if (a.mode == 1)
        hipLaunchKernelGGL((nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 1, 1>), grid, block, 0, stream, p);
    else if (a.mode == 0)
        hipLaunchKernelGGL((nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 0, 2>), grid, block, 0, stream, p);
    else if (a.gather)
        hipLaunchKernelGGL((nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 2, 1>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 2, 2>), grid, block, 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // namespace

// Measured on MI355X, weights cold (us, the whole layer, with gradients where
// marked; E experts of F x K with k a token):
//                                              128 x 32   128 x 64   256 x 64   256 x 128
//   n = 30    E = 64  k = 8  F = 1408 K = 5120      150        175        166         204
//   n = 100                                         184        197        194         254
//   n = 1500                                       1009        776        750         786
//   n = 700   E = 32  k = 4  F = 1280 K = 2048 *    252        235        249         305
//   n = 4000  *                                    1060        820        802         823
//   n = 300   E = 8   k = 2  F = 1024 K = 4096 *    123        143        188         271
// A larger tile dequantises a weight for more rows, but an expert's last tile is
// seldom full, and the smaller ones leave room for four workgroups a compute unit.
int nvfp4_moe_tile_tokens(int rows, int E, int F)
{
    const int each = (rows + E - 1) / E;   // rows of an expert where all are chosen alike
    const long long workgroups = (rows / 64 + (E + 1) / 2) * (2LL * F + 127) / 128;
    return each <= 40 || workgroups < 384 ? 32 : 64;
}

int nvfp4_moe_tile_rows(int rows, int E, int tokens)
{
    return tokens == 64 && rows / E >= 128 ? 256 : 128;
}

long long nvfp4_moe_max_tiles(int rows, int E, int tokens)
{
    return rows / tokens + (rows < E ? rows : E);
}

int nvfp4_launch_moe_gemm(const nvfp4_moe_gemm_args &a, hipStream_t stream)
{
    GroupedGemmParams p = {};
    p.codes = reinterpret_cast<const u32x4 *>(a.codes);
    p.scales = reinterpret_cast<const char *>(a.scales);
    p.X = a.X;
    p.ldx = a.ldx;
    p.n = a.rows;
    p.K = a.K;
    p.T = (int)k_tiles(a.K);
    p.RG = a.row_groups;
    p.ks = 1;
    p.tp = p.T;
    p.e = a.epi;
    p.tile = a.order.tile;
    p.offset = a.order.offset;
    p.pair = a.order.pair;
    p.k = a.k;
    p.xrows = a.xrows;
    p.xexp = a.xexp;
    p.hexp = a.hexp;
    p.nexp = a.nexp;
    p.hrest = a.hrest;
    p.rest = a.rest;
    p.gscale = a.gscale;
    p.up_gscale = a.up_gscale;
    p.cstride = a.cstride;
    p.sstride = a.sstride;
    if (a.tile_tokens == 32)
        return launch_grouped<2, 2, 4, 2>(p, a, stream);
    if (nvfp4_moe_tile_rows(a.rows, a.E, a.tile_tokens) == 256)
        return launch_grouped<4, 4, 4, 1>(p, a, stream);
    return launch_grouped<2, 4, 4, 1>(p, a, stream);
}
