// Token-tiled product of bf16 activations with an NVFP4 weight, with a fused
// epilogue: the many-token form of the fused operators, and (on the transposed
// copy of the weight) of their input gradients.
#include "fused_gemm_kernel.h"

namespace {

template <int RG, int TB, int RW, int KG>
int launch_one(FusedGemmParams p, int mode, hipStream_t stream)
{
    p.tiles_x = (p.RG + RW * RG - 1) / (RW * RG);
    p.tiles_y = (p.n + TB * 16 - 1) / (TB * 16);
    const long long total = (long long)p.tiles_x * p.tiles_y * p.ks;
    if (total > INT32_MAX || (long long)p.T * RG * 1024 > INT32_MAX)
        return NVFP4_ERR_SHAPE;   // a wave's codes must stay within a 32-bit buffer offset
    auto k = mode == 0 ? nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 0>
                       : (mode == 1 ? nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 1> : nvfp4_fused_gemm_kernel<RG, TB, RW, KG, 2>);
    hipLaunchKernelGGL(k, dim3((unsigned)total), dim3(64 * RW * KG), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// Tile shapes: row groups a wave, 16-token blocks, waves along the rows, K
// groups, workgroups that fit a compute unit, and what an iteration (a step of
// every K group) costs (ns) with one workgroup on its unit and, per workgroup,
// with the unit full.
struct Tile {
    int rg, tb, rw, kg, full;
    double alone, shared;
};
constexpr Tile kTiles[] = {
    {2, 2, 1, 4, 2, 750, 415},      //  32 rows x  32 tokens
    {2, 2, 1, 8, 1, 1015, 885},
    {2, 2, 2, 4, 2, 820, 680},      //  64 x  32
    {2, 4, 2, 4, 1, 1315, 1170},    //  64 x  64
    {2, 4, 4, 2, 2, 995, 805},      // 128 x  64
    {4, 8, 4, 2, 1, 2655, 2530},    // 256 x 128
    {4, 8, 4, 1, 2, 1680, 1235},
};
constexpr int kParts[] = {1, 2, 3, 4, 6, 8, 12};
constexpr double kStart = 2.55;         // a workgroup's start and epilogue, in iterations
constexpr double kTail = 0.82;          // uneven end of a grid of several rounds, in workgroups a unit
constexpr double kReduceNs = 4100;      // the second launch
constexpr double kReduceSumNs = 9.2e-4; // a partial sum written and read again

}  // namespace

// The tile and part count of least modelled time.  Smaller tiles, K groups and
// K parts fill the chip where the largest tile leaves units idle; larger tiles
// dequantise a weight for more tokens, K groups add their sums in LDS where
// parts write them and need a second launch.  A step of the small tiles is
// bound by issue (64 rows x 32 tokens with 8 groups: 16 waves, 4 a SIMD, take
// 2.0 us an iteration warm or cold, with 4 groups 1.0), so that a grid which
// leaves units idle wants fewer waves a workgroup: 32 rows.  The constants were
// fitted to 120 shapes x 8 tiles x every part count measured on MI355X with
// weights that come from HBM (64 .. 34816 rows, K 1024 .. 34816, n 17 .. 8000):
// over them the choice is within 0.8% of the best measured one on average, 17%
// at worst.  Both sides of some choices (us):
//   4096 x 1024   n = 20    32 x 32, 4 groups 4.9; 64 x 32 5.6, 128 x 64 8.6
//   1237 x 2064   n = 47    32 x 32, 8 groups 7.0; 4 groups 7.2, 64 x 32 8.3
//   5120 x 6144^T n = 24    32 x 32, 8 groups 12.4; 64 x 32 in 2 parts 13.1, 1 part 15.7
//   16384 x 5120  n = 17    64 x 32 16.7; 32 x 32 18.5, 64 x 64 20.0
//   16384 x 5120  n = 64    64 x 64 24.1; 64 x 32 25.5, 128 x 64 32.2
//   16384 x 5120  n = 128   128 x 64 34.1; 64 x 64 42.5, 256 x 128 71
//   5120 x 6144   n = 1000  256 x 128 in 3 parts 78; 2 groups 81, 128 x 64 86, 1 part 97
//   gated 2 x 17408 x 5120  n = 1024  256 x 128 342; 2 groups 379, 128 x 64 402
nvfp4_fused_gemm_plan nvfp4_plan_fused_gemm(int n, int row_groups, int K)
{
    const int T = (int)k_tiles(K);
    nvfp4_fused_gemm_plan best = {};
    double best_cost = -1;
    for (int c = 0; c < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++c) {
        const Tile &t = kTiles[c];
        const long long tiles =
            (long long)((row_groups + t.rw * t.rg - 1) / (t.rw * t.rg)) * ((n + 16 * t.tb - 1) / (16 * t.tb));
        for (const int ks : kParts) {
            const int tp = (T + ks - 1) / ks;
            if (ks > 1 && (tp < 2 || tiles >= 2048))
                break;
            if ((long long)(ks - 1) * tp >= T)
                continue;   // the last part would be empty
            const long long units = tiles * ks, resident = (units + 255) / 256;
            const double per = resident <= t.full ? (double)resident : units * (1.0 / 256) + kTail;
            const double step = per * t.shared > t.alone ? per * t.shared : t.alone;
            double cost = ((tp + t.kg - 1) / t.kg + kStart) * step;
            if (ks > 1)
                cost += kReduceNs + (double)ks * n * row_groups * kRowsPerGroup * kReduceSumNs;
            if (best_cost < 0 || cost < best_cost) {
                best_cost = cost;
                best.tile = c;
                best.ks = ks;
                best.tp = tp;
            }
        }
    }
    return best;
}

void nvfp4_fused_gemm_tile(int tile, int *rows, int *tokens, int *k_groups)
{
    const Tile &t = kTiles[tile];
    *rows = kRowsPerGroup * t.rw * t.rg;
    *tokens = 16 * t.tb;
    *k_groups = t.kg;
}

int nvfp4_launch_fused_gemm(const nvfp4_fused_gemm_args &a, const nvfp4_fused_gemm_plan &plan, hipStream_t stream)
{
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    FusedGemmParams p = {};
    p.codes = reinterpret_cast<const u32x4 *>(a.codes);
    p.scales = reinterpret_cast<const char *>(a.scales);
    p.X = a.X;
    p.ldx = a.ldx;
    p.n = a.n;
    p.K = a.K;
    p.T = (int)k_tiles(a.K);
    p.RG = a.row_groups;
    p.e = a.epi;
    p.ks = plan.ks;
    p.tp = plan.tp;
    p.partial = a.partial;
    switch (plan.tile) {
    case 0: return launch_one<2, 2, 1, 4>(p, a.mode, stream);
    case 1: return launch_one<2, 2, 1, 8>(p, a.mode, stream);
    case 2: return launch_one<2, 2, 2, 4>(p, a.mode, stream);
    case 3: return launch_one<2, 4, 2, 4>(p, a.mode, stream);
    case 4: return launch_one<2, 4, 4, 2>(p, a.mode, stream);
    case 5: return launch_one<4, 8, 4, 2>(p, a.mode, stream);
    default: return launch_one<4, 8, 4, 1>(p, a.mode, stream);
    }
}
