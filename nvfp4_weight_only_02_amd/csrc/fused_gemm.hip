// Token-tiled product of bf16 activations with an NVFP4 weight, with a fused
// epilogue: the many-token form of the fused operators, and (on the transposed
// copy of the weight) of their input gradients.
#include "fused_gemm.h"

#include "epilogue.h"

namespace {

struct FusedGemmParams {
    const u32x4 *codes;    // packed codes, [RG][T][64 lanes] x 16 B
    const char *scales;    // packed scales, 128 B a tile
    const uint16_t *X;     // bf16 [n][ldx]
    long long ldx;
    int n, K, T, RG;       // K: columns contracted (a multiple of 8), T its tiles
    int tiles_x, tiles_y;  // row and token tiles
    int ks, tp;            // K parts of tp tiles (the last may be shorter)
    float *partial;        // ks > 1: unscaled sums [ks][n][16 RG]
    nvfp4_epi_params e;
};

constexpr int kQuad = 4 * kTileK * 2 + 64;   // LDS bytes of four tokens' 128 columns, padded (see below)

// Exact bf16 of the 8 weights of one lane of a transposed tile, dword `w` of
// its codes: two blocks of 4 contracted rows, each row with its own E4M3 scale
// (bytes of s0 and s1).
__device__ __forceinline__ u32x4 dequant_rows(u32 w, u32 s0, u32 s1)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const auto sa = __builtin_amdgcn_cvt_pk_f32_fp8((int)s0, false);
    const auto sb = __builtin_amdgcn_cvt_pk_f32_fp8((int)s0, true);
    const auto sc = __builtin_amdgcn_cvt_pk_f32_fp8((int)s1, false);
    const auto sd = __builtin_amdgcn_cvt_pk_f32_fp8((int)s1, true);
    const bf16x2 o0 = {(__bf16)(a[0] * sa[0]), (__bf16)(a[1] * sa[1])};
    const bf16x2 o1 = {(__bf16)(b[0] * sb[0]), (__bf16)(b[1] * sb[1])};
    const bf16x2 o2 = {(__bf16)(c[0] * sc[0]), (__bf16)(c[1] * sc[1])};
    const bf16x2 o3 = {(__bf16)(d[0] * sd[0]), (__bf16)(d[1] * sd[1])};
    return u32x4{__builtin_bit_cast(u32, o0), __builtin_bit_cast(u32, o1), __builtin_bit_cast(u32, o2),
                 __builtin_bit_cast(u32, o3)};
}

// LDS-direct load: lane l's 16 bytes go to `lds` + 16 l (a wave-uniform LDS
// address); offsets past the resource write zeros.  No register is written, so
// only the vmcnt wait before the barrier orders it.
__device__ __forceinline__ void load_lds_b128(u32x4 rsrc, unsigned voff, unsigned soff, unsigned lds)
{
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds) : "memory");   // M0 is reserved: the compiler keeps nothing in it
}

__device__ __forceinline__ u32x4 buffer_load_b128_s(u32x4 rsrc, unsigned voff, unsigned soff)
{
    u32x4 v;
    asm volatile("buffer_load_dwordx4 %0, %1, %2, %3 offen" : "=v"(v) : "v"(voff), "s"(rsrc), "s"(soff));
    return v;
}

// Byte address of LDS memory, as the M0 of an LDS-direct load takes it.
__device__ __forceinline__ unsigned lds_address(const void *p)
{
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// One workgroup: 4 waves x RG row groups (64 * RG weight rows) times 16 * TB
// tokens, over the steps of one K part.  A step covers 128 contracted columns:
// the tokens' slice and the scales go straight to LDS, each wave turns its own
// code tiles into MFMA operands in registers.  NB LDS buffers: the loads of
// step s + NB - 1 are issued before step s is computed.  With two buffers the
// codes are loaded into registers (LDS would leave room for one workgroup a
// compute unit only), with more they go through LDS too.  MODE: 0 linear, 1
// gated (row groups alternate gate, up), 2 transposed weight, plain output.
//
// LDS layout of the slice: token t's 16-byte chunk c (8 columns) at
//     (t / 4) * kQuad + (t % 4) * 256 + (c ^ (t % 4)) * 16.
// An operand is two 8-byte pieces, columns 32j + 4g and 32j + 16 + 4g, of 16
// tokens a read; the XOR and the 64 bytes between quads put the 16 tokens in
// 16 different 16-byte slots of the 256-byte bank row, and leave the step j
// and the token block as constant offsets.  A quad is 1 KiB of consecutive
// LDS, one LDS-direct load of a wave.
template <int RG, int TB, int NB, int MODE>
__global__ __launch_bounds__(256, 2) void nvfp4_fused_gemm_kernel(FusedGemmParams p)
{
    constexpr int BM = TB * 16;
    constexpr bool kLdsCodes = NB > 2;
    constexpr int kSlice = BM / 4 * kQuad;         // LDS bytes of a step's token slice
    constexpr int kCodes = kSlice + 4 * RG * 128;  // after the waves' scales
    constexpr int kBuf = kCodes + (kLdsCodes ? 4 * RG * 1024 : 0);
    constexpr int XL = TB;                         // quads a wave stages: BM / 4 / 4 waves
    constexpr int kLoads = XL + 1 + RG;            // loads of a step and wave
    static_assert((NB - 2) * kLoads <= 63, "vmcnt is a 6-bit field");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;

    // Tile of this workgroup.  Consecutive workgroups go to the 8 XCDs in
    // turn; each XCD takes a contiguous share of the tiles, in blocks of 8 row
    // tiles x every token tile, so that the workgroups that run on it together
    // share both operands through its L2.
    int tx, ty, part;
    {
        const int total = p.tiles_x * p.tiles_y;
        const int b = blockIdx.x, x = b & 7;
        const int per = (int)gridDim.x >> 3, rem = gridDim.x & 7;
        const int all = x * per + min(x, rem) + (b >> 3);
        part = all / total;
        const int idx = all % total;
        const int block = 8 * p.tiles_y;
        const int x0 = idx / block * 8, w = min(8, p.tiles_x - x0), at = idx % block;
        tx = x0 + at % w;
        ty = at / w;
    }
    const int rg0 = (tx * 4 + wave) * RG;
    const int tok0 = ty * BM;
    const int ntok = min(BM, p.n - tok0);
    const int nrg = max(0, min(RG, p.RG - rg0)), rgb = min(rg0, p.RG);
    const int s0 = part * p.tp, s1 = min(p.T, s0 + p.tp);
    __shared__ __align__(1024) char lds[NB][kBuf];

    // Loads past these ranges (tokens beyond n, row groups beyond RG) read
    // zeros without touching memory.
    const u32x4 xrsrc = uniform(buffer_rsrc(p.X + tok0 * p.ldx, (unsigned)(((ntok - 1) * p.ldx + p.K) * 2)));
    const u32x4 crsrc = uniform(buffer_rsrc(p.codes + (size_t)rgb * p.T * 64, (unsigned)(nrg * p.T) * 1024u));
    const u32x4 srsrc = uniform(buffer_rsrc(p.scales + (size_t)rgb * p.T * 128, (unsigned)(nrg * p.T) * 128u));
    const int ldx2 = (int)p.ldx * 2;
    const int xcol = 8 * (i ^ g);   // lane (i, g) stages chunk i ^ g of token 4 q + g
    const unsigned xoff = (unsigned)((wave * XL * 4 + g) * ldx2 + xcol * 2);
    const unsigned soff = (unsigned)((lane >> 3) * p.T * 128 + (lane & 7) * 16);
    const unsigned ldsb = lds_address(lds) + wave * XL * kQuad;
    const unsigned ldss = lds_address(lds) + kSlice + wave * RG * 128;
    const unsigned ldsc = lds_address(lds) + kCodes + wave * RG * 1024;

    u32x4 cw[RG];
    // Loads of step s into LDS buffer `b`.  Steps past the part read zeros
    // (every step issues the same loads, so that the waits can count them).
    auto issue = [&](int s, int b) {
        const unsigned buf = b * kBuf;
        const bool live = s < s1;
        const unsigned xv = live && s * kTileK + xcol < p.K ? xoff : kOutOfRange;
#pragma unroll
        for (int u = 0; u < XL; ++u)
            load_lds_b128(xrsrc, xv, (unsigned)(u * 4 * ldx2 + s * 256), ldsb + buf + u * kQuad);
        if (lane < 8 * RG)   // the wave's 128 RG bytes of scales
            load_lds_b128(srsrc, live ? soff : kOutOfRange, (unsigned)(s * 128), ldss + buf);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            const unsigned at = (unsigned)((r * p.T + s) * 1024);
            if constexpr (kLdsCodes)
                load_lds_b128(crsrc, live ? (unsigned)(lane * 16) : kOutOfRange, at, ldsc + buf + r * 1024);
            else
                cw[r] = buffer_load_b128_s(crsrc, (unsigned)(lane * 16), at);
        }
    };
    // Wait for the oldest step in flight, of NB - 1.
    auto land = [&]() {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NB - 2) * kLoads) : "memory");
        if constexpr (!kLdsCodes) {
#pragma unroll
            for (int r = 0; r < RG; ++r)
                asm volatile("" : "+v"(cw[r]));
        }
        __syncthreads();
    };

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 acc[RG][TB];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
            acc[r][tb] = zero;

    const int xa = (i >> 2) * kQuad + (i & 3) * 256 + 8 * (g & 1);
    const int x0 = xa + ((g >> 1) ^ (i & 3)) * 16, x1 = xa + (((g >> 1) | 2) ^ (i & 3)) * 16;
    const int sa = kSlice + wave * RG * 128 + (MODE == 2 ? g * 32 : i * 8);

    auto compute = [&](int b, const u32x4 *c) {
        const char *buf = lds[b];
        u32x2 sw[RG];
        if constexpr (MODE != 2) {
#pragma unroll
            for (int r = 0; r < RG; ++r)
                sw[r] = *reinterpret_cast<const u32x2 *>(buf + sa + r * 128);
        }
        bf16x8 w[2][RG];
        auto dequant = [&](auto jc, int q) {
            constexpr int j = decltype(jc)::value;
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                if constexpr (MODE == 2) {
                    const u32x2 sv = *reinterpret_cast<const u32x2 *>(buf + sa + r * 128 + 8 * j);
                    w[q][r] = __builtin_bit_cast(bf16x8, dequant_rows(c[r][j], sv[0], sv[1]));
                } else {
                    w[q][r] = __builtin_bit_cast(bf16x8, dequant_pair<(j & 1) != 0>(c[r][j], sw[r][j >> 1]));
                }
            }
        };
        dequant(std::integral_constant<int, 0>{}, 0);
        static_for<4>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (j < 3)
                dequant(std::integral_constant<int, j + 1>{}, (j + 1) & 1);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                const u32x2 lo = *reinterpret_cast<const u32x2 *>(buf + x0 + tb * 4 * kQuad + 64 * j);
                const u32x2 hi = *reinterpret_cast<const u32x2 *>(buf + x1 + tb * 4 * kQuad + 64 * j);
                const bf16x8 x = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
                for (int r = 0; r < RG; ++r)
                    acc[r][tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j & 1][r], x, acc[r][tb], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);   // one substep's operands live at a time
        });
    };

    if constexpr (kLdsCodes) {
        static_for<NB - 1>([&](auto q) { issue(s0 + decltype(q)::value, decltype(q)::value); });
        land();
        int b = 0;
        for (int s = s0; s < s1; ++s) {
            const int free = b == 0 ? NB - 1 : b - 1;   // the buffer computed from in the last step
            issue(s + NB - 1, free);
            u32x4 c[RG];
#pragma unroll
            for (int r = 0; r < RG; ++r)
                c[r] = *reinterpret_cast<const u32x4 *>(lds[b] + kCodes + (wave * RG + r) * 1024 + lane * 16);
            compute(b, c);
            land();
            b = b == NB - 1 ? 0 : b + 1;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing still writes LDS
    } else {
        issue(s0, 0);
        land();
        for (int s = s0; s < s1; ++s) {
            const int b = (s - s0) & 1;
            u32x4 c[RG];
#pragma unroll
            for (int r = 0; r < RG; ++r)
                c[r] = cw[r];
            if (s + 1 < s1)
                issue(s + 1, b ^ 1);
            compute(b, c);
            land();
        }
    }

    // A K part stores its sums as they are: nvfp4_fused_reduce_kernel adds the
    // parts in order and runs the epilogue.
    if (p.ks > 1) {
        const int pitch = p.RG * kRowsPerGroup;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            const int tok = tok0 + 16 * tb + i;
            if (tok >= p.n)
                continue;
            float *dst = p.partial + ((long long)part * p.n + tok) * pitch + rg0 * kRowsPerGroup + 4 * g;
#pragma unroll
            for (int r = 0; r < RG; ++r)
                if (rg0 + r < p.RG)
                    *reinterpret_cast<f32x4 *>(dst + r * kRowsPerGroup) = acc[r][tb];
        }
        return;
    }

    // Epilogue, one token block at a time through LDS, so that a wave writes
    // whole lines of consecutive outputs and the epilogue's code exists once.
    // Component v of lane (g, i) of acc[r][tb]: weight row 16*(rg0 + r) + 4g + v
    // of token tok0 + 16*tb + i.
    constexpr int kRows = 64 * RG, kPitch = kRows + 4;
    constexpr int kOuts = MODE == 1 ? kRows / 2 : kRows;   // outputs a token
    static_assert(16 * kPitch * 4 <= sizeof(lds), "the staged block fits the slice's LDS");
    float *stage = reinterpret_cast<float *>(lds);
    const int out0 = tx * kOuts;
#pragma unroll 1
    for (int b = 0; b < TB && tok0 + 16 * b < p.n; ++b) {
        __syncthreads();
        static_for<TB>([&](auto tc) {
            constexpr int tb = decltype(tc)::value;
            if (tb == b) {
#pragma unroll
                for (int r = 0; r < RG; ++r)
                    *reinterpret_cast<f32x4 *>(stage + i * kPitch + (wave * RG + r) * 16 + 4 * g) = acc[r][tb];
            }
        });
        __syncthreads();
#pragma unroll 1
        for (int q = tid * 4; q < 16 * kOuts; q += 1024) {
            const int t = q / kOuts, o = q % kOuts;
            const int tok = tok0 + 16 * b + t;
            if (tok >= p.n)
                break;
            if constexpr (MODE == 1) {
                const float *src = stage + t * kPitch + (o >> 4) * 32 + (o & 15);
                gated_out4(p.e, tok, out0 + o, *reinterpret_cast<const f32x4 *>(src),
                           *reinterpret_cast<const f32x4 *>(src + 16));
            } else {
                linear_out4(p.e, tok, out0 + o, *reinterpret_cast<const f32x4 *>(stage + t * kPitch + o));
            }
        }
    }
}

template <int RG, int TB, int NB>
int launch_one(FusedGemmParams p, int mode, hipStream_t stream)
{
    p.tiles_x = (p.RG + 4 * RG - 1) / (4 * RG);
    p.tiles_y = (p.n + TB * 16 - 1) / (TB * 16);
    const long long total = (long long)p.tiles_x * p.tiles_y * p.ks;
    if (total > INT32_MAX || (long long)p.T * RG * 1024 > INT32_MAX)
        return NVFP4_ERR_SHAPE;   // a wave's codes must stay within a 32-bit buffer offset
    auto k = mode == 0 ? nvfp4_fused_gemm_kernel<RG, TB, NB, 0>
                       : (mode == 1 ? nvfp4_fused_gemm_kernel<RG, TB, NB, 1> : nvfp4_fused_gemm_kernel<RG, TB, NB, 2>);
    hipLaunchKernelGGL(k, dim3((unsigned)total), dim3(256), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// Tile shapes: row groups a wave, token blocks, and what a step of one
// workgroup costs (ns) with one workgroup on its compute unit and with `full`
// of them there (per workgroup).
struct Tile {
    int rg, tb, full;
    int alone, shared;
};
constexpr Tile kTiles[] = {
    {2, 2, 2, 900, 500},
    {2, 4, 2, 1000, 600},
    {4, 8, 2, 2440, 1750},
};

}  // namespace

nvfp4_fused_gemm_plan nvfp4_plan_fused_gemm(int n, int row_groups, int K)
{
    const int T = (int)k_tiles(K);
    nvfp4_fused_gemm_plan best = {};
    double best_cost = -1;
    for (int c = 0; c < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++c) {
        const Tile &t = kTiles[c];
        if (t.tb > 2 && n <= 8 * t.tb)
            continue;   // a smaller token tile holds them
        const long long tiles = (long long)((row_groups + 4 * t.rg - 1) / (4 * t.rg)) * ((n + 16 * t.tb - 1) / (16 * t.tb));
        for (int ks = 1; ks <= 16; ++ks) {
            const int tp = (T + ks - 1) / ks;
            if (ks > 1 && (tp < 4 || (long long)(ks - 1) * tp >= T))
                continue;
            const long long units = tiles * ks, slots = 256LL * t.full;
            const long long rest = units % slots;
            const int r = (int)((rest + 255) / 256);
            double cost = (double)(units / slots) * t.full * t.shared;
            if (r == 1)
                cost += t.alone;
            else
                cost += (double)r * t.shared;
            cost = cost * tp + 3000;
            if (ks > 1)
                cost += 3000 + (double)ks * n * row_groups * 16 * 8 / 5500;
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
    case 0: return launch_one<2, 2, 3>(p, a.mode, stream);
    case 1: return launch_one<2, 4, 3>(p, a.mode, stream);
    default: return launch_one<4, 8, 2>(p, a.mode, stream);
    }
}
