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

// One workgroup: 4 waves x RG row groups (64 * RG weight rows) times 16 * TB
// tokens.  A step covers 128 contracted columns: the tokens' slice goes
// through LDS, each wave turns its own code tiles into MFMA operands in
// registers.  MODE: 0 linear, 1 gated (row groups alternate gate, up), 2
// transposed weight, plain output.
//
// LDS layout of the slice: token t's 16-byte chunk c (8 columns) at
//     (t / 4) * kQuad + (t % 4) * 256 + (c ^ (t % 4)) * 16.
// An operand is two 8-byte pieces, columns 32j + 4g and 32j + 16 + 4g, of 16
// tokens a read; the XOR and the 64 bytes between quads put the 16 tokens in
// 16 different 16-byte slots of the 256-byte bank row, and leave the step j
// and the token block as constant offsets.
template <int RG, int TB, int MODE>
__global__ __launch_bounds__(256) void nvfp4_fused_gemm_kernel(FusedGemmParams p)
{
    constexpr int BM = TB * 16;
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int rg0 = (blockIdx.x * 4 + wave) * RG;
    const int tok0 = blockIdx.y * BM;
    __shared__ __align__(16) char xs[BM / 4 * kQuad < 16 * (64 * RG + 4) * 4 ? 16 * (64 * RG + 4) * 4 : BM / 4 * kQuad];

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 acc[RG][TB];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
            acc[r][tb] = zero;

    const char *xa = xs + (i >> 2) * kQuad + (i & 3) * 256 + 8 * (g & 1);
    const char *x0 = xa + (((g >> 1)) ^ (i & 3)) * 16;
    const char *x1 = xa + (((g >> 1) | 2) ^ (i & 3)) * 16;

    for (int s = 0; s < p.T; ++s) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < TB; ++u) {
            const int t = (tid >> 4) + 16 * u, c = tid & 15;
            const int k = s * kTileK + 8 * c;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (tok0 + t < p.n && k < p.K)
                v = *reinterpret_cast<const u32x4 *>(p.X + (tok0 + t) * p.ldx + k);
            *reinterpret_cast<u32x4 *>(xs + (t >> 2) * kQuad + (t & 3) * 256 + (c ^ (t & 3)) * 16) = v;
        }
        u32x4 cw[RG];
        u32x4 sa[RG], sb[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            const long long tile = (long long)min(rg0 + r, p.RG - 1) * p.T + s;   // rows past the end: any tile, not stored
            cw[r] = p.codes[tile * 64 + lane];
            if constexpr (MODE == 2) {
                const u32x4 *src = reinterpret_cast<const u32x4 *>(p.scales + tile * 128 + g * 32);
                sa[r] = src[0];
                sb[r] = src[1];
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(p.scales + tile * 128 + i * 8);
                sa[r][0] = v[0];
                sa[r][1] = v[1];
            }
        }
        __syncthreads();
        static_for<4>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            bf16x8 w[RG];
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                if constexpr (MODE == 2) {
                    const u32x4 sv = j < 2 ? sa[r] : sb[r];
                    w[r] = __builtin_bit_cast(bf16x8, dequant_rows(cw[r][j], sv[2 * (j & 1)], sv[2 * (j & 1) + 1]));
                } else {
                    w[r] = __builtin_bit_cast(bf16x8, dequant_pair<(j & 1) != 0>(cw[r][j], sa[r][j >> 1]));
                }
            }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                const u32x2 lo = *reinterpret_cast<const u32x2 *>(x0 + tb * 4 * kQuad + 64 * j);
                const u32x2 hi = *reinterpret_cast<const u32x2 *>(x1 + tb * 4 * kQuad + 64 * j);
                const bf16x8 x = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
                for (int r = 0; r < RG; ++r)
                    acc[r][tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[r], x, acc[r][tb], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);   // one substep's operands live at a time
        });
    }

    // Epilogue, one token block at a time through LDS, so that a wave writes
    // whole lines of consecutive outputs and the epilogue's code exists once.
    // Component v of lane (g, i) of acc[r][tb]: weight row 16*(rg0 + r) + 4g + v
    // of token tok0 + 16*tb + i.
    constexpr int kRows = 64 * RG, kPitch = kRows + 4;
    constexpr int kOuts = MODE == 1 ? kRows / 2 : kRows;   // outputs a token
    static_assert(16 * kPitch * 4 <= sizeof(xs), "the staged block fits the slice's LDS");
    float *stage = reinterpret_cast<float *>(xs);
    const int out0 = blockIdx.x * kOuts;
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

template <int RG, int TB, int MODE>
int launch_one(const FusedGemmParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.RG + 4 * RG - 1) / (4 * RG)), (unsigned)((p.n + TB * 16 - 1) / (TB * 16)));
    hipLaunchKernelGGL((nvfp4_fused_gemm_kernel<RG, TB, MODE>), grid, dim3(256), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

template <int MODE>
int launch_mode(const FusedGemmParams &p, hipStream_t stream)
{
    if (p.n <= 32)
        return launch_one<2, 2, MODE>(p, stream);
    return launch_one<2, 4, MODE>(p, stream);
}

}  // namespace

int nvfp4_launch_fused_gemm(const nvfp4_fused_gemm_args &a, hipStream_t stream)
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
    switch (a.mode) {
    case 0: return launch_mode<0>(p, stream);
    case 1: return launch_mode<1>(p, stream);
    default: return launch_mode<2>(p, stream);
    }
}
