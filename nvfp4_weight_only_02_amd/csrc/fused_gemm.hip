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

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Exact bf16 (an E2M1 code times an E4M3 scale has at most 6 significant bits)
// of the codes in half H of w: 2 bytes, low nibble first, scales s.
template <int H>
__device__ __forceinline__ u32x2 dequant4(u32 w, f32x2 sa, f32x2 sb)
{
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2 * H);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2 * H + 1);
    const bf16x2 x = {(__bf16)(a[0] * sa[0]), (__bf16)(a[1] * sa[1])};
    const bf16x2 y = {(__bf16)(b[0] * sb[0]), (__bf16)(b[1] * sb[1])};
    return u32x2{__builtin_bit_cast(u32, x), __builtin_bit_cast(u32, y)};
}

template <bool H>
__device__ __forceinline__ f32x2 scales2(u32 w)
{
    const auto s = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, H);
    return f32x2{s[0], s[1]};
}

// LDS-direct load: lane l's 16 bytes go to `lds` + 16 l (a wave-uniform LDS
// address); offsets past the resource write zeros (the scalar offset stays 0:
// the range check need not include it).  No register is written, so only the
// vmcnt wait before the barrier orders it.  M0 is reserved, the compiler keeps
// nothing in it; one wait state separates its write from the load.
__device__ __forceinline__ void load_lds_b128(u32x4 rsrc, unsigned off, unsigned lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(off), "s"(rsrc), "s"(lds) : "memory");
}

// Byte address of LDS memory, as the M0 of an LDS-direct load takes it.
__device__ __forceinline__ unsigned lds_address(const void *p)
{
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// One workgroup: RW waves x RG row groups (16 * RW * RG weight rows) times 16 *
// TB tokens, over the steps of one K part, which KG groups of RW waves take in
// turn and whose sums they add through LDS in the end, in group order.  A step
// covers 128 contracted columns: the tokens' slice and the scales go straight
// to LDS, each wave turns its own code tiles into MFMA operands in registers.
// The loads of step s + 1 are issued before step s is computed and waited for
// after it: two LDS buffers, which leave room for two workgroups a compute unit
// at the largest tile (a third buffer, with the codes through LDS as well,
// measured no faster at 17 .. 64 tokens: 16384 x 5120, n = 24: 17.0 against
// 16.8 us; weights alone two steps ahead 1 .. 4% slower at n = 17 .. 512: the
// small tiles are bound by issue).  MODE: 0 linear, 1 gated (row groups
// alternate gate, up), 2 transposed weight, plain output.
//
// LDS layout of the slice: token t's 16-byte chunk c (8 columns) at
//     (t / 4) * kQuad + (t % 4) * 256 + (c ^ (t % 4)) * 16.
// An operand is a chunk of 32 tokens; the XOR and the 64 bytes between quads
// put 16 of them in 16 different 16-byte slots of the 256-byte bank row, and
// leave the substep and the token block as constant offsets.  A quad is 1 KiB
// of consecutive LDS, one LDS-direct load of a wave.
//
// The MFMA is v_mfma_f32_32x32x16_bf16 (rows x tokens): two row groups fill
// its 32 rows.  A code tile's lane (i, g) holds row i's columns 16b + 4g + e;
// one v_permlane16_swap a code dword of two row groups gives every lane (row
// 16 (g % 2) + i, half h = g / 2) the columns 16b + 8h + 0 .. 3 in one dword
// and + 4 .. 7 in the other: the 8 consecutive columns of a chunk, so that the
// tokens' operand is one 16-byte read.  Against the 16-row form (whose operand
// is two 8-byte reads) it halves the MFMA and LDS instructions that the
// dequantisation has to share the issue slots with.
template <int RG, int TB, int RW, int KG, int MODE>
__global__ __launch_bounds__(64 * RW * KG, RW * KG <= 4 ? 2 : 1) void nvfp4_fused_gemm_kernel(FusedGemmParams p)
{
    constexpr int BM = TB * 16;
    constexpr int kThreads = 64 * RW * KG;
    constexpr int kSlice = BM / 4 * kQuad;         // LDS bytes of a step's token slice
    constexpr int kBuf = kSlice + RW * RG * 128;   // and of the waves' scales
    constexpr int XL = BM / 4 / RW;                // quads a wave stages
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % RW;
    const int kg = __builtin_amdgcn_readfirstlane(tid >> 6) / RW;
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
    const int rg0 = (tx * RW + wave) * RG;
    const int tok0 = ty * BM;
    const int s0 = part * p.tp, s1 = min(p.T, s0 + p.tp);
    __shared__ __align__(1024) char lds[KG][2][kBuf];

    // What lies past a resource (tokens beyond n, row groups beyond RG, and by an
    // offset past all of them the columns beyond K) is read as zeros without
    // touching memory.  Each quad of tokens has one of its own, so that a step
    // needs one vector offset for all of them.
    u32x4 xrsrc[XL];
#pragma unroll
    for (int u = 0; u < XL; ++u) {
        const int t = tok0 + (wave * XL + u) * 4, live = min(4, p.n - t);
        xrsrc[u] = uniform(live > 0 ? buffer_rsrc(p.X + t * p.ldx, (unsigned)(((live - 1) * p.ldx + p.K) * 2))
                                    : buffer_rsrc(p.X, 0u));
    }
    const int nrg = max(0, min(RG, p.RG - rg0)), rgb = min(rg0, p.RG);
    const u32x4 crsrc = uniform(buffer_rsrc(p.codes + (size_t)rgb * p.T * 64, (unsigned)(nrg * p.T) * 1024u));
    const u32x4 srsrc = uniform(buffer_rsrc(p.scales + (size_t)rgb * p.T * 128, (unsigned)(nrg * p.T) * 128u));
    const int xcol = 8 * (i ^ g);   // lane (i, g) stages chunk i ^ g of token g of a quad
    const unsigned xoff = (unsigned)(g * (int)p.ldx + xcol) * 2u;
    const unsigned soff = (unsigned)((lane >> 3) * p.T * 128 + (lane & 7) * 16);
    const unsigned ldsb = lds_address(lds[kg]) + wave * XL * kQuad;
    const unsigned ldss = lds_address(lds[kg]) + kSlice + wave * RG * 128;

    u32x4 cw[RG];
    auto issue = [&](int s, int b) {
        const unsigned buf = b * kBuf;
        const unsigned xv = s * kTileK + xcol < p.K ? xoff + s * (kTileK * 2) : kOutOfRange;
#pragma unroll
        for (int u = 0; u < XL; ++u)
            load_lds_b128(xrsrc[u], xv, ldsb + buf + u * kQuad);
        if (lane < 8 * RG)   // the wave's 128 RG bytes of scales
            load_lds_b128(srsrc, soff + s * 128, ldss + buf);
#pragma unroll
        for (int r = 0; r < RG; ++r)
            cw[r] = buffer_load_b128(crsrc, (unsigned)((r * p.T + s) * 1024 + lane * 16));
    };
    auto land = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int r = 0; r < RG; ++r)
            asm volatile("" : "+v"(cw[r]));
        __syncthreads();
    };

    constexpr int RP = RG / 2, TP = TB / 2;   // 32-row and 32-token blocks
    f32x16 acc[RP][TP];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
        for (int t = 0; t < TP; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[r][t][v] = 0.f;

    const int h = lane >> 5, tl = lane & 31;   // column half, token of the operand
    const int xa = (tl >> 2) * kQuad + (tl & 3) * 256;
    const int x0 = xa + (h ^ (tl & 3)) * 16, x1 = xa + ((h | 2) ^ (tl & 3)) * 16;
    const int sa = kSlice + wave * RG * 128 + (g & 1) * 128 + (MODE == 2 ? h * 64 : i * 8);

    auto compute = [&](int b, const u32x4 *c) {
        const char *buf = lds[kg][b];
        u32 lo[RP][4], hi[RP][4];   // columns 8h + 0..3 and 4..7 of each block
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto q = __builtin_amdgcn_permlane16_swap(c[2 * r][j], c[2 * r + 1][j], false, false);
                lo[r][j] = q[0];
                hi[r][j] = q[1];
            }
        u32x2 sw[RP];
        if constexpr (MODE != 2) {
#pragma unroll
            for (int r = 0; r < RP; ++r)
                sw[r] = *reinterpret_cast<const u32x2 *>(buf + sa + r * 256);
        }
        bf16x8 w[2][RP][2];   // of substep j: blocks 2j and 2j + 1
        auto dequant = [&](auto jc, int q) {
            constexpr int j = decltype(jc)::value;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                u32x2 l0, l1, h0, h1;
                if constexpr (MODE == 2) {
                    // a scale for each contracted row: of columns 8h + 0..3, and 4..7
                    const u32x2 s = *reinterpret_cast<const u32x2 *>(buf + sa + r * 256 + 8 * j);
                    const u32x2 t = *reinterpret_cast<const u32x2 *>(buf + sa + r * 256 + 8 * j + 32);
                    l0 = dequant4<0>(lo[r][j], scales2<false>(s[0]), scales2<true>(s[0]));
                    h0 = dequant4<0>(hi[r][j], scales2<false>(t[0]), scales2<true>(t[0]));
                    l1 = dequant4<1>(lo[r][j], scales2<false>(s[1]), scales2<true>(s[1]));
                    h1 = dequant4<1>(hi[r][j], scales2<false>(t[1]), scales2<true>(t[1]));
                } else {
                    const f32x2 s = scales2<(j & 1) != 0>(sw[r][j >> 1]);   // of blocks 2j and 2j + 1
                    const f32x2 s0 = {s[0], s[0]}, s1 = {s[1], s[1]};
                    l0 = dequant4<0>(lo[r][j], s0, s0);
                    h0 = dequant4<0>(hi[r][j], s0, s0);
                    l1 = dequant4<1>(lo[r][j], s1, s1);
                    h1 = dequant4<1>(hi[r][j], s1, s1);
                }
                w[q][r][0] = __builtin_bit_cast(bf16x8, u32x4{l0[0], l0[1], h0[0], h0[1]});
                w[q][r][1] = __builtin_bit_cast(bf16x8, u32x4{l1[0], l1[1], h1[0], h1[1]});
            }
        };
        dequant(std::integral_constant<int, 0>{}, 0);
        static_for<4>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (j < 3)
                dequant(std::integral_constant<int, j + 1>{}, (j + 1) & 1);
#pragma unroll
            for (int t = 0; t < TP; ++t) {
                const bf16x8 a = *reinterpret_cast<const bf16x8 *>(buf + x0 + t * 8 * kQuad + 64 * j);
                const bf16x8 d = *reinterpret_cast<const bf16x8 *>(buf + x1 + t * 8 * kQuad + 64 * j);
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j & 1][r][0], a, acc[r][t], 0, 0, 0);
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j & 1][r][1], d, acc[r][t], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);   // one substep's operands live at a time
        });
    };

    if (s0 + kg < s1)
        issue(s0 + kg, 0);
    land();
    int b = 0;
    for (int sb = s0; sb < s1; sb += KG, b ^= 1) {
        const int s = sb + kg;
        u32x4 c[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r)
            c[r] = cw[r];
        if (s + KG < s1)
            issue(s + KG, b ^ 1);
        if (KG == 1 || s < s1)
            compute(b, c);
        land();
    }

    // Components 4q .. 4q + 3 of acc[r][t]: weight rows 8q + 4h .. + 3 of the
    // 32 of row pair r, token 32 t + lane % 32.
    auto sums = [&](const f32x16 &c, auto qc) {
        constexpr int q = 4 * decltype(qc)::value;
        return f32x4{c[q], c[q + 1], c[q + 2], c[q + 3]};
    };
    const int pitch = p.RG * kRowsPerGroup;
    float *partial = p.partial + (long long)part * p.n * pitch;

    // A K part stores its sums as they are: nvfp4_fused_reduce_kernel adds the
    // parts in order and runs the epilogue.
    if (KG == 1 && p.ks > 1) {
#pragma unroll
        for (int t = 0; t < TP; ++t) {
            const int tok = tok0 + 32 * t + tl;
            if (tok >= p.n)
                continue;
            float *dst = partial + (long long)tok * pitch + rg0 * kRowsPerGroup + 4 * h;
#pragma unroll
            for (int r = 0; r < RP; ++r)
                static_for<4>([&](auto qc) {
                    constexpr int q = decltype(qc)::value;
                    if (rg0 + 2 * r + q / 2 < p.RG)
                        *reinterpret_cast<f32x4 *>(dst + r * 32 + 8 * q) = sums(acc[r][t], qc);
                });
        }
        return;
    }

    // Epilogue, one token block at a time through LDS, so that a wave writes
    // whole lines of consecutive outputs and the epilogue's code exists once.
    constexpr int kRows = 16 * RW * RG, kPitch = kRows + 4;
    constexpr int kOuts = MODE == 1 ? kRows / 2 : kRows;   // outputs a token
    static_assert(KG * 32 * kPitch * 4 <= sizeof(lds), "the staged block fits the slices' LDS");
    float *stage = reinterpret_cast<float *>(lds);
    auto staged = [&](int t, int row) {
        const float *src = stage + t * kPitch + row;
        f32x4 v = *reinterpret_cast<const f32x4 *>(src);
#pragma unroll
        for (int k = 1; k < KG; ++k)
            v += *reinterpret_cast<const f32x4 *>(src + k * 32 * kPitch);
        return v;
    };
#pragma unroll 1
    for (int b = 0; b < TP && tok0 + 32 * b < p.n; ++b) {
        __syncthreads();
        static_for<TP>([&](auto tc) {
            constexpr int t = decltype(tc)::value;
            if (t == b) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    static_for<4>([&](auto qc) {
                        *reinterpret_cast<f32x4 *>(stage + (kg * 32 + tl) * kPitch + (wave * RG + 2 * r) * 16 +
                                                   8 * decltype(qc)::value + 4 * h) = sums(acc[r][t], qc);
                    });
            }
        });
        __syncthreads();
        if (KG > 1 && p.ks > 1) {
#pragma unroll 1
            for (int q = tid * 4; q < 32 * kRows; q += 4 * kThreads) {
                const int tok = tok0 + 32 * b + q / kRows, o = q % kRows;
                if (tok < p.n && tx * kRows + o < pitch)
                    *reinterpret_cast<f32x4 *>(partial + (long long)tok * pitch + tx * kRows + o) = staged(q / kRows, o);
            }
            continue;
        }
#pragma unroll 1
        for (int q = tid * 4; q < 32 * kOuts; q += 4 * kThreads) {
            const int t = q / kOuts, o = q % kOuts;
            const int tok = tok0 + 32 * b + t;
            if (tok >= p.n)
                break;
            if constexpr (MODE == 1) {
                const int row = (o >> 4) * 32 + (o & 15);
                gated_out4(p.e, tok, tx * kOuts + o, staged(t, row), staged(t, row + 16));
            } else {
                linear_out4(p.e, tok, tx * kOuts + o, staged(t, o));
            }
        }
    }
}

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
