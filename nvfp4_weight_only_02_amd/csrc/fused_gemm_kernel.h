// The kernel of the many-token product (fused_gemm.hip: one weight; moe_gemm.hip:
// an expert's weight for each token tile).
#ifndef NVFP4_FUSED_GEMM_KERNEL_H
#define NVFP4_FUSED_GEMM_KERNEL_H

#include "epilogue.h"
#include "fused_gemm.h"

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

// Rows grouped by expert: E weights of one shape in turn, and the rows (pairs of
// a token and an expert) in the experts' order.
struct GroupedGemmParams : FusedGemmParams {
    const int *tile;              // [1 + 2 tiles]: token tiles in use, then expert and first row of each
    const int *offset;            // [E + 1]: first row of each expert, and the end
    const int *pair;              // [rows]: the pair of each row; the token of pair q is q / k
    int k, xrows;                 // GROUP 1: X's rows are the tokens
    const float *gscale, *up_gscale;   // [E], or null (1)
    const int *xexp;              // GROUP 2: exponents of X's rows, [rows][nexp], or MODE 2: [rows]
    int *hexp;                    // MODE 1: of the rows it writes, likewise
    uint16_t *hrest;              // MODE 1: second parts of the rows (store_block_rest), or null
    int rest;                     // 0; else X holds second parts: 1, or GROUP 2 (bits below the first ones'
                                  // exponent) kRestBits.  The sums are added to the rows that are there
    int nexp;                     // an even number
    long long cstride, sstride;   // bytes of an expert's codes and scales
};

template <int GROUP>
using GemmParams = std::conditional_t<GROUP != 0, GroupedGemmParams, FusedGemmParams>;

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

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The same in fp16 (between 2^-10 and 2688: exact too), scales s.
template <int H>
__device__ __forceinline__ u32x2 dequant4(u32 w, f16x2 sa, f16x2 sb)
{
    const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * H));
    const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2 * H + 1));
    return u32x2{__builtin_bit_cast(u32, a * sa), __builtin_bit_cast(u32, b * sb)};
}

template <bool H>
__device__ __forceinline__ f16x2 half_scales2(u32 w)
{
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, H));
}

template <bool H>
__device__ __forceinline__ f32x2 scales2(u32 w)
{
    const auto s = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, H);
    return f32x2{s[0], s[1]};
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
// GROUP: 0 one weight; else a token tile takes rows of one expert, whose weight
// it multiplies.  The number of tiles in use is known on the device alone: the
// grid is the most there can be, and the workgroups past it end.  1: the tokens'
// rows of X are gathered through `pair`, by the vector offset of the LDS-direct
// loads (no copy of X in the experts' order: 168 MB of it for 1500 tokens of
// 5120 columns with 8 experts each); 2: X's rows are in the experts' order
// themselves, values between two products as fp16 (store_block), of MODE 2 with an
// exponent for a row, which its producer can know, of MODE 0 with one for each 64
// columns.  There a lane multiplies its operands by 2 to the difference from the
// row's largest exponent, at most 1 and exact down to 2^-24 of the row's largest
// value; the sums are scaled by the latter.  One bf16 number for a value adds as much
// to the result's error as the result's own rounding (2.3e-3 of the norm against
// 1.7e-3); two bf16 parts, added by a second matrix instruction, take twice the
// tokens' LDS.  E = 64, F = 1408, K = 5120, n = 1500, k = 8, the down product: 237 us,
// 220 from one bf16 number (without the lanes' products where a step's exponents are
// alike, in a second copy of the loop's body: 275, it takes too many registers);
// E = 32, F = 1280, K = 2048, n = 700, k = 4, the gradient's: 50, 68 with an exponent
// for each 64, 55 from bf16.  (fp16 has a packed product, so that the weights'
// dequantisation is shorter than to bf16.)  Of an fp32 result a second launch multiplies
// the values' second parts and adds its sums: the whole layer 1040 us for 740, 3.9e-7
// of the norm for 2.1e-4.
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
template <int RG, int TB, int RW, int KG, int MODE, int GROUP = 0>
__global__ __launch_bounds__(64 * RW * KG, RW * KG <= 4 ? 2 : 1) void nvfp4_fused_gemm_kernel(GemmParams<GROUP> p)
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
    int tok0, tok1;   // tokens of the tile, or rows in the experts' order: up to tok1 they exist
    if constexpr (GROUP) {
        // Each XCD a contiguous share of the tiles in use, row tiles fastest:
        // the workgroups that run on it together share an expert's weight.
        const int total = p.tiles_x * p.tile[0];
        const int x = blockIdx.x & 7, at = blockIdx.x >> 3, per = total >> 3, rem = total & 7;
        if (at >= per + (x < rem ? 1 : 0))
            return;
        const int idx = x * per + min(x, rem) + at;
        part = 0;
        tx = idx % p.tiles_x;
        ty = idx / p.tiles_x;
        const int expert = p.tile[1 + 2 * ty];
        tok0 = p.tile[2 + 2 * ty];
        tok1 = p.offset[expert + 1];
        p.codes += expert * p.cstride / 16;
        p.scales += expert * p.sstride;
        if (p.gscale)
            p.e.gscale = p.gscale[expert];
        if (p.up_gscale)
            p.e.up_gscale = p.up_gscale[expert];
    } else {
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
        tok0 = ty * BM;
        tok1 = p.n;
    }
    const int rg0 = (tx * RW + wave) * RG;
    const int s0 = part * p.tp, s1 = min(p.T, s0 + p.tp);
    __shared__ __align__(1024) char lds[KG][2][kBuf];

    // What lies past a resource (tokens beyond n, row groups beyond RG, and by an
    // offset past all of them the columns beyond K) is read as zeros without
    // touching memory.  Each quad of tokens has one of its own, so that a step
    // needs one vector offset for all of them.
    u32x4 xrsrc[GROUP == 1 ? 1 : XL];
    unsigned xrow[GROUP == 1 ? XL : 1];   // GROUP 1: this lane's row of each quad, in bytes
    const int xcol = 8 * (i ^ g);   // lane (i, g) stages chunk i ^ g of token g of a quad
    if constexpr (GROUP == 1) {
        xrsrc[0] = uniform(buffer_rsrc(p.X, (unsigned)(((p.xrows - 1) * p.ldx + p.K) * 2)));
#pragma unroll
        for (int u = 0; u < XL; ++u) {
            const int t = tok0 + (wave * XL + u) * 4 + g;
            // (past the last row: past the resource with any column added, see moe.hip's limit)
            xrow[u] = t < tok1 ? (unsigned)(p.pair[t] / p.k * p.ldx + xcol) * 2u : kOutOfRange;
        }
    } else {
#pragma unroll
        for (int u = 0; u < XL; ++u) {
            const int t = tok0 + (wave * XL + u) * 4, live = min(4, tok1 - t);
            xrsrc[u] = uniform(live > 0 ? buffer_rsrc(p.X + t * p.ldx, (unsigned)(((live - 1) * p.ldx + p.K) * 2))
                                        : buffer_rsrc(p.X, 0u));
        }
    }
    const int nrg = max(0, min(RG, p.RG - rg0)), rgb = min(rg0, p.RG);
    const u32x4 crsrc = uniform(buffer_rsrc(p.codes + (size_t)rgb * p.T * 64, (unsigned)(nrg * p.T) * 1024u));
    const u32x4 srsrc = uniform(buffer_rsrc(p.scales + (size_t)rgb * p.T * 128, (unsigned)(nrg * p.T) * 128u));
    const unsigned xoff = (unsigned)(g * (int)p.ldx + xcol) * 2u;
    const unsigned soff = (unsigned)((lane >> 3) * p.T * 128 + (lane & 7) * 16);
    const unsigned ldsb = lds_address(lds[kg]) + wave * XL * kQuad;
    const unsigned ldss = lds_address(lds[kg]) + kSlice + wave * RG * 128;

    // GROUP 2: the tokens of this lane's operands, and the largest exponent of each
    constexpr bool kBlocks = GROUP == 2 && MODE == 0;   // an exponent for each 64 columns
    constexpr int NE = GROUP == 2 ? TB / 2 : 1;
    const int *xexp[NE];
    int top[NE], ex[NE][2];
    __shared__ int tops[GROUP == 2 ? BM : 1];
    if constexpr (GROUP == 2) {
#pragma unroll
        for (int t = 0; t < NE; ++t)
            xexp[t] = p.xexp + (long long)min(tok0 + 32 * t + (lane & 31), tok1 - 1) * (kBlocks ? p.nexp : 1);
    }
    // (lanes l and l + 32 take every other pair of a token's, eight loads at a time)
    auto find_tops = [&]() {
        const int used = (p.K + 63) / 64, last = (used - 1) & ~1;
#pragma unroll
        for (int t = 0; t < NE; ++t)
            top[t] = kNoExponent;
        for (int t = 0; !kBlocks && t < NE; ++t)
            top[t] = *xexp[t];
        for (int b0 = 2 * (lane >> 5); kBlocks && b0 < used; b0 += 32) {
            u32x2 v[NE][8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int t = 0; t < NE; ++t)
                    v[t][q] = *reinterpret_cast<const u32x2 *>(xexp[t] + min(b0 + 4 * q, last));
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int t = 0; t < NE; ++t) {
                    top[t] = max(top[t], (int)v[t][q][0]);
                    if (min(b0 + 4 * q, last) + 1 < used)
                        top[t] = max(top[t], (int)v[t][q][1]);
                }
        }
#pragma unroll
        for (int t = 0; t < NE; ++t) {
            if constexpr (kBlocks)
                top[t] = max(top[t], __shfl_xor(top[t], 32));
            if (tid < 32)
                tops[32 * t + tid] = top[t];
        }
    };

    u32x4 cw[RG];
    auto issue = [&](int s, int b) {
        const unsigned buf = b * kBuf;
        const bool in = s * kTileK + xcol < p.K;
        if constexpr (GROUP == 1) {
#pragma unroll
            for (int u = 0; u < XL; ++u)
                load_lds_b128(xrsrc[0], in ? xrow[u] + s * (kTileK * 2) : kOutOfRange, ldsb + buf + u * kQuad);
        } else {
            const unsigned xv = in ? xoff + s * (kTileK * 2) : kOutOfRange;
#pragma unroll
            for (int u = 0; u < XL; ++u)
                load_lds_b128(xrsrc[u], xv, ldsb + buf + u * kQuad);
        }
        if (lane < 8 * RG)   // the wave's 128 RG bytes of scales
            load_lds_b128(srsrc, soff + s * 128, ldss + buf);
#pragma unroll
        for (int r = 0; r < RG; ++r)
            cw[r] = buffer_load_b128(crsrc, (unsigned)((r * p.T + s) * 1024 + lane * 16));
        if constexpr (kBlocks) {
#pragma unroll
            for (int t = 0; t < NE; ++t) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(xexp[t] + 2 * s);
                ex[t][0] = (int)v[0];
                ex[t][1] = (int)v[1];
            }
        }
    };
    auto land = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int r = 0; r < RG; ++r)
            asm volatile("" : "+v"(cw[r]));
        if constexpr (kBlocks) {
#pragma unroll
            for (int t = 0; t < NE; ++t)
                asm volatile("" : "+v"(ex[t][0]), "+v"(ex[t][1]));
        }
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

    // 32-token blocks with rows (an expert's last tile is seldom full: the others
    // would cost their matrix instructions and the power these are bound by)
    const int blocks = GROUP ? __builtin_amdgcn_readfirstlane(min(TP, (tok1 - tok0 + 31) >> 5)) : TP;
    const int h = lane >> 5, tl = lane & 31;   // column half, token of the operand
    const int xa = (tl >> 2) * kQuad + (tl & 3) * 256;
    const int x0 = xa + (h ^ (tl & 3)) * 16, x1 = xa + ((h | 2) ^ (tl & 3)) * 16;
    const int sa = kSlice + wave * RG * 128 + (g & 1) * 128 + (MODE == 2 ? h * 64 : i * 8);

    auto compute = [&](int b, const u32x4 *c, const f16x2 (*factor)[2]) {
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
        u32x4 w[2][RP][2];   // of substep j: blocks 2j and 2j + 1
        auto dequant = [&](auto jc, int q) {
            constexpr int j = decltype(jc)::value;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                u32x2 l0, l1, h0, h1;
                if constexpr (MODE == 2 && GROUP == 2) {
                    const u32x2 s = *reinterpret_cast<const u32x2 *>(buf + sa + r * 256 + 8 * j);
                    const u32x2 t = *reinterpret_cast<const u32x2 *>(buf + sa + r * 256 + 8 * j + 32);
                    l0 = dequant4<0>(lo[r][j], half_scales2<false>(s[0]), half_scales2<true>(s[0]));
                    h0 = dequant4<0>(hi[r][j], half_scales2<false>(t[0]), half_scales2<true>(t[0]));
                    l1 = dequant4<1>(lo[r][j], half_scales2<false>(s[1]), half_scales2<true>(s[1]));
                    h1 = dequant4<1>(hi[r][j], half_scales2<false>(t[1]), half_scales2<true>(t[1]));
                } else if constexpr (GROUP == 2) {
                    const f16x2 s = half_scales2<(j & 1) != 0>(sw[r][j >> 1]);
                    const f16x2 s0 = {s[0], s[0]}, s1 = {s[1], s[1]};
                    l0 = dequant4<0>(lo[r][j], s0, s0);
                    h0 = dequant4<0>(hi[r][j], s0, s0);
                    l1 = dequant4<1>(lo[r][j], s1, s1);
                    h1 = dequant4<1>(hi[r][j], s1, s1);
                } else if constexpr (MODE == 2) {
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
                w[q][r][0] = u32x4{l0[0], l0[1], h0[0], h0[1]};
                w[q][r][1] = u32x4{l1[0], l1[1], h1[0], h1[1]};
            }
        };
        dequant(std::integral_constant<int, 0>{}, 0);
        static_for<4>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (j < 3)
                dequant(std::integral_constant<int, j + 1>{}, (j + 1) & 1);
#pragma unroll
            for (int t = 0; t < TP; ++t) {
                if (GROUP && TP > 1 && t >= blocks)
                    break;
                const u32x4 a = *reinterpret_cast<const u32x4 *>(buf + x0 + t * 8 * kQuad + 64 * j);
                const u32x4 d = *reinterpret_cast<const u32x4 *>(buf + x1 + t * 8 * kQuad + 64 * j);
                if constexpr (GROUP == 2) {
                    f16x8 af = __builtin_bit_cast(f16x8, a), df = __builtin_bit_cast(f16x8, d);
                    if constexpr (kBlocks) {
                        const f16x2 f = factor[t][j >> 1];
                        const f16x8 f8 = {f[0], f[1], f[0], f[1], f[0], f[1], f[0], f[1]};
                        af *= f8;
                        df *= f8;
                    }
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w[j & 1][r][0]), af,
                                                                           acc[r][t], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w[j & 1][r][1]), df,
                                                                           acc[r][t], 0, 0, 0);
                } else {
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w[j & 1][r][0]),
                                                                            __builtin_bit_cast(bf16x8, a), acc[r][t], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w[j & 1][r][1]),
                                                                            __builtin_bit_cast(bf16x8, d), acc[r][t], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // one substep's operands live at a time
        });
    };

    if (s0 + kg < s1)
        issue(s0 + kg, 0);
    if constexpr (GROUP == 2)
        find_tops();
    land();
    int b = 0;
    for (int sb = s0; sb < s1; sb += KG, b ^= 1) {
        const int s = sb + kg;
        u32x4 c[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r)
            c[r] = cw[r];
        f16x2 factor[NE][2];
        if constexpr (kBlocks) {
#pragma unroll
            for (int t = 0; t < NE; ++t)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // (an exponent behind the last column is none: its columns are zeros)
                    const _Float16 f = (_Float16)__builtin_amdgcn_ldexpf(1.0f, min(max(ex[t][q] - top[t], -30), 0));
                    factor[t][q] = f16x2{f, f};
                }
        }
        if (s + KG < s1)
            issue(s + KG, b ^ 1);
        if (KG == 1 || s < s1)
            compute(b, c, factor);
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
    if (GROUP == 0 && KG == 1 && p.ks > 1) {
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
    for (int b = 0; b < TP && tok0 + 32 * b < tok1; ++b) {
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
        if (GROUP == 0 && KG > 1 && p.ks > 1) {
#pragma unroll 1
            for (int q = tid * 4; q < 32 * kRows; q += 4 * kThreads) {
                const int tok = tok0 + 32 * b + q / kRows, o = q % kRows;
                if (tok < p.n && tx * kRows + o < pitch)
                    *reinterpret_cast<f32x4 *>(partial + (long long)tok * pitch + tx * kRows + o) = staged(q / kRows, o);
            }
            continue;
        }
        // GROUP: sums as they are, in rows of their own (whole vectors: outputs come
        // in sixteens), or h with the activation chosen once.
        if constexpr (GROUP && MODE != 1) {
#pragma unroll 2
            for (int q = tid * 4; q < 32 * kOuts; q += 4 * kThreads) {
                const int t = q / kOuts, o = q % kOuts, tok = tok0 + 32 * b + t;
                if (tok >= tok1)
                    break;
                if (tx * kOuts + o >= p.e.N)
                    continue;
                f32x4 v = staged(t, o);
                f32x4 *dst = reinterpret_cast<f32x4 *>(static_cast<float *>(p.e.out) + (long long)tok * p.e.ldo + tx * kOuts + o);
                if constexpr (GROUP == 2) {
                    const int top = tops[32 * b + t] - p.rest;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = __builtin_amdgcn_ldexpf(p.e.gscale * v[j], top);
                } else {
                    v = p.e.gscale * v;
                }
                if (p.rest)
                    v += *dst;
                *dst = v;
            }
            continue;
        } else if constexpr (GROUP) {
            with_activation(p.e.flags & kEpiAct, [&](auto act) {
                constexpr int kTurns = 8 * kOuts / kThreads;
                static_assert(kTurns * kThreads == 8 * kOuts && kOuts % 64 == 0, "sixteen lanes: a block of 64 columns");
#pragma unroll
                for (int turn = 0; turn < kTurns; ++turn) {
                    const int q = tid * 4 + turn * 4 * kThreads;
                    const int t = q / kOuts, o = q % kOuts, tok = tok0 + 32 * b + t, r = tx * kOuts + o;
                    if (tok >= tok1)
                        break;
                    const bool in = r < p.e.N;
                    const int row = (o >> 4) * 32 + (o & 15);
                    const f32x4 z = p.e.gscale * staged(t, row), u = p.e.up_gscale * staged(t, row + 16);
                    if (p.e.preact && in) {
                        float *pre = p.e.preact + (long long)tok * p.e.ldp;
                        *reinterpret_cast<f32x4 *>(pre + gated_row(r, 0)) = z;
                        *reinterpret_cast<f32x4 *>(pre + gated_row(r, 1)) = u;
                    }
                    f32x4 y;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        y[v] = in ? activate(z[v], decltype(act)::value) * u[v] : 0.f;
                    const int exponent = block_exponent(row_max(top_bits(y)));
                    if (in) {
                        store_block(static_cast<uint16_t *>(p.e.out) + (long long)tok * p.e.ldo + r, y, exponent);
                        if (p.hrest)
                            store_block_rest(p.hrest + (long long)tok * p.e.ldo + r, y, exponent);
                        if (r % 64 == 0)
                            p.hexp[(long long)tok * p.nexp + r / 64] = exponent;
                    }
                }
            });
            continue;
        }
#pragma unroll 1
        for (int q = tid * 4; q < 32 * kOuts; q += 4 * kThreads) {
            const int t = q / kOuts, o = q % kOuts;
            const int tok = tok0 + 32 * b + t;
            if (tok >= tok1)
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

}  // namespace

#endif  // NVFP4_FUSED_GEMM_KERNEL_H
