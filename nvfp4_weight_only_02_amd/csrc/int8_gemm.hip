// Token-tiled product in 8-bit integers: many tokens.
#include "epilogue.h"
#include "int8.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct Int8GemmParams {
    const char *codes;
    const int8_t *X;
    const float *wscale, *xscale;
    long long ldx;
    int n, K, T, RG;       // T: 128-column steps
    int tiles_x, tiles_y;
    int ks, tp;
    int *partial;
    nvfp4_epi_params e;
};

constexpr int kStep = 128;              // columns of a step, bytes of a token's slice

// One workgroup: RW x TW waves of RG row groups x TB 16-token blocks, times KG
// groups that take the 128-column steps of a K part in turn and add their sums
// through LDS in the end (integers: exact in any order).  Tokens' slices go
// straight to LDS, weights to registers, both a step ahead.
//
// LDS: eight tokens' 128-byte slices are 1 KiB, one LDS-direct load of a wave;
// token t's 16-byte chunk c lies at slot c ^ (t % 8) of its slice, so that the
// lanes of an operand read (one chunk of 32 tokens) take every slot of the bank
// row in turn.
//
// The MFMA is v_mfma_i32_32x32x32_i8, weights as rows: one permlane16 swap a
// dword of two row groups' tiles gives lane (row 16 (g % 2) + i, half h = g / 2)
// columns 32 h + 0 .. 15 and 32 h + 16 .. 31 of the 64.
template <int RG, int TB, int RW, int TW, int KG>
__global__ __launch_bounds__(64 * RW * TW * KG, RW * TW * KG <= 4 ? 2 : 1) void nvfp4_int8_gemm_kernel(Int8GemmParams p)
{
    constexpr int kTokens = TB * TW * 16;
    constexpr int kThreads = 64 * RW * TW * KG;
    constexpr int kSlice = kTokens * kStep;
    constexpr int XL = kTokens / 8 / (RW * TW);   // 1 KiB loads a wave stages a step
    static_assert(XL * 8 * RW * TW == kTokens, "the waves stage the tokens evenly");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6) % (RW * TW);
    const int kg = __builtin_amdgcn_readfirstlane(tid >> 6) / (RW * TW);
    const int rw = wv % RW, tw = wv / RW;
    int tx, ty, part;
    {
        // XCD-aware: consecutive workgroups go to the 8 XCDs in turn; each takes a
        // contiguous share, in blocks of 8 row tiles x every token tile.
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
    const int rg0 = (tx * RW + rw) * RG, tok0 = ty * kTokens;
    const int s0 = part * p.tp, s1 = min(p.T, s0 + p.tp);
    constexpr int kRows = 16 * RW * RG, kPitch = kRows + 4;   // of the epilogue's staged blocks
    constexpr int kSlices = KG * 2 * kSlice, kStaged = KG * TW * 32 * kPitch * 4;
    __shared__ __align__(1024) char lds[kSlices > kStaged ? kSlices : kStaged];

    // Lane l stages token l / 8 of a group of eight, the chunk that belongs in slot l % 8.
    const int xtok = lane >> 3, xcol = 16 * ((lane & 7) ^ xtok);
    u32x4 xrsrc[XL];
#pragma unroll
    for (int u = 0; u < XL; ++u) {
        const int t = tok0 + (wv * XL + u) * 8, live = min(8, p.n - t);
        xrsrc[u] = uniform(live > 0 ? buffer_rsrc(p.X + t * p.ldx, (unsigned)((live - 1) * p.ldx + p.K))
                                    : buffer_rsrc(p.X, 0u));
    }
    const unsigned xoff = (unsigned)(xtok * (int)p.ldx + xcol);
    const unsigned ldsb = lds_address(lds) + kg * 2 * kSlice + wv * XL * 1024;
    const int nrg = max(0, min(RG, p.RG - rg0)), rgb = min(rg0, p.RG);
    const auto crsrc = resource(p.codes + (size_t)rgb * p.T * 2048, (unsigned)(nrg * p.T) * 2048u);

    u32x4 cw[RG][2];
    auto issue = [&](int s, int b) {
        const unsigned xv = s * kStep + xcol < p.K ? xoff + s * kStep : kOutOfRange;
#pragma unroll
        for (int u = 0; u < XL; ++u)
            load_lds_b128(xrsrc[u], xv, ldsb + b * kSlice + u * 1024);
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                cw[r][q] = __builtin_amdgcn_raw_buffer_load_b128(crsrc, (r * p.T + s) * 2048 + q * 1024 + lane * 16, 0, 0);
    };
    // The compiler counts the waits of the weights' loads, and places them here,
    // before the loads of the next step; it does not know of the LDS-direct ones.
    auto land = [&]() {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int r = 0; r < RG; ++r)
            asm volatile("" : "+v"(cw[r][0]), "+v"(cw[r][1]));
        __syncthreads();
    };

    constexpr int RP = RG / 2, TP = TB / 2;
    i32x16 acc[RP][TP];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
        for (int t = 0; t < TP; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[r][t][v] = 0;
    const int h = lane >> 5, tl = lane & 31;
    const int xa = (tw * TB * 16 + tl) * kStep;

    auto compute = [&](int b, const u32x4 (&c)[RG][2]) {
        const char *buf = lds + (kg * 2 + b) * kSlice;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            i32x4 w[2][RP];
#pragma unroll
            for (int r = 0; r < RP; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const auto a = __builtin_amdgcn_permlane16_swap(c[2 * r][q][j], c[2 * r + 1][q][j], false, false);
                    w[0][r][j] = (int)a[0];
                    w[1][r][j] = (int)a[1];
                }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int slot = ((4 * q + 2 * h + m) ^ (tl & 7)) * 16;
#pragma unroll
                for (int t = 0; t < TP; ++t) {
                    const i32x4 x = *reinterpret_cast<const i32x4 *>(buf + xa + t * 32 * kStep + slot);
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        acc[r][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[m][r], x, acc[r][t], 0, 0, 0);
                }
            }
        }
    };

    if (s0 + kg < s1)
        issue(s0 + kg, 0);
    land();
    int b = 0;
    for (int sb = s0; sb < s1; sb += KG, b ^= 1) {
        const int s = sb + kg;
        u32x4 c[RG][2];
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                c[r][q] = cw[r][q];
        if (s + KG < s1)
            issue(s + KG, b ^ 1);
        if (KG == 1 || s < s1)
            compute(b, c);
        land();
    }

    // Epilogue, 32 tokens at a time through LDS, so that a wave writes whole lines
    // of consecutive outputs.  Components 4q .. 4q + 3 of acc[r][t]: weight rows
    // 8q + 4h .. + 3 of row pair r, token 32 t + lane % 32.
    int *stage = reinterpret_cast<int *>(lds);
    const int pitch = p.RG * kRowsPerGroup;
    int *partial = p.partial + (long long)part * p.n * pitch;
#pragma unroll 1
    for (int blk = 0; blk < TP; ++blk) {
        __syncthreads();
        static_for<TP>([&](auto tc) {
            constexpr int t = decltype(tc)::value;
            if (t == blk) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    static_for<4>([&](auto qc) {
                        constexpr int q = 4 * decltype(qc)::value;
                        *reinterpret_cast<i32x4 *>(stage + ((kg * TW + tw) * 32 + tl) * kPitch + (rw * RG + 2 * r) * 16 +
                                                   2 * q + 4 * h) =
                            i32x4{acc[r][t][q], acc[r][t][q + 1], acc[r][t][q + 2], acc[r][t][q + 3]};
                    });
            }
        });
        __syncthreads();
#pragma unroll 1
        for (int q = tid * 4; q < TW * 32 * kRows; q += 4 * kThreads) {
            const int line = q / kRows, o = q % kRows;
            const int tok = tok0 + line / 32 * (TB * 16) + 32 * blk + line % 32;
            const int row = tx * kRows + o;
            if (tok >= p.n || row >= pitch)
                continue;
            i32x4 v = *reinterpret_cast<const i32x4 *>(stage + line * kPitch + o);
#pragma unroll
            for (int k = 1; k < KG; ++k)
                v += *reinterpret_cast<const i32x4 *>(stage + (k * TW * 32 + line) * kPitch + o);
            if (p.ks > 1) {
                *reinterpret_cast<i32x4 *>(partial + (long long)tok * pitch + row) = v;
                continue;
            }
            const float sx = p.xscale[tok];
            f32x4 z;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                z[j] = row + j < p.e.N ? (float)v[j] * sx * p.wscale[row + j] : 0.f;
            linear_out4(p.e, tok, row, z);
        }
    }
}

template <int RG, int TB, int RW, int TW, int KG>
int launch_one(Int8GemmParams p, hipStream_t stream)
{
    p.tiles_x = (p.RG + RW * RG - 1) / (RW * RG);
    p.tiles_y = (p.n + TB * TW * 16 - 1) / (TB * TW * 16);
    const long long total = (long long)p.tiles_x * p.tiles_y * p.ks;
    if (total > INT32_MAX || (long long)p.T * RG * 2048 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL((nvfp4_int8_gemm_kernel<RG, TB, RW, TW, KG>), dim3((unsigned)total), dim3(64 * RW * TW * KG), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

struct Tile {
    int rows, tokens, kg;
};
constexpr Tile kTiles[] = {{64, 32, 4}, {128, 64, 2}, {256, 256, 1}};

}  // namespace

nvfp4_int8_plan nvfp4_plan_int8(int n, int row_groups, int K)
{
    const int T = (int)k_tiles(K);
    nvfp4_int8_plan plan = {};
    plan.tile = n <= 32 ? 0 : (n <= 512 ? 1 : 2);
    const Tile &t = kTiles[plan.tile];
    const long long tiles = (long long)((row_groups * 16 + t.rows - 1) / t.rows) * ((n + t.tokens - 1) / t.tokens);
    int ks = 1;
    while (ks < 8 && tiles * ks * 2 <= 256 && T / (2 * ks) >= 4 * t.kg)
        ks *= 2;
    plan.tp = (T + ks - 1) / ks;
    plan.ks = (T + plan.tp - 1) / plan.tp;
    return plan;
}

int nvfp4_launch_int8_gemm(const nvfp4_int8_args &a, const nvfp4_int8_plan &plan, hipStream_t stream)
{
    Int8GemmParams p = {};
    p.codes = reinterpret_cast<const char *>(a.codes);
    p.X = a.X;
    p.wscale = a.wscale;
    p.xscale = a.xscale;
    p.ldx = a.ldx;
    p.n = a.n;
    p.K = a.K;
    p.T = (int)k_tiles(a.K);
    p.RG = (int)row_groups(a.N);
    p.ks = plan.ks;
    p.tp = plan.tp;
    p.partial = a.partial;
    p.e = a.epi;
    switch (plan.tile) {
    case 0: return launch_one<2, 2, 2, 1, 4>(p, stream);
    case 1: return launch_one<2, 4, 4, 1, 2>(p, stream);
    default: return launch_one<4, 8, 4, 2, 1>(p, stream);
    }
}
