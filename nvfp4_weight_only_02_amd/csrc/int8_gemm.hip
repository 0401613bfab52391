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
    int n, K, T, RG;       // T: 64-column steps
    int tiles_x, tiles_y;
    int ks, tp;
    int *partial;
    nvfp4_epi_params e;
};

constexpr int kStep = 64;               // columns of a step, bytes of a token's slice

// One workgroup: RW x TW waves of RG row groups x TB 16-token blocks, times KG
// groups that take the 64-column steps of a K part in turn and add their sums
// through LDS in the end (integers: exact in any order).  Tokens' slices go
// straight to LDS, weights to registers, both kRing - 1 steps ahead: a step is 512
// cycles of a wave's matrix instructions, less than half of what a load takes when
// all compute units load.  Every step issues the same number of loads (behind the
// last step they read nothing), so the wait for a step is the constant count of
// the newer steps' loads; the barrier after it makes the other waves' slices
// visible and frees the buffer of the step before, which the next loads go to.
//
// LDS: token t's 16-byte chunk c lies at slot c ^ (t / 4 % 4) of its 64 bytes: the
// 16 tokens of a quarter of an operand read take 16 different 16-byte slots.  1 KiB
// (16 tokens) is one LDS-direct load of a wave.
//
// The MFMA is v_mfma_i32_32x32x32_i8, weights as rows: one permlane16 swap a
// dword of two row groups' tiles gives lane (row 16 (g % 2) + i, half h = g / 2)
// columns 32 h + 0 .. 15 and 32 h + 16 .. 31 of the 64.
constexpr int kRing = 4;

template <int RG, int TB, int RW, int TW, int KG>
__global__ __launch_bounds__(64 * RW * TW * KG, RW * TW * KG <= 4 ? 2 : 1) void nvfp4_int8_gemm_kernel(Int8GemmParams p)
{
    constexpr int kTokens = TB * TW * 16;
    constexpr int kThreads = 64 * RW * TW * KG;
    constexpr int kSlice = kTokens * kStep;
    constexpr int XL = kTokens / 16 / (RW * TW);   // 1 KiB loads a wave stages a step
    static_assert(XL * 16 * RW * TW == kTokens, "the waves stage the tokens evenly");
    constexpr int kLoads = XL + RG;                // of a wave and step
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
    constexpr int kSlices = KG * kRing * kSlice, kStaged = KG * TW * 32 * kPitch * 4;
    __shared__ __align__(1024) char lds[kSlices > kStaged + kTokens * 4 ? kSlices : kStaged + kTokens * 4];

    // Lane l stages token l / 4 of sixteen, the chunk that belongs in slot l % 4.
    const int xtok = lane >> 2, xcol = 16 * ((lane & 3) ^ (xtok >> 2));
    u32x4 xrsrc[XL];
#pragma unroll
    for (int u = 0; u < XL; ++u) {
        const int t = tok0 + (wv * XL + u) * 16, live = min(16, p.n - t);
        xrsrc[u] = uniform(live > 0 ? buffer_rsrc(p.X + t * p.ldx, (unsigned)((live - 1) * p.ldx + p.K))
                                    : buffer_rsrc(p.X, 0u));
    }
    const unsigned xoff = (unsigned)(xtok * (int)p.ldx + xcol);
    const unsigned ldsb = lds_address(lds) + kg * kRing * kSlice + wv * XL * 1024;
    const int nrg = max(0, min(RG, p.RG - rg0)), rgb = min(rg0, p.RG);
    const u32x4 crsrc = uniform(buffer_rsrc(p.codes + (size_t)rgb * p.T * 1024, (unsigned)(nrg * p.T) * 1024u));

    u32x4 cw[kRing][RG];
    auto issue = [&](int s, auto bc) {
        constexpr int b = decltype(bc)::value;
        const bool in = s < s1;
        const unsigned xv = in && s * kStep + xcol < p.K ? xoff + s * kStep : kOutOfRange;
#pragma unroll
        for (int u = 0; u < XL; ++u)
            load_lds_b128(xrsrc[u], xv, ldsb + b * kSlice + u * 1024);
#pragma unroll
        for (int r = 0; r < RG; ++r)
            cw[b][r] = buffer_load_b128(crsrc, in ? (unsigned)((r * p.T + s) * 1024 + lane * 16) : kOutOfRange);
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
    const char *mine = lds + kg * kRing * kSlice + (tw * TB * 16 + tl) * kStep;
    const int slot0 = ((2 * h) ^ (tl >> 2 & 3)) * 16, slot1 = ((2 * h + 1) ^ (tl >> 2 & 3)) * 16;

    auto compute = [&](auto bc) {
        constexpr int b = decltype(bc)::value;
        i32x4 w[2][RP];
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto a = __builtin_amdgcn_permlane16_swap(cw[b][2 * r][j], cw[b][2 * r + 1][j], false, false);
                w[0][r][j] = (int)a[0];
                w[1][r][j] = (int)a[1];
            }
#pragma unroll
        for (int t = 0; t < TP; ++t) {
            const i32x4 x0 = *reinterpret_cast<const i32x4 *>(mine + b * kSlice + t * 32 * kStep + slot0);
            const i32x4 x1 = *reinterpret_cast<const i32x4 *>(mine + b * kSlice + t * 32 * kStep + slot1);
#pragma unroll
            for (int r = 0; r < RP; ++r)
                acc[r][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[0][r], x0, acc[r][t], 0, 0, 0);
#pragma unroll
            for (int r = 0; r < RP; ++r)
                acc[r][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[1][r], x1, acc[r][t], 0, 0, 0);
        }
    };

    // Step of group kg, counted from s0: kg, kg + KG, ...
    static_for<kRing - 1>([&](auto bc) { issue(s0 + kg + decltype(bc)::value * KG, bc); });
    for (int sb = s0; sb < s1; sb += kRing * KG) {
        static_for<kRing>([&](auto bc) {
            constexpr int b = decltype(bc)::value;
            constexpr int n = (b + kRing - 1) % kRing;
            if constexpr (RG == 4)
                asm volatile("s_waitcnt vmcnt(%4)" : "+v"(cw[b][0]), "+v"(cw[b][1]), "+v"(cw[b][2]), "+v"(cw[b][3])
                             : "n"((kRing - 2) * kLoads) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(%2)" : "+v"(cw[b][0]), "+v"(cw[b][1]) : "n"((kRing - 2) * kLoads) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            issue(sb + kg + (b + kRing - 1) * KG, std::integral_constant<int, n>{});
            compute(bc);   // (behind the last step: zeros)
            // every read of the slice is done before the barrier that frees it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        });
    }
    // (the loads behind the last step still write their registers)
#pragma unroll
    for (int b = 0; b < kRing; ++b)
#pragma unroll
        for (int r = 0; r < RG; ++r)
            asm volatile("s_waitcnt vmcnt(0)" : "+v"(cw[b][r])::"memory");

    // Epilogue, 32 tokens at a time through LDS, so that a wave writes whole lines
    // of consecutive outputs.  Components 4q .. 4q + 3 of acc[r][t]: weight rows
    // 8q + 4h .. + 3 of row pair r, token 32 t + lane % 32.  A thread finishes the
    // same four rows of every line it takes, so their scales and biases are loaded
    // once, the tokens' scales lie in LDS, and kBatch residuals are in flight
    // together (loaded one by one in the loop they cost 28 us a 256 x 256 tile).
    int *stage = reinterpret_cast<int *>(lds);
    float *xs = reinterpret_cast<float *>(lds + kStaged);
    const int pitch = p.RG * kRowsPerGroup;
    int *partial = p.partial + (long long)part * p.n * pitch;
    constexpr int kLines = 4 * kThreads / kRows, kTotal = TW * 32 / kLines, kBatch = kTotal < 4 ? kTotal : 4;
    static_assert(4 * kThreads % kRows == 0 && kTotal % kBatch == 0, "a thread keeps its rows");
    const int o = tid * 4 % kRows, row = tx * kRows + o, line0 = tid * 4 / kRows;
    f32x4 scale = {0.f, 0.f, 0.f, 0.f}, bias = scale;
    if (p.ks == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row + j < p.e.N) {
                scale[j] = p.wscale[row + j];
                if (p.e.bias)
                    bias[j] = load_any(p.e.bias, row + j, p.e.flags & kEpiBiasF32);
            }
    }
    __syncthreads();
    for (int t = tid; p.ks == 1 && t < kTokens; t += kThreads)
        xs[t] = tok0 + t < p.n ? p.xscale[tok0 + t] : 0.f;
    const bool vec = (p.e.flags & kEpiVec) && row + 3 < p.e.N;
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
        for (int l0 = 0; l0 < kTotal; l0 += kBatch) {
            f32x4 residual[kBatch];
#pragma unroll
            for (int l = 0; l < kBatch; ++l) {
                const int line = line0 + (l0 + l) * kLines, t = line / 32 * (TB * 16) + 32 * blk + line % 32;
                residual[l] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (p.e.residual && vec && tok0 + t < p.n)
                    residual[l] = load_any4(p.e.residual, (long long)(tok0 + t) * p.e.ldr + row, p.e.flags & kEpiResidualF32);
            }
#pragma unroll
            for (int l = 0; l < kBatch; ++l) {
                const int line = line0 + (l0 + l) * kLines, t = line / 32 * (TB * 16) + 32 * blk + line % 32;
                const int tok = tok0 + t;
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
                const float sx = xs[t];
                f32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    // (each operation rounded, as for up to 16 tokens: the same bits for any n)
                    y[j] = activate(__fadd_rn(__fmul_rn(__fmul_rn((float)v[j], sx), scale[j]), bias[j]), p.e.flags & kEpiAct);
                if (vec) {
                    if (p.e.residual)
                        y += residual[l];
                    store_any4(p.e.out, (long long)tok * p.e.ldo + row, p.e.flags & kEpiOutF32, y);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + j < p.e.N) {
                        if (p.e.residual)
                            y[j] += load_any(p.e.residual, (long long)tok * p.e.ldr + row + j, p.e.flags & kEpiResidualF32);
                        store_any(p.e.out, (long long)tok * p.e.ldo + row + j, p.e.flags & kEpiOutF32, y[j]);
                    }
            }
        }
    }
}

template <int RG, int TB, int RW, int TW, int KG>
int launch_one(Int8GemmParams p, hipStream_t stream)
{
    p.tiles_x = (p.RG + RW * RG - 1) / (RW * RG);
    p.tiles_y = (p.n + TB * TW * 16 - 1) / (TB * TW * 16);
    const long long total = (long long)p.tiles_x * p.tiles_y * p.ks;
    if (total > INT32_MAX || (long long)p.T * RG * 1024 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL((nvfp4_int8_gemm_kernel<RG, TB, RW, TW, KG>), dim3((unsigned)total), dim3(64 * RW * TW * KG), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

struct Tile {
    int rows, tokens, kg;
};
constexpr Tile kTiles[] = {{64, 32, 4}, {128, 64, 2}, {256, 256, 1}, {256, 128, 1}, {128, 128, 1}, {128, 128, 2}, {256, 64, 1}, {128, 64, 1}, {256, 64, 2}};

}  // namespace

nvfp4_int8_plan nvfp4_plan_int8(int n, int row_groups, int K)
{
    const int T = 2 * (int)k_tiles(K);
    nvfp4_int8_plan plan = {};
    plan.tile = n <= 32 ? 0 : (n <= 256 ? 1 : 3);
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
    p.T = 2 * (int)k_tiles(a.K);
    p.RG = (int)row_groups(a.N);
    p.ks = plan.ks;
    p.tp = plan.tp;
    p.partial = a.partial;
    p.e = a.epi;
    switch (plan.tile) {
    case 0: return launch_one<2, 2, 2, 1, 4>(p, stream);
    case 1: return launch_one<2, 4, 4, 1, 2>(p, stream);
    case 2: return launch_one<4, 8, 4, 2, 1>(p, stream);
    case 3: return launch_one<4, 8, 4, 1, 1>(p, stream);
    case 4: return launch_one<4, 4, 2, 2, 1>(p, stream);
    case 5: return launch_one<4, 4, 2, 2, 2>(p, stream);
    case 6: return launch_one<4, 4, 4, 1, 1>(p, stream);
    case 7: return launch_one<2, 4, 4, 1, 1>(p, stream);
    default: return launch_one<4, 4, 4, 1, 2>(p, stream);
    }
}
