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
//
// The large tiles have the weights in LDS too (WL), where the waves that share row
// groups read them once.  16384 x 5120, n = 4096: 327 us on 256 x 256, 2.1 POP/s,
// bound by the matrix instructions and power (a library product: 2.2).
constexpr int kRing = 4;

// a * b, a + b, rounded: the compiler makes no fma of them.  A result has the same
// bits for any n, and the form for up to 16 tokens rounds each operation.
__device__ __forceinline__ float mul_rounded(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

__device__ __forceinline__ float add_rounded(float a, float b)
{
#pragma clang fp contract(off)
    return a + b;
}

template <int RG, int TB, int RW, int TW, int KG, bool WL>
__global__ __launch_bounds__(64 * RW * TW * KG, RW * TW * KG <= 4 ? 2 : 1) void nvfp4_int8_gemm_kernel(Int8GemmParams p)
{
    constexpr int kTokens = TB * TW * 16;
    constexpr int kThreads = 64 * RW * TW * KG;
    constexpr int kCodes = WL ? RW * RG * 1024 : 0;   // LDS bytes of a step's weights
    constexpr int kTok = kTokens * kStep, kSlice = kTok + kCodes;
    constexpr int WLL = RW * RG / (RW * TW);          // 1 KiB loads of weights a wave stages
    constexpr int XL = kTokens / 16 / (RW * TW);   // 1 KiB loads a wave stages a step
    static_assert(XL * 16 * RW * TW == kTokens, "the waves stage the tokens evenly");
    constexpr int kLoads = XL + (WL ? WLL : RG);   // of a wave and step
    static_assert(WL || RG == 2, "the waits name a step's registers");
    static_assert(!WL || WLL * TW == RG, "the waves stage the weights evenly");
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
    // (WL: of all the workgroup's row groups, which the waves stage between them)
    const int first = WL ? tx * RW * RG : rg0;
    const int nrg = max(0, min(WL ? RW * RG : RG, p.RG - first)), rgb = min(first, p.RG);
    const u32x4 crsrc = uniform(buffer_rsrc(p.codes + (size_t)rgb * p.T * 1024, (unsigned)(nrg * p.T) * 1024u));

    u32x4 cw[WL ? 1 : kRing][WL ? 1 : RG];
    const unsigned ldsw = lds_address(lds) + kg * kRing * kSlice + kTok + wv * WLL * 1024;
    auto issue = [&](int s, auto bc) {
        constexpr int b = decltype(bc)::value;
        const bool in = s < s1;
        const unsigned xv = in && s * kStep + xcol < p.K ? xoff + s * kStep : kOutOfRange;
#pragma unroll
        for (int u = 0; u < XL; ++u)
            load_lds_b128(xrsrc[u], xv, ldsb + b * kSlice + u * 1024);
        if constexpr (WL) {
#pragma unroll
            for (int u = 0; u < WLL; ++u)
                load_lds_b128(crsrc, in ? (unsigned)(((wv * WLL + u) * p.T + s) * 1024 + lane * 16) : kOutOfRange,
                              ldsw + b * kSlice + u * 1024);
        } else {
#pragma unroll
            for (int r = 0; r < RG; ++r)
                cw[b][r] = buffer_load_b128(crsrc, in ? (unsigned)((r * p.T + s) * 1024 + lane * 16) : kOutOfRange);
        }
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
    // lane (row 16 (g % 2) + i of a pair of row groups, half h): chunks 2h and 2h + 1 of the row
    const char *codes = lds + kg * kRing * kSlice + kTok + rw * RG * 1024 + (lane >> 4 & 1) * 1024 + (32 * h + (lane & 15)) * 16;
    const int slot0 = ((2 * h) ^ (tl >> 2 & 3)) * 16, slot1 = ((2 * h + 1) ^ (tl >> 2 & 3)) * 16;

    // Operands of one half (m) of a step: 16 of each lane's 32 columns.
    struct Half {
        i32x4 w[RP], x[TP];
    };
    auto tokens_of = [&](auto bc, int m, Half &f) {
        constexpr int b = decltype(bc)::value;
#pragma unroll
        for (int t = 0; t < TP; ++t)
            f.x[t] = *reinterpret_cast<const i32x4 *>(mine + b * kSlice + t * 32 * kStep + (m ? slot1 : slot0));
    };
    auto codes_of = [&](auto bc, int m, Half &f) {
        constexpr int b = decltype(bc)::value;
#pragma unroll
        for (int r = 0; r < RP; ++r)
            f.w[r] = *reinterpret_cast<const i32x4 *>(codes + b * kSlice + r * 2048 + m * 256);
    };
    auto swap_codes = [&](auto bc, Half &f0, Half &f1) {
        if constexpr (!WL) {
            constexpr int b = decltype(bc)::value;
#pragma unroll
            for (int r = 0; r < RP; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const auto a = __builtin_amdgcn_permlane16_swap(cw[b][2 * r][j], cw[b][2 * r + 1][j], false, false);
                    f0.w[r][j] = (int)a[0];
                    f1.w[r][j] = (int)a[1];
                }
        }
    };
    auto multiply = [&](const Half &f) {
#pragma unroll
        for (int t = 0; t < TP; ++t)
#pragma unroll
            for (int r = 0; r < RP; ++r)
                acc[r][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[r], f.x[t], acc[r][t], 0, 0, 0);
    };
    // Waits for a step's loads, kRing - 2 newer ones under way.
    auto landed = [&](auto bc) {
        constexpr int b = decltype(bc)::value;
        if constexpr (WL)
            asm volatile("s_waitcnt vmcnt(%0)" :: "n"((kRing - 2) * kLoads) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(%2)" : "+v"(cw[b][0]), "+v"(cw[b][1]) : "n"((kRing - 2) * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // Step of group kg, counted from s0: kg, kg + KG, ...  The waves run in step
    // from barrier to barrier, so each half's operands are read while the half
    // before is multiplied, across the barrier too (read and multiplied in turn,
    // 768 of LDS and 1024 cycles of matrix instructions a 256 x 256 step added up).
    Half f0, f1, g1;
    static_for<kRing - 1>([&](auto bc) { issue(s0 + kg + decltype(bc)::value * KG, bc); });
    landed(std::integral_constant<int, 0>{});
    swap_codes(std::integral_constant<int, 0>{}, f0, f1);
    if constexpr (WL)
        codes_of(std::integral_constant<int, 0>{}, 0, f0);
    tokens_of(std::integral_constant<int, 0>{}, 0, f0);
    issue(s0 + kg + (kRing - 1) * KG, std::integral_constant<int, kRing - 1>{});
    for (int sb = s0; sb < s1; sb += kRing * KG) {
        static_for<kRing>([&](auto bc) {
            constexpr int b = decltype(bc)::value;
            constexpr std::integral_constant<int, (b + 1) % kRing> nc{};
            if constexpr (WL)
                codes_of(bc, 1, f1);
            tokens_of(bc, 1, f1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f0);   // (behind the last step: zeros)
            __builtin_amdgcn_sched_barrier(0);
            // every read of this step's slice is done before the barrier that frees it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            landed(nc);
            if constexpr (WL)
                codes_of(nc, 0, f0);
            else
                swap_codes(nc, f0, g1);
            tokens_of(nc, 0, f0);
            issue(sb + kg + (b + kRing) * KG, bc);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f1);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!WL) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    f1.w[r] = g1.w[r];
            }
        });
    }
    // (the loads behind the last step still write their registers)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (!WL) {
#pragma unroll
        for (int b = 0; b < kRing; ++b)
#pragma unroll
            for (int r = 0; r < RG; ++r)
                asm volatile("" : "+v"(cw[b][r]));
    }

    // Epilogue, 32 tokens at a time through LDS, so that a wave writes whole lines
    // of consecutive outputs.  Components 4q .. 4q + 3 of acc[r][t]: weight rows
    // 8q + 4h .. + 3 of row pair r, token 32 t + lane % 32.  A thread finishes the
    // same four rows of every line it takes, so their scales and biases are loaded
    // once and the tokens' scales lie in LDS; kBatch residuals are in flight
    // together, and the activation is chosen once.  (Bound by its instructions:
    // loads and choices made for each four outputs cost 28 us a 256 x 256 tile, the
    // activation's choice alone 17.)
    int *stage = reinterpret_cast<int *>(lds);
    float *xs = reinterpret_cast<float *>(lds + kStaged);
    const int pitch = p.RG * kRowsPerGroup;
    int *partial = p.partial + (long long)part * p.n * pitch;
    constexpr int kLines = 4 * kThreads / kRows, kTotal = TW * 32 / kLines, kBatch = kTotal < 4 ? kTotal : 4;
    static_assert(4 * kThreads % kRows == 0 && kTotal % kBatch == 0, "a thread keeps its rows");
    const int o = tid * 4 % kRows, row = tx * kRows + o, line0 = tid * 4 / kRows;
    f32x4 scale = {0.f, 0.f, 0.f, 0.f}, bias = {-0.f, -0.f, -0.f, -0.f};   // (adding -0 changes nothing)
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
        // The sums of line l of this thread, whose token is t of the tile's.
        auto token_of = [&](int l) {
            const int line = line0 + l * kLines;
            return line / 32 * (TB * 16) + 32 * blk + line % 32;
        };
        auto staged = [&](int l) {
            const int *src = stage + (line0 + l * kLines) * kPitch + o;
            i32x4 v = *reinterpret_cast<const i32x4 *>(src);
#pragma unroll
            for (int k = 1; k < KG; ++k)
                v += *reinterpret_cast<const i32x4 *>(src + k * TW * 32 * kPitch);
            return v;
        };
        if (p.ks > 1) {
#pragma unroll 2
            for (int l = 0; l < kTotal; ++l) {
                const int tok = tok0 + token_of(l);
                if (tok < p.n && row < pitch)
                    *reinterpret_cast<i32x4 *>(partial + (long long)tok * pitch + row) = staged(l);
            }
            continue;
        }
        with_activation(p.e.flags & kEpiAct, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
#pragma unroll 1
            for (int l0 = 0; l0 < kTotal; l0 += kBatch) {
                f32x4 residual[kBatch];
#pragma unroll
                for (int l = 0; l < kBatch; ++l) {
                    const int tok = tok0 + token_of(l0 + l);
                    residual[l] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (p.e.residual && vec && tok < p.n)
                        residual[l] = load_any4(p.e.residual, (long long)tok * p.e.ldr + row, p.e.flags & kEpiResidualF32);
                }
#pragma unroll
                for (int l = 0; l < kBatch; ++l) {
                    const int t = token_of(l0 + l), tok = tok0 + t;
                    const i32x4 v = staged(l0 + l);
                    const float sx = xs[t];
                    f32x4 y;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] = activate(add_rounded(mul_rounded(mul_rounded((float)v[j], sx), scale[j]), bias[j]), kAct);
                    if (tok >= p.n)
                        continue;
                    if (vec) {
                        if (p.e.residual) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                y[j] = add_rounded(y[j], residual[l][j]);
                        }
                        store_any4(p.e.out, (long long)tok * p.e.ldo + row, p.e.flags & kEpiOutF32, y);
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (row + j < p.e.N) {
                            if (p.e.residual)
                                y[j] = add_rounded(y[j], load_any(p.e.residual, (long long)tok * p.e.ldr + row + j, p.e.flags & kEpiResidualF32));
                            store_any(p.e.out, (long long)tok * p.e.ldo + row + j, p.e.flags & kEpiOutF32, y[j]);
                        }
                }
            }
        });
    }
}

template <int RG, int TB, int RW, int TW, int KG, bool WL>
int launch_one(Int8GemmParams p, hipStream_t stream)
{
    p.tiles_x = (p.RG + RW * RG - 1) / (RW * RG);
    p.tiles_y = (p.n + TB * TW * 16 - 1) / (TB * TW * 16);
    const long long total = (long long)p.tiles_x * p.tiles_y * p.ks;
    if (total > INT32_MAX || (long long)p.T * RG * (WL ? RW : 1) * 1024 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL((nvfp4_int8_gemm_kernel<RG, TB, RW, TW, KG, WL>), dim3((unsigned)total), dim3(64 * RW * TW * KG), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// Tile shapes: weight rows, tokens, K groups, workgroups that fit a compute unit,
// and what an iteration (a step of every K group) costs (ns) with one workgroup on
// its unit and, per workgroup, with the unit full; a workgroup's start and
// epilogue, in iterations; the uneven end of a grid of several rounds, in
// workgroups a unit.
struct Tile {
    int rows, tokens, kg, full;
    double alone, shared, start, tail;
};
constexpr Tile kTiles[] = {
    {64, 32, 4, 4, 375, 336, 3.1, 0},
    {128, 64, 2, 2, 163, 362, 4.6, 0.47},
    {128, 64, 1, 4, 219, 197, 4.9, 0},
    {128, 128, 1, 2, 244, 274, 8.0, 0.65},
    {256, 128, 1, 1, 338, 411, 12.5, 0.91},
    {256, 256, 1, 1, 411, 656, 11.5, 1.05},
};
constexpr int kParts[] = {1, 2, 3, 4, 6, 8};
constexpr double kBaseNs = 1500, kReduceNs = 7500, kReduceSumNs = 8e-4;   // a launch, the second one, a partial sum

}  // namespace

// The tile and part count of least modelled time, fitted to 99 shapes (640 ..
// 20000 rows, K 1024 .. 17408, n 17 .. 4096) x 6 tiles x every part count measured
// on MI355X with weights that mostly come from HBM: the choice is within 2% of the
// best measured one on average, 22% at worst.  Both sides of some choices (us):
//   640 x 4096     n = 96     64 x 32 8.8; 128 x 64 11.0, 128 x 128 12.5
//   5120 x 17408   n = 64     128 x 64 in 6 parts 27.6; 128 x 128 29.8, 64 x 32 in 3 34.1
//   5120 x 6144    n = 300    128 x 64, 2 groups 25.2; 128 x 128 26.3, 128 x 64 26.7
//   8192 x 2048    n = 300    128 x 64 14.4; 2 groups 17.0, 128 x 128 17.0, 64 x 32 20.3
//   5120 x 17408   n = 300    256 x 128 in 4 parts 50; 128 x 128 in 2 52, 256 x 256 in 6 57
//   2048 x 8192    n = 2048   128 x 128 45; 128 x 64 48, 256 x 128 in 2 parts 53
//   16384 x 5120   n = 1000   256 x 256 91; 256 x 128 101, 128 x 128 112
//   16384 x 5120   n = 4096   256 x 256 338; 256 x 128 379, 128 x 64 490
nvfp4_int8_plan nvfp4_plan_int8(int n, int row_groups, int K)
{
    const int T = 2 * (int)k_tiles(K);
    nvfp4_int8_plan best = {};
    double best_cost = -1;
    for (int c = 0; c < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++c) {
        const Tile &t = kTiles[c];
        const long long tiles = ((long long)row_groups * kRowsPerGroup + t.rows - 1) / t.rows * ((n + t.tokens - 1) / t.tokens);
        for (const int parts : kParts) {
            const int tp = (T + parts - 1) / parts, ks = (T + tp - 1) / tp;
            if (parts > 1 && (tp < 4 || tiles >= 2048))
                break;
            const long long units = tiles * ks, resident = (units + 255) / 256;
            const double per = resident <= t.full ? (double)resident : units * (1.0 / 256) + t.tail;
            const double step = per * t.shared > t.alone ? per * t.shared : t.alone;
            double cost = ((tp + t.kg - 1) / t.kg + t.start) * step + kBaseNs;
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

void nvfp4_int8_tile(int tile, int *rows, int *tokens, int *k_groups)
{
    const Tile &t = kTiles[tile];
    *rows = t.rows;
    *tokens = t.tokens;
    *k_groups = t.kg;
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
    case 0: return launch_one<2, 2, 2, 1, 4, false>(p, stream);
    case 1: return launch_one<2, 4, 4, 1, 2, false>(p, stream);
    case 2: return launch_one<2, 4, 4, 1, 1, false>(p, stream);
    case 3: return launch_one<4, 4, 2, 2, 1, true>(p, stream);
    case 4: return launch_one<4, 4, 4, 2, 1, true>(p, stream);
    default: return launch_one<4, 8, 4, 2, 1, true>(p, stream);
    }
}
