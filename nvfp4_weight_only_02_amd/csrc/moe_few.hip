// The expert layer for up to 16 tokens in two launches: gate and up projections
// of every chosen expert with the activation, then the down projections with
// the sum over each token's experts.
//
// Which experts are chosen is known on the device alone, so every workgroup
// reads the n k choices and builds the list of the distinct ones (ascending, so
// that the list does not depend on the order of the choices).  An expert's
// weights are read once however many tokens it has.
//
// Every sum's order depends on the layer's sizes and k alone: a dot product's on
// the columns, a token's over its experts on its own slots.  So a token's result
// does not depend on the others of the batch.
#include "epilogue.h"
#include "moe.h"

namespace {

constexpr int kFewTokens = 16;
constexpr int kMaxSlots = 32;                        // experts of a token
constexpr int kMaxPairs = kFewTokens * kMaxSlots;
constexpr int kMaxExperts = 1024;
constexpr int kThreads = kWaves * 64;
static_assert(kMaxPairs <= kThreads, "a thread for each pair");

struct MoeFewParams {
    const char *gu_codes, *gu_scales, *d_codes, *d_scales;
    const float *gscale;          // [3][E]
    const uint16_t *X;
    const int *experts;           // [n][k]
    const float *weights;         // [n][k]
    uint16_t *h;                  // [n k][128 Td], columns of a tile in the lanes' order
    int ldx, n, k, E, F, K, act;
    int T, Td, P;                 // 128-column tiles of K and of F, pairs of row groups of a gated weight
    int ws, tpw;                  // waves that share an expert's down projection, and the tiles of each
    nvfp4_epi_params e;
};

// The choices of the batch in LDS.
struct Routes {
    int expert[kMaxPairs];                   // of each pair, -1 if none
    unsigned short first[kMaxPairs];         // the token's first pair with the same expert
    unsigned short list[kMaxPairs];          // the distinct experts, ascending
    unsigned tokens[kMaxPairs];              // of each of them: its tokens, a bit each
    unsigned short pair[kMaxPairs][kFewTokens];   // and the pair of its j-th token
    u32 bits[kMaxExperts / 32];
    int count;
};

// All threads of the workgroup; a barrier ends it.
__device__ __forceinline__ void build_routes(Routes &r, const MoeFewParams &p, bool pairs)
{
    const int tid = threadIdx.x, nk = p.n * p.k, words = (p.E + 31) / 32;
    int e = -1;
    if (tid < nk) {
        e = p.experts[tid];
        if (e < 0 || e >= p.E)
            e = -1;
        r.expert[tid] = e;
        r.tokens[tid] = 0;
    }
    if (tid < words)
        r.bits[tid] = 0;
    __syncthreads();
    const int t = tid / p.k;
    bool first = e >= 0;
    if (first) {
        int f = tid;
        for (int q = tid - 1; q >= t * p.k; --q)
            if (r.expert[q] == e)
                f = q;
        first = f == tid;
        r.first[tid] = (unsigned short)f;
        if (first)
            atomicOr(&r.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int a = 0;
    if (first) {
        for (int w = 0; w < e >> 5; ++w)
            a += __popc(r.bits[w]);
        a += __popc(r.bits[e >> 5] & ((1u << (e & 31)) - 1));
        r.list[a] = (unsigned short)e;
        if (pairs)
            atomicOr(&r.tokens[a], 1u << t);
    }
    if (tid == kThreads - 1) {
        int c = 0;
        for (int w = 0; w < words; ++w)
            c += __popc(r.bits[w]);
        r.count = c;
    }
    __syncthreads();
    if (pairs) {
        if (first)
            r.pair[a][__popc(r.tokens[a] & ((1u << t) - 1))] = (unsigned short)tid;
        __syncthreads();
    }
}

// Raw buffer over [base, base + bytes), for loads whose waits the compiler counts.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void *base, unsigned bytes)
{
    const unsigned long long a = (unsigned long long)base;
    const unsigned lo = __builtin_amdgcn_readfirstlane((int)(u32)a), hi = __builtin_amdgcn_readfirstlane((int)(u32)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)((unsigned long long)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), kBufferWord3);
}

constexpr unsigned kBehind = 0x40000000u;   // added to an offset: behind any h
constexpr int kNt = 2;   // read once: streamed past the caches

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, unsigned off, int more = 0)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)(off + more), 0, 0);
}

__device__ __forceinline__ u32x4 load16_nt(__amdgpu_buffer_rsrc_t r, unsigned off)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kNt);
}

__device__ __forceinline__ u32x2 load8_nt(__amdgpu_buffer_rsrc_t r, unsigned off)
{
    return __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, kNt);
}

// One 16-row x 128-column tile: acc[v] += sum over its 8 blocks of scale times
// the product of the block's codes with the operand x.
template <int NV>
__device__ __forceinline__ void tile_product(f32x4 &acc, const u32x4 c, const u32x2 s, const u32x2 *x)
{
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 p1 = zero, p2 = zero;
    float s1 = 0.f, s2 = 0.f;
    float sc[kBlocksPerTile];
    static_for<4>([&](auto hc) {
        constexpr int h = decltype(hc)::value;
        const auto f2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)s[h >> 1], (h & 1) != 0);
        sc[2 * h] = f2[0];
        sc[2 * h + 1] = f2[1];
    });
#pragma unroll
    for (int b = 0; b < kBlocksPerTile; ++b) {
        const u32 cw = c[b >> 1];
        const u32 lo = fp4x2_to_bf16x2(cw, (b & 1) * 2), hi = fp4x2_to_bf16x2(cw, (b & 1) * 2 + 1);
        const f32x4 pr = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, x[b]),
                                                                   __builtin_bit_cast(s16x4, u32x2{lo, hi}), zero, 0, 0, 0);
        if (b >= 2) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                acc[v] = __builtin_fmaf(s2, p2[v], acc[v]);
        }
        p2 = p1;
        s2 = s1;
        p1 = pr;
        s1 = sc[b];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
        acc[v] = __builtin_fmaf(s1, p1[v], __builtin_fmaf(s2, p2[v], acc[v]));
}

// Position of column r of a 128-column tile in the order of the lanes' operands:
// lane group g of block b takes columns 16 b + 4 g + 0 .. 3, eight blocks in turn.
__device__ __forceinline__ int operand_order(int r)
{
    return (r & ~127) + 32 * ((r >> 2) & 3) + 4 * ((r >> 4) & 7) + (r & 3);
}

// Gate and up: the row groups of all chosen experts as one sequence, gate and up
// in turn, cut into equal shares for the workgroups; the eight waves split K.
// All tokens' rows stay in registers as MFMA operands (rows that an expert was
// not chosen for cost nothing: the matrix instruction has 16 rows anyway), and
// the weights stream past them, a row group ahead.
template <int MT, int NV>
__global__ __launch_bounds__(kThreads) void nvfp4_moe_up_kernel(MoeFewParams p)
{
    constexpr int W = kWaves;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    __shared__ Routes routes;
    __shared__ f32x4 part[kSlots][W][64];

    // Lane (i, g) loads 16-byte chunks (block 2j + g % 2, half g / 2) of its
    // token's tile; a swap between lane groups then leaves columns 4g .. 4g + 3
    // of both blocks.
    const int tok = 4 * (i & 3) + (i >> 2);
    u32x2 x[MT][kBlocksPerTile];
    {
        const auto xr = resource(p.X, (unsigned)(((p.n - 1) * p.ldx + p.K) * 2));
        u32x4 raw[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = (wave + W * t) * kTileK + 32 * j + 16 * (g & 1) + 8 * (g >> 1);
                raw[t][j] = load16(xr, tok < p.n && col < p.K ? (unsigned)(tok * p.ldx + col) * 2u : kOutOfRange);
            }
        build_routes(routes, p, false);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 r = raw[t][j];
                const auto a = __builtin_amdgcn_permlane16_swap(r[0], r[2], false, false);
                const auto b = __builtin_amdgcn_permlane16_swap(r[1], r[3], false, false);
                x[t][2 * j] = u32x2{a[0], b[0]};
                x[t][2 * j + 1] = u32x2{a[1], b[1]};
            }
    }

    const int units = __builtin_amdgcn_readfirstlane(routes.count) * p.P;
    const int per = units / (int)gridDim.x, rem = units % (int)gridDim.x, wg = blockIdx.x;
    const int u0 = wg * per + min(wg, rem), u1 = u0 + per + (wg < rem ? 1 : 0);
    if (u0 >= u1)
        return;
    const long long rows = 2LL * p.P;   // row groups of an expert
    const unsigned tb = p.T * 1024u, sb = p.T * 128u;
    u32x4 c[MT];
    u32x2 s[MT];
    // Of gate (half 0) or up row group of a unit; nothing where there is none.
    auto codes_of = [&](int u, int half, bool in) {
        const long long rg = (long long)routes.list[u / p.P] * rows + 2 * (u % p.P) + half;
        return resource(p.gu_codes + rg * tb, in ? tb : 0u);
    };
    auto scales_of = [&](int u, int half, bool in) {
        const long long rg = (long long)routes.list[u / p.P] * rows + 2 * (u % p.P) + half;
        return resource(p.gu_scales + rg * sb, in ? sb : 0u);
    };
    const unsigned coff = (unsigned)(wave * 1024 + lane * 16), soff = (unsigned)(wave * 128 + i * 8);
    {
        const auto cr = codes_of(u0, 0, true), sr = scales_of(u0, 0, true);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            s[t] = load8_nt(sr, soff + t * (W * 128));
            c[t] = load16_nt(cr, coff + t * (W * 1024));
        }
    }
    for (int b0 = u0; b0 < u1; b0 += kSlots / 2) {
        const int b1 = min(b0 + kSlots / 2, u1);
        for (int q = 2 * b0; q < 2 * b1; ++q) {
            const int nu = min((q + 1) >> 1, u1 - 1);
            const bool more = (q + 1) >> 1 < u1;
            const auto cr = codes_of(nu, (q + 1) & 1, more), sr = scales_of(nu, (q + 1) & 1, more);
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            static_for<MT>([&](auto tc) {
                constexpr int t = decltype(tc)::value;
                tile_product<NV>(acc, c[t], s[t], x[t]);
                s[t] = load8_nt(sr, soff + t * (W * 128));
                c[t] = load16_nt(cr, coff + t * (W * 1024));
                __builtin_amdgcn_sched_barrier(0);
            });
            part[q - 2 * b0][wave][lane] = acc;
        }
        __syncthreads();
        // unit v: component v % NV (token 4v + g) of pair v / NV of the batch
        for (int v = wave; v < (b1 - b0) * NV; v += W) {
            const int u = b0 + v / NV, slot = 2 * (v / NV), comp = v % NV;
            const float *src = reinterpret_cast<const float *>(&part[slot][0][lane]) + comp;
            float gate = src[0], up = src[W * 256];
#pragma unroll
            for (int w = 1; w < W; ++w) {
                gate += src[w * 256];
                up += src[(W + w) * 256];
            }
            const int e = routes.list[u / p.P], pr = u % p.P;
            const int t = 4 * comp + g;
            const float hv = activate(p.gscale[e] * gate, p.act) * (p.gscale[p.E + e] * up);
            if (t < p.n) {
                for (int sl = 0; sl < p.k; ++sl) {
                    if (routes.expert[t * p.k + sl] != e)
                        continue;
                    uint16_t *row = p.h + (long long)(t * p.k + sl) * (p.Td * kTileK);
                    row[operand_order(pr * 16 + i)] = f32_to_bf16_bits(hv);
                    // the columns behind the last one, up to a whole tile
                    if (pr == p.P - 1)
                        for (int r = p.P * 16 + i; r < p.Td * kTileK; r += 16)
                            row[operand_order(r)] = 0;
                    break;
                }
            }
        }
        if (b1 < u1)
            __syncthreads();
    }
}

// Down: a workgroup has 16 outputs of every token, its waves an expert each in
// turn (ws of them share one expert's F where a token has fewer experts than
// that takes); the rows of an expert's own tokens are its operand.  The sums of
// all pairs meet in LDS, and a thread adds those of its token, weighted, in slot
// order.
template <int TP>
__global__ __launch_bounds__(kThreads) void nvfp4_moe_down_kernel(MoeFewParams p)
{
    constexpr int W = kWaves;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int rg = blockIdx.x, nk = p.n * p.k;
    __shared__ Routes routes;
    __shared__ float mix[kMaxPairs];
    extern __shared__ float sums[];   // [n k][ws][16]
    build_routes(routes, p, true);
    if (tid < nk) {
        const int e = routes.expert[tid];
        mix[tid] = e < 0 ? 0.f : p.weights[tid] * p.gscale[2 * p.E + e];
    }
    const int units = __builtin_amdgcn_readfirstlane(routes.count) * p.ws;
    const long long groups = p.K / kRowsPerGroup;
    const unsigned tb = p.Td * 1024u, sb = p.Td * 128u;
    const auto hr = resource(p.h, (unsigned)(nk * p.Td * kTileK * 2));

    // This wave's units, an expert or its part each, in steps of TP tiles; the
    // operands of a step are loaded while the one before is computed.
    u32x4 c[TP], h[TP][4];
    u32x2 s[TP];
    int unit = wave, tile = 0, end = 0, cnt = 0;   // of the step that is loaded next
    unsigned row = kOutOfRange;                    // this lane's operand row in h, bytes
    auto open = [&](int u) {
        unit = u;
        if (u >= units)
            return;
        const int a = u / p.ws;
        tile = u % p.ws * p.tpw;
        end = min(p.Td, tile + p.tpw);
        cnt = __builtin_amdgcn_readfirstlane(__popc(routes.tokens[a]));
        const int j = 4 * (i & 3) + (i >> 2);
        row = j < cnt ? (unsigned)(routes.pair[a][j] * p.Td * kTileK + 32 * g) * 2u : kOutOfRange;
    };
    // A unit's tiles end where its resources do: what lies behind reads zeros.
    auto codes_of = [&](int u) {
        const long long at = u < units ? (long long)routes.list[u / p.ws] * groups + rg : 0;
        return resource(p.d_codes + at * tb, u < units ? end * 1024u : 0u);
    };
    auto scales_of = [&](int u) {
        const long long at = u < units ? (long long)routes.list[u / p.ws] * groups + rg : 0;
        return resource(p.d_scales + at * sb, u < units ? end * 128u : 0u);
    };
    auto load = [&](__amdgpu_buffer_rsrc_t cr, __amdgpu_buffer_rsrc_t sr, auto tc) {
        constexpr int t = decltype(tc)::value;
        s[t] = load8_nt(sr, (unsigned)((tile + t) * 128 + i * 8));
        c[t] = load16_nt(cr, (unsigned)((tile + t) * 1024 + lane * 16));
        const unsigned at = row + (tile + t) * (kTileK * 2) + (tile + t < end ? 0u : kBehind);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[t][q] = load16(hr, at, 16 * q);
    };
    open(wave);
    if (unit < units) {
        {
            const auto cr = codes_of(unit), sr = scales_of(unit);
            static_for<TP>([&](auto tc) { load(cr, sr, tc); });
        }
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        while (true) {
            const int done = unit, had = cnt;
            tile += TP;
            const bool last = tile >= end;
            if (last)
                open(unit + W);
            const auto cr = codes_of(unit), sr = scales_of(unit);
            static_for<TP>([&](auto tc) {
                constexpr int t = decltype(tc)::value;
                const u32x2 x[8] = {{h[t][0][0], h[t][0][1]}, {h[t][0][2], h[t][0][3]}, {h[t][1][0], h[t][1][1]},
                                    {h[t][1][2], h[t][1][3]}, {h[t][2][0], h[t][2][1]}, {h[t][2][2], h[t][2][3]},
                                    {h[t][3][0], h[t][3][1]}, {h[t][3][2], h[t][3][3]}};
                if (had <= 4)
                    tile_product<1>(acc, c[t], s[t], x);
                else
                    tile_product<4>(acc, c[t], s[t], x);
                load(cr, sr, tc);
                __builtin_amdgcn_sched_barrier(0);
            });
            if (last) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int j = 4 * v + g;
                    if (j < had)
                        sums[(routes.pair[done / p.ws][j] * p.ws + done % p.ws) * 16 + i] = acc[v];
                    acc[v] = 0.f;
                }
            }
            if (unit >= units)
                break;
        }
    }
    __syncthreads();
    if (tid < p.n * 16) {
        const int t = tid >> 4, r = tid & 15;
        float y = 0.f;
        for (int sl = 0; sl < p.k; ++sl) {
            const int q = t * p.k + sl;
            if (routes.expert[q] < 0)
                continue;
            const float *src = sums + routes.first[q] * p.ws * 16 + r;
            float o = src[0];
            for (int w = 1; w < p.ws; ++w)
                o += src[w * 16];
            y = __builtin_fmaf(mix[q], o, y);
        }
        linear_out(p.e, t, rg * 16 + r, y);
    }
}

typedef void (*UpKernel)(MoeFewParams);

template <int NV, int... MT>
UpKernel pick_up(int mt, std::integer_sequence<int, MT...>)
{
    UpKernel k = nullptr;
    ((mt == MT + 1 ? (void)(k = nvfp4_moe_up_kernel<MT + 1, NV>) : (void)0), ...);
    return k;
}

// Waves that share an expert's down projection: a function of the layer's k, so
// that the order of a sum is.
int down_split(int k, int Td)
{
    int ws = 1;
    while (ws < kWaves && k * ws < kWaves && 2 * ws <= Td)
        ws *= 2;
    return ws;
}

}  // namespace

bool nvfp4_moe_is_few(int n, int K)
{
    return n <= kFewTokens && K <= kWaves * kMaxTilesPerWave * kTileK;
}

size_t nvfp4_moe_few_bytes(int n, int k, int F)
{
    return (size_t)n * k * k_tiles(F) * kTileK * 2;
}

int nvfp4_launch_moe_few(const nvfp4_moe_few_args &a, hipStream_t stream)
{
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    MoeFewParams p = {};
    p.gu_codes = reinterpret_cast<const char *>(a.gu_codes);
    p.gu_scales = reinterpret_cast<const char *>(a.gu_scales);
    p.d_codes = reinterpret_cast<const char *>(a.d_codes);
    p.d_scales = reinterpret_cast<const char *>(a.d_scales);
    p.gscale = a.gscale;
    p.X = a.X;
    p.experts = a.experts;
    p.weights = a.weights;
    p.h = a.h;
    p.ldx = a.ldx;
    p.n = a.n;
    p.k = a.k;
    p.E = a.E;
    p.F = a.F;
    p.K = a.K;
    p.act = a.act;
    p.T = (int)k_tiles(a.K);
    p.Td = (int)k_tiles(a.F);
    p.P = a.F / kRowsPerGroup;
    p.ws = down_split(a.k, p.Td);
    p.tpw = (p.Td + p.ws - 1) / p.ws;
    p.e = a.epi;
    const int mt = (p.T + kWaves - 1) / kWaves;
    constexpr auto mts = std::make_integer_sequence<int, kMaxTilesPerWave>{};
    const UpKernel up = a.n <= 4 ? pick_up<1>(mt, mts) : (a.n <= 8 ? pick_up<2>(mt, mts) : pick_up<4>(mt, mts));
    const long long most = (long long)(a.n * a.k < a.E ? a.n * a.k : a.E) * p.P;
    hipLaunchKernelGGL(up, dim3((unsigned)(most < cus ? most : cus)), dim3(kThreads), 0, stream, p);
    if (hipGetLastError() != hipSuccess)
        return NVFP4_ERR_LAUNCH;
    hipLaunchKernelGGL(nvfp4_moe_down_kernel<4>, dim3((unsigned)(a.K / kRowsPerGroup)), dim3(kThreads),
                       (unsigned)(a.n * a.k * p.ws * 16 * sizeof(float)), stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}
