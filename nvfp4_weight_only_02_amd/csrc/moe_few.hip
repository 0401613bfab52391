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
    uint16_t *h;                  // [n k][Td][2][128]: the two bf16 parts of a value (bf16_rest),
                                  // columns of a tile in the lanes' order
    int ldx, n, k, E, F, K, act;
    int T, Td, P;                 // 128-column tiles of K and of F, pairs of row groups of a gated weight
    int ws, tpw;                  // parts of an expert's F in the down projection, and the tiles of each
    int rows;                     // outputs of a workgroup of the down projection
    nvfp4_epi_params e;
};

// The choices of the batch in LDS.
struct Routes {
    int expert[kMaxPairs];                   // of each pair, -1 if none
    unsigned short list[kMaxPairs];          // the distinct experts, ascending
    u32 bits[kMaxExperts / 32];
    int count;
};

// The expert of thread tid's pair, -1 if none.
__device__ __forceinline__ int load_choice(const MoeFewParams &p)
{
    int e = -1;
    if (threadIdx.x < (unsigned)(p.n * p.k))
        e = p.experts[threadIdx.x];
    return e;
}

// All threads of the workgroup, e from load_choice; a barrier ends it.  Returns
// the place of this thread's expert in the list if it is the first pair of its
// token with that expert, else -1; *first is that pair.
__device__ __forceinline__ int build_routes(Routes &r, const MoeFewParams &p, int e, int *first)
{
    const int tid = threadIdx.x, nk = p.n * p.k, words = (p.E + 31) / 32;
    if (e < 0 || e >= p.E)
        e = -1;
    if (tid < nk)
        r.expert[tid] = e;
    if (tid < words)
        r.bits[tid] = 0;
    __syncthreads();
    int f = tid;
    if (e >= 0) {
        for (int q = tid - 1; q >= tid / p.k * p.k; --q)
            if (r.expert[q] == e)
                f = q;
        if (f == tid)
            atomicOr(&r.bits[e >> 5], 1u << (e & 31));
    }
    *first = f;
    __syncthreads();
    int a = -1;
    if (e >= 0 && f == tid) {
        a = __popc(r.bits[e >> 5] & ((1u << (e & 31)) - 1));
        for (int w = 0; w < e >> 5; ++w)
            a += __popc(r.bits[w]);
        r.list[a] = (unsigned short)e;
    }
    if (tid == kMaxPairs - 1) {
        int c = 0;
        for (int w = 0; w < words; ++w)
            c += __popc(r.bits[w]);
        r.count = c;
    }
    __syncthreads();
    return a;
}

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
// Each tile's columns come twice: the values' first parts, then the second ones.
__device__ __forceinline__ int operand_order(int r)
{
    return 2 * (r & ~127) + 32 * ((r >> 2) & 3) + 4 * ((r >> 4) & 7) + (r & 3);
}

// Gate and up: the row groups of all chosen experts as one sequence, gate and up
// in turn, cut into equal shares for the workgroups; the eight waves split K.
// All tokens' rows stay in registers as MFMA operands (rows that an expert was
// not chosen for cost nothing: the matrix instruction has 16 rows anyway), and
// the weights stream past them, a row group ahead.  Bound by the weights' bytes and
// the start: E = 64, F = 1408, K = 5120, k = 8: 15.7 us for n = 1 (65 MB), 79 for 16
// (450 MB, 5.7 TB/s).
template <int MT, int NV>
__global__ __launch_bounds__(kThreads) void nvfp4_moe_up_kernel(MoeFewParams p)
{
    constexpr int W = kWaves;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    __shared__ Routes routes;
    __shared__ f32x4 part[kSlots][W][64];

    const int choice = load_choice(p);
    int first;
    build_routes(routes, p, choice, &first);
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
    // Lane (i, g) loads 16-byte chunks (block 2j + g % 2, half g / 2) of its
    // token's tile; a swap between lane groups then leaves columns 4g .. 4g + 3
    // of both blocks.
    const int tok = 4 * (i & 3) + (i >> 2);
    u32x4 raw[MT][4];
    const auto xr = resource(p.X, (unsigned)(((p.n - 1) * p.ldx + p.K) * 2));
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = (wave + W * t) * kTileK + 32 * j + 16 * (g & 1) + 8 * (g >> 1);
            raw[t][j] = load16(xr, tok < p.n && col < p.K ? (unsigned)(tok * p.ldx + col) * 2u : kOutOfRange);
        }
    __builtin_amdgcn_sched_barrier(0);
    {
        const auto cr = codes_of(u0, 0, true), sr = scales_of(u0, 0, true);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            s[t] = load8_nt(sr, soff + t * (W * 128));
            c[t] = load16_nt(cr, coff + t * (W * 1024));
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    u32x2 x[MT][kBlocksPerTile];
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
                    uint16_t *row = p.h + (long long)(t * p.k + sl) * (p.Td * 2 * kTileK);
                    const uint16_t high = f32_to_bf16_bits(hv);
                    row[operand_order(pr * 16 + i)] = high;
                    row[operand_order(pr * 16 + i) + kTileK] = f32_to_bf16_bits(bf16_rest(hv, high));
                    // the columns behind the last one, up to a whole tile
                    if (pr == p.P - 1)
                        for (int r = p.P * 16 + i; r < p.Td * kTileK; r += 16)
                            row[operand_order(r)] = row[operand_order(r) + kTileK] = 0;
                    break;
                }
            }
        }
        if (b1 < u1)
            __syncthreads();
    }
}

// A piece of the down projection of 16 outputs: up to four tokens of an expert,
// over a part of F.
struct Unit {
    unsigned short expert, part;
    unsigned short tile, end;
    unsigned short pair[4];       // 0xFFFF: none
};
constexpr int kNoPair = 0xFFFF;

// Down: a workgroup has p.rows outputs of every token, in NW windows of 16 rows
// (of which the last may use fewer, and which need not begin with a row group).
// Its waves take units from a queue: an expert with up to four of its tokens (an
// expert with more has several units, whose weights come from cache after the
// first; four tokens, whose values are two bf16 parts each, cost the matrix
// instruction two components and 2 KiB of LDS a tile), or a part of its F where a
// token has few experts.  A unit's tiles of
// weights go to registers and its tokens' rows straight to LDS, D tiles ahead:
// always the same loads a tile in the same order, so that the wait for a tile is
// the constant count of the newer ones, across the units' ends too.  The sums of
// all pairs meet in LDS, and a thread adds those of its token, weighted, in slot
// order.
//
// Rows are dealt out evenly over the compute units, in fours (64 bytes of each
// column quarter of a tile): a unit reads little faster than its share of the
// memory's bandwidth (24 KB/us were measured with most others done, against 25 for
// 6.4 TB/s over 256), so a second workgroup on some of them would be what the
// launch waits for.  13 experts 400 x 1040, n = 7: 10.2 us with 16 rows a
// workgroup, 7.5 with 8; E = 64, F = 1408, K = 5120, k = 8, n = 16 (225 MB): 59 us,
// 53 with one bf16 number for a value; the codes alone take 42.
template <int NW, int D>
__global__ __launch_bounds__(kThreads, 4) void nvfp4_moe_down_kernel(MoeFewParams p)
{
    constexpr int W = kWaves;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * p.rows, nk = p.n * p.k;
    __shared__ Routes routes;
    __shared__ unsigned tokens[kMaxPairs];        // of each expert of the list: its tokens, a bit each
    __shared__ unsigned short firsts[kMaxPairs];  // of each pair: the token's first pair with its expert
    __shared__ float mix[kMaxPairs];              // of each pair: its weight times the tensor scale
    __shared__ int queue, count;                  // next unit, units
    extern __shared__ __align__(1024) char dynamic[];
    char *rows = dynamic;                                                      // [W][D][2] KiB
    Unit *table = reinterpret_cast<Unit *>(dynamic + W * D * 2048);            // [n k ws]
    float *sums = reinterpret_cast<float *>(table + nk * p.ws);                // [n k][ws][16 NW]
    unsigned short *pairs = reinterpret_cast<unsigned short *>(rows);          // [n k][16], before the rows come
    static_assert(W * D * 2048 >= kMaxPairs * kFewTokens * 2, "the pairs fit the rows");
    {
        const int e = load_choice(p);
        const float w = tid < nk ? p.weights[tid] : 0.f;
        if (tid < nk)
            tokens[tid] = 0;
        if (tid == 0) {
            queue = W;
            count = 0;
        }
        int first;
        const int a = build_routes(routes, p, e, &first), t = tid / p.k;
        if (a >= 0)
            atomicOr(&tokens[a], 1u << t);
        if (tid < nk)
            firsts[tid] = (unsigned short)first;
        const float scale = tid < nk && routes.expert[tid] >= 0 ? p.gscale[2 * p.E + routes.expert[tid]] : 0.f;
        __syncthreads();
        const int j = a >= 0 ? __popc(tokens[a] & ((1u << t) - 1)) : 0;
        if (a >= 0)
            pairs[a * kFewTokens + j] = (unsigned short)tid;
        __syncthreads();
        // the first of each four tokens makes their units
        if (a >= 0 && j % 4 == 0) {
            const int n = __popc(tokens[a]);
            for (int part = 0; part < p.ws; ++part) {
                Unit u;
                u.expert = routes.list[a];
                u.part = (unsigned short)part;
                u.tile = (unsigned short)(part * p.tpw);
                u.end = (unsigned short)min(p.Td, (part + 1) * p.tpw);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    u.pair[q] = j + q < n ? pairs[a * kFewTokens + j + q] : kNoPair;
                table[atomicAdd(&count, 1)] = u;
            }
        }
        if (tid < nk)
            mix[tid] = routes.expert[tid] < 0 ? 0.f : w * scale;
        __syncthreads();
    }
    const int units = __builtin_amdgcn_readfirstlane(count);
    const unsigned tb = p.Td * 1024u, sb = p.Td * 128u;
    const u32x4 hrsrc = uniform(buffer_rsrc(p.h, (unsigned)(nk * p.Td * kTileK * 4)));
    const unsigned slots = lds_address(rows) + wave * (D * 2048);

    // This lane's row of each window: its offsets within an expert's codes and scales.
    unsigned coff[NW], soff[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int at = 16 * w + i, r = row0 + at;
        const bool in = at < p.rows && r < p.K;
        coff[w] = in ? (unsigned)(r >> 4) * tb + (unsigned)((g * 16 + (r & 15)) * 16) : kOutOfRange;
        soff[w] = in ? (unsigned)(r >> 4) * sb + (unsigned)((r & 15) * 8) : kOutOfRange;
    }
    u32x4 c[D][NW];
    u32x2 s[D][NW];
    int unit = wave, tile = 0, end = 0;   // of the tile that is loaded next
    u32x4 crsrc, srsrc;
    unsigned high, low;                   // this lane's 16 bytes of its row of the unit's h, of each part
    auto begin = [&]() {
        const bool in = unit < units;
        const Unit &u = table[in ? unit : 0];
        const int expert = in ? __builtin_amdgcn_readfirstlane(u.expert) : 0;
        tile = in ? __builtin_amdgcn_readfirstlane(u.tile) : 0;
        end = in ? __builtin_amdgcn_readfirstlane(u.end) : 1 << 30;
        const int pair = u.pair[g];
        const unsigned groups = p.K / kRowsPerGroup;
        crsrc = uniform(buffer_rsrc(p.d_codes + (long long)expert * groups * tb, in ? groups * tb : 0u));
        srsrc = uniform(buffer_rsrc(p.d_scales + (long long)expert * groups * sb, in ? groups * sb : 0u));
        // chunk c of token g's part j goes to slot c ^ (2 g + j) of its 256 bytes: the
        // operand's reads (chunk 4 g + q of part i % 2 of token i / 4) then fall into
        // eight different 16-byte slots a lane group
        const unsigned row = pair * p.Td * (kTileK * 4);
        high = in && pair != kNoPair ? row + 16 * (i ^ 2 * g) : kOutOfRange;
        low = in && pair != kNoPair ? row + 256 + 16 * (i ^ (2 * g + 1)) : kOutOfRange;
    };
    auto load = [&](auto tc) {
        constexpr int t = decltype(tc)::value;
        load_lds_b128(hrsrc, high + tile * (kTileK * 4), slots + t * 2048);
        load_lds_b128(hrsrc, low + tile * (kTileK * 4), slots + t * 2048 + 1024);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            s[t][w] = buffer_load_b64_nt(srsrc, soff[w] + tile * 128);
            c[t][w] = buffer_load_b128_nt(crsrc, coff[w] + tile * 1024);
        }
    };
    // The tile after; its unit, if another begins, from the queue.
    auto advance = [&]() {
        if (++tile < end)
            return;
        int next = 0;
        if (lane == 0)
            next = atomicAdd(&queue, 1);
        unit = __builtin_amdgcn_readfirstlane(next);
        begin();
    };
    const char *mine = rows + wave * (D * 2048) + (i & 1) * 1024 + (i >> 2) * 256;
    const int turn = 2 * (i >> 2) + (i & 1);
    f32x4 acc[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w)
        acc[w] = f32x4{0.f, 0.f, 0.f, 0.f};
    begin();
    int what[D];                  // of each slot: twice its unit, and 1 on the unit's last tile; -1: none
    static_for<D>([&](auto tc) {
        constexpr int t = decltype(tc)::value;
        what[t] = unit < units ? unit * 2 + (tile + 1 == end) : -1;
        load(tc);
        advance();
    });
    while (what[0] >= 0) {
        static_for<D>([&](auto tc) {
            constexpr int t = decltype(tc)::value;
            if constexpr (NW == 1)
                asm volatile("s_waitcnt vmcnt(%2)" : "+v"(c[t][0]), "+v"(s[t][0]) : "n"(4 * (D - 1)) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(%4)" : "+v"(c[t][0]), "+v"(s[t][0]), "+v"(c[t][1]), "+v"(s[t][1])
                             : "n"(6 * (D - 1)) : "memory");
            u32x2 x[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(mine + t * 2048 + ((4 * g + q) ^ turn) * 16);
                x[2 * q] = u32x2{v[0], v[1]};
                x[2 * q + 1] = u32x2{v[2], v[3]};
            }
#pragma unroll
            for (int w = 0; w < NW; ++w)
                tile_product<2>(acc[w], c[t][w], s[t][w], x);
            if (what[t] >= 0 && (what[t] & 1)) {
                const Unit &u = table[what[t] >> 1];
                const int pair = u.pair[g];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    if (pair != kNoPair)
                        sums[(pair * p.ws + u.part) * (16 * NW) + 16 * w + i] = acc[w][0] + acc[w][1];
                    acc[w][0] = acc[w][1] = 0.f;
                }
            }
            what[t] = unit < units ? unit * 2 + (tile + 1 == end) : -1;
            // the slot has been read before the next tile's rows are sent to it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            load(tc);
            advance();
        });
    }
    // (the loads behind the last tile still write their registers)
#pragma unroll
    for (int t = 0; t < D; ++t)
#pragma unroll
        for (int w = 0; w < NW; ++w)
            asm volatile("s_waitcnt vmcnt(0)" : "+v"(c[t][w]), "+v"(s[t][w])::"memory");
    __syncthreads();
    const int t = tid / (16 * NW), r = tid % (16 * NW);
    if (t < p.n && r < p.rows && row0 + r < p.K) {
        float y = 0.f;
        for (int sl = 0; sl < p.k; ++sl) {
            const int q = t * p.k + sl;
            if (routes.expert[q] < 0)
                continue;
            const float *src = sums + firsts[q] * p.ws * (16 * NW) + r;
            float o = src[0];
            for (int w = 1; w < p.ws; ++w)
                o += src[w * (16 * NW)];
            y = __builtin_fmaf(mix[q], o, y);
        }
        linear_out(p.e, t, row0 + r, y);
    }
}

constexpr int kMaxDownRows = 32;   // two windows
static_assert(kFewTokens * kMaxDownRows <= kThreads, "a thread for each output of a workgroup");

typedef void (*FewKernel)(MoeFewParams);

template <int NV, int... MT>
FewKernel pick_up(int mt, std::integer_sequence<int, MT...>)
{
    FewKernel k = nullptr;
    ((mt == MT + 1 ? (void)(k = nvfp4_moe_up_kernel<MT + 1, NV>) : (void)0), ...);
    return k;
}

// Outputs of a workgroup of the down projection: in fours, so that every compute unit
// has a workgroup; of few units some have several.
int down_rows(int K, int cus)
{
    const long long each = 4LL * cus, rows = (K + each - 1) / each * 4;
    return rows < kMaxDownRows ? (int)rows : kMaxDownRows;
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

int nvfp4_moe_decode_geometry(int K, int compute_units, int *outputs_per_workgroup)
{
    if (!outputs_per_workgroup)
        return NVFP4_ERR_NULL;
    if (K < 1 || compute_units < 1)
        return NVFP4_ERR_RANGE;
    if (K % 16 != 0 || !nvfp4_moe_is_few(1, K))
        return NVFP4_ERR_SHAPE;
    *outputs_per_workgroup = down_rows(K, compute_units);
    return NVFP4_OK;
}

size_t nvfp4_moe_few_bytes(int n, int k, int F)
{
    return (size_t)n * k * k_tiles(F) * kTileK * 4;
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
    p.ws = (p.Td + p.tpw - 1) / p.tpw;   // no part is empty
    p.e = a.epi;
    const int mt = (p.T + kWaves - 1) / kWaves;
    constexpr auto mts = std::make_integer_sequence<int, kMaxTilesPerWave>{};
    const FewKernel up = a.n <= 4 ? pick_up<1>(mt, mts) : (a.n <= 8 ? pick_up<2>(mt, mts) : pick_up<4>(mt, mts));
    const long long most = (long long)(a.n * a.k < a.E ? a.n * a.k : a.E) * p.P;
    hipLaunchKernelGGL(up, dim3((unsigned)(most < cus ? most : cus)), dim3(kThreads), 0, stream, p);
    if (hipGetLastError() != hipSuccess)
        return NVFP4_ERR_LAUNCH;
    p.rows = down_rows(a.K, cus);
    const int nk = a.n * a.k, nw = (p.rows + 15) / 16;
    const dim3 grid((unsigned)((a.K + p.rows - 1) / p.rows));
    // Six tiles ahead where the sums leave the LDS for it (of 160 KiB, of which the
    // kernel's own arrays take less than 10), else four.
    const unsigned units = (unsigned)(nk * p.ws * (sizeof(Unit) + 64 * nw));
    const bool six = units + kWaves * 6 * 2048 <= 150 * 1024;
    const unsigned lds = units + kWaves * (six ? 6 : 4) * 2048;
    const FewKernel down = nw == 1 ? (six ? nvfp4_moe_down_kernel<1, 6> : nvfp4_moe_down_kernel<1, 4>)
                                  : (six ? nvfp4_moe_down_kernel<2, 6> : nvfp4_moe_down_kernel<2, 4>);
    hipLaunchKernelGGL(down, grid, dim3(kThreads), lds, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}
