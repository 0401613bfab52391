// The expert layer of include/nvfp4.h: argument checks and dispatch, the router,
// the order of the pairs by expert, and the elementwise steps around the grouped
// products of many tokens.
#include "checks.h"
#include "epilogue.h"
#include "moe.h"

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSlots = 32;           // experts of a token
constexpr int kMaxF = 1 << 18;
constexpr int kMaxLd = 1 << 18;         // row strides of X and dY
constexpr int kChunkPairs = 1 << 16;

// ---- router --------------------------------------------------------------------------

struct RouteParams {
    const void *logits;
    const float *bias;
    float *weights;
    int *experts;
    const int *chosen;        // backward
    const float *dweights;
    void *dlogits;
    long long ldl, ldd;
    int n, E, k, bf16, sigmoid, normalize;
    float scale;
};

// Dword v of another lane: STEP 0 and 1 of the lane 1 and 2 away, 2 and 3 of the
// mirror of its eight and sixteen, 4 and 5 of the other sixteen and half of the wave.
// Without LDS: the router's rounds wait for one reduction after another (16 x 64,
// k = 8: 3.9 us, 5.4 through __shfl_xor; k = 4: 3.4).
template <int STEP>
__device__ __forceinline__ int other_lane(int v)
{
    if constexpr (STEP < 4) {
        constexpr int kControl[] = {0xB1, 0x4E, 0x141, 0x140};
        return __builtin_amdgcn_update_dpp(v, v, kControl[STEP], 0xF, 0xF, false);
    } else {
        const auto s = STEP == 4 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                 : __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (threadIdx.x & (STEP == 4 ? 16 : 32)) ? s[0] : s[1];
    }
}

// v combined over the wave (all lanes on) in a fixed order; every lane has the result.
template <typename T, typename F>
__device__ __forceinline__ T wave_all(T v, F f)
{
    static_for<6>([&](auto sc) {
        constexpr int kStep = decltype(sc)::value;
        struct Dwords {
            int d[sizeof(T) / 4];
        } w = __builtin_bit_cast(Dwords, v);
#pragma unroll
        for (int j = 0; j < (int)(sizeof(T) / 4); ++j)
            w.d[j] = other_lane<kStep>(w.d[j]);
        v = f(v, __builtin_bit_cast(T, w));
    });
    return v;
}

// v of lane `at`, the same in all lanes.
__device__ __forceinline__ float of_lane(float v, int at)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), at));
}

__device__ __forceinline__ float wave_sum(float v)
{
    return wave_all(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ u32 wave_max(u32 v)
{
    return wave_all(v, [](u32 a, u32 b) { return a > b ? a : b; });
}

// Unsigned integers in the order of the floats; NaN above all, the zeros alike.
__device__ __forceinline__ u32 ordered(float x)
{
    const u32 b = __builtin_bit_cast(u32, x + 0.0f);
    return x != x ? 0xFFFFFFFFu : (b >> 31 ? ~b : b | 0x80000000u);
}

__device__ __forceinline__ unsigned long long ordered(double x)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, x + 0.0);
    return x != x ? ~0ULL : (b >> 63 ? ~b : b | 0x8000000000000000ULL);
}

constexpr u32 kMasked = 0x007FFFFFu;    // ordered(-infinity)

// log sigmoid(x), without loss on either side
__device__ __forceinline__ float log_sigmoid(float x)
{
    return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}

__device__ __forceinline__ float load_logit(const RouteParams &p, long long row, int e)
{
    return e < p.E ? load_any(p.logits, row * p.ldl + e, !p.bf16) : -__builtin_inff();
}

// One wave a token, E / 64 logits a lane.  Each round takes the largest key that
// is left, ties to the lowest index: keys are the logits (both score functions
// ascend with them), or with a bias the scores plus it in 64 bits, where
// neighbours in the order may lie closer than 32 bits can tell.  Masked experts
// (-infinity) are never taken.  A normalized weight is a softmax over the chosen
// experts' logits, or log sigmoids: no sum of scores that could be zero.  8000 x 256,
// k = 8 with bias: 22 us, bound by the 64-bit exponentials and divisions of every
// score (8 MB read would take 2).
template <int NE, bool BIAS>
__global__ __launch_bounds__(256) void nvfp4_moe_route_kernel(RouteParams p)
{
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.n)
        return;
    float l[NE];
    u32 key[NE];
    unsigned long long wide[BIAS ? NE : 1];
#pragma unroll
    for (int r = 0; r < NE; ++r) {
        l[r] = load_logit(p, t, r * 64 + lane);
        key[r] = ordered(l[r]);
    }
    u32 top = key[0];
#pragma unroll
    for (int r = 1; r < NE; ++r)
        top = key[r] > top ? key[r] : top;
    top = wave_max(top);
    // the largest logit; of an all-masked row any finite value will do
    const float m = top == kMasked ? 0.0f : (top == 0xFFFFFFFFu ? __builtin_nanf("")
                                                                 : __builtin_bit_cast(float, top >> 31 ? top & 0x7FFFFFFFu : ~top));
    float total = 1.0f;
    if (!p.sigmoid && !p.normalize) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < NE; ++r)
            s += expf(l[r] - m);
        total = wave_sum(s);
    }
    if constexpr (BIAS) {
        double s[NE], sum = 0.0;
#pragma unroll
        for (int r = 0; r < NE; ++r) {
            s[r] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[r])) : exp((double)l[r] - (double)m);
            sum += s[r];
        }
        sum = p.sigmoid ? 1.0 : wave_all(sum, [](double a, double b) { return a + b; });
#pragma unroll
        for (int r = 0; r < NE; ++r) {
            const int e = r * 64 + lane;
            wide[r] = key[r] == kMasked ? 0ULL : ordered(s[r] / sum + (e < p.E ? (double)p.bias[e] : 0.0));
        }
    }
    int mine = -1;              // lane s: the expert of slot s, and its logit
    float logit = -__builtin_inff();
    for (int s = 0; s < p.k; ++s) {
        // the largest key, then the lowest expert that has it
        u32 best = 0, low = 0;
        if constexpr (BIAS) {
            unsigned long long b = 0;
#pragma unroll
            for (int r = 0; r < NE; ++r)
                b = wide[r] > b ? wide[r] : b;
            best = wave_max((u32)(b >> 32));
            low = wave_max((u32)(b >> 32) == best ? (u32)b : 0u);
            if (!best && !low)
                break;
        } else {
#pragma unroll
            for (int r = 0; r < NE; ++r)
                best = key[r] > best ? key[r] : best;
            best = wave_max(best);
            if (best <= kMasked)
                break;
        }
        bool found = false;
#pragma unroll
        for (int r = 0; r < NE; ++r) {
            const bool is = BIAS ? wide[BIAS ? r : 0] == ((unsigned long long)best << 32 | low) : key[r] == best;
            const unsigned long long mask = __ballot(is && !found);
            if (mask && !found) {
                const int at = __ffsll((long long)mask) - 1;
                const float v = of_lane(l[r], at);
                if (lane == s) {
                    mine = r * 64 + at;
                    logit = v;
                }
                if (lane == at) {
                    key[r] = 0;
                    if constexpr (BIAS)
                        wide[r] = 0;
                }
                found = true;
            }
        }
    }
    const bool live = lane < p.k && mine >= 0;
    // (in 64 bits behind the exponential, whose error of one step is most of a weight's)
    double w;
    if (p.normalize) {
        const float u = p.sigmoid ? log_sigmoid(logit) : logit;
        // largest of the chosen ones; NaN stays
        float um = live ? u : -__builtin_inff();
        um = wave_all(um, [](float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); });
        const double ex = live ? expf(u - um) : 0.0f;
        w = ex / wave_all(ex, [](double a, double b) { return a + b; });
    } else {
        w = p.sigmoid ? 1.0 / (1.0 + (double)expf(-logit)) : (double)expf(logit - m) / (double)total;
    }
    if (lane < p.k) {
        p.experts[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = live ? (float)(w * p.scale) : 0.0f;
    }
}

// d logits from d weights: with q the weights over the scale,
//   normalized:          scale q_s (dw_s - sum_j q_j dw_j), times sigmoid(-l_s) for sigmoid scores;
//   sigmoid:             scale q_s sigmoid(-l_s) dw_s;
//   softmax of the row:  scale p_e (dw_e - sum_j p_j dw_j) for every expert, dw_e = 0 where not chosen.
template <int NE>
__global__ __launch_bounds__(256) void nvfp4_moe_route_grad_kernel(RouteParams p)
{
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.n)
        return;
    const int chosen = lane < p.k ? p.chosen[t * p.k + lane] : -1;
    const bool live = chosen >= 0 && chosen < p.E;
    const float logit = live ? load_logit(p, t, chosen) : -__builtin_inff();
    const float dw = live ? p.dweights[t * p.k + lane] : 0.0f;
    const bool dense = !p.sigmoid && !p.normalize;
    float l[NE];
    float m = 0.0f, inv = 0.0f, q;
    if (dense) {
        m = -__builtin_inff();
#pragma unroll
        for (int r = 0; r < NE; ++r) {
            l[r] = load_logit(p, t, r * 64 + lane);
            m = l[r] != l[r] ? l[r] : (m != m ? m : fmaxf(m, l[r]));
        }
        m = wave_all(m, [](float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); });
        if (m == -__builtin_inff())
            m = 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < NE; ++r)
            s += expf(l[r] - m);
        s = wave_sum(s);
        inv = s > 0.0f || s != s ? 1.0f / s : 0.0f;
        q = expf(logit - m) * inv;
    } else if (p.normalize) {
        const float u = p.sigmoid ? log_sigmoid(logit) : logit;
        float um = live ? u : -__builtin_inff();
        um = wave_all(um, [](float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); });
        const float ex = live ? expf(u - um) : 0.0f;
        q = ex / wave_sum(ex);
    } else {
        q = 1.0f / (1.0f + expf(-logit));
    }
    const float dot = p.normalize || dense ? wave_sum(live ? q * dw : 0.0f) : 0.0f;
    float d = dense ? dw : q * (dw - dot);
    if (p.sigmoid)
        d *= 1.0f / (1.0f + expf(logit));
    d = live ? d : 0.0f;
    float out[NE];
#pragma unroll
    for (int r = 0; r < NE; ++r)
        out[r] = 0.0f;
    for (int s = 0; s < p.k; ++s) {
        const int es = __builtin_amdgcn_readlane(chosen, s);
        const float ds = of_lane(d, s);
#pragma unroll
        for (int r = 0; r < NE; ++r)
            if (es == r * 64 + lane)
                out[r] += ds;
    }
#pragma unroll
    for (int r = 0; r < NE; ++r) {
        const int e = r * 64 + lane;
        float v = out[r];
        if (dense)
            v = l[r] == -__builtin_inff() ? 0.0f : expf(l[r] - m) * inv * (v - dot);
        if (e < p.E)
            store_any(p.dlogits, t * p.ldd + e, !p.bf16, v * p.scale);
    }
}

template <int NE>
int launch_route(const RouteParams &p, bool grad, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.n + 3) / 4));
    if (grad)
        hipLaunchKernelGGL((nvfp4_moe_route_grad_kernel<NE>), grid, dim3(256), 0, stream, p);
    else if (p.bias)
        hipLaunchKernelGGL((nvfp4_moe_route_kernel<NE, true>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((nvfp4_moe_route_kernel<NE, false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int route(const RouteParams &p, bool grad, hipStream_t stream)
{
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    if (p.E <= 64)
        return launch_route<1>(p, grad, stream);
    if (p.E <= 128)
        return launch_route<2>(p, grad, stream);
    if (p.E <= 256)
        return launch_route<4>(p, grad, stream);
    if (p.E <= 512)
        return launch_route<8>(p, grad, stream);
    return launch_route<16>(p, grad, stream);
}

// ---- the pairs in the experts' order ----------------------------------------------------

// Stable counting sort of the n k pairs by expert, one workgroup: each of the 16
// waves counts a contiguous share, the shares' counts become their first rows,
// and each wave places its share 64 pairs at a time, equal experts in lane order
// (matched by one ballot for each bit of the expert).  Also the token tiles of
// the grouped products.  position: the row of each pair, or -1.  Bound by the
// latency of reading the choices, so kHeld of a lane's are read together and kept
// from the counting to the placing (12000 pairs: 18.4 us read one by one).
constexpr int kSortWaves = 16, kHeld = 16;

__global__ __launch_bounds__(1024) void nvfp4_moe_sort_kernel(const int *experts, int pairs, int E, int bm, int *position,
                                                              int *pair, int *offset, int *tile)
{
    __shared__ int count[kSortWaves][kMaxExperts];
    __shared__ int start[kMaxExperts + 1], tiles[kMaxExperts + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int share = ((pairs + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int q0 = min(pairs, wave * share), q1 = min(pairs, q0 + share);
    int held[kHeld];              // experts of the pairs q0 + 64 j + lane, -1: none
    auto fetch = [&](int q) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int at = q + 64 * j + lane;
            held[j] = at < q1 ? experts[at] : -1;
        }
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (held[j] >= E)
                held[j] = -1;
    };
    fetch(q0);
    for (int i = tid; i < kSortWaves * E; i += 1024)
        count[i / E][i % E] = 0;
    __syncthreads();
    for (int q = q0; q < q1; q += 64 * kHeld) {
        if (q > q0)
            fetch(q);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (held[j] >= 0)
                atomicAdd(&count[wave][held[j]], 1);
    }
    __syncthreads();
    // totals, then (one wave, 16 experts a lane) their running sums
    int total = 0;
    if (tid < E)
        for (int w = 0; w < kSortWaves; ++w)
            total += count[w][tid];
    start[tid] = total;
    tiles[tid] = (total + bm - 1) / bm;
    __syncthreads();
    if (wave == 0) {
        int a[16], b[16], sa = 0, sb = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            a[j] = sa;
            b[j] = sb;
            sa += start[lane * 16 + j];
            sb += tiles[lane * 16 + j];
        }
        int pa = sa, pb = sb;
        for (int d = 1; d < 64; d *= 2) {
            const int ua = __shfl_up(pa, d), ub = __shfl_up(pb, d);
            if (lane >= d) {
                pa += ua;
                pb += ub;
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            start[lane * 16 + j] = pa - sa + a[j];
            tiles[lane * 16 + j] = pb - sb + b[j];
        }
        if (lane == 63) {
            start[kMaxExperts] = pa;
            tiles[kMaxExperts] = pb;
        }
    }
    __syncthreads();
    if (tid < E) {
        int at = start[tid];
        offset[tid] = at;
        for (int i = 0; i * bm < total; ++i) {
            tile[1 + 2 * (tiles[tid] + i)] = tid;
            tile[2 + 2 * (tiles[tid] + i)] = at + i * bm;
        }
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = count[w][tid];
            count[w][tid] = at;
            at += c;
        }
    }
    if (tid == 0) {
        offset[E] = start[kMaxExperts];
        tile[0] = tiles[kMaxExperts];
    }
    __syncthreads();
    int bits = 0;
    while (bits < 10 && (E - 1) >> bits)
        ++bits;
    for (int q = q0; q < q1; q += 64 * kHeld) {
        if (q1 - q0 > 64 * kHeld)
            fetch(q);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int at = q + 64 * j;
            if (at >= q1)
                break;
            const int e = held[j];
            const bool ok = e >= 0;
            unsigned long long same = __ballot(ok);
            for (int b = 0; b < bits; ++b) {
                const unsigned long long set = __ballot(ok && (e >> b & 1));
                same &= e >> b & 1 ? set : ~set;
            }
            int row = -1;
            if (ok) {
                row = count[wave][e] + __popcll(same & ((1ULL << lane) - 1));
                pair[row] = at + lane;
            }
            if (at + lane < q1)
                position[at + lane] = row;
            // the last of each expert's lanes moves its counter on (after every lane has read it)
            __builtin_amdgcn_wave_barrier();
            if (ok && !(same >> lane >> 1))
                count[wave][e] = row + 1;
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---- combine ------------------------------------------------------------------------------

// Outputs of a token: sum over its slots, in order, of weight times the pair's
// row, then the residual.  Memory bound: 4 k bytes read for an output (12000 rows of
// 5120: 41 us, 6 TB/s).  (The rows
// are sums, so they stay in 32 bits.)
template <int SLOTS>
__global__ __launch_bounds__(256) void nvfp4_moe_combine_kernel(nvfp4_epi_params e, const float *rows, const int *position,
                                                                const float *weights, int n, int k, int cols)
{
    const int quads = cols / 4;
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(idx / quads), c = (int)(idx % quads) * 4;
    if (t >= n)
        return;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < k; s0 += SLOTS) {
        f32x4 v[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int q = t * k + s0 + s;
            const int at = s0 + s < k ? position[q] : -1;
            w[s] = at < 0 ? 0.f : (weights ? weights[q] : 1.f);
            v[s] = at < 0 ? f32x4{0.f, 0.f, 0.f, 0.f}
                          : __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(rows + (long long)at * cols + c));
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = __builtin_fmaf(w[s], v[s][j], y[j]);
    }
    linear_out4(e, t, c, y);
}

// ---- the elementwise half of the gradients ---------------------------------------------------

// One workgroup a pair: with d = dY . Wd (for weight one), the weight's gradient
// is the dot product of d with h = act(G) U, unrounded; dG = w d U act'(G) and dU
// = w d act(G), times their tensor scales, become operands of the next product, fp16
// with an exponent for the row (as bf16, dX was off by 2.3e-3 of its norm, of which
// its own rounding is 1.7e-3).  They stay in registers until the row's largest is
// known, kHeldTurns a thread; of longer rows the rest is computed again.  Memory
// bound: 2800 pairs of F = 1280 take 13 us for 57 MB.
constexpr int kHeldTurns = 4;

__global__ __launch_bounds__(256) void nvfp4_moe_grad_kernel(const float *d, const float *preact, const int *position,
                                                             const int *experts, const float *weights, const float *gscale,
                                                             float *dweights, uint16_t *dz, int *dzexp, long long ldp, int E,
                                                             int F, int act)
{
    const int q = blockIdx.x, tid = threadIdx.x;
    const int row = position[q];
    if (row < 0) {
        if (tid == 0 && dweights)
            dweights[q] = 0.f;
        return;
    }
    const int e = experts[q];
    const float w = weights[q], gg = gscale[e], gu = gscale[E + e];
    const float *src = preact + (long long)row * ldp;
    uint16_t *dst = dz + (long long)row * 2 * F;
    float dot = 0.f;
    struct Grads {
        f32x4 g, u;
    };
    auto grads = [&](int c) {
        const f32x4 dh = *reinterpret_cast<const f32x4 *>(d + (long long)row * F + c);
        const f32x4 g = *reinterpret_cast<const f32x4 *>(src + gated_row(c, 0));
        const f32x4 u = *reinterpret_cast<const f32x4 *>(src + gated_row(c, 1));
        Grads r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = activate(g[j], act);
            dot = __builtin_fmaf(dh[j], a * u[j], dot);
            r.g[j] = w * dh[j] * u[j] * activate_grad(g[j], act) * gg;
            r.u[j] = w * dh[j] * a * gu;
        }
        return r;
    };
    Grads held[kHeldTurns];
    u32 top = 0;
    static_for<kHeldTurns>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int c = tid * 4 + 1024 * j;
        if (c < F) {
            held[j] = grads(c);
            top = max(top, max(top_bits(held[j].g), top_bits(held[j].u)));
        }
    });
    for (int c = tid * 4 + 1024 * kHeldTurns; c < F; c += 1024) {
        const Grads r = grads(c);
        top = max(top, max(top_bits(r.g), top_bits(r.u)));
    }
    __shared__ float part[4];
    __shared__ u32 tops[4];
    dot = wave_sum(dot);
    top = wave_max(top);
    if ((tid & 63) == 0) {
        part[tid >> 6] = dot;
        tops[tid >> 6] = top;
    }
    __syncthreads();
    if (tid == 0 && dweights)
        dweights[q] = (part[0] + part[1]) + (part[2] + part[3]);
    if (!dz)
        return;
    const int exponent = block_exponent(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    if (tid == 0)
        dzexp[row] = exponent;
    static_for<kHeldTurns>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int c = tid * 4 + 1024 * j;
        if (c < F) {
            store_block(dst + gated_row(c, 0), held[j].g, exponent);
            store_block(dst + gated_row(c, 1), held[j].u, exponent);
        }
    });
    for (int c = tid * 4 + 1024 * kHeldTurns; c < F; c += 1024) {
        const Grads r = grads(c);
        store_block(dst + gated_row(c, 0), r.g, exponent);
        store_block(dst + gated_row(c, 1), r.u, exponent);
    }
}

// bf16 rows of an fp32 or unaligned matrix, or of one whose rows lie far apart, for the
// product; rest: the second parts of fp32 values (bf16_rest).
__global__ __launch_bounds__(256) void nvfp4_moe_rows_kernel(const void *src, int f32, int rest, long long ld, int n, int cols,
                                                             uint16_t *dst)
{
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(idx / cols), c = (int)(idx % cols);
    if (t >= n)
        return;
    const float v = load_any(src, t * ld + c, f32);
    const uint16_t high = f32_to_bf16_bits(v);
    dst[(long long)t * cols + c] = rest ? f32_to_bf16_bits(bf16_rest(v, high)) : high;
}

// ---- host side --------------------------------------------------------------------------------

size_t round256(size_t bytes)
{
    return (bytes + 255) / 256 * 256;
}

// Tokens handled at a time: bounded work memory, and offsets of their rows (below
// the 0x7FFFFFF0 that stands for "outside") within 32 bits.  By k and K alone: the
// pre-activations are in the experts' order within such a chunk, so the forward and
// the backward call cut the tokens alike, whatever strides their rows have.
constexpr int64_t kMaxOffset = 0x7FFF0000LL / 2 - kMaxLd;   // in elements

int chunk_tokens(int k, int K)
{
    const int by_pairs = kChunkPairs / k, by_bytes = (int)(kMaxOffset / K);
    return by_pairs < by_bytes ? by_pairs : by_bytes;
}

// Whether a chunk's rows lie too far apart for 32 bits: they are copied next to each other.
bool far_apart(int tokens, int64_t ld)
{
    return tokens > 1 && tokens * ld > kMaxOffset;
}

bool is_few(int n, int K)
{
    return nvfp4_moe_is_few(n, K);
}

// The order's arrays, at the head of a workspace.
struct Order {
    int *position, *pair, *offset, *tile;
};

// (grows with the pairs, whatever tile they take: a shorter last chunk fits the
// workspace of a whole one)
size_t order_bytes(int pairs, int E)
{
    return round256(4 * ((size_t)2 * pairs + E + 1 + 1 + 2 * (size_t)nvfp4_moe_max_tiles(pairs, E, 32)));
}

Order order_at(void *ws, int pairs, int E)
{
    int *p = static_cast<int *>(ws);
    return {p, p + pairs, p + 2 * pairs, p + 2 * pairs + E + 1};
}

int launch_sort(const Order &o, const int *experts, int pairs, int E, int tile_tokens, hipStream_t stream)
{
    hipLaunchKernelGGL(nvfp4_moe_sort_kernel, dim3(1), dim3(1024), 0, stream, experts, pairs, E,
                       tile_tokens, o.position, o.pair, o.offset, o.tile);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int launch_rows(const void *src, bool f32, bool rest, long long ld, int n, int cols, uint16_t *dst, hipStream_t stream)
{
    hipLaunchKernelGGL(nvfp4_moe_rows_kernel, dim3((unsigned)(((long long)n * cols + 255) / 256)), dim3(256), 0, stream, src, f32,
                       rest, ld, n, cols, dst);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int launch_combine(const nvfp4_epi_params &e, const float *rows, const Order &o, const float *weights, int n, int k, int cols,
                   hipStream_t stream)
{
    const dim3 grid((unsigned)(((long long)n * (cols / 4) + 255) / 256));
    if (k <= 2)
        hipLaunchKernelGGL(nvfp4_moe_combine_kernel<2>, grid, dim3(256), 0, stream, e, rows, o.position, weights, n, k, cols);
    else if (k <= 4)
        hipLaunchKernelGGL(nvfp4_moe_combine_kernel<4>, grid, dim3(256), 0, stream, e, rows, o.position, weights, n, k, cols);
    else
        hipLaunchKernelGGL(nvfp4_moe_combine_kernel<8>, grid, dim3(256), 0, stream, e, rows, o.position, weights, n, k, cols);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int check_sizes(const nvfp4_experts *w, int n, int k)
{
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || k < 1 || k > kMaxSlots || w->E < 1 || w->E > kMaxExperts || w->F < 1 || w->K < 1)
        return NVFP4_ERR_RANGE;
    if (w->K % 16 != 0 || w->F % 16 != 0 || w->K > kMaxK || w->F > kMaxF)
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

nvfp4_epi_params plain_out(void *out, int64_t ldo, bool f32, int N)
{
    nvfp4_epi_params e = {};
    e.out = out;
    e.ldo = (int)ldo;
    e.gscale = e.up_gscale = 1.0f;
    e.N = N;
    e.flags = f32 ? kEpiOutF32 : 0;
    if (ldo % 4 == 0 && is_aligned(out, f32 ? 16 : 8))
        e.flags |= kEpiVec;
    return e;
}

struct Bytes {
    size_t gu_codes, gu_scales, d_codes, d_scales;   // of one expert
};

Bytes expert_bytes(const nvfp4_experts *w, bool transposed)
{
    const int rows = 2 * w->F;   // F is a multiple of 16: nvfp4_gated_rows(F)
    return transposed ? Bytes{nvfp4_transposed_codes_bytes(rows, w->K), nvfp4_transposed_scales_bytes(rows, w->K),
                              nvfp4_transposed_codes_bytes(w->K, w->F), nvfp4_transposed_scales_bytes(w->K, w->F)}
                      : Bytes{nvfp4_packed_codes_bytes(rows, w->K), nvfp4_packed_scales_bytes(rows, w->K),
                              nvfp4_packed_codes_bytes(w->K, w->F), nvfp4_packed_scales_bytes(w->K, w->F)};
}

// Exponents of a row of h: one for 64 columns, an even number.
int exponents(int F)
{
    return (F + 127) / 128 * 2;
}

size_t exponents_bytes(int rows, int F)
{
    return round256((size_t)rows * exponents(F) * 4);
}

// Workspace of a forward call of several tokens: the order, h with its exponents, its
// second parts (of a call whose result is fp32) and the rows.
size_t forward_bytes(int n, int k, const nvfp4_experts *w)
{
    const int by_pairs = kChunkPairs / k, m = n < by_pairs ? n : by_pairs, pairs = m * k;
    return order_bytes(pairs, w->E) + 2 * round256((size_t)pairs * w->F * 2) + exponents_bytes(pairs, w->F) +
           round256((size_t)pairs * w->K * 4);
}

// (a copy of dY, which the first product reads, lies where the last one's rows will,
// or without them in a place of its own)
size_t backward_bytes(int n, int k, const nvfp4_experts *w, bool dx, bool copy)
{
    const int by_pairs = kChunkPairs / k, m = n < by_pairs ? n : by_pairs, pairs = m * k;
    size_t b = order_bytes(pairs, w->E) + round256((size_t)pairs * w->F * 4);
    if (dx)
        b += round256((size_t)pairs * w->F * 4) + round256((size_t)pairs * 4) + round256((size_t)pairs * w->K * 4);
    else if (copy || far_apart(m, kMaxLd))
        b += round256((size_t)m * w->K * 2);
    return b;
}

bool usable_dy(const void *p, int dtype, int64_t ld, int n)
{
    return dtype == NVFP4_DTYPE_BF16 && is_aligned(p, 16) && (n < 2 || ld % 8 == 0);
}

int check_pointers(const nvfp4_experts *w)
{
    if (!w->gate_up_codes || !w->gate_up_scales || !w->down_codes || !w->down_scales || !w->gscale)
        return NVFP4_ERR_NULL;
    if (!is_aligned(w->gate_up_codes, 16) || !is_aligned(w->gate_up_scales, 16) || !is_aligned(w->down_codes, 16) ||
        !is_aligned(w->down_scales, 16) || !is_aligned(w->gscale, 4))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_moe_route(const void *logits, int dtype, int64_t ldl, const float *bias, int n, int E, int k, int scoring,
                    int normalize, float scale, float *weights, int32_t *experts, void *stream)
{
    if (n > 0 && (!logits || !weights || !experts))
        return NVFP4_ERR_NULL;
    if (n < 0 || E < 1 || E > kMaxExperts || k < 1 || k > kMaxSlots || k > E || !valid_dtype(dtype) || ldl < E ||
        (scoring != NVFP4_SCORE_SOFTMAX && scoring != NVFP4_SCORE_SIGMOID))
        return NVFP4_ERR_RANGE;
    if (!is_aligned(logits, dtype_size(dtype)) || !is_aligned(bias, 4) || !is_aligned(weights, 4) || !is_aligned(experts, 4))
        return NVFP4_ERR_ALIGN;
    const Region in[] = {matrix(logits, n, ldl, E, dtype_size(dtype)), array(bias, 4 * (size_t)E)};
    const Region w = array(weights, (size_t)n * k * 4), e = array(experts, (size_t)n * k * 4);
    if (any_overlap(w, in) || any_overlap(e, in) || overlap(w, e))
        return NVFP4_ERR_OVERLAP;
    if (n == 0)
        return NVFP4_OK;
    RouteParams p = {};
    p.logits = logits;
    p.bias = bias;
    p.weights = weights;
    p.experts = experts;
    p.ldl = ldl;
    p.n = n;
    p.E = E;
    p.k = k;
    p.bf16 = dtype == NVFP4_DTYPE_BF16;
    p.sigmoid = scoring == NVFP4_SCORE_SIGMOID;
    p.normalize = normalize != 0;
    p.scale = scale;
    return route(p, false, (hipStream_t)stream);
}

int nvfp4_moe_route_backward(const void *logits, int dtype, int64_t ldl, const int32_t *experts, const float *dweights, int n,
                             int E, int k, int scoring, int normalize, float scale, void *dlogits, int64_t ldd, void *stream)
{
    if (n > 0 && (!logits || !experts || !dweights || !dlogits))
        return NVFP4_ERR_NULL;
    if (n < 0 || E < 1 || E > kMaxExperts || k < 1 || k > kMaxSlots || k > E || !valid_dtype(dtype) || ldl < E || ldd < E ||
        (scoring != NVFP4_SCORE_SOFTMAX && scoring != NVFP4_SCORE_SIGMOID))
        return NVFP4_ERR_RANGE;
    const int size = dtype_size(dtype);
    if (!is_aligned(logits, size) || !is_aligned(dlogits, size) || !is_aligned(experts, 4) || !is_aligned(dweights, 4))
        return NVFP4_ERR_ALIGN;
    const Region in[] = {matrix(logits, n, ldl, E, size), array(experts, (size_t)n * k * 4), array(dweights, (size_t)n * k * 4)};
    if (any_overlap(matrix(dlogits, n, ldd, E, size), in))
        return NVFP4_ERR_OVERLAP;
    if (n == 0)
        return NVFP4_OK;
    RouteParams p = {};
    p.logits = logits;
    p.chosen = experts;
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ldl = ldl;
    p.ldd = ldd;
    p.n = n;
    p.E = E;
    p.k = k;
    p.bf16 = dtype == NVFP4_DTYPE_BF16;
    p.sigmoid = scoring == NVFP4_SCORE_SIGMOID;
    p.normalize = normalize != 0;
    p.scale = scale;
    return route(p, true, (hipStream_t)stream);
}

size_t nvfp4_moe_workspace_bytes(int n, int k, int E, int F, int K, int preact)
{
    nvfp4_experts w = {};
    w.E = E;
    w.F = F;
    w.K = K;
    if (check_sizes(&w, n, k) != NVFP4_OK || n == 0)
        return 0;
    return !preact && is_few(n, K) ? nvfp4_moe_few_bytes(n, k, F) : forward_bytes(n, k, &w);
}

int nvfp4_moe_geometry(int n, int k, int E, int F, int K, int *rows_per_workgroup, int *tokens_per_workgroup)
{
    if (!rows_per_workgroup || !tokens_per_workgroup)
        return NVFP4_ERR_NULL;
    nvfp4_experts w = {};
    w.E = E;
    w.F = F;
    w.K = K;
    const int st = n < 1 ? NVFP4_ERR_RANGE : check_sizes(&w, n, k);
    if (st != NVFP4_OK)
        return st;
    const int by_pairs = kChunkPairs / k, pairs = (n < by_pairs ? n : by_pairs) * k;   // (a shorter last chunk may differ)
    *tokens_per_workgroup = nvfp4_moe_tile_tokens(pairs, E, F);
    *rows_per_workgroup = nvfp4_moe_tile_rows(pairs, E, *tokens_per_workgroup);
    return NVFP4_OK;
}

int nvfp4_moe(const nvfp4_experts *w, const uint16_t *X, int64_t ldx, const int32_t *experts, const float *weights, int n, int k,
              void *Y, int64_t ldy, const nvfp4_epilogue *epilogue, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!w || !epilogue)
        return NVFP4_ERR_NULL;
    const nvfp4_epilogue &ep = *epilogue;
    int st = check_sizes(w, n, k);
    if (st != NVFP4_OK)
        return st;
    st = check_pointers(w);
    if (st != NVFP4_OK)
        return st;
    if (n > 0 && (!X || !experts || !weights || !Y))
        return NVFP4_ERR_NULL;
    const int F = w->F, K = w->K, E = w->E;
    if (ep.activation < NVFP4_ACT_NONE || ep.activation > NVFP4_ACT_GELU_TANH || !valid_dtype(ep.out_dtype) ||
        (ep.residual && !valid_dtype(ep.residual_dtype)) || ep.bias || ep.up_bias)
        return NVFP4_ERR_RANGE;
    if (ldx < K || ldy < K || (ep.residual && ep.ldr < K) || (ep.preact && ep.ldp < 2 * (int64_t)F))
        return NVFP4_ERR_RANGE;
    if (ldx > kMaxLd || ldy > INT32_MAX || ep.ldr > INT32_MAX || ep.ldp > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    const int os = dtype_size(ep.out_dtype), rs = dtype_size(ep.residual_dtype);
    if (!is_aligned(X, 16) || (n > 1 && ldx % 8 != 0) || !is_aligned(experts, 4) || !is_aligned(weights, 4) || !is_aligned(Y, os) ||
        (ep.residual && !is_aligned(ep.residual, rs)) || (ep.preact && (!is_aligned(ep.preact, 16) || ep.ldp % 8 != 0)))
        return NVFP4_ERR_ALIGN;
    if (n == 0)
        return NVFP4_OK;
    const bool few = !ep.preact && is_few(n, K);
    const size_t need = nvfp4_moe_workspace_bytes(n, k, E, F, K, ep.preact != nullptr);
    if (!workspace || workspace_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    if (!is_aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const Bytes b = expert_bytes(w, false);
    const size_t pairs_bytes = (size_t)n * k * 4;
    const Region in[] = {matrix(X, n, ldx, K, 2), array(experts, pairs_bytes), array(weights, pairs_bytes),
                         array(w->gate_up_codes, E * b.gu_codes), array(w->gate_up_scales, E * b.gu_scales),
                         array(w->down_codes, E * b.d_codes), array(w->down_scales, E * b.d_scales),
                         array(w->gscale, 12 * (size_t)E)};
    const Region y = matrix(Y, n, ldy, K, os), z = matrix(ep.preact, ep.preact ? n * k : 0, ep.ldp, 2 * (int64_t)F, 4);
    const Region residual = matrix(ep.residual, n, ep.ldr, K, rs), space = array(workspace, need);
    const bool in_place = ep.residual == Y && ep.ldr == ldy && ep.residual_dtype == ep.out_dtype;
    if (any_overlap(y, in) || any_overlap(z, in) || any_overlap(space, in) || overlap(y, z) || overlap(z, residual) ||
        overlap(space, y) || overlap(space, z) || overlap(space, residual) || (!in_place && overlap(y, residual)))
        return NVFP4_ERR_OVERLAP;

    nvfp4_epi_params e = plain_out(Y, ldy, ep.out_dtype == NVFP4_DTYPE_F32, K);
    e.residual = ep.residual;
    e.ldr = (int)ep.ldr;
    if (ep.residual_dtype == NVFP4_DTYPE_F32)
        e.flags |= kEpiResidualF32;
    if (ep.residual && (ep.ldr % 4 != 0 || !is_aligned(ep.residual, 4 * rs)))
        e.flags &= ~kEpiVec;
    hipStream_t s = (hipStream_t)stream;
    if (few) {
        nvfp4_moe_few_args a = {};
        a.gu_codes = w->gate_up_codes;
        a.gu_scales = w->gate_up_scales;
        a.d_codes = w->down_codes;
        a.d_scales = w->down_scales;
        a.gscale = w->gscale;
        a.X = X;
        a.experts = experts;
        a.weights = weights;
        a.h = static_cast<uint16_t *>(workspace);
        a.ldx = (int)ldx;
        a.n = n;
        a.k = k;
        a.E = E;
        a.F = F;
        a.K = K;
        a.act = ep.activation;
        a.epi = e;
        return nvfp4_launch_moe_few(a, s);
    }
    int cus = 0;
    st = nvfp4_device_cus(&cus);
    const int step = chunk_tokens(k, K);
    for (int t0 = 0; t0 < n && st == NVFP4_OK; t0 += step) {
        const int m = n - t0 < step ? n - t0 : step, pairs = m * k, tokens = nvfp4_moe_tile_tokens(pairs, E, F);
        char *ws = static_cast<char *>(workspace);
        const Order o = order_at(ws, pairs, E);
        ws += order_bytes(pairs, E);
        uint16_t *h = reinterpret_cast<uint16_t *>(ws);
        ws += round256((size_t)pairs * F * 2);
        uint16_t *hrest = reinterpret_cast<uint16_t *>(ws);
        ws += round256((size_t)pairs * F * 2);
        int *hexp = reinterpret_cast<int *>(ws);
        float *rows = reinterpret_cast<float *>(ws + exponents_bytes(pairs, F));
        const uint16_t *x = X + (size_t)t0 * ldx;
        long long ld = ldx;
        if (far_apart(m, ldx)) {
            uint16_t *near = reinterpret_cast<uint16_t *>(rows);   // (which the second product writes)
            st = launch_rows(x, false, false, ldx, m, K, near, s);
            if (st != NVFP4_OK)
                break;
            x = near;
            ld = K;
        }
        st = launch_sort(o, experts + (size_t)t0 * k, pairs, E, tokens, s);
        if (st != NVFP4_OK)
            break;
        nvfp4_moe_gemm_args a = {};
        a.mode = 1;
        a.gather = true;
        a.codes = w->gate_up_codes;
        a.scales = w->gate_up_scales;
        a.cstride = (long long)b.gu_codes;
        a.sstride = (long long)b.gu_scales;
        a.X = x;
        a.ldx = ld;
        a.xrows = m;
        a.k = k;
        a.rows = pairs;
        a.tile_tokens = tokens;
        a.E = E;
        a.K = K;
        a.row_groups = 2 * F / kRowsPerGroup;
        a.gscale = w->gscale;
        a.up_gscale = w->gscale + E;
        a.order = {o.tile, o.offset, o.pair};
        a.hexp = hexp;
        a.hrest = ep.out_dtype == NVFP4_DTYPE_F32 ? hrest : nullptr;
        a.nexp = exponents(F);
        a.epi = plain_out(h, F, false, F);
        a.epi.flags |= ep.activation;
        if (ep.preact) {
            a.epi.preact = ep.preact + (size_t)t0 * k * ep.ldp;
            a.epi.ldp = (int)ep.ldp;
        }
        st = nvfp4_launch_moe_gemm(a, s);
        if (st != NVFP4_OK)
            break;
        a.mode = 0;
        a.gather = false;
        a.codes = w->down_codes;
        a.scales = w->down_scales;
        a.cstride = (long long)b.d_codes;
        a.sstride = (long long)b.d_scales;
        a.X = h;
        a.xexp = hexp;
        a.ldx = F;
        a.K = F;
        a.row_groups = K / kRowsPerGroup;
        a.gscale = w->gscale + 2 * (size_t)E;
        a.up_gscale = nullptr;
        a.epi = plain_out(rows, K, true, K);
        st = nvfp4_launch_moe_gemm(a, s);
        if (st != NVFP4_OK)
            break;
        if (a.hrest) {
            a.X = hrest;
            a.rest = kRestBits;
            st = nvfp4_launch_moe_gemm(a, s);
            if (st != NVFP4_OK)
                break;
        }
        nvfp4_epi_params c = e;
        c.out = static_cast<char *>(e.out) + (size_t)t0 * ldy * os;
        if (c.residual)
            c.residual = static_cast<const char *>(e.residual) + (size_t)t0 * ep.ldr * rs;
        st = launch_combine(c, rows, o, weights + (size_t)t0 * k, m, k, K, s);
    }
    return st;
}

size_t nvfp4_moe_backward_workspace_bytes(int n, int k, int E, int F, int K, int dx, int copy)
{
    nvfp4_experts w = {};
    w.E = E;
    w.F = F;
    w.K = K;
    if (check_sizes(&w, n, k) != NVFP4_OK || n == 0)
        return 0;
    return backward_bytes(n, k, &w, dx != 0, copy != 0);
}

int nvfp4_moe_backward(const nvfp4_experts *wt, const void *dY, int dy_dtype, int64_t ldy, const int32_t *experts,
                       const float *weights, const float *preact, int64_t ldp, int activation, int n, int k, uint16_t *dX,
                       int64_t ldx, float *dweights, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!wt)
        return NVFP4_ERR_NULL;
    int st = check_sizes(wt, n, k);
    if (st != NVFP4_OK)
        return st;
    st = check_pointers(wt);
    if (st != NVFP4_OK)
        return st;
    if (n > 0 && (!dY || !experts || !weights || !preact))
        return NVFP4_ERR_NULL;
    const int F = wt->F, K = wt->K, E = wt->E;
    if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_GELU_TANH || !valid_dtype(dy_dtype) || ldy < K ||
        ldp < 2 * (int64_t)F || (dX && ldx < K))
        return NVFP4_ERR_RANGE;
    if (ldy > kMaxLd || ldp > INT32_MAX || ldx > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    const int ds = dtype_size(dy_dtype);
    if (!is_aligned(dY, ds) || !is_aligned(experts, 4) || !is_aligned(weights, 4) || !is_aligned(preact, 16) || ldp % 8 != 0 ||
        !is_aligned(dX, 2) || !is_aligned(dweights, 4))
        return NVFP4_ERR_ALIGN;
    if (n == 0 || (!dX && !dweights))
        return NVFP4_OK;
    const bool copy = !usable_dy(dY, dy_dtype, ldy, n);
    const size_t need = backward_bytes(n, k, wt, dX != nullptr, copy);
    if (!workspace || workspace_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    if (!is_aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const Bytes b = expert_bytes(wt, true);
    const size_t pairs_bytes = (size_t)n * k * 4;
    const Region in[] = {matrix(dY, n, ldy, K, ds), array(experts, pairs_bytes), array(weights, pairs_bytes),
                         matrix(preact, n * k, ldp, 2 * (int64_t)F, 4), array(wt->gate_up_codes, E * b.gu_codes),
                         array(wt->gate_up_scales, E * b.gu_scales), array(wt->down_codes, E * b.d_codes),
                         array(wt->down_scales, E * b.d_scales), array(wt->gscale, 12 * (size_t)E)};
    const Region out[] = {matrix(dX, n, ldx, K, 2), array(dweights, pairs_bytes), array(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        if (any_overlap(out[i], in))
            return NVFP4_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return NVFP4_ERR_OVERLAP;
    }
    int cus = 0;
    st = nvfp4_device_cus(&cus);
    hipStream_t s = (hipStream_t)stream;
    const int step = chunk_tokens(k, K);
    for (int t0 = 0; t0 < n && st == NVFP4_OK; t0 += step) {
        const int m = n - t0 < step ? n - t0 : step, pairs = m * k, tokens = nvfp4_moe_tile_tokens(pairs, E, F);
        char *ws = static_cast<char *>(workspace);
        const Order o = order_at(ws, pairs, E);
        ws += order_bytes(pairs, E);
        float *d = reinterpret_cast<float *>(ws);
        ws += round256((size_t)pairs * F * 4);
        uint16_t *dz = dX ? reinterpret_cast<uint16_t *>(ws) : nullptr;
        ws += dX ? round256((size_t)pairs * F * 4) : 0;
        int *dzexp = reinterpret_cast<int *>(ws);
        ws += dX ? round256((size_t)pairs * 4) : 0;
        float *rows = reinterpret_cast<float *>(ws);
        const char *from = static_cast<const char *>(dY) + (size_t)t0 * ldy * ds;
        const uint16_t *dy = reinterpret_cast<const uint16_t *>(from);
        long long ld = ldy;
        const bool f32 = dy_dtype == NVFP4_DTYPE_F32;
        uint16_t *near = reinterpret_cast<uint16_t *>(ws);
        if (copy || far_apart(m, ldy)) {
            st = launch_rows(from, f32, false, ldy, m, K, near, s);
            if (st != NVFP4_OK)
                break;
            dy = near;
            ld = K;
        }
        const int *ids = experts + (size_t)t0 * k;
        st = launch_sort(o, ids, pairs, E, tokens, s);
        if (st != NVFP4_OK)
            break;
        nvfp4_moe_gemm_args a = {};
        a.mode = 2;
        a.gather = true;
        a.codes = wt->down_codes;
        a.scales = wt->down_scales;
        a.cstride = (long long)b.d_codes;
        a.sstride = (long long)b.d_scales;
        a.X = dy;
        a.ldx = ld;
        a.xrows = m;
        a.k = k;
        a.rows = pairs;
        a.tile_tokens = tokens;
        a.E = E;
        a.K = K;
        a.row_groups = F / kRowsPerGroup;
        a.gscale = wt->gscale + 2 * (size_t)E;
        a.order = {o.tile, o.offset, o.pair};
        a.epi = plain_out(d, F, true, F);
        st = nvfp4_launch_moe_gemm(a, s);
        if (st != NVFP4_OK)
            break;
        if (f32) {
            a.rest = 1;
            st = launch_rows(from, true, true, ldy, m, K, near, s);
            if (st == NVFP4_OK)
                st = nvfp4_launch_moe_gemm(a, s);
            if (st != NVFP4_OK)
                break;
            a.rest = 0;
        }
        hipLaunchKernelGGL(nvfp4_moe_grad_kernel, dim3((unsigned)pairs), dim3(256), 0, s, d, preact + (size_t)t0 * k * ldp,
                           o.position, ids, weights + (size_t)t0 * k, wt->gscale,
                           dweights ? dweights + (size_t)t0 * k : nullptr, dz, dzexp, (long long)ldp, E, F, activation);
        st = hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
        if (!dX || st != NVFP4_OK)
            continue;
        a.gather = false;
        a.codes = wt->gate_up_codes;
        a.scales = wt->gate_up_scales;
        a.cstride = (long long)b.gu_codes;
        a.sstride = (long long)b.gu_scales;
        a.X = dz;
        a.xexp = dzexp;
        a.ldx = 2 * (long long)F;
        a.K = 2 * F;
        a.row_groups = K / kRowsPerGroup;
        a.gscale = nullptr;   // dz carries the tensor scales
        a.epi = plain_out(rows, K, true, K);
        st = nvfp4_launch_moe_gemm(a, s);
        if (st != NVFP4_OK)
            break;
        st = launch_combine(plain_out(dX + (size_t)t0 * ldx, ldx, false, K), rows, o, nullptr, m, k, K, s);
    }
    return st;
}

}  // extern "C"
