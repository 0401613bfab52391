// The 8-bit projection of include/nvfp4.h: argument checks and dispatch, the
// layout step of its weights, the quantisation of tokens and the product for up
// to 16 tokens.
#include "checks.h"
#include "epilogue.h"
#include "int8.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxInt8K = 131056;   // 128 * 128 * K stays below 2^31
constexpr int kMaxInt8Rows = 1 << 30;
constexpr int kMaxInt8Ld = 1 << 22;

// ---- layout -----------------------------------------------------------------------

__global__ __launch_bounds__(256) void nvfp4_int8_pack_kernel(const int8_t *src, int N, int K, int T, long long chunks,
                                                              u32x4 *dst)
{
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    if (idx >= chunks)
        return;
    const int lane = (int)(idx & 63);
    const long long tile = idx >> 6;
    const int t = (int)(tile % (2 * T));
    const long long row = tile / (2 * T) * 16 + (lane & 15);
    const int col = t * 64 + 16 * (lane >> 4);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (row < N && col < K) {
        const int8_t *s = src + row * K + col;
#pragma unroll
        for (int b = 0; b < 16; ++b)
            v[b / 4] |= (u32)(uint8_t)s[b] << (8 * (b % 4));
    }
    dst[idx] = v;
}

// ---- quantisation ------------------------------------------------------------------

// A row's quantisation: scale = amax / 127, q = rint(127 x / amax), halves to the
// even integer.  `top`: the bits of amax.  For bf16 the quotient of two 8-bit
// mantissas (one times 127) is either a half-integer exactly or at least 2^-17 of
// its value away from one; the product with the reciprocal and one correction by
// its exact remainder is within 2^-23 of it, and gives a representable quotient
// itself: rounding decides as exact arithmetic would.  fp32 rows are divided.
// Both sides of the quotient are first scaled by a power of two that keeps 127 x
// and the reciprocal in range.  A row that holds a NaN or an infinity has scale
// NaN and q = 0; a row of zeros has scale 0.
struct RowScale {
    float mul, div, rcp, scale;
    bool finite;
    __device__ __forceinline__ explicit RowScale(u32 top)
    {
        finite = top < 0x7F800000u;
        const float amax = __builtin_bit_cast(float, top);
        scale = finite ? amax / 127.0f : __builtin_nanf("");
        const float by = amax > 0x1p60f ? 0x1p-64f : (amax < 0x1p-60f ? 0x1p100f : 1.0f);
        mul = 127.0f * by;
        div = finite && top ? amax * by : 1.0f;
        rcp = __builtin_amdgcn_rcpf(div);
    }
    template <bool F32>
    __device__ __forceinline__ int quantize(u32 bits) const
    {
        const float t = __builtin_bit_cast(float, bits) * mul;
        float q;
        if constexpr (F32) {
            q = t / div;
        } else {
            const float q0 = t * rcp;
            q = __builtin_fmaf(__builtin_fmaf(-q0, div, t), rcp, q0);
        }
        return finite ? (int)__builtin_rintf(q) : 0;
    }
};

// One workgroup a row, whose values stay in registers between the maximum and the
// division (the first kHeld vectors of a thread; a longer row is read again).
constexpr int kHeld = 4;

template <bool F32, int kQuantThreads>
__global__ __launch_bounds__(kQuantThreads) void nvfp4_int8_quantize_kernel(const void *src, long long ldx, int K, int8_t *q,
                                                                           long long ldq, float *scale)
{
    const long long t = blockIdx.x;
    const int tid = threadIdx.x;
    const char *row = static_cast<const char *>(src) + t * ldx * (F32 ? 4 : 2);
    struct Vec {
        u32 v[8];   // fp32 bits
    };
    // (a row may be longer than 2^31 bytes)
    auto fetch = [&](int c) {
        Vec r;
        if constexpr (F32) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(row + c * 32LL), b = *reinterpret_cast<const u32x4 *>(row + c * 32LL + 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r.v[j] = a[j];
                r.v[4 + j] = b[j];
            }
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(row + c * 16LL);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r.v[2 * j] = a[j] << 16;
                r.v[2 * j + 1] = a[j] & 0xFFFF0000u;
            }
        }
        return r;
    };
    const int chunks = K / 8;
    Vec held[kHeld];
    u32 top = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int c = tid + j * kQuantThreads;
        if (c < chunks)
            held[j] = fetch(c);
        else
            held[j] = Vec{};
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, held[j].v[e] & 0x7FFFFFFFu);
    for (int c = tid + kHeld * kQuantThreads; c < chunks; c += kQuantThreads) {
        const Vec r = fetch(c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, r.v[e] & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = max(top, (u32)__shfl_xor((int)top, d));
    __shared__ u32 tops[kQuantThreads / 64];
    if ((tid & 63) == 0)
        tops[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 64; ++w)
        top = max(top, tops[w]);
    const RowScale row_scale(top);
    if (tid == 0)
        scale[t] = row_scale.scale;
    auto store = [&](int c, const Vec &r) {
        u32 w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e / 4] |= (u32)(row_scale.quantize<F32>(r.v[e]) & 255) << (8 * (e % 4));
        }
        *reinterpret_cast<u32x2 *>(q + t * ldq + c * 8LL) = u32x2{w[0], w[1]};
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int c = tid + j * kQuantThreads;
        if (c < chunks)
            store(c, held[j]);
    }
    for (int c = tid + kHeld * kQuantThreads; c < chunks; c += kQuantThreads)
        store(c, fetch(c));
}

// ---- up to 16 tokens ------------------------------------------------------------------

struct Int8GemvParams {
    const char *codes;
    const float *wscale, *xscale;
    const void *X;        // int8, or bf16 that the launch quantises
    long long ldx;
    int n, K, T2, RG;     // T2: 64-column tiles
    int rows;             // of a workgroup
    nvfp4_epi_params e;
};

// Most activations a decode launch quantises itself, of eight tokens at most.  Both
// ways, us, weights cold (inside / a launch of its own):
//   n = 1   5120 x 6144 10.0 / 12.5    16384 x 8192 28.0 / 30.8    1024 x 17408 10.2 / 14.9
//   n = 8   5120 x 4096  9.8 / 11.2    16384 x 4096 17.0 / 19.2    1024 x 4096   6.7 / 7.9
//   n = 4   5120 x 8192 13.2 / 14.9    16384 x 12288 43.0 / 40.8   1024 x 12288 11.7 / 11.9
//   n = 8   5120 x 6144 13.7 / 12.8    16384 x 6144 24.2 / 23.0    1024 x 6144   9.9 / 9.9
//   n = 6   5120 x 8192 17.3 / 15.3    16384 x 8192 33.0 / 30.9    1024 x 8192  12.1 / 10.3
//   beyond  n = 8  5120 x 8192 17.6 / 15.6    n = 4  16384 x 17408 58.5 / 54.6
// What decides is a wave's share, whatever the rows: inside is faster up to the 4096
// values that a wave holds, as fast to 2 us slower from 6144 on.
constexpr int kQuantInside = 49152;

// A workgroup has p.rows weight rows, in R windows of 16 (of which the last may use
// fewer, and which need not begin with a row group); its eight waves take
// 64-column tiles in turn.  A window's 1 KiB is one 16-byte load a lane and the
// operand of one v_mfma_i32_16x16x64_i8 as it stands; the tokens' operand is read
// beside it once for the R windows.  Bound by the weight stream; rows are dealt
// out evenly, in fours, since a compute unit reads no faster than its share of the
// memory's bandwidth (5120 x 6144, n = 1, 16 rows a workgroup: 320 of them on 256
// units took 9.4 us).
//
// QUANT: every workgroup quantises the bf16 activations itself, into LDS, while
// its first weights are under way; a launch for it costs 2.5 us more (5120 x 6144,
// n = 1).  Up to eight tokens, a wave each, and kQuantInside values: beyond, the
// arithmetic outlasts the loads that it hides behind.
template <int R, int U, bool QUANT>
__global__ __launch_bounds__(kWaves * 64) void nvfp4_int8_gemv_kernel(Int8GemvParams p)
{
    constexpr int W = kWaves;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int row0 = blockIdx.x * p.rows;
    __shared__ i32x4 part[R][W][64];
    __shared__ u32 tops[W];
    __shared__ float xs[W];
    extern __shared__ __align__(16) char xq[];   // QUANT: [n][64 T2]
    // This lane's row of each window: its offset from the first row group.
    const int rg0 = row0 >> 4, nrg = min((row0 + p.rows + 15) >> 4, p.RG) - rg0;
    const auto cr = resource(p.codes + (size_t)rg0 * p.T2 * 1024, (unsigned)(nrg * p.T2) * 1024u);
    unsigned off[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int at = 16 * r + i, row = row0 + at;
        off[r] = at < p.rows ? (unsigned)(((row >> 4) - rg0) * p.T2 * 1024 + (g * 16 + (row & 15)) * 16) : kOutOfRange;
    }
    u32x4 c[U][R], x[U];
    auto load_codes = [&](int tile, int u) {
        const unsigned behind = tile < p.T2 ? 0 : 1u << 30;   // past the resource: no memory is touched
#pragma unroll
        for (int r = 0; r < R; ++r)
            c[u][r] = __builtin_amdgcn_raw_buffer_load_b128(cr, (int)(off[r] + tile * 1024 + behind), 0, 2);
    };
    const auto xr = resource(p.X, (unsigned)((p.n - 1) * p.ldx + p.K));   // int8
    auto load_x = [&](int tile, int u) {
        const int col = tile * 64 + 16 * g;
        if constexpr (QUANT)
            x[u] = i < p.n && tile < p.T2 ? *reinterpret_cast<const u32x4 *>(xq + i * (p.T2 * 64) + col) : u32x4{0u, 0u, 0u, 0u};
        else
            x[u] = __builtin_amdgcn_raw_buffer_load_b128(xr, i < p.n && col < p.K ? (int)(i * p.ldx + col) : (int)kOutOfRange, 0, 0);
    };
    int tile = wave;
    // QUANT: 8, 4, 2 or 1 waves a token; what a lane reads for the maximum it keeps
    // for the division (a long row's rest is read again).  Loads come back in order:
    // the activations first, the weights while they are quantised.
    constexpr int kHold = 8;
    const int share = p.n == 1 ? 8 : (p.n == 2 ? 4 : (p.n <= 4 ? 2 : 1)), sub = wave % share, t = wave / share;
    const int chunks = p.K / 8, step = 64 * share, c0 = sub * 64 + lane;
    const u32x4 *row = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p.X) + (QUANT && t < p.n ? t : 0) * p.ldx);
    u32x4 held[QUANT ? kHold : 1];
    if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < kHold; ++j)
            held[j] = t < p.n && c0 + j * step < chunks ? row[c0 + j * step] : u32x4{0u, 0u, 0u, 0u};
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        load_codes(tile + u * W, u);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (QUANT) {
        u32 top = 0;
        auto largest = [&](const u32x4 v) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                top = max(top, max((v[q] << 16) & 0x7FFF0000u, v[q] & 0x7FFF0000u));
        };
        if (t < p.n) {
#pragma unroll
            for (int j = 0; j < kHold; ++j)
                largest(held[j]);
            for (int c = c0 + kHold * step; c < chunks; c += step)
                largest(row[c]);
#pragma unroll
            for (int d = 1; d < 64; d *= 2)
                top = max(top, (u32)__shfl_xor((int)top, d));
            if (lane == 0)
                tops[wave] = top;
        }
        __syncthreads();
        if (t < p.n) {
            for (int w = 0; w < share; ++w)
                top = max(top, tops[t * share + w]);
            const RowScale scale(top);
            if (sub == 0 && lane == 0)
                xs[t] = scale.scale;
            auto store = [&](int c, const u32x4 v) {
                u32 w[2] = {0u, 0u};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const u32 lo = scale.quantize<false>(v[q] << 16) & 255, hi = scale.quantize<false>(v[q] & 0xFFFF0000u) & 255;
                    w[q / 2] |= (lo | hi << 8) << (16 * (q % 2));
                }
                *reinterpret_cast<u32x2 *>(xq + t * (p.T2 * 64) + c * 8) = u32x2{w[0], w[1]};
            };
#pragma unroll
            for (int j = 0; j < kHold; ++j)
                if (c0 + j * step < p.T2 * 8)      // (the columns behind K are zeros)
                    store(c0 + j * step, held[j]);
            for (int c = c0 + kHold * step; c < p.T2 * 8; c += step)
                store(c, c < chunks ? row[c] : u32x4{0u, 0u, 0u, 0u});
        }
        __syncthreads();
    }
    i32x4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        acc[r] = i32x4{0, 0, 0, 0};
    if constexpr (!QUANT) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_x(tile + u * W, u);
    }
    for (; tile < p.T2; tile += W * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (QUANT)
                load_x(tile + u * W, u);
#pragma unroll
            for (int r = 0; r < R; ++r)
                acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x[u]), __builtin_bit_cast(i32x4, c[u][r]),
                                                               acc[r], 0, 0, 0);
            load_codes(tile + W * (U + u), u);
            if constexpr (!QUANT)
                load_x(tile + W * (U + u), u);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        part[r][wave][lane] = acc[r];
    __syncthreads();
    // lane (i, g), component v: token 4 g + v, weight row i
    for (int o = tid; o < R * 256; o += kWaves * 64) {
        const int r = o >> 8, l = (o >> 2) & 63, v = o & 3;
        const int tok = 4 * (l >> 4) + v, at = 16 * r + (l & 15), row = row0 + at;
        if (tok >= p.n || at >= p.rows || row >= p.e.N)
            continue;
        int s = 0;
#pragma unroll
        for (int w = 0; w < W; ++w)
            s += reinterpret_cast<const int *>(&part[r][w][l])[v];
        linear_out(p.e, tok, row, (float)s * (QUANT ? xs[tok] : p.xscale[tok]) * p.wscale[row]);
    }
}

// Whether a decode launch quantises its activations itself.
bool quant_inside(int n, int K)
{
    return n <= kWaves && (long long)n * K <= kQuantInside;
}

template <bool QUANT>
int launch_gemv(Int8GemvParams p, hipStream_t stream)
{
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    // one workgroup a compute unit, or as many as keep them at 64 rows
    const long long units = ((long long)p.e.N + 64LL * cus - 1) / (64LL * cus) * cus;
    p.rows = (int)((p.e.N + 4 * units - 1) / (4 * units) * 4);
    const dim3 grid((unsigned)((p.e.N + p.rows - 1) / p.rows)), block(kWaves * 64);
    const unsigned lds = QUANT ? (unsigned)(p.n * p.T2 * 64) : 0u;
    switch ((p.rows + 15) / 16) {
    case 1: hipLaunchKernelGGL((nvfp4_int8_gemv_kernel<1, 8, QUANT>), grid, block, lds, stream, p); break;
    case 2: hipLaunchKernelGGL((nvfp4_int8_gemv_kernel<2, 6, QUANT>), grid, block, lds, stream, p); break;
    case 3: hipLaunchKernelGGL((nvfp4_int8_gemv_kernel<3, 4, QUANT>), grid, block, lds, stream, p); break;
    default: hipLaunchKernelGGL((nvfp4_int8_gemv_kernel<4, 4, QUANT>), grid, block, lds, stream, p); break;
    }
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int launch_gemv(const nvfp4_int8_args &a, const void *X, long long ldx, hipStream_t stream)
{
    Int8GemvParams p = {};
    p.codes = reinterpret_cast<const char *>(a.codes);
    p.wscale = a.wscale;
    p.xscale = a.xscale;
    p.X = X;
    p.ldx = ldx;
    p.n = a.n;
    p.K = a.K;
    p.T2 = 2 * (int)k_tiles(a.K);
    p.RG = (int)row_groups(a.N);
    p.e = a.epi;
    return a.xscale ? launch_gemv<false>(p, stream) : launch_gemv<true>(p, stream);
}

// K parts added, then the epilogue: four outputs of a token a thread.
__global__ __launch_bounds__(256) void nvfp4_int8_reduce_kernel(nvfp4_epi_params e, const int *P, const float *wscale,
                                                                const float *xscale, int n, int pitch, int ks)
{
    const int quads = (e.N + 3) / 4;
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long tok = idx / quads;
    if (tok >= n)
        return;
    const int r = (int)(idx % quads) * 4;
    i32x4 s = {0, 0, 0, 0};
    for (int k = 0; k < ks; ++k)
        s += *reinterpret_cast<const i32x4 *>(P + ((long long)k * n + tok) * pitch + r);
    const float sx = xscale[tok];
    f32x4 z;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        z[j] = r + j < e.N ? (float)s[j] * sx * wscale[r + j] : 0.f;
    linear_out4(e, (int)tok, r, z);
}

size_t round256(size_t bytes)
{
    return (bytes + 255) / 256 * 256;
}

struct Space {
    size_t q, scale, parts;   // quantised tokens, their scales, K parts
    size_t total() const { return q + scale + parts; }
};

Space space_of(int n, int N, int K, bool quantize)
{
    Space s = {};
    if (n < 1)
        return s;
    if (quantize && !quant_inside(n, K)) {
        s.q = round256((size_t)n * K);
        s.scale = round256((size_t)n * 4);
    }
    if (n > NVFP4_MAX_TOKENS) {
        const int rg = (int)row_groups(N), ks = nvfp4_plan_int8(n, rg, K).ks;
        s.parts = ks > 1 ? round256((size_t)ks * n * rg * 16 * 4) : 0;
    }
    return s;
}

int check_shape(int n, int N, int K)
{
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || N < 1 || N > kMaxInt8Rows || K < 1)
        return NVFP4_ERR_RANGE;
    return K % 16 != 0 || K > kMaxInt8K ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

int launch_quantize(const void *X, int dtype, long long ldx, int n, int K, int8_t *q, long long ldq, float *scale, hipStream_t s)
{
    // (a row of 8192 stays in the registers of 256 threads; n = 300, K = 17408: 9.1 us
    // with 256, 7.8 with 1024)
    const bool f32 = dtype == NVFP4_DTYPE_F32;
    if (K <= 8192) {
        auto k = f32 ? nvfp4_int8_quantize_kernel<true, 256> : nvfp4_int8_quantize_kernel<false, 256>;
        hipLaunchKernelGGL(k, dim3((unsigned)n), dim3(256), 0, s, X, ldx, K, q, ldq, scale);
    } else {
        auto k = f32 ? nvfp4_int8_quantize_kernel<true, 1024> : nvfp4_int8_quantize_kernel<false, 1024>;
        hipLaunchKernelGGL(k, dim3((unsigned)n), dim3(1024), 0, s, X, ldx, K, q, ldq, scale);
    }
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t nvfp4_int8_packed_bytes(int N, int K)
{
    return check_shape(0, N, K) == NVFP4_OK ? (size_t)row_groups(N) * k_tiles(K) * 2048 : 0;
}

int nvfp4_int8_pack(const int8_t *codes, int N, int K, int8_t *packed, void *stream)
{
    if (!codes || !packed)
        return NVFP4_ERR_NULL;
    int st = check_shape(0, N, K);
    if (st != NVFP4_OK)
        return st;
    if (!is_aligned(packed, 16))
        return NVFP4_ERR_ALIGN;
    const size_t bytes = nvfp4_int8_packed_bytes(N, K);
    if (overlap(codes, (size_t)N * K, packed, bytes))
        return NVFP4_ERR_OVERLAP;
    const long long chunks = (long long)(bytes / 16);
    if ((chunks + 255) / 256 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    int cus = 0;
    st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    hipLaunchKernelGGL(nvfp4_int8_pack_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, (hipStream_t)stream, codes, N,
                       K, (int)k_tiles(K), chunks, (u32x4 *)packed);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

int nvfp4_int8_quantize(const void *X, int dtype, int64_t ldx, int n, int K, int8_t *q, int64_t ldq, float *scale, void *stream)
{
    if (n > 0 && (!X || !q || !scale))
        return NVFP4_ERR_NULL;
    if (n < 0 || K < 1 || !valid_dtype(dtype) || ldx < K || ldq < K)
        return NVFP4_ERR_RANGE;
    if (K % 16 != 0)
        return NVFP4_ERR_SHAPE;
    const int size = dtype_size(dtype);
    if (!is_aligned(X, 16) || (n > 1 && ldx * size % 16 != 0) || !is_aligned(q, 16) || (n > 1 && ldq % 16 != 0) || !is_aligned(scale, 4))
        return NVFP4_ERR_ALIGN;
    const Region x = matrix(X, n, ldx, K, size), y = matrix(q, n, ldq, K, 1), s = array(scale, (size_t)n * 4);
    if (overlap(x, y) || overlap(x, s) || overlap(y, s))
        return NVFP4_ERR_OVERLAP;
    if (n == 0)
        return NVFP4_OK;
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    return st != NVFP4_OK ? st : launch_quantize(X, dtype, ldx, n, K, q, ldq, scale, (hipStream_t)stream);
}

int nvfp4_int8_geometry(int n, int N, int K, int *rows_per_workgroup, int *tokens_per_workgroup, int *k_groups, int *k_parts)
{
    if (!rows_per_workgroup || !tokens_per_workgroup || !k_groups || !k_parts)
        return NVFP4_ERR_NULL;
    if (n <= NVFP4_MAX_TOKENS)
        return NVFP4_ERR_RANGE;
    const int st = check_shape(n, N, K);
    if (st != NVFP4_OK)
        return st;
    const nvfp4_int8_plan plan = nvfp4_plan_int8(n, (int)row_groups(N), K);
    nvfp4_int8_tile(plan.tile, rows_per_workgroup, tokens_per_workgroup, k_groups);
    *k_parts = plan.ks;
    return NVFP4_OK;
}

size_t nvfp4_int8_linear_workspace_bytes(int n, int N, int K, int quantize)
{
    return check_shape(n, N, K) == NVFP4_OK ? space_of(n, N, K, quantize != 0).total() : 0;
}

int nvfp4_int8_linear(const int8_t *Wq, const float *wscale, const void *X, int64_t ldx, const float *xscale, void *Y, int64_t ldy,
                      int n, int N, int K, const nvfp4_epilogue *epilogue, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!Wq || !wscale || !epilogue || (n > 0 && (!X || !Y)))
        return NVFP4_ERR_NULL;
    const nvfp4_epilogue &ep = *epilogue;
    int st = check_shape(n, N, K);
    if (st != NVFP4_OK)
        return st;
    const bool quantize = !xscale;
    const int xs = quantize ? 2 : 1;
    if (ep.activation < NVFP4_ACT_NONE || ep.activation > NVFP4_ACT_GELU_TANH || !valid_dtype(ep.out_dtype) ||
        (ep.bias && !valid_dtype(ep.bias_dtype)) || (ep.residual && !valid_dtype(ep.residual_dtype)) || ep.up_bias || ep.preact ||
        ldx < K || ldy < N || (ep.residual && ep.ldr < N))
        return NVFP4_ERR_RANGE;
    if (ldx > kMaxInt8Ld || ldy > INT32_MAX || ep.ldr > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    const int os = dtype_size(ep.out_dtype), bs = dtype_size(ep.bias_dtype), rs = dtype_size(ep.residual_dtype);
    if (!is_aligned(Wq, 16) || !is_aligned(wscale, 4) || !is_aligned(X, 16) || (n > 1 && ldx * xs % 16 != 0) ||
        !is_aligned(xscale, 4) || !is_aligned(Y, os) || (ep.bias && !is_aligned(ep.bias, bs)) ||
        (ep.residual && !is_aligned(ep.residual, rs)))
        return NVFP4_ERR_ALIGN;
    if (n == 0)
        return NVFP4_OK;
    const Space w = space_of(n, N, K, quantize);
    if (w.total() && (!workspace || workspace_bytes < w.total()))
        return NVFP4_ERR_WORKSPACE;
    if (w.total() && !is_aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const Region in[] = {array(Wq, nvfp4_int8_packed_bytes(N, K)), array(wscale, 4 * (size_t)N), matrix(X, n, ldx, K, xs),
                         array(xscale, 4 * (size_t)n), array(ep.bias, (size_t)N * bs)};
    const Region y = matrix(Y, n, ldy, N, os), residual = matrix(ep.residual, n, ep.ldr, N, rs);
    const Region space = array(workspace, w.total());
    const bool in_place = ep.residual == Y && ep.ldr == ldy && ep.residual_dtype == ep.out_dtype;
    if (any_overlap(y, in) || any_overlap(space, in) || overlap(space, y) || overlap(space, residual) ||
        (!in_place && overlap(y, residual)))
        return NVFP4_ERR_OVERLAP;
    int cus = 0;
    st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    char *ws = static_cast<char *>(workspace);
    nvfp4_int8_args a = {};
    a.codes = Wq;
    a.wscale = wscale;
    a.n = n;
    a.N = N;
    a.K = K;
    if (w.q) {
        int8_t *q = reinterpret_cast<int8_t *>(ws);
        float *scale = reinterpret_cast<float *>(ws + w.q);
        st = launch_quantize(X, NVFP4_DTYPE_BF16, ldx, n, K, q, K, scale, s);
        if (st != NVFP4_OK)
            return st;
        a.X = q;
        a.ldx = K;
        a.xscale = scale;
    } else {
        a.X = static_cast<const int8_t *>(X);
        a.ldx = ldx;
        a.xscale = xscale;
    }
    a.partial = reinterpret_cast<int32_t *>(ws + w.q + w.scale);
    nvfp4_epi_params &e = a.epi;
    e.bias = ep.bias;
    e.residual = ep.residual;
    e.out = Y;
    e.ldr = (int)ep.ldr;
    e.ldo = (int)ldy;
    e.gscale = 1.0f;
    e.N = N;
    e.flags = ep.activation | (ep.bias_dtype == NVFP4_DTYPE_F32 ? kEpiBiasF32 : 0) |
              (ep.residual_dtype == NVFP4_DTYPE_F32 ? kEpiResidualF32 : 0) | (ep.out_dtype == NVFP4_DTYPE_F32 ? kEpiOutF32 : 0);
    if (ldy % 4 == 0 && is_aligned(Y, 4 * os) && (!ep.bias || is_aligned(ep.bias, 4 * bs)) &&
        (!ep.residual || (ep.ldr % 4 == 0 && is_aligned(ep.residual, 4 * rs))))
        e.flags |= kEpiVec;
    if (n <= NVFP4_MAX_TOKENS)
        return w.q || !quantize ? launch_gemv(a, a.X, a.ldx, s) : launch_gemv(a, X, ldx, s);
    const nvfp4_int8_plan plan = nvfp4_plan_int8(n, (int)row_groups(N), K);
    st = nvfp4_launch_int8_gemm(a, plan, s);
    if (st != NVFP4_OK || plan.ks == 1)
        return st;
    const long long quads = ((long long)N + 3) / 4 * n;
    hipLaunchKernelGGL(nvfp4_int8_reduce_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, e, a.partial, wscale,
                       a.xscale, n, (int)row_groups(N) * 16, plan.ks);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

}  // extern "C"
