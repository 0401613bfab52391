// The fused operators of include/nvfp4.h: argument checks and dispatch, the
// layout steps of their weights, the epilogue of K parts and the elementwise
// half of their gradients.
#include "epilogue.h"
#include "fused_gemm.h"

namespace {

// ---- layout steps (once, at load time) -------------------------------------------

// Row groups of two packed weights in turn: gate 0, up 0, gate 1, up 1, ...
// `per` 16-byte words a row group.
__global__ void nvfp4_interleave_kernel(const u32x4 *gate, const u32x4 *up, long long per, long long words, u32x4 *out)
{
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= words)
        return;
    const long long rg = idx / per;
    out[idx] = (rg & 1 ? up : gate)[(rg >> 1) * per + idx % per];
}

// Transposed tiles from packed ones.  One thread per 16-byte lane chunk of a
// transposed tile: lane (i, g) of tile (kb, rt) holds column 16 kb + i at the
// rows rt*128 + 16 b + 4 g + e (b = 0..7, e = 0..3), the same order in which a
// packed tile's lane holds columns.
__global__ void nvfp4_transpose_codes_kernel(const uint8_t *codes, int T, int RG, int TT, long long chunks, u32x4 *out)
{
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= chunks)
        return;
    const int l = (int)(idx & 63);
    const long long tile = idx >> 6;
    const int rt = (int)(tile % TT);
    const int k = (int)(tile / TT) * 16 + (l & 15);
    const int g = l >> 4;
    // within a row's tile: lane 16 * (k % 16 / 4) + row % 16, byte and nibble of k
    const int kt = k / kTileK, kk = k % kTileK;
    const int byte = 2 * (kk >> 4) + ((kk & 3) >> 1), shift = 4 * (kk & 1);
    u32 w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int q = 0; q < 32; ++q) {
        const int r = rt * kTileK + 16 * (q >> 2) + 4 * g + (q & 3);
        const int rg = r >> 4;
        if (rg < RG) {
            const long long src = ((long long)rg * T + kt) * 64 + ((kk & 15) >> 2) * 16 + (r & 15);
            w[q >> 3] |= (u32)((codes[src * 16 + byte] >> shift) & 15) << (4 * (q & 7));
        }
    }
    out[idx] = u32x4{w[0], w[1], w[2], w[3]};
}

// One thread per 4 scale bytes: of block column kb, rows rt*128 + 16 b + 4 g + e
// at byte g*32 + b*4 + e of the tile's 128.
__global__ void nvfp4_transpose_scales_kernel(const uint8_t *scales, int T, int RG, int TT, long long words, u32 *out)
{
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (idx >= words)
        return;
    const int q = (int)(idx & 31);
    const long long tile = idx >> 5;
    const int rt = (int)(tile % TT);
    const int kb = (int)(tile / TT);
    const int g = q >> 3, b = q & 7;
    u32 w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = rt * kTileK + 16 * b + 4 * g + e;
        const int rg = r >> 4;
        if (rg < RG)
            w |= (u32)scales[(((long long)rg * T + kb / kBlocksPerTile) * 16 + (r & 15)) * 8 + kb % kBlocksPerTile]
                 << (8 * e);
    }
    out[idx] = w;
}

// ---- K parts ------------------------------------------------------------------------

// The parts of each output added in part order, then the epilogue: one thread
// for four consecutive outputs of a token, the parts of a batch in flight
// together.  P: [ks][n][pitch].
template <bool GATED>
__global__ __launch_bounds__(256) void nvfp4_fused_reduce_kernel(nvfp4_epi_params e, const float *P, int n, int pitch, int ks)
{
    const int quads = (e.N + 3) / 4;
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long tok = idx / quads;
    if (tok >= n)
        return;
    const int r = (int)(idx % quads) * 4;
    const long long count = (long long)n * pitch;
    auto total = [&](long long row) {
        const f32x4 *src = reinterpret_cast<const f32x4 *>(P + tok * pitch + row);
        constexpr int kBatch = 4;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        for (int q0 = 0; q0 < ks; q0 += kBatch) {
            f32x4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                v[j] = q0 + j < ks ? __builtin_nontemporal_load(src + (q0 + j) * count / 4) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (q0 + j < ks)
                    s = q0 + j == 0 ? v[j] : s + v[j];
        }
        return s;
    };
    if constexpr (GATED)
        gated_out4(e, (int)tok, r, total(gated_row(r, 0)), total(gated_row(r, 1)));
    else
        linear_out4(e, (int)tok, r, total(r));
}

// ---- the elementwise half of the gradients ---------------------------------------------

struct GradParams {
    const void *dy;
    const float *z;          // pre-activations, or null (identity)
    uint16_t *dz;            // bf16, or null
    float *partial;          // [row blocks][halves][cols] column sums, or null
    void *db[2];             // bias gradients, or null
    long long ldy, ldz, lddz;
    int n, N, cols;          // outputs a token; columns visited (padded with zero gradients)
    int act, dy_f32, db_f32, vec;
    int rows_per_block;
    float gscale[2];
};

constexpr int kGradCols = 256;   // columns of a block: 32 threads x 8, times 8 rows at once

__device__ __forceinline__ void store_db(const GradParams &p, int half, int col, float v)
{
    if (p.db[half] && col < p.N)
        store_any(p.db[half], col, p.db_f32, v);
}

// dZ = dY act'(Z) (linear), or of a gate and up row (dH U act'(G), dH act(G))
// times its tensor scale (gated, so that one product with the gated weight
// serves both), each rounded to bf16; and the column sums of the unrounded,
// unscaled values.  The rounding makes dZ an operand of the bf16 matrix
// instructions: dX is then off by 2.3e-3 of its norm, of which its own rounding
// to bf16 is 1.7e-3 (linear 16384 x 5120, n = 1536; gated 2 x 17408 x 5120, n =
// 1024).  A second operand for the remainder would double the matrix
// instructions of that product, seven eighths of the backward pass.  Memory
// bound: dY (bf16) and Z (fp32) in, dZ out, 8 bytes an output (gated 14).  A
// block takes rows_per_block rows, eight at a time, sums them in a fixed order,
// and blocks are added in order: no atomics.
template <bool GATED>
__global__ __launch_bounds__(256) void nvfp4_grad_kernel(GradParams p)
{
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c0 = blockIdx.x * kGradCols + cx * 8;
    const int t1 = min(p.n, (int)(blockIdx.y + 1) * p.rows_per_block);
    float sum[2][8] = {};
    if (c0 < p.cols) {
        for (int t = blockIdx.y * p.rows_per_block + ry; t < t1; t += 8) {
            float dy[8];
            const long long at = t * p.ldy + c0;
            if (p.vec && c0 + 8 <= p.N) {
                const f32x4 a = load_any4(p.dy, at, p.dy_f32), b = load_any4(p.dy, at + 4, p.dy_f32);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dy[e] = a[e];
                    dy[4 + e] = b[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dy[e] = c0 + e < p.N ? load_any(p.dy, at + e, p.dy_f32) : 0.f;
            }
            float z[2][8] = {};
            // (a gated row has all the columns up to a multiple of 16)
            auto fetch = [&](int half, long long col) {
                const float *row = p.z + t * p.ldz + col;
                if (GATED || c0 + 8 <= p.N) {
                    const f32x4 a = reinterpret_cast<const f32x4 *>(row)[0], b = reinterpret_cast<const f32x4 *>(row)[1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[half][e] = a[e];
                        z[half][4 + e] = b[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[half][e] = c0 + e < p.N ? row[e] : 0.f;
                }
            };
            if (p.z)
                fetch(0, GATED ? gated_row(c0, 0) : c0);
            if constexpr (GATED)
                fetch(1, gated_row(c0, 1));
            u32x4 out[2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d[2];
                // past the last output the pre-activations are not defined
                const bool in = c0 + e < p.N;
                if constexpr (GATED) {
                    d[0] = in ? dy[e] * z[1][e] * activate_grad(z[0][e], p.act) : 0.f;
                    d[1] = in ? dy[e] * activate(z[0][e], p.act) : 0.f;
                } else {
                    d[0] = in ? (p.act == NVFP4_ACT_NONE ? dy[e] : dy[e] * activate_grad(z[0][e], p.act)) : 0.f;
                    d[1] = 0.f;
                }
#pragma unroll
                for (int h = 0; h < (GATED ? 2 : 1); ++h) {
                    sum[h][e] += d[h];
                    const u32 b = f32_to_bf16_bits(GATED ? d[h] * p.gscale[h] : d[h]);
                    out[h][e >> 1] = e & 1 ? out[h][e >> 1] | b << 16 : b;
                }
            }
            if (p.dz) {
                *reinterpret_cast<u32x4 *>(p.dz + t * p.lddz + (GATED ? gated_row(c0, 0) : c0)) = out[0];
                if constexpr (GATED)
                    *reinterpret_cast<u32x4 *>(p.dz + t * p.lddz + gated_row(c0, 1)) = out[1];
            }
        }
    }
    if (!p.db[0] && !p.db[1])
        return;
    __shared__ float part[8][kGradCols + 8];
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[ry][cx * 8 + e] = sum[h][e];
        __syncthreads();
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y)
            s += part[y][threadIdx.x];
        const int col = blockIdx.x * kGradCols + threadIdx.x;
        if (col >= p.cols)
            continue;
        if (gridDim.y == 1)
            store_db(p, h, col, s);
        else
            p.partial[((long long)blockIdx.y * (GATED ? 2 : 1) + h) * p.cols + col] = s;
    }
}

// Bias gradients from the row blocks' sums, added in block order.
__global__ __launch_bounds__(256) void nvfp4_grad_sum_kernel(GradParams p, int blocks, int halves)
{
    const int col = blockIdx.x * 256 + threadIdx.x;
    const int h = blockIdx.y;
    if (col >= p.N)
        return;
    float s = 0.f;
    constexpr int kBatch = 8;   // loads in flight together
    for (int y0 = 0; y0 < blocks; y0 += kBatch) {
        float v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            v[j] = y0 + j < blocks ? p.partial[((long long)(y0 + j) * halves + h) * p.cols + col] : 0.f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            s += v[j];
    }
    store_db(p, h, col, s);
}

// ---- host side --------------------------------------------------------------------------

constexpr int kMaxRows = 1 << 30;     // of a packed weight: rounded up to a tile they stay within 32 bits
constexpr int kMaxStride = 1 << 22;   // elements between rows: keeps a token tile's offsets within 32 bits

bool is_aligned(const void *p, size_t a)
{
    return ((uintptr_t)p % a) == 0;
}

// Memory an argument covers, in bytes: an array, or a matrix whose rows of
// `width` bytes lie `ld` apart.
struct Region {
    const void *p;
    size_t rows, ld, width;
    size_t span() const { return rows ? (rows - 1) * ld + width : 0; }
};

Region array(const void *p, size_t bytes)
{
    return {p, p && bytes ? 1u : 0u, 0, bytes};
}

Region matrix(const void *p, int n, int64_t ld, int64_t cols, int size)
{
    return {p, p && n > 0 ? (size_t)n : 0u, (size_t)ld * size, (size_t)cols * size};
}

// Rows that take turns in memory with one stride (neighbouring columns of one
// buffer) lie apart although their spans do not.
bool overlap(const Region &a, const Region &b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (!a.rows || !b.rows || x >= y + b.span() || y >= x + a.span())
        return false;
    const size_t ld = a.rows > 1 ? a.ld : b.ld;   // one row fits any stride
    if ((a.rows == 1 && b.rows == 1) || (a.rows > 1 && b.rows > 1 && a.ld != b.ld) || a.width > ld || b.width > ld)
        return true;
    const size_t from = (y % ld + ld - x % ld) % ld;   // b's first column, in a's rows
    return from < a.width || from + b.width > ld;
}

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    return overlap(array(a, an), array(b, bn));
}

// Whether an output overlaps an argument.
template <int I>
bool any_overlap(const Region &out, const Region (&args)[I])
{
    for (const Region &a : args)
        if (overlap(out, a))
            return true;
    return false;
}

bool valid_dtype(int d)
{
    return d == NVFP4_DTYPE_F32 || d == NVFP4_DTYPE_BF16;
}

int dtype_size(int d)
{
    return d == NVFP4_DTYPE_F32 ? 4 : 2;
}

// Shapes, strides and pointers that linear and gated share.  N: outputs a
// token; rows: rows of the packed weight.
int validate_forward(const uint8_t *Wq, const uint8_t *Wscale, const uint16_t *X, int64_t ldx, const void *out,
                     int64_t ldo, int n, int N, int rows, int K, const nvfp4_epilogue *ep, bool gated)
{
    if (!Wq || !Wscale || !ep || (n > 0 && (!X || !out)))
        return NVFP4_ERR_NULL;
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || N < 1 || N > kMaxRows || K < 1)
        return NVFP4_ERR_RANGE;
    if (K % 16 != 0 || K > kMaxK)
        return NVFP4_ERR_SHAPE;
    if (ep->activation < NVFP4_ACT_NONE || ep->activation > NVFP4_ACT_GELU_TANH || !valid_dtype(ep->out_dtype) ||
        ((ep->bias || ep->up_bias) && !valid_dtype(ep->bias_dtype)) ||
        (ep->residual && !valid_dtype(ep->residual_dtype)))
        return NVFP4_ERR_RANGE;
    if ((gated && ep->residual) || (!gated && ep->up_bias))
        return NVFP4_ERR_RANGE;
    const int64_t pre_cols = gated ? rows : N;
    if (ldx < K || ldo < N || (ep->residual && ep->ldr < N) || (ep->preact && ep->ldp < pre_cols))
        return NVFP4_ERR_RANGE;
    if (ldx > kMaxStride || ldo > INT32_MAX || ep->ldr > INT32_MAX || ep->ldp > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    const int os = dtype_size(ep->out_dtype);
    if (!is_aligned(Wq, 16) || !is_aligned(Wscale, 16) || !is_aligned(X, 16) || (n > 1 && ldx % 8 != 0) ||
        !is_aligned(out, os) || (ep->bias && !is_aligned(ep->bias, dtype_size(ep->bias_dtype))) ||
        (ep->up_bias && !is_aligned(ep->up_bias, dtype_size(ep->bias_dtype))) ||
        (ep->residual && !is_aligned(ep->residual, dtype_size(ep->residual_dtype))))
        return NVFP4_ERR_ALIGN;
    if (ep->preact && (!is_aligned(ep->preact, 16) || ep->ldp % 8 != 0))
        return NVFP4_ERR_ALIGN;
    // Workgroups read what others write unless the outputs lie apart.  The
    // residual may be the output itself: each element is read by the thread
    // that then writes it.
    const size_t bn = (size_t)N * dtype_size(ep->bias_dtype);
    const Region y = matrix(out, n, ldo, N, os), z = matrix(ep->preact, n, ep->ldp, pre_cols, 4);
    const Region residual = matrix(ep->residual, n, ep->ldr, N, dtype_size(ep->residual_dtype));
    const Region in[] = {matrix(X, n, ldx, K, 2), array(Wq, nvfp4_packed_codes_bytes(rows, K)),
                         array(Wscale, nvfp4_packed_scales_bytes(rows, K)), array(ep->bias, bn), array(ep->up_bias, bn)};
    const bool in_place = ep->residual == out && ep->ldr == ldo && ep->residual_dtype == ep->out_dtype;
    if (any_overlap(y, in) || any_overlap(z, in) || overlap(y, z) || overlap(z, residual) ||
        (!in_place && overlap(y, residual)))
        return NVFP4_ERR_OVERLAP;
    return NVFP4_OK;
}

nvfp4_epi_params epi_params(const nvfp4_epilogue *ep, float gscale, float up_gscale, void *out, int64_t ldo, int N,
                            int64_t pre_cols)
{
    nvfp4_epi_params e = {};
    e.bias = ep->bias;
    e.up_bias = ep->up_bias;
    e.residual = ep->residual;
    e.preact = ep->preact;
    e.out = out;
    e.ldr = (int)ep->ldr;
    e.ldp = (int)ep->ldp;
    e.ldo = (int)ldo;
    e.gscale = gscale;
    e.up_gscale = up_gscale;
    e.N = N;
    e.flags = ep->activation | (ep->bias_dtype == NVFP4_DTYPE_F32 ? kEpiBiasF32 : 0) |
              (ep->residual_dtype == NVFP4_DTYPE_F32 ? kEpiResidualF32 : 0) |
              (ep->out_dtype == NVFP4_DTYPE_F32 ? kEpiOutF32 : 0);
    const int bs = 4 * dtype_size(ep->bias_dtype), rs = 4 * dtype_size(ep->residual_dtype);
    const int os = 4 * dtype_size(ep->out_dtype);
    const bool vec = ldo % 4 == 0 && is_aligned(out, os) && (!ep->bias || is_aligned(ep->bias, bs)) &&
            (!ep->up_bias || is_aligned(ep->up_bias, bs)) &&
            (!ep->residual || (ep->ldr % 4 == 0 && is_aligned(ep->residual, rs)));
    if (vec)
        e.flags |= kEpiVec;
    return e;
}

int padded_rows(int rows)
{
    return (int)(kRowsPerGroup * row_groups(rows));
}

// Workspace of a call that runs in K parts: fp32 sums [ks][n][rows to 16].
size_t parts_bytes(int n, int rows, int K)
{
    if (n < 1)
        return 0;
    const int ks = n <= NVFP4_MAX_TOKENS ? nvfp4_gemv_kparts(rows, K)
                                         : nvfp4_plan_fused_gemm(n, (int)row_groups(rows), K).ks;
    return ks > 1 ? (size_t)ks * n * padded_rows(rows) * sizeof(float) : 0;
}

// A workspace for the partial sums of a product with a packed weight of
// row_groups x T tiles: large enough, aligned, apart from what the two launches
// read and write.
int check_workspace(const void *workspace, size_t bytes, size_t need, const uint8_t *codes, const uint8_t *scales,
                    long long tiles, const uint16_t *X, long long ldx, int n, int K, const nvfp4_epi_params &e,
                    long long pre_cols)
{
    if (!need)
        return NVFP4_OK;
    if (!workspace || bytes < need)
        return NVFP4_ERR_WORKSPACE;
    if (!is_aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const size_t bn = (size_t)e.N * (e.flags & kEpiBiasF32 ? 4 : 2);
    const Region others[] = {array(codes, tiles * 1024), array(scales, tiles * 128), matrix(X, n, ldx, K, 2),
                             array(e.bias, bn), array(e.up_bias, bn),
                             matrix(e.out, n, e.ldo, e.N, e.flags & kEpiOutF32 ? 4 : 2),
                             matrix(e.residual, n, e.ldr, e.N, e.flags & kEpiResidualF32 ? 4 : 2),
                             matrix(e.preact, n, e.ldp, pre_cols, 4)};
    if (any_overlap(array(workspace, need), others))
        return NVFP4_ERR_OVERLAP;
    return NVFP4_OK;
}

// The second launch of a call in K parts.
int launch_reduce(const nvfp4_epi_params &e, const float *partial, int n, int pitch, int ks, bool gated, hipStream_t stream)
{
    const long long quads = ((long long)e.N + 3) / 4 * n;
    const dim3 grid((unsigned)((quads + 255) / 256));
    if (gated)
        hipLaunchKernelGGL(nvfp4_fused_reduce_kernel<true>, grid, dim3(256), 0, stream, e, partial, n, pitch, ks);
    else
        hipLaunchKernelGGL(nvfp4_fused_reduce_kernel<false>, grid, dim3(256), 0, stream, e, partial, n, pitch, ks);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// The many-token product; rows: of the packed weight (its K tiles when transposed).
int launch_product(nvfp4_fused_gemm_args a, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const nvfp4_fused_gemm_plan plan = nvfp4_plan_fused_gemm(a.n, a.row_groups, a.K);
    const int pitch = a.row_groups * kRowsPerGroup;
    int st = check_workspace(workspace, workspace_bytes, plan.ks > 1 ? (size_t)plan.ks * a.n * pitch * sizeof(float) : 0,
                             a.codes, a.scales, (long long)a.row_groups * k_tiles(a.K), a.X, a.ldx, a.n, a.K, a.epi, a.mode == 1 ? pitch : a.epi.N);
    if (st != NVFP4_OK)
        return st;
    a.partial = static_cast<float *>(workspace);
    st = nvfp4_launch_fused_gemm(a, plan, stream);
    if (st != NVFP4_OK || plan.ks == 1)
        return st;
    return launch_reduce(a.epi, a.partial, a.n, pitch, plan.ks, a.mode == 1, stream);
}

// rows: rows of the packed weight; gated: its row groups alternate gate, up.
int forward(const uint8_t *Wq, const uint8_t *Wscale, const uint16_t *X, int64_t ldx, int n, int rows, int K,
            const nvfp4_epi_params &e, bool gated, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (n <= NVFP4_MAX_TOKENS) {
        const int ks = nvfp4_gemv_kparts(rows, K);
        if (ks < 1)
            return -ks;
        nvfp4_fused_gemv_args a = {};
        a.codes = Wq;
        a.scales = Wscale;
        a.X = X;
        a.ldx = (int)ldx;
        a.n = n;
        a.K = K;
        a.rows = padded_rows(rows);
        a.units = (int)(row_groups(rows) / (gated && ks == 1 ? 2 : 1));
        a.ks = ks;
        a.epi = e;
        if (ks == 1)
            return gated ? nvfp4_launch_fused_gemv_gated(a, stream) : nvfp4_launch_fused_gemv_linear(a, stream);
        int st = check_workspace(workspace, workspace_bytes, parts_bytes(n, rows, K), Wq, Wscale,
                                 row_groups(rows) * k_tiles(K), X, ldx, n, K, e, gated ? rows : e.N);
        if (st != NVFP4_OK)
            return st;
        a.partials = static_cast<float *>(workspace);
        st = nvfp4_launch_fused_gemv_partial(a, stream);
        return st != NVFP4_OK ? st : launch_reduce(e, a.partials, n, a.rows, ks, gated, stream);
    }
    nvfp4_fused_gemm_args a = {};
    a.mode = gated ? 1 : 0;
    a.codes = Wq;
    a.scales = Wscale;
    a.X = X;
    a.ldx = ldx;
    a.n = n;
    a.K = K;
    a.row_groups = (int)row_groups(rows);
    a.epi = e;
    return launch_product(a, workspace, workspace_bytes, stream);
}

// Rows of the packed weight of a gated block of F outputs.
long long gated_rows(long long F)
{
    return 2 * kRowsPerGroup * row_groups(F);
}

// Token rows a block of the gradient kernel sums: from the shape alone, so that
// the order of the sums is.  About 2048 blocks where n allows.
int grad_rows_per_block(int n, int cols)
{
    const long long bx = (cols + kGradCols - 1) / kGradCols;
    const long long by = (2048 + bx - 1) / bx;
    return (int)(((n + by - 1) / by + 7) / 8 * 8);
}

int grad_blocks(int n, int cols)
{
    const int rows = n > 0 ? grad_rows_per_block(n, cols) : 8;
    return n > 0 ? (n + rows - 1) / rows : 1;
}

size_t grad_bytes(int n, int cols, int halves)
{
    const int by = grad_blocks(n, cols);
    return by > 1 ? (size_t)by * halves * cols * sizeof(float) : 0;
}

int launch_grad(GradParams p, bool gated, hipStream_t stream)
{
    const int halves = gated ? 2 : 1;
    const bool sums = p.db[0] || p.db[1];
    if (!sums && (!p.dz || p.n == 0))
        return NVFP4_OK;
    const int by = grad_blocks(p.n, p.cols);
    p.rows_per_block = p.n > 0 ? grad_rows_per_block(p.n, p.cols) : 8;
    const dim3 grid((unsigned)((p.cols + kGradCols - 1) / kGradCols), (unsigned)by);
    if (gated)
        hipLaunchKernelGGL(nvfp4_grad_kernel<true>, grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL(nvfp4_grad_kernel<false>, grid, dim3(256), 0, stream, p);
    if (hipGetLastError() != hipSuccess)
        return NVFP4_ERR_LAUNCH;
    if (sums && by > 1) {
        hipLaunchKernelGGL(nvfp4_grad_sum_kernel, dim3((unsigned)((p.N + 255) / 256), (unsigned)halves), dim3(256), 0,
                           stream, p, by, halves);
        if (hipGetLastError() != hipSuccess)
            return NVFP4_ERR_LAUNCH;
    }
    return NVFP4_OK;
}

// A backward call: dZ (unless dY serves as it is), the bias gradients, dX.
struct Backward {
    const uint8_t *codes_t, *scales_t;   // needed with dX
    float gscale;
    const void *dy;
    const float *preact;
    uint16_t *dx;
    void *db[2];
    int64_t ldy, ldp, ldx;
    int dy_dtype, db_dtype, act, n, N, K;
    float gate_gscale, up_gscale;
    bool gated;

    int rows() const { return gated ? (int)gated_rows(N) : (N + 7) / 8 * 8; }   // columns of dZ
};

size_t round256(size_t bytes)
{
    return (bytes + 255) / 256 * 256;
}

// Parts of the workspace, each on a multiple of 256 bytes.
struct BackwardSpace {
    size_t dz, sums, parts;
    size_t total() const { return dz + sums + parts; }
};

BackwardSpace backward_space(int n, int N, int K, bool gated, bool dx, bool db, bool copy)
{
    const int rows = gated ? (int)gated_rows(N) : (N + 7) / 8 * 8;
    BackwardSpace w = {};
    if (n < 1)
        return w;
    if (dx && copy)
        w.dz = round256((size_t)n * rows * 2);
    if (db)
        w.sums = round256(grad_bytes(n, gated ? rows / 2 : rows, gated ? 2 : 1));
    if (dx) {
        const int ks = nvfp4_plan_fused_gemm(n, K / 16, rows).ks;
        w.parts = ks > 1 ? round256((size_t)ks * n * K * sizeof(float)) : 0;
    }
    return w;
}

// dY's rows can be loaded by the product as they are.
bool usable_rows(const void *p, int dtype, int64_t ld, int n, int N)
{
    return dtype == NVFP4_DTYPE_BF16 && N % 8 == 0 && is_aligned(p, 16) && (n < 2 || (ld % 8 == 0 && ld <= kMaxStride));
}

int backward(const Backward &b, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int n = b.n, N = b.N;
    const bool sums = b.db[0] || b.db[1];
    if (b.dx && (!b.codes_t || !b.scales_t))
        return NVFP4_ERR_NULL;
    if (n > 0 && (!b.dy || (!b.preact && (b.gated || b.act != NVFP4_ACT_NONE))))
        return NVFP4_ERR_NULL;
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || N < 1 || N > (1 << 29) || b.act < NVFP4_ACT_NONE ||
        b.act > NVFP4_ACT_GELU_TANH || !valid_dtype(b.dy_dtype) || (sums && !valid_dtype(b.db_dtype)) ||
        (b.dx && b.K < 1))
        return NVFP4_ERR_RANGE;
    if (b.dx && (b.K % 16 != 0 || b.K > kMaxK))
        return NVFP4_ERR_SHAPE;
    const int64_t pre_cols = b.gated ? b.rows() : N;
    if (b.ldy < N || (b.preact && b.ldp < pre_cols) || (b.dx && b.ldx < b.K))
        return NVFP4_ERR_RANGE;
    if (b.ldy > INT32_MAX || b.ldp > INT32_MAX || b.ldx > INT32_MAX || (b.dx && b.rows() > kMaxStride))
        return NVFP4_ERR_SHAPE;
    const int ds = dtype_size(b.dy_dtype), bs = dtype_size(b.db_dtype);
    if (!is_aligned(b.dy, ds) || (b.preact && (!is_aligned(b.preact, 16) || b.ldp % 8 != 0)) || !is_aligned(b.dx, 2) ||
        !is_aligned(b.codes_t, 16) || !is_aligned(b.scales_t, 16) || !is_aligned(b.db[0], bs) || !is_aligned(b.db[1], bs))
        return NVFP4_ERR_ALIGN;
    const bool copy = b.gated || b.act != NVFP4_ACT_NONE || !usable_rows(b.dy, b.dy_dtype, b.ldy, n, N);
    const BackwardSpace w = backward_space(n, N, b.K, b.gated, b.dx != nullptr, sums, copy);
    if (w.total() && (!workspace || workspace_bytes < w.total()))
        return NVFP4_ERR_WORKSPACE;
    if (w.total() && !is_aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const size_t bn = (size_t)N * bs;
    const Region in[] = {matrix(b.dy, n, b.ldy, N, ds), matrix(b.preact, n, b.ldp, pre_cols, 4),
                         array(b.codes_t, b.dx ? nvfp4_transposed_codes_bytes(b.rows(), b.K) : 0),
                         array(b.scales_t, b.dx ? nvfp4_transposed_scales_bytes(b.rows(), b.K) : 0)};
    const Region out[] = {matrix(b.dx, n, b.ldx, b.K, 2), array(b.db[0], bn), array(b.db[1], bn),
                          array(workspace, w.total())};
    for (int i = 0; i < 4; ++i) {
        if (any_overlap(out[i], in))
            return NVFP4_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return NVFP4_ERR_OVERLAP;
    }
    int cus = 0;
    int status = nvfp4_device_cus(&cus);
    if (status != NVFP4_OK)
        return status;
    char *ws = static_cast<char *>(workspace);
    GradParams p = {};
    p.dy = b.dy;
    p.z = b.act == NVFP4_ACT_NONE && !b.gated ? nullptr : b.preact;
    p.dz = w.dz ? reinterpret_cast<uint16_t *>(ws) : nullptr;
    p.partial = reinterpret_cast<float *>(ws + w.dz);
    p.db[0] = b.db[0];
    p.db[1] = b.db[1];
    p.ldy = b.ldy;
    p.ldz = b.ldp;
    p.lddz = b.rows();
    p.n = n;
    p.N = N;
    p.cols = b.gated ? b.rows() / 2 : b.rows();
    p.act = b.act;
    p.dy_f32 = b.dy_dtype == NVFP4_DTYPE_F32;
    p.db_f32 = b.db_dtype == NVFP4_DTYPE_F32;
    p.vec = b.ldy % 4 == 0 && is_aligned(b.dy, 4 * ds);
    p.gscale[0] = b.gate_gscale;
    p.gscale[1] = b.up_gscale;
    status = launch_grad(p, b.gated, stream);
    if (status != NVFP4_OK || !b.dx || n == 0)
        return status;
    nvfp4_epilogue ep = {};
    ep.out_dtype = ep.bias_dtype = ep.residual_dtype = NVFP4_DTYPE_BF16;
    nvfp4_fused_gemm_args a = {};
    a.mode = 2;
    a.codes = b.codes_t;
    a.scales = b.scales_t;
    a.X = w.dz ? p.dz : static_cast<const uint16_t *>(b.dy);
    a.ldx = w.dz ? p.lddz : b.ldy;
    a.n = n;
    a.K = b.rows();
    a.row_groups = b.K / 16;
    a.epi = epi_params(&ep, b.gscale, 0.f, b.dx, b.ldx, b.K, b.K);
    return launch_product(a, w.parts ? ws + w.dz + w.sums : nullptr, w.parts, stream);
}

unsigned blocks_of(long long items)
{
    return (unsigned)((items + 255) / 256);
}

}  // namespace

extern "C" {

// ---- weights ----

size_t nvfp4_gated_rows(int F)
{
    return F > 0 && F <= (1 << 30) ? (size_t)gated_rows(F) : 0;
}

int nvfp4_pack_gated(const uint8_t *gate_codes, const uint8_t *gate_scales, const uint8_t *up_codes,
                     const uint8_t *up_scales, int F, int K, uint8_t *codes, uint8_t *scales, void *stream)
{
    if (!gate_codes || !gate_scales || !up_codes || !up_scales || !codes || !scales)
        return NVFP4_ERR_NULL;
    if (F < 1 || F > (1 << 30) || K < 1)
        return NVFP4_ERR_RANGE;
    if (K % 16 != 0 || K > kMaxK)
        return NVFP4_ERR_SHAPE;
    for (const uint8_t *q : {gate_codes, gate_scales, up_codes, up_scales, (const uint8_t *)codes, (const uint8_t *)scales})
        if (!is_aligned(q, 16))
            return NVFP4_ERR_ALIGN;
    const size_t cb = nvfp4_packed_codes_bytes(F, K), sb = nvfp4_packed_scales_bytes(F, K);
    if (overlap(codes, 2 * cb, gate_codes, cb) || overlap(codes, 2 * cb, up_codes, cb) ||
        overlap(scales, 2 * sb, gate_scales, sb) || overlap(scales, 2 * sb, up_scales, sb) ||
        overlap(codes, 2 * cb, scales, 2 * sb) || overlap(codes, 2 * cb, gate_scales, sb) ||
        overlap(codes, 2 * cb, up_scales, sb) || overlap(scales, 2 * sb, gate_codes, cb) ||
        overlap(scales, 2 * sb, up_codes, cb))
        return NVFP4_ERR_OVERLAP;
    const long long T = k_tiles(K), RG = row_groups(F);
    const long long cw = 2 * RG * T * 64, sw = 2 * RG * T * 8;
    if ((cw + 255) / 256 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    hipLaunchKernelGGL(nvfp4_interleave_kernel, dim3(blocks_of(cw)), dim3(256), 0, s, (const u32x4 *)gate_codes,
                       (const u32x4 *)up_codes, T * 64, cw, (u32x4 *)codes);
    hipLaunchKernelGGL(nvfp4_interleave_kernel, dim3(blocks_of(sw)), dim3(256), 0, s, (const u32x4 *)gate_scales,
                       (const u32x4 *)up_scales, T * 8, sw, (u32x4 *)scales);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

size_t nvfp4_transposed_codes_bytes(int N, int K)
{
    return N > 0 && K > 0 && K % 16 == 0 ? (size_t)(K / 16) * k_tiles(N) * 1024 : 0;
}

size_t nvfp4_transposed_scales_bytes(int N, int K)
{
    return N > 0 && K > 0 && K % 16 == 0 ? (size_t)(K / 16) * k_tiles(N) * 128 : 0;
}

int nvfp4_pack_transposed(const uint8_t *codes_packed, const uint8_t *scales_packed, int N, int K, uint8_t *codes_t,
                          uint8_t *scales_t, void *stream)
{
    if (!codes_packed || !scales_packed || !codes_t || !scales_t)
        return NVFP4_ERR_NULL;
    if (N < 1 || N > (1 << 30) || K < 1)
        return NVFP4_ERR_RANGE;
    if (K % 16 != 0 || K > kMaxK)
        return NVFP4_ERR_SHAPE;
    for (const uint8_t *q : {codes_packed, scales_packed, (const uint8_t *)codes_t, (const uint8_t *)scales_t})
        if (!is_aligned(q, 16))
            return NVFP4_ERR_ALIGN;
    const size_t cb = nvfp4_packed_codes_bytes(N, K), sb = nvfp4_packed_scales_bytes(N, K);
    const size_t ct = nvfp4_transposed_codes_bytes(N, K), stb = nvfp4_transposed_scales_bytes(N, K);
    if (overlap(codes_t, ct, codes_packed, cb) || overlap(codes_t, ct, scales_packed, sb) ||
        overlap(scales_t, stb, codes_packed, cb) || overlap(scales_t, stb, scales_packed, sb) ||
        overlap(codes_t, ct, scales_t, stb))
        return NVFP4_ERR_OVERLAP;
    const int T = (int)k_tiles(K), RG = (int)row_groups(N), TT = (int)k_tiles(N);
    const long long chunks = (long long)(K / 16) * TT * 64, words = (long long)(K / 16) * TT * 32;
    if ((chunks + 255) / 256 > INT32_MAX)
        return NVFP4_ERR_SHAPE;
    int cus = 0;
    const int st = nvfp4_device_cus(&cus);
    if (st != NVFP4_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    hipLaunchKernelGGL(nvfp4_transpose_codes_kernel, dim3(blocks_of(chunks)), dim3(256), 0, s, codes_packed, T, RG, TT,
                       chunks, (u32x4 *)codes_t);
    hipLaunchKernelGGL(nvfp4_transpose_scales_kernel, dim3(blocks_of(words)), dim3(256), 0, s, scales_packed, T, RG, TT,
                       words, (u32 *)scales_t);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// ---- forward ----

int nvfp4_fused_geometry(int n, int rows, int K, int *rows_per_workgroup, int *tokens_per_workgroup, int *k_groups,
                         int *k_parts)
{
    if (!rows_per_workgroup || !tokens_per_workgroup || !k_groups || !k_parts)
        return NVFP4_ERR_NULL;
    if (n <= NVFP4_MAX_TOKENS || n > NVFP4_MAX_GEMM_TOKENS || rows < 1 || rows > (1 << 30) || K < 1 || K > (1 << 30))
        return NVFP4_ERR_RANGE;
    if (K % 8 != 0)
        return NVFP4_ERR_SHAPE;
    const nvfp4_fused_gemm_plan plan = nvfp4_plan_fused_gemm(n, (int)row_groups(rows), K);
    nvfp4_fused_gemm_tile(plan.tile, rows_per_workgroup, tokens_per_workgroup, k_groups);
    *k_parts = plan.ks;
    return NVFP4_OK;
}

size_t nvfp4_linear_workspace_bytes(int n, int N, int K)
{
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || N < 1 || N > kMaxRows || K < 1 || K % 16 != 0 || K > kMaxK)
        return 0;
    return parts_bytes(n, N, K);
}

int nvfp4_linear(const uint8_t *Wq, const uint8_t *Wscale, float gscale, const uint16_t *X, int64_t ldx, void *Y,
                 int64_t ldy, int n, int N, int K, const nvfp4_epilogue *epilogue, void *workspace,
                 size_t workspace_bytes, void *stream)
{
    const int st = validate_forward(Wq, Wscale, X, ldx, Y, ldy, n, N, N, K, epilogue, false);
    if (st != NVFP4_OK || n == 0)
        return st;
    return forward(Wq, Wscale, X, ldx, n, N, K, epi_params(epilogue, gscale, 0.f, Y, ldy, N, N), false, workspace,
                   workspace_bytes, (hipStream_t)stream);
}

size_t nvfp4_gated_workspace_bytes(int n, int F, int K)
{
    if (n < 0 || n > NVFP4_MAX_GEMM_TOKENS || F < 1 || F > (1 << 29) || K < 1 || K % 16 != 0 || K > kMaxK)
        return 0;
    return parts_bytes(n, (int)gated_rows(F), K);
}

int nvfp4_gated(const uint8_t *Wq, const uint8_t *Wscale, float gate_gscale, float up_gscale, const uint16_t *X,
                int64_t ldx, void *H, int64_t ldh, int n, int F, int K, const nvfp4_epilogue *epilogue, void *workspace,
                size_t workspace_bytes, void *stream)
{
    if (F < 1 || F > (1 << 29))
        return NVFP4_ERR_RANGE;
    const int rows = (int)gated_rows(F);
    const int st = validate_forward(Wq, Wscale, X, ldx, H, ldh, n, F, rows, K, epilogue, true);
    if (st != NVFP4_OK || n == 0)
        return st;
    return forward(Wq, Wscale, X, ldx, n, rows, K, epi_params(epilogue, gate_gscale, up_gscale, H, ldh, F, rows), true,
                   workspace, workspace_bytes, (hipStream_t)stream);
}

// ---- backward ----

size_t nvfp4_linear_backward_workspace_bytes(int n, int N, int K, int dx, int dbias, int copy)
{
    if (n < 1 || n > NVFP4_MAX_GEMM_TOKENS || N < 1 || N > (1 << 29) || (dx && (K < 1 || K % 16 != 0 || K > kMaxK)))
        return 0;
    return backward_space(n, N, K, false, dx != 0, dbias != 0, copy != 0).total();
}

int nvfp4_linear_backward(const uint8_t *codes_t, const uint8_t *scales_t, float gscale, const void *dY, int dy_dtype,
                          int64_t ldy, const float *preact, int64_t ldp, int activation, uint16_t *dX, int64_t ldx,
                          void *dbias, int bias_dtype, int n, int N, int K, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    Backward b = {};
    b.codes_t = codes_t;
    b.scales_t = scales_t;
    b.gscale = gscale;
    b.dy = dY;
    b.dy_dtype = dy_dtype;
    b.ldy = ldy;
    b.preact = preact;
    b.ldp = ldp;
    b.act = activation;
    b.dx = dX;
    b.ldx = ldx;
    b.db[0] = dbias;
    b.db_dtype = bias_dtype;
    b.n = n;
    b.N = N;
    b.K = K;
    return backward(b, workspace, workspace_bytes, (hipStream_t)stream);
}

size_t nvfp4_gated_backward_workspace_bytes(int n, int F, int K, int dx, int dbias)
{
    if (n < 1 || n > NVFP4_MAX_GEMM_TOKENS || F < 1 || F > (1 << 29) || (dx && (K < 1 || K % 16 != 0 || K > kMaxK)))
        return 0;
    return backward_space(n, F, K, true, dx != 0, dbias != 0, true).total();
}

int nvfp4_gated_backward(const uint8_t *codes_t, const uint8_t *scales_t, float gate_gscale, float up_gscale,
                         const void *dH, int dh_dtype, int64_t ldh, const float *preact, int64_t ldp, int activation,
                         uint16_t *dX, int64_t ldx, void *dgate_bias, void *dup_bias, int bias_dtype, int n, int F,
                         int K, void *workspace, size_t workspace_bytes, void *stream)
{
    Backward b = {};
    b.codes_t = codes_t;
    b.scales_t = scales_t;
    b.gscale = 1.0f;   // the gradient rows carry the two tensor scales
    b.gate_gscale = gate_gscale;
    b.up_gscale = up_gscale;
    b.dy = dH;
    b.dy_dtype = dh_dtype;
    b.ldy = ldh;
    b.preact = preact;
    b.ldp = ldp;
    b.act = activation;
    b.dx = dX;
    b.ldx = ldx;
    b.db[0] = dgate_bias;
    b.db[1] = dup_bias;
    b.db_dtype = bias_dtype;
    b.n = n;
    b.N = F;
    b.K = K;
    b.gated = true;
    return backward(b, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
