// What the fused operators do with a finished sum: scale, bias, activation,
// residual (linear) or the product of the activated gate with the up row
// (gated), in fp32, rounded once when stored.  The pre-activations that a
// backward pass will want are stored in fp32: rounded to bf16 they would be as
// large an error of the gradient as the rounding of dZ for its matrix product
// (gated 2 x 17408 x 5120, n = 1024: dX off by 2.9e-3 of its norm against
// 2.3e-3), for 4% of the training step's time.
#ifndef NVFP4_EPILOGUE_H
#define NVFP4_EPILOGUE_H

#include "../../include/nvfp4.h"
#include "device.h"
#include "internal.h"

namespace {

// exp(-z) is off by about |z| 2^-24 of its value (the product with log2(e) is
// rounded), and so is the left tail.
__device__ __forceinline__ float sigmoid_f(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));   // 0 and 1 at the ends; rcp is within 1 ulp
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// Phi(z), the normal distribution function, as 1 - erfc(x) / 2 for z = sqrt(2) x
// >= 0 and erfc(x) / 2 for -z.  erfc(x) = t exp(p(t) - x^2) with t = 1 / (1 +
// 0.4 x): p is a Chebyshev fit of degree 9, in t, of ln(erfc(x) exp(x^2) / t),
// relative error 9e-8 before rounding.  exp(-x^2) = 2^-(z^2 log2(e) / 2) takes
// the remainders of the square and of the product: a rounding of the exponent y
// would be a relative error of y 2^-24 (7e-6 of Phi(-8), 1.8e-5 of Phi(-13)).
// Phi(z) is within 8e-7 of its value for every z, and 0 below 2^-126.  The math
// library's erfc takes about four times the instructions: gelu added 22 us to
// the 158 of 16384 x 5120 at n = 1024, and adds 14 this way (9 without the
// remainders).
// *density receives exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float *density)
{
    constexpr float kC = 0.72134752044448170f;                              // log2(e) / 2
    constexpr float kCLow = (float)(0.72134752044448170 - (double)kC);
    const float a = fminf(fabsf(z), 16.0f);                                 // 0 by then
    const float q = a * a, y = q * kC;
    const float low = __builtin_fmaf(__builtin_fmaf(a, a, -q), kC, __builtin_fmaf(q, kCLow, __builtin_fmaf(q, kC, -y)));
    const float e = __builtin_amdgcn_exp2f(-y);
    const float d = __builtin_fmaf(-0.69314718f * low, e, e);               // 2^-low, low < 2^-16
    *density = d;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f * kSqrtHalf, a, 1.0f));
    float p = 0.0683646575f;
    p = __builtin_fmaf(p, t, -0.581891f);
    p = __builtin_fmaf(p, t, 1.81158173f);
    p = __builtin_fmaf(p, t, -2.67597985f);
    p = __builtin_fmaf(p, t, 1.99297822f);
    p = __builtin_fmaf(p, t, -0.977739036f);
    p = __builtin_fmaf(p, t, 0.484770298f);
    p = __builtin_fmaf(p, t, 0.360483378f);
    p = __builtin_fmaf(p, t, 1.0063802f);
    p = __builtin_fmaf(p, t, -1.48894858f);
    const float half = 0.5f * t * __expf(p) * d;
    return z < 0.0f ? half : 1.0f - half;
}

// act(z).  gelu is z Phi(z), whose left tail keeps its relative precision;
// gelu_tanh is 0.5 z (1 + tanh(u)) = z sigmoid(2u).
__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case NVFP4_ACT_RELU: return z < 0.0f ? 0.0f : z;   // NaN stays NaN
    case NVFP4_ACT_SILU: return z * sigmoid_f(z);
    case NVFP4_ACT_GELU: {
        float density;
        return z * normal_cdf(z, &density);
    }
    case NVFP4_ACT_GELU_TANH: return z * sigmoid_f(kTanhC * (z + kTanhA * z * z * z));
    default: return z;
    }
}

// act'(z)
__device__ __forceinline__ float activate_grad(float z, int act)
{
    switch (act) {
    case NVFP4_ACT_RELU: return z <= 0.0f ? 0.0f : 1.0f;
    case NVFP4_ACT_SILU: {
        const float s = sigmoid_f(z);
        return s * (1.0f + z * (1.0f - s));
    }
    case NVFP4_ACT_GELU: {
        float density;
        const float cdf = normal_cdf(z, &density);
        return cdf + z * kInvSqrt2Pi * density;
    }
    case NVFP4_ACT_GELU_TANH: {
        // s (1 - s) is 0 well before |z| = 16: beyond it the square would only
        // overflow, to 0 * inf
        const float s = sigmoid_f(kTanhC * (z + kTanhA * z * z * z)), c = fminf(fabsf(z), 16.0f);
        return s + z * s * (1.0f - s) * kTanhC * (1.0f + 3.0f * kTanhA * c * c);
    }
    default: return 1.0f;
    }
}

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b)
{
    return __builtin_bit_cast(float, (u32)b << 16);
}

// The two halves of an fp32 value, the lower one zero for bf16.
struct Halves {
    u32 lo, hi;
    __device__ __forceinline__ float value() const { return __builtin_bit_cast(float, hi << 16 | lo); }
};

// Element i of an fp32 or bf16 array.  Both types go through the same load of
// the upper 16 bits: a register that one of two branches loads looks, to the
// build's check of loads in flight, as if both might.
__device__ __forceinline__ Halves load_halves(const void *p, long long i, int f32)
{
    const uint16_t *h = static_cast<const uint16_t *>(p) + (f32 ? 2 * i : i);
    u32 lo = 0;
    if (f32)
        lo = h[0];
    return {lo, h[f32 ? 1 : 0]};
}

__device__ __forceinline__ float load_any(const void *p, long long i, int f32)
{
    return load_halves(p, i, f32).value();
}

__device__ __forceinline__ void store_any(void *p, long long i, int f32, float v)
{
    if (f32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = f32_to_bf16_bits(v);
}

// Position of output row r of the gate (up: 0 or 1) among the rows of a gated
// weight, whose 16-row groups alternate gate, up.
__device__ __forceinline__ long long gated_row(int r, int up)
{
    return (long long)(r >> 4) * 32 + up * 16 + (r & 15);
}

// One output of the linear epilogue: row r < N of token tok, `sum` unscaled.
__device__ __forceinline__ void linear_out(const nvfp4_epi_params e, int tok, int r, float sum, float bias,
                                           float residual)
{
    float z = e.gscale * sum;
    if (e.bias)
        z += bias;
    if (e.preact)
        e.preact[(long long)tok * e.ldp + r] = z;
    float y = activate(z, e.flags & kEpiAct);
    if (e.residual)
        y += residual;
    store_any(e.out, (long long)tok * e.ldo + r, e.flags & kEpiOutF32, y);
}

__device__ __forceinline__ void linear_out(const nvfp4_epi_params e, int tok, int r, float sum)
{
    linear_out(e, tok, r, sum, e.bias ? load_any(e.bias, r, e.flags & kEpiBiasF32) : 0.f,
               e.residual ? load_any(e.residual, (long long)tok * e.ldr + r, e.flags & kEpiResidualF32) : 0.f);
}

// One output of the gated epilogue.
__device__ __forceinline__ void gated_out(const nvfp4_epi_params e, int tok, int r, float gate, float up, float bias,
                                          float up_bias)
{
    float z = e.gscale * gate, u = e.up_gscale * up;
    if (e.bias)
        z += bias;
    if (e.up_bias)
        u += up_bias;
    if (e.preact) {
        e.preact[(long long)tok * e.ldp + gated_row(r, 0)] = z;
        e.preact[(long long)tok * e.ldp + gated_row(r, 1)] = u;
    }
    store_any(e.out, (long long)tok * e.ldo + r, e.flags & kEpiOutF32, activate(z, e.flags & kEpiAct) * u);
}

__device__ __forceinline__ void gated_out(const nvfp4_epi_params e, int tok, int r, float gate, float up)
{
    gated_out(e, tok, r, gate, up, e.bias ? load_any(e.bias, r, e.flags & kEpiBiasF32) : 0.f,
              e.up_bias ? load_any(e.up_bias, r, e.flags & kEpiBiasF32) : 0.f);
}

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 load_any4(const void *p, long long i, int f32)
{
    const u32x2 *w = reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(p) + (f32 ? 2 * i : i));
    u32x2 b = {0u, 0u};
    if (f32)
        b = w[1];
    const u32x2 a = w[0];
    const u32x4 v = f32 ? u32x4{a[0], a[1], b[0], b[1]}
                        : u32x4{a[0] << 16, a[0] & 0xFFFF0000u, a[1] << 16, a[1] & 0xFFFF0000u};
    return __builtin_bit_cast(f32x4, v);
}

__device__ __forceinline__ u16x4 to_bf16x4(const f32x4 v)
{
    return u16x4{f32_to_bf16_bits(v[0]), f32_to_bf16_bits(v[1]), f32_to_bf16_bits(v[2]), f32_to_bf16_bits(v[3])};
}

__device__ __forceinline__ void store_any4(void *p, long long i, int f32, const f32x4 v)
{
    if (f32)
        *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + i) = v;
    else
        *reinterpret_cast<u16x4 *>(static_cast<uint16_t *>(p) + i) = to_bf16x4(v);
}

// Four consecutive rows r .. r+3 of a token: as vectors where `vec` allows and
// all four exist, else one by one.
__device__ __forceinline__ void linear_out4(const nvfp4_epi_params e, int tok, int r, const f32x4 sum)
{
    if (!((e.flags & kEpiVec) && r + 3 < e.N)) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (r + v < e.N)
                linear_out(e, tok, r + v, sum[v]);
        return;
    }
    f32x4 z = e.gscale * sum;
    if (e.bias)
        z += load_any4(e.bias, r, e.flags & kEpiBiasF32);
    if (e.preact)
        *reinterpret_cast<f32x4 *>(e.preact + (long long)tok * e.ldp + r) = z;
    f32x4 y;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        y[v] = activate(z[v], e.flags & kEpiAct);
    if (e.residual)
        y += load_any4(e.residual, (long long)tok * e.ldr + r, e.flags & kEpiResidualF32);
    store_any4(e.out, (long long)tok * e.ldo + r, e.flags & kEpiOutF32, y);
}

__device__ __forceinline__ void gated_out4(const nvfp4_epi_params e, int tok, int r, const f32x4 gate, const f32x4 up)
{
    if (!((e.flags & kEpiVec) && r + 3 < e.N)) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (r + v < e.N)
                gated_out(e, tok, r + v, gate[v], up[v]);
        return;
    }
    f32x4 z = e.gscale * gate, u = e.up_gscale * up;
    if (e.bias)
        z += load_any4(e.bias, r, e.flags & kEpiBiasF32);
    if (e.up_bias)
        u += load_any4(e.up_bias, r, e.flags & kEpiBiasF32);
    if (e.preact) {
        *reinterpret_cast<f32x4 *>(e.preact + (long long)tok * e.ldp + gated_row(r, 0)) = z;
        *reinterpret_cast<f32x4 *>(e.preact + (long long)tok * e.ldp + gated_row(r, 1)) = u;
    }
    f32x4 y;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        y[v] = activate(z[v], e.flags & kEpiAct) * u[v];
    store_any4(e.out, (long long)tok * e.ldo + r, e.flags & kEpiOutF32, y);
}

}  // namespace

#endif  // NVFP4_EPILOGUE_H
