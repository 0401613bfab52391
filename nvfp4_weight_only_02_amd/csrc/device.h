// Device-side basics shared by the translation units of libnvfp4: the tile
// sizes of the packed layout, buffer resources and hand-counted buffer loads,
// and the exact NVFP4 dequantisation.
#ifndef NVFP4_DEVICE_H
#define NVFP4_DEVICE_H

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>
#include <utility>

namespace {

typedef unsigned int u32;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRowsPerGroup = 16;      // MFMA N dimension: weight rows per tile
constexpr int kTileK = 128;            // K columns per tile (8 NVFP4 blocks)
constexpr int kBlocksPerTile = kTileK / 16;
constexpr int kMaxTilesPerWave = 8;    // X slice of a wave: 16 VGPRs per tile
constexpr int kMaxTilesChunked = 7;    // per wave and K chunk when K needs several chunks
constexpr int kWaves = 8;            // waves per workgroup, one K-slice each
constexpr int kBufferWord3 = 0x00020000;   // gfx9 raw buffer resource: 32-bit data, no swizzle
constexpr unsigned kOutOfRange = 0x7FFFFFF0u;   // buffer offset past any resource: reads zeros
constexpr int kSlots = 8;                        // row-group partials parked in LDS
constexpr int kMaxK = 1 << 18;                   // keeps every buffer offset within 32 bits
constexpr int kMaxKParts = 64;                   // K parts of a split launch

// 16-row groups of N rows and 128-column tiles of K columns, rounded up in
// 64-bit arithmetic (no int near INT_MAX overflows).
constexpr long long row_groups(long long N)
{
    return (N + kRowsPerGroup - 1) / kRowsPerGroup;
}
constexpr long long k_tiles(long long K)
{
    return (K + kTileK - 1) / kTileK;
}

struct GemvParams {
    const u32x4 *codes;    // packed codes, [RG][T][64 lanes] x 16 B
    const u32x2 *scales;   // packed scales, [RG][T][16 rows] x 8 B
    const uint16_t *X;     // bf16 [n][K]
    uint16_t *Y;           // bf16 output, token stride ldy
    float gscale;
    int n, N, K, T, RG;
    int kc;                // K chunks (passes) of a K part: chunk c covers its tiles [c*8*MT, (c+1)*8*MT)
    int rg_base, rg_rem;   // row groups per workgroup: rg_base, +1 for the first rg_rem
    int start1, start2;    // first row of the 2nd and 3rd projection (N if absent)
    long long off0, off1, off2, ldy;
    // K split: workgroups [q*wpp, (q+1)*wpp) own the tiles [q*tp, min((q+1)*tp, T))
    // of K part q.  With P set they store fp32 partials P[q][t][r] (unscaled)
    // instead of Y; nvfp4_ksplit_reduce_kernel then sums the parts.
    int tp, wpp;
    float *P;

    __device__ __forceinline__ int x_stride() const { return K; }
    __device__ __forceinline__ unsigned x_bytes() const { return (unsigned)(n * K * 2); }
};

// Two E2M1 codes (byte `sel` of w) -> two bf16 values, unscaled (scale 1.0).
__device__ __forceinline__ u32 fp4x2_to_bf16x2(u32 w, int sel)
{
    bf16x2 v;
    switch (sel) {
    case 0: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0); break;
    case 1: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1); break;
    case 2: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2); break;
    default: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3); break;
    }
    return __builtin_bit_cast(u32, v);
}

// Calls f(std::integral_constant<int, j>) for j = 0 .. N-1.
template <typename F, int... J>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, J...>)
{
    (f(std::integral_constant<int, J>{}), ...);
}

template <int N, typename F>
__device__ __forceinline__ void static_for(F &&f)
{
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// A raw buffer resource over [base, base + bytes) (gfx9 layout: 48-bit base,
// stride 0, byte-granular range check).
__device__ __forceinline__ u32x4 buffer_rsrc(const void *base, unsigned bytes)
{
    const unsigned long long a = (unsigned long long)base;
    return u32x4{(u32)a, (u32)(a >> 32) & 0xFFFFu, bytes, (u32)kBufferWord3};
}

// Loads whose completion is tracked by hand (see the vmcnt bookkeeping in
// the kernel).  Offsets past the resource's range return zeros.
__device__ __forceinline__ u32x4 buffer_load_b128(u32x4 rsrc, unsigned off)
{
    u32x4 v;
    asm volatile("buffer_load_dwordx4 %0, %1, %2, 0 offen" : "=v"(v) : "v"(off), "s"(rsrc));
    return v;
}

__device__ __forceinline__ u32x4 buffer_load_b128_nt(u32x4 rsrc, unsigned off)
{
    u32x4 v;
    asm volatile("buffer_load_dwordx4 %0, %1, %2, 0 offen nt" : "=v"(v) : "v"(off), "s"(rsrc));
    return v;
}

// Wait until at most N vector-memory operations are outstanding; the
// registers passed are the ones the wait makes valid (tied in and out, so no
// read of them can be scheduled before it).
template <int N>
__device__ __forceinline__ void vm_wait4(u32x4 &a, u32x4 &b, u32x4 &c, u32x4 &d, std::integral_constant<int, N>)
{
    static_assert(N >= 0 && N <= 63, "vmcnt is a 6-bit field");
    asm volatile("s_waitcnt vmcnt(%4)" : "+v"(a), "+v"(b), "+v"(c), "+v"(d) : "n"(N));
}

__device__ __forceinline__ uint16_t f32_to_bf16_bits(float f)
{
    return __builtin_bit_cast(uint16_t, (__bf16)f);   // v_cvt_pk_bf16_f32: RNE
}

template <int N>
__device__ __forceinline__ void vm_wait1(u32x4 &a, std::integral_constant<int, N>)
{
    static_assert(N >= 0 && N <= 63, "vmcnt is a 6-bit field");
    asm volatile("s_waitcnt vmcnt(%1)" : "+v"(a) : "n"(N));
}

// A wave-uniform value the compiler cannot prove uniform, moved to SGPRs.
__device__ __forceinline__ u32x4 uniform(u32x4 v)
{
    return u32x4{(u32)__builtin_amdgcn_readfirstlane((int)v[0]), (u32)__builtin_amdgcn_readfirstlane((int)v[1]),
                 (u32)__builtin_amdgcn_readfirstlane((int)v[2]), (u32)__builtin_amdgcn_readfirstlane((int)v[3])};
}

__device__ __forceinline__ u32x2 buffer_load_b64_nt(u32x4 rsrc, unsigned off)
{
    u32x2 v;
    asm volatile("buffer_load_dwordx2 %0, %1, %2, 0 offen nt" : "=v"(v) : "v"(off), "s"(rsrc));
    return v;
}

// Exact bf16 of the 8 weights of one lane for blocks 2j and 2j+1: codes in
// dword `w` (bytes 0, 1: block 2j; bytes 2, 3: block 2j+1; low nibble first),
// E4M3 scales of the two blocks in bytes 2H, 2H+1 of `sw`.
template <bool H>
__device__ __forceinline__ u32x4 dequant_pair(u32 w, u32 sw)
{
    const auto s2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)sw, H);
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const bf16x2 o0 = {(__bf16)(a[0] * s2[0]), (__bf16)(a[1] * s2[0])};
    const bf16x2 o1 = {(__bf16)(b[0] * s2[0]), (__bf16)(b[1] * s2[0])};
    const bf16x2 o2 = {(__bf16)(c[0] * s2[1]), (__bf16)(c[1] * s2[1])};
    const bf16x2 o3 = {(__bf16)(d[0] * s2[1]), (__bf16)(d[1] * s2[1])};
    return u32x4{__builtin_bit_cast(u32, o0), __builtin_bit_cast(u32, o1), __builtin_bit_cast(u32, o2),
                 __builtin_bit_cast(u32, o3)};
}

}  // namespace

#endif  // NVFP4_DEVICE_H
