// What the operators on 4-bit weights share: 16-bit element types, unpacking of
// code words, activations, and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cq.h"

namespace cq {

constexpr int kGroup = 128;       // inputs per scale
constexpr int kWordsPerGroup = 16;

// Masks a code in each half of a register.  Kernels get it as an argument: with both the mask and the
// magic number known, (x & mask) | magic becomes two instructions with an immediate each; from
// a register it is one (one row of the 37,888 x 8,192 layer: 45 us with two).
constexpr uint32_t kLow = 0x000F000Fu;

// One 16-bit element type: packed integers, conversions, packed arithmetic.
// magic | u, u < 16, is the value 2^p + u of the type (p its mantissa bits), so
// subtracting 2^p + z + 1 leaves u - (z + 1) exactly.
struct BF16 {
    using pair = __nv_bfloat162;
    static constexpr uint32_t kMagic = 0x43004300u;  // 128
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        const pair d = __hsub2(reinterpret_cast<const pair &>(a), reinterpret_cast<const pair &>(b));
        return reinterpret_cast<const uint32_t &>(d);
    }
    // u - z - 1 of codes q and q + 4 of a word; zero as zero_pair gives it, low is kLow.
    static __device__ __forceinline__ uint32_t code_pair(uint32_t word, int q, uint32_t zero, uint32_t low)
    {
        return sub(((word >> (4 * q)) & low) | kMagic, zero);
    }
    static __device__ __forceinline__ float to_float(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
    static __device__ __forceinline__ uint16_t from_float(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
    static __device__ __forceinline__ uint32_t from_floats(float lo, float hi)
    {
        const pair p = __floats2bfloat162_rn(lo, hi);
        return reinterpret_cast<const uint32_t &>(p);
    }
};

struct FP16 {
    using pair = __half2;
    static constexpr uint32_t kMagic = 0x64006400u;  // 1024
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        const pair d = __hsub2(reinterpret_cast<const pair &>(a), reinterpret_cast<const pair &>(b));
        return reinterpret_cast<const uint32_t &>(d);
    }
    // u - z - 1 of codes q and q + 4 of a word; zero as zero_pair gives it, low is kLow.  Ten mantissa bits hold an
    // odd code where it stands, as 1024 + 16 u; a sixteenth of that less 64 + z + 1 is exact, and a shift is saved.
    static __device__ __forceinline__ uint32_t code_pair(uint32_t word, int q, uint32_t zero, uint32_t low)
    {
        const uint32_t w = word >> (8 * (q / 2));
        if (q % 2 == 0)
            return sub((w & low) | kMagic, zero);
        const uint32_t v = (w & (low << 4)) | kMagic;
        const pair offset = __hsub2(__float2half2_rn(960.0f), reinterpret_cast<const pair &>(zero));
        const pair d = __hfma2(reinterpret_cast<const pair &>(v), __float2half2_rn(0.0625f), offset);
        return reinterpret_cast<const uint32_t &>(d);
    }
    static __device__ __forceinline__ float to_float(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    static __device__ __forceinline__ uint16_t from_float(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ uint32_t from_floats(float lo, float hi)
    {
        const pair p = __floats2half2_rn(lo, hi);
        return reinterpret_cast<const uint32_t &>(p);
    }
};

// magic + z + 1 in both halves: what sub() takes from magic | u.
template <class T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t nibble)
{
    return T::kMagic + (nibble + 1u) * 0x00010001u;
}

__device__ __forceinline__ float half_bits(uint16_t b)
{
    return __half2float(__ushort_as_half(b));
}

// act(z) for a result that is rounded to 16 bits: exp and the quotient to a few units of
// 2^-22, far inside that rounding.  The quotients' limits hold: exp(-z) = inf gives 0.
template <int n>
__device__ __forceinline__ void activate(float (&z)[n], int act)
{
    if (act == CQ_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = z[i] < 0.0f ? 0.0f : z[i];
    } else if (act == CQ_ACT_GELU) {  // erfc keeps the small values of large negative z
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = 0.5f * z[i] * erfcf(z[i] * -0.7071067811865476f);
    } else if (act == CQ_ACT_GELU_TANH) {  // z/2 (1 + tanh u) = z / (1 + exp(-2u))
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = __fdividef(z[i], 1.0f + __expf(-1.5957691216057308f * (z[i] + 0.044715f * z[i] * z[i] * z[i])));
    } else if (act == CQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = __fdividef(z[i], 1.0f + __expf(-z[i]));
    }
}

__device__ __forceinline__ float activation_slope(float z, int act)
{
    constexpr float kC = 0.7978845608028654f;
    switch (act) {
    case CQ_ACT_RELU:
        return z > 0.0f ? 1.0f : 0.0f;
    case CQ_ACT_GELU:
        return 0.5f * erfcf(z * -0.7071067811865476f) + z * (0.3989422804014327f * expf(-0.5f * z * z));
    case CQ_ACT_GELU_TANH: {
        const float t = tanhf(kC * (z + 0.044715f * z * z * z));
        return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * (kC * (1.0f + 0.134145f * z * z));
    }
    case CQ_ACT_SILU: {
        const float p = 1.0f / (1.0f + expf(-z));
        return p * (1.0f + z * (1.0f - p));
    }
    default:
        return 1.0f;
    }
}

inline bool is_aligned(const void *p, size_t a)
{
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// A [T][n] operand of 16-bit values: 16-byte rows.
inline bool good_rows(const void *p, int64_t ld, int64_t n)
{
    return p && is_aligned(p, 16) && ld >= n && ld % 8 == 0;
}

}  // namespace cq
