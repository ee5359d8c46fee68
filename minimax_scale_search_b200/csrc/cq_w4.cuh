// What the operators on 4-bit weights share: 16-bit element types, unpacking of
// code words, activations, and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <utility>

#include "cq.h"

namespace cq {

constexpr int kGroup = 128;       // inputs per scale
constexpr int kWordsPerGroup = 16;

// Masks a code in each half of a register.  Kernels get it as an argument: with both the mask and the
// magic number known, (x & mask) | magic becomes two instructions with an immediate each; from
// a register it is one (one row through 30,336 x 16,384: 68 us for 82).
constexpr uint32_t kLow = 0x000F000Fu;

// One 16-bit element type: packed integers, conversions, packed arithmetic.
// magic | u, u < 16, is the value 2^p + u of the type (p its mantissa bits), so
// subtracting 2^p + z + 1 leaves u - (z + 1) exactly.
struct BF16 {
    using pair = __nv_bfloat162;
    static constexpr uint32_t kMagic = 0x43004300u;  // 128
    // Codes that enter products as integers do so times 2^-11 (mantissas of 2^-4), so that 128 inputs of any size times
    // codes of up to 16 stay in fp32 where the scale brings the result back into it; the smallest input times 2^-11
    // is an fp32 value still.
    static constexpr uint32_t kCodeMagic = 0x3D803D80u;
    static constexpr float kCodeUnit = 2048.0f;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        const pair d = __hsub2(reinterpret_cast<const pair &>(a), reinterpret_cast<const pair &>(b));
        return reinterpret_cast<const uint32_t &>(d);
    }
    // (u - z - 1) / kCodeUnit of codes q and q + 4 of a word; zero as code_zero_pair gives it, low is kLow.
    static __device__ __forceinline__ uint32_t code_pair(uint32_t word, int q, uint32_t zero, uint32_t low)
    {
        return sub(((word >> (4 * q)) & low) | kCodeMagic, zero);
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
    static constexpr uint32_t kCodeMagic = kMagic;   // 128 inputs below 2^16 times 16 are below 2^27
    static constexpr float kCodeUnit = 1.0f;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b)
    {
        const pair d = __hsub2(reinterpret_cast<const pair &>(a), reinterpret_cast<const pair &>(b));
        return reinterpret_cast<const uint32_t &>(d);
    }
    // u - z - 1 of codes q and q + 4 of a word; zero as code_zero_pair gives it, low is kLow.  Ten mantissa bits hold an
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

// The same for code_pair().
template <class T>
__device__ __forceinline__ uint32_t code_zero_pair(uint32_t nibble)
{
    return T::kCodeMagic + (nibble + 1u) * 0x00010001u;
}

__device__ __forceinline__ float half_bits(uint16_t b)
{
    return __half2float(__ushort_as_half(b));
}

// Phi(z), the normal distribution function, and phi(z), its density: the tail beyond |z| is phi M(|z|), M the ratio of
// Mills, here a polynomial of degree 8 in 1 / (1 + 0.3 |z|), fitted on [0, 14] and there within 2.1e-7 of it (4.8e-7 as evaluated in
// fp32), so that the small values of large negative z keep their digits.  17 instructions, where erfc has three times as many.
__device__ __forceinline__ float normal_distribution(float z, float &phi)
{
    const float t = __fdividef(1.0f, fmaf(0.3f, fabsf(z), 1.0f));
    float m = 0.08939834282074922f;
    m = fmaf(m, t, -0.3938665763259987f);
    m = fmaf(m, t, 0.5167975709357504f);
    m = fmaf(m, t, -0.13402152701818226f);
    m = fmaf(m, t, 0.3219068215590072f);
    m = fmaf(m, t, 0.2505677419384999f);
    m = fmaf(m, t, 0.30266395988252076f);
    m = fmaf(m, t, 0.2998676368875933f);
    phi = 0.3989422804014327f * __expf(-0.5f * z * z);
    const float tail = phi * (m * t);
    return z < 0.0f ? tail : 1.0f - tail;
}

// 1 / (1 + exp(-a)), its small values to their own last digits: only exp(-|a|) is taken, so that the divisor lies between
// 1 and 2 (the fast quotient gives 0 for divisors above 2^126, where bf16 still has normal results).
__device__ __forceinline__ float sigmoid(float a)
{
    const float e = __expf(-fabsf(a)), p = __fdividef(1.0f, 1.0f + e);
    return a < 0.0f ? e * p : p;
}

// act(z) for a result that is rounded to 16 bits.  exp(x) of the fast instruction is within (2 + 1.2 |x|) 2^-23 of
// its value and x within 5 roundings: 2^-14 in all where exp(x) is about to leave fp32, 2^-19 for |x| < 2.
template <int n>
__device__ __forceinline__ void activate(float (&z)[n], int act)
{
    if (act == CQ_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = z[i] < 0.0f ? 0.0f : z[i];
    } else if (act == CQ_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < n; i++) {
            float phi;
            z[i] *= normal_distribution(z[i], phi);
        }
    } else if (act == CQ_ACT_GELU_TANH) {  // z/2 (1 + tanh u) = z / (1 + exp(-2u))
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] *= sigmoid(1.5957691216057308f * (z[i] + 0.044715f * z[i] * z[i] * z[i]));
    } else if (act == CQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] *= sigmoid(z[i]);
    }
}

// act'(z), each of its terms as far off as that.
template <int n>
__device__ __forceinline__ void slopes(float (&z)[n], int act)
{
    constexpr float kC = 0.7978845608028654f;  // sqrt(2 / pi)
    if (act == CQ_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = z[i] > 0.0f ? 1.0f : 0.0f;
    } else if (act == CQ_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < n; i++) {
            float phi;
            const float p = normal_distribution(z[i], phi);
            z[i] = fmaf(z[i], phi, p);
        }
    } else if (act == CQ_ACT_GELU_TANH) {  // p = (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), 1 - tanh^2 u = 4 p (1 - p)
#pragma unroll
        for (int i = 0; i < n; i++) {
            const float q = fminf(z[i] * z[i], 1e6f);  // p is 0 or 1 long before; inf would meet its 1 - p = 0
            const float p = sigmoid(2.0f * kC * z[i] * (1.0f + 0.044715f * q));
            z[i] = p + z[i] * (2.0f * p * (1.0f - p)) * (kC * (1.0f + 0.134145f * q));
        }
    } else if (act == CQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < n; i++) {
            const float p = sigmoid(z[i]);
            z[i] = p * (1.0f + z[i] * (1.0f - p));
        }
    } else {
#pragma unroll
        for (int i = 0; i < n; i++)
            z[i] = 1.0f;
    }
}

inline bool is_aligned(const void *p, size_t a)
{
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

template <class D>
__device__ __forceinline__ void widen(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        v[2 * j] = D::to_float(static_cast<uint16_t>(w[j]));
        v[2 * j + 1] = D::to_float(static_cast<uint16_t>(w[j] >> 16));
    }
}

template <class D>
__device__ __forceinline__ uint4 narrow(const float (&v)[8])
{
    return make_uint4(D::from_floats(v[0], v[1]), D::from_floats(v[2], v[3]), D::from_floats(v[4], v[5]),
                      D::from_floats(v[6], v[7]));
}

// SMs of the current device, and whether a kernel has been set up on it: asked once per device.
constexpr int kMostDevices = 64;

inline int current_device()
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

inline int sm_count()
{
    static std::atomic<int> known[kMostDevices];
    const int dev = current_device();
    if (dev >= 0 && dev < kMostDevices && known[dev].load(std::memory_order_relaxed) > 0)
        return known[dev].load(std::memory_order_relaxed);
    int sms = 0;
    if (dev < 0 || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return 148;
    if (dev < kMostDevices)
        known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Lets `kernel` have `bytes` of dynamic shared memory on the current device.
template <auto kernel>
cudaError_t allow_shared(int bytes)
{
    static std::atomic<bool> done[kMostDevices];
    const int dev = current_device();
    const bool kept = dev >= 0 && dev < kMostDevices;
    if (kept && done[dev].load(std::memory_order_relaxed))
        return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && kept)
        done[dev].store(true, std::memory_order_relaxed);
    return e;
}

inline cq_status launched()
{
    return cudaGetLastError() == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

// Launches of one call that follow each other on a stream.  The first says early on that the next may begin; that
// one is launched by launch_next, may run beside the first's last CTAs, and calls wait_for_previous before it touches
// what the first wrote, or before its end where it touches none of it.  It never ends before the first has, so what
// comes after it on the stream comes after both; the first is an ordinary launch, so what came before is done.
// Saves the launch and what a wave's last CTAs leave idle: both gradients of 777 x 1,032 x 2,176 in 22.7 us for 24.7,
// of 4,096 x 14,336 x 4,096 in 769 for 778; a table's gradient of 16 tokens in 8.3 us for 12.
__device__ __forceinline__ void let_next_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void wait_for_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cq_status launch_next(void (*kernel)(P...), unsigned ctas, int threads, int bytes, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(ctas);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    config.attrs = attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, std::forward<A>(args)...) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

// A [T][n] operand of 16-bit values: 16-byte rows.
inline bool good_rows(const void *p, int64_t ld, int64_t n)
{
    return p && is_aligned(p, 16) && ld >= n && ld % 8 == 0;
}

}  // namespace cq
