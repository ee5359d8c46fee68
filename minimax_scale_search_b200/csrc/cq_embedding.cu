// Rows of a quantised table, and the gradient of its group scales.
//
// The table is the selection's own output for a [V][K] matrix: scales
// [V * K/128] and code words [V * K/128][16], so a row's words are contiguous.
#include "cq_w4.cuh"

namespace cq {
namespace {

constexpr int kThreads = 256;

struct Ids {
    const void *p;
    int wide;  // int64 ids
    int64_t V;
    // The row of token t, or -1 for an id outside [0, V).
    __device__ __forceinline__ int64_t row(int64_t t) const
    {
        const int64_t v = wide ? static_cast<const int64_t *>(p)[t] : static_cast<const int32_t *>(p)[t];
        return v >= 0 && v < V ? v : -1;
    }
};

// Eight values from a code word: q = u - 8.
__device__ __forceinline__ void unpack(uint32_t word, float (&q)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j++)
        q[j] = static_cast<float>(static_cast<int>((word >> (4 * j)) & 15u) - 8);
}

template <int DT>
__device__ __forceinline__ void store8(void *out, int64_t i, const float (&v)[8])
{
    if (DT == CQ_DTYPE_FP32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + i);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            h[j] = DT == CQ_DTYPE_BF16 ? BF16::from_floats(v[2 * j], v[2 * j + 1]) : FP16::from_floats(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + i) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

template <int DT>
__device__ __forceinline__ void load8(const void *in, int64_t i, float (&v)[8])
{
    if (DT == CQ_DTYPE_FP32) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(in) + i));
        const float4 b = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(in) + i) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(in) + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint16_t b = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
            v[j] = DT == CQ_DTYPE_BF16 ? BF16::to_float(b) : FP16::to_float(b);
        }
    }
}

// One thread per code word.
template <int DT>
__global__ void __launch_bounds__(kThreads) embedding_kernel(Ids ids, int64_t T, const uint16_t *scales,
                                                             const uint32_t *codes, int64_t K8, float multiplier, void *out)
{
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads, n = T * K8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
        const int64_t t = i / K8, k = i - t * K8, v = ids.row(t);
        float q[8] = {};
        if (v >= 0) {
            const float s = half_bits(scales[v * (K8 / kWordsPerGroup) + k / kWordsPerGroup]);
            unpack(codes[v * K8 + k], q);
#pragma unroll
            for (int j = 0; j < 8; j++)
                q[j] = multiplier * (s * q[j]);
        }
        store8<DT>(out, i * 8, q);
    }
}

// dots[t][g] = sum_{i in g} dout[t][i] q[id_t][i]: 16 lanes per group.
template <int DT>
__global__ void __launch_bounds__(kThreads) token_dots_kernel(const void *dout, Ids ids, int64_t T, const uint32_t *codes,
                                                              int64_t K8, float *dots)
{
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads, n = T * K8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {  // n % 16 == 0
        const int64_t t = i / K8, k = i - t * K8, v = ids.row(t);
        float s = 0.0f;
        if (v >= 0) {
            float d[8], q[8];
            load8<DT>(dout, i * 8, d);
            unpack(codes[v * K8 + k], q);
#pragma unroll
            for (int j = 0; j < 8; j++)
                s = fmaf(d[j], q[j], s);
        }
        const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
        for (int o = 8; o > 0; o >>= 1)
            s += __shfl_xor_sync(mask, s, o, 16);
        if ((threadIdx.x & 15) == 0)
            dots[i / kWordsPerGroup] = s;
    }
}

// order[rank] = t and key[rank] = id (V for no row), rank the number of tokens that
// come before t by (id, t).
__global__ void __launch_bounds__(kThreads) rank_kernel(Ids ids, int64_t T, int64_t *key, int32_t *order)
{
    __shared__ int64_t other[kThreads];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    int64_t mine = -1;
    if (t < T) {
        mine = ids.row(t);
        mine = mine < 0 ? ids.V : mine;
    }
    int64_t rank = 0;
    for (int64_t j0 = 0; j0 < T; j0 += kThreads) {
        __syncthreads();
        if (j0 + threadIdx.x < T) {
            const int64_t v = ids.row(j0 + threadIdx.x);
            other[threadIdx.x] = v < 0 ? ids.V : v;
        }
        __syncthreads();
        const int m = static_cast<int>(T - j0 < kThreads ? T - j0 : kThreads);
        for (int j = 0; j < m; j++)
            rank += other[j] < mine || (other[j] == mine && j0 + j < t);
    }
    if (t < T) {
        key[rank] = mine;
        order[rank] = static_cast<int32_t>(t);
    }
}

// One thread per (first token of a run of equal ids, group): sums the run in fp64.
__global__ void __launch_bounds__(kThreads) run_sums_kernel(const int64_t *key, const int32_t *order, int64_t T, int64_t V,
                                                            const float *dots, int64_t ng, float multiplier, float *dscales)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= T * ng)
        return;
    const int64_t j0 = i / ng, g = i - j0 * ng, v = key[j0];
    if (v >= V || (j0 > 0 && key[j0 - 1] == v))
        return;
    double s = 0.0;
    for (int64_t j = j0; j < T && key[j] == v; j++)
        s += dots[order[j] * ng + g];
    dscales[v * ng + g] = static_cast<float>(s * multiplier);
}

unsigned grid_for(int64_t n)
{
    const int64_t blocks = (n + kThreads - 1) / kThreads, cap = 148 * 64;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

cq_status check_table(int64_t T, int64_t V, int64_t K, int dtype, int ids64, const void *ids, const void *codes,
                      float multiplier)
{
    if (T < 0 || V < 0 || K <= 0 || K % kGroup != 0 || dtype < CQ_DTYPE_BF16 || dtype > CQ_DTYPE_FP32 ||
        (ids64 != 0 && ids64 != 1) || !(multiplier - multiplier == 0.0f))
        return CQ_ERR_INVALID_ARG;
    constexpr int64_t kMost = static_cast<int64_t>(1) << 31;
    if (T >= kMost || V >= kMost || K >= kMost)
        return CQ_ERR_UNSUPPORTED;
    if ((T > 0 && (!ids || !is_aligned(ids, ids64 ? 8 : 4))) || (T > 0 && V > 0 && (!codes || !is_aligned(codes, 4))))
        return CQ_ERR_INVALID_ARG;
    return CQ_OK;
}

size_t round256(size_t n)
{
    return (n + 255) / 256 * 256;
}

cq_status launched()
{
    return cudaGetLastError() == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // namespace
}  // namespace cq

using namespace cq;

extern "C" {

cq_status cq_w4_embedding(const void *ids, int ids64, int64_t T, const uint16_t *scales, const uint32_t *codes, int64_t V,
                          int64_t K, float multiplier, int dtype, void *out, void *stream)
{
    const cq_status st = check_table(T, V, K, dtype, ids64, ids, codes, multiplier);
    if (st != CQ_OK)
        return st;
    if (T == 0)
        return CQ_OK;
    if ((V > 0 && (!scales || !is_aligned(scales, 2))) || !out || !is_aligned(out, 16))
        return CQ_ERR_INVALID_ARG;
    const Ids in = {ids, ids64, V};
    auto kernel = dtype == CQ_DTYPE_BF16   ? embedding_kernel<CQ_DTYPE_BF16>
                  : dtype == CQ_DTYPE_FP16 ? embedding_kernel<CQ_DTYPE_FP16>
                                           : embedding_kernel<CQ_DTYPE_FP32>;
    kernel<<<grid_for(T * (K / 8)), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(in, T, scales, codes, K / 8,
                                                                                      multiplier, out);
    return launched();
}

size_t cq_w4_embedding_backward_workspace_bytes(int64_t T, int64_t K)
{
    if (T <= 0 || K <= 0)
        return 256;
    const size_t n = static_cast<size_t>(T);
    return round256(n * 8) + round256(n * 4) + round256(n * static_cast<size_t>(K / kGroup) * 4);
}

cq_status cq_w4_embedding_backward(const void *dout, int dtype, const void *ids, int ids64, int64_t T, const uint32_t *codes,
                                   int64_t V, int64_t K, float multiplier, float *dscales, void *workspace,
                                   size_t workspace_bytes, void *stream)
{
    const cq_status st = check_table(T, V, K, dtype, ids64, ids, codes, multiplier);
    if (st != CQ_OK)
        return st;
    if (V == 0)
        return CQ_OK;
    if (!dscales || !is_aligned(dscales, 4) || (T > 0 && (!dout || !is_aligned(dout, 16))))
        return CQ_ERR_INVALID_ARG;
    if (T > 0 && (!workspace || !is_aligned(workspace, 256) ||
                  workspace_bytes < cq_w4_embedding_backward_workspace_bytes(T, K)))
        return CQ_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t ng = K / kGroup;
    if (cudaMemsetAsync(dscales, 0, static_cast<size_t>(V) * ng * 4, s) != cudaSuccess)
        return CQ_ERR_CUDA;
    if (T == 0)
        return CQ_OK;
    char *p = static_cast<char *>(workspace);
    int64_t *key = reinterpret_cast<int64_t *>(p);
    int32_t *order = reinterpret_cast<int32_t *>(p + round256(static_cast<size_t>(T) * 8));
    float *dots = reinterpret_cast<float *>(p + round256(static_cast<size_t>(T) * 8) + round256(static_cast<size_t>(T) * 4));
    const Ids in = {ids, ids64, V};
    auto kernel = dtype == CQ_DTYPE_BF16   ? token_dots_kernel<CQ_DTYPE_BF16>
                  : dtype == CQ_DTYPE_FP16 ? token_dots_kernel<CQ_DTYPE_FP16>
                                           : token_dots_kernel<CQ_DTYPE_FP32>;
    kernel<<<grid_for(T * (K / 8)), kThreads, 0, s>>>(dout, in, T, codes, K / 8, dots);
    if (launched() != CQ_OK)
        return CQ_ERR_CUDA;
    rank_kernel<<<static_cast<unsigned>((T + kThreads - 1) / kThreads), kThreads, 0, s>>>(in, T, key, order);
    if (launched() != CQ_OK)
        return CQ_ERR_CUDA;
    run_sums_kernel<<<static_cast<unsigned>((T * ng + kThreads - 1) / kThreads), kThreads, 0, s>>>(key, order, T, V, dots, ng,
                                                                                             multiplier, dscales);
    return launched();
}

}  // extern "C"
