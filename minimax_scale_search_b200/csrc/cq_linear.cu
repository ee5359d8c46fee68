// Linear layers on 4-bit weights, and their gradients (the plain versions).
#include <cooperative_groups.h>

#include "cq_w4.cuh"

namespace cg = cooperative_groups;

namespace cq {
namespace {

struct Layer {
    const uint32_t *qweight;   // [K/8][R]
    const uint32_t *qzeros;    // [K/128][R/8]
    const uint16_t *scales;    // [K/128][R]
    int64_t R, K;
};

__device__ __forceinline__ int code_of(const Layer &w, int64_t r, int64_t k)
{
    const int u = (w.qweight[(k >> 3) * w.R + r] >> (4 * (k & 7))) & 15;
    const int z = (w.qzeros[(k >> 7) * (w.R >> 3) + (r >> 3)] >> (4 * (r & 7))) & 15;
    return u - (z + 1);
}

constexpr int kTile = 32;

// y tile of 32 rows of T x 32 outputs, one thread per element.
template <class D>
__global__ void __launch_bounds__(1024) linear_plain(const uint16_t *x, int64_t ldx, int64_t T, Layer w,
                                                     const uint16_t *bias, int act, const uint16_t *res, int64_t ldres,
                                                     uint16_t *y, int64_t ldy, uint16_t *pre, int64_t ldpre)
{
    __shared__ float xs[kTile][kTile + 1], ws[kTile][kTile + 1];
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kTile + tx, t = static_cast<int64_t>(blockIdx.y) * kTile + ty;
    float acc = 0.0f;
    for (int64_t k0 = 0; k0 < w.K; k0 += kTile) {
        xs[ty][tx] = t < T ? D::to_float(x[t * ldx + k0 + tx]) : 0.0f;
        const int64_t k = k0 + ty;
        ws[ty][tx] = r < w.R ? half_bits(w.scales[(k >> 7) * w.R + r]) * code_of(w, r, k) : 0.0f;
        __syncthreads();
        for (int i = 0; i < kTile; i++)
            acc = fmaf(xs[ty][i], ws[i][tx], acc);
        __syncthreads();
    }
    if (t >= T || r >= w.R)
        return;
    const float z = acc + (bias ? D::to_float(bias[r]) : 0.0f);
    if (pre)
        pre[t * ldpre + r] = D::from_float(z);
    float v = activate(z, act);
    if (res)
        v += D::to_float(res[t * ldres + r]);
    y[t * ldy + r] = D::from_float(v);
}

template <class D>
__global__ void __launch_bounds__(1024) input_gradient_plain(const uint16_t *dz, int64_t lddz, int64_t T, Layer w,
                                                             uint16_t *dx, int64_t lddx)
{
    __shared__ float ds[kTile][kTile + 1], ws[kTile][kTile + 1];
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * kTile + tx, t = static_cast<int64_t>(blockIdx.y) * kTile + ty;
    float acc = 0.0f;
    for (int64_t r0 = 0; r0 < w.R; r0 += kTile) {
        ds[ty][tx] = t < T && r0 + tx < w.R ? D::to_float(dz[t * lddz + r0 + tx]) : 0.0f;
        const int64_t r = r0 + ty;
        ws[ty][tx] = r < w.R ? half_bits(w.scales[(k >> 7) * w.R + r]) * code_of(w, r, k) : 0.0f;
        __syncthreads();
        for (int i = 0; i < kTile; i++)
            acc = fmaf(ds[ty][i], ws[i][tx], acc);
        __syncthreads();
    }
    if (t < T)
        dx[t * lddx + k] = D::from_float(acc);
}

// One CTA per group and 8 outputs: thread (i, j) sums dz[t][r_j] x[t][i] over t.
template <class D>
__global__ void __launch_bounds__(1024) scale_gradient_plain(const uint16_t *dz, int64_t lddz, const uint16_t *x,
                                                             int64_t ldx, int64_t T, Layer w, float *dscales)
{
    __shared__ float part[8][kGroup];
    const int i = threadIdx.x, j = threadIdx.y;
    const int64_t g = blockIdx.y, r = static_cast<int64_t>(blockIdx.x) * 8 + j, k = g * kGroup + i;
    float acc = 0.0f;
    for (int64_t t = 0; t < T; t++)
        acc = fmaf(D::to_float(dz[t * lddz + r]), D::to_float(x[t * ldx + k]), acc);
    part[j][i] = acc * code_of(w, r, k);
    __syncthreads();
    if (i == 0) {
        float s = 0.0f;
        for (int n = 0; n < kGroup; n++)
            s += part[j][n];
        dscales[g * w.R + r] = s;
    }
}

constexpr int kActCluster = 8;
constexpr int kActSlab = 64;                          // columns per cluster
constexpr int kActSlots = 32;                         // row slots per CTA: 8 lanes x 8 columns cover a slab's row
constexpr int kActThreads = kActSlots * kActSlab / 8;

// dz = dy act'(pre) and its column sums.  A cluster of 8 CTAs owns 64 columns; its 256
// row slots take every 256th row, a thread 8 adjacent columns (16-byte accesses).  The
// sums meet in shared memory and through distributed shared memory, in a fixed order.
// Bound by HBM: 6 bytes per element.
template <class D>
__global__ void __cluster_dims__(kActCluster, 1, 1) __launch_bounds__(kActThreads)
    activation_backward_kernel(const uint16_t *dy, int64_t lddy, const uint16_t *pre, int64_t ldpre, int64_t T, int64_t R,
                               int act, uint16_t *dz, int64_t lddz, float *dbias)
{
    __shared__ float part[kActSlots][kActSlab];
    __shared__ float cta_sum[kActSlab];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int64_t col0 = static_cast<int64_t>(blockIdx.x / kActCluster) * kActSlab;
    const int lane = threadIdx.x % (kActSlab / 8), slot = threadIdx.x / (kActSlab / 8);
    const int64_t col = col0 + 8 * lane;
    float acc[8] = {};
    if (col < R) {
        for (int64_t t = rank * kActSlots + slot; t < T; t += kActCluster * kActSlots) {
            const uint4 a = *reinterpret_cast<const uint4 *>(dy + t * lddy + col);
            const uint4 b = *reinterpret_cast<const uint4 *>(pre + t * ldpre + col);
            const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float lo = D::to_float(static_cast<uint16_t>(av[j])) *
                                 activation_slope(D::to_float(static_cast<uint16_t>(bv[j])), act);
                const float hi = D::to_float(static_cast<uint16_t>(av[j] >> 16)) *
                                 activation_slope(D::to_float(static_cast<uint16_t>(bv[j] >> 16)), act);
                acc[2 * j] += lo;
                acc[2 * j + 1] += hi;
                o[j] = D::from_floats(lo, hi);
            }
            *reinterpret_cast<uint4 *>(dz + t * lddz + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        part[slot][8 * lane + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < kActSlab) {
        float s = 0.0f;
        for (int i = 0; i < kActSlots; i++)
            s += part[i][threadIdx.x];
        cta_sum[threadIdx.x] = s;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x < kActSlab && dbias && col0 + threadIdx.x < R) {
        float s = 0.0f;
        for (int i = 0; i < kActCluster; i++)
            s += cluster.map_shared_rank(cta_sum, i)[threadIdx.x];
        dbias[col0 + threadIdx.x] = s;
    }
    cluster.sync();  // peers keep their shared memory until rank 0 has read it
}

cq_status check_layer(int64_t T, int dtype, int64_t R, int64_t K, const void *qweight, const void *qzeros,
                      const void *scales)
{
    if (T < 0 || R < 0 || K <= 0 || R % 8 != 0 || K % kGroup != 0 || (dtype != CQ_DTYPE_BF16 && dtype != CQ_DTYPE_FP16))
        return CQ_ERR_INVALID_ARG;
    constexpr int64_t kMost = static_cast<int64_t>(1) << 31;
    if (T >= kMost || R >= kMost || K >= kMost)
        return CQ_ERR_UNSUPPORTED;
    if (R > 0 && (!qweight || !qzeros || !scales || !is_aligned(qweight, 16) || !is_aligned(qzeros, 4) ||
                  !is_aligned(scales, 16)))
        return CQ_ERR_INVALID_ARG;
    return CQ_OK;
}

cq_status launched()
{
    return cudaGetLastError() == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // namespace
}  // namespace cq

using namespace cq;

extern "C" {

cq_status cq_w4_linear(const void *x, int64_t ldx, int dtype, int64_t T, const int32_t *qweight, const int32_t *qzeros,
                       const uint16_t *gptq_scales, int64_t R, int64_t K, const void *bias, int activation,
                       const void *residual, int64_t ldres, void *y, int64_t ldy, void *pre, int64_t ldpre, void *stream)
{
    const cq_status st = check_layer(T, dtype, R, K, qweight, qzeros, gptq_scales);
    if (st != CQ_OK)
        return st;
    if (activation < CQ_ACT_NONE || activation > CQ_ACT_SILU)
        return CQ_ERR_INVALID_ARG;
    if (T == 0 || R == 0)
        return CQ_OK;
    if (!good_rows(x, ldx, K) || !good_rows(y, ldy, R) || (residual && !good_rows(residual, ldres, R)) ||
        (pre && !good_rows(pre, ldpre, R)) || (bias && !is_aligned(bias, 2)))
        return CQ_ERR_INVALID_ARG;
    const Layer w = {reinterpret_cast<const uint32_t *>(qweight), reinterpret_cast<const uint32_t *>(qzeros), gptq_scales, R, K};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>((R + kTile - 1) / kTile), static_cast<unsigned>((T + kTile - 1) / kTile));
    auto kernel = dtype == CQ_DTYPE_BF16 ? linear_plain<BF16> : linear_plain<FP16>;
    kernel<<<grid, dim3(kTile, kTile), 0, s>>>(
        static_cast<const uint16_t *>(x), ldx, T, w, static_cast<const uint16_t *>(bias), activation,
        static_cast<const uint16_t *>(residual), ldres, static_cast<uint16_t *>(y), ldy, static_cast<uint16_t *>(pre), ldpre);
    return launched();
}

cq_status cq_w4_linear_backward(const void *dz, int64_t lddz, const void *x, int64_t ldx, int dtype, int64_t T,
                                const int32_t *qweight, const int32_t *qzeros, const uint16_t *gptq_scales, int64_t R,
                                int64_t K, void *dx, int64_t lddx, float *dscales, void *stream)
{
    const cq_status st = check_layer(T, dtype, R, K, qweight, qzeros, gptq_scales);
    if (st != CQ_OK)
        return st;
    if (!is_aligned(dscales, 16) || (T > 0 && ((R > 0 && !good_rows(dz, lddz, R)) || (dx && !good_rows(dx, lddx, K)) ||
                                               (dscales && R > 0 && !good_rows(x, ldx, K)))))
        return CQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Layer w = {reinterpret_cast<const uint32_t *>(qweight), reinterpret_cast<const uint32_t *>(qzeros), gptq_scales, R, K};
    const uint16_t *d = static_cast<const uint16_t *>(dz), *xs = static_cast<const uint16_t *>(x);
    if (dx && T > 0) {
        const dim3 grid(static_cast<unsigned>(K / kTile), static_cast<unsigned>((T + kTile - 1) / kTile));
        auto kernel = dtype == CQ_DTYPE_BF16 ? input_gradient_plain<BF16> : input_gradient_plain<FP16>;
        kernel<<<grid, dim3(kTile, kTile), 0, s>>>(d, lddz, T, w, static_cast<uint16_t *>(dx), lddx);
        if (launched() != CQ_OK)
            return CQ_ERR_CUDA;
    }
    if (dscales && R > 0) {
        const dim3 grid(static_cast<unsigned>(R / 8), static_cast<unsigned>(K / kGroup));
        auto kernel = dtype == CQ_DTYPE_BF16 ? scale_gradient_plain<BF16> : scale_gradient_plain<FP16>;
        kernel<<<grid, dim3(kGroup, 8), 0, s>>>(d, lddz, xs, ldx, T, w, dscales);
        if (launched() != CQ_OK)
            return CQ_ERR_CUDA;
    }
    return CQ_OK;
}

cq_status cq_activation_backward(const void *dy, int64_t lddy, const void *pre, int64_t ldpre, int dtype, int64_t T,
                                 int64_t R, int activation, void *dz, int64_t lddz, float *dbias, void *stream)
{
    if (T < 0 || R < 0 || R % 8 != 0 || (dtype != CQ_DTYPE_BF16 && dtype != CQ_DTYPE_FP16) || activation < CQ_ACT_NONE ||
        activation > CQ_ACT_SILU || !is_aligned(dbias, 4))
        return CQ_ERR_INVALID_ARG;
    if (R >= (static_cast<int64_t>(1) << 31) || T >= (static_cast<int64_t>(1) << 31))
        return CQ_ERR_UNSUPPORTED;
    if (R == 0)
        return CQ_OK;
    if (T > 0 && (!good_rows(dy, lddy, R) || !good_rows(pre, ldpre, R) || !good_rows(dz, lddz, R)))
        return CQ_ERR_INVALID_ARG;
    const unsigned grid = static_cast<unsigned>((R + kActSlab - 1) / kActSlab * kActCluster);
    auto kernel = dtype == CQ_DTYPE_BF16 ? activation_backward_kernel<BF16> : activation_backward_kernel<FP16>;
    kernel<<<grid, kActThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t *>(dy), lddy, static_cast<const uint16_t *>(pre), ldpre, T, R, activation,
        static_cast<uint16_t *>(dz), lddz, dbias);
    return launched();
}

}  // extern "C"
