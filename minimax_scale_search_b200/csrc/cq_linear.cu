// Linear layers on 4-bit weights, and their gradients.
#include <cooperative_groups.h>

#include "cq_tensor.cuh"
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

// ---- tensor-core products with the weights ------------------------------------------------
//
// One kernel serves the layer and its input gradient: out[t][m] = sum_c act[t][c] Wm[m][c].
//   layer            m = output r, c = input k,  act = x
//   input gradient   m = input k,  c = output r, act = dz
// A tile is 128 values of m (the tensor core's rows) by N tokens; a stage 64 of c.  The
// weights' words travel as 128 outputs x 16 word rows (one group: 8 KB of codes with
// their scales and zero points), so they cross HBM and L2 at half a byte a weight.
// Eight warps turn them into 16-bit values and store them as the tensor core's A operand: a
// word is 8 adjacent inputs of one output, 16 bytes of a 128-byte shared row [r][64 k],
// chunks swizzled by r mod 8.  The layer contracts along such rows, the input gradient
// across them, so both take the same image and differ in the operand descriptor alone.
//
// Warps: 0-3 epilogue, 4-11 unpack, 12 copies activations (tensor map), 13 issues the
// matrix instructions, 14 copies weights.  CTAs are persistent; two accumulators in tensor memory let
// a tile's epilogue run under the next tile's products.

constexpr int kM = 128;
constexpr int kChunk = 64;                     // contraction per stage
constexpr int kAStage = kM * kChunk * 2;
constexpr int kRawWords = 8192;                // 16 word rows x 128 outputs
constexpr int kRawStage = kRawWords + 512;     // and 128 scales (256 B), 16 zero words (64 B)
constexpr int kUnpackWarps = 8;
constexpr int kTensorThreads = 32 * 15;

// Stages of (A, B) and of raw weights, by what 227 KB of shared memory hold.
template <int N>
struct Stages {
    static constexpr int kB = N * kChunk * 2;
    static constexpr int kOperands = N >= 256 ? 4 : 5;
    static constexpr int kRaw = N >= 256 ? 3 : N >= 128 ? 6 : 10;
    static constexpr int kBarriers = 2 * kOperands + 2 * kRaw + 4;
    static constexpr int kBytes = kOperands * (kAStage + kB) + kRaw * kRawStage + 8 * kBarriers + 16 + 1024;
    static constexpr int kColumns = 2 * N < 32 ? 32 : 2 * N;
    static_assert(kBytes <= 232448, "shared memory");
};

__device__ int g_gave_up;  // set when a wait in a kernel ran out; read by cq_w4_status

// Eight codes of a word as 16-bit values s (u - z - 1), in order, each rounded once.
template <class D>
struct Unpack;

// n = u - z - 1 of the word's eight codes: pairs of adjacent inputs.
template <class D>
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t zero, uint32_t (&n)[4])
{
    const uint32_t high = w >> 4;  // byte j of w starts with code 2j, byte j of this with code 2j + 1
#pragma unroll
    for (int j = 0; j < 4; j++)
        n[j] = D::sub((__byte_perm(w, high, j | (4 + j) << 8) & 0x000F000Fu) | D::kMagic, zero);
}

// fp16: the packed product rounds once.
template <>
struct Unpack<FP16> {
    uint32_t zero;
    __half2 s;
    __device__ __forceinline__ Unpack(uint16_t scale, uint32_t nibble)
        : zero(zero_pair<FP16>(nibble)), s(__half2half2(__ushort_as_half(scale)))
    {
    }
    __device__ __forceinline__ uint4 operator()(uint32_t w) const
    {
        uint32_t n[4];
        unpack_codes<FP16>(w, zero, n);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const __half2 p = __hmul2(reinterpret_cast<const __half2 &>(n[j]), s);
            n[j] = reinterpret_cast<const uint32_t &>(p);
        }
        return make_uint4(n[0], n[1], n[2], n[3]);
    }
};

// bf16: s = hi + lo, hi the scale rounded to 8 bits and lo the at most 3 bits left, so
// n lo is exact and fma(n, hi, n lo) rounds n s once.
template <>
struct Unpack<BF16> {
    uint32_t zero;
    __nv_bfloat162 hi, lo;
    __device__ __forceinline__ Unpack(uint16_t scale, uint32_t nibble) : zero(zero_pair<BF16>(nibble))
    {
        const float s = half_bits(scale);
        const __nv_bfloat16 h = __float2bfloat16_rn(s);
        hi = __bfloat162bfloat162(h);
        lo = __bfloat162bfloat162(__float2bfloat16_rn(s - __bfloat162float(h)));
    }
    __device__ __forceinline__ uint4 operator()(uint32_t w) const
    {
        uint32_t n[4];
        unpack_codes<BF16>(w, zero, n);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const __nv_bfloat162 v = reinterpret_cast<const __nv_bfloat162 &>(n[j]);
            const __nv_bfloat162 p = __hfma2(v, hi, __hmul2(v, lo));
            n[j] = reinterpret_cast<const uint32_t &>(p);
        }
        return make_uint4(n[0], n[1], n[2], n[3]);
    }
};

struct Epilogue {
    const uint16_t *bias, *res;
    uint16_t *y, *pre;
    int64_t ldres, ldy, ldpre;
    int act;
};

// A ring's slot and the parity of its phase.
template <int kSlots>
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) {
            slot = 0;
            parity ^= 1;
        }
    }
};

template <class D, int N, bool kGradient>
__global__ void __launch_bounds__(kTensorThreads, 1)
    weights_product_kernel(const __grid_constant__ CUtensorMap act_map, const __grid_constant__ CUtensorMap word_map,
                           Layer w, int64_t T, Epilogue ep)
{
    using S = Stages<N>;
    extern __shared__ char shared_raw[];
    const uint32_t base = (tc::smem_address(shared_raw) + 1023) & ~1023u;
    char *shared = shared_raw + (base - tc::smem_address(shared_raw));
    const uint32_t raw0 = base + S::kOperands * (kAStage + S::kB), bars = raw0 + S::kRaw * kRawStage;
    auto a_at = [&](int i) { return base + i * (kAStage + S::kB); };
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 8 * (S::kOperands + i); };
    auto raw_full = [&](int i) { return bars + 8 * (2 * S::kOperands + i); };
    auto raw_empty = [&](int i) { return bars + 8 * (2 * S::kOperands + S::kRaw + i); };
    auto sums_full = [&](int i) { return bars + 8 * (2 * S::kOperands + 2 * S::kRaw + i); };
    auto sums_empty = [&](int i) { return bars + 8 * (2 * S::kOperands + 2 * S::kRaw + 2 + i); };
    volatile int *stop = reinterpret_cast<volatile int *>(shared + (bars - base) + 8 * S::kBarriers);
    uint32_t *tmem_at = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(stop + 1));

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t rows = kGradient ? w.K : w.R, depth = kGradient ? (w.R + kM - 1) / kM : w.K / kM;  // in steps of 128
    const int64_t tiles_n = (T + N - 1) / N, tiles = (rows + kM - 1) / kM * tiles_n;

    if (warp == 13)
        tc::tmem_alloc(tc::smem_address(tmem_at), S::kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kOperands; i++) {
            tc::barrier_init(full(i), kUnpackWarps + 1);
            tc::barrier_init(empty(i), 1);
        }
        for (int i = 0; i < S::kRaw; i++) {
            tc::barrier_init(raw_full(i), 32 + 1);
            tc::barrier_init(raw_empty(i), kUnpackWarps);
        }
        for (int i = 0; i < 2; i++) {
            tc::barrier_init(sums_full(i), 1);
            tc::barrier_init(sums_empty(i), 4);
        }
        *stop = 0;
        tc::barrier_init_fence();
    }
    if (threadIdx.x == 32) {
        tc::prefetch_map(&act_map);
        tc::prefetch_map(&word_map);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_at;

    if (warp < 4) {  // epilogue: a thread has one m, a chunk of 32 tokens at a time
        Ring<2> sums;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int64_t m = tile / tiles_n * kM + 32 * warp + lane, t0 = tile % tiles_n * N;
            const float bias = ep.bias && m < rows ? D::to_float(ep.bias[m]) : 0.0f;
            if (!tc::barrier_wait_warp(sums_full(sums.slot), sums.parity, stop))
                break;
            tc::fence_after();
            for (int c = 0; c < N; c += 32) {
                if (t0 + c >= T)
                    break;
                uint32_t v[32];
                __syncwarp();
                tc::tmem_load32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * N + c, v);
                if (m < rows) {
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        const int64_t t = t0 + c + j;
                        if (t >= T)
                            break;
                        const float z = __uint_as_float(v[j]) + bias;
                        if (kGradient) {
                            ep.y[t * ep.ldy + m] = D::from_float(z);
                            continue;
                        }
                        if (ep.pre)
                            ep.pre[t * ep.ldpre + m] = D::from_float(z);
                        float o = activate(z, ep.act);
                        if (ep.res)
                            o += D::to_float(ep.res[t * ep.ldres + m]);
                        ep.y[t * ep.ldy + m] = D::from_float(o);
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(sums_empty(sums.slot));
            sums.next();
        }
    } else if (warp < 4 + kUnpackWarps) {  // unpack
        const int i = threadIdx.x - 128;
        Ring<S::kRaw> raw;
        Ring<S::kOperands> op;
        bool going = true;
        for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
            for (int64_t g = 0; going && g < depth; g++) {
                going = tc::barrier_wait_warp(raw_full(raw.slot), raw.parity, stop);
                const char *slot = shared + (raw0 - base) + raw.slot * kRawStage;
                const uint32_t *words = reinterpret_cast<const uint32_t *>(slot);
                const uint16_t *scales = reinterpret_cast<const uint16_t *>(slot + kRawWords);
                const uint32_t *zeros = reinterpret_cast<const uint32_t *>(slot + kRawWords + 256);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (!going)
                        break;
                    // layer: 128 outputs x 8 word rows; gradient: 64 outputs x 16 word rows
                    const int r = kGradient ? h * 64 + (i & 63) : i & 127;
                    const int k8 = kGradient ? (i >> 6) * 4 : h * 8 + (i >> 7) * 4;
                    const Unpack<D> unpack(scales[r], (zeros[r >> 3] >> (4 * (r & 7))) & 15u);
                    uint32_t word[4];
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        word[j] = words[(k8 + j) * kM + r];
                    going = tc::barrier_wait_warp(empty(op.slot), op.parity ^ 1, stop);
                    if (!going)
                        break;
                    char *a = shared + (a_at(op.slot) - base) + (kGradient ? (k8 >> 3) * (kAStage / 2) + (i & 63) * 128 : r * 128);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        *reinterpret_cast<uint4 *>(a + (((k8 + j) & 7) ^ (r & 7)) * 16) = unpack(word[j]);
                    tc::fence_shared_writes();
                    __syncwarp();
                    if (lane == 0)
                        tc::barrier_arrive(full(op.slot));
                    op.next();
                }
                if (going && lane == 0)
                    tc::barrier_arrive(raw_empty(raw.slot));
                raw.next();
            }
        }
    } else if (warp == 12) {  // activations
        if (lane == 0) {
            Ring<S::kOperands> op;
            bool going = true;
            for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
                const int t0 = static_cast<int>(tile % tiles_n * N);
                for (int64_t c = 0; c < 2 * depth; c++) {
                    going = tc::barrier_wait(empty(op.slot), op.parity ^ 1, stop);
                    if (!going)
                        break;
                    tc::barrier_expect(full(op.slot), S::kB);
                    tc::copy_box(a_at(op.slot) + kAStage, &act_map, static_cast<int>(c * kChunk), t0, full(op.slot));
                    op.next();
                }
            }
        }
    } else if (warp == 13) {  // matrix instructions
        if (lane == 0) {
            constexpr uint32_t kInstr = tc::instruction(D::kMagic == BF16::kMagic, kGradient, false, N);
            Ring<S::kOperands> op;
            Ring<2> sums;
            bool going = true;
            for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
                going = tc::barrier_wait(sums_empty(sums.slot), sums.parity ^ 1, stop);
                if (!going)
                    break;
                tc::fence_after();
                for (int64_t c = 0; c < 2 * depth; c++) {
                    going = tc::barrier_wait(full(op.slot), op.parity, stop);
                    if (!going)
                        break;
                    tc::fence_after();
                    const uint32_t a = a_at(op.slot), b = a + kAStage;
#pragma unroll
                    for (int k = 0; k < kChunk / 16; k++) {
                        const uint64_t da = kGradient ? tc::descriptor(a + k * 2048, kAStage / 2, 1024)
                                                      : tc::descriptor(a + k * 32, 16, 1024);
                        tc::mma(tmem + sums.slot * N, da, tc::descriptor(b + k * 32, 16, 1024), kInstr, c > 0 || k > 0);
                    }
                    tc::commit(empty(op.slot));
                    op.next();
                }
                if (!going)
                    break;
                tc::commit(sums_full(sums.slot));
                sums.next();
            }
        }
    } else {  // weights
        Ring<S::kRaw> raw;
        bool going = true;
        for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
            const int64_t m0 = tile / tiles_n * kM;
            for (int64_t g = 0; g < depth; g++) {
                going = tc::barrier_wait_warp(raw_empty(raw.slot), raw.parity ^ 1, stop);
                if (!going)
                    break;
                const int64_t r0 = kGradient ? g * kM : m0, group = kGradient ? m0 / kGroup : g;
                const uint32_t at = raw0 + raw.slot * kRawStage;
                if (lane == 0) {
                    tc::barrier_expect(raw_full(raw.slot), kRawWords);
                    tc::copy_box(at, &word_map, static_cast<int>(r0), static_cast<int>(group * kWordsPerGroup), raw_full(raw.slot));
                }
                const int64_t r = r0 + 8 * (lane & 15);  // 8 outputs: a 16-byte run of scales, a word of zeros
                const bool inside = r < w.R;
                if (lane < 16)
                    tc::copy_async<16>(at + kRawWords + 16 * lane, w.scales + (inside ? group * w.R + r : 0), inside);
                else
                    tc::copy_async<4>(at + kRawWords + 256 + 4 * (lane - 16), w.qzeros + (inside ? (group * w.R + r) / 8 : 0), inside);
                tc::copy_async_arrive(raw_full(raw.slot));
                raw.next();
            }
        }
        tc::copy_async_wait();
    }
    __syncthreads();
    if (*stop) {
        tc::let_copies_land();
        g_gave_up = 1;
    }
    if (warp == 13)
        tc::tmem_free(tmem, S::kColumns);
}

// ---- scale gradient ----------------------------------------------------------------------------
//
// dscales[g][r] = sum_{i in g} n[r][i] dW[r][i], dW = dz^T x.  A tile is 128 outputs by
// 256 inputs (two groups) of dW, contracted over the tokens 64 at a time; both operands come
// straight from the row-major dz and x (contracted across their rows).  The
// epilogue multiplies a lane's 128 sums of a group by its codes and adds them up, so dW stays in
// tensor memory.  Two accumulators, persistent CTAs; warps 0-3 epilogue, 4 copies, 5 issues.

constexpr int kGradN = 256;
constexpr int kGradB = kGradN * kChunk * 2;
constexpr int kGradStages = 4;
constexpr int kGradThreads = 32 * 6;
constexpr int kGradBytes = kGradStages * (kAStage + kGradB) + 8 * (2 * kGradStages + 4) + 16 + 1024;

template <class D>
__global__ void __launch_bounds__(kGradThreads, 1)
    scale_gradient_kernel(const __grid_constant__ CUtensorMap dz_map, const __grid_constant__ CUtensorMap x_map, Layer w,
                          int64_t T, float *dscales)
{
    extern __shared__ char shared_raw[];
    const uint32_t base = (tc::smem_address(shared_raw) + 1023) & ~1023u;
    char *shared = shared_raw + (base - tc::smem_address(shared_raw));
    const uint32_t bars = base + kGradStages * (kAStage + kGradB);
    auto a_at = [&](int i) { return base + i * (kAStage + kGradB); };
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 8 * (kGradStages + i); };
    auto sums_full = [&](int i) { return bars + 8 * (2 * kGradStages + i); };
    auto sums_empty = [&](int i) { return bars + 8 * (2 * kGradStages + 2 + i); };
    volatile int *stop = reinterpret_cast<volatile int *>(shared + (bars - base) + 8 * (2 * kGradStages + 4));
    uint32_t *tmem_at = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(stop + 1));

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t tiles_k = (w.K + kGradN - 1) / kGradN, tiles = (w.R + kM - 1) / kM * tiles_k;
    const int64_t chunks = (T + kChunk - 1) / kChunk;

    if (warp == 5)
        tc::tmem_alloc(tc::smem_address(tmem_at), 2 * kGradN);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kGradStages; i++) {
            tc::barrier_init(full(i), 1);
            tc::barrier_init(empty(i), 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::barrier_init(sums_full(i), 1);
            tc::barrier_init(sums_empty(i), 4);
        }
        *stop = 0;
        tc::barrier_init_fence();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_at;

    if (warp < 4) {
        Ring<2> sums;
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int64_t r = tile / tiles_k * kM + 32 * warp + lane, g0 = tile % tiles_k * (kGradN / kGroup);
            if (!tc::barrier_wait_warp(sums_full(sums.slot), sums.parity, stop))
                break;
            tc::fence_after();
            for (int64_t g = g0; g < g0 + kGradN / kGroup && g < w.K / kGroup; g++) {
                const bool inside = r < w.R;
                const int z1 = inside ? static_cast<int>((w.qzeros[(g * w.R + r) / 8] >> (4 * (r & 7))) & 15u) + 1 : 0;
                float total = 0.0f;
                for (int c = 0; c < kGroup; c += 32) {
                    uint32_t v[32];
                    __syncwarp();
                    tc::tmem_load32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * kGradN +
                                        static_cast<uint32_t>(g - g0) * kGroup + c, v);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const uint32_t word = inside ? w.qweight[(g * kWordsPerGroup + c / 8 + j) * w.R + r] : 0u;
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            total = fmaf(__uint_as_float(v[8 * j + i]),
                                         static_cast<float>(static_cast<int>((word >> (4 * i)) & 15u) - z1), total);
                    }
                }
                if (inside)
                    dscales[g * w.R + r] = total;
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(sums_empty(sums.slot));
            sums.next();
        }
    } else if (warp == 4) {
        if (lane == 0) {
            Ring<kGradStages> op;
            bool going = true;
            for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
                const int r0 = static_cast<int>(tile / tiles_k * kM), k0 = static_cast<int>(tile % tiles_k * kGradN);
                for (int64_t c = 0; c < chunks; c++) {
                    going = tc::barrier_wait(empty(op.slot), op.parity ^ 1, stop);
                    if (!going)
                        break;
                    const int t0 = static_cast<int>(c * kChunk);
                    tc::barrier_expect(full(op.slot), kAStage + kGradB);
#pragma unroll
                    for (int j = 0; j < kM / 64; j++)
                        tc::copy_box(a_at(op.slot) + j * 8192, &dz_map, r0 + 64 * j, t0, full(op.slot));
#pragma unroll
                    for (int j = 0; j < kGradN / 64; j++)
                        tc::copy_box(a_at(op.slot) + kAStage + j * 8192, &x_map, k0 + 64 * j, t0, full(op.slot));
                    op.next();
                }
            }
        }
    } else if (lane == 0) {
        constexpr uint32_t kInstr = tc::instruction(D::kMagic == BF16::kMagic, true, true, kGradN);
        Ring<kGradStages> op;
        Ring<2> sums;
        bool going = true;
        for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
            going = tc::barrier_wait(sums_empty(sums.slot), sums.parity ^ 1, stop);
            if (!going)
                break;
            tc::fence_after();
            for (int64_t c = 0; c < chunks; c++) {
                going = tc::barrier_wait(full(op.slot), op.parity, stop);
                if (!going)
                    break;
                tc::fence_after();
                const uint32_t a = a_at(op.slot), b = a + kAStage;
#pragma unroll
                for (int k = 0; k < kChunk / 16; k++)
                    tc::mma(tmem + sums.slot * kGradN, tc::descriptor(a + k * 2048, 8192, 1024),
                            tc::descriptor(b + k * 2048, 8192, 1024), kInstr, c > 0 || k > 0);
                tc::commit(empty(op.slot));
                op.next();
            }
            if (!going)
                break;
            tc::commit(sums_full(sums.slot));
            sums.next();
        }
    }
    __syncthreads();
    if (*stop) {
        tc::let_copies_land();
        g_gave_up = 1;
    }
    if (warp == 5)
        tc::tmem_free(tmem, 2 * kGradN);
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

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 148;
    return sms > 0 ? sms : 148;
}

cq_status launched()
{
    return cudaGetLastError() == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

template <class D>
CUtensorMapDataType map_type()
{
    return D::kMagic == BF16::kMagic ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

template <class D, int N, bool kGradient>
cq_status run_product(const uint16_t *act, int64_t ld, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    CUtensorMap act_map, word_map;
    const int64_t rows = kGradient ? w.K : w.R;
    if (!tc::make_map(&act_map, map_type<D>(), 2, act, T, kGradient ? w.R : w.K, ld, N, kChunk, true) ||
        !tc::make_map(&word_map, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, w.qweight, w.K / 8, w.R, w.R, kWordsPerGroup, kM, false))
        return CQ_ERR_CUDA;
    auto kernel = weights_product_kernel<D, N, kGradient>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Stages<N>::kBytes) != cudaSuccess)
        return CQ_ERR_CUDA;
    const int64_t tiles = (rows + kM - 1) / kM * ((T + N - 1) / N), sms = sm_count();
    kernel<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kTensorThreads, Stages<N>::kBytes, stream>>>(act_map, word_map, w, T, ep);
    return launched();
}

// Tokens per tile: the least time by a count of waves, where a stage of N tokens takes the tensor
// core 2 N cycles and the unpacking warps about 200.
template <class D, bool kGradient>
cq_status product(const uint16_t *act, int64_t ld, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    const int64_t m = ((kGradient ? w.K : w.R) + kM - 1) / kM, sms = sm_count();
    int64_t least = INT64_MAX;
    int best = 256;
    for (int n = 256; n >= 32; n /= 2) {
        const int64_t waves = (m * ((T + n - 1) / n) + sms - 1) / sms, cost = waves * (2 * n > 200 ? 2 * n : 200);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best == 256   ? run_product<D, 256, kGradient>(act, ld, T, w, ep, stream)
           : best == 128 ? run_product<D, 128, kGradient>(act, ld, T, w, ep, stream)
           : best == 64  ? run_product<D, 64, kGradient>(act, ld, T, w, ep, stream)
                         : run_product<D, 32, kGradient>(act, ld, T, w, ep, stream);
}

template <class D>
cq_status scale_gradient(const uint16_t *dz, int64_t lddz, const uint16_t *x, int64_t ldx, int64_t T, const Layer &w,
                         float *dscales, cudaStream_t stream)
{
    if (T == 0)
        return cudaMemsetAsync(dscales, 0, static_cast<size_t>(w.K / kGroup) * w.R * 4, stream) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
    CUtensorMap dz_map, x_map;
    if (!tc::make_map(&dz_map, map_type<D>(), 2, dz, T, w.R, lddz, kChunk, 64, true) ||
        !tc::make_map(&x_map, map_type<D>(), 2, x, T, w.K, ldx, kChunk, 64, true))
        return CQ_ERR_CUDA;
    auto kernel = scale_gradient_kernel<D>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradBytes) != cudaSuccess)
        return CQ_ERR_CUDA;
    const int64_t tiles = (w.R + kM - 1) / kM * ((w.K + kGradN - 1) / kGradN), sms = sm_count();
    kernel<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kGradThreads, kGradBytes, stream>>>(dz_map, x_map, w, T, dscales);
    return launched();
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
    const uint16_t *in = static_cast<const uint16_t *>(x);
    const Epilogue ep = {static_cast<const uint16_t *>(bias), static_cast<const uint16_t *>(residual),
                         static_cast<uint16_t *>(y), static_cast<uint16_t *>(pre), ldres, ldy, ldpre, activation};
    return dtype == CQ_DTYPE_BF16 ? product<BF16, false>(in, ldx, T, w, ep, s) : product<FP16, false>(in, ldx, T, w, ep, s);
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
        if (R == 0)
            return cudaMemset2DAsync(dx, static_cast<size_t>(lddx) * 2, 0, static_cast<size_t>(K) * 2, static_cast<size_t>(T), s) == cudaSuccess
                       ? CQ_OK
                       : CQ_ERR_CUDA;
        const Epilogue ep = {nullptr, nullptr, static_cast<uint16_t *>(dx), nullptr, 0, lddx, 0, CQ_ACT_NONE};
        const cq_status did = dtype == CQ_DTYPE_BF16 ? product<BF16, true>(d, lddz, T, w, ep, s) : product<FP16, true>(d, lddz, T, w, ep, s);
        if (did != CQ_OK)
            return did;
    }
    if (dscales && R > 0)
        return dtype == CQ_DTYPE_BF16 ? scale_gradient<BF16>(d, lddz, xs, ldx, T, w, dscales, s)
                                      : scale_gradient<FP16>(d, lddz, xs, ldx, T, w, dscales, s);
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
