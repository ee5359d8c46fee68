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
// Warps: 0-3 epilogue, 4-19 unpack, then one that copies activations (tensor map), one that
// issues the matrix instructions, one that copies weights.  CTAs are persistent; two accumulators in tensor memory let
// a tile's epilogue run under the next tile's products.

constexpr int kM = 128;
constexpr int kChunk = 64;                     // contraction per stage
constexpr int kAStage = kM * kChunk * 2;
constexpr int kRawWords = 8192;                // 16 word rows x 128 outputs
constexpr int kRawStage = kRawWords + 512;     // and 128 scales (256 B), 16 zero words (64 B)
constexpr int kUnpackSets = 4, kSetWarps = 4;   // a set fills a stage
constexpr int kUnpackWarps = kSetWarps * kUnpackSets;
constexpr int kSetWords = kM * kChunk / 8 / (32 * kSetWarps);  // words of a stage per thread
constexpr int kCopyWarp = 4 + kUnpackWarps, kIssueWarp = kCopyWarp + 1;
constexpr int kTensorThreads = 32 * (kIssueWarp + 2);

// Stages of (A, B) and of raw weights, by what 227 KB of shared memory hold.
template <int N>
struct Stages {
    static constexpr int kB = N * kChunk * 2;
    static constexpr int kOperands = N >= 128 ? 4 : 5;
    static constexpr int kRaw = N >= 256 ? 3 : N >= 128 ? 9 : 10;
    static constexpr int kBarriers = 2 * kOperands + 2 * kRaw + 4;
    static constexpr int kControl = 8 * kBarriers + 16;      // barriers, the stop flag, tensor memory's address
    static constexpr int kTurn = 4 * 16 * 33 * 4;            // the epilogue's turn from lanes to rows
    static constexpr int kBytes = kOperands * (kAStage + kB) + kRaw * kRawStage + kControl + kTurn + 1024;
    static constexpr int kColumns = 2 * N < 32 ? 32 : 2 * N;
    static_assert(kBytes <= 232448, "shared memory");
    // A set that has filled stage c goes on to c + kUnpackSets.  It knows that c - kOperands has been read, and the
    // parity of its next wait needs c + kUnpackSets - 2 kOperands to have been.
    static_assert(kUnpackSets % 2 == 0 && kUnpackSets <= kOperands, "phases");
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
    __device__ __forceinline__ void skip(int n)
    {
        for (int i = 0; i < n; i++)
            next();
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

    const int warp = tc::uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int64_t rows = kGradient ? w.K : w.R, depth = kGradient ? (w.R + kM - 1) / kM : w.K / kM;  // in steps of 128
    const int64_t tiles_n = (T + N - 1) / N, tiles = (rows + kM - 1) / kM * tiles_n;

    if (warp == kIssueWarp)
        tc::tmem_alloc(tc::smem_address(tmem_at), S::kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kOperands; i++) {
            tc::barrier_init(full(i), kSetWarps + 1);
            tc::barrier_init(empty(i), 1);
        }
        for (int i = 0; i < S::kRaw; i++) {
            tc::barrier_init(raw_full(i), 32 + 1);
            tc::barrier_init(raw_empty(i), 2 * kSetWarps);
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
    const uint32_t tmem = tc::uniform(*tmem_at);

    if (warp < 4) {
        // Epilogue, a warp's 32 m by 16 tokens at a time: a thread has one m in tensor memory;
        // through 2 KB of shared memory it gets 8 adjacent m of one token, 16 bytes of every row it touches.
        float *turn = reinterpret_cast<float *>(shared + (bars - base) + S::kControl) + warp * (16 * 33);
        Ring<2> sums;
        const int tok = lane >> 2, part = 8 * (lane & 3);
        for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int64_t m0 = tile / tiles_n * kM + 32 * warp, t0 = tile % tiles_n * N, m = m0 + part;
            const float bias = ep.bias && m0 + lane < rows ? D::to_float(ep.bias[m0 + lane]) : 0.0f;
            const int64_t left = T - t0;
            const int tokens = left < N ? static_cast<int>(left) : N;
            if (!tc::barrier_wait_warp(sums_full(sums.slot), sums.parity, stop))
                break;
            tc::fence_after();
            for (int c = 0; c < tokens; c += 16) {
                uint4 res[2];
#pragma unroll
                for (int h = 0; h < 2; h++)
                    if (!kGradient && ep.res && m < rows && c + 8 * h + tok < tokens)
                        res[h] = *reinterpret_cast<const uint4 *>(ep.res + (t0 + c + 8 * h + tok) * ep.ldres + m);
                uint32_t v[16];
                tc::tmem_load16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * N + c, v);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 16; j++)
                    turn[j * 33 + lane] = __uint_as_float(v[j]) + bias;
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (m >= rows || c + 8 * h + tok >= tokens)  // rows % 8 == 0: eight m in or out together
                        continue;
                    const int64_t t = t0 + c + 8 * h + tok;
                    float z[8];
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        z[j] = turn[(8 * h + tok) * 33 + part + j];
                    if (!kGradient) {
                        if (ep.pre)
                            *reinterpret_cast<uint4 *>(ep.pre + t * ep.ldpre + m) = narrow<D>(z);
                        activate(z, ep.act);
                        if (ep.res) {
                            float r[8];
                            widen<D>(res[h], r);
#pragma unroll
                            for (int j = 0; j < 8; j++)
                                z[j] += r[j];
                        }
                    }
                    *reinterpret_cast<uint4 *>(ep.y + t * ep.ldy + m) = narrow<D>(z);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(sums_empty(sums.slot));
            sums.next();
        }
    } else if (warp < 4 + kUnpackWarps) {  // unpack
        // Sets of warps take the stages in turn: half a group each (h).
        const int i = threadIdx.x % (32 * kSetWarps), set = (warp - 4) / kSetWarps, h = set & 1;
        const int r = kGradient ? h * 64 + (i & 63) : i & 127;                                 // output within the 128
        const int k8 = kGradient ? (i >> 6) * kSetWords : h * 8 + (i >> 7) * kSetWords;        // word row within the 16
        const uint32_t a = kGradient ? (k8 >> 3) * (kAStage / 2) + (r & 63) * 128 : r * 128;
        const int64_t mine = static_cast<int64_t>(blockIdx.x) < tiles ? (tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
        Ring<S::kRaw> raw;
        Ring<S::kOperands> op;
        raw.skip(set / 2);
        op.skip(set);
        for (int64_t g = set / 2; g < mine * depth; g += kUnpackSets / 2) {
            if (!tc::barrier_wait_warp(raw_full(raw.slot), raw.parity, stop))
                break;
            const char *slot = shared + (raw0 - base) + raw.slot * kRawStage;
            const uint32_t *words = reinterpret_cast<const uint32_t *>(slot) + k8 * kM + r;
            const Unpack<D> unpack(reinterpret_cast<const uint16_t *>(slot + kRawWords)[r],
                                   (reinterpret_cast<const uint32_t *>(slot + kRawWords + 256)[r >> 3] >> (4 * (r & 7))) & 15u);
            uint32_t word[kSetWords];
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                word[j] = words[j * kM];
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(raw_empty(raw.slot));
            raw.skip(kUnpackSets / 2);
            uint4 values[kSetWords];
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                values[j] = unpack(word[j]);
            if (!tc::barrier_wait_warp(empty(op.slot), op.parity ^ 1, stop))
                break;
            char *to = shared + (a_at(op.slot) - base) + a;
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                *reinterpret_cast<uint4 *>(to + (((k8 + j) & 7) ^ (r & 7)) * 16) = values[j];
            tc::fence_shared_writes();
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(full(op.slot));
            op.skip(kUnpackSets);
        }
    } else if (warp == kCopyWarp) {  // activations
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
    } else if (warp == kIssueWarp) {  // matrix instructions: the loop is the whole warp's, so that what it computes stays uniform
        constexpr uint32_t kInstr = tc::instruction(D::kMagic == BF16::kMagic, kGradient, false, N);
        constexpr uint32_t kStep = kGradient ? 2048 : 32;  // 16 of the contraction in A: 16 rows, or 32 bytes of a row
        const uint64_t a_first = tc::descriptor(base, kGradient ? kAStage / 2 : 16, 1024);
        const uint64_t b_first = tc::descriptor(base + kAStage, 16, 1024);
        const int64_t mine = static_cast<int64_t>(blockIdx.x) < tiles ? (tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
        const uint32_t stages = static_cast<uint32_t>(2 * depth);
        Ring<2> sums;
        uint32_t parity = 0, c = 0;
        int64_t left = mine;
        bool going = left > 0;
        while (going) {
#pragma unroll
            for (int slot = 0; slot < S::kOperands; slot++) {  // unrolled: addresses and descriptors stay fixed
                if (c == 0) {
                    going = going && tc::barrier_wait_warp(sums_empty(sums.slot), sums.parity ^ 1, stop);
                    tc::fence_after();
                }
                going = going && tc::barrier_wait_warp(full(slot), parity, stop);
                if (!going)
                    break;
                tc::fence_after();
                const uint64_t a = a_first + static_cast<uint32_t>(slot * (kAStage + S::kB) / 16);
                const uint64_t b = b_first + static_cast<uint32_t>(slot * (kAStage + S::kB) / 16);
                const uint32_t d = tmem + sums.slot * N;
                const bool last = ++c == stages;
                if (tc::elected()) {
                    tc::mma(d, a, b, kInstr, c > 1);
#pragma unroll
                    for (int k = 1; k < kChunk / 16; k++)
                        tc::mma_add(d, a + k * (kStep / 16), b + k * (32 / 16), kInstr);
                    tc::commit(empty(slot));
                    if (last)
                        tc::commit(sums_full(sums.slot));
                }
                __syncwarp();
                if (last) {
                    c = 0;
                    sums.next();
                    if (--left == 0) {
                        going = false;
                        break;
                    }
                }
            }
            parity ^= 1;
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
    if (warp == kIssueWarp)
        tc::tmem_free(tmem, S::kColumns);
}

// ---- few rows ----------------------------------------------------------------------------------
//
// Up to 16 rows the weights' bytes are the work: a CTA has 32 outputs, its 8 warps (of all
// the CTAs of a cluster) take the groups in turn.  A thread loads 4 outputs' words at once (16 bytes,
// 4 lanes of a word row make 128-byte runs over 8 lanes); a word is 8 inputs, whose pairs (q, q + 4)
// come out of it with a shift and a mask.  That order of the inputs is as good as any for the
// m16n8k16 product if the activations' pairs are the same.  The codes enter as integers and each
// group's fp32 sum is scaled after, so the weights are exact.
// The warps' and the cluster's sums meet in shared memory in a fixed order.

constexpr int kFewWarps = 8;
constexpr int kFewRows = 32;   // outputs per CTA

template <class D>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);

template <>
__device__ __forceinline__ void mma_16x8x16<BF16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <>
__device__ __forceinline__ void mma_16x8x16<FP16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a thread needs of one group: 4 word rows of its 4 outputs, their scales and
// zero points, and 32 inputs of one token of each tile of 8.
template <int NT>
struct GroupData {
    uint4 words[4];
    uint2 scales;
    uint32_t zeros;
    uint4 x[NT][4];
};

template <class D, int NT>
__global__ void __launch_bounds__(32 * kFewWarps)
    few_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int T, Layer w, Epilogue ep)
{
    __shared__ float sums[kFewWarps][8 * NT * kFewRows];
    __shared__ float cta_sums[8 * NT * kFewRows];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int quad = lane >> 2, c = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / ranks) * kFewRows, r = r0 + 4 * quad;
    const bool inside = r < w.R;  // R % 8 == 0: four outputs in or out together
    const int64_t groups = w.K / kGroup;

    auto load = [&](int64_t g, GroupData<NT> &d) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            d.words[j] = inside ? __ldcs(reinterpret_cast<const uint4 *>(w.qweight + (g * kWordsPerGroup + 4 * j + c) * w.R + r))
                                : make_uint4(0, 0, 0, 0);
        d.scales = inside ? *reinterpret_cast<const uint2 *>(w.scales + g * w.R + r) : make_uint2(0, 0);
        d.zeros = inside ? w.qzeros[(g * w.R + r) / 8] >> (4 * (r & 7)) : 0u;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                d.x[n][j] = 8 * n + quad < T
                                ? *reinterpret_cast<const uint4 *>(x + (8 * n + quad) * ldx + g * kGroup + 8 * (4 * j + c))
                                : make_uint4(0, 0, 0, 0);
    };

    float total[2][NT][4] = {};
    auto multiply = [&](const GroupData<NT> &d) {
        float acc[2][NT][4] = {};
        uint32_t zero[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            zero[i] = zero_pair<D>((d.zeros >> (4 * i)) & 15u);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t word[4] = {d.words[j].x, d.words[j].y, d.words[j].z, d.words[j].w};
            uint32_t pair[4][4];  // [output][q]: inputs q and q + 4
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    pair[i][q] = D::sub(((word[i] >> (4 * q)) & 0x000F000Fu) | D::kMagic, zero[i]);
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const uint4 v = d.x[n][j];
                const uint32_t b[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                       __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
                for (int p = 0; p < 2; p++) {
#pragma unroll
                    for (int s = 0; s < 2; s++) {
                        const uint32_t a[4] = {pair[2 * p][2 * s], pair[2 * p + 1][2 * s], pair[2 * p][2 * s + 1],
                                               pair[2 * p + 1][2 * s + 1]};
                        mma_16x8x16<D>(acc[p][n], a, b[2 * s], b[2 * s + 1]);
                    }
                }
            }
        }
        const float s[4] = {half_bits(static_cast<uint16_t>(d.scales.x)), half_bits(static_cast<uint16_t>(d.scales.x >> 16)),
                            half_bits(static_cast<uint16_t>(d.scales.y)), half_bits(static_cast<uint16_t>(d.scales.y >> 16))};
#pragma unroll
        for (int p = 0; p < 2; p++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    total[p][n][i] = fmaf(s[2 * p + (i >> 1)], acc[p][n][i], total[p][n][i]);
    };

    const int64_t step = static_cast<int64_t>(ranks) * kFewWarps;
    int64_t g = static_cast<int64_t>(rank) * kFewWarps + warp;
    if (g < groups) {
        GroupData<NT> now, next;
        load(g, now);
        for (; g < groups; g += step) {
            if (g + step < groups)
                load(g + step, next);
            multiply(now);
            now = next;
        }
    }
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                sums[warp][(8 * n + 2 * c + (i & 1)) * kFewRows + 4 * quad + 2 * p + (i >> 1)] = total[p][n][i];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const int e = threadIdx.x + n * 32 * kFewWarps;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kFewWarps; i++)
            s += sums[i][e];
        cta_sums[e] = s;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    const int share = 8 * NT * kFewRows / ranks;
    if (static_cast<int>(threadIdx.x) < share || NT > 1) {
        for (int i = threadIdx.x; i < share; i += 32 * kFewWarps) {
            const int e = rank * share + i, t = e / kFewRows;
            const int64_t out = r0 + e % kFewRows;
            float z[1] = {0.0f};
            for (int k = 0; k < ranks; k++)
                z[0] += ranks > 1 ? cluster.map_shared_rank(cta_sums, k)[e] : cta_sums[e];
            if (t >= T || out >= w.R)
                continue;
            z[0] += ep.bias ? D::to_float(ep.bias[out]) : 0.0f;
            if (ep.pre)
                ep.pre[t * ep.ldpre + out] = D::from_float(z[0]);
            activate(z, ep.act);
            if (ep.res)
                z[0] += D::to_float(ep.res[t * ep.ldres + out]);
            ep.y[t * ep.ldy + out] = D::from_float(z[0]);
        }
    }
    if (ranks > 1)
        cluster.sync();  // peers keep their shared memory until it has been read
}

// ---- scale gradient ----------------------------------------------------------------------------
//
// dscales[g][r] = sum_{i in g} n[r][i] dW[r][i], dW = dz^T x.  A tile is 128 outputs by
// 256 inputs (two groups) of dW, contracted over the tokens 64 at a time; both operands come
// straight from the row-major dz and x (contracted across their rows).  The
// epilogue multiplies a lane's 128 sums of a group by its codes and adds them up, so dW stays in
// tensor memory.  The tensor core's fp32 sums are cut off, not rounded, at each of its steps of 16 tokens;
// kSpan bounds the drift: every span of tokens has sums of its own, which the epilogue adds up.  Two accumulators, persistent CTAs; warps 0-3 epilogue, 4 copies, 5 issues.

constexpr int kGradN = 256;
constexpr int kGradB = kGradN * kChunk * 2;
constexpr int kGradStages = 4;
constexpr int kSpan = 16;  // stages (1,024 tokens)
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

    const int warp = tc::uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
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
    const uint32_t tmem = tc::uniform(*tmem_at);

    if (warp < 4) {
        Ring<2> sums;
        bool going = true;
        for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
            const int64_t r = tile / tiles_k * kM + 32 * warp + lane, g0 = tile % tiles_k * (kGradN / kGroup);
            const bool inside = r < w.R;
            float total[kGradN / kGroup] = {};
            for (int64_t c0 = 0; c0 < chunks; c0 += kSpan) {
                going = tc::barrier_wait_warp(sums_full(sums.slot), sums.parity, stop);
                if (!going)
                    break;
                tc::fence_after();
#pragma unroll
                for (int i = 0; i < kGradN / kGroup; i++) {
                    const int64_t g = g0 + i;
                    if (g >= w.K / kGroup)
                        continue;
                    const int z1 = inside ? static_cast<int>((w.qzeros[(g * w.R + r) / 8] >> (4 * (r & 7))) & 15u) + 1 : 0;
                    float part = 0.0f;
                    for (int c = 0; c < kGroup; c += 32) {
                        uint32_t word[4], v[32];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            word[j] = inside ? w.qweight[(g * kWordsPerGroup + c / 8 + j) * w.R + r] : 0u;
                        __syncwarp();
                        tc::tmem_load32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * kGradN + i * kGroup + c, v);
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            part = fmaf(__uint_as_float(v[j]),
                                        static_cast<float>(static_cast<int>((word[j / 8] >> (4 * (j % 8))) & 15u) - z1), part);
                    }
                    total[i] += part;
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::barrier_arrive(sums_empty(sums.slot));
                sums.next();
            }
#pragma unroll
            for (int i = 0; i < kGradN / kGroup; i++)
                if (going && inside && g0 + i < w.K / kGroup)
                    dscales[(g0 + i) * w.R + r] = total[i];
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
    } else {
        constexpr uint32_t kInstr = tc::instruction(D::kMagic == BF16::kMagic, true, true, kGradN);
        const uint64_t a_first = tc::descriptor(base, 8192, 1024), b_first = tc::descriptor(base + kAStage, 8192, 1024);
        Ring<kGradStages> op;
        Ring<2> sums;
        bool going = true;
        for (int64_t tile = blockIdx.x; going && tile < tiles; tile += gridDim.x) {
            for (int64_t c = 0; going && c < chunks; c++) {
                const bool first = c % kSpan == 0, last = c + 1 == chunks || (c + 1) % kSpan == 0;
                if (first)
                    going = tc::barrier_wait_warp(sums_empty(sums.slot), sums.parity ^ 1, stop);
                going = going && tc::barrier_wait_warp(full(op.slot), op.parity, stop);
                if (!going)
                    break;
                tc::fence_after();
                const uint32_t d = tmem + sums.slot * kGradN;
                const uint64_t a = a_first + static_cast<uint32_t>(op.slot * (kAStage + kGradB) / 16);
                const uint64_t b = b_first + static_cast<uint32_t>(op.slot * (kAStage + kGradB) / 16);
                if (tc::elected()) {
                    tc::mma(d, a, b, kInstr, !first);
#pragma unroll
                    for (int k = 1; k < kChunk / 16; k++)
                        tc::mma_add(d, a + k * 128, b + k * 128, kInstr);
                    tc::commit(empty(op.slot));
                    if (last)
                        tc::commit(sums_full(sums.slot));
                }
                __syncwarp();
                op.next();
                if (last)
                    sums.next();
            }
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

// Tokens per tile: the least time by a count of waves, a stage of N tokens costing 2 N cycles on the tensor
// core but never less than about 450, what the chain of waits between the warps takes.
template <class D, bool kGradient>
cq_status product(const uint16_t *act, int64_t ld, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    const int64_t m = ((kGradient ? w.K : w.R) + kM - 1) / kM, sms = sm_count();
    int64_t least = INT64_MAX;
    int best = 256;
    for (int n = 256; n >= 32; n /= 2) {
        const int64_t waves = (m * ((T + n - 1) / n) + sms - 1) / sms, cost = waves * (2 * n > 450 ? 2 * n : 450);
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

// CTAs per cluster: enough warps to keep the memory busy, at least one group for each.
template <class D, int NT>
cq_status few_rows(const uint16_t *x, int64_t ldx, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    const int64_t tiles = (w.R + kFewRows - 1) / kFewRows, groups = w.K / kGroup, sms = sm_count();
    int ranks = 1;
    while (ranks < 8 && tiles * ranks * 2 <= 4 * sms && ranks * 2 * kFewWarps <= groups)
        ranks *= 2;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(static_cast<unsigned>(tiles * ranks));
    config.blockDim = dim3(32 * kFewWarps);
    config.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    config.attrs = attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, few_rows_kernel<D, NT>, x, ldx, static_cast<int>(T), w, ep) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

template <class D>
cq_status layer(const uint16_t *x, int64_t ldx, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    if (T <= 8)
        return few_rows<D, 1>(x, ldx, T, w, ep, stream);
    if (T <= CQ_W4_EXACT_ROWS)
        return few_rows<D, 2>(x, ldx, T, w, ep, stream);
    return product<D, false>(x, ldx, T, w, ep, stream);
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
    return dtype == CQ_DTYPE_BF16 ? layer<BF16>(in, ldx, T, w, ep, s) : layer<FP16>(in, ldx, T, w, ep, s);
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
