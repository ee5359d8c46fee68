// Linear layers on 4-bit weights, and their gradients.
//
//   z = x W^T + bias, y = act(z) + residual;   W[r][i] = s[g][r] n[r][i], n = u - (zero + 1), g = i / 128
//   dx = dz W;   dscales[g][r] = sum_{i in g} n[r][i] (dz^T x)[r][i];   dz = dy act'(z), dbias = its column sums
//
// Up to 16 rows of x: few_rows_kernel, bound by the weights' bytes.  More: weights_product_kernel, on the tensor
// cores, which the input gradient shares.  The scale gradient is a product of its own whose result stays in tensor memory.
#include <cooperative_groups.h>

#include <utility>

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
    uint32_t low;              // kLow
};

// ---- tensor-core products with the weights ------------------------------------------------
//
// One kernel serves the layer and its input gradient: out[t][m] = sum_c act[t][c] Wm[m][c].
//   layer            m = output r, c = input k,  act = x
//   input gradient   m = input k,  c = output r, act = dz
// A tile is 128 values of m (the tensor core's rows) by N tokens; a stage 64 of c.  The
// weights' words travel by the stage (4 KB of codes with their scales and zero
// points), so they cross HBM and L2 at half a byte a weight.
// Sixteen warps turn them into 16-bit values, s n rounded once to the activations' type (the tensor core takes
// both operands of one type; with bf16 this doubles the square of the result's own rounding error, with fp16 less:
// many of the products fit), and store them as the tensor core's A operand: a
// word is 8 adjacent inputs of one output, 16 bytes of a 128-byte shared row [r][64 k],
// chunks swizzled by r mod 8.  The layer contracts along such rows, the input gradient
// across them, so both take the same image and differ in the operand descriptor alone.
//
// Warps: 0-3 epilogue, 4-19 unpack, then one each that copies activations, copies words, issues the matrix
// instructions, copies scales and zero points.  CTAs are persistent; two accumulators in tensor memory let
// a tile's epilogue run under the next tile's products.  Where there are too few tiles for the SMs, a cluster shares
// a tile's contraction and adds its sums up through distributed shared memory, in the order of its ranks.
// The tensor core's fp32 sums are cut off, not rounded, at each step: 16,384 terms of one sign come out 3e-5 low, a
// sixteenth of half a step of fp16, and nothing is done against it here (the scale gradient, whose results are fp32, has spans).
//
// Measured (bf16, events, one B200): 4,096 x 14,336 x 4,096 in 355 us, 1.35 PFLOP/s, 0.80 of the measured cuBLAS burst; 390 us
// the input gradient.  Run for seconds the power limit holds them at 1.36 and 1.43 GHz: 417 and 453 us, 680 and 720 cycles a stage of
// 256 tokens, where cuBLAS, of weights already unpacked, takes 395 us at 1.24 GHz (the tensor core alone needs 512 cycles; 96 KB go
// through shared memory).  64 x 30,336 x 16,384: 130 us, 2.0 TB/s, bound by issue slots (305 of 500 cycles a stage: unpacking).

constexpr int kM = 128;
constexpr int kChunk = 64;                     // contraction per stage
constexpr int kAStage = kM * kChunk * 2;
constexpr int kRawWords = 4096;                // a stage's words: 8 word rows x 128 outputs, or 16 x 64
constexpr int kRawStage = kRawWords + 512;     // and up to 128 scales (256 B) and 16 zero words (64 B)
constexpr int kUnpackSets = 4, kSetWarps = 4;   // a set fills a stage
constexpr int kUnpackWarps = kSetWarps * kUnpackSets;
constexpr int kSetWords = kM * kChunk / 8 / (32 * kSetWarps);  // words of a stage per thread
constexpr int kCopyWarp = 4 + kUnpackWarps, kWordWarp = kCopyWarp + 1, kIssueWarp = kWordWarp + 1;
constexpr int kTensorThreads = 32 * (kIssueWarp + 2);

// Slots of unpacked weights (A), of activations (B) and of raw weights, by what 227 KB of shared memory hold.  Copies
// take about 1,000 cycles from L2, a stage of few tokens under 300: their rings are the deeper, the smaller N is.
template <int N>
struct Stages {
    static constexpr int kB = N * kChunk * 2;
    static constexpr int kASlots = 4;
    static constexpr int kBSlots = N >= 256 ? 3 : N >= 128 ? 5 : N >= 64 ? 10 : 14;
    static constexpr int kRaw = N >= 256 ? 8 : N >= 128 ? 8 : 12;
    static constexpr int kBarriers = 2 * (kASlots + kBSlots + kRaw) + 4;
    static constexpr int kControl = 8 * kBarriers + 16;      // barriers, the stop flag, tensor memory's address
    static constexpr int kTurn = 4 * 16 * 33 * 4;            // the epilogue's turn from lanes to rows
    static constexpr int kBytes = kASlots * kAStage + kBSlots * kB + kRaw * kRawStage + kControl + kTurn + 1024;
    static constexpr int kColumns = 2 * N < 32 ? 32 : 2 * N;
    static_assert(kBytes <= 232448, "shared memory");
    // A slot of raw weights belongs to one set, as a slot of A does: loads complete in any order, so only the set that
    // has read a slot before knows which of its phases the next wait is for.
    static_assert(kRaw % kUnpackSets == 0, "phases");
};

// Eight codes of a word as 16-bit values s (u - z - 1), in order, each rounded once.
template <class D>
struct Unpack;

// n = u - z - 1 of the word's eight codes: pairs of adjacent inputs.
template <class D>
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t zero, uint32_t low, uint32_t (&n)[4])
{
    const uint32_t high = w >> 4;  // byte j of w starts with code 2j, byte j of this with code 2j + 1
#pragma unroll
    for (int j = 0; j < 4; j++)
        n[j] = D::sub((__byte_perm(w, high, j | (4 + j) << 8) & low) | D::kMagic, zero);
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
    __device__ __forceinline__ uint4 operator()(uint32_t w, uint32_t low) const
    {
        uint32_t n[4];
        unpack_codes<FP16>(w, zero, low, n);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const __half2 p = __hmul2(reinterpret_cast<const __half2 &>(n[j]), s);
            n[j] = reinterpret_cast<const uint32_t &>(p);
        }
        return make_uint4(n[0], n[1], n[2], n[3]);
    }
};

// bf16: s = hi + lo, hi the scale rounded to 8 bits and lo the at most 3 bits left, so
// n lo is exact and fma(n, hi, n lo) rounds n s once.  An infinite scale is hi alone: inf - inf leaves no rest.
template <>
struct Unpack<BF16> {
    uint32_t zero;
    __nv_bfloat162 hi, lo;
    __device__ __forceinline__ Unpack(uint16_t scale, uint32_t nibble) : zero(zero_pair<BF16>(nibble))
    {
        const float s = half_bits(scale);
        const __nv_bfloat16 h = __float2bfloat16_rn(s);
        hi = __bfloat162bfloat162(h);
        lo = __bfloat162bfloat162(__float2bfloat16_rn((scale & 0x7C00u) == 0x7C00u ? 0.0f : s - __bfloat162float(h)));
    }
    __device__ __forceinline__ uint4 operator()(uint32_t w, uint32_t low) const
    {
        uint32_t n[4];
        unpack_codes<BF16>(w, zero, low, n);
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

// z of eight adjacent m of one token -> pre, y.
template <class D, bool kGradient>
__device__ __forceinline__ void finish_row(const Epilogue &ep, int64_t t, int64_t m, float (&z)[8], const uint4 &res)
{
    if (!kGradient) {
        if (ep.pre)
            *reinterpret_cast<uint4 *>(ep.pre + t * ep.ldpre + m) = narrow<D>(z);
        activate(z, ep.act);
        if (ep.res) {
            float r[8];
            widen<D>(res, r);
#pragma unroll
            for (int j = 0; j < 8; j++)
                z[j] += r[j];
        }
    }
    *reinterpret_cast<uint4 *>(ep.y + t * ep.ldy + m) = narrow<D>(z);
}

template <class D, int N, bool kGradient>
__global__ void __launch_bounds__(kTensorThreads, 1)
    weights_product_kernel(const __grid_constant__ CUtensorMap act_map, const __grid_constant__ CUtensorMap word_map,
                           Layer w, int64_t T, Epilogue ep)
{
    using S = Stages<N>;
    extern __shared__ char shared_raw[];
    const uint32_t base = (tc::smem_address(shared_raw) + 1023) & ~1023u;
    char *shared = shared_raw + (base - tc::smem_address(shared_raw));
    const uint32_t b0 = base + S::kASlots * kAStage, raw0 = b0 + S::kBSlots * S::kB, bars = raw0 + S::kRaw * kRawStage;
    auto a_full = [&](int i) { return bars + 8 * i; };
    auto a_empty = [&](int i) { return bars + 8 * (S::kASlots + i); };
    auto b_full = [&](int i) { return bars + 8 * (2 * S::kASlots + i); };
    auto b_empty = [&](int i) { return bars + 8 * (2 * S::kASlots + S::kBSlots + i); };
    auto raw_full = [&](int i) { return bars + 8 * (2 * (S::kASlots + S::kBSlots) + i); };
    auto raw_empty = [&](int i) { return bars + 8 * (2 * (S::kASlots + S::kBSlots) + S::kRaw + i); };
    auto sums_full = [&](int i) { return bars + 8 * (2 * (S::kASlots + S::kBSlots + S::kRaw) + i); };
    auto sums_empty = [&](int i) { return bars + 8 * (2 * (S::kASlots + S::kBSlots + S::kRaw) + 2 + i); };
    volatile int *stop = reinterpret_cast<volatile int *>(shared + (bars - base) + 8 * S::kBarriers);
    uint32_t *tmem_at = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(stop + 1));

    const int warp = tc::uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    // a cluster shares the tile's contraction: this CTA has `depth` steps of 128 of it, from `first`
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t rows = kGradient ? w.K : w.R, steps = kGradient ? (w.R + kM - 1) / kM : w.K / kM;
    const int first = static_cast<int>(steps * rank / ranks), depth = static_cast<int>(steps * (rank + 1) / ranks) - first;
    const int64_t tiles_n = (T + N - 1) / N, tiles = (rows + kM - 1) / kM * tiles_n;
    const int64_t tile0 = blockIdx.x / ranks, tile_step = gridDim.x / ranks;

    if (warp == kIssueWarp)
        tc::tmem_alloc(tc::smem_address(tmem_at), S::kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kASlots; i++) {
            tc::barrier_init(a_full(i), kSetWarps);
            tc::barrier_init(a_empty(i), 1);
        }
        for (int i = 0; i < S::kBSlots; i++) {
            tc::barrier_init(b_full(i), 1);
            tc::barrier_init(b_empty(i), 1);
        }
        for (int i = 0; i < S::kRaw; i++) {
            tc::barrier_init(raw_full(i), 32 + 1);
            tc::barrier_init(raw_empty(i), kSetWarps);
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
    if (kGradient)
        let_next_begin();  // the scale gradient's CTAs, as soon as SMs fall idle

    if (warp < 4) {
        // Epilogue, a warp's 32 m by 16 tokens at a time: a thread has one m in tensor memory;
        // through 2 KB of shared memory it gets 8 adjacent m of one token, 16 bytes of every row it touches.
        float *turn = reinterpret_cast<float *>(shared + (bars - base) + S::kControl) + warp * (16 * 33);
        Ring<2> sums;
        const int tok = lane >> 2, part = 8 * (lane & 3);
        for (int64_t tile = tile0; tile < tiles; tile += tile_step) {
            const int64_t m0 = tile / tiles_n * kM + 32 * warp, t0 = tile % tiles_n * N, m = m0 + part;
            const float bias = ep.bias && m0 + lane < rows ? D::to_float(ep.bias[m0 + lane]) : 0.0f;
            const int64_t left = T - t0;
            const int tokens = left < N ? static_cast<int>(left) : N;
            if (!tc::barrier_wait_warp(sums_full(sums.slot), sums.parity, stop))
                break;
            tc::fence_after();
            if (ranks > 1) {  // the sums go to shared memory, [token][m], for the cluster
                float *to = reinterpret_cast<float *>(shared) + 32 * warp + lane;
                for (int c = 0; c < tokens; c += 16) {
                    uint32_t v[16];
                    tc::tmem_load16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * N + c, v);
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        to[(c + j) * kM] = __uint_as_float(v[j]);
                }
                break;
            }
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
                    finish_row<D, kGradient>(ep, t, m, z, res[h]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::barrier_arrive(sums_empty(sums.slot));
            sums.next();
        }
    } else if (warp < 4 + kUnpackWarps) {  // unpack
        // Sets of warps take the stages in turn, each with its slot of A: a word row of eight a thread.
        static_assert(kSetWords == 8 && kUnpackSets == S::kASlots, "a set fills the same slot each time");
        const int i = threadIdx.x % (32 * kSetWarps), set = (warp - 4) / kSetWarps;
        constexpr int kOutputs = kGradient ? 64 : kM;       // outputs of a stage
        const int r = i % kOutputs, k8 = i / kOutputs * kSetWords;  // output and first word row within it
        const uint32_t to = (base + set * kAStage + (k8 >> 3) * (kAStage / 2) + r * 128) | (r & 7) << 4;  // chunk j lies at ^ j << 4
        const uint32_t full = a_full(set), empty = a_empty(set);
        const int zero_shift = 4 * (r & 7);
        uint32_t parity = 1, raw_parity = 0;
        int raw = set;
        int64_t left = ((tile0 < tiles ? (tiles - 1 - tile0) / tile_step + 1 : 0) * 2 * depth - set + kUnpackSets - 1) / kUnpackSets;
        for (; left > 0; left--) {
            if (!tc::barrier_wait_warp(raw_full(raw), raw_parity, stop))
                break;
            const char *slot = shared + (raw0 - base) + raw * kRawStage;
            const uint32_t *words = reinterpret_cast<const uint32_t *>(slot) + k8 * kOutputs + r;
            uint32_t word[kSetWords];
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                word[j] = words[j * kOutputs];
            const Unpack<D> unpack(reinterpret_cast<const uint16_t *>(slot + kRawWords)[r],
                                   (reinterpret_cast<const uint32_t *>(slot + kRawWords + 256)[r >> 3] >> zero_shift) & 15u);
            uint4 values[kSetWords];
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                values[j] = unpack(word[j], w.low);
            if (!tc::barrier_wait_warp(empty, parity, stop))
                break;
#pragma unroll
            for (int j = 0; j < kSetWords; j++)
                tc::store_shared(to ^ j << 4, values[j]);
            tc::fence_shared_writes();
            __syncwarp();
            // The words are released only here, after stores that needed them: an arrival does not wait for
            // shared loads in flight, and with shared memory busy the next words overtook them.
            if (lane == 0) {
                tc::barrier_arrive(raw_empty(raw));
                tc::barrier_arrive(full);
            }
            parity ^= 1;
            raw += kUnpackSets;
            if (raw >= S::kRaw) {
                raw -= S::kRaw;
                raw_parity ^= 1;
            }
        }
    } else if (warp == kCopyWarp) {  // activations, by tensor map
        Ring<S::kBSlots> op;
        bool going = true;
        for (int64_t tile = tile0; going && tile < tiles; tile += tile_step) {
            const int t0 = static_cast<int>(tile % tiles_n * N), end = (first + depth) * kM;
            for (int c = first * kM; c < end; c += kChunk) {
                going = tc::barrier_wait_warp(b_empty(op.slot), op.parity ^ 1, stop);
                if (!going)
                    break;
                if (tc::elected()) {
                    tc::barrier_expect(b_full(op.slot), S::kB);
                    tc::copy_box(b0 + op.slot * S::kB, &act_map, c, t0, b_full(op.slot));
                }
                __syncwarp();
                op.next();
            }
        }
    } else if (warp == kWordWarp) {  // words, by tensor map
        Ring<S::kRaw> raw;
        bool going = true;
        for (int64_t tile = tile0; going && tile < tiles; tile += tile_step) {
            const int m0 = static_cast<int>(tile / tiles_n * kM);
            int r = kGradient ? first * kM : m0, row = kGradient ? m0 / 8 : first * kWordsPerGroup;
            for (int c = 0; c < 2 * depth; c++) {
                going = tc::barrier_wait_warp(raw_empty(raw.slot), raw.parity ^ 1, stop);
                if (!going)
                    break;
                if (tc::elected()) {
                    tc::barrier_expect(raw_full(raw.slot), kRawWords);
                    tc::copy_box(raw0 + raw.slot * kRawStage, &word_map, r, row, raw_full(raw.slot));
                }
                __syncwarp();
                r += kGradient ? kChunk : 0;
                row += kGradient ? 0 : kChunk / 8;
                raw.next();
            }
        }
    } else if (warp == kIssueWarp) {  // matrix instructions: the loop is the whole warp's, so that what it computes stays uniform
        constexpr uint32_t kInstr = tc::instruction(D::kMagic == BF16::kMagic, kGradient, false, N);
        constexpr uint32_t kStep = kGradient ? 2048 : 32;  // 16 of the contraction in A: 16 rows, or 32 bytes of a row
        const uint64_t a_first = tc::descriptor(base, kGradient ? kAStage / 2 : 16, 1024);
        const uint64_t b_first = tc::descriptor(b0, 16, 1024);
        const bool leader = tc::elected();
        Ring<S::kASlots> a_ring;
        Ring<S::kBSlots> b_ring;
        Ring<2> sums;
        bool going = true;
        for (int64_t tile = tile0; going && tile < tiles; tile += tile_step) {
            going = tc::barrier_wait_warp(sums_empty(sums.slot), sums.parity ^ 1, stop);
            const uint32_t d = tmem + sums.slot * N;
            for (int c = 0; going && c < 2 * depth; c++) {
                going = tc::barrier_wait_both(b_full(b_ring.slot), b_ring.parity, a_full(a_ring.slot), a_ring.parity, stop);
                if (!going)
                    break;
                tc::fence_after();
                const uint64_t a = a_first + static_cast<uint32_t>(a_ring.slot * (kAStage / 16));
                const uint64_t b = b_first + static_cast<uint32_t>(b_ring.slot * (S::kB / 16));
#pragma unroll
                for (int k = 0; k < kChunk / 16; k++)
                    tc::mma(d, a + k * (kStep / 16), b + k * (32 / 16), kInstr, c > 0 || k > 0, leader);
                tc::commit(a_empty(a_ring.slot), leader);
                tc::commit(b_empty(b_ring.slot), leader);
                a_ring.next();
                b_ring.next();
            }
            if (going)
                tc::commit(sums_full(sums.slot), leader);
            sums.next();
        }
    } else {  // half the lanes 16 bytes (8 outputs) of scales, half a word of zero points
        Ring<S::kRaw> raw;
        const int l = lane & 15;
        const uint32_t to = raw0 + kRawWords + (lane < 16 ? 16 * l : 256 + 4 * l);
        const bool mine = !kGradient || l < 8;
        const int64_t group_step = lane < 16 ? 2 * w.R : w.R / 2;
        bool going = true;
        for (int64_t tile = tile0; going && tile < tiles; tile += tile_step) {
            const int64_t m0 = tile / tiles_n * kM;
            int64_t r = (kGradient ? static_cast<int64_t>(first) * kM : m0) + 8 * l;
            const int64_t group = kGradient ? m0 / kGroup : first;
            const char *from = lane < 16 ? reinterpret_cast<const char *>(w.scales + group * w.R + r)
                                         : reinterpret_cast<const char *>(w.qzeros + (group * w.R + r) / 8);
            for (int c = 0; c < 2 * depth; c++) {
                going = tc::barrier_wait_warp(raw_empty(raw.slot), raw.parity ^ 1, stop);
                if (!going)
                    break;
                if (mine) {
                    const bool inside = r < w.R;
                    const char *p = inside ? from : reinterpret_cast<const char *>(w.scales);
                    if (lane < 16)
                        tc::copy_async<16>(to + raw.slot * kRawStage, p, inside);
                    else
                        tc::copy_async<4>(to + raw.slot * kRawStage, p, inside);
                }
                tc::copy_async_arrive(raw_full(raw.slot));
                if (kGradient) {
                    r += kChunk;
                    from += lane < 16 ? kChunk * 2 : kChunk / 2;
                } else if (c & 1) {
                    from += group_step;
                }
                raw.next();
            }
        }
        tc::copy_async_wait();
    }
    __syncthreads();
    tc::report(stop);
    if (warp == kIssueWarp)
        tc::tmem_free(tmem, S::kColumns);
    if (ranks == 1)
        return;
    // the cluster's sums, each CTA a part of the tile's rows, in the order of the ranks
    cluster.sync();
    const int64_t m0 = tile0 / tiles_n * kM, t0 = tile0 % tiles_n * N, left = T - t0;
    const int items = (left < N ? static_cast<int>(left) : N) * (kM / 8);
    for (int i = rank * kTensorThreads + threadIdx.x; i < items; i += ranks * kTensorThreads) {
        const int64_t t = t0 + i / (kM / 8), m = m0 + i % (kM / 8) * 8;
        if (m >= rows)
            continue;
        float z[8] = {};
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (k < ranks) {
                const float4 *from = reinterpret_cast<const float4 *>(cluster.map_shared_rank(reinterpret_cast<float *>(shared), k)) + 2 * i;
                const float4 a = from[0], b = from[1];
                z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
                z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
            }
        if (!kGradient && ep.bias) {
            float b[8];
            widen<D>(*reinterpret_cast<const uint4 *>(ep.bias + m), b);
#pragma unroll
            for (int j = 0; j < 8; j++)
                z[j] += b[j];
        }
        uint4 res = make_uint4(0, 0, 0, 0);
        if (!kGradient && ep.res)
            res = *reinterpret_cast<const uint4 *>(ep.res + t * ep.ldres + m);
        finish_row<D, kGradient>(ep, t, m, z, res);
    }
    cluster.sync();  // peers keep their shared memory until it has been read
}

// ---- few rows ----------------------------------------------------------------------------------
//
// Up to 16 rows the weights' bytes are the work.  A CTA has 128 outputs and a part of the groups (a
// cluster has them all); two warps keep a ring of groups in flight (words by tensor map; scales, zero
// points and the tokens' 128 inputs by asynchronous copies), eight warps in four sets take them in turn,
// 64 outputs a warp.  A thread reads 4 adjacent outputs' words at once; a word is 8 inputs, whose pairs
// (q, q + 4) come out of it with a shift and a mask.  That order of the inputs is as good as any for the
// m16n8k16 product if the activations' pairs are the same.  The codes enter as integers, zero point
// taken off (with bf16 times 2^-11, made good at the end), and each group's fp32 sum is scaled after, so the weights are exact.  The sets' and the
// cluster's sums meet in shared memory in a fixed order.
//
// Measured: 30,336 x 16,384 in 68 us for 1 to 8 rows (3.8 TB/s, 0.59 of HBM), 93 us for 13 (fp16); 14,336 x 4,096 in 12.4 us.
// The copies alone take 42 us.  A word costs 16 instructions (3 shifts, 4 logical operations, 4 subtractions, its share of the
// products), which keep the ALU pipe 43% and the matrix pipe 38% busy at 13 rows; and 237 tiles on 148 SMs leave
// 20% of them idle at the end (splitting each over 2, 4 or 8 CTAs costs as much in starting them: 71, 70, 88 us).

constexpr int kFewSets = 4;
constexpr int kFewWords = 8192;                // 16 word rows x 128 outputs
constexpr int kFewThreads = 32 * (2 * kFewSets + 2);
constexpr int kFewX = kFewWords + 320;       // a stage: words, 256 B of scales, 64 B of zero points, inputs
constexpr int kFewXRow = 272;                // a token's 128 inputs; 16 bytes more keep two rows' reads off each other's banks

template <int NT>
struct FewStages {
    static constexpr int kStage = (kFewX + 8 * NT * kFewXRow + 1023) / 1024 * 1024;
    static constexpr int kStages = 8;
    static constexpr int kBytes = kStages * kStage + 16 * kStages + 16 + 1024;
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
    static_assert((kFewSets + 1) * 8 * NT * kM * 4 <= kStages * kStage, "sums reuse the ring");
    // A stage belongs to one set: loads complete in any order, so only the set that has read a stage before
    // knows which of its phases the next wait is for.
    static_assert(kStages % kFewSets == 0, "phases");
};

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

template <class D, int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
    few_rows_kernel(const __grid_constant__ CUtensorMap word_map, const uint16_t *__restrict__ x, int64_t ldx, int T, Layer w,
                    Epilogue ep)
{
    using S = FewStages<NT>;
    extern __shared__ char shared_raw[];
    const uint32_t base = (tc::smem_address(shared_raw) + 1023) & ~1023u;
    char *shared = shared_raw + (base - tc::smem_address(shared_raw));
    const uint32_t bars = base + S::kStages * S::kStage;
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 8 * (S::kStages + i); };
    volatile int *stop = reinterpret_cast<volatile int *>(shared + (bars - base) + 16 * S::kStages);

    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int warp = tc::uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / ranks) * kM;
    const int groups = static_cast<int>(w.K / kGroup);
    const int first = static_cast<int>(static_cast<int64_t>(groups) * rank / ranks);
    const int count = static_cast<int>(static_cast<int64_t>(groups) * (rank + 1) / ranks) - first;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; i++) {
            tc::barrier_init(full(i), 32 + 1);
            tc::barrier_init(empty(i), 2);
        }
        *stop = 0;
        tc::barrier_init_fence();
    }
    for (int i = threadIdx.x; i < S::kStages * (8 * NT - T) * 16; i += kFewThreads) {  // rows of no token: zeros, never written again
        const int stage = i / ((8 * NT - T) * 16), row = T + i / 16 % (8 * NT - T);
        *reinterpret_cast<uint4 *>(shared + stage * S::kStage + kFewX + row * kFewXRow + i % 16 * 16) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();

    float total[4][NT][4] = {};
    const int half = warp & 1, quad = lane >> 2, c = lane & 3;
    if (warp == 2 * kFewSets) {  // words
        Ring<S::kStages> ring;
        int row = first * kWordsPerGroup;
        for (int i = 0; i < count; i++) {
            if (!tc::barrier_wait_warp(empty(ring.slot), ring.parity ^ 1, stop))
                break;
            if (tc::elected()) {
                tc::barrier_expect(full(ring.slot), kFewWords);
#pragma unroll
                for (int b = 0; b < 4; b++)  // 32 outputs x 16 word rows, swizzled
                    tc::copy_box(base + ring.slot * S::kStage + 2048 * b, &word_map, static_cast<int>(r0) + 32 * b, row, full(ring.slot));
            }
            __syncwarp();
            row += kWordsPerGroup;
            ring.next();
        }
    } else if (warp == 2 * kFewSets + 1) {  // the rest: half the lanes 16 bytes of scales, half a word of zero points; inputs by all
        Ring<S::kStages> ring;
        const int l = lane & 15;
        const bool inside = r0 + 8 * l < w.R;
        const int64_t at = static_cast<int64_t>(first) * w.R + (inside ? r0 + 8 * l : 0);
        const char *from = lane < 16 ? reinterpret_cast<const char *>(w.scales + at) : reinterpret_cast<const char *>(w.qzeros + at / 8);
        const int64_t step = lane < 16 ? 2 * w.R : w.R / 2;
        const uint32_t to = kFewWords + (lane < 16 ? 16 * l : 256 + 4 * l);
        const char *in = reinterpret_cast<const char *>(x + (lane >> 4) * ldx + static_cast<int64_t>(first) * kGroup + 8 * l);
        const int64_t rows = 4 * ldx;
        for (int i = 0; i < count; i++) {
            if (!tc::barrier_wait_warp(empty(ring.slot), ring.parity ^ 1, stop))
                break;
            const uint32_t stage = base + ring.slot * S::kStage;
            if (lane < 16)
                tc::copy_async<16>(stage + to, from, inside);
            else
                tc::copy_async<4>(stage + to, from, inside);
            const char *p = in;
#pragma unroll
            for (int n = 0; n < 4 * NT; n++) {
                if (2 * n + (lane >> 4) < T)
                    tc::copy_async<16>(stage + kFewX + (2 * n + (lane >> 4)) * kFewXRow + 16 * l, p, true);
                p += rows;
            }
            tc::copy_async_arrive(full(ring.slot));
            if (inside)
                from += step;
            in += 2 * kGroup;
            ring.next();
        }
        tc::copy_async_wait();
    } else {
        int slot = warp / 2;
        uint32_t parity = 0;
        for (int i = warp / 2; i < count; i += kFewSets) {
            if (!tc::barrier_wait_warp(full(slot), parity, stop))
                break;
            const char *at = shared + slot * S::kStage;
            float acc[4][NT][4] = {};
            uint32_t zero[2][4];
#pragma unroll
            for (int m = 0; m < 2; m++) {
                const uint32_t z = reinterpret_cast<const uint32_t *>(at + kFewWords + 256)[8 * half + 4 * m + quad / 2] >> (16 * (quad & 1));
#pragma unroll
                for (int k = 0; k < 4; k++)
                    zero[m][k] = code_zero_pair<D>((z >> (4 * k)) & 15u);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int k8 = 8 * (j >> 1) + 2 * c + (j & 1);  // this order of word rows keeps a warp's reads on all banks
                uint32_t b[NT][4];
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(at + kFewX + (8 * n + quad) * kFewXRow + 16 * k8);
                    b[n][0] = __byte_perm(v.x, v.z, 0x5410);
                    b[n][1] = __byte_perm(v.x, v.z, 0x7632);
                    b[n][2] = __byte_perm(v.y, v.w, 0x5410);
                    b[n][3] = __byte_perm(v.y, v.w, 0x7632);
                }
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(at + 2048 * (2 * half + m) + 128 * k8 + 16 * (quad ^ (k8 & 7)));
                    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
                    uint32_t pair[4][4];  // [output][q]: inputs q and q + 4
#pragma unroll
                    for (int k = 0; k < 4; k++)
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            pair[k][q] = D::code_pair(word[k], q, zero[m][k], w.low);
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int p = 0; p < 2; p++)
#pragma unroll
                            for (int q = 0; q < 2; q++) {
                                const uint32_t a[4] = {pair[2 * p][2 * q], pair[2 * p + 1][2 * q], pair[2 * p][2 * q + 1],
                                                       pair[2 * p + 1][2 * q + 1]};
                                mma_16x8x16<D>(acc[2 * m + p][n], a, b[n][2 * q], b[n][2 * q + 1]);
                            }
                }
            }
#pragma unroll
            for (int m = 0; m < 2; m++) {
                const uint2 v = *reinterpret_cast<const uint2 *>(at + kFewWords + 2 * (64 * half + 32 * m + 4 * quad));
                const float s[4] = {half_bits(static_cast<uint16_t>(v.x)), half_bits(static_cast<uint16_t>(v.x >> 16)),
                                    half_bits(static_cast<uint16_t>(v.y)), half_bits(static_cast<uint16_t>(v.y >> 16))};
#pragma unroll
                for (int p = 0; p < 2; p++)
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            total[2 * m + p][n][k] = fmaf(s[2 * p + (k >> 1)], acc[2 * m + p][n][k], total[2 * m + p][n][k]);
            }
            __syncwarp();
            // The arrival's address hangs on sums that hang on every shared load above (w.low is kLow): on its own
            // it would not wait for loads in flight.
            const uint32_t loaded = (__float_as_uint(total[0][0][0]) ^ __float_as_uint(total[2][NT - 1][0])) & (w.low ^ kLow);
            if (lane == 0)
                tc::barrier_arrive(empty(slot) + loaded);
            slot += kFewSets;
            if (slot >= S::kStages) {
                slot -= S::kStages;
                parity ^= 1;
            }
        }
    }
    __syncthreads();  // every copy has landed and been read: the ring becomes the sets' sums
    tc::report(stop);
    float *sums = reinterpret_cast<float *>(shared), *cta_sums = sums + kFewSets * 8 * NT * kM;
    if (warp < 2 * kFewSets) {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int row = 64 * half + 32 * (i >> 1) + 4 * quad + 2 * (i & 1) + (k >> 1), t = 8 * n + 2 * c + (k & 1);
                    sums[((warp / 2) * 8 * NT + t) * kM + row] = total[i][n][k];
                }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < T * kM; e += kFewThreads) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kFewSets; i++)
            s += sums[i * 8 * NT * kM + e];
        cta_sums[e] = s;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    for (int e = rank * kFewThreads + threadIdx.x; e < T * kM; e += ranks * kFewThreads) {
        const int t = e / kM;
        const int64_t r = r0 + e % kM;
        float parts[8];
#pragma unroll
        for (int k = 0; k < 8; k++)  // all on their way at once
            parts[k] = k < ranks ? (ranks > 1 ? cluster.map_shared_rank(cta_sums, k)[e] : cta_sums[e]) : 0.0f;
        float z[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < 8; k++)
            z[0] += parts[k];
        if (r >= w.R)
            continue;
        z[0] *= D::kCodeUnit;
        z[0] += ep.bias ? D::to_float(ep.bias[r]) : 0.0f;
        if (ep.pre)
            ep.pre[t * ep.ldpre + r] = D::from_float(z[0]);
        activate(z, ep.act);
        if (ep.res)
            z[0] += D::to_float(ep.res[t * ep.ldres + r]);
        ep.y[t * ep.ldy + r] = D::from_float(z[0]);
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
// kSpan bounds the drift: every span of 512 tokens has sums of its own, which the epilogue adds up (against 64 bits
// 5e-7 off at 4,096 tokens; 1.1e-6 with spans of 1,024).  Measured: 4,096 x 14,336 x 4,096 in 383 us, 1.26 PFLOP/s, for seconds
// 452 at 1.56 GHz.  Two accumulators, persistent CTAs; warps 0-3 epilogue, 4 copies, 5 issues.

constexpr int kGradN = 256;
constexpr int kGradB = kGradN * kChunk * 2;
constexpr int kGradStages = 4;
constexpr int kSpan = 8;  // stages (512 tokens)
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
                    const uint32_t zero = code_zero_pair<FP16>(inside ? (w.qzeros[(g * w.R + r) / 8] >> (4 * (r & 7))) & 15u : 0u);
                    float part = 0.0f;
                    for (int c = 0; c < kGroup; c += 32) {
                        uint32_t word[4], v[32];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            word[j] = inside ? w.qweight[(g * kWordsPerGroup + c / 8 + j) * w.R + r] : 0u;
                        __syncwarp();
                        tc::tmem_load32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + sums.slot * kGradN + i * kGroup + c, v);
#pragma unroll
                        for (int j = 0; j < 4; j++)
#pragma unroll
                            for (int q = 0; q < 4; q++) {
                                const uint32_t n = FP16::code_pair(word[j], q, zero, w.low);
                                const float2 f = __half22float2(reinterpret_cast<const __half2 &>(n));
                                part = fmaf(__uint_as_float(v[8 * j + q]), f.x, part);
                                part = fmaf(__uint_as_float(v[8 * j + q + 4]), f.y, part);
                            }
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
        const bool leader = tc::elected();
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
#pragma unroll
                for (int k = 0; k < kChunk / 16; k++)
                    tc::mma(d, a + k * 128, b + k * 128, kInstr, !first || k > 0, leader);
                tc::commit(empty(op.slot), leader);
                op.next();
                if (last) {
                    tc::commit(sums_full(sums.slot), leader);
                    sums.next();
                }
            }
        }
    }
    __syncthreads();
    tc::report(stop);
    if (warp == 5)
        tc::tmem_free(tmem, 2 * kGradN);
    wait_for_previous();  // the input gradient before it: the two share inputs only
}

// dz = dy act'(pre) and its column sums.  A cluster of 8 CTAs owns 64 columns; its
// 256 row slots take every 256th row, a thread 8 adjacent columns (16-byte accesses).  A thread's operands come through
// its own places in shared memory, kActAhead rows ahead: bytes in flight are what the rate hangs on, and in registers two rows
// at a time cost more warps than they bring (86 us; one at a time 76; 71, 65, 64 with 2, 3, 4 ahead).  The sums meet
// in shared memory and through distributed shared memory, in a fixed order.
// Bound by HBM: 6 bytes per element, 5.5 TB/s (0.86 of the copy's rate) at 4,096 x 14,336 silu and relu (64 us); by issue slots,
// 85% of them used, gelu (80 us, 4.4 TB/s) and its tanh form (69 to 72 us).
constexpr int kActCluster = 8;
constexpr int kActThreads = 256;
constexpr int kActColumns = 64;    // pieces of 128 bytes of a row (256 bytes: silu 62 us for 64, gelu 83 for 79)
constexpr int kActAhead = 4;

template <class D>
__global__ void __cluster_dims__(kActCluster, 1, 1) __launch_bounds__(kActThreads)
    activation_backward_kernel(const uint16_t *dy, int64_t lddy, const uint16_t *pre, int64_t ldpre, int64_t T, int64_t R,
                               int act, uint16_t *dz, int64_t lddz, float *dbias)
{
    constexpr int kLanes = kActColumns / 8, kSlots = kActThreads / kLanes;
    __shared__ float part[kSlots][kActColumns];
    __shared__ float cta_sum[kActColumns];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int64_t col0 = static_cast<int64_t>(blockIdx.x / kActCluster) * kActColumns;
    const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
    const int64_t col = col0 + 8 * lane;
    __shared__ uint4 ring[kActAhead][2][kActThreads];
    float acc[8] = {};
    if (col < R) {
        constexpr int kStep = kActCluster * kSlots;
        auto fetch = [&](int64_t t, int i) {
            if (t < T) {
                tc::copy_async<16>(tc::smem_address(&ring[i][0][threadIdx.x]), dy + t * lddy + col, true);
                tc::copy_async<16>(tc::smem_address(&ring[i][1][threadIdx.x]), pre + t * ldpre + col, true);
            }
            tc::copy_async_commit();
        };
        const int64_t first = rank * kSlots + slot;
#pragma unroll
        for (int i = 0; i < kActAhead; i++)
            fetch(first + i * kStep, i);
        int at = 0;
        for (int64_t t = first; t < T; t += kStep) {
            float d[8], z[8];
            tc::copy_async_wait_but<kActAhead - 1>();
            widen<D>(ring[at][0][threadIdx.x], d);
            widen<D>(ring[at][1][threadIdx.x], z);
            slopes(z, act);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                z[j] *= d[j];
                acc[j] += z[j];
            }
            *reinterpret_cast<uint4 *>(dz + t * lddz + col) = narrow<D>(z);
            fetch(t + kActAhead * kStep, at);  // behind the store, which hangs on what the slot held
            at = at + 1 < kActAhead ? at + 1 : 0;
        }
        tc::copy_async_wait();
    }
    if (!dbias)
        return;  // the whole cluster
#pragma unroll
    for (int j = 0; j < 8; j++)
        part[slot][8 * lane + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < kActColumns) {
        float s = 0.0f;
#pragma unroll 8
        for (int i = 0; i < kSlots; i++)
            s += part[i][threadIdx.x];
        cta_sum[threadIdx.x] = s;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x < kActColumns && col0 + threadIdx.x < R) {
        float s = 0.0f;
#pragma unroll
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
    if (T >= kMost || R > kMost - kM || K >= kMost)  // the last tile of outputs ends in 31 bits too
        return CQ_ERR_UNSUPPORTED;
    if (R > 0 && (!qweight || !qzeros || !scales || !is_aligned(qweight, 16) || !is_aligned(qzeros, 4) ||
                  !is_aligned(scales, 16)))
        return CQ_ERR_INVALID_ARG;
    return CQ_OK;
}

template <class D>
CUtensorMapDataType map_type()
{
    return D::kMagic == BF16::kMagic ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

template <class... P, class... A>
cq_status launch_clusters(void (*kernel)(P...), int64_t ctas, int ranks, int threads, int bytes, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(static_cast<unsigned>(ctas));
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    config.attrs = attr;
    config.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, std::forward<A>(args)...) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

template <class D, int N, bool kGradient>
cq_status run_product(const uint16_t *act, int64_t ld, int64_t T, const Layer &w, const Epilogue &ep, int ranks, cudaStream_t stream)
{
    CUtensorMap act_map, word_map;
    const int64_t rows = kGradient ? w.K : w.R;
    if (!tc::make_map(&act_map, map_type<D>(), 2, act, T, kGradient ? w.R : w.K, ld, N, kChunk, true) ||
        !tc::make_map(&word_map, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, w.qweight, w.K / 8, w.R, w.R, kGradient ? kWordsPerGroup : kChunk / 8,
                      kGradient ? kChunk : kM, false))
        return CQ_ERR_CUDA;
    constexpr auto kernel = weights_product_kernel<D, N, kGradient>;
    if (allow_shared<kernel>(Stages<N>::kBytes) != cudaSuccess)
        return CQ_ERR_CUDA;
    const int64_t tiles = (rows + kM - 1) / kM * ((T + N - 1) / N), sms = sm_count();
    return launch_clusters(kernel, ranks > 1 ? tiles * ranks : tiles < sms ? tiles : sms, ranks, kTensorThreads, Stages<N>::kBytes,
                           stream, act_map, word_map, w, T, ep);
}

// Tokens per tile and CTAs per tile: the least time by a count of waves.  A stage of N tokens counts 2 N cycles, what the
// tensor core takes, but never less than about 400, what the chain of waits between the warps takes; a call about 3,000 more to start
// and to end, a cluster's sums 2,000 and a few for each token.  It ranks the choices and is no forecast: a stage of 256 tokens
// measures 680 to 820 cycles, and the results of a CTA's only tile, which nothing hides, are not in it (333 x 4,104 x 1,152:
// 10,200 cycles by the rule, 14.5 us measured).  17 x 4,096 x 4,096 took 14.5 us in clusters of 4 where it took 22.5 without.
template <class D, bool kGradient>
cq_status product(const uint16_t *act, int64_t ld, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    const int64_t m = ((kGradient ? w.K : w.R) + kM - 1) / kM, steps = kGradient ? (w.R + kM - 1) / kM : w.K / kM, sms = sm_count();
    int64_t least = INT64_MAX;
    int best = 256, ranks = 1;
    for (int n = 256; n >= 32; n /= 2)
        for (int r = 1; r <= 8 && r <= steps; r *= 2) {
            const int64_t tiles = m * ((T + n - 1) / n);
            if (r > 1 && tiles * r > sms)
                break;
            const int64_t waves = (tiles * r + sms - 1) / sms, stage = 2 * n > 400 ? 2 * n : 400;
            const int64_t cost = waves * 2 * ((steps + r - 1) / r) * stage + 3000 + (r > 1 ? 2000 + 8 * n : 0);
            if (cost <= least) {  // of equals the smallest tile
                least = cost;
                best = n;
                ranks = r;
            }
        }
    return best == 256   ? run_product<D, 256, kGradient>(act, ld, T, w, ep, ranks, stream)
           : best == 128 ? run_product<D, 128, kGradient>(act, ld, T, w, ep, ranks, stream)
           : best == 64  ? run_product<D, 64, kGradient>(act, ld, T, w, ep, ranks, stream)
                         : run_product<D, 32, kGradient>(act, ld, T, w, ep, ranks, stream);
}

// CTAs per cluster: the least number of groups in a row on an SM, a CTA costing about eight groups more
// to start and to end.
template <class D, int NT>
cq_status few_rows(const uint16_t *x, int64_t ldx, int64_t T, const Layer &w, const Epilogue &ep, cudaStream_t stream)
{
    const int64_t tiles = (w.R + kM - 1) / kM, groups = w.K / kGroup, sms = sm_count();
    int ranks = 1;
    int64_t least = INT64_MAX;
    for (int n = 1; n <= 8 && n <= groups; n *= 2) {
        const int64_t cost = (tiles * n + sms - 1) / sms * ((groups + n - 1) / n + 8);
        if (cost < least) {
            least = cost;
            ranks = n;
        }
    }
    CUtensorMap word_map;
    if (!tc::make_map(&word_map, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, w.qweight, w.K / 8, w.R, w.R, kWordsPerGroup, 32, true))
        return CQ_ERR_CUDA;
    constexpr auto kernel = few_rows_kernel<D, NT>;
    if (allow_shared<kernel>(FewStages<NT>::kBytes) != cudaSuccess)
        return CQ_ERR_CUDA;
    return launch_clusters(kernel, tiles * ranks, ranks, kFewThreads, FewStages<NT>::kBytes, stream, word_map, x, ldx,
                           static_cast<int>(T), w, ep);
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
                         float *dscales, bool after_dx, cudaStream_t stream)
{
    if (T == 0)
        return cudaMemsetAsync(dscales, 0, static_cast<size_t>(w.K / kGroup) * w.R * 4, stream) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
    CUtensorMap dz_map, x_map;
    if (!tc::make_map(&dz_map, map_type<D>(), 2, dz, T, w.R, lddz, kChunk, 64, true) ||
        !tc::make_map(&x_map, map_type<D>(), 2, x, T, w.K, ldx, kChunk, 64, true))
        return CQ_ERR_CUDA;
    constexpr auto kernel = scale_gradient_kernel<D>;
    if (allow_shared<kernel>(kGradBytes) != cudaSuccess)
        return CQ_ERR_CUDA;
    const int64_t tiles = (w.R + kM - 1) / kM * ((w.K + kGradN - 1) / kGradN), sms = sm_count();
    const unsigned ctas = static_cast<unsigned>(tiles < sms ? tiles : sms);
    if (after_dx)
        return launch_next(kernel, ctas, kGradThreads, kGradBytes, stream, dz_map, x_map, w, T, dscales);
    kernel<<<ctas, kGradThreads, kGradBytes, stream>>>(dz_map, x_map, w, T, dscales);
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
        (pre && !good_rows(pre, ldpre, R)) || (bias && !is_aligned(bias, 16)))
        return CQ_ERR_INVALID_ARG;
    const Layer w = {reinterpret_cast<const uint32_t *>(qweight), reinterpret_cast<const uint32_t *>(qzeros), gptq_scales, R, K, kLow};
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
    const Layer w = {reinterpret_cast<const uint32_t *>(qweight), reinterpret_cast<const uint32_t *>(qzeros), gptq_scales, R, K, kLow};
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
        return dtype == CQ_DTYPE_BF16 ? scale_gradient<BF16>(d, lddz, xs, ldx, T, w, dscales, dx != nullptr, s)
                                      : scale_gradient<FP16>(d, lddz, xs, ldx, T, w, dscales, dx != nullptr, s);
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
    auto kernel = dtype == CQ_DTYPE_BF16 ? activation_backward_kernel<BF16> : activation_backward_kernel<FP16>;
    const unsigned grid = static_cast<unsigned>((R + kActColumns - 1) / kActColumns * kActCluster);
    kernel<<<grid, kActThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t *>(dy), lddy, static_cast<const uint16_t *>(pre), ldpre, T, R, activation,
        static_cast<uint16_t *>(dz), lddz, dbias);
    return launched();
}

cq_status cq_w4_status(void *stream)
{
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return CQ_ERR_CUDA;
    bool gave_up = false;
    if (tc::take_report(&gave_up) != cudaSuccess)
        return CQ_ERR_CUDA;
    return gave_up ? CQ_ERR_CUDA : CQ_OK;
}

}  // extern "C"
