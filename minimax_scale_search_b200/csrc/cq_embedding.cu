// Rows of a quantised table, and the gradient of its group scales.
//
// The table is the selection's own output for a [V][K] matrix: scales
// [V * K/128] and code words [V * K/128][16], so a row's words are contiguous.
//
// Lookup.  out[t] = m s q of row ids[t]; the bytes of the output bound it.  Sixteen lanes have a unit of up to
// four groups of one token (a word of 8 values of each group a lane), all their loads before the first store.
// 8,192 tokens x 4,096 to fp16: 14.5 us, 5.4 TB/s.
//
// Gradient.  dscales[v][g] = m sum_{t: ids[t] = v} sum_{i in g} dout[t][i] q[v][i], in
// three launches:
//  1. dots[t][g] = sum_{i in g} dout[t][i] q[id_t][i] (fp32, one pass over dout, which is what
//     bounds the whole); the same launch fills dscales with zeros and sorts the tokens by
//     (id, t): up to kRankMost tokens by counting, for each, the tokens before it (T^2
//     comparisons, no further launch), others with a radix sort of its own launches;
//  2. sums over the runs of equal ids within each chunk of 8 sorted tokens, in fp64; a run that
//     lies inside a chunk is done, others leave a part at the chunk's head or tail;
//  3. the runs across chunks, from their parts in order.
// So a row that every token names is summed by many threads, and the order of the sums is fixed.
// 8,192 bf16 tokens x 4,096: 33 us (26 the first launch: its ranking takes 20 on its own, the pass over dout 13 at HBM's
// rate, and they overlap in part); 65,536 x 1,024: 61 us, half of them the radix sort.  Each launch but a call's first begins before the one
// in front of it has ended and waits for it where it needs its results (without: 73 us, 9,000 x 256 41 for 29).
#include <type_traits>

#include "cq_w4.cuh"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / kWordsPerGroup;       // units of a CTA at a time: kGroups groups of one token
// Tokens sorted by counting: what the 48 KB of a CTA's static shared memory hold, and up to there counting is the faster
// (calls of width 1,024 by counting and by radix sort: 12 and 25 us at 1,024 tokens, 15 and 27 at 4,096, 25 and 30 at 8,192;
// of width 4,096: 12 and 24, 21 and 34, 33 and 44);
constexpr int kRankMost = 8192;
constexpr int64_t kRankRows = 1 << 24;                  // and tables whose row numbers fp32 holds
constexpr int kRankBlock = 32;                          // tokens ranked by a CTA, one a lane
constexpr int kChunk = 8;                               // sorted tokens per partial sum
constexpr int kSortTokens = 1024;                       // per CTA of the radix sort

struct Ids {
    const void *p;
    int wide;  // int64 ids
    int64_t V;
    // The row of token t, or V for an id outside [0, V).
    __device__ __forceinline__ uint32_t key(int64_t t) const
    {
        const int64_t v = wide ? static_cast<const int64_t *>(p)[t] : static_cast<const int32_t *>(p)[t];
        return static_cast<uint32_t>(v >= 0 && v < V ? v : V);
    }
};

// Division by the units of a row.  Below 2^31: i d^-1 as a product with ceil(2^(31+s) / d), 2^(s-1) < d <= 2^s,
// whose excess of less than 2^-31 i / 2^s < 1 / d never reaches the next quotient.
struct Divider {
    int64_t d;
    uint32_t factor;  // 0: 64-bit division, or by one
    int shift;
    Divider(int64_t d, int64_t n) : d(d), factor(0), shift(0)
    {
        if (d == 1 || n >= (static_cast<int64_t>(1) << 31))
            return;
        while ((static_cast<int64_t>(1) << shift) < d)
            shift++;
        factor = static_cast<uint32_t>(((static_cast<uint64_t>(1) << (31 + shift)) + d - 1) / d);
        shift--;  // the product's upper half is taken first
    }
    __device__ __forceinline__ void operator()(int64_t i, int64_t &q, int64_t &r) const
    {
        if (factor) {
            const uint32_t n = static_cast<uint32_t>(i), k = __umulhi(n, factor) >> shift;
            q = k;
            r = n - k * static_cast<uint32_t>(d);
        } else {
            q = d == 1 ? i : i / d;
            r = i - q * d;
        }
    }
};

// Eight values u - 8 from a code word: pairs in binary16, where 1024 | u is 1024 + u.
__device__ __forceinline__ void unpack(uint32_t word, uint32_t low, float (&q)[8])
{
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t n = FP16::sub(((word >> (4 * j)) & low) | FP16::kMagic, FP16::kMagic + 0x00080008u);
        const float2 f = __half22float2(reinterpret_cast<const __half2 &>(n));
        q[j] = f.x;
        q[j + 4] = f.y;
    }
}

template <int DT>
__device__ __forceinline__ void store8(void *out, int64_t i, const float (&v)[8])
{
    if (DT == CQ_DTYPE_FP32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + i);
        __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
        const uint4 h = DT == CQ_DTYPE_BF16 ? narrow<BF16>(v) : narrow<FP16>(v);
        __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + i), h);
    }
}

// Eight elements of dout as they lie in memory, and their values.
template <int DT>
struct Eight {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *in, int64_t i)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(in) + i * (DT == CQ_DTYPE_FP32 ? 4 : 2));
        a = __ldcs(p);
        if (DT == CQ_DTYPE_FP32)
            b = __ldcs(p + 1);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        if (DT == CQ_DTYPE_FP32) {
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        } else if (DT == CQ_DTYPE_BF16) {
            widen<BF16>(a, v);
        } else {
            widen<FP16>(a, v);
        }
    }
};

template <int DT, int kGroups>
__global__ void __launch_bounds__(kThreads) embedding_kernel(Ids ids, int64_t T, const uint16_t *__restrict__ scales,
                                                             const uint32_t *__restrict__ codes, int64_t ng, Divider by,
                                                             uint32_t low, float multiplier, void *__restrict__ out)
{
    const int lane = threadIdx.x % kWordsPerGroup;
    for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + threadIdx.x / kWordsPerGroup; unit < T * by.d;
         unit += static_cast<int64_t>(gridDim.x) * kUnits) {
        int64_t t, b;
        by(unit, t, b);
        const uint32_t row = ids.key(t);
        const bool named = row < ids.V;
        const int64_t g0 = b * kGroups;
        const int n = ng - g0 < kGroups ? static_cast<int>(ng - g0) : kGroups;
        const int64_t from = row * ng + g0;
        uint32_t word[kGroups];
        uint16_t scale[kGroups];
#pragma unroll
        for (int u = 0; u < kGroups; u++)
            if (named && u < n) {
                word[u] = codes[(from + u) * kWordsPerGroup + lane];
                scale[u] = scales[from + u];
            }
#pragma unroll
        for (int u = 0; u < kGroups; u++) {
            if (u >= n)
                break;
            float q[8] = {};
            if (named) {
                const float s = half_bits(scale[u]);
                unpack(word[u], low, q);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    q[j] = multiplier * (s * q[j]);
            }
            store8<DT>(out, ((t * ng + g0 + u) * kWordsPerGroup + lane) * 8, q);
        }
    }
}

// ---- gradient ------------------------------------------------------------------------------------

// order[rank] = t, key[rank] = row: for each of a CTA's 32 tokens, one a lane, the number of tokens before it
// by (row, t).  The warps take an eighth of the tokens each to compare with, four per shared read.  A comparison of
// row numbers is the difference clamped to [0, 1], in fp32, where it and its sum are one instruction each.
__device__ void rank_tokens(const Ids &ids, int T, int t0, uint32_t *key, int32_t *order)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ alignas(16) float tile[kRankMost];
    __shared__ int ranks[kWarps][kRankBlock];
    static_assert(kRankMost % kThreads == 0 && kThreads % (32 * kWarps) == 0 && kRankBlock == 32, "shares are blocks of 32");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, t = t0 + lane;
    const uint32_t row = t < T ? ids.key(t) : 0;
    const float mine = static_cast<float>(row);
    const int end = (T + kThreads - 1) / kThreads * kThreads;  // the tokens that are there, and some that are above all
#pragma unroll 8
    for (int j = threadIdx.x; j < end; j += kThreads)
        tile[j] = j < T ? static_cast<float>(ids.key(j)) : 2.0f * kRankRows;
    __syncthreads();
    // (other, j) < (mine, t)  <=>  other < mine + (j < t)
    float rank[4] = {};
    const int share = end / kWarps;  // % 32 == 0
    for (int j0 = warp * share; j0 < (warp + 1) * share; j0 += 32) {
        if (j0 != t0) {
            const float below = mine + (j0 < t0 ? 1.0f : 0.0f);
            const float4 *p = reinterpret_cast<const float4 *>(tile + j0);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float4 o = p[j];
                rank[0] += __saturatef(below - o.x);
                rank[1] += __saturatef(below - o.y);
                rank[2] += __saturatef(below - o.z);
                rank[3] += __saturatef(below - o.w);
            }
        } else {
            for (int j = j0; j < j0 + 32; j++)
                rank[0] += __saturatef(mine + (j < t ? 1.0f : 0.0f) - tile[j]);
        }
    }
    ranks[warp][lane] = static_cast<int>(rank[0] + rank[1] + rank[2] + rank[3]);
    __syncthreads();
    if (warp == 0 && t < T) {
        int r = 0;
#pragma unroll
        for (int i = 0; i < kWarps; i++)
            r += ranks[i][lane];
        key[r] = row;
        order[r] = t;
    }
}

// Sums of kGroups values over 16 lanes, in a fixed order: the sum of value u in lane u * 16 / kGroups.
template <int kGroups>
__device__ __forceinline__ float sum_lanes(float (&v)[kGroups], int lane)
{
    int n = kGroups;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        if (n > 1) {  // a lane keeps half of its values and gets its partner's parts of them
            n /= 2;
#pragma unroll
            for (int u = 0; u < kGroups / 2; u++)
                if (u < n) {
                    const bool upper = lane & o;
                    const float give = upper ? v[u] : v[u + n];
                    v[u] = (upper ? v[u + n] : v[u]) + __shfl_xor_sync(0xFFFFFFFFu, give, o, 16);
                }
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o, 16);
        }
    }
    return v[0];
}

// Blocks below `rank_blocks` sort by counting; the others form the dots and write the zeros.
template <int DT, int kGroups>
__global__ void __launch_bounds__(kThreads) dots_kernel(const void *__restrict__ dout, Ids ids, int64_t T,
                                                        const uint32_t *__restrict__ codes, int64_t ng, Divider by, uint32_t low,
                                                        float *__restrict__ dots, int rank_blocks, uint32_t *key, int32_t *order,
                                                        float *__restrict__ dscales)
{
    let_next_begin();
    if (static_cast<int>(blockIdx.x) < rank_blocks) {
        rank_tokens(ids, static_cast<int>(T), blockIdx.x * kRankBlock, key, order);
        return;
    }
    const int64_t block = blockIdx.x - rank_blocks, blocks = gridDim.x - rank_blocks;
    const int lane = threadIdx.x % kWordsPerGroup;
    for (int64_t unit0 = block * kUnits; unit0 < T * by.d; unit0 += blocks * kUnits) {
        const int64_t unit = unit0 + threadIdx.x / kWordsPerGroup;
        float v[kGroups] = {};
        int64_t t = 0, g0 = 0;
        int n = 0;
        if (unit < T * by.d) {
            int64_t b;
            by(unit, t, b);
            g0 = b * kGroups;
            n = ng - g0 < kGroups ? static_cast<int>(ng - g0) : kGroups;
            uint32_t word[kGroups];
            Eight<DT> d[kGroups];
#pragma unroll
            for (int u = 0; u < kGroups; u++)
                if (u < n)
                    d[u].load(dout, ((t * ng + g0 + u) * kWordsPerGroup + lane) * 8);  // does not wait for the id
            const uint32_t row = ids.key(t);
            if (row < ids.V) {
#pragma unroll
                for (int u = 0; u < kGroups; u++)
                    if (u < n)
                        word[u] = codes[(row * ng + g0 + u) * kWordsPerGroup + lane];
#pragma unroll
                for (int u = 0; u < kGroups; u++)
                    if (u < n) {
                        float x[8], q[8];
                        d[u].values(x);
                        unpack(word[u], low, q);
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            v[u] = fmaf(x[j], q[j], v[u]);
                    }
            }
        }
        const float sum = sum_lanes<kGroups>(v, lane);
        constexpr int kSpread = kWordsPerGroup / kGroups;
        if (lane % kSpread == 0 && lane / kSpread < n)
            dots[t * ng + g0 + lane / kSpread] = sum;
    }
    const int64_t outputs = ids.V * ng;
    for (int64_t i = block * kThreads + threadIdx.x; i < outputs; i += blocks * kThreads)
        dscales[i] = 0.0f;
    wait_for_previous();  // the sort, where it is launches of its own: nothing here reads it
}

// The parts of a run that crosses chunks: [chunk][group], what the chunk has of a run that
// began before it (head) and of one that goes on after it (tail).
struct Parts {
    double *head, *tail;
};

// `width` threads (a power of two) have a chunk's groups.  No __restrict__ on what the launch before wrote: loads
// through it might be moved ahead of the wait.
__global__ void __launch_bounds__(kThreads) chunk_sums_kernel(const uint32_t *key, const int32_t *order, int64_t T, int64_t V,
                                                              const float *dots, int64_t ng, int width, float multiplier,
                                                              Parts parts, float *dscales)
{
    let_next_begin();
    wait_for_previous();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (kThreads / width) + threadIdx.x / width;
    const int64_t p0 = c * kChunk, p1 = p0 + kChunk < T ? p0 + kChunk : T;
    if (p0 >= T)
        return;
    for (int64_t g = threadIdx.x % width; g < ng; g += width) {
        uint32_t current = key[p0];
        bool head = p0 > 0 && key[p0 - 1] == current;
        double sum = 0.0;
        auto finish = [&](bool goes_on) {
            if (current >= V)
                return;
            if (head)
                parts.head[c * ng + g] = sum;
            else if (goes_on)
                parts.tail[c * ng + g] = sum;
            else
                dscales[current * ng + g] = static_cast<float>(sum * multiplier);
        };
        constexpr int kAhead = kChunk;
        for (int64_t p = p0; p < p1; p += kAhead) {
            uint32_t k[kAhead];
            float d[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; u++)
                if (p + u < p1) {
                    k[u] = key[p + u];
                    d[u] = dots[order[p + u] * ng + g];
                }
#pragma unroll
            for (int u = 0; u < kAhead; u++)
                if (p + u < p1) {
                    if (k[u] != current) {
                        finish(false);
                        current = k[u];
                        head = false;
                        sum = 0.0;
                    }
                    sum += d[u];
                }
        }
        finish(p1 < T && key[p1] == current);
    }
}

// Runs that begin in chunk c and go on after it, a warp for each: `width` lanes (a power of two) have
// a group each, 32 / width of them share its parts.
__global__ void __launch_bounds__(kThreads) join_runs_kernel(const uint32_t *key, int64_t T, int64_t V, int64_t ng, int width,
                                                             float multiplier, Parts parts, float *dscales)
{
    wait_for_previous();
    const int lane = threadIdx.x % 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32, p0 = c * kChunk;
    if (p0 + kChunk >= T)
        return;
    const uint32_t v = key[p0 + kChunk];
    if (v >= V || key[p0 + kChunk - 1] != v || (p0 > 0 && key[p0 - 1] == v))
        return;
    // the last chunk that begins with v: 32 candidates at once, 32 chunks apart, then the 31 after the last hit
    const int64_t chunks = (T - 1) / kChunk + 1;
    auto begins = [&](int64_t i) { return i < chunks && key[i * kChunk] == v; };
    int64_t last = c + 1;
    for (int hits = 32; hits == 32;) {
        hits = __popc(__ballot_sync(0xFFFFFFFFu, begins(last + 32 * (lane + 1))));
        last += 32 * hits;
    }
    last += __popc(__ballot_sync(0xFFFFFFFFu, begins(last + lane + 1)));
    const int shares = 32 / width, share = lane / width;
    for (int64_t g0 = 0; g0 < ng; g0 += width) {
        const int64_t g = g0 + lane % width;
        double sum = 0.0;
        if (g < ng) {
            constexpr int kAhead = 16;
            for (int64_t i = c + 1 + share; i <= last; i += kAhead * shares) {
                double part[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; u++)
                    part[u] = i + u * shares <= last ? parts.head[(i + u * shares) * ng + g] : 0.0;
#pragma unroll
                for (int u = 0; u < kAhead; u++)
                    sum += part[u];
            }
            if (share == 0)
                sum += parts.tail[c * ng + g];
        }
        for (int o = 16; o >= width; o >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (g < ng && share == 0)
            dscales[v * ng + g] = static_cast<float>(sum * multiplier);
    }
}

// ---- radix sort of the tokens by row, 8 bits a pass, stable ---------------------------------------

struct SortPass {
    const uint32_t *key_in;   // null in the first pass: the tokens in their order
    const int32_t *order_in;
    uint32_t *key_out;
    int32_t *order_out;
    int32_t *counts;          // [256][blocks]
    int shift;
};

__device__ __forceinline__ uint32_t sort_key(const Ids &ids, const SortPass &s, int64_t i)
{
    return s.key_in ? s.key_in[i] : ids.key(i);
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(Ids ids, int64_t T, SortPass s)
{
    __shared__ int32_t count[256];
    let_next_begin();
    wait_for_previous();
    count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTokens;
    for (int j = threadIdx.x; j < kSortTokens && i0 + j < T; j += kThreads)
        atomicAdd(&count[(sort_key(ids, s, i0 + j) >> s.shift) & 255u], 1);
    __syncthreads();
    s.counts[threadIdx.x * static_cast<int64_t>(gridDim.x) + blockIdx.x] = count[threadIdx.x];
}

// counts -> the number of tokens before each (digit, block), by one CTA.
__global__ void __launch_bounds__(1024) sort_scan_kernel(int32_t *counts, int64_t n)
{
    __shared__ int32_t sums[32];
    let_next_begin();
    wait_for_previous();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    constexpr int kEach = 8;  // counts per thread, n % 256 == 0
    int32_t before = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 1024 * kEach) {
        const int64_t i = i0 + threadIdx.x * kEach;
        int4 a = make_int4(0, 0, 0, 0), b = a;
        if (i < n) {
            a = *reinterpret_cast<const int4 *>(counts + i);
            b = *reinterpret_cast<const int4 *>(counts + i + 4);
        }
        const int32_t mine = a.x + a.y + a.z + a.w + b.x + b.y + b.z + b.w;
        int32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            x += lane >= o ? y : 0;
        }
        if (lane == 31)
            sums[warp] = x;
        __syncthreads();
        int32_t w = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            w += lane >= o ? y : 0;
        }
        const int32_t warps_before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) % 32);
        const int32_t total = __shfl_sync(0xFFFFFFFFu, w, 31);
        if (i < n) {
            int32_t at = before + (warp > 0 ? warps_before : 0) + x - mine;
            int4 p, q;
            p.x = at;
            p.y = at += a.x;
            p.z = at += a.y;
            p.w = at += a.z;
            q.x = at += a.w;
            q.y = at += b.x;
            q.z = at += b.y;
            q.w = at += b.z;
            *reinterpret_cast<int4 *>(counts + i) = p;
            *reinterpret_cast<int4 *>(counts + i + 4) = q;
        }
        before += total;
        __syncthreads();
    }
}

// A warp has 128 tokens in a row; first its digits' counts, then each token's place: the digit's
// start, the warps before, the warp's tokens before.
__global__ void __launch_bounds__(kThreads) sort_scatter_kernel(Ids ids, int64_t T, SortPass s)
{
    constexpr int kWarps = kThreads / 32, kPerWarp = kSortTokens / kWarps;
    __shared__ int32_t count[kWarps][256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int j = threadIdx.x; j < kWarps * 256; j += kThreads)
        count[j / 256][j % 256] = 0;
    let_next_begin();
    wait_for_previous();
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTokens + warp * kPerWarp;
    for (int j = lane; j < kPerWarp; j += 32)
        if (i0 + j < T)
            atomicAdd(&count[warp][(sort_key(ids, s, i0 + j) >> s.shift) & 255u], 1);
    __syncthreads();
    int32_t at = s.counts[threadIdx.x * static_cast<int64_t>(gridDim.x) + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        const int32_t n = count[w][threadIdx.x];
        count[w][threadIdx.x] = at;
        at += n;
    }
    __syncthreads();
    for (int j = lane; j < kPerWarp; j += 32) {
        const bool inside = i0 + j < T;
        const uint32_t k = inside ? sort_key(ids, s, i0 + j) : 0;
        const uint32_t digit = inside ? (k >> s.shift) & 255u : 256u;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
        const int before = __popc(same & ((1u << lane) - 1));
        int32_t place = 0;
        if (inside)
            place = count[warp][digit] + before;
        __syncwarp();
        if (inside) {
            if (before == 0)
                count[warp][digit] += __popc(same);
            s.key_out[place] = k;
            s.order_out[place] = s.key_in ? s.order_in[i0 + j] : static_cast<int32_t>(i0 + j);
        }
        __syncwarp();
    }
}

// CTAs for so many units.
unsigned grid_for(int64_t units)
{
    const int64_t blocks = (units + kUnits - 1) / kUnits, most = static_cast<int64_t>(sm_count()) * 32;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

// Four groups to a unit where rows have them; a single one for rows of one to three groups, whose
// units would stand idle in part.
template <class F>
cq_status by_groups(int64_t ng, F run)
{
    return ng >= 4 ? run(std::integral_constant<int, 4>()) : run(std::integral_constant<int, 1>());
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

// Where the gradient's workspace holds what.
struct Workspace {
    size_t key, order, key2, order2, counts, dots, head, tail, bytes;
    Workspace(int64_t T, int64_t K)
    {
        const size_t n = static_cast<size_t>(T), ng = static_cast<size_t>(K / kGroup), chunks = (n + kChunk - 1) / kChunk;
        size_t at = 0;
        auto take = [&](size_t size) {
            const size_t here = at;
            at += (size + 255) / 256 * 256;
            return here;
        };
        key = take(n * 4);
        order = take(n * 4);
        key2 = take(n * 4);
        order2 = take(n * 4);
        counts = take((n + kSortTokens - 1) / kSortTokens * 256 * 4);
        dots = take(n * ng * 4);
        head = take(chunks * ng * 8);
        tail = take(chunks * ng * 8);
        bytes = at;
    }
};

cq_status sort_tokens(const Ids &ids, int64_t T, char *base, const Workspace &ws, cudaStream_t stream)
{
    const unsigned blocks = static_cast<unsigned>((T + kSortTokens - 1) / kSortTokens);
    int passes = 1;
    while (passes < 4 && (ids.V >> (8 * passes)) != 0)
        passes++;
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(base + ws.key), reinterpret_cast<uint32_t *>(base + ws.key2)};
    int32_t *orders[2] = {reinterpret_cast<int32_t *>(base + ws.order), reinterpret_cast<int32_t *>(base + ws.order2)};
    for (int i = 0; i < passes; i++) {
        const int to = (passes - 1 - i) % 2;  // the last pass ends in the first pair
        SortPass s = {i > 0 ? keys[1 - to] : nullptr, orders[1 - to], keys[to], orders[to],
                      reinterpret_cast<int32_t *>(base + ws.counts), 8 * i};
        cq_status st = CQ_OK;
        if (i == 0) {
            sort_count_kernel<<<blocks, kThreads, 0, stream>>>(ids, T, s);
            st = launched();
        } else {
            st = launch_next(sort_count_kernel, blocks, kThreads, 0, stream, ids, T, s);
        }
        if (st == CQ_OK)
            st = launch_next(sort_scan_kernel, 1, 1024, 0, stream, s.counts, static_cast<int64_t>(blocks) * 256);
        if (st == CQ_OK)
            st = launch_next(sort_scatter_kernel, blocks, kThreads, 0, stream, ids, T, s);
        if (st != CQ_OK)
            return st;
    }
    return CQ_OK;
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
    const int64_t ng = K / kGroup;
    auto run = [&](auto groups) {
        constexpr int kGroups = decltype(groups)::value;
        const int64_t units = (ng + kGroups - 1) / kGroups;
        auto kernel = dtype == CQ_DTYPE_BF16   ? embedding_kernel<CQ_DTYPE_BF16, kGroups>
                      : dtype == CQ_DTYPE_FP16 ? embedding_kernel<CQ_DTYPE_FP16, kGroups>
                                               : embedding_kernel<CQ_DTYPE_FP32, kGroups>;
        kernel<<<grid_for(T * units), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(in, T, scales, codes, ng,
                                                                                        Divider(units, T * units), kLow, multiplier, out);
        return launched();
    };
    return by_groups(ng, run);
}

size_t cq_w4_embedding_backward_workspace_bytes(int64_t T, int64_t K)
{
    if (T <= 0 || K <= 0)
        return 256;
    return Workspace(T, K).bytes;
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t ng = K / kGroup;
    if (T == 0)
        return cudaMemsetAsync(dscales, 0, static_cast<size_t>(V) * ng * 4, s) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
    const Workspace ws(T, K);
    if (!workspace || !is_aligned(workspace, 256) || workspace_bytes < ws.bytes)
        return CQ_ERR_WORKSPACE;
    char *base = static_cast<char *>(workspace);
    uint32_t *key = reinterpret_cast<uint32_t *>(base + ws.key);
    int32_t *order = reinterpret_cast<int32_t *>(base + ws.order);
    float *dots = reinterpret_cast<float *>(base + ws.dots);
    const Parts parts = {reinterpret_cast<double *>(base + ws.head), reinterpret_cast<double *>(base + ws.tail)};
    const Ids in = {ids, ids64, V};

    const bool count = T <= kRankMost && V < kRankRows;
    const int rank_blocks = count ? static_cast<int>((T + kRankBlock - 1) / kRankBlock) : 0;
    if (!count && sort_tokens(in, T, base, ws, s) != CQ_OK)
        return CQ_ERR_CUDA;
    const cq_status made = by_groups(ng, [&](auto groups) {
        constexpr int kGroups = decltype(groups)::value;
        auto kernel = dtype == CQ_DTYPE_BF16   ? dots_kernel<CQ_DTYPE_BF16, kGroups>
                      : dtype == CQ_DTYPE_FP16 ? dots_kernel<CQ_DTYPE_FP16, kGroups>
                                               : dots_kernel<CQ_DTYPE_FP32, kGroups>;
        const int64_t units = (ng + kGroups - 1) / kGroups, zeros = V * ng / 256;  // a CTA's share of zeros costs about one unit
        const unsigned grid = rank_blocks + grid_for(T * units > zeros ? T * units : zeros);
        const Divider by(units, T * units);
        if (!count)
            return launch_next(kernel, grid, kThreads, 0, s, dout, in, T, codes, ng, by, kLow, dots, rank_blocks, key, order, dscales);
        kernel<<<grid, kThreads, 0, s>>>(dout, in, T, codes, ng, by, kLow, dots, rank_blocks, key, order, dscales);
        return launched();
    });
    if (made != CQ_OK)
        return made;
    int width = 1;
    while (width < kThreads && width < ng)
        width *= 2;
    const int64_t chunks = (T + kChunk - 1) / kChunk, per_block = kThreads / width;
    const unsigned grid = static_cast<unsigned>((chunks + per_block - 1) / per_block);
    const cq_status summed = launch_next(chunk_sums_kernel, grid, kThreads, 0, s, key, order, T, V, dots, ng, width, multiplier, parts, dscales);
    if (summed != CQ_OK || chunks == 1)
        return summed;
    return launch_next(join_runs_kernel, static_cast<unsigned>((chunks + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s, key, T, V,
                       ng, width < 32 ? width : 32, multiplier, parts, dscales);
}

}  // extern "C"
