// Wrappers of the sm_100a instructions that the tensor-core kernels issue: mbarriers
// with bounded waits, tensor-map copies, and the tcgen05 family.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cq {
namespace tc {

__device__ __forceinline__ uint32_t smem_address(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// A value that is the same in all lanes, in a form that the compiler knows to be: branches on it are
// uniform, and addresses and descriptors made of it stay in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v)
{
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// One lane of the warp: the one that issues for all.
__device__ __forceinline__ bool elected()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// ---- mbarriers ---------------------------------------------------------------------------------

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void barrier_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void barrier_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

// A wait that has not ended after this long gives up (waits take microseconds).
constexpr uint64_t kMostNanoseconds = 4000000000ull;

__device__ __forceinline__ uint64_t now()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Waits for a phase; false when it did not come, or when another thread of the CTA has
// given up (*stop).  Every role then leaves its loop.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile int *stop, uint64_t most = kMostNanoseconds)
{
    if (barrier_try(bar, parity))
        return true;
    const uint64_t start = now();
    for (uint32_t i = 1;; i++) {
        if (barrier_try(bar, parity))
            return true;
        if (i % 64 == 0) {
            if (*stop)
                return false;
            if (now() - start > most) {
                *stop = 1;
                return false;
            }
        }
    }
}

// The same for a whole warp, with one answer for its lanes.
__device__ __forceinline__ bool barrier_wait_warp(uint32_t bar, uint32_t parity, volatile int *stop, uint64_t most = kMostNanoseconds)
{
    return __all_sync(0xFFFFFFFFu, barrier_wait(bar, parity, stop, most));
}

// Two of them at once.
__device__ __forceinline__ bool barrier_wait_both(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, volatile int *stop)
{
    const bool first = barrier_try(bar0, parity0), second = barrier_try(bar1, parity1);
    if (__all_sync(0xFFFFFFFFu, first && second))
        return true;
    return barrier_wait_warp(bar0, parity0, stop) && barrier_wait_warp(bar1, parity1, stop);
}

// After a wait that gave up: long enough for every copy and product in flight to end.
__device__ __forceinline__ void let_copies_land()
{
    for (int i = 0; i < 1000; i++)
        __nanosleep(1000);
}

static __device__ int g_gave_up;  // set when a wait in a kernel of this file ran out

// By every thread of a CTA whose roles have left their loops.
__device__ __forceinline__ void report(volatile int *stop)
{
    if (*stop) {
        let_copies_land();
        g_gave_up = 1;
    }
}

// Whether a wait has run out on the current device since this was last asked.
static cudaError_t take_report(bool *gave_up)
{
    int set = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&set, g_gave_up, sizeof(set));
    *gave_up = set != 0;
    if (e == cudaSuccess && set) {
        set = 0;
        e = cudaMemcpyToSymbol(g_gave_up, &set, sizeof(set));
    }
    return e;
}

// ---- copies ----------------------------------------------------------------------------------------

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// kBytes from global to shared memory, zeros where not `valid`.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? kBytes : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}

// The barrier gets this thread's arrival when its copy_async have landed.
__device__ __forceinline__ void copy_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void copy_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits for this thread's copies but those of its last kGroups commits.
template <int kGroups>
__device__ __forceinline__ void copy_async_wait_but()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kGroups) : "memory");
}

__device__ __forceinline__ void copy_async_wait()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ void store_shared(uint32_t at, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Shared memory written by this thread becomes visible to the tensor cores.
__device__ __forceinline__ void fence_shared_writes()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory and the matrix instruction --------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The three below are called by a whole warp, and by predicate only its leader issues: in a branch of the leader's
// own the operands could not stay in uniform registers (an instruction then took about 80 cycles to issue).

__device__ __forceinline__ void commit(uint32_t bar, bool leader)
{
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
        "r"(static_cast<uint32_t>(leader))
        : "memory");
}

// d = a b + (add ? d : 0).
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, bool leader)
{
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
        : "memory");
}

// 32 columns of this warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// The same of 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Descriptor of an operand in shared memory, in rows of 128 bytes with the 16-byte chunks
// swizzled by the row number modulo 8.
//  contraction along the row: `stride` bytes between blocks of 8 rows (1024); `lead` unused;
//  contraction across rows: `stride` bytes between blocks of 8 rows of the contraction,
//  `lead` between blocks of 64 elements of the other dimension.
__device__ __forceinline__ uint64_t descriptor(uint32_t address, uint32_t lead, uint32_t stride)
{
    return static_cast<uint64_t>((address & 0x3FFFF) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
           static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: fp32 sums of bf16 (or fp16) products, 128 x n, each operand
// contracted along its rows or across them.
__host__ __device__ constexpr uint32_t instruction(bool bf16, bool a_across, bool b_across, int n)
{
    return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (a_across ? 1u : 0u) << 15 |
           (b_across ? 1u : 0u) << 16 | static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}

// ---- host: tensor maps -----------------------------------------------------------------------------

// A map of [rows][cols] elements, ld elements apart, in boxes of box_rows x box_cols; what lies
// outside reads as zeros.  Swizzled boxes have rows of 128 bytes.
inline bool make_map(CUtensorMap *map, CUtensorMapDataType type, int element, const void *base, int64_t rows, int64_t cols,
                     int64_t ld, int box_rows, int box_cols, bool swizzled)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) == cudaSuccess &&
                       found == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<Encode>(f)
                   : nullptr;
    }();
    if (!encode)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * element};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace cq
