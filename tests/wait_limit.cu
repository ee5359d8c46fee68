// A kernel whose roles hand work on through the library's bounded waits, but for one barrier that gets no arrival.
// The first wait for it runs out after `most` nanoseconds; every role then leaves, and the CTA reports it.
#include "cq_tensor.cuh"

using namespace cq;

__global__ void __launch_bounds__(96) roles_kernel(uint64_t most, int lost, int *left)
{
    __shared__ alignas(8) uint64_t bars[3];
    __shared__ int stop_flag;
    volatile int *stop = &stop_flag;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; i++)
            tc::barrier_init(tc::smem_address(&bars[i]), 1);
        *stop = 0;
        tc::barrier_init_fence();
    }
    __syncthreads();
    // a ring of three roles: each waits for the one before it and lets the next one go; role 0 lets the first round go
    bool going = true;
    int rounds = 0;
    for (; going && rounds < 4; rounds++) {
        if (warp > 0 || rounds > 0)
            going = tc::barrier_wait_warp(tc::smem_address(&bars[warp]), (warp > 0 ? rounds : rounds - 1) & 1, stop, most);
        if (going && threadIdx.x % 32 == 0 && !(warp == 1 && rounds == lost))
            tc::barrier_arrive(tc::smem_address(&bars[(warp + 1) % 3]));
    }
    __syncthreads();
    tc::report(stop);
    if (threadIdx.x % 32 == 0)
        left[warp] = going ? rounds : -rounds;
}

extern "C" int run_roles(uint64_t most, int lost, int *left)
{
    roles_kernel<<<1, 96>>>(most, lost, left);
    return cudaDeviceSynchronize();
}

extern "C" int reported(int *gave_up)
{
    bool set = false;
    const cudaError_t e = tc::take_report(&set);
    *gave_up = set;
    return e;
}
