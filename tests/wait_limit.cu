// wait_limit.cu -- the waits with a limit of async_copy.cuh by themselves, with
// a limit of 2 ms, on a barrier that this block alone completes or leaves be.
#include "async_copy.cuh"

using namespace rlscan::seq;
namespace ptx = rlscan::ptx;

__device__ unsigned int g_timed_out;

// 0: the phase never comes; 1: it has come; 2: it has come, and a thread has given
// up elsewhere; 3: as 0, and the first warp is gone before the second gives up;
// 4: it has come for every other lane alone.
__global__ void __launch_bounds__(64) wait_kernel(int kind, int *threads, int *warps)
{
    constexpr uint64_t kLimitNs = 2'000'000;
    __shared__ uint64_t bar;
    __shared__ int gave_up;
    if (threadIdx.x == 0) {
        gave_up = kind == 2;
        ptx::mbar_init(&bar, 1);
        ptx::fence_mbar_init();
        if (kind == 1 || kind == 2 || kind == 4) ptx::mbar_arrive(&bar);
    }
    __syncthreads();
    if (kind != 3 || threadIdx.x >= 32) {
        const uint32_t parity = kind == 4 ? threadIdx.x & 1u : 0u;
        threads[threadIdx.x] = wait(ptx::smem_u32(&bar), parity, &gave_up, kLimitNs);
        warps[threadIdx.x] = wait_warp(ptx::smem_u32(&bar), parity, &gave_up, kLimitNs);
    }
    leave(&gave_up, &g_timed_out);
}

// -1: a launch failed; else the status, then the status of a second question
extern "C" __attribute__((visibility("default"))) int run_waits(int kind, int *threads, int *warps, int *again, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    wait_kernel<<<1, 64, 0, s>>>(kind, threads, warps);
    if (cudaGetLastError() != cudaSuccess) return -1;
    const rlscan_status first = take_flag(g_timed_out, s);
    *again = take_flag(g_timed_out, s);
    return first;
}
