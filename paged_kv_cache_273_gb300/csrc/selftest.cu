// pkv_selftest_wait_timeout: two threads wait, with the two forms of the
// library's bounded mbarrier wait, on phases that nothing completes.  Each gives
// up after its time limit, and when both have the kernel records
// PKV_EBIT_TIMEOUT in the pool's error word and returns, so the failure path of
// every bounded wait in the library's kernels (report, return, context still
// usable) can be checked without faulting or hanging the device.

#include <cuda_runtime.h>

#include "tc_common.cuh"

namespace pkv {
namespace {

using namespace dev;

__global__ void wait_timeout_kernel(unsigned int *err)
{
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag[2], gave_up[2];
    const int w = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[i], 1);                 // one arrival expected, none comes
            abort_flag[i] = 0;
        }
        mbar_fence_init();
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        gave_up[w] = !(w ? mbar_wait_or_abort(&bar[1], 0u, &abort_flag[1])
                         : mbar_wait_bounded(&bar[0], 0u, &abort_flag[0]));
    __syncthreads();
    if (threadIdx.x == 0 && gave_up[0] && gave_up[1] && abort_flag[1])
        atomicOr(err, PKV_EBIT_TIMEOUT);
}

}  // namespace

int launch_selftest_wait_timeout(const pkv_pool *pool, pkv_stream_t stream)
{
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    wait_timeout_kernel<<<1, 64, 0, s>>>(pool->d_err);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
