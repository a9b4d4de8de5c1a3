// Device check of the chunk kernel's bounded waits: mbar_wait_or_abort gives up after its limit
// on the GPU's clock and makes the other roles stop, gives up when another role has, and takes
// an arrival before that; mbar_wait_bounded with a longer limit waits longer.  Every loop
// here ends by the clock.
#include <cstdio>

#include "tc_common.cuh"

using namespace pkv::dev;

namespace {

struct Result {
    int ok, abort_flag;
    float ms;
};

// Warp 0 waits (limit 0: by mbar_wait_or_abort); after `delay` ms warp 1 arrives (what = 1) or
// sets the abort flag (2), or does neither (0).
__global__ void wait_kernel(uint64_t limit, int what, int delay, Result *out)
{
    __shared__ uint64_t bar;
    __shared__ volatile int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();
    const uint64_t t0 = globaltimer_ns();
    if (threadIdx.x < 32) {
        const bool ok = __all_sync(FULL_MASK, limit ? mbar_wait_bounded(&bar, 0u, &abort_flag, limit)
                                                    : mbar_wait_or_abort(&bar, 0u, &abort_flag));
        if (threadIdx.x == 0) {
            out->ok = ok;
            out->ms = (float)(globaltimer_ns() - t0) * 1e-6f;
        }
    } else if (threadIdx.x == 32 && what) {
        while (globaltimer_ns() - t0 < (uint64_t)delay * 1000000u) {
        }
        if (what == 1)
            mbar_arrive(&bar);
        else
            abort_flag = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        out->abort_flag = abort_flag;
}

int check(const char *name, uint64_t limit, int what, int delay, int ok, float least, float most, Result *r)
{
    wait_kernel<<<1, 64>>>(limit, what, delay, r);
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        std::printf("%s: %s\n", name, cudaGetErrorString(e));
        return 1;
    }
    std::printf("%s: ok %d abort %d, %.1f ms\n", name, r->ok, r->abort_flag, r->ms);
    // (mbar_wait_bounded leaves the flag to its caller)
    return r->ok != ok || r->abort_flag != (!ok && !limit) || r->ms < least || r->ms > most;
}

}  // namespace

int main()
{
    Result *r = nullptr;
    if (cudaMallocManaged(&r, sizeof(Result)) != cudaSuccess)
        return 1;
    int bad = 0;
    // the limit is 1074 ms; a wait looks at the clock every 64 tries
    bad |= check("no arrival", 0, 0, 0, 0, 1050.0f, 1500.0f, r);
    bad |= check("another role gave up", 0, 2, 50, 0, 50.0f, 400.0f, r);
    bad |= check("a late arrival", 0, 1, 300, 1, 300.0f, 700.0f, r);
    bad |= check("no arrival, a short limit", 100000000, 0, 0, 0, 100.0f, 400.0f, r);
    bad |= check("a later arrival, a longer limit", 2 * WAIT_LIMIT_NS, 1, 1500, 1, 1500.0f, 2000.0f, r);
    std::printf(bad ? "wrong\n" : "ok\n");
    return bad;
}
