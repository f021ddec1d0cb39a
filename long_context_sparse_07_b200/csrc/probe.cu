// probe.cu -- a kernel whose only job is to let bounded device-side waits run
// out: one thread waits on an mbarrier that nothing arrives on and gives up
// after the requested time; then a warp waits on another (mbar_wait_warp) of
// which one lane is told to give up, while the barrier completes for the other
// lanes a while later. The kernel records CSA_ERR_TIMEOUT in the device error
// word, exactly as the pipeline kernels do when one of their waits expires,
// with the number of the warp's lanes that gave up (all, if they agree).
// It issues no copy and no tensor-core work, so nothing is in flight when it
// returns and the context stays usable.
#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa {

namespace {

// How long the warp's barrier stays open: the lane that is told to give up looks
// at its flag after a millisecond of tries and 64 more.
constexpr uint64_t kOpenNs = 100000000;

__global__ void wait_probe_kernel(uint64_t limit_ns, unsigned *err)
{
    __shared__ uint64_t bar[2];
    __shared__ int give_up[32];
    if (threadIdx.x == 0) {
        tc::mbar_init(&bar[0], 1);
        tc::mbar_init(&bar[1], 1);
        tc::fence_mbar_init();
    }
    if (threadIdx.x < 32)
        give_up[threadIdx.x] = threadIdx.x == 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        volatile int never = 0;
        const bool out = threadIdx.x == 0 && !tc::mbar_wait(&bar[0], 0, &never, limit_ns);
        __syncwarp();
        const bool ok = tc::mbar_wait_warp(&bar[1], 0, &give_up[threadIdx.x]);
        const unsigned gave_up = __ballot_sync(0xffffffffu, !ok);
        if (out)
            report(err, CSA_ERR_TIMEOUT, K_PROBE, 0, __popc(gave_up));
    } else if (threadIdx.x == 32) {
        const uint64_t t0 = tc::global_ns();
        while (tc::global_ns() - t0 < limit_ns + kOpenNs)
            __nanosleep(10000);
        tc::mbar_arrive(&bar[1]);
    }
}

}  // namespace

cudaError_t launch_wait_probe(uint64_t limit_ns, unsigned *err, cudaStream_t s)
{
    wait_probe_kernel<<<1, 64, 0, s>>>(limit_ns, err);
    return cudaGetLastError();
}

}  // namespace csa
