// selftest.cu -- self-test of the bounded waits that every kernel of the
// library uses, run as a call of its own (no data, no copies, no tensor
// memory).
//
// One CTA of four warps and an mbarrier for each on which nothing ever arrives.
// Warp 0 waits with mbar_wait_bounded (limit limit_ns) and must give up: it
// sets PKV_FLAG_WAIT_TIMEOUT and the CTA's abort flag. The others must stop
// because of the abort flag, soon after warp 0: warp 1 waits with
// mbar_wait_or_abort and a limit 100 times longer, warp 2 with
// mbar_warp_wait_watched and one lane of warp 3 with mbar_wait_watched, which
// have no limit of their own. Warp 0's waiting time goes to elapsed_ns[0], the
// longest of the others' to elapsed_ns[1]. All waits end by construction (the
// global timer bounds warp 0's, whose flag ends the others), so the call cannot
// hang the GPU.
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

__global__ void __launch_bounds__(128, 1) selftest_wait_kernel(uint64_t limit_ns, int32_t* err, uint64_t* elapsed_ns) {
    __shared__ __align__(8) uint64_t bars[4];
    __shared__ int abort_flag;
    __shared__ uint64_t elapsed[4];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars[i]), 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int* ab = &abort_flag;
    const uint64_t t0 = global_ns();
    if (warp == 0) {
        const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bars[0]), 0, limit_ns));
        if (!got && lane == 0) {
            *ab = 1;
            flag_error(err, PKV_FLAG_WAIT_TIMEOUT);
        }
    } else if (warp == 1) {
        (void)__all_sync(0xffffffffu, mbar_wait_or_abort(smem_u32(&bars[1]), 0, ab, 100 * limit_ns));
    } else if (warp == 2) {
        (void)mbar_warp_wait_watched(smem_u32(&bars[2]), 0, ab);
    } else {
        if (lane == 0) (void)mbar_wait_watched(smem_u32(&bars[3]), 0, ab);
        __syncwarp();
    }
    if (lane == 0) elapsed[warp] = global_ns() - t0;
    __syncthreads();
    if (threadIdx.x == 0) {
        elapsed_ns[0] = elapsed[0];
        elapsed_ns[1] = max(elapsed[1], max(elapsed[2], elapsed[3]));
    }
}

}  // namespace

cudaError_t launch_selftest_wait(uint64_t limit_ns, int32_t* err, uint64_t* elapsed_ns, cudaStream_t s) {
    selftest_wait_kernel<<<1, 128, 0, s>>>(limit_ns, err, elapsed_ns);
    return cudaGetLastError();
}

}  // namespace pkv
