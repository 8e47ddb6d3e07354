// selftest.cu -- the failure path of the kernels' bounded waits, run on purpose.
//
// Every wait in the library's kernels is on an mbarrier that a copy (or the
// other warp of a CTA) completes, and gives up after a time limit: the
// kernel then records FKV_DEVERR_TIMEOUT in the device error word and ends
// normally, so the context stays usable.  fkv_selftest_wait runs the three
// wait helpers those kernels use -- the spinning one of the computing warps,
// the sleeping one of a producer warp, and the one of tree and window
// attention (whose giving up also ends the block's other waits) -- on an mbarrier that
// nothing completes, so the path can be seen working on the GPU without a
// fault: the waits end after limit_ns, the error bit is set, later calls
// still work.  With `complete`, the block completes the barrier first and all
// waits must return at once.
#include "tree_attn.cuh"

namespace fkv {

constexpr int kSelftestAfter = 256;                   // waits after one that gave up
constexpr uint64_t kSelftestMaxNs = 10000000000ull;   // at most 10 s of waiting

__global__ void __launch_bounds__(96) selftest_wait_kernel(uint64_t limit_ns, int complete, uint32_t *err,
                                                            uint32_t *result) {
    __shared__ __align__(8) uint64_t bar_word;
    __shared__ int32_t dead;
    __shared__ uint32_t saw[3];                             // per warp: its wait saw the barrier complete
    const uint32_t bar = smem_u32(&bar_word);
    if (threadIdx.x == 0) {
        dead = 0;
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (complete && threadIdx.x == 0) mbar_arrive(bar);     // phase 0 completes
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    const uint64_t t0 = globaltimer_ns();
    bool ok;
    if (warp == 0) ok = mbar_wait_bounded(bar, 0, limit_ns);
    else if (warp == 1) ok = mbar_wait_bounded_sleep(bar, 0, limit_ns);
    else ok = tree_wait(bar, 0, &dead, err, static_cast<uint32_t>(limit_ns >> 10));
    if (warp == 2 && !ok) {
        const uint64_t t1 = globaltimer_ns();
        for (int i = 0; i < kSelftestAfter; ++i) ok |= tree_wait(bar, 0, &dead, err);
        const uint64_t t2 = globaltimer_ns();
        // given up before its limit (ticks of 1024 ns), or the block's other waits still wait: nine tests of 2 us each, and the
        // reading of the clock, are less than 50 us a wait
        if (t1 - t0 + 2048 < limit_ns || t2 - t1 > kSelftestAfter * 50000ull) ok = true;
    }
    if ((threadIdx.x & 31) == 0) {
        if (!ok) atomicOr(err, FKV_DEVERR_TIMEOUT);
        saw[warp] = ok ? 1u : 0u;
    }
    __syncthreads();
    if (threadIdx.x == 0 && result) {
        result[0] = saw[0] == saw[2] ? saw[0] : 2u;         // 2: the two waits that test without a pause do not agree
        result[1] = saw[1];
    }
}

}  // namespace fkv

using namespace fkv;

extern "C" fkv_status fkv_selftest_wait(uint64_t limit_ns, int32_t complete, uint32_t *result, void *stream) {
    if (limit_ns > kSelftestMaxNs) return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    if (!err) return FKV_ERR_CUDA;
    selftest_wait_kernel<<<1, 96, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns, complete ? 1 : 0, err, result);
    return cudaGetLastError() == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
