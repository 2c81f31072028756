// warps.cuh -- what the warp-specialised kernels share: an elected lane, the whole warp's bounded
// wait, a ring's position, the fast power of two.
#pragma once

#include "common.cuh"

namespace rssm {

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// True on one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// The whole warp's bounded wait for phase `parity` of `bar`; false, with the CTA's abort
// flag set, when it ran out on any lane or another warp had given up.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort,
                                              uint64_t wait_ns, int32_t* dev_err) {
    const int w = mbar_wait_abortable(bar, parity, wait_ns, abort);
    if (__all_sync(0xffffffffu, w > 0)) return true;
    if (w == 0) {
        set_dev_err(dev_err, RSSM_DEVERR_TIMEOUT);
        *abort = 1;
    }
    __syncwarp();
    return false;
}

// A ring's slot and the parity of its present use.
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            parity ^= 1;
        }
    }
};

}  // namespace rssm
