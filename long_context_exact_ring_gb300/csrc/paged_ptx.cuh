// paged_ptx.cuh -- what the paged kernels need beside sm103_ptx.cuh: their bit of
// the status word, and a wait without a call.  A file of their own, as the ring
// kernels' recorded counters hold for their own sources as they are.
#pragma once

#include "sm103_ptx.cuh"

namespace ra {

// Device status bit, beside kStatusTimeout and kStatusAborted.
enum : uint32_t {
    kStatusBadPage = 4u,   // a page or slot outside its pool was met and not followed
};
static_assert((kStatusBadPage & (kStatusTimeout | kStatusAborted)) == 0, "a bit of its own");

// mbar_wait without a call: a kernel that moves registers between its warps
// (setmaxnreg) may call no function.
__device__ __forceinline__ bool mbar_wait_inline(uint32_t bar, uint32_t parity, const WaitCtl& w)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (*w.abort_flag) return false;
        if (globaltimer_ns() - t0 > w.limit_ns) {
            *w.abort_flag = 1;
            atomicOr(w.status, kStatusTimeout);
            return false;
        }
    }
}

}  // namespace ra
