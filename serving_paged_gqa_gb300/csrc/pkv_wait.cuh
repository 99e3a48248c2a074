// Bounded waits on mbarriers: every wait of a kernel ends, with a status bit where it gave up.
#pragma once

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

struct WaitCtx {
    volatile int* abort_flag;
    uint32_t* status;
    uint64_t limit_ns = kWaitLimitNs;
};

__device__ __forceinline__ void raise_status(uint32_t* status, uint32_t bits) { atomicOr(status, bits); }

// Warp-collective bounded wait on an mbarrier phase. Returns false if the wait gave up (abort or timeout).
// try_wait suspends the thread until the phase completes or a short hardware time slice ends; the abort flag and
// the global timer are consulted only every kPollEvery slices.
constexpr uint32_t kPollEvery = 256;

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (it % kPollEvery == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            const bool stop = (*ctx.abort_flag != 0) || (now - t0 > ctx.limit_ns);
            if (__any_sync(0xffffffffu, stop)) {
                if ((threadIdx.x & 31) == 0 && *ctx.abort_flag == 0) {
                    *ctx.abort_flag = 1;
                    raise_status(ctx.status, PKV_STATUS_TIMEOUT);
                }
                return false;
            }
        }
    }
}

// The same for one thread of a warp.
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (it % kPollEvery == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (*ctx.abort_flag != 0 || now - t0 > ctx.limit_ns) {
                if (*ctx.abort_flag == 0) {
                    *ctx.abort_flag = 1;
                    raise_status(ctx.status, PKV_STATUS_TIMEOUT);
                }
                return false;
            }
        }
    }
}

// Bounded wait that ignores the abort flag (used to drain a warp's own copies before it returns).
__device__ __forceinline__ void warp_drain(uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it) {
        if (it % kPollEvery == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > kWaitLimitNs)) return;
        }
    }
}

}  // namespace pkv
