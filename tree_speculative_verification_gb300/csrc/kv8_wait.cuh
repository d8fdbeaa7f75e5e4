// kv8_wait.cuh -- bounded waits of the 8-bit cache's attention kernel. Every
// wait is for other warps of the same CTA, or for copies and products that they
// or this warp have issued.
#pragma once
#include "ts_internal.cuh"

namespace ts {
namespace {

// A wait's tries. The hardware suspends each for up to 20 us, measured 4 us:
// 2 s, about kWaitCycles. (By count: a clock in this loop, which stands in every
// loop over tiles, or a look at a word that other warps set when they give up,
// costs code: 64 requests of 47 nodes, 56 heads, 1024 keys 211 and 208 us
// against 204.)
constexpr int kWaitTries = 1 << 19;

// Wait for a phase: false after kWaitTries.
__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t phase) {
#pragma unroll 1
    for (int i = 0; i < kWaitTries; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(phase), "r"(20000)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// The same by a whole warp, one verdict for every lane; a look first, which most waits in the tile loop need no more
// than (long-context case: 453 us against 462).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(phase)
                 : "memory");
    return __all_sync(~0u, ok) || __all_sync(~0u, wait1(bar, phase));
}

}  // namespace
}  // namespace ts
