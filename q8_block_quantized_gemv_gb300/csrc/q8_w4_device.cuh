// Device pieces shared by the kernels over 4-bit weights: codes to exact bf16, scales, bulk copies and bounded waits.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q8_w4.h"

namespace q8 {

// Rows 8t + 2p and 8t + 2p + 1 of a word as the bf16 pair 128 + c: bf16's mantissa unit at 128 is 1, so the four bits go
// under the exponent as they are.
template <int P> __device__ __forceinline__ uint32_t w4_raised(uint32_t w) {
    uint32_t d;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(d) : "r"(P ? w >> (4 * P) : w));
    return d;
}
// ... less the pair 128 + z: c - z, exact (|c - z| <= 127 has at most 7 bits).
template <int P> __device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t raised_zero) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w4_raised<P>(w)), "r"(raised_zero));
    return d;
}
constexpr uint32_t kRaisedEight = 0x43084308u;  // the pair 128 + 8
__device__ __forceinline__ uint32_t w4_raised_zero(unsigned char z) { return (0x4300u | z) * 0x10001u; }

// A scale's value: bf16 is the top half of an fp32.
__device__ __forceinline__ float w4_scale(uint16_t s, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)s << 16) : __half2float(__ushort_as_half(s));
}

__device__ __forceinline__ uint32_t w4_smem(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void w4_bar_init(uint64_t *bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(w4_smem(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void w4_bar_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void w4_arrive_tx(uint64_t *bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(w4_smem(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void w4_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(w4_smem(bar)) : "memory");
}
// Bytes of global memory to shared memory; both 16-byte aligned, a multiple of 16.
__device__ __forceinline__ void w4_copy(void *dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     w4_smem(dst)),
                 "l"(src), "r"(bytes), "r"(w4_smem(bar))
                 : "memory");
}
__device__ __forceinline__ bool w4_look(uint64_t *bar, unsigned parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(w4_smem(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for the phase of the given parity, two seconds at most; false when that time ran out.
__device__ __noinline__ bool w4_wait_long(uint64_t *bar, unsigned parity);
__device__ __forceinline__ bool w4_wait(uint64_t *bar, unsigned parity) {
    return w4_look(bar, parity) || w4_wait_long(bar, parity);
}
__device__ __noinline__ bool w4_wait_long(uint64_t *bar, unsigned parity) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (unsigned n = 1;; ++n) {
        if (w4_look(bar, parity)) return true;
        if ((n & 63u) == 0) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (t - t0 > 2000000000ull) return false;
        }
    }
}

}  // namespace q8
