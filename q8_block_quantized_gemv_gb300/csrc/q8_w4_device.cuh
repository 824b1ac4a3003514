// Device pieces shared by the kernels over 4-bit weights: codes to exact bf16, scales, bulk copies and bounded waits.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q8_w4.h"

namespace q8 {

// Rows 8t + 2P and 8t + 2P + 1 of a word as the exact bf16 pair (c - z) / 64.  The byte v under a zero exponent is the bf16
// number v * 2^-133 (subnormals and the binade after them are one arithmetic progression), so four bits where they stand,
// in the low or the high half of the byte, are c * 2^-133 or c * 2^-129: one packed fma times 2^127 or 2^123 less z / 64
// is exact (|c - z| <= 127 has 7 bits).  Eight codes cost one shift, four ands and four fmas; putting each pair under the
// exponent of 128 and subtracting takes three shifts.  `zero` holds -z / 64 twice.
template <int P> __device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t zero) {
    const uint32_t v = (P >= 2 ? w >> 8 : w) & (P & 1 ? 0x00F000F0u : 0x000F000Fu);
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(P & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(zero));
    return d;
}
constexpr float kW4Unit = 64.0f;            // what the products are short of
constexpr uint32_t kW4Eight = 0xBE00BE00u;  // -8 / 64
__device__ __forceinline__ uint32_t w4_zero(unsigned char z) {  // 2 - (128 + z) / 64
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"((0x4300u | z) * 0x10001u), "r"(0xBC80BC80u), "r"(0x40004000u));
    return d;
}

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
constexpr long long kW4Patience = 4000000000ll;  // clocks
__device__ __forceinline__ bool w4_look(uint64_t *bar, unsigned parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(w4_smem(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for the phase of the given parity, some two seconds at most (of the SM's clock: reading the global timer first takes
// 650 clocks); false when that time ran out.
__device__ __forceinline__ bool w4_wait(uint64_t *bar, unsigned parity) {
    if (w4_look(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (w4_look(bar, parity)) return true;
    } while (clock64() - t0 < kW4Patience);
    return false;
}

}  // namespace q8
