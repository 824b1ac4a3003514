// q8_attn_prefill: causal attention of a chunk of new tokens over the paged cache, on the 5th-generation tensor cores.
//
// 4 dim flops a visible (query row, key) pair against 4 dim bytes a key: from some hundred rows the tensor cores bound
// it, so the kernel is built around keeping them fed.  A work item is two 128-row query tiles of one cache head -- the
// tokens' rows with the heads that share the cache head packed beside each other, whole tokens to a tile, so shared
// heads fill tiles as tokens do -- that take turns: while the softmax warps work on one tile's scores, the tensor cores
// compute the other's.  For each 128-key tile:
//     S = Q K^T (tcgen05.mma, both operands in shared memory, fp32 S in tensor memory)
//     P = 2^(S scale log2(e) - m), rounded to 16 bits, written over S in tensor memory
//     O += P V (P read from tensor memory, V from shared memory, fp32 O in tensor memory)
// with a running m that only moves when weights against it grow past what their type and the sums take (2^15 in fp16,
// 2^32 in bf16; then the row's O is rescaled in place).  The weights multiply V with 16 bits, as that product wants them: bf16's
// 8 significant ones over a bf16 cache, whose range they share; over a Q8_0 cache fp16's 11 down to 2^-14 of the row's
// largest and fewer below.  Their sum is fp32.
//
// Warps: 0-3 and 4-7 the softmax of tiles A and B, one row a thread; 8 issues the MMAs; 9 requests keys and values;
// the rest load Q and prepare values:
//   bf16 cache: K and V tiles arrive by TMA straight in the MMA's 128-byte swizzle; the helpers (two warps) look through
//     the V tiles that some row does not see whole, and clear what nobody sees;
//   Q8_0 cache: codes and scales arrive by bulk copies, and the helpers (six warps) turn them into fp16 operands,
//     code * scale / unit with one power of two `unit` a tile, as the softmax threads do Q with one a row: 11 significant
//     bits for scales down to 2^-21 of the tile's largest (for values, of the largest so far), fewer below.  For scores that is
//     what fp32 sums of the largest keep.  An output block so small beside the largest values that it may have lost bits is
//     computed again in fp32 by its row's thread (a rare, slow walk).  (bf16 operands would cost the scores and values 8-bit
//     roundings: measured 0.0029 against 0.0017 relative error.)
//
// The tiles of all items are one list, cut into equal spans, one for each CTA (one CTA per SM); an item that crosses
// spans leaves fp32 parts in the workspace, which the CTA that arrives last adds in span order.
//
// A weight of zero times a value that is not finite is NaN, so a value that one row sees and another of its tile does
// not must not reach the MMA unless finite: such values are cleared, and the rows that do see them get them added at
// the end (a rare, slow walk).
//
// Every wait is bounded (about two seconds); one that runs out records a fault, and the CTA drains and returns.
//
// Measured, 32 heads of 128 over 8 cache heads: a prompt of 8,192 rows 351 us over a bf16 cache = 1.56 PFLOP/s (80% of a
// large bf16 product's rate: the MMAs wait for the softmax some of the time, 68% of the tensor pipe's cycles are taken),
// 581 us over a Q8_0 cache, where a tile goes through five hands (codes, conversion, S, softmax, O) and nothing is full:
// 27% of the tensor pipe's cycles and 38% of the issue slots in a chunk of 509 rows, which takes 68 us (1.5 us more with
// four conversion warps; as long with the conversion finished in registers before its operand's place is free, or with
// the values' place given back before the keys').
// 512 rows after 4,096 tokens, 32 cache heads: 51 us.  A call's fixed part is 11 us: the cut of the list 2, the first Q
// and keys 3, a join 4 and the launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "q8_attn.h"
#include "q8_device.cuh"

namespace q8 {
namespace {

constexpr int kTile = 128;   // keys of a tile, and rows of a query tile
constexpr int kRows = 256;   // query rows of an item
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kHelpWarp = 10;
constexpr unsigned kTmemColumns = 512;
constexpr unsigned kSteps = 16;  // a power of two above 10 (see Control::step)
constexpr uint32_t kColP = 64;   // the weights (16 bits) over the upper half of their scores
constexpr unsigned kFaultAttnWait = 8u;

__device__ unsigned int g_attn_fault = 0;

template <int D, bool Q8> struct Cfg {
    static constexpr int kSub = D / 64;                    // 128-byte-wide column blocks of an operand
    // Tensor memory: score buffers of 128 columns, then the tiles' O.  With two buffers a tile's next scores follow its
    // last weights, which lie over the last scores.  Heads of 64 leave room for a third: the jobs A, B, A, B ... take the
    // buffers in turn, and a tile's next scores are there before its softmax is done with the last.
    static constexpr int kBufs = D == 64 ? 3 : 2;
    static constexpr uint32_t kColO = kBufs * 128;
    static constexpr int kOp = kSub * kTile * 128;         // bytes of a K, V or Q operand tile
    static constexpr int kRaw = Q8 ? kTile * D + kTile * (D / 32) * 4 : 0;
    static constexpr int kSlots = Q8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int kRawSlots = Q8 ? (D == 128 ? 3 : 4) : 0;
    static constexpr int kHelpers = Q8 ? 6 : 2;            // warps
    static constexpr int kThreads = 32 * (kHelpWarp + kHelpers);
    // What an item costs beside its tiles, in tiles: loading Q, the pipe's fill and drain, the epilogue.  Without it the
    // CTAs of a long prompt's first rows, 44 short items each, took 835,000 clocks where the others took 740,000.  2, 3, 4, 5
    // and 6, heads of 128, 32 over 8: a prompt of 4,096 rows takes 121, 116, 116, 119 and 119 us, under a window of 1,024 87
    // each, 512 rows of 9 requests 44, 41, 41, 41 and 41; over a Q8_0 cache 220, 204, 193, 195 and 196, 138, 136, 136, 139 and
    // 139, 61, 56, 56, 58 and 58.  Heads of 64 are alike.  Prompts of full heads, 32 over 32, would have more (bf16 145, 134,
    // 129, 128 and 130; Q8_0 260, 246, 232, 216 and 214), their 512 rows of 9 requests less (70, 71, 72, 73 and 75; 105, 97, 98,
    // 98 and 99).
    static constexpr int kItemCost = Q8 ? 4 : 3;
    static constexpr int kRing = 2 * kOp;                  // after Q's two tiles
    static constexpr int kRawAt = kRing + kSlots * kOp;
    static constexpr int kCtl = kRawAt + kRawSlots * kRaw;
    static constexpr int kSmem = kCtl + (Q8 ? 4096 : 2048);
    static_assert(kSmem <= 226 * 1024, "");
    // The list of items is cut before the operands come, in their place: the requests' sums of query tiles (R + 1), then,
    // for up to kCopied requests, copies of row_start (R + 1) and lens (R), which otherwise are read where they are.
    static constexpr int kCopied = (kCtl / 4 - 2) / 3;
    static_assert((Q8_MAX_REQUESTS + 1) * 4 <= kCtl && (3 * kCopied + 2) * 4 <= kCtl, "the list ends before the control block");
};

// Control block in shared memory.
template <int D, bool Q8> struct Control {
    using C = Cfg<D, Q8>;
    // Operands: landed, usable.  Over a Q8_0 cache `ready` goes by place of the ring.  Over a bf16 cache both go by key
    // tile, at most five of which are on their way: keys are full[n % 5], values full[5 + n % 5] and, after the helpers,
    // ready[n % 5].  So a barrier's every phase has the same waiters: one that places shared between keys, which the
    // helpers have no business with, and values could complete twice before a helper had looked.
    uint64_t full[10], ready[10];
    // A step's MMAs are done, and with them what it used is free.  Who waits for a step must not find its barrier a whole
    // turn further on: the loads wait for what a place held up to five tiles ago (ten places), and in items of one tile,
    // whose first scores are a step of their own, the MMAs are up to ten steps past that by then.
    uint64_t step[kSteps];
    uint64_t raw_full[4], raw_empty[4];        // raw ring (Q8_0)
    uint64_t q_raw, q_full, q_empty, drain;  // q_raw: landed, before the conversion (Q8_0)
    uint64_t s_full[3], p_ready[3];            // by score buffer: scores computed, weights written
    uint64_t o_full[2], joined, decided;
    uint64_t idle;  // a segment in which tile B has no rows: its warps have seen the end of A's
    // Of key tile number n of this CTA at n & 7 (no role is more than five tiles behind the requests):
    // its first place, and bits: which 16-token groups lie on a page (0-7); whether some row of tile A (8) or B (9) does
    // not see all of it
    int2 tile[8];
    float unit[2][8];   // Q8_0: log2 of the keys' and the values' unit
    uint32_t tmem;
    int abort, last;
    int poison, lost;   // values were cleared; or are below fp16's normal range (Q8_0)
    int first_r, first_qt;
    long long first_start;
    long long scan[20];
};
static_assert(sizeof(Control<128, true>) <= 4096 && sizeof(Control<128, false>) <= 2048, "");

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t *bar, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ void bar_arrive_tx(uint64_t *bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, unsigned parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(saddr(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Wait for a phase of `bar`; false when the CTA is aborting, or after about two seconds (which starts the abort).
__device__ __forceinline__ bool bar_wait(uint64_t *bar, unsigned parity, volatile int *abort) {
    uint64_t t0 = 0;  // the timer is slow to read: looked at once in a long while
    for (unsigned n = 1;; ++n) {
        if (bar_try(bar, parity)) return true;
        if ((n & 255u) == 0) {
            if (*abort) return false;
            const uint64_t t = now_ns();
            if (!t0) t0 = t;
            if (t - t0 > 2000000000ull) {
                *abort = 1;
                atomicOr(&g_attn_fault, kFaultAttnWait);
                return false;
            }
        }
    }
}
// The same for a whole warp, one answer for all lanes; the first look is a few instructions.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, unsigned parity, volatile int *abort) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " vote.sync.all.pred q, p, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(done)
        : "r"(saddr(bar)), "r"(parity)
        : "memory");
    return done ? true : __all_sync(0xffffffffu, bar_wait(bar, parity, abort));
}
// Whether three phases are complete: the looks overlap.
__device__ __forceinline__ bool look3(uint64_t *b0, unsigned p0, uint64_t *b1, unsigned p1, uint64_t *b2, unsigned p2) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p, q, r;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n"
        " and.pred p, p, q;\n and.pred p, p, r;\n vote.sync.all.pred q, p, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(done)
        : "r"(saddr(b0)), "r"(p0), "r"(saddr(b1)), "r"(p1), "r"(saddr(b2)), "r"(p2)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar))
                 : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle (layout 2).  K-major operands (Q, K): rows of 128 bytes, groups of
// 8 rows 1024 bytes apart.  MN-major (V): 64 values of dim in 128 bytes, groups of 8 keys 1024 bytes apart, the next
// 64 values `lead` bytes on.
constexpr uint64_t desc128_high = ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
__device__ __forceinline__ uint32_t desc128_low(uint32_t addr, uint32_t lead) {
    return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
// One lane of a converged warp.  The warp that issues MMAs runs its loop with all lanes, so that addresses and
// descriptors stay in uniform registers, and picks a lane for the instructions themselves: inside a one-lane branch
// each MMA moved its operands over anew, 67 to 85 clocks of issue for 64 of work.
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
// A value that all lanes hold, so that the compiler knows it.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Descriptors come as their low words; the high ones are desc128's constant.
constexpr uint32_t kDescHigh = (uint32_t)(desc128_high >> 32);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n"
        " mov.b64 db, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max32(const uint32_t (&v)[32]) {
    float a = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
    float b = max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
#pragma unroll
    for (int k = 6; k < 30; k += 4) {
        a = max3(a, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        b = max3(b, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
    }
    return max3(a, b, fmaxf(__uint_as_float(v[30]), __uint_as_float(v[31])));
}
// The lowest n of 32 bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ void bulk(uint32_t dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(saddr(bar))
                 : "memory");
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar))
        : "memory");
}

// 32 values of an output row; wide: 32-byte stores, whole sectors (every row 32-byte aligned).
__device__ __forceinline__ void store_row(uint16_t *p, const float (&o)[32], bool wide) {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = bf16x2(o[2 * k], o[2 * k + 1]);
    if (wide) {
#pragma unroll
        for (int k = 0; k < 16; k += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 2 * k), "r"(w[k]),
                         "r"(w[k + 1]), "r"(w[k + 2]), "r"(w[k + 3]), "r"(w[k + 4]), "r"(w[k + 5]), "r"(w[k + 6]),
                         "r"(w[k + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<uint4 *>(p + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
    }
}

__device__ __forceinline__ int2 tile_info(const int2 *p) {
    int2 v;
    asm volatile("ld.shared.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(saddr(p)) : "memory");
    return v;
}

// A row of Q to fp16, in place, by one thread: times a power of two that takes its largest magnitude to [2^9, 2^10), which
// the result undoes.  Out of line, for the registers of the softmax's loop.
template <int D> __device__ __noinline__ float row_to_half(unsigned char *row, int swizzle) {
    uint4 *at = reinterpret_cast<uint4 *>(row);
    uint32_t mx = 0u;
#pragma unroll 1  // short code: what a CTA runs once or a few times waits for its instructions
    for (int c0 = 0; c0 < D / 8; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = at[(c0 / 8) * kTile * 8 + (c ^ swizzle)];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu)),
                          __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu));
    }
    const int ex = min(max((int)(max(mx & 0xFFFFu, mx >> 16) >> 7), 1), 254), up = min(127 + 9 - ex, 126);
    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll 1
    for (int c0 = 0; c0 < D / 8; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = at[(c0 / 8) * kTile * 8 + (c ^ swizzle)];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = f16x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
            at[(c0 / 8) * kTile * 8 + (c ^ swizzle)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    return __uint_as_float((uint32_t)(127 - up) << 23);
}

// The scores at ts that their row does not see become -inf in place: it sees columns c_lo .. c_hi and 0 .. c_sink - 1
// of the 16-column groups that have a bit.
__device__ __forceinline__ void hide_scores_here(uint32_t ts, int c_hi, int c_lo, int c_sink, unsigned groups) {
    // By 32 columns: most are seen by all 32 rows of the warp, or by none.
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t see = bits_below(c_hi + 1 - c0) & (~bits_below(c_lo - c0) | bits_below(c_sink - c0));
        see &= ((groups >> (c0 / 16) & 1u) ? 0xFFFFu : 0u) | ((groups >> (c0 / 16 + 1) & 1u) ? 0xFFFF0000u : 0u);
        if (__all_sync(0xffffffffu, see == ~0u)) continue;
        uint32_t v[32];
        if (__any_sync(0xffffffffu, see != 0u)) {
            tm_ld32(ts + c0, v);
            tm_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = (see >> k & 1u) ? v[k] : 0xFF800000u;
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0xFF800000u;
        }
        tm_st32(ts + c0, v);
    }
    tm_wait_st();
}

// Over a bf16 cache, where the softmax's loop is what the tensor cores wait for, as a function of its own, which leaves the
// loop to the tiles without any; over a Q8_0 cache inline.  Own and inline, 4,096 rows, 32 heads over 8, without and with a
// window of 1,024: bf16, heads of 128 117 and 120 us (window 87 and 88), heads of 64 91 and 95 (70 and 69); Q8_0, heads of
// 128 195 and 194 (137 and 136), heads of 64 140 and 139 (102 and 100).
__device__ __noinline__ void hide_scores_call(uint32_t ts, int c_hi, int c_lo, int c_sink, unsigned groups) {
    hide_scores_here(ts, c_hi, c_lo, c_sink, groups);
}
template <bool Q8>
__device__ __forceinline__ void hide_scores(uint32_t ts, int c_hi, int c_lo, int c_sink, unsigned groups) {
    if (Q8) hide_scores_here(ts, c_hi, c_lo, c_sink, groups);
    else hide_scores_call(ts, c_hi, c_lo, c_sink, groups);
}
// A row's largest score, and n columns of a row times f: the rare part of a softmax step, out of its loop too.
__device__ __noinline__ float max_score(uint32_t ts) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 64) {
        uint32_t v[2][32];
        tm_ld32(ts + c0, v[0]);
        tm_ld32(ts + c0 + 32, v[1]);
        tm_wait_ld();
        mx = max3(mx, max32(v[0]), max32(v[1]));
    }
    return mx;
}
__device__ __noinline__ void scale_columns(uint32_t to, int n, float f) {
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += 32) {
        uint32_t o[32];
        tm_ld32(to + c0, o);
        tm_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
        tm_st32(to + c0, o);
    }
}

// a / b for a >= 0, b > 0: a 64-bit division is some 100 instructions, and hardly ever needed.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

struct PrefillArgs {
    AttnArgs a;
    int run;         // consecutive tokens of a tile that lie on one page wherever they start: gcd(page_size, 128)
    int tile_tokens; // tokens of a query tile: 128 / group
    int item_cost;   // in key tiles
};

// Two query tiles of one cache head: tokens tok0 .. tok0 + tokens - 1 of request r, tile_tokens to a tile; row y of a tile
// is token y / group, head y % group of those that share the cache head.  The item's keys are a list cut into tiles: the
// first `sinks` places hold the sinks (whole runs), the others keys from the window's first run on, place v key v + jump.
// (Whole tiles for the sinks and for the window, from multiples of 128, took 61.5 us for a prompt of 4097 rows, window
// 1024, 4 sinks; the window from its first run 59; the one list 54.  Calls without a window take 1 to 2 us longer with it:
// a chunk of 512 rows 50 and 51, a prompt of 8192 rows 346 and 348.)  In the list of all items an item takes item_cost + n
// places, the tiles last.
struct Item {
    int r, qt, h;
    long long start;  // of its tiles in the list, the fixed cost behind it
    int row0, all, pos0;  // the request's first row, its rows, the position of its first row
    int tok0, tokens;
    int p_min, p_max, end, lo, sinks, jump, n;

    __device__ __forceinline__ int key(int v) const { return v < sinks ? v : v + jump; }
    // Whether some row of the item does not see all of the tile from place v0, pages aside.
    __device__ __forceinline__ bool partial(const AttnArgs &a, int v0) const { return partial(a, v0, p_min, p_max); }
    // The same for its rows at positions p0 .. p1.
    __device__ __forceinline__ bool partial(const AttnArgs &a, int v0, int p0, int p1) const {
        const int last = key(v0 + kTile - 1);
        if (last >= end || last > p0) return true;
        if (!a.window) return false;
        if (v0 < sinks && min(sinks, v0 + kTile) > a.sinks) return true;  // a run that sinks end inside
        return last >= a.sinks && p1 - key(max(v0, sinks)) >= a.window;
    }
};
// Key tiles that rows at positions p_min .. p_max visit.
__device__ __forceinline__ void span_of(const PrefillArgs &pa, Item &x) {
    const AttnArgs &a = pa.a;
    x.end = min(max(x.p_max + 1, 0), a.width * a.page_size);
    x.lo = a.window ? min(max(max(x.p_min, 0) - a.window + 1, 0), x.end) : 0;  // a position may be negative, a window 2^31 - 1
    const int ul = x.lo & -pa.run, sinks = a.window ? min(a.sinks, ul) : 0;
    x.sinks = (sinks + pa.run - 1) & -pa.run;  // not past ul, which is whole runs too
    x.jump = sinks == a.sinks ? ul - x.sinks : 0;
    if (!x.jump) x.sinks = 0;  // no gap: one stretch of keys
    x.n = (max(x.end - x.jump, 0) + kTile - 1) / kTile;
}
__device__ __forceinline__ void request_of(const int *row_start, const int *lens, int rows, Item &x) {
    const int t0 = min(max(row_start[x.r], 0), rows), t1 = min(max(row_start[x.r + 1], t0), rows);
    x.row0 = t0;
    x.all = t1 - t0;
    x.pos0 = max(lens[x.r], 0) - x.all;
}
__device__ __forceinline__ void request_of(const AttnArgs &a, Item &x) { request_of(a.row_start, a.lens, a.rows, x); }
__device__ __forceinline__ int q_tiles(const PrefillArgs &pa, int tokens) {
    return (tokens + 2 * pa.tile_tokens - 1) / (2 * pa.tile_tokens);
}
__device__ __forceinline__ void q_tile_of(const PrefillArgs &pa, Item &x) {
    x.tok0 = x.qt * 2 * pa.tile_tokens;
    x.tokens = min(2 * pa.tile_tokens, x.all - x.tok0);
    x.p_min = x.pos0 + x.tok0;
    x.p_max = x.p_min + x.tokens - 1;
    span_of(pa, x);
}
__device__ __forceinline__ long long cost_of(const PrefillArgs &pa, const Item &x) {
    return x.n ? x.n + pa.item_cost : 0;
}
__device__ __forceinline__ void next_item(const PrefillArgs &pa, Item &x) {
    x.start += x.n + pa.item_cost;
    if (++x.h < pa.a.kv_heads) return;
    x.h = 0;
    do {
        if (++x.qt >= q_tiles(pa, x.all)) {
            do {
                if (++x.r >= pa.a.R) return;  // never reached: the walk ends within the list
                request_of(pa.a, x);
            } while (x.all == 0);
            x.qt = 0;
        }
        q_tile_of(pa, x);
    } while (x.n == 0);
}

// Whether the row at position p sees key j (pages aside).
__device__ __forceinline__ bool sees(const AttnArgs &a, int p, int j) {
    return j <= p && (!a.window || p - j < a.window || j < a.sinks);
}

// Values that are not finite in tiles that only some rows see were cleared before the MMA; add them to the rows that
// do see them.  o: 32 of the row's values from column c0.
template <int D, bool Q8>
__device__ __noinline__ void add_nonfinite(const AttnArgs &a, const Item it, int i0, int i1, int p, int c0, float *o) {
    for (int i = i0; i < i1; ++i) {
        const int v0 = i * kTile;
        for (int c = 0; c < kTile; ++c) {
            const int j = it.key(v0 + c);
            if (j >= it.end) break;
            if (!sees(a, p, j)) continue;
            const int page = a.table[(size_t)it.r * a.pitch + j / a.page_size];
            if (page < 0 || page >= a.pages) continue;
            // only tiles that some row does not see whole were cleared
            bool cleared = it.partial(a, v0);
            for (int b = 0; b < kTile / 16 && !cleared; ++b) {
                const int pg = a.table[(size_t)it.r * a.pitch + it.key(v0 + 16 * b) / a.page_size];
                cleared = pg < 0 || pg >= a.pages;
            }
            if (!cleared) break;
            const long long at =
                (long long)page * a.page_stride + ((long long)it.h * a.page_size + j % a.page_size) * D + c0;
            for (int d = 0; d < 32; ++d) {
                float v;
                if (Q8) v = (float)static_cast<const signed char *>(a.v)[at + d] * a.vs[(at + d) / 32];
                else v = __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.v)[at + d] << 16);
                if (!(fabsf(v) < INFINITY)) o[d] += v;
            }
        }
    }
}

// 32 of a row's values from column c0 once more, in fp32 from the Q8_0 cache itself, where none is as large as `least`.  The
// row: token tok, head gh of those that share the cache head; M: its maximum as the softmax has it; o: times inv.
template <int D>
__device__ __noinline__ void attend_again(const AttnArgs &a, const Item it, int i0, int i1, int tok, int gh, float M, float inv,
                                          float least, int c0, float *o) {
    float most = 0.0f;
    for (int d = 0; d < 32; ++d) most = fmaxf(most, fabsf(o[d]));
    if (!(most < least) || isnan(o[0])) return;
    const int p = it.p_min + tok;
    const uint16_t *q = a.q + (size_t)(it.row0 + it.tok0 + tok) * a.ldq + (it.h * a.group + gh) * D;
    for (int d = 0; d < 32; ++d) o[d] = 0.0f;
    for (int v = i0 * kTile; v < i1 * kTile; ++v) {
        const int j = it.key(v);
        if (j >= it.end) break;
        if (!sees(a, p, j)) continue;
        const int page = a.table[(size_t)it.r * a.pitch + j / a.page_size];
        if (page < 0 || page >= a.pages) continue;
        const long long at = (long long)page * a.page_stride + ((long long)it.h * a.page_size + j % a.page_size) * D;
        const float scale = a.vs[(at + c0) / 32];
        if (!(fabsf(scale) < INFINITY)) continue;  // add_nonfinite's
        float s = 0.0f;
        for (int b = 0; b < D / 32; ++b) {
            float sum = 0.0f;
            for (int d = 32 * b; d < 32 * b + 32; ++d)
                sum = fmaf(__uint_as_float((uint32_t)q[d] << 16), (float)static_cast<const signed char *>(a.k)[at + d], sum);
            s = fmaf(sum, a.ks[at / 32 + b], s);
        }
        const float w = ex2(s * (a.scale * kLog2e) - M) * inv * scale;
        for (int d = 0; d < 32; ++d) o[d] = fmaf(w, (float)static_cast<const signed char *>(a.v)[at + c0 + d], o[d]);
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs pa, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap) {
    using C = Cfg<D, Q8>;
    const AttnArgs &a = pa.a;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control<D, Q8> &ctl = *reinterpret_cast<Control<D, Q8> *>(smem + C::kCtl);
    volatile int *abort = &ctl.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = (int)uniform(tid >> 5);
    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            bar_init(&ctl.ready[i], C::kHelpers);
        }
        for (int i = 0; i < 10; ++i) bar_init(&ctl.full[i], 1);
        for (unsigned i = 0; i < kSteps; ++i) bar_init(&ctl.step[i], 1);
        for (int i = 0; i < C::kRawSlots; ++i) {
            bar_init(&ctl.raw_full[i], 1);
            bar_init(&ctl.raw_empty[i], C::kHelpers);
        }
        bar_init(&ctl.q_raw, 1);
        bar_init(&ctl.q_full, Q8 ? 8 : 1);
        bar_init(&ctl.q_empty, 1);
        bar_init(&ctl.drain, 1);
        bar_init(&ctl.joined, 8);
        bar_init(&ctl.decided, 1);
        for (int i = 0; i < C::kBufs; ++i) {
            bar_init(&ctl.s_full[i], 1);
            bar_init(&ctl.p_ready[i], 4);
        }
        for (int i = 0; i < 2; ++i) bar_init(&ctl.o_full[i], 1);
        bar_init(&ctl.idle, 4);
        ctl.abort = 0;
        ctl.poison = ctl.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&ctl.tmem)),
                     "r"(kTmemColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the list and this CTA's span: query tiles of each request, then key tiles of each query tile ----
    int *qsum = reinterpret_cast<int *>(smem);  // [R + 1] exclusive sums (the operands come later)
    constexpr int T = C::kThreads;
    long long total = 0, b0 = 0, b1 = 0, span = 1;
    {
        const int *starts = a.row_start, *lens = a.lens;
        if (a.R <= C::kCopied) {  // what follows looks at them over and over
            int *s = qsum + a.R + 1, *l = s + a.R + 1;
            for (int r = tid; r <= a.R; r += T) {
                s[r] = a.row_start[r];
                if (r < a.R) l[r] = a.lens[r];
            }
            starts = s;
            lens = l;
        }
        __syncthreads();
        const int each = (a.R + T - 1) / T, ra = min(a.R, tid * each), rb = min(a.R, ra + each);
        Item x;
        int mine = 0;
        for (x.r = ra; x.r < rb; ++x.r) {
            request_of(starts, lens, a.rows, x);
            mine += q_tiles(pa, x.all);
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) ctl.scan[warp] = upto;
        __syncthreads();
        int before = upto - mine, tiles = 0;
        for (int w = 0; w < T / 32; ++w) {
            if (w < warp) before += (int)ctl.scan[w];
            tiles += (int)ctl.scan[w];
        }
        for (x.r = ra; x.r < rb; ++x.r) {
            request_of(starts, lens, a.rows, x);
            qsum[x.r] = before;
            before += q_tiles(pa, x.all);
        }
        if (tid == 0) qsum[a.R] = tiles;
        __syncthreads();
        // this thread's query tiles of all of them
        const int qe = (tiles + T - 1) / T, qa = min(tiles, tid * qe), qb = min(tiles, qa + qe);
        long long keys = 0;
        auto seek = [&](int q) {  // x at query tile q of the list
            int lo = 0, hi = a.R - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (qsum[mid] <= q) lo = mid; else hi = mid - 1;
            }
            x.r = lo;
            x.qt = q - qsum[lo];
            request_of(starts, lens, a.rows, x);
            q_tile_of(pa, x);
        };
        for (int q = qa; q < qb; ++q) {
            seek(q);
            keys += cost_of(pa, x);
        }
        long long sum = keys;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        __syncthreads();  // every thread has read scan
        if (lane == 31) ctl.scan[warp] = sum;
        __syncthreads();
        long long ahead = sum - keys;
        for (int w = 0; w < T / 32; ++w) {
            if (w < warp) ahead += ctl.scan[w];
            total += ctl.scan[w];
        }
        total *= a.kv_heads;
        span = max(quotient(total + gridDim.x - 1, gridDim.x), 4ll + C::kItemCost);
        b0 = span * blockIdx.x;
        b1 = min(total, b0 + span);
        if (b0 < b1 && ahead * a.kv_heads <= b0 && b0 < (ahead + keys) * a.kv_heads) {
            for (int q = qa;; ++q) {  // exactly one thread holds unit b0
                seek(q);
                if (b0 < (ahead + cost_of(pa, x)) * a.kv_heads) break;
                ahead += cost_of(pa, x);
            }
            ctl.first_r = x.r;
            ctl.first_qt = x.qt;
            ctl.first_start = ahead * a.kv_heads;
        }
    }
    fence_before();
    fence_async();
    __syncthreads();  // also: qsum is read, the operands may land over it
    fence_after();
    const uint32_t tmem = uniform(ctl.tmem);
    const bool work = b0 < b1;
    Item it;
    if (work) {
        it.r = ctl.first_r;
        it.qt = ctl.first_qt;
        request_of(a, it);
        q_tile_of(pa, it);
        it.h = (int)quotient(b0 - ctl.first_start, cost_of(pa, it));
        it.start = ctl.first_start + it.h * cost_of(pa, it) + pa.item_cost;
    }
    // An item's tiles [i0, i1) that fall into this span; none of the last item's when only its fixed cost does.
    int i0 = 0, i1 = 0;
    auto segment = [&]() {
        i0 = (int)max(0ll, b0 - it.start);
        i1 = (int)min((long long)it.n, b1 - it.start);
    };
    bool more = work;
    if (more) segment();
    auto advance = [&]() {
        more = it.start + it.n < b1;
        if (more) {
            next_item(pa, it);
            segment();
            more = i1 > 0;
        }
    };

    // Who fills the operand ring waits for the step that used a slot's last contents: key tile i is used in step i - i0 of
    // its segment, its values in the next.  Lane s remembers slot s's step.
    unsigned steps = 0, last_step = 0;
    auto slot_free = [&](unsigned s) {
        const unsigned n = __shfl_sync(0xffffffffu, last_step, s);
        return warp_wait(&ctl.step[n % kSteps], n / kSteps & 1, abort);
    };
    auto slot_used = [&](unsigned s, unsigned step) {
        if (lane == (int)s) last_step = step;
    };
    // The landing of load number c (keys of tile c / 2, or its values), and the phase: bf16 operands, or raw Q8_0 data.
    auto landed = [&](unsigned c) {
        if constexpr (Q8) return &ctl.raw_full[c % C::kRawSlots];
        else return &ctl.full[(c & 1) * 5 + (c >> 1) % 5];
    };
    auto landed_phase = [](unsigned c) {
        if constexpr (Q8) return c / C::kRawSlots & 1;
        else return (c >> 1) / 5 & 1;
    };
    if (warp == kLoadWarp) {
        // ---- keys and values: lane i requests run i of each tile ----
        const int runs = kTile / pa.run, per = pa.run / 16;
        unsigned cnt = 0, seg = 0;
        bool ok = true;
        for (; more; advance()) {
            if (!ok) break;
            if (seg && !(ok = warp_wait(&ctl.q_empty, (seg - 1) & 1, abort))) break;
            ++seg;
            if (lane == 0) {  // Q: boxes of 64 values, the cache head's heads, a tile's tokens
                uint64_t *bar = Q8 ? &ctl.q_raw : &ctl.q_full;
                const int nx = it.tokens > pa.tile_tokens ? 2 : 1;
                bar_arrive_tx(bar, (unsigned)(nx * C::kSub * 128 * a.group * pa.tile_tokens));
                for (int x = 0; x < nx; ++x)
                    for (int sub = 0; sub < C::kSub; ++sub)
                        tma3(saddr(smem) + x * C::kOp + sub * kTile * 128, &qmap, 64 * sub, it.h * a.group,
                             it.row0 + it.tok0 + x * pa.tile_tokens, bar);
            }
            __syncwarp();
            const int *row = a.table + (size_t)it.r * a.pitch;
            int page = -1, off = 0;
            auto look = [&](int i) {
                const int j = it.key(i * kTile + lane * pa.run);
                page = -1;
                if (lane < runs && j < it.end) {
                    page = row[j / a.page_size];
                    off = j % a.page_size;
                }
            };
            look(i0);
            for (int i = i0; i < i1 && ok; ++i) {
                const bool there = page >= 0 && page < a.pages;
                const unsigned got = __ballot_sync(0xffffffffu, there);
                unsigned groups = 0;  // a bit for each 16 tokens
                for (int b = 0; b < runs; ++b)
                    if (got >> b & 1u) groups |= ((1u << per) - 1u) << (b * per);
                const int mypage = page, myoff = off;
                if (i + 1 < i1) look(i + 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++cnt) {
                    const unsigned slots = Q8 ? C::kRawSlots : C::kSlots;
                    const unsigned s = cnt % slots, turn = cnt / slots;
                    uint64_t *full = landed(cnt);
                    if (cnt >= slots) {
                        if (Q8) ok = warp_wait(&ctl.raw_empty[s], (turn - 1) & 1, abort);
                        else ok = slot_free(s);
                        if (!ok) break;
                    }
                    if (!Q8) slot_used(s, steps + (i - i0) + kv);
                    if (lane == 0) {
                        if (kv == 0) {
                            const int v0 = i * kTile, pb = it.p_min + pa.tile_tokens;
                            const bool gone = groups != 0xFFu;
                            ctl.tile[(cnt >> 1) & 7] = make_int2(
                                v0, (int)groups | (gone || it.partial(a, v0, it.p_min, min(pb - 1, it.p_max)) ? 256 : 0) |
                                               (pb <= it.p_max && (gone || it.partial(a, v0, pb, it.p_max)) ? 512 : 0));
                        }
                        const unsigned bytes = __popc(groups) * 16 * (Q8 ? D + D / 32 * 4 : 2 * D);
                        bar_arrive_tx(full, bytes);
                    }
                    __syncwarp();
                    if (there) {
                        if (!Q8) {
                            const uint32_t dst = saddr(smem + C::kRing + s * C::kOp) + lane * pa.run * 128;
#pragma unroll
                            for (int sub = 0; sub < C::kSub; ++sub)
                                tma3(dst + sub * kTile * 128, kv ? &vmap : &kmap, 64 * sub, it.h * a.page_size + myoff,
                                     mypage, full);
                        } else {
                            const long long at = (long long)mypage * a.page_stride +
                                                 ((long long)it.h * a.page_size + myoff) * D;
                            const uint32_t dst = saddr(smem + C::kRawAt + s * C::kRaw);
                            bulk(dst + lane * pa.run * D, static_cast<const signed char *>(kv ? a.v : a.k) + at,
                                 pa.run * D, full);
                            bulk(dst + kTile * D + lane * pa.run * (D / 32) * 4, (kv ? a.vs : a.ks) + at / 32,
                                 pa.run * (D / 32) * 4, full);
                        }
                    }
                }
            }
            steps += i1 - i0 + 1;
        }
        if (!ok) {  // the copies in flight land before the shared memory goes
            const unsigned slots = Q8 ? C::kRawSlots : C::kSlots;
            for (unsigned c = cnt > slots ? cnt - slots : 0; c < cnt; ++c) {
                const uint64_t t0 = now_ns();
                while (!bar_try(landed(c), landed_phase(c)) && now_ns() - t0 < 2000000000ull) {
                }
            }
            const uint64_t t0 = now_ns();
            while (seg && !bar_try(Q8 ? &ctl.q_raw : &ctl.q_full, (seg - 1) & 1) && now_ns() - t0 < 2000000000ull) {
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---- the MMAs ----
        // The tensor cores work on what is queued while this warp looks at barriers, as long as a batch follows a batch.  A
        // turn is a batch: the O of a job, and the S that its score buffer (with three, the one behind it) is free for.
        constexpr uint32_t fmt = Q8 ? 0u : 1u;  // fp16 or bf16 operands
        const uint32_t id_s = (1u << 4) | (fmt << 7) | (fmt << 10) | (a.scale < 0.0f ? 1u << 13 : 0u) |
                              ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
        constexpr uint32_t id_o = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((D >> 3) << 17) |
                                  ((kTile >> 4) << 24);
        const uint32_t q_desc = desc128_low(saddr(smem), 16), k_desc = desc128_low(saddr(smem + C::kRing), 16);
        const uint32_t v_desc = desc128_low(saddr(smem + C::kRing), kTile * 128);
        constexpr int AHEAD = C::kBufs - 1;  // key tiles that A's scores are ahead of its O
        unsigned seg = 0, steps = 0, pbits = 0;              // pbits: the weight barriers' phases
        // Of the next keys to wait for, the next values: place (Q8_0) or tile modulo 5 (bf16), and phase.
        unsigned knext = 0, kphase = 0, vnext = Q8 ? 1 : 0, vphase = 0;
        unsigned jobs = 0;                                   // the buffer of A's next O
        bool ok = true;
        auto tile_on = [](unsigned &next, unsigned &phase) {
            constexpr unsigned by = Q8 ? 2 : 1, around = Q8 ? C::kSlots : 5;
            next += by;
            if (next >= around) {
                next -= around;
                phase ^= 1;
            }
        };
        auto key_bar = [&]() { return Q8 ? &ctl.ready[knext] : &ctl.full[knext]; };
        auto place_of = [](unsigned next, unsigned kv) {  // in the ring
            if constexpr (Q8) return next;
            const unsigned s = 2 * next + kv;
            return s >= C::kSlots ? s - C::kSlots : s;
        };
        auto issue_s = [&](int x, unsigned b, unsigned slot) {  // one lane
            const uint32_t qd = q_desc + x * (C::kOp >> 4), kd = k_desc + slot * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const unsigned o = ((k / 4) * kTile * 128 + (k % 4) * 32) >> 4;
                mma_ss(tmem + b * kTile, qd + o, kd + o, id_s, k > 0);
            }
            commit(&ctl.s_full[b]);
        };
        auto issue_o = [&](int x, unsigned b, unsigned slot, uint32_t more_o) {
            const uint32_t vd = v_desc + slot * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                mma_ts(tmem + C::kColO + x * D, tmem + b * kTile + kColP + k * 8, vd + (k * 2048 >> 4), id_o,
                       k > 0 ? 1u : more_o);
        };
        auto buffer = [](unsigned j) { return C::kBufs == 2 ? j & 1u : (j >= 6 ? j - 6 : j >= 3 ? j - 3 : j); };
        for (; more; advance()) {
            const bool two = it.tokens > pa.tile_tokens;  // tile B has rows
            if (!(ok = warp_wait(&ctl.q_full, seg & 1, abort))) break;
            // the first scores
            unsigned key1 = 0;  // slot of the keys that B's next scores need
            for (int n = 0; n < AHEAD && i0 + n < i1; ++n) {
                if (!(ok = warp_wait(key_bar(), kphase, abort))) break;
                key1 = uniform(place_of(knext, 0));
                tile_on(knext, kphase);
                const unsigned b = uniform(jobs);
                fence_after();
                if (elect()) {
                    issue_s(0, buffer(b + 2 * n), key1);
                    if (n == 0 && two) issue_s(1, buffer(b + 1), key1);
                    if (n + 1 == AHEAD || i0 + n + 1 == i1) {
                        commit(&ctl.step[steps % kSteps]);
                        if (i1 - i0 == 1) commit(&ctl.q_empty);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            ++steps;
            for (int i = i0; i < i1; ++i) {
                const unsigned u = uniform(vnext | (jobs << 8)), vn = u & 255u, ba = u >> 8, bb = buffer(ba + 1);
                const unsigned vs = place_of(vn, 1);
                const uint32_t more_o = i > i0;
                // ---- A ----
                {
                    const bool keys = C::kBufs == 2 && i + 1 < i1;  // two buffers: A's next scores in this turn
                    uint64_t *const pbar = &ctl.p_ready[ba], *const kbar = keys ? key_bar() : pbar;
                    const unsigned pp = pbits >> ba & 1u, kp = keys ? kphase : pp;
                    if (!look3(pbar, pp, &ctl.ready[vn], vphase, kbar, kp)) {
                        if (!(ok = warp_wait(&ctl.ready[vn], vphase, abort))) break;
                        if (!(ok = warp_wait(kbar, kp, abort))) break;
                        if (!(ok = warp_wait(pbar, pp, abort))) break;
                    }
                    pbits ^= 1u << ba;
                    if (keys) {
                        key1 = uniform(place_of(knext, 0));
                        tile_on(knext, kphase);
                    }
                    fence_after();
                    if (elect()) {
                        issue_o(0, ba, vs, more_o);
                        if (i + 1 == i1) commit(&ctl.o_full[0]);
                        if (C::kBufs == 2) {
                            if (keys) issue_s(0, ba, key1);
                        } else if (two && i + 1 < i1) {
                            issue_s(1, ba, key1);
                        }
                    }
                    __syncwarp();
                }
                // ---- B ----
                {
                    const bool keys = C::kBufs == 3 && i + 2 < i1;  // three: A's scores of the tile after the next
                    if (two || keys) {
                        uint64_t *const kbar = keys ? key_bar() : &ctl.p_ready[bb], *const pbar = two ? &ctl.p_ready[bb] : kbar;
                        const unsigned kp = keys ? kphase : pbits >> bb & 1u, pp = two ? pbits >> bb & 1u : kp;
                        if (!look3(pbar, pp, kbar, kp, pbar, pp)) {
                            if (!(ok = warp_wait(kbar, kp, abort))) break;
                            if (!(ok = warp_wait(pbar, pp, abort))) break;
                        }
                        if (two) pbits ^= 1u << bb;
                    }
                    unsigned key2 = 0;
                    if (keys) {
                        key2 = uniform(place_of(knext, 0));
                        tile_on(knext, kphase);
                    }
                    fence_after();
                    if (elect()) {
                        if (two) {
                            issue_o(1, bb, vs, more_o);
                            if (i + 1 == i1) commit(&ctl.o_full[1]);
                        }
                        if (C::kBufs == 2) {
                            if (two && i + 1 < i1) issue_s(1, bb, key1);
                        } else if (keys) {
                            issue_s(0, bb, key2);
                        }
                        commit(&ctl.step[steps % kSteps]);
                        if (i + 2 == i1) commit(&ctl.q_empty);
                    }
                    __syncwarp();
                    if (keys) key1 = key2;
                }
                tile_on(vnext, vphase);
                if (C::kBufs == 3) jobs = buffer(jobs + 2);
                ++steps;
            }
            if (!ok) break;
            ++seg;
        }
        __syncwarp();
    } else if (warp >= kHelpWarp) {
        // ---- what the tiles need before the MMAs ----
        const int ht = tid - 32 * kHelpWarp;
        constexpr int HT = 32 * C::kHelpers;
        unsigned cnt = 0, seg = 0;
        bool ok = true;
        for (; more; advance()) {
            if (!ok) break;
            constexpr int CH = D / 8;  // 16-byte chunks of an operand row
            int v_ex = 0;
            for (int i = i0; i < i1 && ok; ++i) {
                const int v0 = i * kTile;
                // a key that some row of the item may see
                auto live = [&](int c, unsigned groups) {
                    const int j = it.key(v0 + c);
                    return (groups >> (c >> 4) & 1u) && j < it.end && (j >= it.lo || j < a.sinks);
                };
                for (int kv = 0; kv < 2 && ok; ++kv, ++cnt) {
                    const unsigned s = cnt % C::kSlots;
                    unsigned char *op = smem + C::kRing + s * C::kOp;
                    if constexpr (!Q8) {
                        if (!kv) continue;  // keys go to the MMAs as they are
                        if (!(ok = warp_wait(landed(cnt), landed_phase(cnt), abort))) break;
                        const int info = ctl.tile[(cnt >> 1) & 7].y;
                        const unsigned groups = info & 255u;
                        if (info & 768) {
                            // Thread ht takes chunk ht % CH of every RS-th key, eight loads in flight.
                            bool found = false;
                            constexpr int RS = HT / CH, B = 8;
                            static_assert(kTile % (RS * B) == 0, "");
                            uint4 *at = reinterpret_cast<uint4 *>(op + (ht % CH / 8) * kTile * 128 + ht / CH * 128 + ht % 8 * 16);
#pragma unroll 1
                            for (int y = 0; y < kTile / RS; y += B) {
                                uint4 v[B];
#pragma unroll
                                for (int z = 0; z < B; ++z) v[z] = at[(y + z) * RS * 8];
#pragma unroll
                                for (int z = 0; z < B; ++z) {
                                    const int c = (y + z) * RS + ht / CH;
                                    if (!live(c, groups)) {
                                        at[(y + z) * RS * 8] = make_uint4(0u, 0u, 0u, 0u);
                                        continue;
                                    }
                                    const auto odd = [](uint32_t w) {  // the halves that are not finite, in their top bits
                                        return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;
                                    };
                                    const uint32_t b[4] = {odd(v[z].x), odd(v[z].y), odd(v[z].z), odd(v[z].w)};
                                    if (b[0] | b[1] | b[2] | b[3]) {
                                        found = true;
                                        at[(y + z) * RS * 8] = make_uint4(
                                            v[z].x & ~((b[0] >> 15) * 0xFFFFu), v[z].y & ~((b[1] >> 15) * 0xFFFFu),
                                            v[z].z & ~((b[2] >> 15) * 0xFFFFu), v[z].w & ~((b[3] >> 15) * 0xFFFFu));
                                    }
                                }
                            }
                            if (found) *(volatile int *)&ctl.poison = 1;
                            fence_async();
                        }
                        __syncwarp();
                        if (lane == 0) bar_arrive(&ctl.ready[(cnt >> 1) % 5]);
                        continue;
                    }
                    // Q8_0: codes and scales to fp16
                    const unsigned rs = cnt % (C::kRawSlots ? C::kRawSlots : 1);
                    if (cnt >= (unsigned)C::kSlots && !(ok = slot_free(s))) break;
                    slot_used(s, steps + (i - i0) + kv);
                    if (!(ok = warp_wait(landed(cnt), landed_phase(cnt), abort))) break;
                    const unsigned char *raw = smem + C::kRawAt + rs * C::kRaw;
                    const float *scl = reinterpret_cast<const float *>(raw + kTile * D);
                    const int info = ctl.tile[(cnt >> 1) & 7].y;
                    const unsigned groups = info & 255u;
                    const bool part = (info & 768) != 0;
                    constexpr int NB = D / 32;
                    // The tile's largest finite scale, by its bits: every warp looks for itself, four at a time.
                    uint32_t mx = 0u;
#pragma unroll
                    for (int y = 0; y < kTile * NB / 128; ++y) {
                        const uint4 f = *reinterpret_cast<const uint4 *>(scl + (y * 32 + lane) * 4);
                        mx = max(mx, max(max(f.x & 0x7FFFFFFFu, f.y & 0x7FFFFFFFu), max(f.z & 0x7FFFFFFFu, f.w & 0x7FFFFFFFu)));
                    }
                    mx = __reduce_max_sync(0xffffffffu, mx);
                    if (part || mx >= 0x7F800000u) {  // one by one, what somebody sees and is finite
                        mx = 0u;
#pragma unroll 1
                        for (int e = lane; e < kTile * NB; e += 32) {
                            const uint32_t m = __float_as_uint(scl[e]) & 0x7FFFFFFFu;
                            if (m < 0x7F800000u && (!part || live(e / NB, groups))) mx = max(mx, m);
                        }
                        mx = __reduce_max_sync(0xffffffffu, mx);
                    }
                    // The values' unit only grows within a segment, and neither is below 2^-70, so that a tile of
                    // zeros does not take the row sums, which are kept apart from the units, out of fp32's range.
                    int ex = min(max((int)(mx >> 23), 64), 252);
                    if (kv) ex = v_ex = max(v_ex, ex);
                    // The unit is 2^-7 of the largest scale's power of two: scale / unit is below 2^8, any int8 code times
                    // it within fp16's range, and its smallest normal 2^-21 of the largest.
                    const float down = __uint_as_float((uint32_t)(254 + 7 - ex) << 23);  // 2^-(ex - 7 - 127)
                    bool found = false, lost = false;
                    // Thread ht takes 16 codes of rows r0, r0 + HT / RC, ...: a step of whole swizzle periods, so that
                    // all addresses are its first ones plus constants.
                    constexpr int RC = D / 16, RS = HT / RC;  // chunks of 16 codes a row, rows a pass
                    static_assert(RS % 8 == 0, "");
                    const int ch = ht % RC, r0 = ht / RC;
                    const unsigned char *src = raw + r0 * D + ch * 16;
                    const float *sc = scl + r0 * NB + ch / 2;
                    unsigned char *to = op + (ch / 4) * kTile * 128 + r0 * 128;
                    // Two threads of a quarter warp that read the same chunk's place write its halves in turn, so that
                    // they write different banks.
                    const bool swap = (ch >> 2) & 1;
                    const int da = (((2 * ch) & 7) ^ (r0 & 7)) * 16, db = da ^ 16;
                    unsigned char *first = to + (swap ? db : da), *second = to + (swap ? da : db);
                    constexpr int B = 3;  // rows at a time, so that their loads are in flight together
#pragma unroll
                    for (int y = 0; y * RS < kTile; y += B) {
                        uint4 v[B];
                        float f[B];
#pragma unroll
                        for (int z = 0; z < B; ++z) {
                            if ((y + z + 1) * RS > kTile && r0 + (y + z) * RS >= kTile) break;
                            v[z] = *reinterpret_cast<const uint4 *>(src + (y + z) * RS * D);
                            f[z] = sc[(y + z) * RS * NB] * down;
                        }
                        if (part) {
#pragma unroll
                            for (int z = 0; z < B; ++z) {
                                const bool see = live(r0 + (y + z) * RS, groups);
                                if (r0 + (y + z) * RS < kTile && (!see || (kv && !(fabsf(f[z]) < INFINITY)))) {
                                    found = found || see;
                                    v[z] = make_uint4(0u, 0u, 0u, 0u);
                                    f[z] = 0.0f;
                                }
                            }
                        }
#pragma unroll
                        for (int z = 0; z < B; ++z) {
                            if ((y + z + 1) * RS > kTile && r0 + (y + z) * RS >= kTile) break;
                            const __half2 f2 = __float2half2_rn(f[z]);
                            // not 0 and below 2^-14, fp16's smallest normal
                            lost = lost || (__float_as_uint(f[z]) & 0x7FFFFFFFu) - 1u < 0x38800000u - 1u;
                            const uint32_t w[4] = {(swap ? v[z].z : v[z].x) ^ 0x80808080u, (swap ? v[z].w : v[z].y) ^ 0x80808080u,
                                                   (swap ? v[z].x : v[z].z) ^ 0x80808080u, (swap ? v[z].y : v[z].w) ^ 0x80808080u};
                            uint32_t h[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t b = __byte_perm(w[k / 2], 0x64646464u, k % 2 ? 0x4342 : 0x4140);
                                const __half2 q = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&b),
                                                                  __half2half2(__ushort_as_half(0x6480))), f2);
                                h[k] = *reinterpret_cast<const uint32_t *>(&q);
                            }
                            *reinterpret_cast<uint4 *>(first + (y + z) * RS * 128) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4 *>(second + (y + z) * RS * 128) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                    }
                    if (found) *(volatile int *)&ctl.poison = 1;
                    if (kv && lost) *(volatile int *)&ctl.lost = 1;
                    if (ht == 0) ctl.unit[kv][(cnt >> 1) & 7] = (float)(ex - 7 - 127);
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&ctl.raw_empty[rs]);
                        bar_arrive(&ctl.ready[s]);
                    }
                }
            }
            steps += i1 - i0 + 1;
            ++seg;
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = row of tile x ----
        const int x = warp >> 2, quarter = warp & 3;
        const int y = quarter * 32 + lane, rx = x * kTile + y;
        const int tok = x * pa.tile_tokens + y / a.group, gh = y % a.group;  // of this row: the item's token, the head
        const bool whole_row = y < pa.tile_tokens * a.group;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t to = tmem + lanes + C::kColO + x * D;
        // The largest sum of a row's 128 weights: below fp16's largest value; for bf16 weights, which have fp32's range,
        // such that sums over values of up to 2^90 do not overflow on the way to a result that does not.
        constexpr float kMostSum = Q8 ? 32768.0f : 4294967296.0f;  // 2^15, 2^32
        constexpr float kLeast = 1.17549435e-38f;  // a factor of 0 would make NaN of a hidden score's -inf
        const float sc0 = fmaxf(fabsf(a.scale) * kLog2e, kLeast);
        unsigned cnt = 0, ends = 0, shared = 0, seg = 0;  // ends: the phases of o_full (bit 0) and idle (bit 1)
        unsigned job = 0, sbits = 0;  // the buffer of A's next scores; the score barriers' phases
        bool ok = true;
        for (; more; advance()) {
            if (!ok) break;
            const bool two = it.tokens > pa.tile_tokens, active = x == 0 || two;
            const bool row_live = whole_row && tok < it.tokens;
            const int p = it.p_min + tok;
            float M = row_live ? -INFINITY : 0.0f, l = 0.0f;  // rows beyond the item's ask for nothing
            float back = 1.0f;
            if constexpr (Q8) {
                if (!(ok = warp_wait(&ctl.q_raw, seg & 1, abort))) break;
                if (row_live) back = row_to_half<D>(smem + x * C::kOp + y * 128, y & 7);
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(&ctl.q_full);
            }
            if (active) {
                float sc = sc0;
                for (int i = i0; i < i1 && ok; ++i) {
                    const unsigned ba = job, bb = C::kBufs == 2 ? 1u : (job == 2 ? 0u : job + 1);
                    const unsigned b = x ? bb : ba, parity = sbits >> b & 1u;
                    sbits ^= (1u << ba) ^ (two ? 1u << bb : 0u);
                    if (C::kBufs == 3) job = job == 0 ? 2u : job - 1;  // two on
                    const uint32_t ts = tmem + lanes + b * kTile;
                    const unsigned ck = cnt + 2 * (i - i0), at = (ck >> 1) & 7;
                    if (!(ok = warp_wait(&ctl.s_full[b], parity, abort))) break;
                    fence_after();
                    float shift = 0.0f;  // log2 of the values' unit (Q8_0)
                    const int2 info = tile_info(&ctl.tile[at]);
                    if (Q8) {
                        const unsigned cv = ck + 1;
                        if (!(ok = warp_wait(&ctl.ready[cv % C::kSlots], (cv / C::kSlots) & 1, abort))) break;
                        sc = fmaxf(sc0 * back * ex2(*(volatile float *)&ctl.unit[0][at]), kLeast);
                        shift = *(volatile float *)&ctl.unit[1][at];
                    }
                    if (info.y >> (8 + x) & 1) {
                        // columns [c_lo, c_hi] and [0, c_sink) are visible
                        const int j0 = info.x + it.jump;
                        hide_scores<Q8>(ts, min(p, it.end - 1) - j0, a.window ? max(max(p, 0) - (a.window - 1), j0) - j0 : 0,
                                       a.window ? a.sinks - info.x : 0, info.y);
                    }
                    // The weights are taken against the running maximum as it stands: a row's maximum is only looked
                    // for where their sum shows that a score passed it too far (or there is none yet).
                    unsigned long long sc2, off2, sum2;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(sc2) : "f"(sc));
                    float sum;
                    uint32_t w[4][16];
                    auto weights = [&](const uint32_t (&r)[32], uint32_t (&to)[16]) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            unsigned long long e;
                            float p0, p1;
                            asm("{\n .reg .b64 s;\n mov.b64 s, {%1, %2};\n fma.rn.f32x2 %0, s, %3, %4;\n}"
                                : "=l"(e) : "r"(r[2 * k]), "r"(r[2 * k + 1]), "l"(sc2), "l"(off2));
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(p0), "=f"(p1) : "l"(e));
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            asm("{\n .reg .b64 s;\n mov.b64 s, {%1, %2};\n add.rn.f32x2 %0, %0, s;\n}"
                                : "+l"(sum2) : "f"(p0), "f"(p1));
                            to[k] = Q8 ? f16x2(p0, p1) : bf16x2(p0, p1);
                        }
                    };
                    for (int again = __any_sync(0xffffffffu, M == -INFINITY) ? 1 : 0;; again = 1) {
                        if (again) {
                            float mx = max_score(ts);
                            mx = mx == -INFINITY ? mx : fmaf(mx, sc, shift);
                            const float now = fmaxf(M, mx), f = now == M ? 1.0f : ex2(M - now);  // 0 from -inf
                            M = now;
                            l *= f;
                            if (i > i0) {
                                // With three buffers these scores may have come before the last tile's O: it is at
                                // rest once that tile's turns are done.
                                if (C::kBufs == 3) {
                                    const unsigned n = steps + (i - i0);
                                    if (!(ok = warp_wait(&ctl.step[n % kSteps], n / kSteps & 1, abort))) break;
                                    fence_after();
                                }
                                scale_columns(to, D, f);
                            }
                        }
                        const float off = shift - (M == -INFINITY ? 0.0f : M);
                        asm("mov.b64 %0, {%1, %1};" : "=l"(off2) : "f"(off));
                        sum2 = 0ull;
                        uint32_t va[32], vb[32];
                        tm_ld32(ts, va);
                        tm_ld32(ts + 32, vb);
                        tm_wait_ld();
                        weights(va, w[0]);
                        tm_ld32(ts + 64, va);
                        weights(vb, w[1]);
                        tm_wait_ld();
                        tm_ld32(ts + 96, vb);
                        weights(va, w[2]);
                        tm_wait_ld();
                        weights(vb, w[3]);
                        float sum_hi;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(sum), "=f"(sum_hi) : "l"(sum2));
                        sum += sum_hi;
                        if (again || !__any_sync(0xffffffffu, row_live && sum > kMostSum)) break;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) tm_st16(ts + kColP + 16 * y, w[y]);
                    l += Q8 ? sum * ex2(-shift) : sum;
                    tm_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&ctl.p_ready[b]);
                }
                if (ok) ok = warp_wait(&ctl.o_full[x], ends & 1, abort);
                if (ok && !two) ok = warp_wait(&ctl.idle, ends >> 1 & 1, abort);
                ends ^= two ? 1u : 3u;
                fence_after();
            } else {
                // Tile B without rows keeps count of the buffers, and does not run ahead: a barrier tells a phase from the
                // one before it, not from the one before that.
                for (int i = i0; i < i1; ++i) {
                    sbits ^= 1u << job;
                    if (C::kBufs == 3) job = job == 0 ? 2u : job - 1;
                }
                // A waits for it in turn: it must not be two ends further on when this warp looks.  (Its wait, needed only
                // then, costs all calls 1%: a prompt of 8192 rows 350 and 353 us.)
                ok = warp_wait(&ctl.o_full[0], seg & 1, abort);
                if (lane == 0) bar_arrive(&ctl.idle);
            }
            steps += i1 - i0 + 1;
            cnt += 2 * (i1 - i0);
            ++seg;
            // ---- the segment's end ----
            const long long last_unit = it.start + it.n - 1;
            const int c0 = (int)quotient(it.start, span), c1 = (int)quotient(last_unit, span);
            const bool wide = (((uintptr_t)a.out | (uintptr_t)(2 * a.ldo)) & 31) == 0;
            const bool poison = *(volatile int *)&ctl.poison != 0, rare = poison || (Q8 && *(volatile int *)&ctl.lost);
            float *base = reinterpret_cast<float *>(a.work + kPrefillPartAt);
            uint16_t *orow = a.out + (size_t)(it.row0 + it.tok0 + (row_live ? tok : 0)) * a.ldo + (it.h * a.group + gh) * D;
            float *part = base + ((long long)blockIdx.x * 2 + (it.start >= b0)) * kPrefillPartFloats;
            if (active && ok) {
                const float inv = c0 == c1 ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t v[32];
                    tm_ld32(to + cc, v);
                    tm_wait_ld();
                    float o[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(v[k]) * inv;
                    if (rare && row_live) {
                        float extra[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) extra[k] = o[k];
                        // values below fp16's normal range are off by 2^-18 units at most, a sum of them by l 2^-18
                        if (Q8 && *(volatile int *)&ctl.lost) {
                            const float shift = *(volatile float *)&ctl.unit[1][(cnt / 2 - 1) & 7];  // of the last tile
                            attend_again<D>(a, it, i0, i1, tok, gh, M, inv, l * inv * ex2(shift - 8.0f), cc, extra);
                        }
                        if (poison) add_nonfinite<D, Q8>(a, it, i0, i1, p, cc, extra);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = extra[k];
                    }
                    if (c0 == c1) {
                        if (row_live) store_row(orow + cc, o, wide);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4 *>(part + ((cc / 4 + k) * kRows + rx) * 4) =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
            }
            if (c0 != c1) *reinterpret_cast<float2 *>(part + kRows * 128 + 2 * rx) = make_float2(M, l);
            fence_before();
            if (c0 != c1 && ok) {
                // ---- shared with other CTAs: the last to arrive adds the parts in span order ----
                // (one thread's fence covers what the barrier has ordered before it)
                __syncwarp();
                if (lane == 0) bar_arrive(&ctl.joined);
                if (tid == 0 && bar_wait(&ctl.joined, shared & 1, abort)) {
                    int *count = reinterpret_cast<int *>(a.work + kPrefillCounterAt) + c0;
                    __threadfence();
                    const int seen = atomicAdd(count, 1);
                    ctl.last = seen == c1 - c0;
                    if (seen == c1 - c0) {
                        *count = 0;
                        __threadfence();
                    }
                    bar_arrive(&ctl.decided);
                }
                ok = warp_wait(&ctl.decided, shared++ & 1, abort);
                if (ok && *(volatile int *)&ctl.last && row_live) {
                    constexpr int J = Q8 || D == 64 ? 32 : 64;  // columns at a time: J / 4 loads in flight, J sums
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += J) {
                        float o[J], m2 = -INFINITY, l2 = 0.0f;
#pragma unroll
                        for (int k = 0; k < J; ++k) o[k] = 0.0f;
#pragma unroll 1
                        for (int z = c0; z <= c1; ++z) {
                            const float *from = base + ((long long)z * 2 + (z == c0)) * kPrefillPartFloats;
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(from + kRows * 128 + 2 * rx));
                            float4 v[J / 4];
#pragma unroll
                            for (int k = 0; k < J / 4; ++k)
                                v[k] = __ldcg(reinterpret_cast<const float4 *>(from + ((cc / 4 + k) * kRows + rx) * 4));
                            const float now = fmaxf(m2, ml.x);
                            const float fa = m2 == now ? 1.0f : ex2(m2 - now), fb = ml.x == now ? 1.0f : ex2(ml.x - now);
                            m2 = now;
                            l2 = l2 * fa + ml.y * fb;
                            const bool none = ml.x == -INFINITY;  // a part that saw nothing has no O
#pragma unroll
                            for (int k = 0; k < J / 4; ++k) {
                                o[4 * k] = fmaf(none ? 0.0f : v[k].x, fb, o[4 * k] * fa);
                                o[4 * k + 1] = fmaf(none ? 0.0f : v[k].y, fb, o[4 * k + 1] * fa);
                                o[4 * k + 2] = fmaf(none ? 0.0f : v[k].z, fb, o[4 * k + 2] * fa);
                                o[4 * k + 3] = fmaf(none ? 0.0f : v[k].w, fb, o[4 * k + 3] * fa);
                            }
                        }
                        const float inv = l2 == 0.0f ? 0.0f : 1.0f / l2;
#pragma unroll
                        for (int k = 0; k < J; ++k) o[k] *= inv;
#pragma unroll
                        for (int k = 0; k < J; k += 32)
                            store_row(orow + cc + k, *reinterpret_cast<const float(*)[32]>(o + k), wide);
                    }
                }
            }
        }
    }

    // ---- drain: every MMA issued is done (o_full was waited for), unless the CTA aborted ----
    fence_before();
    __syncthreads();
    if (*abort && tid == 32 * kMmaWarp) {
        commit(&ctl.drain);
        const uint64_t t0 = now_ns();
        while (!bar_try(&ctl.drain, 0) && now_ns() - t0 < 2000000000ull) {
        }
    }
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns) : "memory");
    // ---- rows that see nothing: padding, and rows before the first key ----
    for (int row = blockIdx.x * T + tid; row < a.rows; row += gridDim.x * T) {
        int lo = 0, hi = a.R;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.row_start[mid] <= row) lo = mid; else hi = mid - 1;
        }
        Item x;
        x.n = 0;
        if (lo < a.R) {
            x.r = lo;
            request_of(a, x);
            x.p_min = x.p_max = x.pos0 + (row - x.row0);
            span_of(pa, x);
        }
        if (x.n == 0)
            for (int e = 0; e < a.heads * D / 8; ++e)
                *reinterpret_cast<uint4 *>(a.out + (size_t)row * a.ldo + 8 * e) = make_uint4(0u, 0u, 0u, 0u);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? p : nullptr);
    }();
    return fn;
}

// A map of 16-bit values [dims[2]][dims[1]][dims[0]], boxes of 64 x b1 x b2 values, 128-byte swizzle.
bool encode_boxes(CUtensorMap *map, const void *p, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2], int b1,
                  int b2) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    if (!encode) return false;
    const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8> cudaError_t launch_one(const AttnArgs &a, int sms, cudaStream_t stream) {
    using C = Cfg<D, Q8>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(prefill_kernel<D, Q8>, C::kSmem, &allowed);
    if (e != cudaSuccess) return e;
    PrefillArgs pa = {a, 16, kTile / a.group, C::kItemCost};
    while (pa.run < kTile && a.page_size % (2 * pa.run) == 0) pa.run *= 2;
    // K and V as [pages][heads * page_size][dim], boxes of `run` tokens; Q as [rows][heads][dim], boxes of a tile's
    // tokens and their heads.
    CUtensorMap kmap = {}, vmap = {}, qmap = {};
    const cuuint64_t kd[3] = {D, (cuuint64_t)a.kv_heads * a.page_size, (cuuint64_t)a.pages};
    const cuuint64_t ks[2] = {D * 2, (cuuint64_t)a.page_stride * 2};
    const cuuint64_t qd[3] = {D, (cuuint64_t)a.heads, (cuuint64_t)a.rows}, qs[2] = {D * 2, (cuuint64_t)a.ldq * 2};
    if (!encode_boxes(&qmap, a.q, qd, qs, a.group, pa.tile_tokens) ||
        (!Q8 && (!encode_boxes(&kmap, a.k, kd, ks, pa.run, 1) || !encode_boxes(&vmap, a.v, kd, ks, pa.run, 1))))
        return cudaErrorNotSupported;
    return kv_launch(prefill_kernel<D, Q8>, dim3((unsigned)sms, 1, 1), C::kThreads, C::kSmem, stream, pa, kmap, vmap,
                     qmap);
}

}  // namespace

cudaError_t read_attn_fault(unsigned *out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attn_fault, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_fault, &zero, sizeof(unsigned));
}

cudaError_t launch_attn_prefill(const AttnArgs &a, int dim, bool q8, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count_of_device(&sms);
    if (e != cudaSuccess) return e;
    if (sms > kAttnMaxCtas) sms = kAttnMaxCtas;
    if (dim == 128) return q8 ? launch_one<128, true>(a, sms, stream) : launch_one<128, false>(a, sms, stream);
    return q8 ? launch_one<64, true>(a, sms, stream) : launch_one<64, false>(a, sms, stream);
}

}  // namespace q8
