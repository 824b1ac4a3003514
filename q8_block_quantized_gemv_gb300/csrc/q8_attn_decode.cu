// q8_attn_decode: attention of one new token a request over the paged cache, split over the cache's length and joined.
//
// Every visible key and value is read once for up to 16 query heads of its cache head (once more for each further 16), 4
// flops a byte and head: HBM bounds the kernel until contexts are so short that latency does.  So the work is cut by bytes,
// not by requests: the visible tokens of all items in a row -- an item is a request's cache head with 8 or 16 of its query
// heads -- are a list of 16-token units, and each CTA (one per SM) takes an equal contiguous span of it, computed on the
// device from lens.  Its 8 warps (12 over a Q8_0 cache, up to 8 heads to a
// cache head) take the span's units in turn, each with a ring of its own in shared memory filled by cp.async (prefetch
// runs on across items; no CTA barrier but at an item's end), a running maximum and sum, and accumulators in registers.
//
// Products run transposed on mma.sync m16n8k16, as 16 tokens (or 16 of the head's values) by 8 query heads: a unit's
// S^T = K Q^T, then O^T += V^T P^T, so up to 8 heads sharing a cache head cost what one does.  tcgen05 has nothing to
// add: its smallest tile is 64 rows, and one to 16 query rows leave the tensor pipe nearly idle either way.
//
// At an item's end the warps' parts are summed through shared memory in warp order.  An item that crosses spans
// leaves parts in the workspace; the CTA that arrives last (a counter per first CTA, left at zero) adds them in span
// order, so the result does not depend on who was last.
//
// Measured, heads of 128, 32 over 8 cache heads: one request of 131,072 tokens, bf16, 84 us = 6.4 TB/s (95% of a copy's
// rate); 15 requests with 81,000 tokens in all, Q8_0, 43 us = 4.4 TB/s.  There a unit costs about 550 instructions (the
// codes' way to fp16, the scales), 137 for each of the SM's schedulers, and 200 clocks of the SM's share of the memory, and
// neither is full: 51% of the issue slots, 64% of the bandwidth.  8 warps take 44 us, 16 with their 128 registers 56.
// Heads of 64, 24 over 8, a window of 4,096 in 64 requests: 89 us = 6.0 TB/s.  One request of 203 tokens, 32 heads: 5.2
// us, the chain from its length over table, keys and sums to the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "q8_attn.h"
#include "q8_device.cuh"

namespace q8 {
namespace {

constexpr int kUnit = 16;  // tokens of a unit; a page holds whole units
constexpr int kMinSpan = 16;  // units: two a warp, below which a further CTA would cost more to join than it takes over
constexpr int kWholeUnits = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // log2: the running maximum moves when a score passes it by more than this

template <int D, bool Q8, int NT> struct Cfg {
    static constexpr int kWarps = Q8 && NT == 1 ? 12 : 8;
    static constexpr int kRow = Q8 ? D : 2 * D;                    // bytes of a token's values
    static constexpr int kVals = kUnit * kRow;                     // of a unit, K or V
    static constexpr int kScales = Q8 ? kUnit * (D / 32) * 4 : 0;  // of a unit, K or V
    static constexpr int kStage = 2 * (kVals + kScales);
    static constexpr int kPart = NT * 8 * D * 4 + NT * 8 * 8;      // a warp's O, then its (m, l)
    static constexpr int kFit = (226 * 1024 - kWarps * kPart) / (kWarps * kStage);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kWarps * (kStages * kStage + kPart);
    static_assert(kStages >= 2, "");
};

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// 16 tokens by 32 codes, transposed: lane (g, t) gets tokens 4t .. 4t + 3 of codes g, g + 8, g + 16 and g + 24.
__device__ __forceinline__ void ldsm8t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b + c, c the same for both token halves.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
template <int N> __device__ __forceinline__ void load_scales(float (&d)[N], uint32_t a) {
    if (N == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[N - 2]), "=f"(d[N - 1]) : "r"(a) : "memory");
    else
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(d[0]), "=f"(d[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Where 16-byte chunk `ch` of a token's row goes in its stage.  The bf16 rows and the codes' values are read by
// (transposing) matrix loads, eight rows of one chunk at a time; the codes' keys by 8-byte loads of 32-byte groups from
// the rows ta of four consecutive g (row ta + 2 keeps its place).  Either way the rows read together land on different banks.
template <int D, bool Q8> __device__ __forceinline__ int key_chunk(int row, int ch) {
    if (!Q8) return ch ^ (row & 7);
    return D == 128 ? ch ^ (((row & 1) | ((row >> 1) & 2)) << 1) : ch ^ (((row >> 2) & 1) << 1);
}
template <int D, bool Q8> __device__ __forceinline__ int value_chunk(int row, int ch) {
    return Q8 && D == 64 ? ch ^ ((row >> 1) & 3) : ch ^ (row & 7);
}

// What a request's token sees, as units: [0, us) hold its sinks, [ul, ul + n - us) the rest.
struct Seen {
    int end;      // keys [0, end) exist
    int lo;       // keys [lo, end) are in the window
    int us, ul, n;
};
__device__ __forceinline__ Seen seen_of(const AttnArgs &a, int len) {
    Seen s;
    s.end = min(max(len, 0), a.width * a.page_size);
    s.lo = a.window ? min(max(len - a.window, 0), s.end) : 0;
    const int sinks = a.window ? min(a.sinks, s.lo) : 0;
    s.us = (sinks + kUnit - 1) / kUnit;
    s.ul = max(s.lo / kUnit, s.us);
    s.n = s.us + max(0, (s.end + kUnit - 1) / kUnit - s.ul);
    return s;
}

// A place in the list of units: item (r, tile) begins at unit `start` of the list and has s.n units.
struct Cursor {
    int r, tile;
    long long start;
    Seen s;
    __device__ __forceinline__ void next(const AttnArgs &a, int tiles) {
        start += s.n;
        if (++tile == tiles) {
            tile = 0;
            do {
                ++r;
                s = seen_of(a, r < a.R ? a.lens[r] : 0x7FFFFFFF);  // past the end: units without end stop the walk
            } while (r < a.R && s.n == 0);
        }
    }
};

// A stored int8 word (q, four bytes) flipped to q + 128; bytes E and E + 1 as the fp16 pair q + 1152: each byte in the
// low mantissa of 1024.
template <int E> __device__ __forceinline__ uint32_t biased_f16x2(uint32_t flipped) {
    uint32_t p;
    asm("prmt.b32 %0, %1, 0x64646464, %2;" : "=r"(p) : "r"(flipped), "n"(E == 0 ? 0x4140 : 0x4342));
    return p;
}
// The exact fp16 pair of q.
template <int E> __device__ __forceinline__ uint32_t codes_f16x2(uint32_t flipped) {
    const uint32_t p = biased_f16x2<E>(flipped);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&p), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The fp16 pair of (p0, p1) * d * per.
__device__ __forceinline__ uint32_t weights_f16x2(float p0, float p1, float d, const uint32_t (&per)[2]) {
    float w0, w1;
    asm("{\n .reg .b64 p, d, u;\n mov.b64 p, {%2, %3};\n mov.b64 d, {%4, %4};\n mov.b64 u, {%5, %6};\n"
        " mul.rn.f32x2 p, p, d;\n mul.rn.f32x2 p, p, u;\n mov.b64 {%0, %1}, p;\n}"
        : "=f"(w0), "=f"(w1) : "f"(p0), "f"(p1), "f"(d), "r"(per[0]), "r"(per[1]));
    return f16x2(w0, w1);
}

// 2^-n, 0 below the smallest normal.
__device__ __forceinline__ float two_to_minus(int n) { return n > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - n) << 23); }
// The 32 values of a block that belong to head x of a lane's two, times f.
__device__ __forceinline__ void scale_block(float (&lo)[4], float (&hi)[4], int x, float f) {
    lo[x] *= f;
    lo[x + 2] *= f;
    hi[x] *= f;
    hi[x + 2] *= f;
}
constexpr int kMostPer = 253;  // exponent field of 2^126, the largest power of two with a normal reciprocal

// x / d for x < 2^27 as (x * mul) >> shift.  mul = ceil(2^shift / d) with 2^shift >= 2^27 d is off by less than one
// part in 2^27, so the quotient is exact, and x * mul < 2^56.
struct UnitDiv {
    unsigned mul;
    int shift;
};
inline UnitDiv unit_div(int d) {
    int log = 0;
    while ((1ll << log) < d) ++log;
    return {(unsigned)(((1ull << (27 + log)) + d - 1) / d), 27 + log};
}

template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(32 * Cfg<D, Q8, NT>::kWarps, 1) attn_decode_kernel(AttnArgs a, int tiles_a_head, UnitDiv div) {
    using C = Cfg<D, Q8, NT>;
    constexpr int W = C::kWarps;
    constexpr int KS = D / 16;       // k-steps of S, value tiles of O
    constexpr int NB = D / 32;       // quantized blocks of a head
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[W + 2];
    __shared__ int s_first[1];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int tiles = a.kv_heads * tiles_a_head;  // items a request
    unsigned char *ring = smem + warp * (C::kStages * C::kStage);
    unsigned char *parts = smem + W * C::kStages * C::kStage;
    const uint32_t ring_s = saddr(ring);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    long long span, b0, b1;  // the CTA's span [b0, b1) of the list
    Cursor c;                // the item being computed
    // ---- few short items: one a CTA, nothing to join ----
    // Splitting an item costs its CTAs a round through memory to hand their parts over, some 3 us; 64 units are 8 a
    // warp.  (One request of 203 tokens, 32 heads of 128: 11.5 us split, 5.2 us whole.  32 heads over 8, one request of 1,008
    // tokens 10.6 and 8.5, 1,500 tokens 10.9 and 10.7, 2,048 tokens 8.3 and 12.9; 16 requests of 1,008 tokens 14.0 and 9.1, of
    // 2,048 26.1 and 22.6; Q8_0, one of 1,008 14.6 and 11.8, of 2,048 10.7 and 16.9; heads of 64 are alike.)
    bool whole_items = (long long)a.R * tiles <= gridDim.x;
    if (whole_items)  // at most a request a thread: a.R <= gridDim.x < the block
        whole_items = !__syncthreads_or(tid < a.R && seen_of(a, a.lens[tid]).n > kWholeUnits);
    if (whole_items) {
        span = 1ll << 40;
        c.r = min((int)blockIdx.x / tiles, a.R - 1);
        c.tile = blockIdx.x % tiles;
        c.start = b0 = 0;
        c.s = seen_of(a, a.lens[c.r]);
        b1 = (int)blockIdx.x < a.R * tiles ? c.s.n : 0;
    } else {
    // ---- the list's length and this CTA's span of it ----
    const int each = (a.R + 32 * W - 1) / (32 * W);
    const int ra = min(a.R, tid * each), rb = min(a.R, ra + each);
    long long mine = 0;
    for (int r = ra; r < rb; ++r) mine += seen_of(a, a.lens[r]).n;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long before = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    total *= tiles;
    span = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinSpan);
    b0 = span * blockIdx.x;
    b1 = min(total, b0 + span);
    if (b0 < b1) {
        if (before * tiles <= b0 && b0 < (before + mine) * tiles) {  // exactly one thread: the request of unit b0
            int r = ra;
            for (;; ++r) {
                const int n = seen_of(a, a.lens[r]).n;
                if (b0 < (before + n) * tiles) break;
                before += n;
            }
            s_first[0] = r;
            s_scan[W] = before * tiles;
        }
        __syncthreads();
        c.r = s_first[0];
        c.s = seen_of(a, a.lens[c.r]);
        c.tile = (int)((b0 - s_scan[W]) / c.s.n);
        c.start = s_scan[W] + (long long)c.tile * c.s.n;
    }
    }
    if (b0 < b1) {
        Cursor p = c;  // runs ahead of c, filling the ring

        // ---- the ring: the warp's next unit into stage `slot`; zeros where no token is visible ----
        int todo = b1 - b0 > warp ? (int)((b1 - b0 - warp + W - 1) / W) : 0;  // this warp's units
        int pi = (int)(b0 + warp - p.start);                                  // the next one, within p's item
        const int *table_row = nullptr;  // of p's item, and its cache head's first value in a page
        int head_at = 0;
        auto place = [&]() {
            table_row = a.table + (size_t)p.r * a.pitch;
            head_at = (p.tile / tiles_a_head) * a.page_size * D;
        };
        place();
        int page_ahead = -1, unit_ahead = 0, at_ahead = 0;
        auto look_up = [&]() {  // where the next request finds its unit
            if (todo == 0) return;
            if (pi >= p.s.n) {
                do {
                    pi -= p.s.n;
                    p.next(a, tiles);
                } while (pi >= p.s.n);
                place();
            }
            unit_ahead = pi < p.s.us ? pi : p.s.ul + (pi - p.s.us);
            const int page = (int)(((unsigned long long)(unsigned)unit_ahead * div.mul) >> div.shift);
            page_ahead = table_row[page];
            at_ahead = head_at + (unit_ahead * kUnit - page * a.page_size) * D;
        };
        constexpr int CH = C::kRow / 16;  // 16-byte chunks a row
        constexpr int RP = 32 / CH;       // rows a pass of the warp's lanes
        constexpr int NX = kUnit / RP;    // passes
        const int ch = lane % CH, row0 = lane / CH;
        uint32_t kd[NX], vd[NX];  // where this lane's chunks go in a stage
#pragma unroll
        for (int x = 0; x < NX; ++x) {
            const int row = x * RP + row0;
            kd[x] = ring_s + row * C::kRow + key_chunk<D, Q8>(row, ch) * 16;
            vd[x] = ring_s + C::kVals + row * C::kRow + value_chunk<D, Q8>(row, ch) * 16;
        }
        const unsigned char *const kl = static_cast<const unsigned char *>(a.k) + lane * 16;
        const unsigned char *const vl = static_cast<const unsigned char *>(a.v) + lane * 16;
        const unsigned char *const sl =
            reinterpret_cast<const unsigned char *>(lane < 16 ? a.ks : a.vs) + (lane & 15) * (NB * 4);
        const uint32_t sd = ring_s + 2 * C::kVals + lane * (NB * 4);  // K's scales on lanes 0-15, V's on 16-31
        int slot = 0;
        unsigned whole_bits = 0;  // bit: the stage's unit lies on a page and all its tokens are visible
        unsigned there_bits = 0;  // bit: it lies on a page
        auto request = [&]() {
            if (todo > 0) {
                const bool there = (unsigned)page_ahead < (unsigned)a.pages;
                const int j0 = unit_ahead * kUnit;
                const bool whole = there && j0 + kUnit <= p.s.end && (j0 >= p.s.lo || j0 + kUnit <= a.sinks);
                const unsigned bit = 1u << slot;
                there_bits = there ? there_bits | bit : there_bits & ~bit;
                whole_bits = whole ? whole_bits | bit : whole_bits & ~bit;
                const long long at = there ? page_ahead * a.page_stride + at_ahead : 0;
                const uint32_t dst = slot * C::kStage;
                const unsigned char *kp = kl + at * (Q8 ? 1 : 2), *vp = vl + at * (Q8 ? 1 : 2);
                if (whole) {
#pragma unroll
                    for (int x = 0; x < NX; ++x) {
                        cp16(dst + kd[x], kp + x * 512);
                        cp16(dst + vd[x], vp + x * 512);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < NX; ++x) {
                        const int j = j0 + x * RP + row0;
                        const bool ok = there && j < p.s.end && (j >= p.s.lo || j < a.sinks);
                        cp16(dst + kd[x], ok ? kp + x * 512 : a.k, ok);
                        cp16(dst + vd[x], ok ? vp + x * 512 : a.v, ok);
                    }
                }
                if (Q8) {
                    const int j = j0 + (lane & 15);
                    const bool ok = whole || (there && j < p.s.end && (j >= p.s.lo || j < a.sinks));
                    const void *src = ok ? static_cast<const void *>(sl + at / 8) : a.ks;
                    if (NB == 4) cp16(dst + sd, src, ok);
                    else cp8(dst + sd, src, ok);
                }
                --todo;
                pi += W;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
            look_up();
        };
        look_up();
#pragma unroll
        for (int x = 0; x < C::kStages - 1; ++x) request();

        // Where this lane reads in a stage.  Over a Q8_0 cache rows g and g + 8 of the score product are tokens ta and
        // ta + 2, so that the weights come out in the token order of the transposed codes.
        const int ta = 4 * (g >> 1) + (g & 1);
        uint32_t kr[NB], vr[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            kr[b] = ring_s + ta * C::kRow + key_chunk<D, true>(ta, 2 * b) * 16 + t * 8;
            const int row = lane & 15;
            vr[b] = ring_s + C::kVals + row * C::kRow + value_chunk<D, true>(row, 2 * b + (lane >> 4)) * 16;
        }
        const uint32_t sr = ring_s + 2 * C::kVals + ta * (NB * 4);
        int ci = (int)(b0 + warp - c.start);  // the next unit to compute, within c's item
        int stage = 0;
        while (c.start < b1) {
            const int seg = (int)min((long long)c.s.n, b1 - c.start);  // c's units end here, or at the span's end
            const int kv_head = c.tile / tiles_a_head;
            const int head0 = kv_head * a.group + (c.tile % tiles_a_head) * (8 * NT);
            const int heads = min(8 * NT, (kv_head + 1) * a.group - head0);
            // ---- this item's queries as B fragments (8 heads a tile; absent heads are zeros) ----
            uint32_t qf[NT][KS][2];
            float off[NT][Q8 ? NB : 1][2];
            float sc[NT][2];  // scale * log2(e) of this lane's two heads (2t, 2t + 1)
            float m[NT][2], l[NT][2], o[NT][KS][4];
            // Over a Q8_0 cache a head's 32 values of block b in o are in units of 1 / per[n][b], a power of two that
            // follows the largest p * scale met: the weights p * scale * per then keep fp16's 11 bits down to 2^-22 of
            // the largest, however far apart the scales of tokens that weigh much and little are.
            uint32_t per[NT][Q8 ? NB : 1][2];  // as fp32 bits
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < (Q8 ? NB : 1); ++b) per[n][b][0] = per[n][b][1] = kMostPer << 23;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint16_t *qr = a.q + (size_t)c.r * a.ldq + (size_t)(head0 + 8 * n + g) * D;
                const bool ok = 8 * n + g < heads;
                if (!Q8) {
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            qf[n][k][x] = ok ? *reinterpret_cast<const uint32_t *>(qr + 16 * k + 8 * x + 2 * t) : 0u;
                    sc[n][0] = sc[n][1] = a.scale * kLog2e;
                } else {
                    // The keys are exact fp16 integers, so q is taken in fp16 too, exactly: scaled by a power of two
                    // to a largest magnitude in [2^9, 2^10) (values 2^-23 of the largest and smaller lose bits that
                    // fp32 sums would not hold).  Lane t holds values 8t .. 8t + 7 of each 32, as the keys' lanes do.
                    uint32_t mx = 0u;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint4 v = ok ? *reinterpret_cast<const uint4 *>(qr + 32 * b + 8 * t) : make_uint4(0, 0, 0, 0);
                        qf[n][2 * b][0] = v.x; qf[n][2 * b][1] = v.y; qf[n][2 * b + 1][0] = v.z; qf[n][2 * b + 1][1] = v.w;
                        const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx = max(mx, max(vv[e] & 0x7FFFu, (vv[e] >> 16) & 0x7FFFu));
                    }
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    // exponent field of the largest; subnormals count as the smallest normal
                    const int ex = min(max((int)(mx >> 7), 1), 254);
                    const int up = min(127 + 9 - ex, 126);  // q * 2^up
                    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t v = qf[n][k][x];
                            const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * f,
                                                                __uint_as_float(v & 0xFFFF0000u) * f);
                            qf[n][k][x] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    // The keys enter as code + 1152 (one instruction a pair): each block's sum begins at -1152 times the
                    // sum of its fp16 queries.  The detour costs fp32 about 2^-24 * 1152 sum |q| a block, some 20
                    // times the rounding of the plain sum and 1e-5 of a score.
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float sum = 0.0f;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t v = qf[n][2 * b + (x >> 1)][x & 1];
                            const float2 f2 = __half22float2(*reinterpret_cast<const __half2 *>(&v));
                            sum += f2.x + f2.y;
                        }
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            off[n][b][x] = -1152.0f * __shfl_sync(0xffffffffu, sum, (2 * t + x) * 4);
                    }
                    const float back = __uint_as_float((uint32_t)(127 - up) << 23);  // 2^-up
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        sc[n][x] = __shfl_sync(0xffffffffu, back, (2 * t + x) * 4) * (a.scale * kLog2e);
                }
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[n][k][x] = 0.0f;
            }
            // ---- this warp's units of the item ----
            for (; ci < seg; ci += W) {
                asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
                __syncwarp();  // every lane's copies of the stage have landed; the stage read last is free
                request();
                const uint32_t at = stage * C::kStage;
                const bool whole = (whole_bits >> stage) & 1u, there = (there_bits >> stage) & 1u;
                stage = stage + 1 == C::kStages ? 0 : stage + 1;
                // ---- s = q k: rows of tokens ja (s[0], s[1]) and jb (s[2], s[3]), heads 2t and 2t + 1 ----
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
                if (!Q8) {
                    const int row = lane & 15;
                    const uint32_t base = ring_s + at + row * C::kRow;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t kf[4];
                        ldsm4(kf, base + (((2 * k + (lane >> 4)) ^ (row & 7)) << 4));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_bf16(s[n], kf, qf[n][k][0], qf[n][k][1]);
                    }
                } else {
                    float d0[NB], d1[NB];
                    load_scales<NB>(d0, at + sr);
                    load_scales<NB>(d1, at + sr + 2 * NB * 4);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {  // lane t: codes 8t .. 8t + 7 of the block
                        const uint2 r0 = lds64(at + kr[b]), r1 = lds64(at + kr[b] + 2 * C::kRow);
                        const uint32_t x0 = r0.x ^ 0x80808080u, y0 = r0.y ^ 0x80808080u;
                        const uint32_t x1 = r1.x ^ 0x80808080u, y1 = r1.y ^ 0x80808080u;
                        const uint32_t f0[4] = {biased_f16x2<0>(x0), biased_f16x2<0>(x1), biased_f16x2<2>(x0),
                                                biased_f16x2<2>(x1)};
                        const uint32_t f1[4] = {biased_f16x2<0>(y0), biased_f16x2<0>(y1), biased_f16x2<2>(y0),
                                                biased_f16x2<2>(y1)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float z[4];
                            mma_f16(z, f0, qf[n][2 * b][0], qf[n][2 * b][1], off[n][b][0], off[n][b][1]);
                            mma_f16(z, f1, qf[n][2 * b + 1][0], qf[n][2 * b + 1][1]);
                            s[n][0] = fmaf(d0[b], z[0], s[n][0]);
                            s[n][1] = fmaf(d0[b], z[1], s[n][1]);
                            s[n][2] = fmaf(d1[b], z[2], s[n][2]);
                            s[n][3] = fmaf(d1[b], z[3], s[n][3]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[n][x] *= sc[n][x & 1];
                if (!whole) {
                    const int u = ci < c.s.us ? ci : c.s.ul + (ci - c.s.us);
                    const int ja = u * kUnit + (Q8 ? ta : g), jb = ja + (Q8 ? 2 : 8);
                    const bool va = there && ja < c.s.end && (ja >= c.s.lo || ja < a.sinks);
                    const bool vb = there && jb < c.s.end && (jb >= c.s.lo || jb < a.sinks);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[n][x] = (x < 2 ? va : vb) ? s[n][x] : -INFINITY;
                }
                // ---- weights p = 2^(s - m) ----
                float p[NT][4];
                bool above = !whole;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        p[n][x] = s[n][x] - m[n][x & 1];
                        above = above || !(p[n][x] <= kSlack);  // true of -inf less -inf, while all scores were -inf
                    }
                if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float mx = fmaxf(s[n][x], s[n][x + 2]);
#pragma unroll
                            for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                            if (Q8) mx = ceilf(mx);  // maxima are whole numbers: what follows takes powers of two
                            mx = fmaxf(mx, m[n][x]);
                            if (!Q8) {
                                const float f = mx == m[n][x] ? 1.0f : ex2(m[n][x] - mx);
                                l[n][x] *= f;
#pragma unroll
                                for (int k = 0; k < KS; ++k) {
                                    o[n][k][x] *= f;
                                    o[n][k][x + 2] *= f;
                                }
                            } else if (mx != m[n][x]) {  // o stays, its units shrink with the weights
                                const int down = (int)fminf(mx - m[n][x], 1024.0f);
                                l[n][x] *= two_to_minus(down);
#pragma unroll
                                for (int b = 0; b < NB; ++b) {
                                    const int e = (int)(per[n][b][x] >> 23) + down;
                                    if (e > kMostPer) scale_block(o[n][2 * b], o[n][2 * b + 1], x, two_to_minus(e - kMostPer));
                                    per[n][b][x] = (uint32_t)min(e, kMostPer) << 23;
                                }
                            }
                            m[n][x] = mx;
                            const float m0 = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet: weights 0
                            p[n][x] = s[n][x] - m0;
                            p[n][x + 2] = s[n][x + 2] - m0;
                        }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) p[n][x] = ex2(p[n][x]);
                    l[n][0] += p[n][0] + p[n][2];
                    l[n][1] += p[n][1] + p[n][3];
                }
                // ---- O^T += V^T P^T ----
                if (!Q8) {
                    uint32_t pf[NT][2];  // weights rounded to bf16, v's type, for the product; their sum is fp32
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        pf[n][0] = transposed8x8(bf16x2(p[n][0], p[n][1]));
                        pf[n][1] = transposed8x8(bf16x2(p[n][2], p[n][3]));
                    }
                    const int row = (lane & 7) + ((lane >> 4) << 3);
                    const uint32_t base = ring_s + at + C::kVals + row * C::kRow;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t vf[4];
                        ldsm4t(vf, base + (((2 * k + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_bf16(o[n][k], vf, pf[n][0], pf[n][1]);
                    }
                } else {
                    // The codes are exact in fp16; the tokens' scales go to the weights, p * scale * per, rounded to fp16.
                    float da[NB], db[NB];
                    load_scales<NB>(da, at + sr + C::kScales);
                    load_scales<NB>(db, at + sr + C::kScales + 2 * NB * 4);
                    uint32_t wa[NT][NB], wb[NT][NB];  // of tokens ja and jb
                    auto weigh = [&]() {
                        __half2 top = __float2half2_rn(0.0f);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                wa[n][b] = weights_f16x2(p[n][0], p[n][1], da[b], per[n][b]);
                                wb[n][b] = weights_f16x2(p[n][2], p[n][3], db[b], per[n][b]);
                                top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&wa[n][b])));
                                top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&wb[n][b])));
                            }
                        // some weight above 2^15 (0x7800; infinity is 0x7C00)
                        return ((*reinterpret_cast<const uint32_t *>(&top) + 0x07FF07FFu) & 0x80008000u) != 0u;
                    };
                    if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int b = 0; b < NB; ++b)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    float mx = fmaxf(p[n][x] * fabsf(da[b]), p[n][x + 2] * fabsf(db[b]));
#pragma unroll
                                    for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                                    const int old = (int)(per[n][b][x] >> 23);
                                    if (mx * __uint_as_float(per[n][b][x]) > 32768.0f) {
                                        // the largest weight comes to [2^8, 2^9)
                                        const int e = 127 + 127 + 8 - (int)(__float_as_uint(mx) >> 23);
                                        scale_block(o[n][2 * b], o[n][2 * b + 1], x, two_to_minus(old - e));
                                        per[n][b][x] = (uint32_t)e << 23;
                                    }
                                }
                        weigh();
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t w[4];
                        ldsm8t(w, at + vr[b]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) w[x] ^= 0x80808080u;
                        const uint32_t v0[4] = {codes_f16x2<0>(w[0]), codes_f16x2<0>(w[1]), codes_f16x2<2>(w[0]),
                                                codes_f16x2<2>(w[1])};
                        const uint32_t v1[4] = {codes_f16x2<0>(w[2]), codes_f16x2<0>(w[3]), codes_f16x2<2>(w[2]),
                                                codes_f16x2<2>(w[3])};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t q0 = transposed8x8(wa[n][b]);
                            const uint32_t q1 = transposed8x8(wb[n][b]);
                            mma_f16(o[n][2 * b], v0, q0, q1);
                            mma_f16(o[n][2 * b + 1], v1, q0, q1);
                        }
                    }
                }
            }
            // ---- the item's end: the warps' parts through shared memory ----
            float *po = reinterpret_cast<float *>(parts + warp * C::kPart);
            float2 *pml = reinterpret_cast<float2 *>(parts + warp * C::kPart + NT * 8 * D * 4);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], sh);
                    float *row = po + (8 * n + 2 * t + x) * D;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const float f = Q8 ? __uint_as_float(0x7F000000u - per[n][Q8 ? k / 2 : 0][x]) : 1.0f;
                        row[16 * k + g] = o[n][k][x] * f;
                        row[16 * k + g + 8] = o[n][k][x + 2] * f;
                    }
                    if (g == 0) pml[8 * n + 2 * t + x] = make_float2(m[n][x], l[n][x]);
                }
            __syncthreads();
            const long long end = c.start + c.s.n;
            const int c0 = (int)(c.start / span), c1 = (int)((end - 1) / span);  // the CTAs that share the item
            float *base = reinterpret_cast<float *>(a.work + kAttnCounterBytes);
            // four values of one head a thread and pass
            constexpr int PASS = NT * 8 * (D / 4);
            for (int e = tid; e < PASS; e += 32 * W) {
                const int h = e / (D / 4), d4 = e % (D / 4);
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    mx = fmaxf(mx, reinterpret_cast<const float2 *>(parts + w * C::kPart + NT * 8 * D * 4)[h].x);
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 ml = reinterpret_cast<const float2 *>(parts + w * C::kPart + NT * 8 * D * 4)[h];
                    const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - mx);
                    const float4 v = *reinterpret_cast<const float4 *>(parts + w * C::kPart + (h * D + 4 * d4) * 4);
                    sum = fmaf(ml.y, f, sum);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
                if (c0 == c1) {
                    if (h < heads) {
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                        *reinterpret_cast<uint2 *>(a.out + (size_t)c.r * a.ldo + (size_t)(head0 + h) * D + 4 * d4) =
                            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
                    }
                } else {
                    float *part = base + ((long long)blockIdx.x * 2 + (c.start >= b0)) * kDecodePartFloats;
                    *reinterpret_cast<float4 *>(part + h * D + 4 * d4) = acc;
                    if (d4 == 0) *reinterpret_cast<float2 *>(part + kDecodeHeads * 128 + 2 * h) = make_float2(mx, sum);
                }
            }
            if (c0 != c1) {
                // ---- an item shared with other CTAs: whoever arrives last adds the parts, in span order ----
                int *count = reinterpret_cast<int *>(a.work) + c0;
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    const int seen = atomicAdd(count, 1);
                    s_last = seen == c1 - c0;
                    if (s_last) *count = 0;
                }
                __syncthreads();
                if (s_last) {
                    __threadfence();
                    for (int e = tid; e < PASS; e += 32 * W) {
                        const int h = e / (D / 4), d4 = e % (D / 4);
                        if (h >= heads) continue;
                        float mx = -INFINITY, sum = 0.0f;
                        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int x = c0; x <= c1; ++x) {
                            const float *part = base + ((long long)x * 2 + (x == c0)) * kDecodePartFloats;
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + kDecodeHeads * 128 + 2 * h));
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + h * D + 4 * d4));
                            const float nm = fmaxf(mx, ml.x);
                            const float fa = mx == nm ? 1.0f : ex2(mx - nm);
                            const float fb = ml.x == nm ? 1.0f : ex2(ml.x - nm);
                            mx = nm;
                            sum = sum * fa + ml.y * fb;
                            acc.x = acc.x * fa + v.x * fb;
                            acc.y = acc.y * fa + v.y * fb;
                            acc.z = acc.z * fa + v.z * fb;
                            acc.w = acc.w * fa + v.w * fb;
                        }
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                        *reinterpret_cast<uint2 *>(a.out + (size_t)c.r * a.ldo + (size_t)(head0 + h) * D + 4 * d4) =
                            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
                    }
                }
            }
            __syncthreads();  // the parts are free for the next item
            if (c.start + seg == b1) break;
            ci -= c.s.n;
            c.next(a, tiles);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // ---- rows that see nothing ----
    for (int r = blockIdx.x; r < a.R; r += gridDim.x)
        if (seen_of(a, a.lens[r]).n == 0)
            for (int e = tid; e < a.heads * D / 8; e += 32 * W)
                *reinterpret_cast<uint4 *>(a.out + (size_t)r * a.ldo + 8 * e) = make_uint4(0u, 0u, 0u, 0u);
}

template <int D, bool Q8, int NT> cudaError_t launch_one(const AttnArgs &a, int sms, cudaStream_t stream) {
    using C = Cfg<D, Q8, NT>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(attn_decode_kernel<D, Q8, NT>, C::kSmem, &allowed);
    if (e != cudaSuccess) return e;
    const int tiles_a_head = (a.group + 8 * NT - 1) / (8 * NT);
    return kv_launch(attn_decode_kernel<D, Q8, NT>, dim3((unsigned)sms, 1, 1), 32 * C::kWarps, C::kSmem, stream, a,
                     tiles_a_head, unit_div(a.page_size / kUnit));
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs &a, int dim, bool q8, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count_of_device(&sms);
    if (e != cudaSuccess) return e;
    if (sms > kAttnMaxCtas) sms = kAttnMaxCtas;
    const bool wide = a.group > 8;  // 16 query heads a pass over the keys instead of 8
    if (dim == 128) {
        if (q8) return wide ? launch_one<128, true, 2>(a, sms, stream) : launch_one<128, true, 1>(a, sms, stream);
        return wide ? launch_one<128, false, 2>(a, sms, stream) : launch_one<128, false, 1>(a, sms, stream);
    }
    if (q8) return wide ? launch_one<64, true, 2>(a, sms, stream) : launch_one<64, true, 1>(a, sms, stream);
    return wide ? launch_one<64, false, 2>(a, sms, stream) : launch_one<64, false, 1>(a, sms, stream);
}

}  // namespace q8
