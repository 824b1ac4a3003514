// Products of more than 16 rows over 4-bit weights on the 5th-generation tensor cores: one CTA computes 128 columns for up
// to 256 rows over its range of K.
//
// The weights are the MMA's A operand (M = 128 columns of W), the activations B (N = up to 256 rows), so that one pass over
// the weight and one conversion of it serve all rows of the tile, and each lane of the accumulator is one column: a group's
// scale is one number for a thread that folds.  A group's sums (the codes less zero points and the activations exact in
// bf16) go to a fresh accumulator in tensor memory and are folded with its scales into fp32 carries in registers.  A gated
// pair's tile is two strips of the gate and the same two of the up projection, 64 columns of output.
//
// 16 warps, one CTA per SM, K in chunks of 128 rows and steps of 64:
//   fold        warps 0-3 (FW = 1) or 0-7 (FW = 2, half of the rows each): a thread reads its lane of a finished accumulator,
//               times its column's scale (packed fp32x2), into at most 128 carries
//   convert     the warps up to 11, in two teams that take steps in turn: codes to bf16 in the 128-byte swizzle (two
//               columns and two 32-row blocks a thread at a time; odd columns store their second block first, so that
//               eight lanes' 16-byte stores fall on all banks)
//   load        warp 12: units by bulk copies; warp 14: activations by TMA (64 values x the tile's rows; rows past m are
//               zeros).  One warp for both kept the activations of a chunk behind the fold of the one before.
//   multiply    warp 13, converged, one lane elected for the instructions (a lane alone in the loop was 2 to 4% slower)
// The fold's 128 carries and a look at tensor memory want 184 to 208 registers a thread; the others give theirs up (setmaxnreg,
// of the launch's 512 x 128).
//
// What bounds it: up to 128 rows the latency of the hand-overs, a step's 450 clocks of waits and instructions of the multiplying
// warp and 600 of a team, beside 200 of MMAs.  Beyond, in groups of 32 and 64, the fold (256 rows of 4096 x 9000 in groups of
// 32 40.9 us, with the fold left out 29.7; the gated pair of 301 rows in groups of 64 92.4 and 78.2, without conversion
// 83.4); in groups of 128 no one part: 512 rows of 4096 x 14336 take 49.1 us, without conversion 44.5, without MMAs 46.8,
// without activations 46.8, without the fold 47.7, and 32.9 with all four left out, of which the copies of the units, the
// hand-overs and the two launches' beginnings and ends remain.  Hence waits without divergence and loops whose counts the
// compiler knows: with branches on the tile's rows 24 rows of 4096 x 9000 in groups of 32 took 30 us, without 18, and, handing
// over four groups at a time, 12.9.  Measured: 512 rows of 4096 x 14336, groups of 128, 49 us (1.22 PFLOP/s); the gated pair of
// 301 rows, 4096 x 14336, groups of 64, 92 us; 61 rows of 2048 x 2048, groups of 32, with the norm 9.2 us.  The converted codes
// in tensor memory instead of shared memory (640 threads, tiles of 160 rows) took 71 us for the first: a step then costs 600
// clocks for 128 rows.
//
// Where the tiles do not fill the SMs, K is split over a cluster, whose carries are added in rank order through shared
// memory.  Every wait ends after some two seconds: the CTA then stops, waits as long for what is in flight, and reports a
// fault.  No such clock starts while the kernel before may still run, however long that takes: a warp waits for its end
// (griddepcontrol.wait) ahead of the first barrier that hangs on its results or on room that those free.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "q8_attn.h"
#include "q8_launch.h"
#include "q8_w4_device.cuh"

namespace q8 {
namespace {

constexpr int kCols = 128;     // columns of W in a tile
constexpr int kStepK = 64;     // rows of K in a step: 128 bytes of bf16
constexpr int kChunkK = 128;   // rows of K in a raw stage
constexpr int kThreadsG = 512;
constexpr int kConvertEnd = 12, kLoadWarp = 12, kMmaWarp = 13, kXWarp = 14;
constexpr int kOperand = kCols * kStepK * 2;  // 16 KB: one converted step
constexpr int kMostRows = 256;
constexpr int kMaxSmemG = 227 * 1024;
constexpr int kMaxStages = 8, kMaxAcc = 4;
constexpr int kMostSplit = 4;  // clusters of eight whole SMs find no place for all at once (61 rows of 2048 x 2048 13.3 -> 19.6 us)

__device__ unsigned int g_w4_gemm_fault = 0;

struct Gemm4 {
    int tile0;   // the launch's first tile of columns
    int rows;    // of a tile: kRows of the kernel
    int slots;   // stages of converted weights and activations
    int raws;    // stages of units
    int accs;    // sets of accumulators
    int ks;      // CTAs of a cluster splitting K
    int prefetch;
};

struct Control {
    uint64_t raw_full[kMaxStages], raw_empty[kMaxStages], full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[kMaxAcc], acc_empty[kMaxAcc], drain;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ bool wait(uint64_t *bar, unsigned parity, volatile int *abort) {
    if (w4_look(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (w4_look(bar, parity)) return true;
    } while (!*abort && clock64() - t0 < kW4Patience);
    if (!*abort) {
        *abort = 1;
        atomicOr(&g_w4_gemm_fault, kW4Fault);
    }
    return false;
}
// The same by a whole warp, without a branch that its lanes could take differently.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, unsigned parity, volatile int *abort) {
    if (__all_sync(0xffffffffu, w4_look(bar, parity))) return true;
    const long long t0 = clock64();
    do {
        if (__all_sync(0xffffffffu, w4_look(bar, parity))) return true;
    } while (__all_sync(0xffffffffu, !*abort && clock64() - t0 < kW4Patience));
    if (!*abort) {
        *abort = 1;
        atomicOr(&g_w4_gemm_fault, kW4Fault);
    }
    return false;
}

__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(w4_smem(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptors of K-major operands in the 128-byte swizzle: rows of 128 bytes, groups of 8 rows 1024 bytes
// apart (the high word), the address (the low one).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n"
        " mov.b64 db, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
// 16 or 64 columns of the warp's lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld64(uint32_t a, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, "
        "[%64];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
        : "r"(a));
}
__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint32_t lo, uint32_t hi) {
    asm("{\n .reg .b64 v;\n mov.b64 v, {%2, %3};\n fma.rn.f32x2 %0, %1, v, %0;\n}" : "+l"(d) : "l"(a), "r"(lo), "r"(hi));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int k, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            w4_smem(dst)),
        "l"(map), "r"(k), "r"(row), "r"(w4_smem(bar))
        : "memory");
}

// Two columns (g and g + 8 of a 16-column tile) of rows 32 blk + 8t .. + 7 of a step, blk = first and then the other, as
// they go into the operand: row n of 128 bytes, 16-byte chunk c at c ^ (n % 8).
__device__ __forceinline__ void store8(unsigned char *row, int chunk, int g, uint32_t w, uint32_t zero) {
    *reinterpret_cast<uint4 *>(row + ((chunk ^ g) << 4)) =
        make_uint4(w4_pair<0>(w, zero), w4_pair<1>(w, zero), w4_pair<2>(w, zero), w4_pair<3>(w, zero));
}

// Groups whose sums are handed to the fold at a time: as many of a chunk as fit twice into tensor memory, where tiles are small
// (24 rows of 4096 x 9000 in groups of 32 18.3 -> 12.9 us, in groups of 64 12.6 -> 12.1; 64 rows 20.1 -> 15.1 and 15.0 -> 13.5);
// one in tiles of 96 rows and more, whose sums then take long to read (100 rows 25.4 -> 31.9 us with two, 17.1 -> 19.0).
constexpr int groups_at_once(int G, int rows) {
    int t = rows <= 64 ? kChunkK / G : 1;
    while (t > 1 && 2 * t * rows > 512) t /= 2;
    return t;
}

template <int G, int FW, int PIECES>
__global__ void __launch_bounds__(kThreadsG, 1)
    gemm4_kernel(const __grid_constant__ W4Args a, const Gemm4 p, const __grid_constant__ CUtensorMap xmap) {
    namespace cg = cooperative_groups;
    constexpr int CG = kChunkK / G;  // groups of a chunk
    constexpr int kConvert = 4 * FW, kTeam = FW == 1 ? 4 : 2;  // warps of a team, of two
    constexpr int kLook = FW == 1 || PIECES < 5 ? 64 : PIECES == 5 ? 80 : PIECES == 6 ? 48 : 32;  // columns of tensor memory
    constexpr int kRows = 16 * FW * PIECES, kHalf = 16 * PIECES;  // of the tile; of a folding thread
    constexpr int T = groups_at_once(G, kRows);
    extern __shared__ __align__(1024) unsigned char smem_g[];
    const int chunk_bytes = CG * a.unit, raw_bytes = 4 * chunk_bytes;
    const int x_bytes = kRows * 128, slot_bytes = kOperand + x_bytes;
    unsigned char *slots = smem_g, *raws = slots + p.slots * slot_bytes;
    Control &ctl = *reinterpret_cast<Control *>(raws + p.raws * raw_bytes);
    volatile int *abort = &ctl.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the tile: four strips of one part, or two of the gate and then two of the up projection
    const bool pair = a.epi == kW4Glu;
    const int width = pair ? 2 : 4;  // strips of output
    int part = 0, tile = p.tile0 + blockIdx.x;
    if (!pair)
        for (int first = 0, tiles;; ++part, tile -= tiles, first = a.part[part - 1].strip_end) {
            tiles = (a.part[part].strip_end - first + 3) / 4;
            if (tile < tiles || part + 1 == a.nparts) break;
        }
    const W4Part &to = a.part[part];
    const int here = min(width, to.Np / kW4Strip - width * tile);  // strips that exist
    const int row0 = blockIdx.y * kRows;
    const int groups = a.K / G, chunks = (groups + CG - 1) / CG;
    const int c0 = (int)((long long)chunks * blockIdx.z / p.ks), c1 = (int)((long long)chunks * (blockIdx.z + 1) / p.ks);
    const int rows_k = min(a.K, c1 * kChunkK) - c0 * kChunkK;  // of K in this CTA's range
    const int n_chunks = c1 - c0, n_steps = (rows_k + kStepK - 1) / kStepK, n_groups = rows_k / G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.raws; ++i) {
            w4_bar_init(&ctl.raw_full[i], 1);
            w4_bar_init(&ctl.raw_empty[i], 2 * kTeam + 4 * FW);  // a team for each of two steps, the folding warps
        }
        for (int i = 0; i < p.slots; ++i) {
            w4_bar_init(&ctl.full[i], kTeam + 1);  // a team, the activations' announcement
            w4_bar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < p.accs; ++i) {
            w4_bar_init(&ctl.acc_full[i], 1);
            w4_bar_init(&ctl.acc_empty[i], 4 * FW);
        }
        w4_bar_init(&ctl.drain, 1);
        ctl.abort = 0;
        w4_bar_fence();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(w4_smem(&ctl.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl.tmem;

    if (warp < 4 * FW) {
        // ---- fold ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FW == 1 ? 208 : 184));
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint64_t acc[kHalf / 2];  // two rows each
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) acc[i] = 0;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int first = (warp >> 2) * kHalf;
        int raw = 0, buf = 0;
        unsigned raw_phase = 0, acc_phase = 0;
        for (int gi = 0; gi < n_groups;) {
            if ((gi & (CG - 1)) == 0 && !warp_wait(&ctl.raw_full[raw], raw_phase, abort)) break;
            if (!warp_wait(&ctl.acc_full[buf], acc_phase, abort)) break;
            fence_after();
            // strip (warp % 4) of the tile is the warp's lanes
            const unsigned char *u =
                raws + raw * raw_bytes + (warp & 3) * chunk_bytes + (gi & (CG - 1)) * a.unit + 16 * G + 2 * lane;
            uint32_t at = tmem + lanes + (uint32_t)(buf * T * kRows + first);
            const int end = min(gi + T, n_groups);
            do {
                const float f = w4_scale(*reinterpret_cast<const uint16_t *>(u), a.bf16);
                uint64_t s;
                asm("mov.b64 %0, {%1, %1};" : "=l"(s) : "r"(__float_as_uint(f)));
#pragma unroll
                for (int c = 0; c < kHalf; c += kLook) {
                    uint32_t v[kLook];
                    constexpr int kLong = kLook >= 64 && kHalf >= 64 ? 64 : 0;
                    if (kLong && c + 64 <= kHalf) tmem_ld64(at + c, v);
#pragma unroll
                    for (int k = 0; k < kLook; k += 16)
                        if ((k >= kLong || c + 64 > kHalf) && c + k < kHalf) tmem_ld16(at + c + k, v + k);
                    tmem_wait();
#pragma unroll
                    for (int k = 0; k < kLook; k += 2)
                        if (c + k < kHalf) fma2(acc[(c + k) / 2], s, v[k], v[k + 1]);
                }
                u += a.unit, at += kRows;
            } while (++gi < end);
            fence_before();
            __syncwarp();
            const bool chunk_done = (gi & (CG - 1)) == 0;
            if (lane == 0) {
                w4_arrive(&ctl.acc_empty[buf]);
                if (chunk_done) w4_arrive(&ctl.raw_empty[raw]);
            }
            if (++buf == p.accs) buf = 0, acc_phase ^= 1;
            if (chunk_done && ++raw == p.raws) raw = 0, raw_phase ^= 1;
        }
        // The last group's sums are in: every MMA of the CTA is done, and with them every use of the operands, where the
        // carries go now, [rows][128].  Straight from registers to the output, a store and a residual's load at a time,
        // the same took 25 us for 256 rows.
        float *red = reinterpret_cast<float *>(smem_g);
        float *to = red + first * kCols + 32 * (warp & 3) + lane;
#pragma unroll
        for (int e = 0; e < kHalf; ++e) to[e * kCols] = __uint_as_float((uint32_t)(e & 1 ? acc[e / 2] >> 32 : acc[e / 2]));
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FW == 1 ? 96 : 72));
        if (warp < kConvertEnd) {
            // ---- convert ----
            const int team = (warp - kConvert) / kTeam, strip0 = (warp & (kTeam - 1)) * (4 / kTeam);
            const int g = lane >> 2, t = lane & 3, odd = g & 1;
            int raw = 0, slot = team;
            unsigned raw_phase = 0, phase = 1;  // a fresh barrier passes for the phase before its first
            const int early = p.prefetch ? min(p.slots, 2 * p.raws) : 0;  // steps that need nothing of the kernel before
            for (int j = team; j < n_steps; j += 2) {  // a team has one step of every chunk
                if (j >= early && j < early + 2) asm volatile("griddepcontrol.wait;" ::: "memory");
                if (!warp_wait(&ctl.raw_full[raw], raw_phase, abort)) break;
                if (!warp_wait(&ctl.empty[slot], phase, abort)) break;
#pragma unroll
                for (int k = 0; k < 4 / kTeam; ++k) {
                    const int strip = strip0 + k;
                    const unsigned char *from = raws + raw * raw_bytes + strip * chunk_bytes;
                    unsigned char *operand = slots + slot * slot_bytes + strip * 32 * 128 + g * 128;
                    // the step's units: half of one, one, or two
                    const unsigned char *u0 = from + (j & 1) * (G == 128 ? 1024 : G == 64 ? a.unit : 2 * a.unit);
                    uint32_t zero[2][2][2];  // [block][tile][h]
                    const unsigned char *z = (G == 128 ? from : u0) + 16 * G + 64 + g;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                zero[b][jj][h] = !a.zeros         ? kW4Eight
                                                 : G > 32 && b == 1 ? zero[0][jj][h]
                                                                    : w4_zero(z[b * a.unit + 16 * jj + 8 * h]);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        uint4 w;
                        if (G == 32) {
                            const uint2 lo = *reinterpret_cast<const uint2 *>(u0 + 256 * jj + 8 * lane);
                            const uint2 hi = *reinterpret_cast<const uint2 *>(u0 + a.unit + 256 * jj + 8 * lane);
                            w = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        } else {
                            w = *reinterpret_cast<const uint4 *>(u0 + 512 * jj + 16 * lane);
                        }
                        const int first = odd ? 4 + t : t, second = first ^ 4;
                        unsigned char *row = operand + 16 * jj * 128;
                        store8(row, first, g, odd ? w.z : w.x, odd ? zero[1][jj][0] : zero[0][jj][0]);
                        store8(row, second, g, odd ? w.x : w.z, odd ? zero[0][jj][0] : zero[1][jj][0]);
                        store8(row + 8 * 128, first, g, odd ? w.w : w.y, odd ? zero[1][jj][1] : zero[0][jj][1]);
                        store8(row + 8 * 128, second, g, odd ? w.y : w.w, odd ? zero[0][jj][1] : zero[1][jj][1]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    w4_arrive(&ctl.full[slot]);
                    w4_arrive(&ctl.raw_empty[raw]);
                }
                if (++raw == p.raws) raw = 0, raw_phase ^= 1;
                if ((slot += 2) >= p.slots) slot -= p.slots, phase ^= 1;
            }
        } else if (warp == kLoadWarp) {
            // ---- load units (one lane) ----
            if (lane == 0) {
                const size_t strip_bytes = (size_t)groups * a.unit;
                const size_t at = (size_t)tile * width * strip_bytes + (size_t)c0 * chunk_bytes;
                const int early = p.prefetch ? p.raws : 0;  // chunks that find an empty stage
                int i = 0, raw = 0;
                unsigned raw_phase = 1;
                for (; i < n_chunks; ++i) {
                    if (i == early) asm volatile("griddepcontrol.wait;" ::: "memory");
                    if (!wait(&ctl.raw_empty[raw], raw_phase, abort)) break;
                    const unsigned bytes = (unsigned)(min(CG, groups - (c0 + i) * CG) * a.unit);
                    w4_arrive_tx(&ctl.raw_full[raw], bytes * (unsigned)(pair ? 2 * here : here));
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int of = pair ? s & 1 : s;
                        if (of < here)
                            w4_copy(raws + raw * raw_bytes + s * chunk_bytes,
                                    (pair && s > 1 ? a.part[1].w : to.w) + at + of * strip_bytes + (size_t)i * chunk_bytes,
                                    bytes, &ctl.raw_full[raw]);
                    }
                    if (++raw == p.raws) raw = 0, raw_phase ^= 1;
                }
                if (*abort)  // what was asked for lands before the memory is used again
                    for (int k = max(0, i - p.raws); k < i; ++k) w4_wait(&ctl.raw_full[k % p.raws], (k / p.raws) & 1);
            }
            __syncwarp();
        } else if (warp == kXWarp) {
            // ---- load activations (one lane) ----
            if (lane == 0) {
                asm volatile("griddepcontrol.wait;" ::: "memory");
                int j = 0, slot = 0;
                unsigned phase = 1;
                for (; j < n_steps; ++j) {
                    if (!wait(&ctl.empty[slot], phase, abort)) break;
                    w4_arrive_tx(&ctl.full[slot], (unsigned)x_bytes);
                    tma_rows(slots + slot * slot_bytes + kOperand, &xmap, c0 * kChunkK + j * kStepK, row0,
                             &ctl.full[slot]);
                    if (++slot == p.slots) slot = 0, phase ^= 1;
                }
                // `full` waits for the teams too, which may have stopped: time for the copies in flight instead
                if (*abort)
                    for (int k = max(0, j - p.slots); k < j; ++k) w4_wait(&ctl.full[k % p.slots], (k / p.slots) & 1);
            }
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ---- multiply ----
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kRows >> 3) << 17) |
                                   ((uint32_t)(kCols >> 4) << 24);
            int slot = 0, buf = 0;
            unsigned phase = 0, acc_phase = 1;
            uint32_t da = __shfl_sync(0xffffffffu, desc_low(w4_smem(slots)), 0);  // the slot's operand; its activations
            const uint32_t base = da, next = (uint32_t)slot_bytes >> 4, xat = (uint32_t)kOperand >> 4;
            for (int j = 0; j < n_steps; ++j) {
                const int ksteps = G > 32 ? 4 : min(4, (rows_k - j * kStepK) / 16);
                // a set of accumulators is of several steps, one, or half of one
                constexpr int kSteps = T * G / kStepK, kSets = kSteps ? 1 : 2;
                const int of = kSteps > 1 ? j & (kSteps - 1) : 0;  // the step in its set
                const int buf1 = buf + 1 == p.accs ? 0 : buf + 1;
                // (all looked at together where all are there)
                const unsigned phase1 = buf1 ? acc_phase : acc_phase ^ 1;
                const bool second = kSets == 2 && ksteps > 2;
                bool there = w4_look(&ctl.full[slot], phase) & w4_look(&ctl.acc_empty[buf], acc_phase);
                if (second) there &= w4_look(&ctl.acc_empty[buf1], phase1);
                if (!__all_sync(0xffffffffu, there)) {
                    bool ok = warp_wait(&ctl.full[slot], phase, abort) && warp_wait(&ctl.acc_empty[buf], acc_phase, abort);
                    if (second) ok = ok && warp_wait(&ctl.acc_empty[buf1], phase1, abort);
                    if (!ok) break;
                }
                const uint32_t d0 = tmem + (uint32_t)((buf * T + of * kStepK / G) * kRows), d1 = tmem + (uint32_t)(buf1 * kRows);
                const bool done = of == kSteps - 1 || j + 1 == n_steps;
                fence_after();
                if (elect()) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (G > 32 || s < ksteps) {
                            const uint32_t d = s * 16 < G ? d0 : kSets == 2 ? d1 : d0 + kRows;
                            mma(d, da + (32 * s >> 4), da + xat + (32 * s >> 4), idesc, 16 * s % G > 0 || (G > kStepK && of > 0));
                            if (kSets == 2 && s % 2) commit(&ctl.acc_full[s < 2 ? buf : buf1]);
                        }
                    if (kSets == 1 && done) commit(&ctl.acc_full[buf]);
                    commit(&ctl.empty[slot]);
                }
                __syncwarp();
                if (kSets == 2 || done)
                    for (int i = 0; i < (kSets == 2 ? ksteps / 2 : 1); ++i)
                        if (++buf == p.accs) buf = 0, acc_phase ^= 1;
                da += next;
                if (++slot == p.slots) slot = 0, phase ^= 1, da = base;
            }
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // All MMAs are done (the last group's commit was waited for) and all copies have landed, unless the CTA stopped.
    fence_before();
    __syncthreads();
    if (*abort && warp == kMmaWarp) {
        if (elect()) commit(&ctl.drain);
        w4_wait(&ctl.drain, 0);
    }
    __syncthreads();
    fence_after();

    // A rank's share of the tile's rows, the ranks' carries added in order, four columns a thread.
    const float *red = reinterpret_cast<float *>(smem_g);
    cg::cluster_group cluster = cg::this_cluster();
    if (p.ks > 1) cluster.sync();
    const int live = min(kRows, a.m - row0);
    const int r0 = live * (int)blockIdx.z / p.ks, r1 = live * ((int)blockIdx.z + 1) / p.ks;
    const int of_row = pair ? 16 : 32;  // lanes
    const int c = 4 * (lane % of_row), n = tile * width * kW4Strip + c;
    if (n < to.Np && !*abort) {
        auto total = [&](int at, float (&v)[4]) {
            float4 f = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(red, 0) + at);
#pragma unroll 2
            for (int k = 1; k < p.ks; ++k) {
                const float4 o = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(red, k) + at);
                f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
            }
            v[0] = kW4Unit * f.x, v[1] = kW4Unit * f.y, v[2] = kW4Unit * f.z, v[3] = kW4Unit * f.w;
        };
        constexpr int kTogether = 4;  // rows of a thread at a time
        const int apart = kThreadsG / of_row;
        for (int r = r0 + (int)threadIdx.x / of_row; r < r1; r += apart * kTogether) {
            float res[kTogether][4] = {};
            if (a.epi == kW4Residual) {
#pragma unroll
                for (int i = 0; i < kTogether; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (r + i * apart < r1 && n + e < to.N)
                            res[i][e] = __ldcg(a.res + (size_t)(row0 + r + i * apart) * to.Np + n + e);
            }
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                if (r + i * apart >= r1) break;
                float v[4];
                total((r + i * apart) * kCols + c, v);
                if (pair) {
                    float u[4];
                    total((r + i * apart) * kCols + kCols / 2 + c, u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = v[e] / (1.0f + expf(-v[e])) * u[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = n + e < to.N ? v[e] + res[i][e] : 0.0f;
                const size_t at = (size_t)(row0 + r + i * apart) * to.Np + n;
                if (to.y) *reinterpret_cast<float4 *>(to.y + at) = make_float4(v[0], v[1], v[2], v[3]);
                if (a.ybf) {
                    __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2 *>(a.ybf + at) =
                        make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
                }
            }
        }
    }
    if (p.ks > 1) cluster_sync_after_reads();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int G, int FW, int PIECES>
cudaError_t launch_kernel(const W4Args &a, const Gemm4 &p, int tiles, int smem, const CUtensorMap &map, cudaStream_t stream) {
    // the shares of setmaxnreg are of what the launch brings: a build that brings less is refused
    static const cudaError_t brings = [] {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, gemm4_kernel<G, FW, PIECES>);
        return e != cudaSuccess ? e : f.numRegs < 128 ? cudaErrorNotSupported : cudaSuccess;
    }();
    if (brings != cudaSuccess) return brings;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(gemm4_kernel<G, FW, PIECES>, kMaxSmemG, &allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)((a.m + p.rows - 1) / p.rows), (unsigned)p.ks);
    cfg.blockDim = dim3(kThreadsG, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.ks > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = (unsigned)p.ks;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, gemm4_kernel<G, FW, PIECES>, a, p, map);
}

// Four warps fold where that is the lesser part, the groups long beside the rows: 24 rows of 4096 x 9000 take 11.6 us with four
// and 12.9 with eight in groups of 128, 12.1 and 13.3 in groups of 64, 12.9 and 13.9 in groups of 32; 64 rows 12.7 and 13.7,
// 13.5 and 14.4, 15.3 and 15.1; 100 rows 14.3 and 15.1, 19.2 and 17.1, 29.4 and 25.4.
template <int G, int ROWS>
cudaError_t launch_rows(const W4Args &a, const Gemm4 &p, int tiles, int smem, const CUtensorMap &map, cudaStream_t stream) {
    constexpr int FW = ROWS <= G ? 1 : 2;
    return launch_kernel<G, FW, ROWS / 16 / FW>(a, p, tiles, smem, map, stream);
}

template <int G>
cudaError_t launch_group(const W4Args &a, const Gemm4 &p, int tiles, int smem, const CUtensorMap &map, cudaStream_t stream) {
    switch (p.rows) {
        case 32: return launch_rows<G, 32>(a, p, tiles, smem, map, stream);
        case 64: return launch_rows<G, 64>(a, p, tiles, smem, map, stream);
        case 96: return launch_rows<G, 96>(a, p, tiles, smem, map, stream);
        case 128: return launch_rows<G, 128>(a, p, tiles, smem, map, stream);
        case 160: return launch_rows<G, 160>(a, p, tiles, smem, map, stream);
        case 192: return launch_rows<G, 192>(a, p, tiles, smem, map, stream);
        default: return launch_rows<G, 256>(a, p, tiles, smem, map, stream);
    }
}

}  // namespace

cudaError_t read_w4_gemm_fault(unsigned *out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_w4_gemm_fault, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_w4_gemm_fault, &zero, sizeof(unsigned));
}

cudaError_t launch_w4_gemm(const W4Args &a, bool constant_weights, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count_of_device(&sms);
    if (e != cudaSuccess) return e;
    Gemm4 p = {};
    p.prefetch = constant_weights;
    const int row_tiles = (a.m + kMostRows - 1) / kMostRows;
    const int rows = (a.m + row_tiles - 1) / row_tiles;
    p.rows = rows <= 192 ? (rows + 31) / 32 * 32 : 256;
    int tiles = a.epi == kW4Glu ? (a.part[0].strip_end + 1) / 2 : 0;
    if (a.epi != kW4Glu)
        for (int i = 0; i < a.nparts; ++i) tiles += (a.part[i].strip_end - (i ? a.part[i - 1].strip_end : 0) + 3) / 4;
    const int chunks = (a.K + kChunkK - 1) / kChunkK;
    p.accs = 512 / (groups_at_once(a.group, p.rows) * p.rows);
    if (p.accs > kMaxAcc) p.accs = kMaxAcc;
    const int raw = 4 * (kChunkK / a.group) * a.unit, slot = kOperand + p.rows * 128, fixed = (int)sizeof(Control);
    p.slots = p.rows <= 64 ? 6 : 4;  // with three 64 rows of 4096 x 9000 took 13.6 us for 12.7, 512 of 4096 x 14336 51 for 49
    p.raws = (kMaxSmemG - fixed - p.slots * slot) / raw;
    if (p.raws > kMaxStages) p.raws = kMaxStages;
    const int smem = fixed + p.slots * slot + p.raws * raw;

    // K splits, in chunks of a CTA's time, which beside its own takes some eight for its beginning and end: of all tiles; or
    // the waves that are full unsplit and the tiles of the last one apart, split, in a launch of their own (512 rows of
    // 4096 x 14336, 224 tiles on 152 SMs, 62 -> 53 us).
    auto waves = [&](int t, int k) { return (double)(((long long)t * row_tiles * k + sms - 1) / sms); };
    auto cost = [&](int t, int k) { return waves(t, k) * (8.0 + (double)((chunks + k - 1) / k)); };
    auto best = [&](int t) {
        int ks = 1;
        for (int k = 2; k <= kMostSplit && k <= chunks; k *= 2)
            if (cost(t, k) < cost(t, ks)) ks = k;
        return ks;
    };
    int whole = (int)((long long)tiles * row_tiles / sms * sms / row_tiles);  // tiles of the full waves
    const int all = best(tiles), rest = whole < tiles ? best(tiles - whole) : 1;
    if (whole > 0 && whole < tiles && cost(whole, 1) + cost(tiles - whole, rest) < 0.95 * cost(tiles, all))
        p.ks = 1;
    else
        p.ks = all, whole = tiles;

    CUtensorMap map;
    if (!encode_bf16_rows(&map, a.x, a.m, a.K, kStepK, p.rows)) return cudaErrorNotSupported;
    for (int done = 0; done < tiles; done += whole, whole = tiles - done, p.ks = rest) {
        p.tile0 = done;
        switch (a.group) {
            case 32: e = launch_group<32>(a, p, whole, smem, map, stream); break;
            case 64: e = launch_group<64>(a, p, whole, smem, map, stream); break;
            default: e = launch_group<128>(a, p, whole, smem, map, stream); break;
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace q8
