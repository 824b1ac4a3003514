// Products of up to 16 rows over 4-bit weights: every warp streams its own run of units and contracts them on the tensor
// cores with exact bf16 operands.
//
// y[r, n] = sum_g s[g, n] * sum_{k in g} x[r, k] (c[k, n] - z[g, n]).  At 4.1 to 4.75 bits a weight the call is bound by the
// bytes of the weight; what has to keep up with them is the conversion (w4_pair: 9 instructions for 8 codes), which is why
// each code is converted once for all rows.
//
//   - A CTA's eight warps split K; the warps share nothing before the end.  A warp's work comes in stages of 128 rows of S
//     strips of 32 columns (of a strip one, two or four units, contiguous) and those rows' activations, bulk copies into
//     a ring of its own, one barrier a stage.
//   - The weights are the MMA's A operand (m16n8k16: 16 columns of W), the activations B (8 rows).  The order of the
//     reduction is free, so a lane's four k-pairs of two MMAs are the 8 rows of one stored word, and its activations 16
//     consecutive bytes.  With the activations as A half of every MMA would be empty rows for m <= 8.  Rows past m are
//     columns of B that nothing reads: they repeat the last row.
//   - A group's sums start from zero and are folded with its scales into an fp32 carry; (c - z) / 64 and x are exact in bf16.
//   - S strips share the activations' way from L2, which at m = 16 are as long as two strips' codes.
//   - Measured, groups of 128: one row of 4096 x 128256 53.5 us (5.1 TB/s of the 6.8 that a copy reaches; 70% of the issue
//     slots: conversion, MMAs, and the beginning and end of each of the 2004 CTAs), the gated pair of 4096 x 14336 14.6 us
//     (4.2 TB/s), 16 rows of 4096 x 6144 7.2 us; one row of 4096 x 4096 in groups of 32 4.8 us, nearly all of it latency.
//   - The warps' carries are added in shared memory in order, then, where the strips are too few for the SMs and K is split
//     over a cluster, those of its CTAs in rank order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "q8_attn.h"
#include "q8_launch.h"
#include "q8_w4_device.cuh"

namespace q8 {

__device__ unsigned int g_w4_fault = 0;

namespace {

constexpr int kWarps4 = 8;
constexpr int kThreads4 = 32 * kWarps4;
constexpr int kChunk = 128;              // rows of K in a stage
constexpr int kXPitch4 = 2 * kChunk + 64;  // bytes between activation rows in a stage: 64 past a multiple of 128, so that
                                         // the 16-byte loads of two rows and four lanes fall on all banks
// A stage: the activations, whose boxes start on the 512 bytes that their swizzle repeats over, then the strips' units.
__host__ __device__ constexpr int xbytes(int m, int xrows) { return xrows ? xrows * 2 * kChunk : m * kXPitch4; }
__host__ __device__ constexpr int stage_bytes(int units, int m, int xrows) {
    return (units + xbytes(m, xrows) + (xrows ? 511 : 15)) & (xrows ? ~511 : ~15);
}
struct Stream4 {
    int xrows;  // rows of a box of activations; 0: rows are copied one by one
    int depth;  // stages of a ring
    int ks;     // CTAs of a cluster splitting K
    int prefetch;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One 32-row block of a strip: word[j][h] of tile j, columns 16j + g and 16j + 8 + g; xb[nt] the lane's 8 activations.
template <int NT>
__device__ __forceinline__ void block32(float (&d)[2][NT][4], const uint32_t (&word)[2][2], const uint32_t (&zero)[2][2],
                                        const uint4 (&xb)[NT]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t lo[4] = {w4_pair<0>(word[j][0], zero[j][0]), w4_pair<0>(word[j][1], zero[j][1]),
                                w4_pair<1>(word[j][0], zero[j][0]), w4_pair<1>(word[j][1], zero[j][1])};
        const uint32_t hi[4] = {w4_pair<2>(word[j][0], zero[j][0]), w4_pair<2>(word[j][1], zero[j][1]),
                                w4_pair<3>(word[j][0], zero[j][0]), w4_pair<3>(word[j][1], zero[j][1])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(d[j][nt], lo, xb[nt].x, xb[nt].y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(d[j][nt], hi, xb[nt].z, xb[nt].w);
    }
}

// S strips a warp: of one part, or half of them of the gate and half of the up projection.
template <int G, int NT, int S>
__global__ void __launch_bounds__(kThreads4, NT * S == 1 ? 4 : NT * S == 2 ? 3 : 2)
    stream4_kernel(const __grid_constant__ W4Args a, const Stream4 p, const __grid_constant__ CUtensorMap xmap) {
    namespace cg = cooperative_groups;
    constexpr int CG = kChunk / G;  // groups of a chunk
    extern __shared__ __align__(1024) unsigned char smem4[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int depth = p.depth;
    const int chunk = CG * a.unit, stage = stage_bytes(S * chunk, a.m, p.xrows), wat = xbytes(a.m, p.xrows);
    unsigned char *ring = smem4 + warp * depth * stage;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem4 + kWarps4 * depth * stage) + warp * depth;

    // the CTA's tile: S strips of one part, or S / 2 of the gate and of the up projection
    const bool pair = a.epi == kW4Glu;
    const int width = pair ? S / 2 : S;  // strips of output
    int part = 0, tile = blockIdx.x;
    if (!pair)
        for (int first = 0, tiles;; ++part, tile -= tiles, first = a.part[part - 1].strip_end) {
            tiles = (a.part[part].strip_end - first + S - 1) / S;
            if (tile < tiles || part + 1 == a.nparts) break;
        }
    const W4Part &to = a.part[part];
    const int here = min(width, to.Np / kW4Strip - tile * width);  // strips that exist

    // the warp's run of chunks
    const int groups = a.K / G, chunks = (groups + CG - 1) / CG, runs = kWarps4 * p.ks;
    const int run = blockIdx.y * kWarps4 + warp;
    const int c0 = (int)((long long)chunks * run / runs);
    const int n = (int)((long long)chunks * (run + 1) / runs) - c0;
    const size_t strip_bytes = (size_t)groups * a.unit;
    const size_t src = (size_t)tile * width * strip_bytes + (size_t)c0 * chunk;
    auto groups_of = [&](int i) { return CG == 1 ? 1 : min(CG, groups - (c0 + i) * CG); };
    // strip s of a stage is strip s of the tile, or s / 2 of the gate (even s) and of the up projection (odd)
    auto ask_w = [&](int i, int slot) {  // lane 0: all bytes of the stage are announced, the weights' asked for
        const int gr = groups_of(i);
        const unsigned bytes = (unsigned)(gr * a.unit);
        uint64_t *bar = full + slot;
        w4_arrive_tx(bar, bytes * (pair ? 2 * here : here) + (unsigned)(gr * G * 2 * (p.xrows ? p.xrows : a.m)));
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int of = pair ? s >> 1 : s;
            if (of < here)
                w4_copy(ring + slot * stage + wat + s * chunk,
                        (pair && (s & 1) ? a.part[1].w : to.w) + src + of * strip_bytes + (size_t)i * chunk, bytes, bar);
        }
    };
    // The stage's activations: m rows (lanes 0 .. m - 1) 64 bytes past a multiple of 128 apart, or boxes of 32 values of all
    // rows in the 64-byte swizzle (lane 0).  Either way the 16-byte loads of two rows and four lanes fall on all banks.
    auto ask_x = [&](int i, int slot) {
        unsigned char *to = ring + slot * stage;
        const int k0 = (c0 + i) * kChunk, rows_k = groups_of(i) * G;
        if (p.xrows == 0) {
            if (lane < a.m)
                w4_copy(to + lane * kXPitch4, a.x + (size_t)lane * a.K + k0, (unsigned)(rows_k * 2), full + slot);
        } else if (lane == 0) {
            for (int b = 0; b < rows_k / 32; ++b)
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                        "r"(w4_smem(to + b * p.xrows * 64)),
                    "l"(&xmap), "r"(k0 + 32 * b), "r"(0), "r"(w4_smem(full + slot))
                    : "memory");
        }
    };

    if (lane == 0) {
        for (int s = 0; s < depth; ++s) w4_bar_init(full + s, 1);
        w4_bar_fence();
        if (p.prefetch)
            for (int i = 0; i < depth && i < n; ++i) ask_w(i, i);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (lane == 0 && !p.prefetch)
        for (int i = 0; i < depth && i < n; ++i) ask_w(i, i);
    __syncwarp();
    for (int i = 0; i < depth && i < n; ++i) ask_x(i, i);

    float acc[S][2][NT][4] = {};
    int xrow[NT];  // where the lane's activations of 32-row block 0 are in a stage; xblock to the next
    const int xblock = p.xrows ? p.xrows * 64 : 64;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + g;
        xrow[nt] = p.xrows ? r * 64 + ((t ^ (r >> 1 & 3)) << 4) : min(r, a.m - 1) * kXPitch4 + 16 * t;
    }
    int slot = 0, i = 0;
    unsigned phase = 0;
    for (; i < n; ++i) {
        if (!__all_sync(0xffffffffu, w4_wait(full + slot, phase))) break;
        const unsigned char *st = ring + slot * stage;
        const int have = groups_of(i);
#pragma unroll
        for (int q = 0; q < CG; ++q) {
            if (q >= have) break;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const unsigned char *u = st + wat + s * chunk + q * a.unit;
                uint32_t zero[2][2] = {{kW4Eight, kW4Eight}, {kW4Eight, kW4Eight}};
                if (a.zeros) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) zero[j][h] = w4_zero(u[16 * G + 64 + 16 * j + 8 * h + g]);
                }
                float d[2][NT][4] = {};
#pragma unroll
                for (int b = 0; b < G / 32; b += 2) {
                    uint32_t w0[2][2], w1[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (G == 32) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(u + 256 * j + 8 * lane);
                            w0[j][0] = v.x, w0[j][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4 *>(u + 512 * (b + j) + 16 * lane);
                            w0[j][0] = v.x, w0[j][1] = v.y, w1[j][0] = v.z, w1[j][1] = v.w;
                        }
                    }
                    uint4 x0[NT], x1[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const unsigned char *row = st + xrow[nt] + (q * (G / 32) + b) * xblock;
                        x0[nt] = *reinterpret_cast<const uint4 *>(row);
                        if (G > 32) x1[nt] = *reinterpret_cast<const uint4 *>(row + xblock);
                    }
                    block32<NT>(d, w0, zero, x0);
                    if (G > 32) block32<NT>(d, w1, zero, x1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f =
                            w4_scale(*reinterpret_cast<const uint16_t *>(u + 16 * G + 2 * (16 * j + 8 * h + g)), a.bf16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            acc[s][j][nt][2 * h] = fmaf(f, d[j][nt][2 * h], acc[s][j][nt][2 * h]);
                            acc[s][j][nt][2 * h + 1] = fmaf(f, d[j][nt][2 * h + 1], acc[s][j][nt][2 * h + 1]);
                        }
                    }
            }
        }
        __syncwarp();
        if (i + depth < n) {
            if (lane == 0) ask_w(i + depth, slot);
            __syncwarp();
            ask_x(i + depth, slot);
        }
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (i < n && lane == 0) {  // what was asked for lands (or two more seconds pass for each) before the memory is used again
        atomicOr(&g_w4_fault, kW4Fault);
        for (int j = i; j < n && j < i + depth; ++j) w4_wait(full + j % depth, (j / depth) & 1);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();

    // carries [8][m][pitch] (a pitch of 4 past a multiple of 32 spreads a fragment's rows over the banks), their sum
    constexpr int cols = 32 * S, pitch = cols + 4;
    const int rows = a.m;
    float *red = reinterpret_cast<float *>(smem4);
    float *sum = red + kWarps4 * rows * pitch;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 8 * nt + 2 * t + (e & 1);
                    if (r < rows) red[(warp * rows + r) * pitch + 32 * s + 16 * j + 8 * (e >> 1) + g] = acc[s][j][nt][e];
                }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (cols / 4); i += kThreads4) {
        const int r = i / (cols / 4), c = 4 * (i - r * (cols / 4));
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kWarps4; ++k) {
            const float4 o = *reinterpret_cast<const float4 *>(red + (k * rows + r) * pitch + c);
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        *reinterpret_cast<float4 *>(sum + r * cols + c) = v;
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (p.ks > 1)
        cluster.sync();
    else
        __syncthreads();

    // a rank's share of the output's columns, four a thread
    const int share = 8 * width, k0 = share * (int)blockIdx.y / p.ks, k1 = share * ((int)blockIdx.y + 1) / p.ks;
    for (int i = threadIdx.x; i < rows * (k1 - k0); i += kThreads4) {
        const int r = i / (k1 - k0), c = 4 * (k0 + i - r * (k1 - k0));
        const int out = tile * width * kW4Strip + c;
        if (out >= to.Np) continue;
        auto total = [&](int at, float (&v)[4]) {
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
            for (int k = 0; k < p.ks; ++k) {
                const float4 o = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(sum, k) + at);
                f.x += o.x, f.y += o.y, f.z += o.z, f.w += o.w;
            }
            v[0] = kW4Unit * f.x, v[1] = kW4Unit * f.y, v[2] = kW4Unit * f.z, v[3] = kW4Unit * f.w;
        };
        float v[4];
        total(r * cols + (pair ? (c >> 5) * 64 + (c & 31) : c), v);
        const size_t at = (size_t)r * to.Np + out;
        if (pair) {
            float u[4];
            total(r * cols + (c >> 5) * 64 + 32 + (c & 31), u);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = v[e] / (1.0f + expf(-v[e])) * u[e];
        }
        if (a.epi == kW4Residual) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (out + e < to.N) v[e] += a.res[at + e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (out + e >= to.N) v[e] = 0.0f;
        if (to.y) *reinterpret_cast<float4 *>(to.y + at) = make_float4(v[0], v[1], v[2], v[3]);
        if (a.ybf) {
            __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2 *>(a.ybf + at) =
                make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
        }
    }
    if (p.ks > 1) cluster_sync_after_reads();
}

constexpr int kMaxSmem4 = 227 * 1024;

int smem_bytes(const W4Args &a, const Stream4 &p, int S) {
    const int ring = kWarps4 * p.depth * (stage_bytes(S * (kChunk / a.group) * a.unit, a.m, p.xrows) + 8);
    const int ends = a.m * (kWarps4 * (32 * S + 4) + 32 * S) * 4;
    return ring > ends ? ring : ends;
}

int tiles_of(const W4Args &a, int S) {
    if (a.epi == kW4Glu) return (a.part[0].strip_end + S / 2 - 1) / (S / 2);
    int tiles = 0;
    for (int i = 0; i < a.nparts; ++i) tiles += (a.part[i].strip_end - (i ? a.part[i - 1].strip_end : 0) + S - 1) / S;
    return tiles;
}

template <int G, int NT, int S>
cudaError_t launch_kernel(const W4Args &a, const Stream4 &p, const CUtensorMap &map, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(stream4_kernel<G, NT, S>, kMaxSmem4, &allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles_of(a, S), (unsigned)p.ks, 1);
    cfg.blockDim = dim3(kThreads4, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem_bytes(a, p, S);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.ks > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = (unsigned)p.ks;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, stream4_kernel<G, NT, S>, a, p, map);
}

template <int G>
cudaError_t launch_group(const W4Args &a, const Stream4 &p, int S, const CUtensorMap &map, cudaStream_t stream) {
    if (a.m > 8) return launch_kernel<G, 2, 2>(a, p, map, stream);
    return S == 1 ? launch_kernel<G, 1, 1>(a, p, map, stream) : launch_kernel<G, 1, 2>(a, p, map, stream);
}

}  // namespace

cudaError_t read_w4_fault(unsigned *out, bool clear) {
    unsigned gemm = 0;
    cudaError_t e = read_w4_gemm_fault(&gemm, clear);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(out, g_w4_fault, sizeof(unsigned));
    *out |= gemm;
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_w4_fault, &zero, sizeof(unsigned));
}

cudaError_t launch_w4_stream(const W4Args &a, bool constant_weights, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count_of_device(&sms);
    if (e != cudaSuccess) return e;
    // Strips a warp: two share the activations' way from L2 from five rows on, where there are enough strips for a wave of
    // such CTAs (4096 x 128256 at one row 56.8 -> 53.5 us), and where the weight is large (14336 x 4096 in groups of 64, four
    // rows 13.3 -> 10.5 us, two 11.6 -> 10.1; 4096 x 4096 in groups of 32, four rows 6.3 -> 5.8, but two 5.1 -> 6.0; one row of
    // 4096 x 14336 8.5 -> 9.5); one otherwise, so that more warps share the weight (5120 x 1500, four rows 4.1 us, with two
    // strips 4.9).
    Stream4 p = {a.m > 8 ? 16 : 0, 1, 1, constant_weights};
    const bool pair = a.epi == kW4Glu;
    const int strips = pair ? 2 * a.part[0].strip_end : a.part[a.nparts - 1].strip_end;
    const int chunks = (a.K + kChunk - 1) / kChunk;
    const long long units = (long long)strips * chunks;
    const bool large = a.m > 2 ? units >= 26ll * sms : units >= 54ll * sms && strips <= sms;
    const int S = pair || a.m > 4 || strips >= 6 * sms || large ? 2 : 1;
    const int fit = a.m > 8 ? 2 : S == 2 ? 3 : 4;  // CTAs an SM by their registers
    // K is split while the CTAs fill no more than three quarters of what fits at once (512 CTAs where 608 fit were no faster
    // than 256, and a second wave costs a whole one), and while each warp has a chunk.
    const int tiles = tiles_of(a, S);
    while (p.ks < 8 && 2ll * p.ks * tiles * 4 <= 3ll * fit * sms && 2 * p.ks * kWarps4 <= chunks) p.ks *= 2;
    // As many stages as leave room for the CTAs that an SM gets.
    const long long ctas = (long long)tiles * p.ks;
    const int each = (int)(ctas >= (long long)fit * sms ? fit : (ctas + sms - 1) / sms);
    while (p.depth < 4 && p.depth * kWarps4 * p.ks < chunks) {
        ++p.depth;
        if (each * (smem_bytes(a, p, S) + 1024) > 228 * 1024) {
            --p.depth;
            break;
        }
    }
    CUtensorMap map = {};
    if (p.xrows && !encode_bf16_rows(&map, a.x, a.m, a.K, 32, p.xrows)) return cudaErrorNotSupported;
    switch (a.group) {
        case 32: return launch_group<32>(a, p, S, map, stream);
        case 64: return launch_group<64>(a, p, S, map, stream);
        default: return launch_group<128>(a, p, S, map, stream);
    }
}

}  // namespace q8
