// The paged key-value cache's bookkeeping and its append: q8_kv_slots and q8_rope_append (formulas in q8_gemv.h).
#include <cuda_bf16.h>
#include <math.h>

#include "q8_device.cuh"
#include "q8_kv.h"

namespace q8 {
namespace {

// ---- slots ----------------------------------------------------------------------------------------------------------
//
// The work is two prefix sums over R requests (new rows, new pages) and one lookup for each row and each new page: a
// few hundred KB at the most, so latency bounds it.  One launch, no CTA waits for another: every CTA takes both prefix
// sums over all R requests for itself (R lengths from L2, the sums in shared memory), then its share of the rows and
// of the new pages, each found by a binary search in the sums.
struct SlotArgs {
    const int *cached, *fresh, *free_pages, *head;
    int *table, *lens, *row_start, *positions, *next_head;
    long long *slots;
    int R, page, n_free, width, pitch, rows;
};

constexpr int kSlotThreads = 512;

__device__ __forceinline__ int ceil_div_dev(int a, int b) { return a / b + (a % b != 0); }

// The largest r in [0, n) with sum[r] <= i (sum ascending, sum[0] = 0): the request that item i belongs to, empty
// requests skipped.
__device__ __forceinline__ int owner(const int *sum, int n, int i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sum[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kSlotThreads) slots_kernel(SlotArgs a) {
    extern __shared__ int sums[];
    int *row0 = sums, *page0 = sums + a.R + 1;  // [R + 1] each: exclusive sums of the new rows and the new pages
    __shared__ int wrow[kSlotThreads / 32], wpage[kSlotThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (a.R + kSlotThreads - 1) / kSlotThreads;
    const int r0 = min(a.R, tid * each), r1 = min(a.R, r0 + each);
    int nrow = 0, npage = 0;
    for (int r = r0; r < r1; ++r) {
        const int c = max(a.cached[r], 0), f = max(a.fresh[r], 0);
        const int have = ceil_div_dev(c, a.page), want = min(a.width, ceil_div_dev(c + f, a.page));
        row0[r] = f;
        page0[r] = max(0, want - have);
        nrow += f;
        npage += max(0, want - have);
    }
    int srow = nrow, spage = npage;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, srow, o), y = __shfl_up_sync(0xffffffffu, spage, o);
        if (lane >= o) { srow += x; spage += y; }
    }
    if (lane == 31) { wrow[warp] = srow; wpage[warp] = spage; }
    __syncthreads();
    int brow = srow - nrow, bpage = spage - npage;
    for (int w = 0; w < warp; ++w) { brow += wrow[w]; bpage += wpage[w]; }
    for (int r = r0; r < r1; ++r) {
        const int f = row0[r], p = page0[r];
        row0[r] = brow;
        page0[r] = bpage;
        brow += f;
        bpage += p;
    }
    if (tid == kSlotThreads - 1) { row0[a.R] = brow; page0[a.R] = bpage; }
    __syncthreads();
    const int total_rows = row0[a.R], total_pages = page0[a.R];
    const int head = a.head ? *a.head : 0;
    const int step = gridDim.x * kSlotThreads, me = blockIdx.x * kSlotThreads + tid;
    auto free_page = [&](int i) {
        const long long at = (long long)head + i;
        return at >= 0 && at < a.n_free ? a.free_pages[at] : -1;
    };
    for (int t = me; t < a.rows; t += step) {
        int pos = -1;
        long long slot = -1;
        if (t < total_rows) {
            const int r = owner(row0, a.R, t);
            const int c = max(a.cached[r], 0);
            pos = c + (t - row0[r]);
            const int idx = pos / a.page, have = ceil_div_dev(c, a.page);
            int entry = -1;
            if (idx < a.width)
                entry = idx < have ? a.table[(size_t)r * a.pitch + idx] : free_page(page0[r] + idx - have);
            if (entry >= 0) slot = (long long)entry * a.page + pos % a.page;
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    for (int i = me; i < total_pages; i += step) {
        const int r = owner(page0, a.R, i);
        const int have = ceil_div_dev(max(a.cached[r], 0), a.page);
        a.table[(size_t)r * a.pitch + have + (i - page0[r])] = free_page(i);
    }
    for (int r = me; r <= a.R; r += step) {
        a.row_start[r] = row0[r];
        if (r < a.R) a.lens[r] = max(a.cached[r], 0) + max(a.fresh[r], 0);
    }
    if (me == 0) *a.next_head = head + total_pages;
}

// ---- append ---------------------------------------------------------------------------------------------------------
//
// One pass over the fp32 outputs of the q/k/v products: 4 bytes read and 2 (bf16) or 1.125 (Q8_0) written a value, a
// handful of operations each, so memory bounds it once there are enough rows, and latency before that.  A head's dim
// values sit on dim / 4 lanes, four a lane, so the norm's sum and the amax of 32 values are shuffles and the partner
// of a half-layout pair is rotary_dim / 8 lanes away.
struct AppendArgs {
    const float *q, *k, *v, *qg, *kg, *table;
    const int *positions;
    const long long *slots;
    uint16_t *qo;
    void *kc, *vc;
    float *ks, *vs;
    long long page_stride, n_slots;
    float eps;
    int ldq, ldk, ldv, ldo, max_pos, rot, rows, q_heads, kv_heads, page;
};

constexpr int kAppendWarps = 8;

__device__ __forceinline__ uint2 pack_bf16x4(float4 v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t *>(&lo);
    o.y = *reinterpret_cast<const uint32_t *>(&hi);
    return o;
}

// D: the head's dim; HALF / pairs; Q8: the cache's type.  A group of D / 4 lanes takes one head of one row.
template <int D, bool INTERLEAVED, bool Q8>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(AppendArgs a) {
    constexpr int L = D / 4;        // lanes a head
    constexpr int G = 32 / L;       // heads a warp takes at once
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, sub = lane % L, warp = threadIdx.x >> 5;
    const int t = blockIdx.y;
    const int total = a.q_heads + 2 * a.kv_heads;
    const int head = (blockIdx.x * kAppendWarps + warp) * G + lane / L;
    const bool live = head < total;
    const int pos = a.positions[t];
    const long long slot = a.slots[t];
    const bool is_q = head < a.q_heads, is_k = !is_q && head < a.q_heads + a.kv_heads;
    const int h = is_q ? head : (is_k ? head - a.q_heads : head - a.q_heads - a.kv_heads);
    const int d0 = 4 * sub;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live && pos >= 0) {
        const float *src = is_q ? a.q + (size_t)t * a.ldq : (is_k ? a.k + (size_t)t * a.ldk : a.v + (size_t)t * a.ldv);
        x = *reinterpret_cast<const float4 *>(src + (size_t)h * D + d0);
    }
    float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int half = a.rot / 2;
    const bool turned = live && pos >= 0 && d0 < a.rot && (is_q || is_k);
    if (turned) {
        if (pos < a.max_pos) {
            const float *row = a.table + (size_t)pos * a.rot;
            if (INTERLEAVED) {
                const float2 c = *reinterpret_cast<const float2 *>(row + 2 * sub);
                const float2 s = *reinterpret_cast<const float2 *>(row + half + 2 * sub);
                cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y;
                sn[0] = sn[1] = s.x; sn[2] = sn[3] = s.y;
            } else {
                const int i = d0 < half ? d0 : d0 - half;
                const float4 c = *reinterpret_cast<const float4 *>(row + i);
                const float4 s = *reinterpret_cast<const float4 *>(row + half + i);
                cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
                sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] = sn[e] = __uint_as_float(0x7FC00000u);
        }
    }
    const float *gamma = is_q ? a.qg : a.kg;
    if (a.qg || a.kg) {  // uniform across the launch: every lane takes the shuffles
        float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (live && (is_q || is_k) && gamma) {
            const float rs = 1.0f / sqrtf(ss / (float)D + a.eps);
            const float4 g = *reinterpret_cast<const float4 *>(gamma + d0);
            x.x = x.x * rs * g.x; x.y = x.y * rs * g.y; x.z = x.z * rs * g.z; x.w = x.w * rs * g.w;
        }
    }
    if (INTERLEAVED) {
        if (turned) {
            const float4 y = x;
            x.x = y.x * cs[0] - y.y * sn[0]; x.y = y.x * sn[1] + y.y * cs[1];
            x.z = y.z * cs[2] - y.w * sn[2]; x.w = y.z * sn[3] + y.w * cs[3];
        }
    } else {
        const bool first = d0 < half;
        const int far = first ? sub + half / 4 : sub - half / 4;
        const int from = (lane - sub) + (d0 < a.rot ? far : sub);
        float4 y;
        y.x = __shfl_sync(0xffffffffu, x.x, from); y.y = __shfl_sync(0xffffffffu, x.y, from);
        y.z = __shfl_sync(0xffffffffu, x.z, from); y.w = __shfl_sync(0xffffffffu, x.w, from);
        if (turned) {
            const float sg = first ? -1.0f : 1.0f;
            x.x = x.x * cs[0] + sg * (y.x * sn[0]); x.y = x.y * cs[1] + sg * (y.y * sn[1]);
            x.z = x.z * cs[2] + sg * (y.z * sn[2]); x.w = x.w * cs[3] + sg * (y.w * sn[3]);
        }
    }
    if (is_q) {
        if (live) *reinterpret_cast<uint2 *>(a.qo + (size_t)t * a.ldo + (size_t)h * D + d0) = pack_bf16x4(x);
    }
    const bool write = live && !is_q && pos >= 0 && slot >= 0 && slot < a.n_slots;
    const long long page = write ? slot / a.page : 0, off = write ? slot - page * a.page : 0;
    const long long base = page * a.page_stride + ((long long)h * a.page + off) * D;
    if (Q8) {
        uint32_t mx = max(max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu),
                          max(__float_as_uint(x.z) & 0x7FFFFFFFu, __float_as_uint(x.w) & 0x7FFFFFFFu));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (write) {
            const float d = act_scale(mx), inv = act_inv(d);
            const uint32_t codes = act_code(x.x, d, inv, mx) | (act_code(x.y, d, inv, mx) << 8) |
                                   (act_code(x.z, d, inv, mx) << 16) | (act_code(x.w, d, inv, mx) << 24);
            *reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(is_k ? a.kc : a.vc) + base + d0) = codes;
            if ((sub & 7) == 0) (is_k ? a.ks : a.vs)[(base + d0) / kBlock] = d;
        }
    } else if (write) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(is_k ? a.kc : a.vc) + base + d0) = pack_bf16x4(x);
    }
}

template <int D> cudaError_t launch_append(const AppendArgs &a, bool interleaved, bool q8, cudaStream_t stream) {
    const int total = a.q_heads + 2 * a.kv_heads, per = kAppendWarps * (128 / D);
    const dim3 grid((unsigned)((total + per - 1) / per), (unsigned)a.rows, 1);
    if (interleaved)
        return q8 ? kv_launch(append_kernel<D, true, true>, grid, 32 * kAppendWarps, 0, stream, a)
                  : kv_launch(append_kernel<D, true, false>, grid, 32 * kAppendWarps, 0, stream, a);
    return q8 ? kv_launch(append_kernel<D, false, true>, grid, 32 * kAppendWarps, 0, stream, a)
              : kv_launch(append_kernel<D, false, false>, grid, 32 * kAppendWarps, 0, stream, a);
}

}  // namespace

q8_status kv_check_cache(const q8_kv_cache *c) {
    if (!c || !c->k || !c->v || (c->k_scale == nullptr) != (c->v_scale == nullptr)) return Q8_ERR_ARG;
    if (c->pages < 1 || c->heads < 1 || c->page_size < 16 || c->page_size % 16 != 0 || (c->dim != 64 && c->dim != 128))
        return Q8_ERR_SHAPE;
    if ((int64_t)c->heads * c->page_size > 0x7FFFFFFFll / c->dim) return Q8_ERR_SHAPE;
    const int64_t dense = (int64_t)c->heads * c->page_size * c->dim;
    if (c->page_stride < dense || c->page_stride % 128 != 0 || c->page_stride > (1ll << 38) / c->pages)
        return Q8_ERR_SHAPE;
    if (!kv_aligned(c->k, 16) || !kv_aligned(c->v, 16) || !kv_aligned(c->k_scale, 16) || !kv_aligned(c->v_scale, 16))
        return Q8_ERR_ALIGN;
    return Q8_OK;
}

bool kv_overlaps_cache(const q8_kv_cache *c, const void *p, int64_t bytes) {
    const int64_t n = kv_span(c), vb = n * (kv_is_q8(c) ? 1 : 2), sb = n / Q8_BLOCK * 4;
    return kv_overlap(p, bytes, c->k, vb) || kv_overlap(p, bytes, c->v, vb) || kv_overlap(p, bytes, c->k_scale, sb) ||
           kv_overlap(p, bytes, c->v_scale, sb);
}

}  // namespace q8

extern "C" q8_status q8_kv_slots(const int *cached, const int *fresh, int R, int page_size, const int *free_pages,
                                 int n_free, const int *head, int *table, int table_width, int table_pitch, int rows,
                                 int *lens, int *row_start, int *positions, int64_t *slots, int *next_head,
                                 q8_stream_t stream) {
    using namespace q8;
    if (!cached || !fresh || !table || !lens || !row_start || !next_head || (n_free > 0 && !free_pages) ||
        (rows > 0 && (!positions || !slots)))
        return Q8_ERR_ARG;
    if (R < 1 || R > Q8_MAX_REQUESTS || page_size < 16 || page_size % 16 != 0 || n_free < 0 || table_width < 1 ||
        table_pitch < table_width || rows < 0)
        return Q8_ERR_SHAPE;
    const void *four[9] = {cached, fresh, free_pages, head, table, lens, row_start, positions, next_head};
    for (const void *p : four)
        if (!kv_aligned(p, 4)) return Q8_ERR_ALIGN;
    if (!kv_aligned(slots, 8)) return Q8_ERR_ALIGN;
    const void *ins[4] = {cached, fresh, free_pages, head};
    const int64_t inb[4] = {4ll * R, 4ll * R, 4ll * n_free, 4};
    const void *outs[6] = {table, lens, row_start, rows ? positions : nullptr, rows ? slots : nullptr, next_head};
    const int64_t outb[6] = {4 * ((int64_t)(R - 1) * table_pitch + table_width), 4ll * R, 4ll * (R + 1), 4ll * rows,
                             8ll * rows, 4};
    for (int o = 0; o < 6; ++o) {
        for (int i = 0; i < 4; ++i)
            if (kv_overlap(outs[o], outb[o], ins[i], inb[i])) return Q8_ERR_ARG;
        for (int p = 0; p < o; ++p)
            if (kv_overlap(outs[o], outb[o], outs[p], outb[p])) return Q8_ERR_ARG;
    }
    const SlotArgs a = {cached, fresh, free_pages, head, table, lens, row_start, positions, next_head,
                        reinterpret_cast<long long *>(slots), R, page_size, n_free, table_width, table_pitch, rows};
    const size_t smem = (size_t)(R + 1) * 8;
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024)
        e = cudaFuncSetAttribute(slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return kv_cuda_fail(e);
    const int most = rows > R + 1 ? rows : R + 1;
    int ctas = (most + kSlotThreads - 1) / kSlotThreads;
    if (ctas > 128) ctas = 128;
    e = kv_launch(slots_kernel, dim3((unsigned)ctas, 1, 1), kSlotThreads, smem, (cudaStream_t)stream, a);
    return e == cudaSuccess ? Q8_OK : kv_cuda_fail(e);
}

extern "C" q8_status q8_rope_append(const float *q, int ldq, const float *k, int ldk, const float *v, int ldv,
                                    const float *q_gamma, const float *k_gamma, float eps, const float *table,
                                    int max_positions, int rotary_dim, const int *positions, const int64_t *slots,
                                    void *q_out, int ldo, const q8_kv_cache *cache, int rows, int q_heads,
                                    unsigned int flags, q8_stream_t stream) {
    using namespace q8;
    if (!q || !k || !v || !positions || !slots || !q_out || !cache || (rotary_dim > 0 && !table)) return Q8_ERR_ARG;
    if (flags & ~Q8_ROPE_INTERLEAVED) return Q8_ERR_ARG;
    if (!(eps >= 0.0f) || !(eps < INFINITY)) return Q8_ERR_ARG;
    q8_status st = kv_check_cache(cache);
    if (st != Q8_OK) return st;
    const int dim = cache->dim;
    if (rows < 1 || rows > 65535 || q_heads < 1 || q_heads > 0x7FFFFFFF / dim || rotary_dim < 0 || rotary_dim > dim ||
        rotary_dim % 8 != 0 || (rotary_dim > 0 && max_positions < 1) || ldq < q_heads * dim || ldo < q_heads * dim ||
        ldk < cache->heads * dim || ldv < cache->heads * dim)
        return Q8_ERR_SHAPE;
    if (ldq % 4 || ldk % 4 || ldv % 4 || ldo % 8) return Q8_ERR_ALIGN;
    const void *p16[7] = {q, k, v, q_gamma, k_gamma, table, q_out};
    for (const void *p : p16)
        if (!kv_aligned(p, 16)) return Q8_ERR_ALIGN;
    if (!kv_aligned(positions, 4) || !kv_aligned(slots, 8)) return Q8_ERR_ALIGN;
    const int64_t ob = 2 * ((int64_t)(rows - 1) * ldo + q_heads * dim);
    const void *ins[8] = {q, k, v, q_gamma, k_gamma, rotary_dim ? table : nullptr, positions, slots};
    const int64_t kvn = (int64_t)cache->heads * dim;
    const int64_t inb[8] = {4 * ((int64_t)(rows - 1) * ldq + q_heads * dim), 4 * ((int64_t)(rows - 1) * ldk + kvn),
                            4 * ((int64_t)(rows - 1) * ldv + kvn), 4ll * dim, 4ll * dim,
                            4ll * max_positions * rotary_dim, 4ll * rows, 8ll * rows};
    for (int i = 0; i < 8; ++i)
        if (kv_overlap(q_out, ob, ins[i], inb[i]) || (ins[i] && kv_overlaps_cache(cache, ins[i], inb[i])))
            return Q8_ERR_ARG;
    if (kv_overlaps_cache(cache, q_out, ob)) return Q8_ERR_ARG;
    const AppendArgs a = {q, k, v, q_gamma, k_gamma, table, positions, reinterpret_cast<const long long *>(slots),
                          static_cast<uint16_t *>(q_out), cache->k, cache->v, cache->k_scale, cache->v_scale,
                          cache->page_stride, (long long)cache->pages * cache->page_size, eps, ldq, ldk, ldv, ldo,
                          max_positions, rotary_dim, rows, q_heads, cache->heads, cache->page_size};
    const bool inter = (flags & Q8_ROPE_INTERLEAVED) != 0, q8c = kv_is_q8(cache);
    const cudaError_t e = dim == 128 ? launch_append<128>(a, inter, q8c, (cudaStream_t)stream)
                                     : launch_append<64>(a, inter, q8c, (cudaStream_t)stream);
    return e == cudaSuccess ? Q8_OK : kv_cuda_fail(e);
}
