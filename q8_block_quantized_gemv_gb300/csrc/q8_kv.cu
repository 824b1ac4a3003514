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
// of the new pages, each found by a binary search in the sums.  (16 requests 3.5 us; 1,500 requests with 30,011 rows 4.7 us.)
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
// One pass over the fp32 outputs of the q/k/v products: 4 bytes read and 2 (bf16) or 1.125 (Q8_0) written a value, so
// memory bounds it once there are enough rows, and latency before that -- if a value costs few enough instructions.
// A lane holds eight values of a head, as two chunks of four: with the half layout a chunk and its partner rotary_dim
// / 2 on, so that the rotation needs no other lane; otherwise two neighbours.  (Four values a lane and shuffles for the
// partners took twice the instructions: 82 us for 8191 rows of 32 + 2 x 8 heads, 55 us now, 5.5 TB/s, with 55% of the
// issue slots taken; 16 rows of 32 + 2 x 32 heads take 1.9 us.)
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

constexpr int kAppendWarps = 4;
constexpr long long kAppendWide = 3ll << 19;  // values (launch_append_type)

__device__ __forceinline__ uint2 pack_bf16x4(float4 v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t *>(&lo);
    o.y = *reinterpret_cast<const uint32_t *>(&hi);
    return o;
}

// D: the head's dim; PAIRS: neighbours (2i, 2i + 1) turn, not halves; Q8: the cache's type; N: heads of its row a group
// of D / 8 lanes takes, all requested before the first is used.
template <int D, bool PAIRS, bool Q8, int N>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(AppendArgs a) {
    constexpr int L = D / 8;   // lanes a head
    constexpr int G = 32 / L;  // heads a warp takes at once
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, sub = lane % L, warp = threadIdx.x >> 5;
    const int total = a.q_heads + 2 * a.kv_heads;
    const unsigned per_row = (unsigned)(total + G * N - 1) / (G * N);  // warps a row
    const unsigned id = blockIdx.x * kAppendWarps + warp;
    const int t = (int)(id / per_row);
    if (t >= a.rows) return;
    const int head0 = (int)(id - t * per_row) * (G * N) + lane / L;  // then every G-th
    const int pos = a.positions[t];
    const long long slot = a.slots[t];
    // this lane's two chunks of four values: c, a pair's first, turns with d, its second
    const int p8 = a.rot / 8;  // chunk pairs that turn (halves)
    const int c = PAIRS ? 2 * sub : (sub < p8 ? sub : 2 * sub), d = PAIRS ? c + 1 : (sub < p8 ? sub + p8 : c + 1);
    float4 in[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int head = head0 + n * G;
        in[n][0] = in[n][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (head < total && pos >= 0) {
            const float *src = head < a.q_heads ? a.q + (size_t)t * a.ldq + head * D
                               : head < a.q_heads + a.kv_heads
                                   ? a.k + (size_t)t * a.ldk + (head - a.q_heads) * D
                                   : a.v + (size_t)t * a.ldv + (head - a.q_heads - a.kv_heads) * D;
            in[n][0] = __ldcs(reinterpret_cast<const float4 *>(src) + c);
            in[n][1] = __ldcs(reinterpret_cast<const float4 *>(src) + d);
        }
    }
    // cos and sin: of the chunk's four pairs (halves), or of each chunk's two (pairs: in x, y of cs[0] and cs[1])
    float4 cs[2], sn[2];
    cs[0] = cs[1] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    sn[0] = sn[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (pos >= 0 && (PAIRS ? 4 * c < a.rot : sub < p8)) {
        const float *row = a.table + (size_t)pos * a.rot;
        const float nan = __uint_as_float(0x7FC00000u);
        if (pos >= a.max_pos) {
            cs[0] = cs[1] = sn[0] = sn[1] = make_float4(nan, nan, nan, nan);
        } else if (PAIRS) {  // rotary_dim is a multiple of 8: both chunks turn or neither
            const float4 cv = *reinterpret_cast<const float4 *>(row + 2 * c);
            const float4 sv = *reinterpret_cast<const float4 *>(row + a.rot / 2 + 2 * c);
            cs[0] = make_float4(cv.x, cv.y, 0.0f, 0.0f);
            cs[1] = make_float4(cv.z, cv.w, 0.0f, 0.0f);
            sn[0] = make_float4(sv.x, sv.y, 0.0f, 0.0f);
            sn[1] = make_float4(sv.z, sv.w, 0.0f, 0.0f);
        } else {
            cs[0] = *reinterpret_cast<const float4 *>(row + 4 * c);
            sn[0] = *reinterpret_cast<const float4 *>(row + a.rot / 2 + 4 * c);
        }
    }
    const bool turns = PAIRS ? 4 * c < a.rot : sub < p8;
    const bool placed = pos >= 0 && slot >= 0 && slot < a.n_slots;
    const long long page = placed ? slot / a.page : 0;
    const long long place = placed ? page * a.page_stride + (slot - page * a.page) * D : 0;  // of head 0
    const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    const bool norms = a.qg || a.kg;
    float4 gq[2] = {one, one}, gk[2] = {one, one};
    if (a.qg) {
        gq[0] = reinterpret_cast<const float4 *>(a.qg)[c];
        gq[1] = reinterpret_cast<const float4 *>(a.qg)[d];
    }
    if (a.kg) {
        gk[0] = reinterpret_cast<const float4 *>(a.kg)[c];
        gk[1] = reinterpret_cast<const float4 *>(a.kg)[d];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int head = head0 + n * G;
        const bool live = head < total;
        const bool is_q = head < a.q_heads, is_k = !is_q && head < a.q_heads + a.kv_heads;
        const int h = is_q ? head : (is_k ? head - a.q_heads : head - a.q_heads - a.kv_heads);
        float4 x = in[n][0], y = in[n][1];
        if (norms) {  // uniform across the launch: every lane takes the shuffles
            float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w))) +
                       fmaf(y.x, y.x, fmaf(y.y, y.y, fmaf(y.z, y.z, y.w * y.w)));
#pragma unroll
            for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (pos >= 0 && ((is_q && a.qg) || (is_k && a.kg))) {  // padding stays 0 whatever eps and gamma are
                const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
                const float4 g0 = is_q ? gq[0] : gk[0], g1 = is_q ? gq[1] : gk[1];
                x.x *= rs * g0.x; x.y *= rs * g0.y; x.z *= rs * g0.z; x.w *= rs * g0.w;
                y.x *= rs * g1.x; y.y *= rs * g1.y; y.z *= rs * g1.z; y.w *= rs * g1.w;
            }
        }
        if (turns && (is_q || is_k)) {
            const float4 u = x, v = y;
            if (PAIRS) {
                x.x = u.x * cs[0].x - u.y * sn[0].x; x.y = u.x * sn[0].x + u.y * cs[0].x;
                x.z = u.z * cs[0].y - u.w * sn[0].y; x.w = u.z * sn[0].y + u.w * cs[0].y;
                y.x = v.x * cs[1].x - v.y * sn[1].x; y.y = v.x * sn[1].x + v.y * cs[1].x;
                y.z = v.z * cs[1].y - v.w * sn[1].y; y.w = v.z * sn[1].y + v.w * cs[1].y;
            } else {
                x.x = u.x * cs[0].x - v.x * sn[0].x; y.x = u.x * sn[0].x + v.x * cs[0].x;
                x.y = u.y * cs[0].y - v.y * sn[0].y; y.y = u.y * sn[0].y + v.y * cs[0].y;
                x.z = u.z * cs[0].z - v.z * sn[0].z; y.z = u.z * sn[0].z + v.z * cs[0].z;
                x.w = u.w * cs[0].w - v.w * sn[0].w; y.w = u.w * sn[0].w + v.w * cs[0].w;
            }
        }
        if (is_q) {
            uint2 *to = reinterpret_cast<uint2 *>(a.qo + (size_t)t * a.ldo + h * D);
            if (PAIRS) {
                const uint2 lo = pack_bf16x4(x), hi = pack_bf16x4(y);
                *reinterpret_cast<uint4 *>(to + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                to[c] = pack_bf16x4(x);
                to[d] = pack_bf16x4(y);
            }
        }
        const bool write = live && !is_q && placed;
        const long long base = place + (long long)h * a.page * D;
        if (Q8) {
            const auto most = [](float4 v) {
                return max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                           max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
            };
            uint32_t m0 = most(x), m1 = most(y);  // of the chunks, then of their blocks of eight chunks
            if (PAIRS) {
                m0 = max(m0, m1);
                m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
                m0 = m1 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
            } else if (a.rot % 64 == 0 && a.rot == D) {  // eight lanes' chunks are a block, first and second alike
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                    m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                }
            } else {  // gather the eight chunks of each block from the lanes that hold them
                uint32_t b0 = 0u, b1 = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int k = ((w ? d : c) & ~7) + e;  // chunk; its lane, and whether it is the second there
                        const int from = k < p8 ? k : (k < 2 * p8 ? k - p8 : k >> 1);
                        const bool second = k < 2 * p8 ? k >= p8 : (k & 1) != 0;
                        const uint32_t f = __shfl_sync(0xffffffffu, m0, lane - sub + from);
                        const uint32_t g = __shfl_sync(0xffffffffu, m1, lane - sub + from);
                        (w ? b1 : b0) = max(w ? b1 : b0, second ? g : f);
                    }
                }
                m0 = b0;
                m1 = b1;
            }
            if (write) {
                unsigned char *codes = static_cast<unsigned char *>(is_k ? a.kc : a.vc) + base;
                float *scales = (is_k ? a.ks : a.vs) + base / kBlock;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const float4 v = w ? y : x;
                    const uint32_t m = w ? m1 : m0;
                    const int k = w ? d : c;
                    const float s = act_scale(m), inv = act_inv(s);
                    *reinterpret_cast<uint32_t *>(codes + 4 * k) =
                        act_code(v.x, s, inv, m) | (act_code(v.y, s, inv, m) << 8) | (act_code(v.z, s, inv, m) << 16) |
                        (act_code(v.w, s, inv, m) << 24);
                    if ((k & 7) == 0) scales[k >> 3] = s;
                }
            }
        } else if (write) {
            uint2 *to = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(is_k ? a.kc : a.vc) + base);
            if (PAIRS) {
                const uint2 lo = pack_bf16x4(x), hi = pack_bf16x4(y);
                *reinterpret_cast<uint4 *>(to + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                to[c] = pack_bf16x4(x);
                to[d] = pack_bf16x4(y);
            }
        }
    }
}

template <int D, bool I, bool Q8> cudaError_t launch_append_type(const AppendArgs &a, cudaStream_t stream) {
    const int total = a.q_heads + 2 * a.kv_heads;
    const auto grid = [&](int n) {
        const long long per = (256 / D) * n, warps = a.rows * ((total + per - 1) / per);
        return dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps), 1, 1);
    };
    // One head a lane group while the rows are few (latency: all of it in flight at once anyway), over a bf16 cache four once
    // there are enough to fill the SMs several times.  One against four, 32 + 2 x 8 heads, halves, without and with norms:
    // heads of 128, 16 rows 1.9 and 2.3 us (2.0 and 2.9), 256 rows (3 2^19 values) 2.8 and 2.7 (3.2 and 3.4), 512 rows 5.2
    // and 4.2 (5.8 and 5.1), 8191 rows 69 and 51 (74 and 56); heads of 64, 512 rows (as many values) 2.8 and 2.8 (3.3 and
    // 3.4), 1024 rows 5.2 and 4.1 (6.0 and 5.2).  Over a Q8_0 cache, whose scales take more instructions than the loads wait
    // for, four are slower everywhere: 16 rows of heads of 128 2.6 and 5.5, 512 rows 6.8 and 7.6, 8191 rows 79 and 88.
    if (!Q8)
        if ((long long)a.rows * total * D >= kAppendWide)
            return kv_launch(append_kernel<D, I, false, 4>, grid(4), 32 * kAppendWarps, 0, stream, a);
    return kv_launch(append_kernel<D, I, Q8, 1>, grid(1), 32 * kAppendWarps, 0, stream, a);
}

template <int D> cudaError_t launch_append(const AppendArgs &a, bool interleaved, bool q8, cudaStream_t stream) {
    if (interleaved || a.rot == 0)
        return q8 ? launch_append_type<D, true, true>(a, stream) : launch_append_type<D, true, false>(a, stream);
    return q8 ? launch_append_type<D, false, true>(a, stream) : launch_append_type<D, false, false>(a, stream);
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
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = smem > 40 * 1024 ? kv_allow_smem(slots_kernel, (Q8_MAX_REQUESTS + 1) * 8, &allowed) : cudaSuccess;
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
