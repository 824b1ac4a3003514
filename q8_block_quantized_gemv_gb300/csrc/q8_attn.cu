// Attention over the paged key-value cache: entry points of q8_attn_decode and q8_attn_prefill (formulas in
// q8_gemv.h), and the kernel behind both.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "q8_attn.h"
#include "q8_device.cuh"

namespace q8 {
namespace {

constexpr int kRowWarps = 4;

// Four consecutive cached values from value index i.
template <bool Q8> __device__ __forceinline__ float2 cached2(const void *p, const float *s, long long i) {
    if (Q8) {
        const char2 c = *reinterpret_cast<const char2 *>(static_cast<const signed char *>(p) + i);
        const float d = s[i / kBlock];
        return make_float2((float)c.x * d, (float)c.y * d);
    }
    const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// One warp per (row, query head): the keys one by one, the head's values on the lanes, with the running maximum and
// sum of the softmax.
template <int D, bool Q8> __global__ void __launch_bounds__(32 * kRowWarps) attn_rows_kernel(AttnArgs a) {
    constexpr int E = D / 64;  // pairs a lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.x * kRowWarps + (threadIdx.x >> 5), t = blockIdx.y;
    if (h >= a.heads) return;
    int r = t, len, pos;
    if (a.row_start) {
        int lo = 0, hi = a.R;  // the last r with row_start[r] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.row_start[mid] <= t) lo = mid; else hi = mid - 1;
        }
        r = lo;
        len = r < a.R ? a.lens[r] : 0;
        pos = r < a.R ? len - (a.row_start[r + 1] - t) : -1;
    } else {
        len = a.lens[r];
        pos = len - 1;
    }
    const int hk = h / a.group;
    float2 q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(a.q + (size_t)t * a.ldq + (size_t)h * D + 64 * e + 2 * lane);
        q[e] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        o[e] = make_float2(0.0f, 0.0f);
    }
    float m = -INFINITY, l = 0.0f;
    const long long most = (long long)a.width * a.page_size;
    const int end = (int)min((long long)min(len, pos + 1), most);
    for (int j = 0; j < end; ++j) {
        if (a.window && j >= a.sinks && pos - j >= a.window) {
            j = max(j, pos - a.window);
            continue;
        }
        const int page = a.table[(size_t)r * a.pitch + j / a.page_size];
        if (page < 0 || page >= a.pages) continue;
        const long long at = (long long)page * a.page_stride + ((long long)hk * a.page_size + j % a.page_size) * D;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 k = cached2<Q8>(a.k, a.ks, at + 64 * e + 2 * lane);
            s = fmaf(q[e].x, k.x, fmaf(q[e].y, k.y, s));
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float old = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * old + p;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 v = cached2<Q8>(a.v, a.vs, at + 64 * e + 2 * lane);
            o[e].x = fmaf(p, v.x, o[e].x * old);
            o[e].y = fmaf(p, v.y, o[e].y * old);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[e].x * inv, o[e].y * inv);
        *reinterpret_cast<uint32_t *>(a.out + (size_t)t * a.ldo + (size_t)h * D + 64 * e + 2 * lane) =
            *reinterpret_cast<const uint32_t *>(&b);
    }
}

cudaError_t launch_rows(const AttnArgs &a, int dim, bool q8, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.heads + kRowWarps - 1) / kRowWarps), (unsigned)a.rows, 1);
    if (dim == 128)
        return q8 ? kv_launch(attn_rows_kernel<128, true>, grid, 32 * kRowWarps, 0, stream, a)
                  : kv_launch(attn_rows_kernel<128, false>, grid, 32 * kRowWarps, 0, stream, a);
    return q8 ? kv_launch(attn_rows_kernel<64, true>, grid, 32 * kRowWarps, 0, stream, a)
              : kv_launch(attn_rows_kernel<64, false>, grid, 32 * kRowWarps, 0, stream, a);
}

// The checks both calls share; fills the arguments.
q8_status attn_args(AttnArgs *a, const void *q, int ldq, const q8_kv_cache *c, const int *table, int width, int pitch,
                    const int *lens, const int *row_start, void *out, int ldo, int rows, int R, int q_heads,
                    float scale, int window, int sinks, void *workspace) {
    if (!q || !c || !table || !lens || !out || !workspace) return Q8_ERR_ARG;
    if (!(fabsf(scale) < INFINITY) || window < 0 || sinks < 0) return Q8_ERR_ARG;
    q8_status st = kv_check_cache(c);
    if (st != Q8_OK) return st;
    if (R < 1 || R > Q8_MAX_REQUESTS || rows < 1 || rows > (1 << 24) || q_heads < 1 || q_heads % c->heads != 0 ||
        q_heads > (1 << 20) / c->dim || width < 1 || pitch < width || ldq < q_heads * c->dim || ldo < q_heads * c->dim ||
        (int64_t)width * c->page_size > 0x7FFFFFFFll)
        return Q8_ERR_SHAPE;
    if (ldq % 8 || ldo % 8 || !kv_aligned(q, 16) || !kv_aligned(out, 16) || !kv_aligned(workspace, 16) ||
        !kv_aligned(table, 4) || !kv_aligned(lens, 4) || !kv_aligned(row_start, 4))
        return Q8_ERR_ALIGN;
    const int64_t n = (int64_t)q_heads * c->dim;
    const int64_t ob = 2 * ((int64_t)(rows - 1) * ldo + n), wb = q8_attn_workspace_bytes();
    const void *ins[4] = {q, table, lens, row_start};
    const int64_t inb[4] = {2 * ((int64_t)(rows - 1) * ldq + n), 4 * ((int64_t)(R - 1) * pitch + width), 4ll * R,
                            4ll * (R + 1)};
    for (int i = 0; i < 4; ++i)
        if (kv_overlap(out, ob, ins[i], inb[i]) || kv_overlap(workspace, wb, ins[i], inb[i])) return Q8_ERR_ARG;
    if (kv_overlaps_cache(c, out, ob) || kv_overlaps_cache(c, workspace, wb) || kv_overlap(out, ob, workspace, wb))
        return Q8_ERR_ARG;
    *a = {static_cast<const uint16_t *>(q), static_cast<uint16_t *>(out), c->k, c->v, c->k_scale, c->v_scale, table,
          lens, row_start, c->page_stride, ldq, ldo, c->pages, c->page_size, width, pitch, rows, R, q_heads, c->heads,
          q_heads / c->heads, scale, window, sinks, static_cast<unsigned char *>(workspace)};
    return Q8_OK;
}

}  // namespace

cudaError_t sm_count_of_device(int *sms) {
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && (*sms = cache[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev >= 0 && dev < 64) cache[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

}  // namespace q8

extern "C" int64_t q8_attn_workspace_bytes(void) { return q8::kAttnWorkspaceBytes; }

extern "C" q8_status q8_attn_decode(const void *q, int ldq, const q8_kv_cache *cache, const int *block_table,
                                    int table_width, int table_pitch, const int *lens, void *out, int ldo, int R,
                                    int q_heads, float scale, int window, int sinks, void *workspace,
                                    q8_stream_t stream) {
    q8::AttnArgs a;
    q8_status st = q8::attn_args(&a, q, ldq, cache, block_table, table_width, table_pitch, lens, nullptr, out, ldo, R,
                                 R, q_heads, scale, window, sinks, workspace);
    if (st != Q8_OK) return st;
    const cudaError_t e = q8::launch_attn_decode(a, cache->dim, q8::kv_is_q8(cache), (cudaStream_t)stream);
    return e == cudaSuccess ? Q8_OK : q8::kv_cuda_fail(e);
}

extern "C" q8_status q8_attn_prefill(const void *q, int ldq, const q8_kv_cache *cache, const int *block_table,
                                     int table_width, int table_pitch, const int *lens, const int *row_start, void *out,
                                     int ldo, int rows, int R, int q_heads, float scale, int window, int sinks,
                                     void *workspace, q8_stream_t stream) {
    if (!row_start) return Q8_ERR_ARG;
    q8::AttnArgs a;
    q8_status st = q8::attn_args(&a, q, ldq, cache, block_table, table_width, table_pitch, lens, row_start, out, ldo,
                                 rows, R, q_heads, scale, window, sinks, workspace);
    if (st != Q8_OK) return st;
    if (rows > 65535) return Q8_ERR_SHAPE;
    const cudaError_t e = q8::launch_rows(a, cache->dim, q8::kv_is_q8(cache), (cudaStream_t)stream);
    return e == cudaSuccess ? Q8_OK : q8::kv_cuda_fail(e);
}
