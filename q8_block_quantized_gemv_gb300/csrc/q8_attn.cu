// Attention over the paged key-value cache: the entry points q8_attn_decode and q8_attn_prefill (formulas in q8_gemv.h)
// and what they check.
#include <math.h>

#include <atomic>

#include "q8_attn.h"

namespace q8 {
namespace {

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
    if (a.group > 128) return Q8_ERR_SHAPE;  // a query tile holds whole tokens
    const cudaError_t e = q8::launch_attn_prefill(a, cache->dim, q8::kv_is_q8(cache), (cudaStream_t)stream);
    return e == cudaSuccess ? Q8_OK : q8::kv_cuda_fail(e);
}
