// Weights of 4 bits with group scales: the tiled form, argument checks and the entry points of their products.
#include <limits.h>
#include <math.h>
#include <string.h>

#include "q8_kv.h"
#include "q8_launch.h"
#include "q8_w4.h"

namespace {

using q8::kv_aligned;
using q8::kv_cuda_fail;
using q8::kv_overlap;

constexpr unsigned kWeightFlags = Q8_W4_ZEROS | Q8_W4_BF16;

q8_status check_plain(const uint8_t *codes, const void *scales, const uint8_t *zeros, int K, int N, int group,
                      unsigned flags, const void *w) {
    if (!codes || !scales || !w || (flags & ~kWeightFlags) || ((flags & Q8_W4_ZEROS) != 0) != (zeros != nullptr))
        return Q8_ERR_ARG;
    const int64_t bytes = q8_w4_bytes(K, N, group, flags);
    if (bytes < 0) return Q8_ERR_SHAPE;
    const int64_t groups = K / group;
    if (kv_overlap(w, bytes, codes, (int64_t)(K / 2) * N) || kv_overlap(w, bytes, scales, groups * N * 2) ||
        kv_overlap(w, bytes, zeros, groups * N))
        return Q8_ERR_ARG;
    return Q8_OK;
}

// The word of rows k0 .. k0 + 7 of column n: row pairs (2p, 2p + 1) are the two halves of codes row k0 / 2 + p.
__host__ __device__ inline uint32_t word_of_column(const uint8_t *codes, int N, int k0, int n) {
    uint32_t w = 0;
    for (int p = 0; p < 4; ++p) {
        const uint32_t c = codes[(int64_t)(k0 / 2 + p) * N + n];
        w |= ((c & 15u) << (4 * p)) | ((c >> 4) << (16 + 4 * p));
    }
    return w;
}

// The part of unit (strip, g) that belongs to column c of the strip.
__host__ __device__ inline void tile_column(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int N,
                                            int group, int n, int g, int c, unsigned char *unit) {
    const bool live = n < N;
    for (int b = 0; b < group / 32; ++b)
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<uint32_t *>(unit + q8::w4_word(group, b, t, c)) =
                live ? word_of_column(codes, N, g * group + 32 * b + 8 * t, n) : 0u;
    *reinterpret_cast<uint16_t *>(unit + 16 * group + 2 * c) = live ? scales[(int64_t)g * N + n] : (uint16_t)0;
    if (zeros) unit[16 * group + 64 + c] = live ? zeros[(int64_t)g * N + n] & 127 : 0;
}

__global__ void tile_kernel(const uint8_t *__restrict__ codes, const uint16_t *__restrict__ scales,
                            const uint8_t *__restrict__ zeros, int N, int group, int groups, int unit, int64_t units,
                            unsigned char *__restrict__ w) {
    const int c = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);  // a warp a unit, a lane a column
    if (u >= units) return;
    const int64_t n = u / groups * q8::kW4Strip + c;
    tile_column(codes, scales, zeros, N, group, n < N ? (int)n : N, (int)(u % groups), c, w + u * unit);
}

// Nothing, behind tile_kernel: a kernel launched without the programmatic attribute starts when all before it has ended and its
// writes are seen, so that a product that starts early starts behind those writes.  Behind tile_kernel itself its first
// copies of a weight declared constant would be ordered by nothing.
__global__ void tiled_kernel() {}

// A product's weight against K; `first` is the call's first weight.
q8_status check_weight(const q8_weight4 *w, const q8_weight4 *first, int K) {
    if (!w || !w->w || (w->flags & ~kWeightFlags) || w->group != first->group || w->flags != first->flags)
        return Q8_ERR_ARG;
    if (q8_w4_bytes(K, w->N, w->group, w->flags) < 0) return Q8_ERR_SHAPE;
    return kv_aligned(w->w, 16) ? Q8_OK : Q8_ERR_ALIGN;
}

int64_t weight_bytes(const q8_weight4 *w, int K) { return q8_w4_bytes(K, w->N, w->group, w->flags); }

q8_status check_call(const void *x, int m, int K, unsigned flags) {
    if (!x || (flags & ~Q8_FLAG_CONSTANT_WEIGHTS)) return Q8_ERR_ARG;
    if (m < 1 || m > Q8_MAX_CHUNK || K <= 0) return Q8_ERR_SHAPE;
    return kv_aligned(x, 16) ? Q8_OK : Q8_ERR_ALIGN;
}

q8::W4Args make_args(const void *x, const q8_weight4 *first, int m, int K) {
    q8::W4Args a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.m = m;
    a.K = K;
    a.group = first->group;
    a.zeros = (first->flags & Q8_W4_ZEROS) != 0;
    a.bf16 = (first->flags & Q8_W4_BF16) != 0;
    a.unit = q8::w4_unit(a.group, a.zeros);
    return a;
}

void add_part(q8::W4Args *a, const q8_weight4 *w, float *y) {
    const int i = a->nparts++, Np = q8_padded_n(w->N);
    a->part[i] = {static_cast<const unsigned char *>(w->w), y, w->N, Np,
                  (i ? a->part[i - 1].strip_end : 0) + Np / q8::kW4Strip};
}

q8_status launch(const q8::W4Args &a, unsigned flags, q8_stream_t stream) {
    const bool constant = (flags & Q8_FLAG_CONSTANT_WEIGHTS) != 0;
    const cudaError_t e = a.m <= q8::kW4StreamRows ? q8::launch_w4_stream(a, constant, (cudaStream_t)stream)
                                                   : q8::launch_w4_gemm(a, constant, (cudaStream_t)stream);
    return e == cudaSuccess ? Q8_OK : kv_cuda_fail(e);
}

}  // namespace

extern "C" int64_t q8_w4_bytes(int K, int N, int group, unsigned int flags) {
    // (the products count rows of K to the end of the last 128 in an int)
    if ((group != 32 && group != 64 && group != 128) || K <= 0 || K > INT_MAX - 127 || K % group != 0 || q8_padded_n(N) < 0 ||
        (flags & ~kWeightFlags))
        return -1;
    return (int64_t)(q8_padded_n(N) / q8::kW4Strip) * (K / group) * q8::w4_unit(group, (flags & Q8_W4_ZEROS) != 0);
}

extern "C" q8_status q8_w4_tile(const uint8_t *codes, const void *scales, const uint8_t *zeros, int K, int N, int group,
                                unsigned int flags, void *w) {
    const q8_status st = check_plain(codes, scales, zeros, K, N, group, flags, w);
    if (st != Q8_OK) return st;
    if (!kv_aligned(w, 4) || !kv_aligned(scales, 2)) return Q8_ERR_ALIGN;
    const int groups = K / group, unit = q8::w4_unit(group, zeros != nullptr);
    unsigned char *to = static_cast<unsigned char *>(w);
    for (int n0 = 0; n0 < q8_padded_n(N); n0 += q8::kW4Strip)
        for (int g = 0; g < groups; ++g, to += unit)
            for (int c = 0; c < q8::kW4Strip; ++c)
                tile_column(codes, static_cast<const uint16_t *>(scales), zeros, N, group, N - n0 > c ? n0 + c : N, g, c, to);
    return Q8_OK;
}

extern "C" q8_status q8_w4_tile_device(const uint8_t *codes, const void *scales, const uint8_t *zeros, int K, int N,
                                       int group, unsigned int flags, void *w, q8_stream_t stream) {
    const q8_status st = check_plain(codes, scales, zeros, K, N, group, flags, w);
    if (st != Q8_OK) return st;
    if (!kv_aligned(w, 16) || !kv_aligned(scales, 2)) return Q8_ERR_ALIGN;
    const int64_t units = (int64_t)(q8_padded_n(N) / q8::kW4Strip) * (K / group);
    if ((units + 7) / 8 > 0x7FFFFFFF) return Q8_ERR_SHAPE;
    tile_kernel<<<(unsigned)((units + 7) / 8), 256, 0, (cudaStream_t)stream>>>(
        codes, static_cast<const uint16_t *>(scales), zeros, N, group, K / group, q8::w4_unit(group, zeros != nullptr),
        units, static_cast<unsigned char *>(w));
    tiled_kernel<<<1, 32, 0, (cudaStream_t)stream>>>();
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q8_OK : kv_cuda_fail(e);
}

extern "C" q8_status q8_w4_repack(const void *blocks, int K, int N, uint8_t *codes, uint16_t *scales) {
    if (!blocks || !codes || !scales) return Q8_ERR_ARG;
    if (K <= 0 || K % 32 != 0 || q8_padded_n(N) < 0) return Q8_ERR_SHAPE;
    const int nb = K / 32;
    const unsigned char *blk = static_cast<const unsigned char *>(blocks);
    for (int n = 0; n < N; ++n)
        for (int b = 0; b < nb; ++b, blk += 18) {
            const uint16_t d = (uint16_t)(blk[0] | (blk[1] << 8));
            if ((d & 0x7C00u) == 0x7C00u) return Q8_ERR_NOT_Q8_0;  // infinite or NaN
            scales[(int64_t)b * N + n] = d;
            for (int i = 0; i < 16; ++i) {
                // rows 2i and 2i + 1 of the block: both in the low halves of bytes 2i, 2i + 1, or both in the high ones
                const unsigned char *two = blk + 2 + 2 * (i & 7);
                const int shift = i < 8 ? 0 : 4;
                codes[((int64_t)b * 16 + i) * N + n] =
                    (uint8_t)(((two[0] >> shift) & 15) | (((two[1] >> shift) & 15) << 4));
            }
        }
    return Q8_OK;
}

extern "C" q8_status q8_gemv4_parts(const void *x, const q8_weight4 *weights, float *const *y, int nparts, int m, int K,
                                    unsigned int flags, q8_stream_t stream) {
    q8_status st = check_call(x, m, K, flags);
    if (st != Q8_OK) return st;
    if (!weights || !y) return Q8_ERR_ARG;
    if (nparts < 1 || nparts > Q8_MAX_PARTS) return Q8_ERR_SHAPE;
    long long strips = 0;
    for (int p = 0; p < nparts; ++p) {
        st = check_weight(&weights[p], &weights[0], K);
        if (st != Q8_OK) return st;
        if (!y[p]) return Q8_ERR_ARG;
        if (!kv_aligned(y[p], 16)) return Q8_ERR_ALIGN;
        strips += q8_padded_n(weights[p].N) / q8::kW4Strip;
    }
    if (strips > 0x3FFFFFFF) return Q8_ERR_SHAPE;
    for (int p = 0; p < nparts; ++p) {
        const int64_t bytes = (int64_t)m * q8_padded_n(weights[p].N) * 4;
        if (kv_overlap(y[p], bytes, x, (int64_t)m * K * 2)) return Q8_ERR_ARG;
        for (int i = 0; i < nparts; ++i)
            if (kv_overlap(y[p], bytes, weights[i].w, weight_bytes(&weights[i], K)) ||
                (i != p && kv_overlap(y[p], bytes, y[i], (int64_t)m * q8_padded_n(weights[i].N) * 4)))
                return Q8_ERR_ARG;
    }
    q8::W4Args a = make_args(x, weights, m, K);
    for (int p = 0; p < nparts; ++p) add_part(&a, &weights[p], y[p]);
    return launch(a, flags, stream);
}

extern "C" q8_status q8_gemv4(const void *x, const q8_weight4 *weight, float *y, int m, int K, unsigned int flags,
                              q8_stream_t stream) {
    return q8_gemv4_parts(x, weight, &y, 1, m, K, flags, stream);
}

extern "C" q8_status q8_gemv4_glu(const void *x, const q8_weight4 *gate, const q8_weight4 *up, float *out, void *out_bf16,
                                  int m, int K, unsigned int flags, q8_stream_t stream) {
    q8_status st = check_call(x, m, K, flags);
    if (st != Q8_OK) return st;
    if (!gate || !up || (!out && !out_bf16)) return Q8_ERR_ARG;
    for (const q8_weight4 *w : {gate, up}) {
        st = check_weight(w, gate, K);
        if (st != Q8_OK) return st;
    }
    if (gate->N != up->N) return Q8_ERR_SHAPE;
    if (!kv_aligned(out, 16) || !kv_aligned(out_bf16, 16)) return Q8_ERR_ALIGN;
    const int64_t values = (int64_t)m * q8_padded_n(gate->N);
    if (kv_overlap(out, values * 4, out_bf16, values * 2)) return Q8_ERR_ARG;
    for (const q8_weight4 *w : {gate, up})
        if (kv_overlap(out, values * 4, w->w, weight_bytes(w, K)) || kv_overlap(out_bf16, values * 2, w->w, weight_bytes(w, K)))
            return Q8_ERR_ARG;
    if (kv_overlap(out, values * 4, x, (int64_t)m * K * 2) || kv_overlap(out_bf16, values * 2, x, (int64_t)m * K * 2))
        return Q8_ERR_ARG;
    q8::W4Args a = make_args(x, gate, m, K);
    a.epi = q8::kW4Glu;
    a.ybf = static_cast<uint16_t *>(out_bf16);
    add_part(&a, gate, out);
    add_part(&a, up, out);
    return launch(a, flags, stream);
}

extern "C" q8_status q8_gemv4_residual_norm(const void *x, const q8_weight4 *weight, const float *residual,
                                            const float *gamma, float eps, float *h, void *out_bf16, int m, int K,
                                            unsigned int flags, q8_stream_t stream) {
    q8_status st = check_call(x, m, K, flags);
    if (st != Q8_OK) return st;
    st = check_weight(weight, weight, K);
    if (st != Q8_OK) return st;
    if (!residual || !gamma || !h || !out_bf16 || !(eps >= 0.0f) || !(eps < INFINITY)) return Q8_ERR_ARG;
    if (!kv_aligned(h, 16) || !kv_aligned(out_bf16, 16) || !kv_aligned(residual, 4) || !kv_aligned(gamma, 4))
        return Q8_ERR_ALIGN;
    const int N = weight->N, Np = q8_padded_n(N);
    const int64_t hb = (int64_t)m * Np * 4, ob = hb / 2;
    if ((h != residual && kv_overlap(h, hb, residual, hb)) || kv_overlap(out_bf16, ob, residual, hb) ||
        kv_overlap(out_bf16, ob, h, hb))
        return Q8_ERR_ARG;
    const void *ins[3] = {x, weight->w, gamma};
    const int64_t inb[3] = {(int64_t)m * K * 2, weight_bytes(weight, K), (int64_t)N * 4};
    for (int i = 0; i < 3; ++i)
        if (kv_overlap(h, hb, ins[i], inb[i]) || kv_overlap(out_bf16, ob, ins[i], inb[i])) return Q8_ERR_ARG;
    q8::W4Args a = make_args(x, weight, m, K);
    a.epi = q8::kW4Residual;
    a.res = residual;
    add_part(&a, weight, h);
    st = launch(a, flags, stream);
    if (st != Q8_OK) return st;
    const q8::NormRows nr = {h, gamma, eps, static_cast<uint16_t *>(out_bf16), nullptr, nullptr, N, Np};
    const cudaError_t e = q8::launch_norm_rows(nr, m, (cudaStream_t)stream, true);
    return e == cudaSuccess ? Q8_OK : kv_cuda_fail(e);
}
