// The rules on logits and the token chosen, first form: one CTA a row, the counts of a window of the vocabulary at a time in
// shared memory, the history read again for each window.
#include <limits.h>
#include <math.h>

#include "q8_device.cuh"
#include "q8_kv.h"

namespace q8 {
namespace {

constexpr int kThreadsC = 512;
constexpr int kWindow = 8192;  // tokens whose counts are in shared memory at a time

// A token's entry: how often it stands in the answer in the low 20 bits, its place among the biases + 1 in the next 11,
// and whether it stands in the prompt.
constexpr uint32_t kCount = 0xFFFFFu, kPrompt = 0x80000000u;

struct ChooseArgs {
    q8_choice c;
    const float *logits;
    float *out;
    int64_t *idx;
    int ldl, ldo, N;
};

__device__ __forceinline__ int64_t token_at(const q8_choice &c, int r, int i) {
    const size_t at = (size_t)r * c.history_pitch + i;
    return c.history_wide ? static_cast<const int64_t *>(c.history)[at] : static_cast<const int *>(c.history)[at];
}

__global__ void __launch_bounds__(kThreadsC) choose_kernel(const __grid_constant__ ChooseArgs a) {
    __shared__ uint32_t entry[kWindow];
    __shared__ unsigned long long best[kThreadsC / 32];
    const q8_choice &c = a.c;
    const int r = blockIdx.x;
    const float rep = c.repetition ? c.repetition[r] : 1.0f, freq = c.frequency ? c.frequency[r] : 0.0f;
    const float pres = c.presence ? c.presence[r] : 0.0f, temp = c.temperature ? c.temperature[r] : 0.0f;
    int length = 0, prompt = 0;
    if (c.history) {
        length = min(max(c.lengths[r], 0), c.history_width);
        prompt = c.prompts ? min(max(c.prompts[r], 0), length) : 0;
    }
    const int mrow = c.mask ? (c.mask_rows ? c.mask_rows[r] : r) : -1;
    const int *mask = mrow >= 0 && mrow < c.mask_count ? c.mask + (size_t)mrow * c.mask_pitch : nullptr;
    unsigned long long key = 0ull;
    for (int n0 = 0; n0 < a.N; n0 += kWindow) {
        const int count = min(kWindow, a.N - n0);
        for (int i = threadIdx.x; i < count; i += kThreadsC) entry[i] = 0u;
        __syncthreads();
        if (c.bias_ids)
            for (int i = threadIdx.x; i < c.bias_width; i += kThreadsC) {
                const int n = c.bias_ids[(size_t)r * c.bias_width + i];
                if (n >= n0 && n < n0 + count) atomicMax(&entry[n - n0], (uint32_t)(i + 1) << 20);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < length; i += kThreadsC) {
            const int64_t n = token_at(c, r, i);
            if (n >= n0 && n < n0 + count) {
                if (i < prompt)
                    atomicOr(&entry[n - n0], kPrompt);
                else
                    atomicAdd(&entry[n - n0], 1u);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kThreadsC) {
            const int n = n0 + i;
            float v = a.logits[(size_t)r * a.ldl + n];
            const uint32_t e = entry[i];
            if (e & (kPrompt | kCount)) v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
            if (e & kCount) {
                v = __fsub_rn(v, __fmul_rn(freq, (float)(e & kCount)));
                v = __fsub_rn(v, pres);
            }
            const uint32_t place = (e & ~kPrompt) >> 20;
            if (place) v = __fadd_rn(v, c.bias[(size_t)r * c.bias_width + place - 1]);
            if (temp > 0.0f) v = __fdiv_rn(v, temp);
            const bool allowed = !mask || (mask[n >> 5] >> (n & 31)) & 1;
            if (allowed) {
                const float score = c.noise && temp > 0.0f ? __fadd_rn(v, c.noise[(size_t)r * c.noise_pitch + n]) : v;
                const unsigned long long k = argmax_key(score, n);
                key = k > key ? k : key;
            }
            if (a.out) a.out[(size_t)r * a.ldo + n] = allowed ? v : -INFINITY;
        }
        __syncthreads();
    }
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
        key = other > key ? other : key;
    }
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = key;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreadsC / 32; ++w) key = best[w] > key ? best[w] : key;
        a.idx[r] = key ? (int64_t)(0xFFFFFFFFull - (key & 0xFFFFFFFFull)) : -1;
    }
}

}  // namespace
}  // namespace q8

extern "C" q8_status q8_choose(const float *logits, int ldl, const q8_choice *rules, float *out, int ldo, int64_t *idx,
                               int m, int N, q8_stream_t stream) {
    using q8::kv_aligned;
    using q8::kv_overlap;
    if (!logits || !idx) return Q8_ERR_ARG;
    if (m < 1 || m > 65535 || N < 1 || N >= INT_MAX - 1023 || ldl < N || (out && ldo < N)) return Q8_ERR_SHAPE;
    q8::ChooseArgs a = {};
    if (rules) a.c = *rules;
    const q8_choice &c = a.c;
    if ((c.history && !c.lengths) || (!c.bias_ids != !c.bias)) return Q8_ERR_ARG;
    if (c.history && (c.history_width < 1 || c.history_width > Q8_MAX_HISTORY || c.history_pitch < c.history_width))
        return Q8_ERR_SHAPE;
    if (c.bias_ids && (c.bias_width < 1 || c.bias_width > Q8_MAX_BIAS)) return Q8_ERR_SHAPE;
    if (c.mask && (c.mask_count < 1 || c.mask_pitch < (N - 1) / 32 + 1)) return Q8_ERR_SHAPE;
    if (c.noise && c.noise_pitch < N) return Q8_ERR_SHAPE;
    const void *words[] = {logits, out, c.repetition, c.frequency, c.presence, c.temperature, c.lengths,
                           c.prompts, c.bias_ids, c.bias, c.mask, c.mask_rows, c.noise};
    for (const void *p : words)
        if (!kv_aligned(p, 4)) return Q8_ERR_ALIGN;
    if (!kv_aligned(idx, 8) || !kv_aligned(c.history, c.history_wide ? 8 : 4)) return Q8_ERR_ALIGN;
    // what the call reads, against what it writes
    const int64_t row = m - 1, lb = (row * ldl + N) * 4, ob = (row * ldo + N) * 4, ib = (int64_t)m * 8;
    const struct { const void *p; int64_t bytes; } ins[] = {
        {c.repetition, m * 4ll}, {c.frequency, m * 4ll}, {c.presence, m * 4ll}, {c.temperature, m * 4ll},
        {c.history, (row * c.history_pitch + c.history_width) * (c.history_wide ? 8 : 4)},
        {c.lengths, m * 4ll}, {c.prompts, m * 4ll}, {c.bias_ids, (int64_t)m * c.bias_width * 4},
        {c.bias, (int64_t)m * c.bias_width * 4}, {c.mask, ((int64_t)(c.mask_count - 1) * c.mask_pitch + (N - 1) / 32 + 1) * 4},
        {c.mask_rows, m * 4ll}, {c.noise, (row * c.noise_pitch + N) * 4}};
    for (const auto &in : ins)
        if (kv_overlap(out, ob, in.p, in.bytes) || kv_overlap(idx, ib, in.p, in.bytes)) return Q8_ERR_ARG;
    if (kv_overlap(idx, ib, logits, lb) || kv_overlap(idx, ib, out, ob)) return Q8_ERR_ARG;
    if (kv_overlap(out, ob, logits, lb) && !(out == logits && ldo == ldl)) return Q8_ERR_ARG;
    a.logits = logits;
    a.out = out;
    a.idx = idx;
    a.ldl = ldl;
    a.ldo = ldo;
    a.N = N;
    q8::choose_kernel<<<m, q8::kThreadsC, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q8_OK : q8::kv_cuda_fail(e);
}
