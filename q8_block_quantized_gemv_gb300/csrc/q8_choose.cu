// The rules on logits and the token chosen (formulas in q8_gemv.h): one cluster of up to eight CTAs a row, one pass over the
// logits.
//
// 8 bytes a logit, 4 more with noise, bound a large step; what has to stay out of their way is the look-up of how often a
// token was said.  Each CTA owns a slice of the vocabulary and holds one word for each of its tokens in shared memory: how
// often it stands in the answer, whether it stands in the prompt, its place among the biases.  The words come from integer
// atomics, whose order does not matter.  A history of up to kLocal tokens is read whole by every CTA of the row, which keeps
// what falls into its slice and needs no word from the others; of a longer one each CTA reads its share and sends what it
// finds to the owner through distributed shared memory.  A vocabulary beyond eight slices of kMostSlice takes several turns.
// The first logits are asked for before the words are made.  Each step of a rule is one fp32 operation rounded once (no
// contraction), so that the bits are those of any other implementation.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include "q8_device.cuh"
#include "q8_kv.h"

namespace q8 {
namespace {

constexpr int kThreadsC = 512;
constexpr int kMostCtas = 8;
constexpr int kMostSlice = 49152;  // 192 KB of words
constexpr int kLocal = 8192;

// A token's word: how often it stands in the answer in the low 20 bits, its place among the biases + 1 in the next 11,
// and whether it stands in the prompt.
constexpr uint32_t kCount = 0xFFFFFu, kPrompt = 0x80000000u;

struct ChooseArgs {
    q8_choice c;
    const float *logits;
    float *out;
    int64_t *idx;
    int ldl, ldo, N;
    int slice;   // tokens of a CTA, a multiple of 128
    bool words;  // whether any rule needs them
};

struct Row {  // a row's numbers
    float rep, freq, pres, temp;
    float inv, span;  // 1 / temp; the quotients that over_temperature makes without a division are of |v| in 1/span .. span
    const float *bias;
};

// The rules of a word on a logit.
__device__ __forceinline__ float ruled(float v, uint32_t word, const Row &w) {
    if (word & (kPrompt | kCount)) v = v > 0.0f ? __fdiv_rn(v, w.rep) : __fmul_rn(v, w.rep);
    if (word & kCount) {
        v = __fsub_rn(v, __fmul_rn(w.freq, (float)(word & kCount)));
        v = __fsub_rn(v, w.pres);
    }
    const uint32_t place = (word & ~kPrompt) >> 20;
    if (place) v = __fadd_rn(v, w.bias[place - 1]);
    return v;
}

// v / temp, rounded once, for every logit of a row.  With y the correctly rounded 1 / temp, v y is within two units in the
// last place, one correction by its remainder makes it one of the two nearest, whose remainder v - q temp is exact in one
// fma, and q + remainder * y is then the correctly rounded quotient (Markstein's theorem), where nothing over- or
// underflows.  Elsewhere, and for zeros, whose sign the remainder loses, the division itself.  A division of each logit took
// more instructions than everything else.
__device__ __forceinline__ float over_temperature(float v, const Row &w) {
    float q = v * w.inv;
    q = fmaf(fmaf(-q, w.temp, v), w.inv, q);
    q = fmaf(fmaf(-q, w.temp, v), w.inv, q);
    const float size = fabsf(v);
    return size <= w.span && size * w.span >= 1.0f ? q : __fdiv_rn(v, w.temp);
}

// VEC: rows of logits, output and noise are 16-byte aligned, a thread takes four tokens in a row; else four that are
// kThreadsC apart.
template <bool VEC, bool WIDE>
__global__ void __launch_bounds__(kThreadsC, 2) choose_kernel(const __grid_constant__ ChooseArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) uint32_t word_of[];
    __shared__ unsigned long long best[kThreadsC / 32], of_rank[kMostCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const q8_choice &c = a.c;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x, r = (int)blockIdx.y, slice = a.slice;
    const int turn = ctas * slice;  // tokens of a turn
    auto clear = [&](int count) {
        for (int i = threadIdx.x; i < (count + 3) / 4; i += kThreadsC)
            reinterpret_cast<uint4 *>(word_of)[i] = make_uint4(0u, 0u, 0u, 0u);
    };
    if (a.words) clear(min(slice, max(0, a.N - rank * slice)));
    asm volatile("griddepcontrol.wait;" ::: "memory");

    Row row;
    row.rep = c.repetition ? c.repetition[r] : 1.0f;
    row.freq = c.frequency ? c.frequency[r] : 0.0f;
    row.pres = c.presence ? c.presence[r] : 0.0f;
    row.temp = c.temperature ? c.temperature[r] : 0.0f;
    const bool hot = row.temp > 0.0f;
    row.inv = __frcp_rn(row.temp);
    row.span = row.temp >= 0x1p-20f && row.temp <= 0x1p20f ? 0x1p80f : 0.0f;  // 0: none
    row.bias = c.bias ? c.bias + (size_t)r * c.bias_width : nullptr;
    int length = 0, prompt = 0;
    if (c.history) {
        length = min(max(c.lengths[r], 0), c.history_width);
        prompt = c.prompts ? min(max(c.prompts[r], 0), length) : 0;
    }
    const int mrow = c.mask ? (c.mask_rows ? c.mask_rows[r] : r) : -1;
    const int *mask = mrow >= 0 && mrow < c.mask_count ? c.mask + (size_t)mrow * c.mask_pitch : nullptr;
    const float *noise = c.noise && hot ? c.noise + (size_t)r * c.noise_pitch : nullptr;
    const float *logits = a.logits + (size_t)r * a.ldl;
    float *out = a.out ? a.out + (size_t)r * a.ldo : nullptr;
    const size_t said = (size_t)r * c.history_pitch;
    const bool far = length > kLocal && ctas > 1;  // a history that the CTAs share out
    const bool any = a.words && (length > 0 || c.bias_ids);
    // The CTAs of a cluster have all started when this is waited for, before the first write into another's memory (a
    // history that is shared out has cluster-wide barriers of its own first).
    if (!far) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    // Four tokens of a thread from n on: their logits, noise, and masks (bit e: token e is allowed)
    struct Batch {
        float x[4], g[4];
        uint32_t allowed;
    };
    auto load4 = [&](const float *p, int n, int end, float (&v)[4]) {
        if (VEC && n + 4 <= end) {
            const float4 f = __ldcs(reinterpret_cast<const float4 *>(p + n));
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = n + (VEC ? e : e * kThreadsC);
                v[e] = at < end ? __ldcs(p + at) : 0.0f;
            }
        }
    };
    auto load = [&](int n, int end, Batch &b) {
        load4(logits, n, end, b.x);
        if (noise) load4(noise, n, end, b.g);
        b.allowed = 15u;
        if (mask) {
            if (VEC) {
                if (n < end) b.allowed = (uint32_t)mask[n >> 5] >> (n & 31);  // whose four are of one word
            } else {
                b.allowed = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = n + e * kThreadsC;
                    if (at < end) b.allowed |= (((uint32_t)mask[at >> 5] >> (at & 31)) & 1u) << e;
                }
            }
        }
    };
    float top = -INFINITY;
    int top_n = INT_MAX;  // the thread's best score and token: none yet
    for (int base = 0; base < a.N; base += turn) {
        const int first = base + rank * slice, end = min(a.N, first + slice);
        constexpr int kTake = 4 * kThreadsC, kAhead = 2;  // tokens of the CTA at a time; as many times in flight
        const int mine = first + (VEC ? 4 : 1) * (int)threadIdx.x;
        Batch ahead[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load(mine + k * kTake, end, ahead[k]);
        if (any) {
            if (base > 0) {
                __syncthreads();
                clear(max(0, end - first));
            }
            __syncthreads();
            if (c.bias_ids) {
                for (int i = threadIdx.x; i < c.bias_width; i += kThreadsC) {
                    const int n = c.bias_ids[(size_t)r * c.bias_width + i];
                    if (n >= first && n < end) atomicMax(word_of + n - first, (uint32_t)(i + 1) << 20);
                }
                __syncthreads();
            }
            if (far) cluster.sync();  // every CTA's words are ready for the others
            const int from = far ? (int)((long long)length * rank / ctas) : 0;
            const int to = far ? (int)((long long)length * (rank + 1) / ctas) : length;
            constexpr int kTokens = 8;  // of a thread in flight
            for (int i0 = from + (int)threadIdx.x; i0 < to; i0 += kTokens * kThreadsC) {
                long long n[kTokens];
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const int i = i0 + k * kThreadsC;
                    n[k] = i >= to  ? -1
                           : WIDE ? static_cast<const long long *>(c.history)[said + i]
                                  : static_cast<const int *>(c.history)[said + i];
                }
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const bool in_prompt = i0 + k * kThreadsC < prompt;
                    uint32_t *w = nullptr;
                    if (!far) {
                        if (n[k] >= first && n[k] < end) w = word_of + (int)(n[k] - first);
                    } else if (n[k] >= base && n[k] < min(a.N, base + turn)) {
                        const int owner = (int)(n[k] - base) / slice;
                        w = cluster.map_shared_rank(word_of, owner) + ((int)(n[k] - base) - owner * slice);
                    }
                    if (w) {
                        if (in_prompt)
                            atomicOr(w, kPrompt);
                        else
                            atomicAdd(w, 1u);
                    }
                }
            }
            if (far)
                cluster.sync();
            else
                __syncthreads();
        }
        for (int n0 = mine; n0 - mine + first < end; n0 += kAhead * kTake) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int n = n0 + k * kTake;
                Batch now = ahead[k];
                load(n + kAhead * kTake, end, ahead[k]);
                if (n < end) {
                    float(&x)[4] = now.x;
                    if (any) {
                        uint32_t words[4];
                        if (VEC) {
                            const uint4 w4 = *reinterpret_cast<const uint4 *>(word_of + (n - first));  // slices of whole 128s
                            words[0] = w4.x, words[1] = w4.y, words[2] = w4.z, words[3] = w4.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                words[e] = n + e * kThreadsC < end ? word_of[n + e * kThreadsC - first] : 0u;
                        }
                        if (words[0] | words[1] | words[2] | words[3]) {  // (past the end what they hold goes nowhere)
#pragma unroll 1
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t w = e == 0 ? words[0] : e == 1 ? words[1] : e == 2 ? words[2] : words[3];
                                if (w) {
                                    const float v = ruled(e == 0 ? x[0] : e == 1 ? x[1] : e == 2 ? x[2] : x[3], w, row);
                                    if (e == 0) x[0] = v;
                                    if (e == 1) x[1] = v;
                                    if (e == 2) x[2] = v;
                                    if (e == 3) x[3] = v;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = n + (VEC ? e : e * kThreadsC);
                        if (hot) x[e] = over_temperature(x[e], row);
                        const bool allowed = (now.allowed >> e) & 1u;
                        if (!allowed) x[e] = -INFINITY;
                        const float score = noise ? __fadd_rn(x[e], now.g[e]) : x[e];
                        // larger, or NaN where there was none, or the first (tokens come in ascending order)
                        if (allowed && at < end && top == top && (!(score <= top) || top_n == INT_MAX)) top = score, top_n = at;
                    }
                    if (out) {
                        if (VEC && n + 4 <= end) {
                            __stcs(reinterpret_cast<float4 *>(out + n), make_float4(x[0], x[1], x[2], x[3]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = n + (VEC ? e : e * kThreadsC);
                                if (at < end) __stcs(out + at, x[e]);
                            }
                        }
                    }
                }
            }
        }
    }
    // the row's best: the highest score, of equal ones the lowest token; 0 for none
    unsigned long long key = top_n == INT_MAX ? 0ull : argmax_key(top, top_n);
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
        key = other > key ? other : key;
    }
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = key;
    __syncthreads();
    if (!far) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreadsC / 32; ++w) key = best[w] > key ? best[w] : key;
        cluster.map_shared_rank(of_rank, 0)[rank] = key;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        key = of_rank[0];
        for (int k = 1; k < ctas; ++k) key = of_rank[k] > key ? of_rank[k] : key;
        a.idx[r] = key ? (int64_t)(0xFFFFFFFFull - (key & 0xFFFFFFFFull)) : -1;
    }
}

template <bool VEC, bool WIDE> cudaError_t launch_choose(const ChooseArgs &a, int ctas, int m, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(choose_kernel<VEC, WIDE>, 4 * kMostSlice, &allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)m, 1);
    cfg.blockDim = dim3(kThreadsC, 1, 1);
    cfg.dynamicSmemBytes = a.words ? 4 * (size_t)a.slice : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, choose_kernel<VEC, WIDE>, a);
}

}  // namespace
}  // namespace q8

extern "C" q8_status q8_choose(const float *logits, int ldl, const q8_choice *rules, float *out, int ldo, int64_t *idx,
                               int m, int N, q8_stream_t stream) {
    using q8::kv_aligned;
    using q8::kv_overlap;
    if (!logits || !idx) return Q8_ERR_ARG;
    if (m < 1 || m > 65535 || N < 1 || N > (1 << 30) || ldl < N || (out && ldo < N)) return Q8_ERR_SHAPE;
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
    a.words = c.history || c.bias_ids;
    // Eight CTAs a row, fewer where a slice would be less than 2048 tokens (one turn of a CTA's threads).
    int ctas = 1;
    while (ctas < q8::kMostCtas && ctas * 2048 < N) ctas *= 2;
    const int slice = ((N + ctas - 1) / ctas + 127) / 128 * 128;
    a.slice = slice < q8::kMostSlice ? slice : q8::kMostSlice;
    auto quad = [](const void *p, int pitch) { return !p || (kv_aligned(p, 16) && pitch % 4 == 0); };
    const bool vec = quad(logits, ldl) && quad(out, ldo) && quad(c.noise, c.noise_pitch);
    const cudaStream_t cs = (cudaStream_t)stream;
    const cudaError_t e = vec ? (c.history_wide ? q8::launch_choose<true, true>(a, ctas, m, cs)
                                                : q8::launch_choose<true, false>(a, ctas, m, cs))
                              : (c.history_wide ? q8::launch_choose<false, true>(a, ctas, m, cs)
                                                : q8::launch_choose<false, false>(a, ctas, m, cs));
    return e == cudaSuccess ? Q8_OK : q8::kv_cuda_fail(e);
}
