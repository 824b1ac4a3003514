// The rules on logits and the token chosen (formulas in q8_gemv.h): one cluster of up to eight CTAs a row, one pass over the
// logits.
//
// 8 bytes a logit, 4 more with noise, bound a large step; what has to stay out of their way is the look-up of how often a
// token was said.  Each CTA owns a slice of the vocabulary and holds one word for each of its tokens in shared memory: how
// often it stands in the answer, whether it stands in the prompt, its place among the biases.  The words come from integer
// atomics, whose order does not matter.  A history of up to kLocal tokens is read whole by every CTA of the row, which keeps
// what falls into its slice and needs no word from the others; of a longer one each CTA reads its share and sends what it
// finds to the owner through distributed shared memory.  A vocabulary beyond eight slices of kMostSlice takes several turns.
// What else bounds it is instructions, 62% of the issue slots in a large step, and a CTA's beginning, when it makes its words and
// streams nothing.  Measured: 256 rows of 128256, histories of 2001, 300 biases, masks and noise 103.5 us (3.8 TB/s of the 6.8
// that a copy reaches), 16 rows with histories of 8191 21.1 us, one row of 32000 5.8 us.
// The first logits are asked for before the words are made.  Each step of a rule is one fp32 operation rounded once (no
// contraction), so that the bits are those of any other implementation.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include "q8_attn.h"
#include "q8_device.cuh"

namespace q8 {
namespace {

constexpr int kMostCtas = 8;
constexpr int kMostSlice = 49152;  // 192 KB of words
// The longest history that every CTA of a row reads whole.  Sharing it out costs two cluster-wide barriers and atomics in other
// SMs' memory.  Measured with 20 biases, masks and noise over 128256 tokens, read whole and shared out: one row with a history
// of 2000 10.7 and 12.0 us, of 8191 12.3 and 15.4, of 16000 14.0 and 18.6; 16 rows 20.5 and 23.7, 23.7 and 30.8, 27.2 and 37.1;
// 64 rows with 16000 45.4 and 65.1.  The two do not meet up to 32000 (16 rows 33.3 and 49.9): for lengths of 8193 to 32000 the
// other side of this border would be the faster one.
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

struct Divisor {  // of many quotients
    float by, inv, span;  // 1 / by; the quotients that need no division are of |v| in 1/span .. span (0: none)
};
__device__ __forceinline__ Divisor divisor(float by) {
    return {by, __frcp_rn(by), by >= 0x1p-20f && by <= 0x1p20f ? 0x1p80f : 0.0f};
}
// v / by, rounded once, where |v| is in the divisor's span.  With y the correctly rounded 1 / by, v y is within two units in
// the last place, one correction by its remainder makes it one of the two nearest, whose remainder v - q by is exact in one
// fma, and q + remainder * y is then the correctly rounded quotient (Markstein's theorem), as nothing over- or underflows.
// (Of a zero the remainder would lose the sign.)  A division of each logit took more instructions than everything else.
__device__ __forceinline__ float quotient(float v, const Divisor &d) {
    float q = v * d.inv;
    q = fmaf(fmaf(-q, d.by, v), d.inv, q);
    return fmaf(fmaf(-q, d.by, v), d.inv, q);
}
__device__ __forceinline__ bool in_span(float most, float least, const Divisor &d) {
    return most <= d.span && least * d.span >= 1.0f;
}

struct Row {  // a row's numbers
    Divisor rep, temp;
    float freq, pres;
    const float *bias;
};

// The rules of a word on a logit.
__device__ __forceinline__ float ruled(float v, uint32_t word, const Row &w) {
    if (word & (kPrompt | kCount)) {
        if (v > 0.0f)
            v = in_span(v, v, w.rep) ? quotient(v, w.rep) : __fdiv_rn(v, w.rep.by);
        else
            v = __fmul_rn(v, w.rep.by);
    }
    if (word & kCount) {
        v = __fsub_rn(v, __fmul_rn(w.freq, (float)(word & kCount)));
        v = __fsub_rn(v, w.pres);
    }
    const uint32_t place = (word & ~kPrompt) >> 20;
    if (place) v = __fadd_rn(v, w.bias[place - 1]);
    return v;
}

// Four logits over the row's temperature.
__device__ __forceinline__ void over_temperature(float (&x)[4], const Divisor &t) {
    float q[4], most = 0.0f, least = INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q[e] = quotient(x[e], t);
        most = fmaxf(most, fabsf(x[e]));
        least = fminf(least, fabsf(x[e]));
        sum += q[e];  // of a NaN among them the others do not tell
    }
    if (in_span(most, least, t) && sum == sum) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = q[e];
    } else {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
            const float v = __fdiv_rn(x[0], t.by);  // the next in turn
            x[0] = x[1], x[1] = x[2], x[2] = x[3], x[3] = v;
        }
    }
}

// VEC: rows of logits, output and noise are 16-byte aligned, a thread takes four tokens in a row; else four that are T
// apart.  T threads: 1024 where every CTA has an SM of its own, else 512, two an SM, of which one streams while the other
// gathers its words.
template <bool VEC, bool WIDE, int T>
__global__ void __launch_bounds__(T, 1024 / T) choose_kernel(const __grid_constant__ ChooseArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) uint32_t word_of[];
    __shared__ unsigned long long best[T / 32], of_rank[kMostCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const q8_choice &c = a.c;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x, r = (int)blockIdx.y, slice = a.slice;
    const int turn = ctas * slice;  // tokens of a turn
    auto clear = [&](int count) {
        for (int i = threadIdx.x; i < (count + 3) / 4; i += T)
            reinterpret_cast<uint4 *>(word_of)[i] = make_uint4(0u, 0u, 0u, 0u);
    };
    if (a.words) clear(min(slice, max(0, a.N - rank * slice)));
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // What needs no other load first is asked for at once: a bias, the first tokens (those past the row's length are dropped
    // when that is known).
    constexpr int kTokens = 4;  // of a thread in flight
    const size_t said = (size_t)r * c.history_pitch;
    auto tokens = [&](int i0, int to, int (&n)[kTokens]) {  // -1 for none and for what is no token
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int i = i0 + k * T;
            n[k] = -1;
            if (i < to) {
                if (WIDE) {
                    const long long t = static_cast<const long long *>(c.history)[said + i];
                    n[k] = t >= 0 && t < a.N ? (int)t : -1;
                } else {
                    n[k] = static_cast<const int *>(c.history)[said + i];
                }
            }
        }
    };
    int early[kTokens];
    tokens((int)threadIdx.x, c.history ? c.history_width : 0, early);
    const int *bias_ids = c.bias_ids ? c.bias_ids + (size_t)r * c.bias_width : nullptr;
    const int first_bias = bias_ids && (int)threadIdx.x < c.bias_width ? bias_ids[threadIdx.x] : -1;
    Row row;
    row.rep = divisor(c.repetition ? c.repetition[r] : 1.0f);
    row.temp = divisor(c.temperature ? c.temperature[r] : 0.0f);
    row.freq = c.frequency ? c.frequency[r] : 0.0f;
    row.pres = c.presence ? c.presence[r] : 0.0f;
    const bool hot = row.temp.by > 0.0f;
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
    const bool far = length > kLocal && ctas > 1;  // a history that the CTAs share out
    const bool any = a.words && (length > 0 || c.bias_ids);
    const int from = far ? (int)((long long)length * rank / ctas) : 0;
    const int to = far ? (int)((long long)length * (rank + 1) / ctas) : length;
    // The CTAs of a cluster have all started when this is waited for, before the first write into another's memory (a
    // history that is shared out has cluster-wide barriers of its own first).
    if (!far) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    // Four tokens of a thread from n on: their logits, noise, and masks' words (of four in a row the same)
    struct Batch {
        float x[4], g[4];
        int mask[VEC ? 1 : 4];
    };
    auto load4 = [&](const float *p, int n, int end, float (&v)[4]) {
        if (VEC && n + 4 <= end) {
            const float4 f = __ldcs(reinterpret_cast<const float4 *>(p + n));
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = n + (VEC ? e : e * T);
                v[e] = at < end ? __ldcs(p + at) : 0.0f;
            }
        }
    };
    auto load = [&](int n, int end, Batch &b) {
        load4(logits, n, end, b.x);
        if (noise) load4(noise, n, end, b.g);
#pragma unroll
        for (int e = 0; e < (VEC ? 1 : 4); ++e) {
            const int at = n + e * T;
            b.mask[e] = mask && at < end ? mask[at >> 5] : -1;
        }
    };
    // The thread's best score above -inf and its token, its first token whose score is NaN: none yet
    float top = -INFINITY;
    int top_n = INT_MAX, nan_n = INT_MAX;
    for (int base = 0; base < a.N; base += turn) {
        const int first = base + rank * slice, end = min(a.N, first + slice);
        constexpr int kTake = 4 * T, kAhead = 2;  // tokens of the CTA at a time; as many times in flight
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
                for (int i = threadIdx.x; i < c.bias_width; i += T) {
                    const int n = i < T ? first_bias : bias_ids[i];
                    if (n >= first && n < end) atomicMax(word_of + n - first, (uint32_t)(i + 1) << 20);
                }
                __syncthreads();
            }
            if (far) cluster.sync();  // every CTA's words are ready for the others
            int next[kTokens];
#pragma unroll
            for (int k = 0; k < kTokens; ++k) next[k] = (int)threadIdx.x + k * T < to ? early[k] : -1;
            if (far) tokens(from + (int)threadIdx.x, to, next);
            for (int i0 = from + (int)threadIdx.x; i0 < to; i0 += kTokens * T) {
                int n[kTokens];
#pragma unroll
                for (int k = 0; k < kTokens; ++k) n[k] = next[k];
                tokens(i0 + kTokens * T, to, next);
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const bool in_prompt = i0 + k * T < prompt;
                    if (far) {
                        if (n[k] >= base && n[k] < min(a.N, base + turn)) {
                            const int owner = (n[k] - base) / slice;
                            uint32_t *w = cluster.map_shared_rank(word_of, owner) + (n[k] - base - owner * slice);
                            if (in_prompt)
                                atomicOr(w, kPrompt);
                            else
                                atomicAdd(w, 1u);
                        }
                    } else if (n[k] >= first && n[k] < end) {
                        if (in_prompt)
                            atomicOr(word_of + n[k] - first, kPrompt);
                        else
                            atomicAdd(word_of + n[k] - first, 1u);
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
                                words[e] = n + e * T < end ? word_of[n + e * T - first] : 0u;
                        }
                        if (words[0] | words[1] | words[2] | words[3]) {  // (past the end they are zeros)
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = ruled(x[e], words[e], row);
                        }
                    }
                    if (hot) over_temperature(x, row.temp);
                    uint32_t seen = 0u;  // bit e: token e is there and allowed
                    if (VEC) {
                        seen = (uint32_t)now.mask[0] >> (n & 31);
                        if (n + 4 > end) seen &= (1u << (end - n)) - 1u;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = n + e * T;
                            seen |= (at < end ? (uint32_t)now.mask[VEC ? 0 : e] >> (at & 31) & 1u : 0u) << e;
                        }
                    }
                    float score[4], sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (!(seen >> e & 1u)) x[e] = -INFINITY;
                        score[e] = noise ? __fadd_rn(x[e], now.g[e]) : x[e];
                        sum += score[e];
                    }
                    if (sum == sum) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // tokens come in ascending order
                            if (score[e] > top) top = score[e], top_n = n + (VEC ? e : e * T);
                    } else {  // a NaN (or infinities of both signs)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = n + (VEC ? e : e * T);
                            if (seen >> e & 1u) {
                                if (score[e] > top) top = score[e], top_n = at;
                                if (score[e] != score[e] && nan_n == INT_MAX) nan_n = at;
                            }
                        }
                    }
                    if (out) {
                        if (VEC && n + 4 <= end) {
                            __stcs(reinterpret_cast<float4 *>(out + n), make_float4(x[0], x[1], x[2], x[3]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int at = n + (VEC ? e : e * T);
                                if (at < end) __stcs(out + at, x[e]);
                            }
                        }
                    }
                }
            }
        }
    }
    // the row's best: the highest score, of equal ones the lowest token; 0 for none
    unsigned long long key = nan_n != INT_MAX ? argmax_key(NAN, nan_n) : top_n != INT_MAX ? argmax_key(top, top_n) : 0ull;
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
        key = other > key ? other : key;
    }
    if ((threadIdx.x & 31) == 0) best[threadIdx.x >> 5] = key;
    __syncthreads();
    if (!far) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int w = 1; w < T / 32; ++w) key = best[w] > key ? best[w] : key;
        cluster.map_shared_rank(of_rank, 0)[rank] = key;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // The others leave once they have told the first CTA (nobody reads their memory any more).
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    key = of_rank[0];
    for (int k = 1; k < ctas; ++k) key = of_rank[k] > key ? of_rank[k] : key;
    if (key == 0ull) {  // nothing above -inf: the first token that is allowed, if any is
        __shared__ int lowest;
        if (threadIdx.x == 0) lowest = mask ? INT_MAX : 0;
        __syncthreads();
        for (int i = threadIdx.x; mask && i <= (a.N - 1) >> 5; i += T) {
            const uint32_t bits = (uint32_t)mask[i] & (32 * i + 32 > a.N ? (1u << (a.N & 31)) - 1u : ~0u);
            if (bits) {
                atomicMin(&lowest, 32 * i + __ffs((int)bits) - 1);
                break;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) a.idx[r] = lowest == INT_MAX ? -1 : lowest;
    } else if (threadIdx.x == 0) {
        a.idx[r] = (int64_t)(0xFFFFFFFFull - (key & 0xFFFFFFFFull));
    }
}

constexpr int choose_smem(int slice) { return 4 * slice; }

template <bool VEC, bool WIDE, int T>
cudaError_t launch_kernel(const ChooseArgs &a, int ctas, int m, int smem, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = kv_allow_smem(choose_kernel<VEC, WIDE, T>, choose_smem(kMostSlice), &allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)m, 1);
    cfg.blockDim = dim3(T, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
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
    return cudaLaunchKernelEx(&cfg, choose_kernel<VEC, WIDE, T>, a);
}

template <bool VEC, bool WIDE> cudaError_t launch_choose(const ChooseArgs &a, int ctas, int m, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = sm_count_of_device(&sms);
    if (e != cudaSuccess) return e;
    const int words = a.words ? choose_smem(a.slice) : 0;
    // Where every CTA can have an SM of its own: a cluster's CTAs are put together on as few SMs as hold them, which these
    // threads do not fit twice.
    if ((long long)ctas * m <= sms) return launch_kernel<VEC, WIDE, 1024>(a, ctas, m, words, stream);
    return launch_kernel<VEC, WIDE, 512>(a, ctas, m, words, stream);
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
    if ((c.history && !c.lengths) || (!c.bias_ids != !c.bias) || (c.mask_rows && !c.mask)) return Q8_ERR_ARG;
    if (c.history && (c.history_width < 1 || c.history_width > Q8_MAX_HISTORY || c.history_pitch < c.history_width))
        return Q8_ERR_SHAPE;
    if (c.bias_ids && (c.bias_width < 1 || c.bias_width > Q8_MAX_BIAS)) return Q8_ERR_SHAPE;
    if (c.mask && (c.mask_count < (c.mask_rows ? 1 : m) || c.mask_pitch < (N - 1) / 32 + 1)) return Q8_ERR_SHAPE;
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
    // Eight CTAs a row, fewer for vocabularies of up to 8192 tokens: doubled while a CTA would have more than 2048, so that
    // slices are of more than 1024 (half a step of 512 threads, four tokens each).
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
