/*
 * q8_gemv.h -- C ABI of the GB300 Q8_0 block-quantized GEMV library (libq8gemv.so).
 *
 * The product (source: "logicaffeine_compile/spatial/passes/from_q8.rs", module doc):
 *
 *     y[r, n] = sum_b s[b, n] * sum_{i<32} x[r, 32b + i] * q[32b + i, n]        r < m, n < N
 *
 * over a weight stored Q8_0: int8 values q (`W__q8`, K x N) and one fp32 scale per 32-row block of each column
 * (`W__q8_scale`, K/32 x N), about 1.125 bytes a weight against 2 for bf16.  Activations x are bf16, accumulation is
 * fp32, and a batch of m <= 16 rows reads the weight once for all its rows.
 *
 * Layouts (all row-major, no strides):
 *   x  bf16    [m][K]        row pitch K elements
 *   q  int8    [K][Np]       row pitch Np bytes; Np = q8_padded_n(N) = N rounded up to a multiple of 32
 *   s  fp32    [K/32][Np]    row pitch Np elements
 *   y  fp32    [m][Np]       row pitch Np elements
 * Columns N .. Np-1 are the zero-padded last 32-column tile ("from_q8.rs", `q8_gemv_applies`): their q and s should
 * be 0 (q8_repack and q8_quantize write them so); the GEMV writes exactly 0.0f into y's pad columns regardless.
 *
 * Conventions shared by every entry point:
 *   - The caller owns every buffer and the library allocates no memory.  Its only state is read-only caches (per
 *     device: SM count, resident clusters, which kernels may use their shared memory; the address of the driver's
 *     tensor-map encoder), the device fault words (q8_device_fault), the planner overrides of
 *     q8_set_tuning, the residual norm's 64 static completion counters (used only by its one-launch fold; see
 *     q8_gemv_residual_norm for the limit this puts on overlapping calls) and the 32 static counters of
 *     q8_gemv_residual_norm_noalloc (see there).
 *   - Device entry points take device pointers and enqueue work on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream).  They are asynchronous: Q8_OK means the work was enqueued.  An argument error is returned
 *     before anything is enqueued.  A CUDA error at launch returns Q8_ERR_CUDA; q8_last_cuda_error() then gives the
 *     cudaError_t value for the calling thread.
 *   - Host entry points take host pointers and run synchronously on the calling thread.
 *   - No entry point aborts, throws or prints.
 *   - Every call is thread-safe; calls on one stream run in order.  The exception is the residual norm's one-launch
 *     fold (q8_set_tuning Q8_TUNE_NORM_FOLD = 1): at most 64 of its row groups may be in flight at once over all
 *     streams and threads.
 */
#ifndef Q8_GEMV_H
#define Q8_GEMV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ABI-identical to cudaStream_t; declared here so that the header needs no CUDA headers. */
struct CUstream_st;
typedef struct CUstream_st *q8_stream_t;

/* Rows of a Q8_0 block ("from_q8.rs", `Q8_BLOCK`). */
#define Q8_BLOCK 32
/* The most activation rows one call takes ("plan.rs", `GEMV_ROWS`: a GEMV launch multiplies at most 16 rows). */
#define Q8_MAX_ROWS 16

/* The most activation rows one call over the tiled storage takes ("plan.rs", `MAX_CHUNK`: the largest prefill chunk
 * a lane compiles, 512; its projections of more rows than the GEMV's 16 run on the tensor cores).  With
 * Q8_FLAG_TILED, m may be 1 .. 512: from 128 rows a plain product of bf16 activations runs as a tensor-core GEMM
 * (tcgen05, 128 x 128 output tiles, each 32-row block contracted exactly and folded with its scales); otherwise the
 * rows run as ceil(m / 16) groups of 16 in one launch, each group's CTAs of a column tile side by side so that the
 * weight is streamed from HBM about once. */
#define Q8_MAX_CHUNK 512

typedef enum {
    Q8_OK = 0,
    Q8_ERR_ARG = 1,      /* a required pointer is NULL, or an enum argument is out of range */
    Q8_ERR_SHAPE = 2,    /* m outside 1..16, K <= 0, K % 32 != 0, N <= 0, or a size that overflows */
    Q8_ERR_ALIGN = 3,    /* a device pointer is not 16-byte aligned */
    Q8_ERR_NOT_Q8_0 = 4, /* a weight or block that is not Q8_0 (see q8_quantize, q8_repack) */
    Q8_ERR_CUDA = 5      /* the CUDA runtime reported an error; see q8_last_cuda_error() */
} q8_status;

/* Kernel family selector for q8_gemv_ex (benchmarking and testing).  AUTO, what q8_gemv takes, runs the streaming
 * kernels: each warp copies its 32-row x 128-column blocks of the row-major weight into a shared-memory ring with
 * cp.async and reads them back transposed (ldmatrix .trans .b8) in the tiled storage's word order, so the row-major
 * weight streams through the same kernels as the tiled one.  The others are earlier designs kept for comparison. */
typedef enum {
    Q8_VARIANT_AUTO = 0,
    Q8_VARIANT_SIMT = 1, /* CUDA-core fp32 FMA, m-row accumulators per thread, weights loaded straight to registers */
    Q8_VARIANT_MMA = 2,  /* int8 -> bf16 exact dequant in registers, bf16 tensor-core MMA, fp32 per-block scale fold */
    Q8_VARIANT_TMA = 3   /* as MMA, the weight streamed by TMA through a 16-stage shared-memory pipeline by a producer
                            warp; launched with programmatic dependent launch.  Needs N > 96 (Np >= 128); smaller N
                            falls back to MMA. */
} q8_variant;

/* N rounded up to whole 32-column tiles ("from_q8.rs", `q8_gemv_applies`: the last tile is zero-padded).
 * Returns -1 when N <= 0 or the result would overflow an int. */
int q8_padded_n(int N);

/* y = x . W over the Q8_0 weight (q, s), m rows (source: "from_q8.rs", module doc and `q8_fold`).
 *   x  device, bf16 [m][K], 16-byte aligned        q  device, int8 [K][Np], 16-byte aligned
 *   s  device, fp32 [K/32][Np], 16-byte aligned    y  device, fp32 [m][Np] (written), 16-byte aligned
 *   1 <= m <= 16 (1 <= m <= 512 over the tiled storage, Q8_MAX_CHUNK), K > 0, K % 32 == 0 ("from_q8.rs",
 *   `q8_gemv_applies`), N > 0.
 * y must not overlap x, q or s.  Every output n < Np is written; outputs n >= N are 0.0f.
 * Each y[r, n] equals the real-number product within 1e-5 * sum_b |s[b,n]| sum_i |x[r,32b+i] q[32b+i,n]| for K up to
 * 14336 (equal terms of 512 rows, whose roundings do not cancel, reach 6.7e-6 there), and beyond within
 * (K / 32 + 64) * 2^-24 of that sum: the fp32 carry is rounded once a block (equal terms reach 1.3e-5 at K = 28672); the
 * summation order is fixed for a given (m, K, N) and device, so repeated calls give identical bits. */
q8_status q8_gemv(const void *x, const int8_t *q, const float *s, float *y, int m, int K, int N, q8_stream_t stream);

/* Flags of q8_gemv_ex. */
#define Q8_FLAG_CONSTANT_WEIGHTS 1u /* no work enqueued before this call on `stream` writes q or s, other than
                                       q8_tile_device (which ends with a launch that orders what follows): the pipelined
                                       kernel may start streaming them before the previous kernel on the stream has
                                       finished (programmatic dependent launch); x and y are still ordered */

#define Q8_FLAG_TILED 2u            /* q and s are in the tiled layout of q8_tile (below), not row-major; read by the
                                       per-warp cp.async streaming kernel (variant must be AUTO) */

#define Q8_FLAG_Q8_ACT 4u           /* x is the quantized form of the activation written by q8_quantize_act (below),
                                       not bf16 values, and the product is the quantized numerics'
                                           y[r, n] = sum_b s[b, n] * d[r, b] * sum_i xq[r, 32b+i] * q[32b+i, n]
                                       (its integer inner sums exact); requires Q8_FLAG_TILED.  Every product entry
                                       point takes it; the bound is as before with xq * d in place of x */

/* q8_gemv with an explicit kernel family (q8_variant) and flags (Q8_FLAG_*; 0 for none).  Same arguments and
 * bound; Q8_ERR_ARG for an unknown variant or flag, for Q8_FLAG_TILED with a variant other than AUTO, or for
 * Q8_FLAG_Q8_ACT without Q8_FLAG_TILED. */
q8_status q8_gemv_ex(const void *x, const int8_t *q, const float *s, float *y, int m, int K, int N, int variant,
                     unsigned int flags, q8_stream_t stream);

/* The product followed by the arg-max that ends a decode step (source: "plan.rs", `Launch::ArgMax`, and
 * "int8_model.rs", `decode_step_lg`: the lowest index among the largest logits; its CUDA arg-max sends equal values to
 * the lower index).
 *   idx     device, int64 [m] (written), 8-byte aligned: idx[r] = the smallest n < N with y[r, n] equal to the
 *           largest y[r, n'] over n' < N, 0-based.  Pad columns never take part.  +0.0 and -0.0 count as equal.
 *           The buffer also serves as the call's cross-block scratch: its contents before the call do not matter.
 *   logits  device, fp32 [m][Np] (written, as q8_gemv's y) or NULL to skip storing the logits.
 * Other arguments as q8_gemv.  Logits that are NaN order above +inf (not reached for finite inputs). */
q8_status q8_gemv_argmax(const void *x, const int8_t *q, const float *s, int64_t *idx, float *logits, int m, int K,
                         int N, q8_stream_t stream);

/* q8_gemv_argmax with flags (Q8_FLAG_CONSTANT_WEIGHTS, Q8_FLAG_TILED). */
q8_status q8_gemv_argmax_ex(const void *x, const int8_t *q, const float *s, int64_t *idx, float *logits, int m,
                            int K, int N, unsigned int flags, q8_stream_t stream);

/* The tiled storage of a Q8_0 weight, for Q8_FLAG_TILED (no counterpart on the pages: a GPU storage order of the
 * same two tensors, made once when the weight is loaded, as the host repack of "from_q8.rs" `Q8Part` is).  Every
 * 32-row x 128-column block becomes one contiguous 4 KB unit laid out in the order the kernel's lanes load it, so a
 * warp streaming one column tile along K reads contiguous memory.  With Nt = q8_tiled_n(N), T = Nt / 128 tiles and
 * nb = K / 32 blocks:
 *   values  uint8 [T][nb][4096]: in unit (t, b), segment 4s + h (s = 0, 1; h = 0..3; 512 bytes each) holds at byte
 *           16 * (4g + u) (g = 0..7, u = 0..3) four words; word w holds weight rows 32b + 16s + 4u + k (byte k,
 *           k = 0..3) of column 128t + 8(4h + w) + g, each value stored as q + 128 (offset binary)
 *   scales  fp32 [T][nb][128]: element c of unit (t, b) is s[b][128t + c]
 * Columns >= N hold q = 0 (byte 128) and scale 0.  Sizes: K * Nt bytes of values, (K / 32) * Nt * 4 bytes of
 * scales. */
int q8_tiled_n(int N); /* N rounded up to a multiple of 128; -1 when N <= 0 or on overflow */

/* Host: row-major q [K][Np], s [K/32][Np] (as q8_gemv takes them) -> tiled qt, st (host buffers, written). */
q8_status q8_tile(const int8_t *q, const float *s, int K, int N, int8_t *qt, float *st);

/* Device: the same transform on device buffers, enqueued on `stream` (q, qt 16-byte aligned; s, st 4-byte aligned;
 * the input and output must not overlap). */
q8_status q8_tile_device(const int8_t *q, const float *s, int K, int N, int8_t *qt, float *st, q8_stream_t stream);

/* The gated pair ("plan.rs", `Launch::GemvGlu`: two projections of one activation through a gate,
 * out = act(x.wg + bg) * (x.wu + bu), silu gating (SwiGLU) by default; here without biases):
 *     out[r, n] = silu(g[r, n]) * u[r, n],   g = x . Wg,  u = x . Wu,   silu(g) = g / (1 + exp(-g)),
 * g and u each the Q8_0 product of q8_gemv (fp32 accumulation), silu and the product in fp32 (CUDA's expf, IEEE
 * division).  One launch (two when the planner splits it, Q8_TUNE_SPLIT, q8_plan_glu_launches): the gate's and the
 * up projection's CTAs of a column tile run side by side in a cluster.
 *   x         device, bf16 [m][K], 16-byte aligned
 *   qg, sg    device, the gate's weight in the tiled storage (q8_tile), 16-byte aligned
 *   qu, su    device, the up projection's weight, tiled, 16-byte aligned
 *   out       device, fp32 [m][Np] (written; pad columns 0), 16-byte aligned, or NULL
 *   out_bf16  device, bf16 [m][Np] (written: out rounded to nearest even; pads 0), 16-byte aligned, or NULL
 *             -- a down projection's activation as q8_gemv takes it (row pitch Np)
 *   flags     Q8_FLAG_TILED (required) | Q8_FLAG_CONSTANT_WEIGHTS
 * Errors: Q8_ERR_ARG (null inputs, both outputs null, flags without Q8_FLAG_TILED or with unknown bits, an output
 * overlapping an input or the other output), Q8_ERR_SHAPE, Q8_ERR_ALIGN, Q8_ERR_CUDA; nothing is launched on an
 * error.  inf and NaN propagate as IEEE arithmetic does (silu(-inf) = -inf / inf = NaN). */
q8_status q8_gemv_glu(const void *x, const int8_t *qg, const float *sg, const int8_t *qu, const float *su, float *out,
                      void *out_bf16, int m, int K, int N, unsigned int flags, q8_stream_t stream);

/* q8_gemv_glu with a third, optional output: out_q8 (device, q8_act_bytes(m, Np) bytes, 16-byte aligned, or NULL)
 * receives the quantized form of the bf16 output -- exactly what q8_quantize_act of out_bf16 (as [m][Np]) writes --
 * from the same launch ("plan.rs": an op may emit fp32, the quantized form, or the two together; `GluActMulQuant`),
 * ready for a Q8_FLAG_Q8_ACT product with K = Np.  At least one of out, out_bf16, out_q8; no two may overlap. */
q8_status q8_gemv_glu_ex(const void *x, const int8_t *qg, const float *sg, const int8_t *qu, const float *su,
                         float *out, void *out_bf16, void *out_q8, int m, int K, int N, unsigned int flags,
                         q8_stream_t stream);

/* A projection followed by the residual add and the following RMS norm ("plan.rs", `Launch::Fold` of a projection
 * with `Launch::Norm`, `gemv_norm_epilogue`: each block of the projection registers on a counter when done, and the
 * block that registers last fetches every result again from L2 and normalises; the norm launch is the lane's
 * "rmsnorm"):
 *     y = x . W (the Q8_0 product of q8_gemv),   h = residual + y,
 *     out[r, n] = h[r, n] / sqrt(mean_{n' < N} h[r, n']^2 + eps) * gamma[n]
 * Every CTA of the product writes its columns of h.  A second launch on the same stream, chained by programmatic
 * dependent launch (it waits for all of h), then runs the norm with one CTA per row: the row's mean square in a fixed
 * order, then out.  The one-launch fold of the source, where the product's last CTA to finish (a completion counter
 * from a fixed set of 64 in static device memory: the library allocates nothing) reads the rows of h back and runs
 * the norm, is kept for comparison (q8_set_tuning Q8_TUNE_NORM_FOLD = 1); measured on GB300 it is slower at every m.
 * Either way the result depends only on the inputs, never on which CTA finishes last.
 *   x, q, s   as q8_gemv, the weight in the tiled storage (q8_tile)
 *   residual  device, fp32 [m][Np], 4-byte aligned (read)
 *   gamma     device, fp32 [N] (at least N values), 4-byte aligned
 *   eps       >= 0 and finite
 *   h         device, fp32 [m][Np] (written: residual + y, pads 0), 16-byte aligned; may be residual itself
 *   out_bf16  device, bf16 [m][Np] (written: out rounded to nearest even, pads 0), 16-byte aligned -- the next
 *             projection's activation as q8_gemv takes it (row pitch Np)
 *   flags     Q8_FLAG_TILED (required) | Q8_FLAG_CONSTANT_WEIGHTS
 * Under the one-launch fold each group of 16 rows takes the next of 64 static completion counters in turn (a counter
 * is back to 0 when its launch ends), so at most 64 row groups may be in flight at once.
 * Errors: Q8_ERR_ARG (null pointers, flags without Q8_FLAG_TILED or unknown bits, eps < 0 or not finite, outputs
 * overlapping an input or each other other than h == residual), Q8_ERR_SHAPE, Q8_ERR_ALIGN, Q8_ERR_CUDA; nothing is
 * launched on an argument error (a Q8_ERR_CUDA from the norm's own launch leaves h written and out unspecified). */
q8_status q8_gemv_residual_norm(const void *x, const int8_t *q, const float *s, const float *residual,
                                const float *gamma, float eps, float *h, void *out_bf16, int m, int K, int N,
                                unsigned int flags, q8_stream_t stream);

/* q8_gemv_residual_norm with the normed output as bf16 (out_bf16) and/or its quantized form (out_q8, q8_act_bytes(m,
 * Np) bytes, 16-byte aligned: what q8_quantize_act of the bf16 rows writes; "plan.rs" `AddNormQuant`); at least one of
 * them, neither overlapping an input, h or the other. */
q8_status q8_gemv_residual_norm_ex(const void *x, const int8_t *q, const float *s, const float *residual,
                                   const float *gamma, float eps, float *h, void *out_bf16, void *out_q8, int m,
                                   int K, int N, unsigned int flags, q8_stream_t stream);

/* The rows one q8_gemv_residual_norm_noalloc call takes at most: its static scratch holds one completion counter per
 * group of 16 rows. */
#define Q8_FOLD_STATIC_MAX_ROWS 512

/* q8_gemv_residual_norm as one kernel launch that needs no device memory beyond its arguments and allocates none.
 * No counterpart on the pages: it serves callers that cannot call cudaMalloc or take memory from an allocator --
 * code running where device allocation is forbidden or would stall the pipeline (a real-time loop, a host
 * framework that owns all device memory and gives its plugins none, a step that must not synchronise the device).
 * It runs the source's one-launch fold (the product's last CTA per group of 16 rows reads h back and normalises),
 * whose completion counters live in a fixed array of this library (Q8_FOLD_STATIC_MAX_ROWS / 16 = 32 counters,
 * 128 bytes held by every GPU that loads the library until the process exits).
 *   Arguments, layouts, the result and its bound as q8_gemv_residual_norm (tiled storage; Q8_FLAG_TILED required,
 *   Q8_FLAG_CONSTANT_WEIGHTS and Q8_FLAG_Q8_ACT accepted), with 1 <= m <= Q8_FOLD_STATIC_MAX_ROWS.
 *   The call enqueues a memset that clears the counters it uses, then the product.
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress) with that device current;
 * make that first call before any stream capture on the device.  Every call shares the one array: calls whose work
 * overlaps on a GPU (other streams, other threads) race on the counters and give wrong results; calls on one stream
 * are ordered and safe.
 * Errors: Q8_ERR_SHAPE for m > Q8_FOLD_STATIC_MAX_ROWS (and as q8_gemv_residual_norm); Q8_ERR_ARG, Q8_ERR_ALIGN,
 * Q8_ERR_CUDA as q8_gemv_residual_norm.  Nothing is enqueued on an argument error. */
q8_status q8_gemv_residual_norm_noalloc(const void *x, const int8_t *q, const float *s, const float *residual,
                                        const float *gamma, float eps, float *h, void *out_bf16, int m, int K, int N,
                                        unsigned int flags, q8_stream_t stream);

/* One weight of a multi-projection call: its Q8_0 values and scales (row-major, or tiled with Q8_FLAG_TILED), its
 * output y [m][q8_padded_n(N)] (written) and its N. */
typedef struct q8_part {
    const int8_t *q;
    const float *s;
    float *y;
    int N;
} q8_part;

#define Q8_MAX_PARTS 8

/* Several Q8_0 products of one activation: y_p = x . W_p for every part p (source: "plan.rs", `Launch::GemmParts`:
 * the projections that share an activation -- q/k/v, or gate/up -- run together, their outputs placed next to each
 * other).
 *   x      device bf16 [m][K], read once for all parts       parts  host array of nparts q8_part (read during the call)
 *   1 <= nparts <= Q8_MAX_PARTS; every part has the same K; N may differ.  Each y_p is as q8_gemv writes it.
 * The parts run as one kernel launch (two when the planner splits it, Q8_TUNE_SPLIT, q8_plan_launches), row-major
 * or (Q8_FLAG_TILED) in the q8_tile layout.  Flags and errors as
 * q8_gemv_ex; an output overlapping x, a weight or another output is Q8_ERR_ARG. */
q8_status q8_gemv_parts(const void *x, const q8_part *parts, int nparts, int m, int K, unsigned int flags,
                        q8_stream_t stream);

/* How many product kernels a q8_gemv_ex (Q8_VARIANT_AUTO), q8_gemv_argmax_ex or q8_gemv_parts call of these sizes
 * launches on the calling thread's current device under the current tuning: 1, or 2 when the planner splits it
 * (Q8_TUNE_SPLIT; plain products of at most 16 rows whose column tiles do not fill the SMs evenly).  The arg-max's
 * memset and index decode are not counted.  No counterpart on the pages: for callers that account for the kernels of
 * a captured graph, and for tests.
 *   Ns  host array of the nparts output widths N (one for q8_gemv_ex and q8_gemv_argmax_ex); 1 <= nparts <= 8
 * Returns the count, or a negative status: -Q8_ERR_ARG (null Ns, nparts out of range, unknown flags), -Q8_ERR_SHAPE
 * (sizes the call would reject), -Q8_ERR_CUDA (the device cannot be queried). */
int q8_plan_launches(int m, int K, const int *Ns, int nparts, unsigned int flags);

/* q8_plan_launches for a q8_gemv_glu(_ex) call of these sizes (flags as that call takes them, Q8_FLAG_TILED among
 * them): 1, or 2 when the planner splits the gated pair in two.  Returns the count or a negative status as
 * q8_plan_launches. */
int q8_plan_glu_launches(int m, int K, int N, unsigned int flags);

/* The quantized form of an activation (source: "plan.rs", `QBLOCK`: 32 consecutive values of the form share one
 * scale; `Buffer::quantized`: int8 codes plus one scale for every 32; `Launch::projected_input`: a product over
 * checkpoint rows takes its activation in this form unless the numerics are the exact ones).  One buffer of
 * q8_act_bytes(m, K) bytes:
 *   values  int8 [m][K]      at byte 0
 *   scales  fp32 [m][K/32]   at byte m * K (16-byte aligned when the buffer is, since K % 32 == 0)
 * The pages fix the form but not its rounding; the rule here is the weight rule of "from_q8.rs" `quantize`
 * (d = amax / 127, q = round(x / d)) in fp32: for each row and block of 32 values, amax = max |x|,
 * d = amax / 127 and q = x / d rounded half away from zero, both quotients IEEE fp32 (round to nearest even,
 * subnormals kept), q clamped to [-127, 127] (a guard: for bf16 input |x / d| <= 127 * (1 + 2^-10)).  A block of
 * zeros gets d = 0 and q = 0; a block holding inf or NaN gets d = NaN and q = 0, so every product over it is NaN. */
int64_t q8_act_bytes(int m, int K); /* m * K + m * (K / 32) * 4; -1 when m < 1, K <= 0 or K % 32 != 0 */

/* Device: quantize x into xa, enqueued on `stream` (asynchronous; errors as q8_gemv).
 *   x   device, bf16 [m][K] row-major, 16-byte aligned
 *   xa  device, q8_act_bytes(m, K) bytes (written), 16-byte aligned, not overlapping x
 * Any m >= 1 (not limited to 16). */
q8_status q8_quantize_act(const void *x, void *xa, int m, int K, q8_stream_t stream);

/* Host repack of checkpoint blocks into the two stored tensors (source: "from_q8.rs", `Q8Part`: the host repacks the
 * checkpoint's blocks into the int8 values `q8_0.values` and the fp32 scales `q8_0.scales`).
 *   blocks  host, N * (K/32) blocks of 36 bytes, column-major by block: column n's blocks b = 0 .. K/32-1 in order;
 *           each block is a little-endian fp32 scale d followed by 32 int8 values (rows 32b .. 32b+31).
 *   q       host, int8 [K][Np] (written, pad columns 0)     s  host, fp32 [K/32][Np] (written, pad columns 0)
 * Returns Q8_ERR_NOT_Q8_0 when a value is -128 (outside the Q8_0 range |q| <= 127) or a scale is not finite; q and s
 * are then left partly written. */
q8_status q8_repack(const void *blocks, int K, int N, int8_t *q, float *s);

/* q8_repack for GGML-style checkpoint blocks ("plan.rs" names the checkpoint format `GgmlType::Q8_0`): each block is
 * 34 bytes, a little-endian IEEE binary16 scale d followed by 32 int8 values, in the same column-major block order.
 * The scale is widened to fp32 exactly (subnormals kept).  Errors as q8_repack (a non-finite scale or a value of
 * -128 is Q8_ERR_NOT_Q8_0). */
q8_status q8_repack_f16(const void *blocks, int K, int N, int8_t *q, float *s);

/* Host Q8_0 quantization of a declared weight (source: "from_q8.rs", `quantize`).
 *   w  host, fp64 [K][N] row-major (the declared values, as the pages' rule takes them)
 *   q  host, int8 [K][Np] (written, pad columns 0)     s  host, fp32 [K/32][Np] (written, pad columns 0)
 * For every 32-row block and column: amax = max |w|; an all-zero block gets q = 0 and s = 0; otherwise
 * d = amax / 127 (in fp64) must be exactly an fp32 value, and every w / d must lie within 1e-9 of an integer r with
 * |r| <= 127 and r * d == w exactly.  Any failure returns Q8_ERR_NOT_Q8_0 (q and s then hold no meaning). */
q8_status q8_quantize(const double *w, int K, int N, int8_t *q, float *s);

/* ---------------------------------------------------------------------------------------------------------------
 * Between the q/k/v products and the output projection: a paged key-value cache, the rotation and the append that
 * fill it, and the attention that reads it.  No counterpart on the pages beyond their key-value rows ("plan.rs"); the
 * formulas are stated with each call.
 * ------------------------------------------------------------------------------------------------------------- */

/* A paged key-value cache.  A page holds `page_size` consecutive tokens of one request for all its heads:
 *   bf16 (k_scale and v_scale NULL):  k, v  bf16 [pages][heads][page_size][dim]
 *   Q8_0 (both given):                k, v  int8 of that shape, and fp32 k_scale, v_scale
 *                                     [pages][heads][page_size][dim / 32]: value = code * scale, the form of
 *                                     q8_quantize_act taken over each 32 values of a head (1.125 bytes a value)
 * page_stride is the number of values from one page to the next (heads * page_size * dim when pages are dense, more
 * when several caches share an allocation); the scales' pages are page_stride / 32 apart.
 *   dim 64 or 128; page_size a positive multiple of 16; page_stride a multiple of 128, at least heads * page_size *
 *   dim, pages * page_stride at most 2^38; k, v and the scales 16-byte aligned.
 * A token's slot is page * page_size + its offset in the page.  A block table is int32 [requests][table_width] (rows
 * table_pitch apart): entry i of a request is the page of its tokens i * page_size and on.  An entry outside
 * [0, pages) names no page: attention sees no token there.  Offsets are 64-bit throughout. */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride;
    int pages, heads, page_size, dim;
} q8_kv_cache;

/* The most requests one call takes. */
#define Q8_MAX_REQUESTS 16384

/* Block tables and slot maps of one step, from the requests' lengths, on the device.  For request r with cached[r]
 * tokens in the cache and fresh[r] new ones (negative lengths count as 0):
 *   have = ceil(cached / page_size), want = min(table_width, ceil((cached + fresh) / page_size)),
 *   need = max(0, want - have), base = the sum of the requests' needs before r,
 *   table[r][have + i] = free_pages[head + base + i] for i < need (-1 where that index is not below n_free),
 *   lens[r] = cached + fresh, row_start[r] = the sum of fresh before r (row_start[R] = the total),
 *   and the row row_start[r] + i of the step's `rows` rows, i < fresh:
 *   positions = cached + i, slots = table[r][position / page_size] * page_size + position % page_size, or -1 where
 *   that entry is missing (beyond table_width, or the free list ran out).
 * Rows past the total are padding: positions and slots -1 (q8_rope_append skips them), so a step captured in a graph
 * can keep a fixed row count.  next_head = head + the sum of the needs: it passes n_free when the list ran out.
 *   cached, fresh  device, int32 [R], 1 <= R <= Q8_MAX_REQUESTS      free_pages  device, int32 [n_free] (may be NULL
 *   head           device, int32 [1], or NULL for 0                                  when n_free is 0)
 *   table          device, int32 [R][table_width], rows table_pitch apart (entries below `have` read, new ones written)
 *   lens int32 [R], row_start int32 [R + 1], positions int32 [rows], slots int64 [rows], next_head int32 [1]: device,
 *   written; none may overlap an input or another output.  The sums must stay below 2^31.
 * Errors: Q8_ERR_ARG (NULL pointers, overlaps), Q8_ERR_SHAPE (R, page_size, table_width, table_pitch < table_width,
 * rows < 0, n_free < 0), Q8_ERR_ALIGN (a pointer not aligned to its type), Q8_ERR_CUDA. */
q8_status q8_kv_slots(const int *cached, const int *fresh, int R, int page_size, const int *free_pages, int n_free,
                      const int *head, int *table, int table_width, int table_pitch, int rows, int *lens,
                      int *row_start, int *positions, int64_t *slots, int *next_head, q8_stream_t stream);

/* Flags of q8_rope_append. */
#define Q8_ROPE_INTERLEAVED 1u /* rotate the pairs (2i, 2i + 1); without it the halves (i, i + rotary_dim / 2) */

/* Norms of q and k per head, the rotation to their positions, and the write of k and v into the cache, in one pass
 * over the fp32 outputs of the q/k/v products.  For each head's `dim` values x of row t:
 *   u = x / sqrt(mean(x^2) + eps) * gamma          (q with q_gamma, k with k_gamma; u = x where gamma is NULL)
 *   (a, b) -> (a cos - b sin, a sin + b cos)       on the rotary_dim / 2 pairs of u's first rotary_dim values, with
 *   cos = table[position][i], sin = table[position][rotary_dim / 2 + i] for pair i
 * q is rounded to bf16 into q_out; k (normed, rotated) and v (as it is) are written at the row's slot in the cache's
 * type: bf16, or codes and scales by the rule of q8_quantize_act taken on the fp32 values.
 *   q          device, fp32 [rows][ldq], heads at column head * dim (q_heads of them); k, v likewise (cache->heads)
 *   q_gamma, k_gamma  device, fp32 [dim], or NULL        table  device, fp32 [max_positions][rotary_dim], or NULL
 *   positions  device, int32 [rows]    slots  device, int64 [rows]     when rotary_dim is 0
 *   q_out      device, bf16 [rows][ldo] (written)
 *   1 <= rows <= 65535; rotary_dim a multiple of 8, 0 .. dim; ldq, ldk, ldv multiples of 4, ldo of 8; all pointers 16-byte aligned
 *   (positions 4, slots 8, gammas 16)
 * A row with a negative position is padding: its q is written as zeros and nothing goes to the cache.  A row with a
 * slot outside the cache writes nothing to it.  A position past the table gives NaN in the rotated values.  Two rows
 * with one slot leave either's values there.
 * Errors: Q8_ERR_ARG (NULL pointers, unknown flags, eps < 0 or not finite, q_out overlapping an input or the cache),
 * Q8_ERR_SHAPE, Q8_ERR_ALIGN, Q8_ERR_CUDA. */
q8_status q8_rope_append(const float *q, int ldq, const float *k, int ldk, const float *v, int ldv,
                         const float *q_gamma, const float *k_gamma, float eps, const float *table, int max_positions,
                         int rotary_dim, const int *positions, const int64_t *slots, void *q_out, int ldo,
                         const q8_kv_cache *cache, int rows, int q_heads, unsigned int flags, q8_stream_t stream);

/* Bytes of device workspace the attention calls take: a constant.  The caller zeroes it once before its first use
 * (the calls leave its counters at zero) and gives calls that may overlap on the GPU one each. */
int64_t q8_attn_workspace_bytes(void);

/* Attention of one new token a request over the paged cache (grouped heads: query head h reads cache head
 * h / (q_heads / cache->heads)):
 *   out[r] = sum_j w_j v_j,   w = softmax over the visible j of scale * (q[r] . k_j)
 * where request r's token has position p = lens[r] - 1 and key j < lens[r] is visible when
 *   window == 0, or p - j < window, or j < sinks
 * and its page is in the table.  A row that sees nothing (lens[r] <= 0) gets zeros.  What is not visible is not read
 * into the result, whatever its bits.  Scores, softmax statistics and sums are fp32.  On the way to them, and from them:
 *   - the weights w_j are rounded before they multiply v: over a bf16 cache to bf16 (each off by 2^-8 of itself at most);
 *     over a Q8_0 cache to fp16, decode w_j times v's scale (2^-11 of itself down to 2^-22 of the head's largest such
 *     product in the block of 32 values, 2^-33 of that below), prefill w_j (2^-11 of itself down to 2^-14 of the row's
 *     largest, 2^-25 of that below);
 *   - prefill over a Q8_0 cache takes code * scale in fp16 (two roundings of 2^-11 down to 2^-21 of the largest scale at
 *     hand; blocks of the result that smaller ones could show in are computed from fp32);
 *   - the result is rounded to bf16.
 * In all some 2e-3 of the result in its 2-norm, most of it that last rounding.
 *   q, out  device, bf16 [R][ldq], [R][ldo]: heads at column head * dim; q_heads a multiple of cache->heads
 *   block_table  device, int32 [R][table_width], rows table_pitch apart      lens  device, int32 [R]
 *   window >= 0, sinks >= 0 (ignored when window is 0); scale finite
 *   workspace  device, q8_attn_workspace_bytes() bytes, 16-byte aligned
 * A long cache is split over the SMs and its parts joined in a fixed order: results do not depend on timing.
 * Errors: Q8_ERR_ARG (NULL pointers, a scale not finite, out overlapping an input, window or sinks < 0),
 * Q8_ERR_SHAPE (R outside 1..Q8_MAX_REQUESTS, heads, dims, widths or pitches), Q8_ERR_ALIGN, Q8_ERR_CUDA. */
q8_status q8_attn_decode(const void *q, int ldq, const q8_kv_cache *cache, const int *block_table, int table_width,
                         int table_pitch, const int *lens, void *out, int ldo, int R, int q_heads, float scale,
                         int window, int sinks, void *workspace, q8_stream_t stream);

/* Attention of a chunk of new tokens, rows row_start[r] .. row_start[r + 1] - 1 being request r's last
 * n = row_start[r + 1] - row_start[r] tokens: row row_start[r] + i has position p = lens[r] - n + i and sees key j <= p
 * by the rule of q8_attn_decode (window, sinks, missing pages).  The chunk's own keys are in the cache already.
 *   q, out  device, bf16 [rows][ldq], [rows][ldo]      row_start  device, int32 [R + 1], ascending from 0, at most rows
 * Rows past row_start[R] are padding and get zeros, as do rows that see nothing.  Other arguments, errors: as
 * q8_attn_decode; 1 <= rows <= 2^24, q_heads at most 128 times cache->heads. */
q8_status q8_attn_prefill(const void *q, int ldq, const q8_kv_cache *cache, const int *block_table, int table_width,
                          int table_pitch, const int *lens, const int *row_start, void *out, int ldo, int rows, int R,
                          int q_heads, float scale, int window, int sinks, void *workspace, q8_stream_t stream);

/* ---------------------------------------------------------------------------------------------------------------
 * Weights of 4 bits with group scales, and the choice of the next token: the products of a decode or prefill step over
 * half the bytes of Q8_0, and what follows the last of them.  No counterpart on the pages.
 * ------------------------------------------------------------------------------------------------------------- */

/* A 4-bit weight: codes c in 0..15, and for each group of `group` consecutive rows of a column a 16-bit scale s and a
 * zero point z:
 *     W[k, n] = s[k / group, n] * (c[k, n] - z[k / group, n])
 *   group  32, 64 or 128; K a multiple of it, at most 2^31 - 128
 *   flags  Q8_W4_ZEROS: the zero points are given (without it z = 8 everywhere); Q8_W4_BF16: the scales are bf16 (without
 *          it fp16)
 * As a checkpoint has it ("plain"):
 *   codes   uint8 [K/2][N]: row 2i of column n in the low four bits of codes[i][n], row 2i + 1 in the high ones
 *   scales  fp16 or bf16 [K/group][N]        zeros  uint8 [K/group][N], 0..127
 * As the products read it ("tiled", q8_w4_tile): strips of 32 columns, of a strip one unit for each group in the order of
 * K, unit (strip, g) at (strip * (K/group) + g) * U bytes, U = 16 * group + 64 (+ 32 with Q8_W4_ZEROS):
 *   codes   words of 8 rows of one column, rows 8t + 2p and 8t + 2p + 1 of a 32-row block in bits 4p .. 4p + 3 and
 *           16 + 4p .. 16 + 4p + 3 (p = 0..3).  With column 16j + 8h + i of the strip (j, h = 0, 1; i = 0..7) and block b of
 *           the group, the word is number 2 (b % 2) + h of the 16 bytes at 512 (2 (b / 2) + j) + 16 (4i + t), or with
 *           group 32 number h of the 8 bytes at 256 j + 8 (4i + t)
 *   scales  32 of 16 bits, in column order        zeros  32 bytes, in column order (Q8_W4_ZEROS)
 * Columns at or past N of the last strip hold code 0, scale 0 and zero point 0.
 * q8_w4_bytes(K, N, group, flags): the tiled form's bytes; -1 for sizes or flags that are not a weight's. */
typedef struct {
    const void *w; /* device, tiled, 16-byte aligned */
    int N, group;
    unsigned int flags;
} q8_weight4;

#define Q8_W4_ZEROS 1u
#define Q8_W4_BF16 2u

int64_t q8_w4_bytes(int K, int N, int group, unsigned int flags);

/* Plain -> tiled, on the host, and on the device enqueued on `stream` (w 16-byte aligned there, scales 2-byte; w may not
 * overlap an input).  zeros is NULL exactly when flags has no Q8_W4_ZEROS.  The low seven bits of a zero point count.
 * On the device two launches, the second only to order what comes after: a product on `stream` may take the weight with
 * Q8_FLAG_CONSTANT_WEIGHTS at once.
 * Errors: Q8_ERR_ARG (NULL pointers, zeros against flags, unknown flags, overlaps), Q8_ERR_SHAPE, Q8_ERR_ALIGN. */
q8_status q8_w4_tile(const uint8_t *codes, const void *scales, const uint8_t *zeros, int K, int N, int group,
                     unsigned int flags, void *w);
q8_status q8_w4_tile_device(const uint8_t *codes, const void *scales, const uint8_t *zeros, int K, int N, int group,
                            unsigned int flags, void *w, q8_stream_t stream);

/* Host repack of GGML-style Q4_0 checkpoint blocks into the plain form (group 32, z = 8, fp16 scales): N * (K/32) blocks of
 * 18 bytes, column-major by block as q8_repack_f16's, each a little-endian binary16 scale and 16 bytes, byte i holding row
 * i of the block in its low and row 16 + i in its high four bits.  Q8_ERR_NOT_Q8_0 for a scale that is not finite. */
q8_status q8_w4_repack(const void *blocks, int K, int N, uint8_t *codes, uint16_t *scales);

/* y_p = x . W_p for every part p, 1 <= nparts <= Q8_MAX_PARTS; all parts have the same K, group and flags.
 *   x  device, bf16 [m][K], 16-byte aligned, 1 <= m <= Q8_MAX_CHUNK        y  host array of device pointers, fp32
 *   [m][q8_padded_n(N_p)] (written, 0 in the pad columns), 16-byte aligned, none overlapping an input or another y
 *   flags  Q8_FLAG_CONSTANT_WEIGHTS (no work enqueued before this call on `stream` writes a weight's tiled form, other than
 *          q8_w4_tile_device; the call may read it before that work has ended) or 0
 * Codes less zero points and activations enter the tensor cores exactly (bf16); a group's sums are fp32, scaled in fp32
 * and added in fp32 in an order fixed for the entry point, m, K, the group, the widths of all the call's weights and the
 * device: repeated calls give identical bits, whatever the other rows and weights hold.  (How K is split follows the tiles of the
 * whole call, so that a weight alone and beside others may differ in the last bits.)  Each output is within
 * max(1e-5, (K / group + 64) * 2^-24) * sum |x s (c - z)| of the real number: one rounding a group where all of K is one
 * carry's, and 64 for the sums within a group and the joins.  Equal terms, whose roundings do not cancel, measured a quarter
 * of it (512 rows, K = 28672 in groups of 32: 1.3e-5; up to 16 rows, whose K is shared by warps, 2e-6 to 8e-6), random
 * positive ones 3e-6 at most.
 * Up to 16 rows run as a stream of the weight, one launch; more on tcgen05, one launch or two (the tiles of a last partial
 * wave apart, with a K split of their own).
 * Errors: Q8_ERR_ARG (NULL pointers, unknown flags, parts that differ in group or flags, overlaps), Q8_ERR_SHAPE (m, K, N,
 * group, nparts), Q8_ERR_ALIGN, Q8_ERR_CUDA. */
q8_status q8_gemv4_parts(const void *x, const q8_weight4 *weights, float *const *y, int nparts, int m, int K,
                         unsigned int flags, q8_stream_t stream);

/* The same for one weight. */
q8_status q8_gemv4(const void *x, const q8_weight4 *weight, float *y, int m, int K, unsigned int flags,
                   q8_stream_t stream);

/* The gated pair: out = silu(x . Wg) * (x . Wu), silu(g) = g / (1 + exp(-g)), as q8_gemv_glu; gate and up have the same N,
 * group and flags.  out fp32 [m][Np], out_bf16 bf16 [m][Np] (rounded to nearest even), either may be NULL; pads 0.
 * Launches, other arguments and errors as q8_gemv4_parts. */
q8_status q8_gemv4_glu(const void *x, const q8_weight4 *gate, const q8_weight4 *up, float *out, void *out_bf16, int m,
                       int K, unsigned int flags, q8_stream_t stream);

/* The product, the residual add and the next RMS norm, as q8_gemv_residual_norm (its arguments and aliasing: h may be
 * residual itself): h = residual + x . W, out = h / sqrt(mean(h^2) + eps) * gamma.  The product's
 * launches (as q8_gemv4_parts) and one more. */
q8_status q8_gemv4_residual_norm(const void *x, const q8_weight4 *weight, const float *residual, const float *gamma,
                                 float eps, float *h, void *out_bf16, int m, int K, unsigned int flags,
                                 q8_stream_t stream);

/* What a step does to its logits before a token is chosen.  Every pointer may be NULL: that rule is then left out.  All are
 * device pointers, aligned to their type. */
typedef struct {
    const float *repetition, *frequency, *presence, *temperature; /* fp32 [m] */
    const void *history;   /* int32 (int64 with history_wide) [m][history_pitch]: the tokens of each row's request */
    const int *lengths;    /* int32 [m]: how many of them there are (required with history) */
    const int *prompts;    /* int32 [m]: how many of those are prompt, not answer (NULL: none) */
    const int *bias_ids;   /* int32 [m][bias_width]: tokens with a bias; ids outside 0..N-1 are unused places */
    const float *bias;     /* fp32 [m][bias_width]: their biases (required with bias_ids) */
    const int *mask;       /* int32 [mask_count][mask_pitch]: bit n % 32 of word n / 32 set: token n is allowed */
    const int *mask_rows;  /* int32 [m]: the mask of each row, none outside 0..mask_count-1 (requires mask; NULL:
                              row r has mask r, and there have to be m of them) */
    const float *noise;    /* fp32 [m][noise_pitch]: added for the choice alone */
    int history_width, history_pitch, history_wide, bias_width, mask_count, mask_pitch, noise_pitch;
} q8_choice;

#define Q8_MAX_HISTORY 1048575
#define Q8_MAX_BIAS 2047

/* The rules on logits, and the token chosen.  For token n < N of row r, in fp32, each step rounded once:
 *     v = logits[r][n]
 *     v = v > 0 ? v / repetition : v * repetition        if n stands anywhere in history[r][0 .. lengths[r])
 *     v = v - frequency * c                              c = how often n stands in history[r][prompts[r] .. lengths[r])
 *     v = v - presence                                   if c > 0
 *     v = v + bias                                       if n is among bias_ids[r] (at several places: the last one counts)
 *     v = v / temperature                                if temperature > 0
 *     out[r][n] = v, or -inf where the row's mask has no bit for n (whatever v is, NaN too)
 *     idx[r] = the lowest n with the largest score among the tokens that the mask allows, -1 if it allows none;
 *              score = v + noise[r][n] where temperature > 0, else v
 * A NaN is larger than +inf, and -0 equals +0, as in q8_gemv_argmax.  With Gumbel noise (-log(-log(u)), u uniform) idx is a
 * sample of softmax(v); a temperature of 0 (or none) is greedy.  A negative or NaN temperature counts as 0.  Without
 * temperature (NULL) the noise is not added.
 *   logits  device, fp32 [m][ldl]      out  device, fp32 [m][ldo], or NULL (only idx is written); may be logits itself with
 *   idx     device, int64 [m]                ldo == ldl (in place), and may not overlap an input otherwise
 *   1 <= m <= 65535, 1 <= N <= 2^30, pitches at least N (history_pitch >= history_width, mask_pitch >= ceil(N / 32))
 *   history_width <= Q8_MAX_HISTORY, bias_width <= Q8_MAX_BIAS, both >= 1 where given
 * Lengths beyond history_width count as it, negative ones as 0, as do prompts; tokens of the history outside 0..N-1 are
 * passed over.  repetition is expected positive.  One launch.
 * Errors: Q8_ERR_ARG (NULL pointers, a rule without its companion, overlaps), Q8_ERR_SHAPE, Q8_ERR_ALIGN, Q8_ERR_CUDA. */
q8_status q8_choose(const float *logits, int ldl, const q8_choice *rules, float *out, int ldo, int64_t *idx, int m, int N,
                    q8_stream_t stream);

/* Reads the device fault word of the current device: nonzero when a kernel's bounded wait on a pipeline barrier ran
 * out (bit 0: a consumer waited about two seconds for a stage's data; bit 1: the producer waited as long for a free
 * stage; bit 2: a wait of the prefill GEMM ran out; bit 3: one of q8_attn_prefill, whose workspace has to be
 * zeroed again; bit 4: one of the products over 4-bit weights) and the kernel finished early -- that call's outputs are then
 * wrong.  Synchronous with respect to the
 * device.  `clear` != 0 resets the word to 0.  Returns Q8_ERR_ARG for a NULL `fault`, Q8_ERR_CUDA on a CUDA error. */
q8_status q8_device_fault(unsigned int *fault, int clear);

/* Planner overrides for tests and benchmarks (no counterpart on the pages).  Process-wide: every later call on every
 * thread and device sees the value, so set them only while no other thread is enqueuing work.  Each option starts
 * from an environment variable, read once, at the first call that plans a launch.
 *   Q8_TUNE_KSPLIT     0: the planner's K split (default); 1..8: every K-split cluster takes this many CTAs (capped
 *                      at the number of K blocks; the gated pair and the prefill GEMM take at most 4).
 *                      Environment: Q8_KSPLIT.
 *   Q8_TUNE_GEMM       -1: the planner's choice (default); 0: calls of 128 rows or more keep the row groups; 1: they
 *                      run on the tcgen05 GEMM whatever the weight's width.  Environment: Q8_GEMM (0 or 1).
 *   Q8_TUNE_NORM_FOLD  0: the residual norm as a launch of its own (default); 1: the one-launch fold, where the
 *                      product's last CTA runs the norm.  Environment: Q8_NORM_LAUNCH=0 selects 1.
 *   Q8_TUNE_SPLIT      1: the planner may run a plain product (q8_gemv, q8_gemv_argmax, q8_gemv_parts) or a gated
 *                      pair (q8_gemv_glu) of m <= 16 rows as two launches, the column tiles that do not fill the
 *                      SMs evenly given their own K split (default); 0: always one launch.  Environment: Q8_SPLIT=0
 *                      selects 0. */
#define Q8_TUNE_KSPLIT 0
#define Q8_TUNE_GEMM 1
#define Q8_TUNE_NORM_FOLD 2
#define Q8_TUNE_SPLIT 3

/* Sets an override.  Returns Q8_ERR_ARG for an unknown option or a value outside its range. */
q8_status q8_set_tuning(int option, int value);

/* The current value of an override (its environment default until set); -2 for an unknown option. */
int q8_get_tuning(int option);

/* A static, human-readable name for a status code. */
const char *q8_status_string(q8_status status);

/* The cudaError_t of the last CUDA failure on the calling thread (0 when none). */
int q8_last_cuda_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int q8_version(void);

#ifdef __cplusplus
}
#endif

#endif /* Q8_GEMV_H */
