/*
 * seqattn.h -- C ABI of libseqattn: sequence-partitioned (chunked) causal
 * attention forward and exact backward on one GB300 (sm_103a).
 *
 * The operation is the per-chunk attention of StreamBP ("StreamBP:
 * Memory-Efficient Exact Backpropagation for Long Sequence Training of LLMs",
 * review page): Property 3.1 ("What carries the argument") says chunk i's
 * output needs only Q^(i), K^(:i), V^(:i); Eq. (1) writes the gradient as a
 * sum of per-chunk terms, and the "Circularity Check" names the partitioned
 * attention of Eqs. (12)-(14) and the running sum that accumulates the
 * per-chunk dK/dV over the prefix.  The same chunk-by-chunk backward with
 * key/value caches as checkpoints is SeCO's ("Training Long-Context LLMs
 * Efficiently via Chunk-wise Optimization", review page, "What carries the
 * argument").
 *
 * Notation: B batch, T = seq_capacity (cache rows), Hq query heads, Hkv
 * key/value heads, G = Hq / Hkv, d = head_dim.  Query head h reads key/value
 * head h / G (contiguous groups).  A chunk is q_len query rows at absolute
 * positions [q_start, q_start + q_len); row r attends keys
 * [q_start - prefix_len, q_start + r] (causal inside the chunk).  prefix_len ==
 * q_start is the method's full prefix K^(:i); a smaller prefix_len starts the
 * window later.
 *
 * Tensor layouts (all dense, row-major, element strides implied):
 *   q, o, d_o : [B, q_len, Hq, d]          chunk-local rows
 *   k, v      : [B, T, Hkv, d]             full cache, row 0 = token 0
 *   lse       : [B, Hq, q_len]   float32   natural-log row logsumexp of the
 *                                          scaled scores (the stored M^(i))
 *   dq        : [B, q_len, Hq, d] float32
 *   dk_accum,
 *   dv_accum  : [B, T, Hkv, d]    float32  running sums over chunks
 * Element type of q, k, v, o, d_o: bfloat16 for SEQATTN_BF16, float32 for
 * SEQATTN_FP32.  Every pointer is a DEVICE pointer owned by the caller and
 * must be 16-byte aligned; the library allocates nothing and keeps no state
 * between calls other than a device-side error word (and the fixed scratch
 * array of seqattn_chunk_bwd_noalloc).
 *
 * All work is enqueued asynchronously on `stream` (a cudaStream_t; 0 is the
 * legacy default stream).  Argument errors are detected on the host before
 * anything is launched.  Launch failures return SEQATTN_ERR_CUDA.  Every
 * device-side wait in the kernels is bounded: a wait that runs out sets the
 * device error word and the kernel returns early; that is reported as
 * SEQATTN_ERR_TIMEOUT by the next call of seqattn_sync_status().
 * No function throws, aborts or prints.
 */
#ifndef SEQATTN_H
#define SEQATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* seqattn_stream_t; /* same type as cudaStream_t */

typedef enum {
  SEQATTN_OK = 0,
  SEQATTN_ERR_INVALID_ARG = 1, /* bad pointer, shape, alignment or scale */
  SEQATTN_ERR_UNSUPPORTED = 2, /* valid request this build does not cover */
  SEQATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
  SEQATTN_ERR_TIMEOUT = 4      /* a bounded device-side wait ran out */
} seqattn_status;

typedef enum { SEQATTN_BF16 = 0, SEQATTN_FP32 = 1 } seqattn_dtype;

typedef struct {
  int32_t batch;        /* B >= 1 */
  int32_t num_q_heads;  /* Hq >= 1 */
  int32_t num_kv_heads; /* Hkv >= 1, Hq % Hkv == 0 */
  int32_t head_dim;     /* d: 64 or 128 */
  int64_t seq_capacity; /* T: rows of the k/v caches and dk/dv accumulators */
  int32_t dtype;        /* seqattn_dtype */
} seqattn_problem;

/*
 * Forward of one chunk: O^(i) = softmax(scale * Q^(i) K^(:i)^T, causal) V^(:i)
 * and the row logsumexp (StreamBP review page, Property 3.1 and Eqs. (12)-(14)
 * named in the "Circularity Check"; the stored row statistic M^(i) of the
 * verdict page's stored-activation list).
 *   q_start, q_len, prefix_len: chunk rows and key window as described above;
 *     requires 0 <= prefix_len <= q_start and q_start + q_len <= T.
 *     q_len == 0 is a no-op.
 *   softmax_scale: finite, > 0 (usually 1/sqrt(d)).
 *   o (out), lse (out): overwritten.
 * Both dtypes accept any q_start, q_len, prefix_len and d in {64, 128}.
 */
seqattn_status seqattn_chunk_fwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                 int64_t prefix_len, float softmax_scale, const void* q,
                                 const void* k, const void* v, void* o, float* lse,
                                 seqattn_stream_t stream);

/*
 * Exact backward of one chunk (StreamBP review page, Eq. (1) and the running
 * sum of the "Circularity Check"; major comment 1 of its referee report names
 * dK^(:i), dV^(:i) over the prefix).  With P = exp(scale*QK^T - lse),
 * dP = dO V^T, Delta = rowsum(dO o O), dS = P o (dP - Delta):
 *   dq (out, overwritten)      = scale * dS K
 *   dk_accum rows [q_start - prefix_len, q_start + q_len) += scale * dS^T Q
 *   dv_accum rows [q_start - prefix_len, q_start + q_len) += P^T dO
 * (summed over the G query heads of each key/value head).  o and lse are the
 * forward's outputs for this chunk.  Other accumulator rows are untouched.
 *   workspace: device scratch of at least seqattn_bwd_workspace_size(pb,
 *     q_len) bytes, 256-byte aligned, caller-owned, contents not preserved.
 * Size rules as for seqattn_chunk_fwd.  Calls on one stream accumulate in
 * order.  SEQATTN_BF16: the accumulator updates are fp32 reduce-adds done in
 * L2 (atomic per element), so calls for different chunks may run concurrently
 * on different streams, each with a workspace of its own (the order of the
 * fp32 additions, and so the last bits of the sums, then varies between
 * runs).  SEQATTN_FP32: the updates are
 * plain read-modify-writes; two calls that update the same accumulator rows
 * must not run concurrently.
 */
seqattn_status seqattn_chunk_bwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                 int64_t prefix_len, float softmax_scale, const void* q,
                                 const void* k, const void* v, const void* o, const float* lse,
                                 const void* d_o, float* dq, float* dk_accum, float* dv_accum,
                                 void* workspace, size_t workspace_bytes,
                                 seqattn_stream_t stream);

/*
 * Backward of one chunk for callers that cannot allocate device memory.  The
 * paper has no counterpart: this is a library convenience.  Some callers own
 * no allocator of their own -- their device memory belongs to another
 * allocator (a framework's caching allocator or a fixed arena) and the
 * interface they call through passes only the tensors -- so they cannot
 * provide the workspace seqattn_chunk_bwd asks for.  This entry point computes
 * exactly what seqattn_chunk_bwd computes, with the same arguments minus the
 * workspace, and calls no allocation routine.
 *
 * Its scratch (the per-row statistics, seqattn_bwd_workspace_size(pb, q_len)
 * bytes) is a fixed device array inside the library of
 * SEQATTN_NOALLOC_MAX_DELTA floats (4 MiB), which every GPU that loads the
 * library holds until the process exits.  Larger requests return
 * SEQATTN_ERR_INVALID_ARG (use seqattn_chunk_bwd instead).  The first
 * call on a device looks up that device's address of the array; make that
 * first call before any stream capture.  Every call shares the one array, so
 * calls that overlap on the GPU (different streams, or different host
 * threads) race on it and must be serialised by the caller.
 */
#define SEQATTN_NOALLOC_MAX_DELTA (1 << 20)
seqattn_status seqattn_chunk_bwd_noalloc(const seqattn_problem* pb, int64_t q_start,
                                         int64_t q_len, int64_t prefix_len, float softmax_scale,
                                         const void* q, const void* k, const void* v,
                                         const void* o, const float* lse, const void* d_o,
                                         float* dq, float* dk_accum, float* dv_accum,
                                         seqattn_stream_t stream);

/* Zero both float32 accumulators ([B, T, Hkv, d] each) before the first chunk
 * of a backward pass (the running sum starts at zero). */
seqattn_status seqattn_reset_accum(const seqattn_problem* pb, float* dk_accum, float* dv_accum,
                                   seqattn_stream_t stream);

/*
 * Multiply rows [row_begin, row_end) of both float32 accumulators by `scale`;
 * scale == 0 stores zeros.  This is the step SpaCO adds to the chunk loop
 * (SeCO review page, "Referee Report": the Summary, where t of the k chunks
 * are backpropagated and the relayed KV-cache gradient is multiplied by k/t,
 * and the major comments on Algorithm 2 and Section 6.4, where the factor
 * is capped at 2).  Before a selected chunk's backward, its own rows --
 * which then hold only what later chunks relayed into them -- are scaled by
 * the compensation factor; the rows of a chunk that is not selected are
 * zeroed, since nothing propagates from them.
 *   0 <= row_begin <= row_end <= seq_capacity; scale finite.  Every batch
 *   entry and every key/value head of those rows is scaled.  dk_accum,
 *   dv_accum: [B, seq_capacity, Hkv, d] float32, 16-byte aligned.
 * Async on `stream`; INVALID_ARG before any launch on a bad argument.
 */
seqattn_status seqattn_scale_accum_rows(const seqattn_problem* pb, int64_t row_begin,
                                        int64_t row_end, float scale, float* dk_accum,
                                        float* dv_accum, seqattn_stream_t stream);

/*
 * Projection weight gradient of rows [row_begin, row_end): the step after the
 * path (SeCO review page, major comment 1 on Algorithm 2 -- once chunk i's
 * cache gradient is complete, chunk i's graph, here the Q/K/V projections
 * X = H W, is backpropagated).  With the last-to-first chunk order the dK/dV
 * rows of chunk i are final right after its backward, so this runs per chunk.
 *   dw[d_model, n] += sum over batch entries b and rows r of h[b, r]^T g[b, r]
 *   h: [batch, seq_len, d_model] bf16 (the projections' input)
 *   g: [batch, seq_len, n] float32 (dQ with n = Hq d, or dK / dV with
 *      n = Hkv d)
 *   dw: [d_model, n] float32, row-major, accumulated (never overwritten)
 * One tensor-core kernel: g is rounded to bf16 (nearest even) as it is read,
 * the products are summed in float32 and each CTA adds its tile into dw with
 * TMA reduce-adds (atomic per element in L2), so calls that update the same
 * dw may run concurrently on different streams (the order of the fp32
 * additions, and so the last bits of dw, then varies between runs).  Rows of
 * h outside [row_begin, row_end) are read only where they meet a zero of g
 * and must be finite.  Requires batch >= 1, 0 <= row_begin <= row_end <= seq_len,
 * d_model and n positive multiples of 8, and 16-byte aligned pointers.  No
 * workspace.  Async on `stream`; INVALID_ARG before any launch on a bad
 * argument; row_begin == row_end is a no-op.
 */
seqattn_status seqattn_proj_wgrad(int32_t batch, int64_t seq_len, int64_t row_begin,
                                  int64_t row_end, int32_t d_model, int32_t n, const void* h,
                                  const float* g, float* dw, seqattn_stream_t stream);

/* ------------------------------------------------------------------------
 * The rest of the attention layer: projections, head norm with rotary
 * positions, and the optimizer step.  (The pages partition the attention and
 * name the projections only as "chunk i's graph"; these calls run that graph
 * chunk by chunk around the attention calls.)
 * ------------------------------------------------------------------------ */

typedef enum {
  SEQATTN_ACT_NONE = 0,
  SEQATTN_ACT_RELU = 1,
  SEQATTN_ACT_SILU = 2,     /* z sigmoid(z) */
  SEQATTN_ACT_GELU = 3,     /* z Phi(z), by erf */
  SEQATTN_ACT_GELU_TANH = 4 /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
} seqattn_act;

/*
 * Linear layer, bf16 with float32 sums: a product and its epilogue in one
 * tensor-core kernel, one rounding to bf16 at the end.
 *   fwd:    z = x w + bias;  y = act(z) + residual
 *   dgrad:  dx = act'(z) o (g w^T) + residual
 *   wgrad:  dw += x^T g;  dbias += sum over rows of g
 * w: [k, n] dense row-major (the layout of the projections' weight gradients).
 * x [rows, k], g [rows, n], y, z [rows, n], dx [rows, k] and residual are
 * row-major with a row stride ld* in elements (so heads of a fused projection
 * or rows of a cache can be passed as they lie).  dw [k, n] and dbias [n] are
 * dense float32 and accumulated, in an order fixed by the shapes; calls that
 * update the same dw or dbias must not overlap.
 *   fwd:    bias [n], residual and z (out: the pre-activation in bf16, for
 *           dgrad) may be NULL.
 *   dgrad:  z is the previous layer's pre-activation, of dx's shape, read
 *           when act is not NONE (else NULL); residual may be NULL.  g is the
 *           gradient of this product's own pre-activation.
 *   wgrad:  dbias may be NULL.
 * residual may be the output itself (same pointer and stride); no other
 * overlap of an output with an operand is allowed (INVALID_ARG where two start
 * at the same address).  Requires k, n and every
 * stride to be positive multiples of 8, strides at least the row length,
 * pointers 16-byte aligned, 0 <= rows < 2^31 - 512; rows == 0 is a no-op.
 * Strides of operands that are NULL are ignored.  No workspace.  Async on
 * `stream`; INVALID_ARG before any launch on a bad argument.
 */
seqattn_status seqattn_linear_fwd(int64_t rows, int32_t k, int32_t n, const void* x, int64_t ldx,
                                  const void* w, const void* bias, int32_t act,
                                  const void* residual, int64_t ldr, void* z, int64_t ldz,
                                  void* y, int64_t ldy, seqattn_stream_t stream);
seqattn_status seqattn_linear_dgrad(int64_t rows, int32_t k, int32_t n, const void* g, int64_t ldg,
                                    const void* w, int32_t act, const void* z, int64_t ldz,
                                    const void* residual, int64_t ldr, void* dx, int64_t lddx,
                                    seqattn_stream_t stream);
seqattn_status seqattn_linear_wgrad(int64_t rows, int32_t k, int32_t n, const void* x, int64_t ldx,
                                    const void* g, int64_t ldg, float* dw, float* dbias,
                                    seqattn_stream_t stream);

/*
 * A rotary embedding over the first rot_dim elements of a head.  Pair i is
 * rotated by position[axis[i]] * turns[i] * 2^-64 turns; turns[i] is the
 * frequency (f_i / 2 pi, radians per position over 2 pi) as an unsigned 64-bit
 * fraction, so the angle of any int64 position is exact modulo a turn.  With
 * interleaved == 0 pair i is elements (i, i + rot_dim / 2), else (2i, 2i + 1).
 * axes == 1: one position a row; more: several (time, height, width).
 */
typedef struct {
  int32_t rot_dim;      /* multiple of 16, at most head_dim */
  int32_t axes;         /* 1 .. 64 */
  int32_t interleaved;  /* 0 or 1 */
  int32_t reserved;     /* 0 */
  uint64_t turns[64];   /* rot_dim / 2 used */
  uint8_t axis[64];     /* each < axes */
} seqattn_rope_plan;

/*
 * Between the projections and seqattn_chunk_fwd, for the chunk's rows
 * [q_start, q_start + q_len): norm every query and key head (RMS over head_dim,
 * times gamma), rotate it, write the queries to the chunk and the keys and
 * values into rows [q_start, q_start + q_len) of the caches.
 *   q_in [B, q_len, Hq, d], k_in, v_in [B, q_len, Hkv, d]: element type pb->dtype,
 *     heads dense, consecutive rows (b, r) ld_q, ld_k, ld_v elements apart
 *     (parts of a fused projection's output can be passed in place).
 *     v_in and v_cache may both be NULL: values are then left alone.
 *   gamma_q, gamma_k [d]: element type; both NULL: no norm (eps is ignored).
 *   plan (host): NULL for no rotation.  positions: device int64 [axes, B, q_len],
 *     or NULL for position q_start + r on every axis.
 *   q (out) [B, q_len, Hq, d]; k_cache, v_cache (out rows) [B, T, Hkv, d].
 * The strides are at least a row's length and multiples of 8 elements;
 * eps >= 0.  Outputs overlap no other operand.  Sums, angles and the rotation are in float32, rounded once.
 */
seqattn_status seqattn_qk_norm_rope_fwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                        const void* q_in, int64_t ld_q, const void* k_in,
                                        int64_t ld_k, const void* v_in, int64_t ld_v,
                                        const void* gamma_q, const void* gamma_k, float eps,
                                        const seqattn_rope_plan* plan, const int64_t* positions,
                                        void* q, void* k_cache, void* v_cache,
                                        seqattn_stream_t stream);

/*
 * Its backward, between seqattn_chunk_bwd (once the chunk's rows of the
 * accumulators are final) and the projections' gradients: reads dq
 * [B, q_len, Hq, d] and rows [q_start, q_start + q_len) of dk_accum, dv_accum
 * [B, T, Hkv, d] (float32) and writes the gradients of q_in, k_in and v_in in
 * the element type (rows ld_dq, ld_dk, ld_dv elements apart).  dgamma_q,
 * dgamma_k [d] float32 are accumulated in a fixed order.
 *   q_in, k_in: the forward's inputs; read for the norm only (NULL without).
 *   dv_accum and dv_in may both be NULL.
 *   workspace: device scratch of seqattn_qk_norm_rope_bwd_workspace_size(pb)
 *     bytes, 256-byte aligned, when there is a norm (else NULL, 0); calls that
 *     overlap need one each, and must not update the same dgamma.
 * Outputs overlap no other operand; dgamma_q and dgamma_k are two vectors, also
 * when one gamma is used for both (their sum is its gradient).
 */
seqattn_status seqattn_qk_norm_rope_bwd(const seqattn_problem* pb, int64_t q_start, int64_t q_len,
                                        const void* q_in, int64_t ld_q, const void* k_in,
                                        int64_t ld_k, const void* gamma_q, const void* gamma_k,
                                        float eps, const seqattn_rope_plan* plan,
                                        const int64_t* positions, const float* dq,
                                        const float* dk_accum, const float* dv_accum, void* dq_in,
                                        int64_t ld_dq, void* dk_in, int64_t ld_dk, void* dv_in,
                                        int64_t ld_dv, float* dgamma_q, float* dgamma_k,
                                        void* workspace, size_t workspace_bytes,
                                        seqattn_stream_t stream);

/* Bytes of workspace seqattn_qk_norm_rope_bwd needs (0 for an invalid problem). */
size_t seqattn_qk_norm_rope_bwd_workspace_size(const seqattn_problem* pb);

/* One tensor of an optimizer step.  Pointers are device pointers, 16-byte
 * aligned (the scales: 4-byte aligned). */
typedef struct {
  float* param;          /* [n] float32 master weights, updated */
  void* lowp;            /* [n] bf16 copy of the updated param, or NULL */
  const void* grad;      /* [n] float32 or bf16 */
  void* m;               /* first moment: [n] float32, or e4m3 codes (8 bit) */
  void* v;               /* second moment: [n] float32, or e4m3 codes of its root */
  float* m_scale;        /* 8 bit: [ceil(n / 256)] scale of each 256 elements */
  float* v_scale;
  int64_t n;             /* >= 0 */
  float weight_decay;    /* finite */
  int32_t grad_bf16;     /* 0: grad is float32, 1: bf16 */
} seqattn_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, grad_scale;
  int64_t step;                 /* 1 for the first step */
  const float* lr_dev;          /* device scalars read when the step runs: lr_dev and */
  const float* grad_scale_dev;  /* step_dev replace lr and step, grad_scale_dev is */
  const int64_t* step_dev;      /* multiplied to grad_scale.  NULL: the host values. */
} seqattn_adamw_params;

/*
 * One AdamW step (decoupled weight decay) over `count` tensors:
 *   g = grad_scale grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * state_bits 32: m and v float32.  state_bits 8: m and u = sqrt(v) are kept as
 * e4m3 codes of m / m_scale and u / v_scale, m_scale and v_scale being the
 * largest magnitude of each 256 consecutive elements over 448; a positive u is
 * never stored as zero, and a block whose largest magnitude is under 1e-30
 * stores zeros.  Zeroed states (codes and scales) are the initial ones.
 * The descriptors (host memory) are read during the call and travel with the
 * launch; a captured call keeps the values it was captured with, so a step
 * meant for replay passes step_dev (and lr_dev).  No two tensors of a call may
 * overlap.  0 <= beta1, beta2 < 1, eps >= 0; lr, eps and grad_scale finite, step >= 1.
 */
seqattn_status seqattn_adamw_step(const seqattn_adamw_tensor* tensors, int32_t count,
                                  int32_t state_bits, const seqattn_adamw_params* params,
                                  seqattn_stream_t stream);

/* Bytes of workspace seqattn_chunk_bwd needs for a chunk of q_len rows
 * (0 for an invalid problem).  Pure host function. */
size_t seqattn_bwd_workspace_size(const seqattn_problem* pb, int64_t q_len);

/* Synchronise `stream`, then read and clear the device error word.  Returns
 * SEQATTN_ERR_TIMEOUT if a kernel gave up a bounded wait since the last
 * check, SEQATTN_ERR_CUDA if the synchronisation failed, else SEQATTN_OK. */
seqattn_status seqattn_sync_status(seqattn_stream_t stream);

/* Limit, in SM clock cycles, of every bounded device-side wait in the kernels
 * launched after this call from any host thread of the process; cycles <= 0
 * restores the default (2e9 cycles, about one second).  This is the knob that
 * lets a caller (or a test) see the timeout path work without a GPU fault: a
 * launch with a limit far below the microseconds its waits normally take has
 * its waits run out, its CTAs let every copy and MMA already issued complete,
 * release their tensor memory and return, and the next seqattn_sync_status()
 * reports SEQATTN_ERR_TIMEOUT; outputs of such a launch are unspecified.
 * Limits below 65536 cycles also make the forward's waits spin instead of
 * sleeping in the barrier.  Pure host function (takes effect at the next
 * launch). */
void seqattn_set_wait_limit(int64_t cycles);

/* Static description of a status code.  Pure host function. */
const char* seqattn_status_string(seqattn_status s);

/* Human-readable reason for the most recent non-OK status returned on the
 * calling host thread ("" if none).  Pure host function. */
const char* seqattn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SEQATTN_H */
