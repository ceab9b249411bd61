/*
 * tpmlp.h -- C ABI of the t-sharded Megatron tensor-parallel MLP block on one
 * GB300 (sm_103a).
 *
 * The block (row convention, all matrices row-major):
 *   GeLU  : A_i = X W1_i,  H_i = GeLU(A_i),                    Y = sum_i H_i W2_i
 *   SwiGLU: G_i = X W1_i,  U_i = X W3_i,  H_i = U_i * Swish(G_i), Y = sum_i H_i W2_i
 * with X [T x d], W1_i / W3_i [d x d_i] (column shard i of W1 / W3),
 * W2_i [d_i x d] (row shard i of W2), H_i [T x d_i], Y [T x d] and
 * sum_i d_i = d_ff.
 *   - Column split of W1 and the identity GeLU(X [W11, W12]) =
 *     [GeLU(X W11), GeLU(X W12)]; row split of W2 and the partial-sum identity
 *     [H1, H2][W21; W22] = H1 W21 + H2 W22; the SwiGLU split: "Parallelism"
 *     tag page of Jiang Yi's homepage, post "megatron-lm", Method / FFN.
 *   - f is the identity forward and a sum (all-reduce) backward; g is a sum
 *     forward and the identity backward: same page, the f/g operator table;
 *     "Tensor parallelism" (brunomaga.github.io), Megatron_f / Megatron_g;
 *     "AI Training Network Primer" ch. 3, section 3.4, Fig. 3.4 and 3.6.
 * Optional biases (any may be NULL): b1_i [d_i] (SwiGLU also b3_i [d_i]) are
 * added to X W1_i (X W3_i) before the activation; b2 [d] is added to Y once,
 * after the g-sum, not once per shard ("Tensor parallelism",
 * brunomaga.github.io, Megatron_FeedForward: fc2 has no bias, fc2_bias is
 * added after the all-reduce).  Their gradients are sums over tokens:
 * db2 = sum_r dY[r, :], db1_i = sum_r dA_i[r, :] (SwiGLU dG_i), db3_i =
 * sum_r dU_i[r, :]; they cost one extra, HBM-bound launch per backward phase
 * that asks for them.
 * On one GPU the t shards sit side by side in HBM and both sums are
 * accumulations in the kernels' fp32 accumulators: the g-sum inside the
 * row-parallel GEMM's K loop, the f-sum inside the dX GEMM's K loop.  There
 * is no collective.
 *
 * Conventions shared by every entry point
 *   - Pointers named X, W*, H, Y, dY, dX, dW*, saved, dact, workspace are
 *     DEVICE pointers owned by the caller; the library never allocates,
 *     frees or retains them.  Arrays of pointers (const void* const* W1 ...)
 *     are HOST arrays of t device pointers, read during the call only.
 *   - Every tensor is a dense row-major 2-D array of the plan's dtype, its
 *     start 16-byte aligned; with bf16, d and every d_i must be multiples of 8
 *     (16-byte rows for the tensor-memory-access engine), with fp32 of 4.
 *   - Calls are asynchronous on the given stream (0 = the legacy default
 *     stream).  Argument errors are reported synchronously before anything
 *     is launched.  A device-side watchdog (a bounded wait inside the
 *     kernels) records TPMLP_ERR_DEVICE_TIMEOUT in the workspace's status
 *     word instead of hanging; tpmlp_check() reads and clears it.
 *   - Outputs are overwritten, never accumulated into.  Results are
 *     deterministic: every reduction has a fixed order, with no atomics
 *     on data (see tpmlp_plan_set_stream_k for the one dependence on the
 *     device's SM count).
 *   - Thread safety: a plan is immutable after creation and may be used from
 *     several threads; calls that share a workspace must be ordered on the
 *     device (same stream or events).
 */
#ifndef TPMLP_H_
#define TPMLP_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define TPMLP_API __attribute__((visibility("default")))
#else
#define TPMLP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* tpmlp_stream_t; /* == cudaStream_t */

typedef enum {
  TPMLP_OK = 0,
  TPMLP_ERR_INVALID_ARG = 1,     /* NULL pointer, bad enum value, NULL plan */
  TPMLP_ERR_SHAPE = 2,           /* T < 0, d < 1, t < 1 or > TPMLP_MAX_SHARDS, some d_i < 1 */
  TPMLP_ERR_ALIGNMENT = 3,       /* a pointer not 16-byte aligned, d or d_i not a multiple of 8 (bf16) / 4 (fp32) */
  TPMLP_ERR_UNSUPPORTED = 4,     /* device is not sm_103 (GB300) or a size beyond the kernels' limits */
  TPMLP_ERR_CUDA = 5,            /* a CUDA runtime/driver call failed; see tpmlp_last_cuda_error() */
  TPMLP_ERR_DEVICE_TIMEOUT = 6,  /* a kernel's bounded wait expired (reported by tpmlp_check) */
  TPMLP_ERR_NOT_IMPLEMENTED = 7
} tpmlp_status;

typedef enum { TPMLP_ACT_GELU = 0, TPMLP_ACT_SWIGLU = 1 } tpmlp_act;
typedef enum { TPMLP_BF16 = 0, TPMLP_FP32 = 1 } tpmlp_dtype;

#define TPMLP_MAX_SHARDS 16

/* Problem description.  d_i points to t shard widths (host memory, copied
 * by tpmlp_plan_create).  Shard i covers hidden units [o_i, o_i + d_i) with
 * o_i = d_0 + ... + d_{i-1}; widths may differ (the pages allow
 * d_1 + d_2 = d_ff with d_1 != d_2).                                          */
typedef struct {
  int64_t T;           /* tokens (b * s); may be 0 */
  int64_t d;           /* hidden size */
  int32_t t;           /* number of shards, 1 .. TPMLP_MAX_SHARDS */
  const int64_t* d_i;  /* t widths, sum = d_ff */
  tpmlp_act act;
  tpmlp_dtype dtype;   /* storage dtype of every tensor; accumulation is fp32 */
} tpmlp_desc;

typedef struct tpmlp_plan tpmlp_plan;

/* Validate desc and build a plan (host memory only).  On error *out is NULL. */
TPMLP_API tpmlp_status tpmlp_plan_create(const tpmlp_desc* desc, tpmlp_plan** out);
/* Free a plan (NULL is a no-op). */
TPMLP_API void tpmlp_plan_destroy(tpmlp_plan* plan);

/* Bytes of device workspace every call needs.  fp32 plans: a 256-byte block
 * holding the device status word (and, once a norm of the heads is set,
 * tpmlp_attn_plan_set_qk_norm_rope, the partial sums of its gains' gradients:
 * 256 bytes and 4 MB with the largest head_dim, which a program that describes the
 * heads more than once takes from the start).  bf16 plans: that block, then
 * the ticket counters and fp32 partial accumulators of the stream-K schedules (16 KB +
 * 160 x 256 KB, about 42 MB; see tpmlp_plan_set_stream_k).  The caller allocates it once,
 * zero-filled, and passes it to every call of this plan; calls that share it
 * must be ordered on the device.                                             */
TPMLP_API size_t tpmlp_workspace_size(const tpmlp_plan* plan);

/* Forward.  Inputs X [T x d]; W1[i], W3[i] (SwiGLU only; pass NULL for GeLU)
 * [d x d_i]; W2[i] [d_i x d]; optional biases b1[i], b3[i] (SwiGLU) [d_i] and
 * b2 [d] (NULL for none; b1 and b3 are arrays of t device pointers).
 * Outputs: Y [T x d]; H[i] [T x d_i]; saved =
 * the pre-activations kept for backward: GeLU t pointers A_i [T x d_i];
 * SwiGLU 2t pointers, G_0..G_{t-1} then U_0..U_{t-1}, each [T x d_i].
 * Two kernels run: the column-parallel GEMM with the activation fused into
 * its epilogue (f forward = identity: X is read by every shard), then the
 * row-parallel GEMM whose K loop walks shard 0..t-1 into one fp32
 * accumulator (the g-sum).                                                    */
TPMLP_API tpmlp_status tpmlp_forward(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                     const void* const* W3, const void* const* W2, const void* const* b1,
                                     const void* const* b3, const void* b2, void* Y, void* const* saved,
                                     void* const* H, void* workspace, tpmlp_stream_t stream);

/* Backward.  Inputs: X, W1, W3, W2 as in forward; saved and H as written by
 * tpmlp_forward; dY [T x d].  Outputs: dact = per-shard activation gradients
 * (GeLU t pointers dA_i; SwiGLU 2t pointers dG_0..dG_{t-1}, dU_0..dU_{t-1},
 * each [T x d_i]), dX [T x d], dW1[i], dW3[i] (SwiGLU only, else NULL)
 * [d x d_i], dW2[i] [d_i x d], and optionally the bias gradients db1[i],
 * db3[i] [d_i] and db2 [d] (NULL: not computed).
 * g backward is the identity (every shard reads the same dY).  Two kernels
 * run: (1) dH_i = dY W2_i^T with act' fused (writes dact) together with
 * dW2_i = H_i^T dY; (2) dX = sum_i dA_i W1_i^T (SwiGLU: + dU_i W3_i^T) with
 * the f-sum in one fp32 accumulator, together with dW1_i = X^T dA_i
 * (dW3_i = X^T dU_i).  With T = 0 the weight gradients are zero-filled.       */
TPMLP_API tpmlp_status tpmlp_backward(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                      const void* const* W3, const void* const* W2, const void* const* saved,
                                      const void* const* H, const void* dY, void* const* dact, void* dX,
                                      void* const* dW1, void* const* dW3, void* const* dW2, void* const* db1,
                                      void* const* db3, void* db2, void* workspace, tpmlp_stream_t stream);

/* Backward with recomputation: the same arguments and results as
 * tpmlp_backward, except that H is not read: the contents of H[i] may have
 * been discarded after tpmlp_forward (only X and the pre-activations in
 * saved must survive), and H[i] is used as scratch that ends up holding the
 * recomputed H_i = act(saved_i).  The first launch computes dact and writes
 * H_i from the saved pre-activations it already reads for act' (GeLU: A_i;
 * SwiGLU: U_i * Swish(G_i)); the second computes dX (the f-sum), dW1, dW3 and
 * dW2 = H_i^T dY.  This trades nothing in FLOPs for not keeping H between the
 * passes ("AI Training Network Primer" ch. 3, section 3.1, and the
 * "Parallelism" page's GPipe post: activation recomputation saves memory by
 * recomputing what the backward pass needs from what was kept).  Because H is
 * recomputed from the bf16 pre-activation rather than from the fp32
 * accumulator, dW2 may differ from tpmlp_backward's in the last bits.       */
TPMLP_API tpmlp_status tpmlp_backward_recompute(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                                const void* const* W3, const void* const* W2,
                                                const void* const* saved, void* const* H, const void* dY,
                                                void* const* dact, void* dX, void* const* dW1, void* const* dW3,
                                                void* const* dW2, void* const* db1, void* const* db3, void* db2,
                                                void* workspace, tpmlp_stream_t stream);

/* The two launches of tpmlp_forward, callable one at a time (same arguments
 * and layouts; each is exactly one kernel launch):
 *   tpmlp_forward_column: saved and H from X, W1 (and W3), b1 (and b3).
 *   tpmlp_forward_row:    Y = sum_i H_i W2_i + b2 (the g-sum in the accumulator). */
TPMLP_API tpmlp_status tpmlp_forward_column(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                            const void* const* W3, const void* const* b1, const void* const* b3,
                                            void* const* saved, void* const* H, void* workspace,
                                            tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_forward_row(const tpmlp_plan* plan, const void* const* W2, const void* b2,
                                         void* const* H, void* Y, void* workspace, tpmlp_stream_t stream);

/* tpmlp_forward_row without a workspace argument, for callers that cannot
 * allocate device memory: code handed only its input and output buffers by a
 * host framework that owns the device allocator (a plugin or an operator
 * inside someone else's runtime), or a latency-bound caller that must not
 * call cudaMalloc because it synchronises the whole device.  The pages have
 * no counterpart: it is an interface variant, not a step of the method.
 *
 * Same arguments, layouts and result as tpmlp_forward_row with b2 = NULL
 * (one launch of the row-parallel GEMM whose K loop carries the g-sum).  Its only scratch, the
 * device status word, lives in a library-owned static device array of
 * 256 bytes (held by every GPU that loads the library until the process
 * exits); the call allocates and frees nothing.  The first call on a device
 * looks up that array's device address (cudaGetSymbolAddress) with the device
 * current.  The address is
 * kept for the life of the process: after a cudaDeviceReset, which destroys
 * the device's context and the array with it, the kept address is stale, and
 * this entry point must not be called again in that process.  Each call clears
 * the status word on the stream, launches, then waits for the stream and
 * reports the kernel's status itself (TPMLP_ERR_DEVICE_TIMEOUT if a bounded
 * wait expired), so it blocks until its kernel has finished.  All calls on a
 * device share the array: calls that overlap on the GPU (other streams, other
 * host threads) race on the status word.  It never uses the stream-K tail
 * (whose flags and partial sums need the full workspace), so its results are
 * those of tpmlp_forward_row with TPMLP_STREAM_K_OFF.                       */
TPMLP_API tpmlp_status tpmlp_forward_row_noalloc(const tpmlp_plan* plan, const void* const* W2, void* const* H,
                                                 void* Y, tpmlp_stream_t stream);

/* The two launches of tpmlp_backward, callable one at a time:
 *   tpmlp_backward_dgrad: dact from dY, W2 and saved (act' fused), and dW2
 *                         from H and dY; db2 (optional) from dY.
 *   tpmlp_backward_fsum:  dX = sum_i dact_i W1_i^T (+ dU_i W3_i^T) (the
 *                         f-sum in the accumulator), dW1 and dW3 from X and
 *                         dact; db1, db3 (optional) from dact.  Must follow
 *                         tpmlp_backward_dgrad.
 * Each is one GEMM launch, plus one column-sum launch when bias gradients are
 * requested.                                                                 */
TPMLP_API tpmlp_status tpmlp_backward_dgrad(const tpmlp_plan* plan, const void* const* W2, const void* const* saved,
                                            const void* const* H, const void* dY, void* const* dact,
                                            void* const* dW2, void* db2, void* workspace, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_backward_fsum(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                           const void* const* W3, const void* const* dact, void* dX,
                                           void* const* dW1, void* const* dW3, void* const* db1, void* const* db3,
                                           void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * Sequence-parallel layout ("AI Training Network Primer" ch. 3, section 3.4,
 * Fig. 3.7): each rank of the TP group keeps a stripe of the tokens; an
 * all-gather rebuilds the full X before the block, and a reduce-scatter after
 * it sums the shards' partial outputs and gives each rank its own stripe of
 * Y; the backward pass mirrors it (all-gather of the dY stripes,
 * reduce-scatter of the partial dX).  On one GPU both collectives are layout:
 * the kernels read X and dY directly from the stripe buffers (the g- and
 * f-sums stay in the accumulators) and write each stripe's rows of Y and dX
 * into that stripe's buffer.  The activations (saved, H, dact) and all
 * weight and bias gradients keep their full layouts.
 *
 * tpmlp_plan_set_sequence_stripes: stripe j holds stripe_rows[j] >= 0
 * consecutive tokens, in token order; the rows sum to the plan's T; every
 * stripe but the first starts at a multiple of 128 tokens (no tensor-memory-
 * access box crosses a stripe).  Copied into the plan; may not be changed
 * while another call uses the plan.
 * Stripe arguments are HOST arrays of nstripes DEVICE pointers, each a dense
 * row-major [stripe_rows[j] x d] array (16-byte aligned; NULL allowed for an
 * empty stripe).  Otherwise the arguments, results and launches are those of
 * tpmlp_forward / tpmlp_backward (no recompute variant); db2 sums dY over all
 * stripes.  Without stripes set on the plan the calls fail with
 * TPMLP_ERR_INVALID_ARG.                                                      */
TPMLP_API tpmlp_status tpmlp_plan_set_sequence_stripes(tpmlp_plan* plan, int32_t nstripes,
                                                       const int64_t* stripe_rows);
TPMLP_API tpmlp_status tpmlp_forward_sp(const tpmlp_plan* plan, const void* const* X_stripes, const void* const* W1,
                                        const void* const* W3, const void* const* W2, const void* const* b1,
                                        const void* const* b3, const void* b2, void* const* Y_stripes,
                                        void* const* saved, void* const* H, void* workspace, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_backward_sp(const tpmlp_plan* plan, const void* const* X_stripes,
                                         const void* const* W1, const void* const* W3, const void* const* W2,
                                         const void* const* saved, const void* const* H,
                                         const void* const* dY_stripes, void* const* dact, void* const* dX_stripes,
                                         void* const* dW1, void* const* dW3, void* const* dW2, void* const* db1,
                                         void* const* db3, void* db2, void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention projections of the tensor-parallel self-attention block.
 *
 * Q/K/V are column-parallel (split by heads: shard i owns a subset of the
 * heads) and the output projection is row-parallel with the g-sum; the f
 * operator sums the shards' input gradients in backward ("Parallelism" tag
 * page of Jiang Yi's homepage, post "megatron-lm", Method / Attention:
 * W_Q = [W_Q1, ..., W_Qh], O = [o_1, ..., o_h] W_O; "Tensor parallelism"
 * (brunomaga.github.io), Megatron_MHA: one column-parallel QKV linear of
 * width 3 x (local heads x head size) whose output is split into q, k, v, and a
 * row-parallel output projection followed by Megatron_g; "AI Training
 * Network Primer" ch. 3, section 3.4, Fig. 3.5: with grouped-query attention
 * a shard owns 16 query heads and one key/value head).  The attention core
 * (scores, mask, softmax, the product with V) runs between these calls and is
 * not part of this library.  Neither projection has a bias (Megatron_MHA
 * builds both linears with bias=False).
 *
 * Per shard i, with dq_i = its query heads x head size, dkv_i = its key/value
 * heads x head size (dkv_i = dq_i without grouped-query attention) and
 * n_i = dq_i + 2 dkv_i:
 *   Wqkv[i] [d x n_i]  = [WQ_i | WK_i | WV_i]  (columns 0..dq_i-1 are WQ_i,
 *                        then dkv_i columns of WK_i, then dkv_i of WV_i)
 *   QKV[i]  [T x n_i]  = X Wqkv[i]             (= [Q_i | K_i | V_i])
 *   O[i]    [T x dq_i]   the attention core's output for the shard's heads
 *   WO[i]   [dq_i x d]   row shard i of the output projection
 *   Z       [T x d]    = sum_i O_i WO_i         (g: summed in the accumulator)
 * Backward, from dZ [T x d] and the core's dQKV[i] [T x n_i] =
 * [dQ_i | dK_i | dV_i]:
 *   dO[i]    = dZ WO_i^T              dWO[i]   = O_i^T dZ
 *   dX       = sum_i dQKV_i Wqkv_i^T  (f: summed in the accumulator)
 *   dWqkv[i] = X^T dQKV_i
 * Every call is one kernel launch; layouts, ownership, alignment, streams and
 * errors follow the conventions above (dq_i and dkv_i play the role of d_i).
 * The plan is an attention plan (tpmlp_attn_plan_create); passing it to an
 * MLP entry point, or an MLP plan here, is TPMLP_ERR_INVALID_ARG.  With T = 0
 * the weight gradients are zero-filled.                                       */
typedef struct {
  int64_t T;             /* tokens (b * s); may be 0 */
  int64_t d;             /* hidden size */
  int32_t t;             /* number of shards, 1 .. TPMLP_MAX_SHARDS */
  const int64_t* dq_i;   /* t query widths (host memory, copied) */
  const int64_t* dkv_i;  /* t key/value widths (host memory, copied) */
  tpmlp_dtype dtype;
} tpmlp_attn_desc;

/* Validate desc and build an attention plan (destroy with tpmlp_plan_destroy;
 * its workspace size is tpmlp_workspace_size's).                              */
TPMLP_API tpmlp_status tpmlp_attn_plan_create(const tpmlp_attn_desc* desc, tpmlp_plan** out);
/* QKV[i] = X Wqkv[i] for every shard (f forward is the identity). */
TPMLP_API tpmlp_status tpmlp_attn_qkv_forward(const tpmlp_plan* plan, const void* X, const void* const* Wqkv,
                                              void* const* QKV, void* workspace, tpmlp_stream_t stream);
/* Z = sum_i O[i] WO[i], the g-sum inside one fp32 accumulator. */
TPMLP_API tpmlp_status tpmlp_attn_out_forward(const tpmlp_plan* plan, const void* const* WO, const void* const* O,
                                              void* Z, void* workspace, tpmlp_stream_t stream);
/* dO[i] = dZ WO[i]^T and dWO[i] = O[i]^T dZ (g backward is the identity). */
TPMLP_API tpmlp_status tpmlp_attn_out_backward(const tpmlp_plan* plan, const void* const* WO, const void* const* O,
                                               const void* dZ, void* const* dO, void* const* dWO, void* workspace,
                                               tpmlp_stream_t stream);
/* dX = sum_i dQKV[i] Wqkv[i]^T (the f-sum) and dWqkv[i] = X^T dQKV[i]. */
TPMLP_API tpmlp_status tpmlp_attn_qkv_backward(const tpmlp_plan* plan, const void* X, const void* const* Wqkv,
                                               const void* const* dQKV, void* dX, void* const* dWqkv,
                                               void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norm of the query and key heads with the position rotation, between the QKV
 * projection and the attention core, and back.
 *
 * Every head x (head_dim elements of Q_i or K_i, one token at position p):
 *   r = (mean(x^2) + eps)^(-1/2)          (norm = 0: r = 1)
 *   u = g x r                             (g: gq for queries, gk for keys; NULL: ones)
 *   pair j < rotary_dim / 2, phi = p f_j: a' = u_a cos phi - u_b sin phi
 *                                         b' = u_b cos phi + u_a sin phi
 * and the elements from rotary_dim on are u.  The partners (a, b) of pair j are
 * the elements (j, j + rotary_dim / 2) (TPMLP_ROPE_HALVES) or (2j, 2j + 1)
 * (TPMLP_ROPE_PAIRS); f_j = base^(-2j / rotary_dim), or inv_freq[j].  All in
 * fp32, rounded once to the plan's dtype.  The angle is p f_j (f_j a double)
 * taken modulo a turn exactly, for any 64-bit position, negative ones
 * included; its error in turns is at most |p f_j| 2^-53 + |p| 2^-65 + 2^-25:
 * positions beyond about 2^40 cost accuracy whatever the frequency.
 * Backward, from dy: w = dy rotated back, n = x r, s = w g:
 *   dx = r (s - n mean(s n)),   dg = sum over tokens, shards and heads of w n
 * (norm = 0: dx = w).  x is the QKV buffer as the projection wrote it: keep it
 * (norm = 0: it is not read, QKV may be NULL in the backward call).
 * A head with a NaN or an infinity spoils itself and the gain's gradient only;
 * so does one whose sum of squares passes the fp32 range (elements above about
 * 10^18).  Without a norm it spoils its pair only, or itself from rotary_dim on.
 *
 * tpmlp_attn_plan_set_qk_norm_rope describes the heads (copied into the plan,
 * inv_freq included; may not run while another call uses the plan).  Every
 * dq_i and dkv_i must be a multiple of head_dim, an even number up to 256, with
 * at most 1024 query heads and 1024 key heads over all shards; rotary_dim is
 * even, 0 (norm only) to head_dim.  With an fp32 plan and
 * norm = 1 tpmlp_workspace_size grows: query it after this call.  Errors:
 * TPMLP_ERR_INVALID_ARG (NULL, an MLP plan, unknown layout, norm not 0 or 1,
 * eps, base or inv_freq not usable), TPMLP_ERR_SHAPE, TPMLP_ERR_UNSUPPORTED
 * (head_dim above 256, or more heads).
 *
 * Forward: QK[i] = [Q_i | K_i] normed and rotated, dense [T x (dq_i + dkv_i)];
 * or in place, QK[i] == QKV[i]: then the query and key columns of the
 * [T x n_i] buffer are overwritten and its value columns left as they are
 * (the backward pass then lacks its input: for inference).  positions: T
 * 64-bit integers (device), NULL for 0 .. T - 1.  One launch.
 * Backward: dQK[i] = the core's [dQ_i | dK_i], dense [T x (dq_i + dkv_i)];
 * dQKV[i] [T x n_i] as tpmlp_attn_qkv_backward takes it.  dV (optional): t
 * dense [T x dkv_i] arrays, copied into the value columns; NULL leaves those
 * columns as they are.  dQK[i] == dQKV[i] is allowed: the query and key
 * columns of the [T x n_i] buffer are then read and overwritten.  dgq, dgk
 * [head_dim] (optional) in the plan's dtype.  One launch, and a second one when
 * a gain's gradient is asked for, which is also when workspace is needed (the
 * plan's, zero-filled or used).  Other overlaps of the [T x ...] arrays, of
 * outputs with inputs or with each other, are refused (TPMLP_ERR_INVALID_ARG).
 * A gain's gradient is added in an order that depends on the device's SM
 * count.  With T = 0 the gradients of the gains are zero-filled.              */
typedef enum { TPMLP_ROPE_HALVES = 0, TPMLP_ROPE_PAIRS = 1 } tpmlp_rope_layout;
typedef struct {
  int32_t head_dim;
  int32_t rotary_dim;
  tpmlp_rope_layout layout;
  int32_t norm;            /* 1: RMS norm, 0: rotation only (no gains then) */
  float eps;               /* > 0 with norm = 1 */
  double base;             /* > 0; read if inv_freq is NULL */
  const double* inv_freq;  /* rotary_dim / 2 radians per position (host memory, copied), or NULL */
} tpmlp_qk_desc;
TPMLP_API tpmlp_status tpmlp_attn_plan_set_qk_norm_rope(tpmlp_plan* plan, const tpmlp_qk_desc* desc);
TPMLP_API tpmlp_status tpmlp_attn_qk_norm_rope_forward(const tpmlp_plan* plan, const void* const* QKV,
                                                       const int64_t* positions, const void* gq, const void* gk,
                                                       void* const* QK, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_attn_qk_norm_rope_backward(const tpmlp_plan* plan, const void* const* QKV,
                                                        const int64_t* positions, const void* gq, const void* gk,
                                                        const void* const* dQK, const void* const* dV,
                                                        void* const* dQKV, void* dgq, void* dgk, void* workspace,
                                                        tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * Activation checkpoints in 8 bits.
 *
 * A checkpoint holds a [rows x cols] tensor in 1.0625 bytes an element: groups
 * of 16 columns of a row, an e4m3 code an element and a power of two 2^e a
 * group.  With m the group's largest magnitude, e is the smallest with
 * m <= 448 * 2^e, within [-117, 120]; a code is the e4m3 number nearest to
 * x 2^-e (ties to even; at most 240 with e = 120, so that no finite number
 * comes back as an infinity).  An element is off by at most 2^-4 of its value,
 * or 2^(e - 10) if that is more.  A group that holds a NaN or an infinity comes
 * back as NaN throughout.  Every kept value is a bf16 number, so unpacking is
 * exact in both dtypes, and packing what was unpacked gives the same codes'
 * values again.
 * Storage (tpmlp_ckpt8_size bytes, 16-byte aligned): blocks of 32 rows x 16
 * columns, 512 bytes each (a row's 16 codes after the other's), the blocks of
 * 32 rows side by side, G = ceil(cols / 16) of them; after the last block one
 * byte e + 127 per group (255: NaN), 32 per block in the blocks' order.  Bytes
 * that stand for rows past the last are neither written nor read; columns past
 * the last within a group are kept as 0.
 *
 * tpmlp_ckpt8_size: 0 for sizes below 0 or above 2^31 - 1.
 * tpmlp_ckpt8_pack / _unpack: any tensor kept between two passes (a layer's
 * input, the attention core's output, QKV).  src / dst: row stride ld >= cols
 * elements; cols and ld multiples of 8 (bf16) / 4 (fp32).  src or dst must not
 * overlap ckpt.  One launch each, none for rows = 0.
 *
 * tpmlp_forward_ckpt8: tpmlp_forward with checkpoints in saved's place: ckpt
 * are t (GeLU: A_i) or 2t (SwiGLU: G_0.., U_0..) buffers of
 * tpmlp_ckpt8_size(T, d_i) bytes, written by the column GEMM's epilogue from
 * its fp32 accumulators.  H (so Y) is that of tpmlp_forward; it is scratch
 * after the call.
 * tpmlp_backward_ckpt8: tpmlp_backward_recompute on the kept values: act' and
 * the recomputed H are taken of them, so that dact, dX, dW1, dW2 and the bias
 * gradients are those of the kept pre-activations.  H is scratch (not read).
 * Both take the plans, layouts and errors of those calls, and as many
 * launches; the plan's token stripes are not used.                           */
TPMLP_API size_t tpmlp_ckpt8_size(int64_t rows, int64_t cols);
TPMLP_API tpmlp_status tpmlp_ckpt8_pack(tpmlp_dtype dtype, int64_t rows, int64_t cols, const void* src, int64_t ld,
                                        void* ckpt, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_ckpt8_unpack(tpmlp_dtype dtype, int64_t rows, int64_t cols, const void* ckpt, void* dst,
                                          int64_t ld, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_forward_ckpt8(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                           const void* const* W3, const void* const* W2, const void* const* b1,
                                           const void* const* b3, const void* b2, void* Y, void* const* ckpt,
                                           void* const* H, void* workspace, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_backward_ckpt8(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                            const void* const* W3, const void* const* W2, const void* const* ckpt,
                                            void* const* H, const void* dY, void* const* dact, void* dX,
                                            void* const* dW1, void* const* dW3, void* const* dW2, void* const* db1,
                                            void* const* db3, void* db2, void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * The residual stream in the epilogue of the row-parallel products.
 *
 * The calls of the same name without _residual, with residual [T x d] added to
 * the product:
 *   Y = residual + sum_i H_i W2_i + b2        Z = residual + sum_i O_i WO_i
 * taken of the fp32 accumulator (after b2) and rounded once.  Y (Z) may be the
 * residual itself; an overlap of the two in any other way is refused
 * (TPMLP_ERR_INVALID_ARG).  As many launches, the same workspace and schedules.
 * The residual's gradient is dY (dZ); the other gradients are those of the calls
 * without it, so the backward passes are the same.  Not for the token-striped
 * layout.                                                                    */
TPMLP_API tpmlp_status tpmlp_forward_row_residual(const tpmlp_plan* plan, const void* const* W2, const void* b2,
                                                  const void* residual, void* const* H, void* Y, void* workspace,
                                                  tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_attn_out_forward_residual(const tpmlp_plan* plan, const void* const* WO,
                                                       const void* const* O, const void* residual, void* Z,
                                                       void* workspace, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_forward_residual(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                              const void* const* W3, const void* const* W2, const void* const* b1,
                                              const void* const* b3, const void* b2, const void* residual, void* Y,
                                              void* const* saved, void* const* H, void* workspace,
                                              tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_forward_ckpt8_residual(const tpmlp_plan* plan, const void* X, const void* const* W1,
                                                    const void* const* W3, const void* const* W2,
                                                    const void* const* b1, const void* const* b3, const void* b2,
                                                    const void* residual, void* Y, void* const* ckpt,
                                                    void* const* H, void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norm of the tokens in front of a block, with the residual stream's sum.
 *
 * Every token x of cols elements:
 *   s = x + residual              (residual NULL: s = x; the sum is kept in the
 *                                 storage type, and what is kept is normed)
 *   mu = mean(s), r = (mean((s - mu)^2) + eps)^(-1/2)   (TPMLP_NORM_RMS: mu = 0)
 *   n = (s - mu) r,  y = n gain + bias      (gain NULL: ones, bias NULL: zeros)
 * Backward, from dy and dsum, the gradient that reaches s past the norm (the
 * residual stream's; NULL: none):
 *   w = dy gain,  dx = r (w - mean(w) - n mean(w n)) + dsum   (RMS: without mean(w))
 *   dgain = sum over tokens of dy n,  dbias = sum over tokens of dy
 * All in fp32, each output rounded once to the storage type.  mu is off by a few fp32
 * roundings of mean|s|, which count in n by r times that: where a mean is 10^4 times
 * the spread, n has about three digits.  dx is the gradient of x and of the residual
 * alike.  A token with a NaN or an infinity spoils its own outputs and the gradients of
 * gain and bias only; so does one whose squares pass the fp32 range (elements above
 * about 10^17).
 *
 * Arrays are [rows x cols] with row strides ld* >= cols in elements; cols and
 * every ld a multiple of 8 (bf16) / 4 (fp32), cols at most 16384.  gain, bias,
 * dgain, dbias: [cols] in the storage type.  stats: [rows x 2] fp32, mu and r of
 * each token; forward may be given NULL, backward reads what forward wrote.
 * Forward: with a residual, sum receives s, which is the x of the backward call.
 * Backward: dgain and dbias are optional (NULL: not computed); workspace,
 * tpmlp_norm_workspace_size bytes, is needed if one of them is asked for (no
 * contents are expected).  One launch each, backward a second one for dgain and
 * dbias.
 * In place: sum may be x or residual, y may be x or residual (where sum is not that
 * array), dx may be x, dy or dsum, each with the same row stride.  Other overlaps
 * of an output with another array are refused (TPMLP_ERR_INVALID_ARG), but for
 * column slices of one buffer that share no element.  The sums over tokens are
 * added in an order that depends on the device's SM count.  With rows = 0 dgain
 * and dbias are zero-filled.                                                 */
typedef enum { TPMLP_NORM_LAYER = 0, TPMLP_NORM_RMS = 1 } tpmlp_norm_kind;
typedef struct {
  int64_t rows, cols;
  tpmlp_norm_kind kind;
  tpmlp_dtype dtype;
  float eps;            /* > 0 */
} tpmlp_norm_desc;
/* 0 for a desc that is not usable. */
TPMLP_API size_t tpmlp_norm_workspace_size(const tpmlp_norm_desc* desc);
TPMLP_API tpmlp_status tpmlp_norm_forward(const tpmlp_norm_desc* desc, const void* x, int64_t ldx,
                                          const void* residual, int64_t ldr, const void* gain, const void* bias,
                                          void* sum, int64_t lds, void* y, int64_t ldy, float* stats,
                                          tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_norm_backward(const tpmlp_norm_desc* desc, const void* x, int64_t ldx,
                                           const float* stats, const void* gain, const void* dy, int64_t lddy,
                                           const void* dsum, int64_t ldds, void* dx, int64_t lddx, void* dgain,
                                           void* dbias, void* workspace, tpmlp_stream_t stream);

/* ---------------------------------------------------------------------------
 * AdamW over many tensors at once, and the gradients' global norm.
 *
 * For every element p of every tensor, with its gradient g:
 *   f = grad_scale, or max_norm / norm where grad_scale norm > max_norm
 *   m = beta1 m + (1 - beta1) f g,   v = beta2 v + (1 - beta2) (f g)^2
 *   p = p - lr weight_decay p
 *         - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32: lr, eps, grad_scale and weight_decay have to be numbers of its range, eps and
 * a max_norm that is not 0 from 2^-126 on (refused otherwise).  v is held in steps of
 * 2^-149 at the least: a gradient whose (1 - beta2) (f g)^2 is below that leaves v as it
 * is, and where eps is far below such a gradient its steps are longer than the
 * formula's.  A tensor is n elements behind one another (any n, 0 too), its start
 * 16-byte aligned like every tensor here.  dtype is that of the parameters,
 * grad_dtype the gradients'.  master (NULL, or an array; bf16 parameters only): an
 * fp32 copy of each parameter, which is what is updated; the parameter is then
 * written only, rounded once.  Without masters a bf16 parameter loses what is
 * below half its last place.
 *
 * tpmlp_grad_norm: norm (one fp32, device) = the root of the sum of the squares
 * of all gradients (without grad_scale), the same on every run; squares in fp32, so
 * that gradients beyond 10^19 give an infinity, and those below 10^-19 lose digits, below
 * 10^-23 all of them.  workspace:
 * tpmlp_grad_norm_workspace_size() bytes, zero-filled or used by this call before.
 * tpmlp_adamw_step: norm (device, or NULL for no norm) is what that call wrote.
 * A norm that is NaN or an infinity skips the step: nothing is written.  So does one that
 * grad_scale takes past the fp32 range, unless max_norm clips it.
 *
 * Moments.  TPMLP_ADAMW_32: n fp32 each.  TPMLP_ADAMW_8: groups of 256 elements,
 * the last one filled up with zeros; M a group's largest magnitude and e =
 * floor(log2 M), one more where M > 1.875 2^e, at least -90.  A code c stands for
 * (1 + (c % 8) / 8) 2^(c / 8) 2^(e - S), for 0 if c = 0: m has 7 bits and its sign
 * in bit 7 (S = 15), v 8 bits (S = 31).  Storage: the groups' 256 codes each, then
 * a byte e + 91 per group (0: all zero; 255: a NaN, an infinity or more than 2^127
 * in the group, which comes back as NaN throughout).  Rounding is stochastic: with r,
 * 16 random bits of the element, the upper one of the two neighbours is taken where
 * the distance from the lower, over the gap, is at least 1 - r / 2^16.  Below the smallest
 * code (1.125 2^(e - S)) m is kept as that code where 2^16 |m| > 2^(e - S) 1.125 r, else as
 * 0, and a v above 0 as that code.  r of element i of a tensor: with h(x) the hash
 * x = (x ^ x >> 16) 0x7feb352d, x = (x ^ x >> 15) 0x846ca68b, x ^ x >> 16 in 32 bits,
 * key = h(h(h(h(seed lo) ^ seed hi) ^ t lo) ^ t hi), q the group's number counted
 * over all tensors, a = h(h(key ^ q lo) ^ q hi), l = i % 256: the low (l even) or high
 * half of h(a + (l / 2) 0x9e3779b9).  The step itself uses m and v before they are
 * rounded.  Moments that are all zero bytes are 0, as before the first step.
 * tpmlp_adamw_state_size: bytes of one moment of n elements (0 for n out of
 * range).  tpmlp_adamw8_unpack: the values of 8-bit moments, as bf16 (exact); m_out
 * or v_out may be NULL.
 *
 * step is t, from 1 on.  step_device (NULL: none): t is read from this 64-bit
 * integer on the device instead, and lr_device (NULL: none) likewise, so that a
 * captured call goes on counting.  weight_decay: one number per tensor, or NULL
 * for 0.  Outputs (parameters, masters, moments, norm) that overlap one another or
 * an input are refused (TPMLP_ERR_INVALID_ARG).  One launch per 400 tensors.    */
typedef enum { TPMLP_ADAMW_32 = 0, TPMLP_ADAMW_8 = 1 } tpmlp_adamw_states;
typedef struct {
  int32_t n;              /* tensors, >= 0 */
  const int64_t* sizes;   /* n numbers of elements (host memory) */
  tpmlp_dtype dtype;
  tpmlp_dtype grad_dtype;
  tpmlp_adamw_states states;
} tpmlp_adamw_desc;
typedef struct {
  double lr, beta1, beta2; /* beta1, beta2 in [0, 1) */
  double eps;              /* >= 2^-126 */
  double grad_scale;       /* finite, >= 0 */
  double max_norm;         /* 0: no clipping; needs norm otherwise */
  int64_t step;            /* >= 1 (not read with step_device) */
  uint64_t seed;           /* of the 8-bit moments' rounding */
  const float* lr_device;
  const int64_t* step_device;
} tpmlp_adamw_hyper;
TPMLP_API size_t tpmlp_adamw_state_size(tpmlp_adamw_states states, int64_t n);
TPMLP_API size_t tpmlp_grad_norm_workspace_size(void);
TPMLP_API tpmlp_status tpmlp_grad_norm(const tpmlp_adamw_desc* desc, const void* const* g, float* norm,
                                       void* workspace, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_adamw_step(const tpmlp_adamw_desc* desc, void* const* p, const void* const* g,
                                        float* const* master, void* const* m, void* const* v,
                                        const double* weight_decay, const tpmlp_adamw_hyper* hyper,
                                        const float* norm, tpmlp_stream_t stream);
TPMLP_API tpmlp_status tpmlp_adamw8_unpack(const tpmlp_adamw_desc* desc, const void* const* m, const void* const* v,
                                           void* const* m_out, void* const* v_out, tpmlp_stream_t stream);

/* Watchdog controls, for testing the failure path without faulting a GPU.
 * Neither may run while another call uses the plan.
 *   tpmlp_plan_set_timeout: bound, in milliseconds (>= 1), of every wait
 *     inside this plan's kernels (default 2000; the environment variable
 *     TPMLP_WAIT_TIMEOUT_MS sets the default of new plans).
 *   tpmlp_plan_set_stall_injection: with enable != 0 the tensor-core kernels
 *     of this plan load nothing, so the first wait of their MMA issuer is
 *     never satisfied and runs out after the timeout; the kernel then records
 *     TPMLP_ERR_DEVICE_TIMEOUT in the status word, every role leaves its loop,
 *     the CTAs free their TMEM and exit, and the CUDA context stays usable.
 *     Outputs are undefined while it is enabled.  The fp32 path has no waits
 *     and ignores it.  enable == 2 instead delays every part of a split
 *     stream-K tile but its first (see tpmlp_plan_set_stream_k) by 20 ms, as
 *     if their CTA pairs ran late: another part than the first then finishes
 *     the tile; results and status must be those of a run without it.      */
TPMLP_API tpmlp_status tpmlp_plan_set_timeout(tpmlp_plan* plan, uint32_t timeout_ms);
TPMLP_API tpmlp_status tpmlp_plan_set_stall_injection(tpmlp_plan* plan, int enable);

/* Stream-K schedules of the bf16 (tensor-core) launches.  A launch deals its
 * 256 x 256 tiles to the resident CTA pairs round robin; when the tile count
 * is not a multiple of the pairs, the last wave leaves pairs idle, and when
 * a launch mixes long-K weight-gradient tiles (K = T) with short ones, the
 * pairs that draw a long tile finish late.  A stream-K schedule cuts the K
 * blocks of some tiles into ranges, one per pair: every part of a split tile
 * leaves its fp32 accumulator in the workspace and takes a ticket; the part
 * that takes the last ticket adds all parts in K order and finishes the
 * tile.  No pair waits for another, so the schedule makes no assumption about
 * which pairs are resident or when they run (other kernels may share the
 * GPU).  The fixed order keeps results deterministic for a given device, but
 * they differ in rounding from the unsplit K sum (within the fp32
 * accumulation bound) and depend on the pair count, i.e. on the device's SM
 * count.
 *   TPMLP_STREAM_K_AUTO (default): per launch, the last partial wave of
 *     equal-depth tiles is split, when that shortens a pair's work by at
 *     least 2 % and 16 K blocks of 128 after charging each extra part its
 *     read-back;
 *   TPMLP_STREAM_K_ALWAYS: the last wave of every launch whose last wave has
 *     at most pairs / 2 tiles, with as many parts as fit (tests);
 *   TPMLP_STREAM_K_BALANCE: the launch's long-K weight-gradient tiles are
 *     placed last and their K blocks spread over the pairs so that every pair
 *     ends with the same estimated work (a launch without such tiles spreads
 *     all of its tiles); a range of K blocks may then end inside one tile,
 *     cover whole tiles and start inside another;
 *   TPMLP_STREAM_K_OFF: plain round robin.
 * tpmlp_forward_row_noalloc never uses it.  Not while another call uses the
 * plan.                                                                      */
#define TPMLP_STREAM_K_OFF 0
#define TPMLP_STREAM_K_AUTO 1
#define TPMLP_STREAM_K_ALWAYS 2
#define TPMLP_STREAM_K_BALANCE 3
TPMLP_API tpmlp_status tpmlp_plan_set_stream_k(tpmlp_plan* plan, int mode);

/* Synchronise the stream, read the workspace's status word and clear it.
 * Returns TPMLP_OK, TPMLP_ERR_DEVICE_TIMEOUT, or TPMLP_ERR_CUDA.               */
TPMLP_API tpmlp_status tpmlp_check(const tpmlp_plan* plan, void* workspace, tpmlp_stream_t stream);

/* Human-readable name of a status code (static string). */
TPMLP_API const char* tpmlp_status_string(tpmlp_status status);
/* The last CUDA error code seen by this thread (0 if none), for TPMLP_ERR_CUDA. */
TPMLP_API int tpmlp_last_cuda_error(void);
/* Description of the last failure on this thread (argument, CUDA or tensor
 * map error; empty string after a successful call).  Static storage per
 * thread, valid until the next call on the same thread.                      */
TPMLP_API const char* tpmlp_last_error(void);
/* ABI version: 100 * major + minor (1.01: optional biases; 1.02: attention
 * projections; 1.03: sequence-parallel layout; 1.04: stream-K tail, larger
 * bf16 workspace; 1.05: tpmlp_last_split_tiles, tpmlp_eval_activation, a
 * 16 KB counter block in the bf16 workspace).  The norm and rotation of the
 * heads, the 8-bit checkpoints, the norm of the tokens, the residual in the
 * row-parallel products and AdamW were added to 1.05; nothing of it changed. */
TPMLP_API int tpmlp_version(void);

/* Kernel launches the last compute call (tpmlp_forward, tpmlp_backward, a
 * phase or an attention entry point) on this thread made (for accounting; 0
 * before the first call).                                                    */
TPMLP_API int tpmlp_last_launch_count(void);

/* Diagnostics of the stream-K schedules (see tpmlp_plan_set_stream_k), for
 * tests that must know which output tiles were computed in parts.
 * launch_kind names a launch of the block:
 *   0 the column-parallel GEMM (tpmlp_forward_column), 1 the row-parallel
 *   GEMM with the g-sum (tpmlp_forward_row), 2 the dgrad launch
 *   (tpmlp_backward_dgrad), 3 the f-sum launch (tpmlp_backward_fsum),
 *   4..7 the attention projections' QKV forward, output forward, output
 *   backward and QKV backward.
 * Returns how many tiles the last launch of that kind made on this thread
 * split into parts (0 if none, or no such launch yet; -1 for an unknown
 * kind) and writes the first min(count, cap) of them to tiles (host memory,
 * may be NULL) as quadruples: the problem's index in its launch, the tile's
 * first output row, its first output column, and the device address of the
 * problem's first output (Y, dX, the pre-activation, dA, dG, dW1, dW2 ... as
 * the caller passed it; 0 for a token-striped output), which identifies the
 * tensor the tile belongs to.                                                */
TPMLP_API int tpmlp_last_split_tiles(int launch_kind, int64_t* tiles, int cap);

/* The activation forms of the kernels' epilogues, evaluated on plain fp32
 * device arrays of n elements (x = the pre-activation A or the gate G, y =
 * the up projection U, dh = the incoming gradient dH), so that they can be
 * checked against a reference over any set of inputs.  The bf16 tensor-core
 * epilogues compute Phi from the rational approximation of erf given as
 * formula 7.1.26 in Abramowitz & Stegun (absolute error at most 1.5e-7) and
 * the sigmoid from the fast exponential and reciprocal; the fp32 path calls
 * erff and expf.  The GeLU forms are those of GeLU(a) = a Phi(a) and
 * GeLU'(a) = Phi(a) + a phi(a); Swish is g sigmoid(g) ("Parallelism" tag page
 * of Jiang Yi's homepage, post "megatron-lm", Method / FFN and the SwiGLU
 * listing; "Tensor parallelism", brunomaga.github.io, Megatron_FeedForward's
 * F.gelu).  Outputs (device, fp32, n elements; unused ones may be NULL):
 *   TPMLP_ACT_EVAL_GELU        out0 = GeLU(x)                       (bf16 column epilogue)
 *   TPMLP_ACT_EVAL_GELU_BWD    out0 = dh GeLU'(x)                   (bf16 dgrad epilogue)
 *   TPMLP_ACT_EVAL_GELU_BWD_H  out0 = dh GeLU'(x), out1 = GeLU(x)   (same, with H recomputed)
 *   TPMLP_ACT_EVAL_SWIGLU      out0 = y Swish(x)                    (bf16 column epilogue)
 *   TPMLP_ACT_EVAL_SWIGLU_BWD  out0 = dG = dh y Swish'(x), out1 = dU = dh Swish(x)
 *   TPMLP_ACT_EVAL_SWIGLU_BWD_H  the same and out2 = y Swish(x)     (H recomputed)
 *   TPMLP_ACT_EVAL_FP32_GELU   out0 = GeLU(x), out1 = dh GeLU'(x)   (fp32 path)
 *   TPMLP_ACT_EVAL_FP32_SWIGLU out0 = y Swish(x), out1 = dG, out2 = dU (fp32 path)
 * Inputs an entry does not read may be NULL.  Asynchronous on the stream;
 * one kernel launch.  Errors: TPMLP_ERR_INVALID_ARG (unknown fn, n < 0, a
 * needed pointer NULL), TPMLP_ERR_ALIGNMENT (a pointer not 4-byte aligned),
 * TPMLP_ERR_UNSUPPORTED (not sm_103), TPMLP_ERR_CUDA.                        */
#define TPMLP_ACT_EVAL_GELU 0
#define TPMLP_ACT_EVAL_GELU_BWD 1
#define TPMLP_ACT_EVAL_GELU_BWD_H 2
#define TPMLP_ACT_EVAL_SWIGLU 3
#define TPMLP_ACT_EVAL_SWIGLU_BWD 4
#define TPMLP_ACT_EVAL_SWIGLU_BWD_H 5
#define TPMLP_ACT_EVAL_FP32_GELU 6
#define TPMLP_ACT_EVAL_FP32_SWIGLU 7
TPMLP_API tpmlp_status tpmlp_eval_activation(int fn, const float* x, const float* y, const float* dh, float* out0,
                                             float* out1, float* out2, int64_t n, tpmlp_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TPMLP_H_ */
