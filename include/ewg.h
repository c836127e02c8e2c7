/*
 * ewg.h -- C ABI of the GB300 sparse embedding weight-gradient library, and of the
 * operators that a training step has beside it: token log probabilities with their
 * gradient (ewg_token_logprobs, the vocabulary's other end), the orthogonalised update of
 * a matrix (ewg_orthogonalize), layer norm with its gradient (ewg_layer_norm) and the AdamW
 * step of many tensors at once (ewg_adamw_step).
 *
 * The operation (Megatron Core API docs, core.fusions.fused_embedding_wgrad,
 * entry accumulate_embedding_wgrad, and the module docstring):
 *
 *     main_grad += embedding_dense_backward(grad, ids)
 *
 * touching only the rows of the ids that occur.  The values are those of PyTorch's
 * sort-based embedding backward followed by main_grad.add_ (module docstring,
 * both bullets): the (token, position) pairs are sorted; each token's gradient rows
 * are summed in position order into fp32 partial sums of at most EWG_NROWS rows,
 * chunked from the token's first row; the partial sums are added in order starting
 * from 0; the total is rounded once to the gradient dtype; that value is added to
 * the main_grad row in fp32 and rounded to main_grad's dtype.  Rows of ids that do
 * not occur are neither read nor written (module docstring, last sentence).
 * Every rounding is IEEE round-to-nearest-even; results are deterministic and
 * independent of the launch configuration.
 *
 * Conventions for every entry point below:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or keeps them.  All tensors must live on the current
 *     CUDA device.
 *   - "stream" is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *     Work is enqueued on it and the call returns without waiting for it.
 *   - Errors a host check can find are returned BEFORE anything is enqueued, so
 *     main_grad is untouched.  Errors found on the device (an id outside
 *     [0, num_embeddings)) make every kernel of the call skip all writes to
 *     main_grad; ewg_read_status() reports them.
 *   - No C++ exception crosses this boundary.  Entry points are thread-safe; two
 *     calls that share a workspace or a main_grad must be ordered by the caller
 *     (same stream, or events).
 */
#ifndef EWG_H_
#define EWG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Fewest tokens accepted: PyTorch's embedding backward takes its sort-based path,
 * whose arithmetic this library reproduces, only above 3072 tokens (module
 * docstring, first bullet; MIN_TOKENS = 3073 on the same page). */
#define EWG_MIN_TOKENS 3073
/* Most tokens accepted.  The page's own limit is 8192 (MAX_TOKENS), set by its
 * single-program sort; this library sorts across many CTAs and keeps 32-bit slot
 * indices, so it accepts up to 2^28 tokens. */
#define EWG_MAX_TOKENS (1 << 28)
/* Partial-sum chunk length (NROWS on the page, NROWS_PER_THREAD in PyTorch). */
#define EWG_NROWS 10
/* Largest hidden size accepted. */
#define EWG_MAX_HIDDEN (1 << 24)

/* Element types (ewg_dtype). */
#define EWG_INT32 0
#define EWG_INT64 1
#define EWG_BF16 2
#define EWG_FP32 3

/* Status codes (ewg_status). */
#define EWG_OK 0
#define EWG_ERR_UNSUPPORTED 1     /* tensors outside what ewg_can_accumulate accepts */
#define EWG_ERR_INVALID 2         /* bad argument: NULL, size, workspace too small, plan mismatch */
#define EWG_ERR_CUDA 3            /* a CUDA runtime call or kernel launch failed */
#define EWG_ERR_ID_OUT_OF_RANGE 4 /* device-detected: an id outside [0, num_embeddings) */
#define EWG_ERR_TIMEOUT 5         /* device-detected: a bounded wait in a kernel gave up;
                                     touched main_grad rows are then unspecified */
#define EWG_ERR_BOUNDS 6          /* device-detected, bounds-checking build (libewg_debug.so)
                                     only: an index a kernel derived from the plan was out of
                                     range; the access was replaced by a safe one, so
                                     main_grad's touched rows are then unspecified */

/*
 * Whether ewg_accumulate supports these tensors (can_accumulate_embedding_wgrad on
 * the page).  Returns 1 or 0 and never enqueues work.
 *
 *   ids        [num_tokens] contiguous, ids_dtype EWG_INT32 or EWG_INT64.  A
 *              multi-dimensional ids tensor is passed flattened in row-major order;
 *              token position p is its flat index.
 *   grad       [num_tokens][hidden], grad_dtype EWG_BF16 or EWG_FP32, unit inner
 *              stride, grad_row_stride elements between rows (>= hidden).
 *   main_grad  [num_embeddings][hidden], EWG_BF16 or EWG_FP32, unit inner stride,
 *              main_grad_row_stride elements between rows (>= hidden).
 *
 * Conditions: EWG_MIN_TOKENS <= num_tokens <= EWG_MAX_TOKENS;
 * 1 <= num_embeddings < 2^31; 8 <= hidden <= EWG_MAX_HIDDEN and hidden % 8 == 0;
 * grad, main_grad and their row strides 16-byte aligned; ids aligned to its element;
 * all three pointers are device (or managed) memory of the current device;
 * main_grad does not overlap grad or ids.  The page's further conditions (Triton
 * present, ids and positions packing into 31 bits, at most 8192 tokens) belong to
 * its own implementation and are not imposed here.
 */
int ewg_can_accumulate(const void* ids, int ids_dtype, int64_t num_tokens,
                       const void* grad, int grad_dtype, int64_t grad_row_stride,
                       const void* main_grad, int main_grad_dtype,
                       int64_t num_embeddings, int64_t hidden,
                       int64_t main_grad_row_stride);

/*
 * Bytes of device workspace that ewg_accumulate / ewg_plan / ewg_apply need for
 * num_tokens tokens of width hidden (an upper bound over every id pattern).  The page
 * has no counterpart: its function allocates its own scratch, while this library leaves
 * every allocation to the caller.  The workspace needs no initialisation and holds no
 * state the caller must keep between calls, except that ewg_apply reads the plan that
 * ewg_plan left in it and ewg_read_status reads the status of the last call.  Returns 0
 * for sizes outside the supported range.
 */
size_t ewg_workspace_bytes(int64_t num_tokens, int64_t hidden);

/*
 * main_grad += embedding_dense_backward(grad, ids), touching only the rows of ids
 * (accumulate_embedding_wgrad on the page).  Arguments as for ewg_can_accumulate,
 * plus a device workspace of at least ewg_workspace_bytes(num_tokens, hidden)
 * bytes, 256-byte aligned, and the stream.  Equivalent to ewg_plan followed by
 * ewg_apply on the same stream.
 *
 * Returns EWG_OK once the work is enqueued, EWG_ERR_UNSUPPORTED /
 * EWG_ERR_INVALID (nothing enqueued, main_grad untouched) or EWG_ERR_CUDA.
 * Out-of-range ids are found on the device: main_grad is then left untouched and
 * ewg_read_status returns EWG_ERR_ID_OUT_OF_RANGE.
 */
int ewg_accumulate(const void* ids, int ids_dtype, int64_t num_tokens,
                   const void* grad, int grad_dtype, int64_t grad_row_stride,
                   void* main_grad, int main_grad_dtype,
                   int64_t num_embeddings, int64_t hidden, int64_t main_grad_row_stride,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * The first half of ewg_accumulate (the page's _sort_tokens_kernel): validates the
 * ids on the device, sorts the (token, position) pairs, finds every token's run of
 * sorted slots and lists its chunks of at most EWG_NROWS rows, writing this plan
 * into the workspace.  Reads only ids; writes only the workspace.
 */
int ewg_plan(const void* ids, int ids_dtype, int64_t num_tokens, int64_t num_embeddings,
             int64_t hidden, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The second half of ewg_accumulate (the page's _partial_sums_kernel and
 * _long_run_sums_kernel): sums the chunks of the plan in the workspace and adds
 * each token's row into main_grad.  num_tokens, num_embeddings
 * and hidden must be those given to the ewg_plan that filled the workspace (the
 * kernel checks them against the plan and writes nothing on a mismatch, reporting
 * EWG_ERR_INVALID through ewg_read_status).  Must be ordered after that ewg_plan.
 */
int ewg_apply(const void* grad, int grad_dtype, int64_t grad_row_stride,
              void* main_grad, int main_grad_dtype, int64_t num_tokens,
              int64_t num_embeddings, int64_t hidden, int64_t main_grad_row_stride,
              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Vocabulary-sharded ewg_accumulate: main_grad holds only the rows
 * [row_begin, row_begin + shard_rows) of the [num_embeddings, hidden] table (its row 0 is
 * table row row_begin), and the call updates exactly the rows of that range that
 * ewg_accumulate would update, with the same bits.  Ids in [0, num_embeddings) outside
 * the range are skipped; ids outside [0, num_embeddings) are errors as in
 * ewg_accumulate.
 *
 * The page has no entry point of its own for this.  It follows from the module
 * docstring of core.fusions.fused_embedding_wgrad: a row's result depends only on that
 * token's own rows, in position order, and rows of absent tokens are not touched, so
 * the rows of a range are computed the same way whatever happens to the other rows.
 * One GPU per range of rows then needs no exchange.
 *
 * ids, grad: as in ewg_accumulate (all num_tokens tokens; the support condition on
 * num_tokens is that of the whole call).  main_grad: shard_rows rows of hidden
 * elements, row stride main_grad_row_stride.  Requires 0 <= row_begin,
 * 1 <= shard_rows and row_begin + shard_rows <= num_embeddings (else
 * EWG_ERR_UNSUPPORTED before anything is enqueued).  Workspace, stream and errors:
 * as ewg_accumulate.
 */
int ewg_accumulate_shard(const void* ids, int ids_dtype, int64_t num_tokens,
                         const void* grad, int grad_dtype, int64_t grad_row_stride,
                         void* main_grad, int main_grad_dtype, int64_t num_embeddings,
                         int64_t row_begin, int64_t shard_rows, int64_t hidden,
                         int64_t main_grad_row_stride, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * The first half of ewg_accumulate_shard: ewg_plan keeping only the ids in
 * [row_begin, row_begin + shard_rows), renumbered from 0.  The ewg_apply that follows
 * takes num_embeddings = shard_rows and the shard's main_grad.
 */
int ewg_plan_shard(const void* ids, int ids_dtype, int64_t num_tokens,
                   int64_t num_embeddings, int64_t row_begin, int64_t shard_rows,
                   int64_t hidden, void* workspace, size_t workspace_bytes, void* stream);

/*
 * ewg_accumulate with ids and grad in pinned host memory (the page's function takes
 * device tensors; this is the same call for a caller whose inputs start on the host).
 *
 * ids_host: num_tokens ids (EWG_INT32 or EWG_INT64), contiguous; grad_host:
 * [num_tokens, hidden] (EWG_BF16 or EWG_FP32), contiguous (row stride = hidden).  Both
 * must be page-locked host memory (cudaHostAlloc / cudaHostRegister / a pinned torch
 * tensor), else EWG_ERR_UNSUPPORTED.  main_grad: a device matrix as in ewg_accumulate.
 * workspace: device memory of at least ewg_host_workspace_bytes(...) bytes; it receives
 * the copies of ids and grad next to the ordinary workspace.
 *
 * Stream-ordered on `stream`: the ids are copied and planned on `stream` while the grad
 * copy runs on a library-owned stream of the device (made on the first call, after the
 * work already queued on `stream`); the apply waits for both.  Calls on one device from
 * several host threads are serialised by the library while they enqueue.  Errors and
 * the device status: as ewg_accumulate (ewg_read_status on the same workspace).
 *
 * The copies read ids_host and grad_host after the call has returned: both buffers must
 * stay allocated and unchanged until `stream` has passed this call (synchronize it, or
 * wait on an event recorded on it after the call).
 *
 * The library keeps ONE copy stream per device for every caller stream, so the grad
 * copy of a call waits for the grad copies of earlier host-input calls on the same
 * device, whatever stream those were made on.
 */
size_t ewg_host_workspace_bytes(int64_t num_tokens, int64_t hidden, int ids_dtype,
                                int grad_dtype);
int ewg_accumulate_host(const void* ids_host, int ids_dtype, int64_t num_tokens,
                        const void* grad_host, int grad_dtype, void* main_grad,
                        int main_grad_dtype, int64_t num_embeddings, int64_t hidden,
                        int64_t main_grad_row_stride, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Size of the library-owned scratch used by ewg_accumulate_static (64 MiB). */
#define EWG_STATIC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * ewg_accumulate without a caller workspace and without any allocation.  The page
 * (Megatron Core API docs, core.fusions.fused_embedding_wgrad) has no counterpart: this
 * is an addition for callers that cannot allocate.
 *
 * For callers that cannot allocate device memory when the gradient is accumulated:
 * code running under a fixed-pool or custom allocator that must not grow, and runtimes
 * that forbid cudaMalloc after start-up.  The library keeps a file-scope __device__ array of
 * EWG_STATIC_SCRATCH_BYTES as the workspace; every device that loads the library
 * holds it until the process exits.  Arguments and results are those of
 * ewg_accumulate, without the workspace.
 *
 * - Sizes whose ewg_workspace_bytes(num_tokens, hidden) exceeds
 *   EWG_STATIC_SCRATCH_BYTES are rejected with EWG_ERR_UNSUPPORTED (and
 *   ewg_last_error says so) before anything is enqueued.  64 MiB covers up to 8192
 *   tokens for hidden sizes up to about 10000.
 * - The call makes no cudaMalloc, cudaFree or other allocating call.  The first call on
 *   a device looks up the array's device address with cudaGetSymbolAddress; make that
 *   first call outside any stream capture.  Under CUDA's lazy module loading (the
 *   default) the array is reserved only then, when that lookup loads the module that
 *   holds it (with CUDA_MODULE_LOADING=EAGER, when the library is loaded): make the
 *   first call at start-up, while the device still has room for it.
 * - Every call on a device uses the same array, which keeps the last call's contents
 *   (nothing in it needs clearing between calls).  Calls that may overlap on the GPU
 *   (different streams without ordering) race on it and must not be made.
 * - If scratch_out is not NULL it receives the array's device address, which can be
 *   passed to ewg_read_status to read the device status of the call.
 */
int ewg_accumulate_static(const void* ids, int ids_dtype, int64_t num_tokens,
                          const void* grad, int grad_dtype, int64_t grad_row_stride,
                          void* main_grad, int main_grad_dtype,
                          int64_t num_embeddings, int64_t hidden,
                          int64_t main_grad_row_stride, void* stream, void** scratch_out);

/* Most alternatives ewg_token_logprobs returns per row. */
#define EWG_MAX_TOP 32

/*
 * Log probabilities of given tokens under rows of logits, with the entropy of each row's
 * distribution and its most likely tokens.  Per row z[0..vocab) with token t,
 * m = max z, x_v = scale (z_v - m), and R the sum of exp(x_v) without one occurrence of
 * the maximum:
 *
 *     log_sum = log1p(R)         logprobs = x_t - log_sum
 *     entropy = log_sum - sum_v exp(x_v) x_v / (1 + R)         row_max = m
 *     top_ids, top_logprobs: the `top` largest logits, best first, equal ones by lower id
 *
 * in 32 bits, the row's sums held relative to its maximum; near-certain tokens keep the
 * relative precision of their small -logprob and entropy (exponentials below 2^-126 are 0).
 *
 *   logits    [num_tokens][vocab], EWG_BF16 or EWG_FP32, unit inner stride,
 *             row_stride elements between rows (>= vocab; any alignment of the element)
 *   targets   [num_tokens] contiguous, EWG_INT32 or EWG_INT64
 *   logprobs, entropy, row_max, log_sum     [num_tokens] fp32
 *   top_logprobs, top_ids     [num_tokens][top] fp32 and int64 (both unused for top = 0)
 *
 * A logit of -inf is a token that cannot occur.  A row of nothing else has log_sum 0,
 * row_max -inf, entropy 0 and logprobs -inf; missing alternatives are id -1 at -inf.  A
 * row with a NaN or +inf has NaN logprobs, entropy and log_sum.  A negative target marks a
 * row without a token (padding): its logits may be anything, its alternatives are missing
 * and its other outputs are 0.  A target of vocab or more makes the row's logprobs NaN and
 * the device status EWG_ERR_ID_OUT_OF_RANGE.
 *
 * Requires 0 <= num_tokens < 2^31 (0: nothing is enqueued, not even the status),
 * 1 <= vocab < 2^31 - 64, finite scale > 0, 0 <= top <= min(vocab, EWG_MAX_TOP); outputs
 * apart from the inputs and each other.  workspace: NULL, or 256 device bytes, 256-byte
 * aligned, that receive the device status for ewg_read_status.  Enqueues one kernel, and for
 * the status of more than 65536 short rows a memset and a kernel over the targets before it;
 * allocates nothing.
 */
int ewg_token_logprobs(const void* logits, int logits_dtype, int64_t row_stride,
                       const void* targets, int targets_dtype, int64_t num_tokens,
                       int64_t vocab, float scale, int top, float* logprobs, float* entropy,
                       float* row_max, float* log_sum, float* top_logprobs, int64_t* top_ids,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gradient of ewg_token_logprobs with respect to the logits.  With p and log p from
 * row_max and log_sum, G = grad_logprobs and E = grad_entropy (E = 0 where it is NULL):
 *
 *     grad_v = scale (G ([v = t] - p_v) - E p_v (log p_v + entropy))
 *
 * computed in 32 bits and rounded once to the logits' dtype; at the token itself
 * G (1 - p_t) is taken as -G expm1(log p_t).
 *
 * logits, targets, scale, row_max, log_sum, entropy: as given to and returned by the
 * forward call (entropy may be NULL where grad_entropy is).  grad_logits:
 * [num_tokens][vocab] of the logits' dtype, grad_row_stride elements between rows; either
 * apart from every input, or the logits themselves (same address and stride), which it
 * then replaces.  Padding rows, rows of -inf only and rows whose target is vocab or more
 * (device status EWG_ERR_ID_OUT_OF_RANGE) get zeros.  Sizes, workspace and errors: as
 * ewg_token_logprobs.
 */
int ewg_token_logprobs_backward(const void* logits, int logits_dtype, int64_t row_stride,
                                const void* targets, int targets_dtype, int64_t num_tokens,
                                int64_t vocab, float scale, const float* row_max,
                                const float* log_sum, const float* entropy,
                                const float* grad_logprobs, const float* grad_entropy,
                                void* grad_logits, int64_t grad_row_stride, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Most Newton-Schulz steps of one ewg_orthogonalize. */
#define EWG_MAX_ORTHO_STEPS 64

/*
 * Bytes of device workspace of ewg_orthogonalize for `batch` matrices of rows x cols (0 for
 * unsupported sizes).  It needs no initialisation.
 */
size_t ewg_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);

/*
 * Newton-Schulz orthogonalisation of updates, as the Muon optimiser applies it to a
 * matrix's (momentum of the) gradient.  For each matrix G, with X0 = G / |G|_F (Frobenius
 * norm; transposed where rows > cols, and back at the end), `steps` times
 *
 *     A = X X^T        X <- a X + (b A + c A^2) X
 *
 * The result is rounded to bf16.  Matrices with a smaller side up to 32 (up to 48 where the
 * larger one is at most 4096) are computed in fp32 throughout and rounded once.  For others
 * the products take fp16 operands with fp32 accumulation; X is kept to 22 bits beside its fp16
 * numbers, and the diagonals of A and of b A + c A^2 exactly to first order.  Five steps with
 * the coefficients below are then within 3e-3 of the exact steps in norm (2.4e-3 where the
 * smaller side is 256 or more), of which the rounding to bf16 is 1.7e-3, for dense updates of
 * any decay of the singular values, low-rank ones included.  Where the singular values are all
 * equal, or the singular vectors are unit vectors, the roundings of fp16 are the same all over
 * and add up: within 4e-3 for orthogonal matrices, 5e-3 for diagonal ones and 9e-3 for the
 * identity.  More steps enlarge this (measured after eight: dense updates 3.3e-3, the
 * identity 2e-2), and each multiplies by `a` what rounding leaves in directions that a low-rank
 * update does not have (after eight steps 2e-2, after twelve as much as the result).
 *
 * The norm is taken over fp32's whole range, so the scale of G does not matter; a zero matrix
 * stays zero, a NaN or an infinity makes its matrix NaN.  The same call gives the same bits; in
 * another batch, or as the transpose of a square matrix, sums may be made otherwise.
 *
 *   grad    [batch][rows][cols], EWG_BF16 or EWG_FP32, unit inner stride; any alignment
 *   out     [batch][rows][cols] bf16, unit inner stride, apart from grad
 *   strides in elements: rows >= cols apart, matrices not overlapping
 *   a, b, c the polynomial (Muon: 3.4445, -4.7750, 2.0315); singular values that it takes
 *           above 1.5 may overflow the fp16 operands
 *
 * Requires 0 <= batch <= 65535 (0: nothing is enqueued), the smaller side at most 16384 and
 * the larger at most 2^20, batch * ceil(rows / 256) * ceil(cols / 256) < 2^30,
 * 1 <= steps <= EWG_MAX_ORTHO_STEPS, finite coefficients, and a workspace as above.
 * Enqueues two small kernels and one cooperative kernel that takes every step, or small ones
 * for every two steps; allocates nothing.  ewg_read_status reports EWG_ERR_TIMEOUT if a bounded
 * wait in it gave up (out is then unspecified).
 */
int ewg_orthogonalize(const void* grad, int grad_dtype, int64_t batch, int64_t rows,
                      int64_t cols, int64_t grad_batch_stride, int64_t grad_row_stride,
                      void* out, int64_t out_batch_stride, int64_t out_row_stride, int steps,
                      float a, float b, float c, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * ewg_orthogonalize with each result transposed: out is [batch][cols][rows], rows of it
 * out_row_stride >= rows elements apart.  (For a grad that is the transpose of a row-major
 * matrix and an out that is row-major, or the other way round.)
 */
int ewg_orthogonalize_transposed(const void* grad, int grad_dtype, int64_t batch, int64_t rows,
                                 int64_t cols, int64_t grad_batch_stride,
                                 int64_t grad_row_stride, void* out, int64_t out_batch_stride,
                                 int64_t out_row_stride, int steps, float a, float b, float c,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Layer norm of rows.  Per row x[0..hidden), with mean and var of its elements:
 *
 *     rstd = 1 / sqrt(var + eps)        out_j = (x_j - mean) rstd weight_j + bias_j
 *
 * in 32 bits (the deviations are taken from the mean before they are squared, and the
 * mean's own rounding is made up for), rounded once.
 *
 *   x       [rows][hidden], EWG_BF16 or EWG_FP32, unit inner stride, row_stride elements
 *           between rows (>= hidden; any alignment of the element)
 *   weight, bias     [hidden] contiguous, both of weight_dtype (EWG_BF16 or EWG_FP32); NULL
 *           stands for ones and zeros (weight_dtype is then of no account if both are)
 *   out     [rows][hidden] of x's dtype, out_row_stride between rows; apart from every input, or
 *           x itself (same address and stride), which it then replaces
 *   mean, rstd       [rows] fp32; both NULL: not wanted (nothing goes back through the rows)
 *
 * A row with a NaN or an infinity gives NaN, and so does one whose elements' or squared
 * deviations' sum leaves fp32's range.  A row of equal elements has rstd 1 / sqrt(eps); its
 * results mean nothing with an eps of 0, or one that is not large beside the square of the mean's
 * rounding (2^-24 of the mean).
 *
 * Requires 0 <= rows < 2^31 (0: nothing is enqueued), 1 <= hidden <= EWG_MAX_HIDDEN, and an eps
 * of 0 or in [2^-126, 2^126].  Enqueues one kernel; allocates nothing.
 */
int ewg_layer_norm(const void* x, int x_dtype, int64_t rows, int64_t hidden, int64_t row_stride,
                   const void* weight, const void* bias, int weight_dtype, double eps, void* out,
                   int64_t out_row_stride, float* mean, float* rstd, void* stream);

/*
 * Bytes of device workspace of ewg_layer_norm_backward (0 for unsupported sizes).  It needs no
 * initialisation.
 */
size_t ewg_layer_norm_workspace_bytes(int64_t rows, int64_t hidden);

/*
 * The gradient of ewg_layer_norm.  With n_j = (x_j - mean) rstd and u_j = grad_j weight_j,
 *
 *     grad_x_j = rstd (u_j - avg(u) - n_j avg(u n))
 *     weight_main_grad_j += sum over rows of grad_j n_j
 *     bias_main_grad_j   += sum over rows of grad_j
 *
 * avg over the row.  Everything is computed and summed in 32 bits; grad_x is rounded once, and
 * a sum over the rows is added to its main_grad element in 32 bits and rounded to the main_grad's
 * dtype.  The order of the sums depends on rows, hidden, the arrays' alignment and the device: the
 * same call gives the same bits.
 *
 *   grad, x    [rows][hidden] of `dtype` (EWG_BF16 or EWG_FP32), unit inner stride, any alignment
 *   mean, rstd [rows] fp32, as ewg_layer_norm left them
 *   weight     [hidden] contiguous of weight_dtype, or NULL for ones
 *   grad_x     [rows][hidden] of `dtype`; apart from every input, or grad or x itself (same
 *              address and stride), which it then replaces
 *   weight_main_grad, bias_main_grad   [hidden] contiguous, both of main_grad_dtype (EWG_BF16 or
 *              EWG_FP32), apart from everything else; NULL: not wanted
 *   workspace  ewg_layer_norm_workspace_bytes(rows, hidden) device bytes, 256-byte aligned; calls
 *              that may run at the same time (two streams, two captured graphs) need one each,
 *              and main_grads of their own
 *
 * Requires sizes as ewg_layer_norm; rows = 0 enqueues nothing and leaves the main_grads as they
 * are.  Enqueues one to three kernels; allocates nothing.
 */
int ewg_layer_norm_backward(const void* grad, int64_t grad_row_stride, const void* x,
                            int64_t x_row_stride, int dtype, int64_t rows, int64_t hidden,
                            const float* mean, const float* rstd, const void* weight,
                            int weight_dtype, void* grad_x, int64_t grad_x_row_stride,
                            void* weight_main_grad, void* bias_main_grad, int main_grad_dtype,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Elements of a tensor that share a scale where AdamW's states are held in 8 bits. */
#define EWG_ADAMW_BLOCK 256

/* One tensor of an AdamW step; every pointer is device memory, contiguous. */
typedef struct ewg_adamw_tensor {
  void* param;          /* [count] of param_dtype: updated */
  const void* grad;     /* [count] of grad_dtype */
  void* exp_avg;        /* [count], fp32, or 8-bit codes (e4m3): updated */
  void* exp_avg_sq;     /* [count], fp32, or 8-bit codes of its root (e4m3): updated */
  float* scales;        /* 8 bits: [ceil(count / EWG_ADAMW_BLOCK)][2], else NULL: updated */
  void* copy;           /* [count] bf16: receives the new param rounded, or NULL */
  int64_t count;        /* elements, 0 included */
  double weight_decay;
  int param_dtype;      /* EWG_BF16 or EWG_FP32 (a copy: EWG_FP32) */
  int grad_dtype;       /* EWG_BF16 or EWG_FP32 */
} ewg_adamw_tensor;

/* Bytes of host memory of a plan for this many tensors (0 for unsupported numbers). */
size_t ewg_adamw_plan_bytes(int64_t num_tensors);

/*
 * Checks the tensors of an AdamW step and writes what ewg_adamw_step launches with into `plan`,
 * host memory of the caller's (8-byte aligned, ewg_adamw_plan_bytes(num_tensors) bytes).
 * Nothing is enqueued, and the tensors' contents are not read.  The plan holds the tensors'
 * addresses: it may be used as long as they stay allocated, on the device that was current.
 * It can be copied, and used by several threads (but steps of the same tensors that may run at
 * the same time, on two streams or in two captured graphs, would get into each other's way).
 *
 * state_bits: 32, or 8.  In 8 bits the two moments of an element are e4m3 codes: its average is
 * code * scales[element / EWG_ADAMW_BLOCK][0], and the root of its second average code *
 * scales[element / EWG_ADAMW_BLOCK][1].  States begin as zeros (codes and scales).
 *
 * Requires 0 <= num_tensors <= 2^20, counts below 2^40, finite weight_decay >= 0, pointers
 * aligned to their element (scales to 8 bytes), memory of the current device, and nothing that is
 * written overlapping anything else (a tensor listed twice among it).
 */
int ewg_adamw_plan(const ewg_adamw_tensor* tensors, int64_t num_tensors, int state_bits,
                   void* plan, size_t plan_bytes);

/*
 * One AdamW step of a plan's tensors.  Per element, in 32 bits, t the step's number (from 1):
 *
 *     g = grad_scale grad       m = beta1 m + (1 - beta1) g       v = beta2 v + (1 - beta2) g^2
 *     param = (1 - lr weight_decay) param
 *             - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *
 * and param is rounded once: what the decay takes and the update are added up first, so that a
 * decay below fp32's rounding of 1 is no less exact (a bf16 param without an fp32 master loses
 * changes below half its step).  An infinite param stays what it is (lr weight_decay <= 1).  The
 * copy is the new param in bf16.  With eps = 0 an element without a gradient so far is 0 / 0.
 *
 * States in 8 bits: after the step, which uses m and v unrounded, m and sqrt(v) are taken
 * relative to their block's scale, its largest magnitude times fl(1 / 448), and rounded to e4m3:
 * a value at share f of the way from one level to the next goes to the upper one where f + h >= 1,
 * h = frac(i A + t B) to 20 bits for element i of the tensor, A and B (for the root B and A) the
 * inverse plastic number's first two powers, 0xC13FA9A9 and 0x91E10DA5 of 2^32.  Over steps and elements h
 * runs evenly through [0, 1), so that changes smaller than a level's width, of which an
 * average over a thousand steps consists, add up instead of being rounded away.  A root above 0 is
 * not rounded to 0.  Blocks whose scale is below 2^-120 are held as zeros.  A gradient that is NaN
 * or infinite makes its element NaN, and in 8 bits, from the next step on, its block.
 *
 *   step, lr, grad_scale     their values; where the pointer beside it is not NULL, it is a device
 *           scalar (int64, fp32, fp32) that is read in the value's place (a step below 1 as 1),
 *           so that a captured call follows a schedule; apart from all that the step writes
 *
 * Requires step >= 1, finite lr >= 0, 0 <= beta1, beta2 < 1, an eps of 0 or in [2^-126, 2^126], finite
 * grad_scale.
 * Every element's result depends on its own tensor alone: the same bits in any plan.  Enqueues one
 * kernel for every 400 tensors; allocates nothing.
 */
int ewg_adamw_step(const void* plan, size_t plan_bytes, int64_t step, const int64_t* step_on_device,
                   double lr, const float* lr_on_device, double beta1, double beta2, double eps,
                   double grad_scale, const float* grad_scale_on_device, void* stream);

/*
 * Waits for `stream`, then copies the device status of the last ewg_plan /
 * ewg_apply / ewg_accumulate that used this workspace into *status (EWG_OK,
 * EWG_ERR_ID_OUT_OF_RANGE, EWG_ERR_INVALID or EWG_ERR_TIMEOUT).  Returns EWG_OK or
 * EWG_ERR_CUDA.  The page has no counterpart: there an out-of-range id stops the
 * process with a device assertion, while here it is reported through this call (the
 * device-status query of the library's boundary).
 */
int ewg_read_status(const void* workspace, void* stream, int* status);

/* Human-readable name of a status code (static storage). */
const char* ewg_status_string(int status);

/* Detail of the last error returned on the calling thread (static storage, "" if none). */
const char* ewg_last_error(void);

/* Library ABI version. */
int ewg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EWG_H_ */
