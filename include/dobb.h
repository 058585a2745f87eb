/*
 * dobb.h -- C ABI of the Dobb optimizer step on one GPU (sm_103a).
 *
 * Dobb ("Dobb: Shard-Local Preconditioning in Block-Diagonal Eigenbases",
 * arXiv 2610.39412, Abstract) keeps, for every weight matrix W (m x n, y = W x,
 * Table 6 notation), the input-activation second moment as B diagonal k x k
 * blocks (k = n / B, Table 3 caption: n^2/B entries per matrix), a complete
 * orthonormal eigenbasis of every block, and a momentum buffer.  One
 * optimizer step projects the momentum into the block bases, takes the sign
 * of the coefficients (the l_inf normalisation of Table 13), reconstructs the
 * update and applies it:
 *
 *     A_b <- beta2 A_b + (1 - beta2) X_b^T X_b / N     dobb_accumulate_moments
 *     Q_b, Lambda_b : A_b = Q_b Lambda_b Q_b^T          dobb_refresh_bases
 *     M <- beta1 M + G ; C_b = M_b Q_b ; S_b = sign(C_b) ;
 *     U_b = S_b Q_b^T ; W <- W - lr * s * U              dobb_step
 *
 * The refresh is the exact eigendecomposition of Table 15; it runs inside the
 * step call every `refresh_period` steps (Table 21 footnote a: the moment
 * reduction runs behind the backward pass, the refresh inside the optimizer
 * call).
 *
 * Conventions shared by every call
 *  - All pointers named *_dev or documented as device pointers are CUDA
 *    device memory of the device that was current at dobb_create; pointer
 *    arrays themselves (const void* const* ...) are host arrays.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Every call is asynchronous on that stream unless stated.
 *  - Matrices are row-major.  X for matrix i is N_i x n_i (one row per token).
 *    W and G are m_i x n_i in the parameter dtype; M is fp32 library state.
 *  - The library never allocates device memory after dobb_create: the state
 *    lives in a caller-provided device buffer of dobb_state_bytes() bytes,
 *    which the caller owns and must keep alive until dobb_destroy.
 *  - Errors: every call returns a dobb_status; on failure dobb_last_error()
 *    (thread-local, valid until the next call on the same thread) gives a
 *    message.  Device-side conditions (non-finite input, non-convergence)
 *    never trap: they set per-block flag bits read by dobb_get_block_flags.
 */
#ifndef DOBB_H
#define DOBB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dobb_ctx* dobb_handle;

typedef enum {
  DOBB_OK = 0,
  DOBB_ERR_INVALID_ARG = 1,   /* bad shape, pointer, size or value          */
  DOBB_ERR_CUDA = 2,          /* a CUDA runtime call failed                  */
  DOBB_ERR_NONFINITE = 3,     /* reserved for callers mapping flag bits      */
  DOBB_ERR_NOT_CONVERGED = 4, /* reserved for callers mapping flag bits      */
  DOBB_ERR_STATE = 5,         /* wrong device, buffer too small, bad handle  */
  DOBB_ERR_UNSUPPORTED = 6    /* shape outside what the kernels support      */
} dobb_status;

typedef enum { DOBB_F32 = 0, DOBB_BF16 = 1 } dobb_dtype;

/* Per-block flag bits, OR-ed on the device, cleared by dobb_clear_block_flags. */
#define DOBB_FLAG_NONFINITE_X 1u     /* accumulate saw a non-finite activation      */
#define DOBB_FLAG_NONFINITE_G 2u     /* step saw a non-finite gradient / momentum   */
#define DOBB_FLAG_NONFINITE_A 4u     /* refresh skipped (A non-finite); basis kept  */
#define DOBB_FLAG_NOT_CONVERGED 8u   /* eigensolver hit its sweep cap; basis written */

/* Which state tensor dobb_state_tensor() returns. */
typedef enum {
  DOBB_T_MOMENTS = 0,  /* A: per matrix B blocks of k x k fp32, row-major, full symmetric */
  DOBB_T_BASES = 1,    /* Q: per matrix B blocks of k x k fp32, row-major; column j is the
                          eigenvector of the j-th largest eigenvalue                         */
  DOBB_T_EIGVALS = 2,  /* Lambda: per matrix B x k fp32, descending within a block         */
  DOBB_T_MOMENTUM = 3, /* M: per matrix m x n fp32, row-major                              */
  DOBB_T_FLAGS = 4,    /* per block uint32 flag bits (all blocks of all matrices)          */
  DOBB_T_STATS = 5,    /* per block 4 fp32: ||U_b||_F^2, ||C_b||_F^2 of the last step,
                          Jacobi sweeps and rotations of the last sweep of the last refresh */
  DOBB_T_ERROR = 6     /* one uint32: nonzero if a device-side wait timed out (the step
                          that set it must be treated as failed); cleared by the caller    */
} dobb_tensor;

/* Bytes of device state for the given matrix set (m[i] x n[i], n[i] % B == 0).
 * Returns 0 if the arguments are invalid (see dobb_last_error). */
size_t dobb_state_bytes(int num_matrices, const int64_t* m, const int64_t* n, int B);

/* Create an optimizer over `num_matrices` matrices.
 *   m, n            host arrays of the matrix shapes; n[i] % B == 0, k = n/B in [1, 8192]
 *   B               blocks per matrix (same for all matrices)
 *   beta1, beta2    momentum and second-moment EMA coefficients, in [0, 1)
 *   refresh_period  T: dobb_step refreshes the bases when t % T == 0; 0 = never
 *   scale_s         update scale s (Table 9), W <- W - lr * s * U
 *   param_dtype     dtype of W and G; act_dtype dtype of X
 *   state_mem       caller-owned device buffer of at least dobb_state_bytes()
 *                   bytes, 256-byte aligned
 * Initialises A = 0, Q = I, Lambda = 0, M = 0, flags = 0, t = 0 on `stream`.
 * The handle is bound to the current CUDA device. */
dobb_status dobb_create(dobb_handle* out, int num_matrices, const int64_t* m,
                        const int64_t* n, int B, float beta1, float beta2,
                        int refresh_period, float scale_s, dobb_dtype param_dtype,
                        dobb_dtype act_dtype, void* state_mem, size_t state_bytes,
                        void* stream);

dobb_status dobb_destroy(dobb_handle h);

/* Thread-local message of the last failed call on this thread ("" if none). */
const char* dobb_last_error(void);

/* Accumulate block second moments (one grouped launch over all matrices):
 * A_b <- beta2 A_b + (1 - beta2) X_b^T X_b / N_i for every block of matrix i.
 *   X   host array of num_matrices device pointers (X[i] may be NULL to skip i)
 *   N   host array of token counts (N[i] == 0 skips matrix i) */
dobb_status dobb_accumulate_moments(dobb_handle h, const void* const* X,
                                    const int64_t* N, void* stream);

/* Recompute Q_b, Lambda_b of every block from the current A_b now (one
 * grouped launch).  Blocks whose A is non-finite keep their basis and get
 * DOBB_FLAG_NONFINITE_A. */
dobb_status dobb_refresh_bases(dobb_handle h, void* stream);

/* One optimizer step over all matrices (one grouped launch, plus the refresh
 * first when refresh_period > 0 and t % refresh_period == 0); then t += 1.
 *   W   host array of device pointers, updated in place (param_dtype)
 *   G   host array of device pointers (param_dtype) */
dobb_status dobb_step(dobb_handle h, void* const* W, const void* const* G,
                      float lr, void* stream);

/* dobb_step that also writes S = sign(C) as int8 (m_i x n_i, row-major) to
 * S_out[i] (device pointers; an entry may be NULL).  Test hook. */
dobb_status dobb_step_with_signs(dobb_handle h, void* const* W, const void* const* G,
                                 float lr, int8_t* const* S_out, void* stream);

/* Host-side step counter. */
dobb_status dobb_get_step(dobb_handle h, int64_t* t);
dobb_status dobb_set_step(dobb_handle h, int64_t t);

/* Coefficient normalisation of the update.
 * DOBB_NORM_SIGN (default): S_b = sign(C_b) ("Dobb", Abstract; l_inf).
 * DOBB_NORM_L2: "Dobb-l2" (Table 11), each column of C_b over all m rows
 *   scaled to l2 norm sqrt(m): S_b[:, j] = sqrt(m) C_b[:, j] / ||C_b[:, j]||
 *   (0 for a zero column), so U / sqrt(m) has Table 9's ||O||_F^2 = n as the
 *   sign update does.  Runs on the FP32 kernels in two passes (momentum and
 *   column norms over all rows, then the update); blocks up to 1024 wide.
 *   dobb_step's optional sign output receives sign(C_b).
 * DOBB_ERR_INVALID_ARG for another value, DOBB_ERR_UNSUPPORTED for wider
 * blocks. */
enum { DOBB_NORM_SIGN = 0, DOBB_NORM_L2 = 1 };
dobb_status dobb_set_normalization(dobb_handle h, int norm);

/* Which axis of a weight the blocks and moments cover ("Dobb", Tables
 * 12-13).  `matrix` is an index, or -1 for every matrix.
 * DOBB_SIDE_INPUT (default): Dobb.  The matrix registered as (m, n) is the
 *   caller's W (m x n, row-major); blocks split its n input columns and
 *   dobb_accumulate_moments takes input activations X (N x n).
 * DOBB_SIDE_OUTPUT: "Dobb-G".  The matrix registered as (m, n) is the
 *   TRANSPOSE of the caller's weight: W, G (and the optional sign output)
 *   are n x m row-major buffers, i.e. a weight with n output rows and m
 *   input columns; blocks split its n output rows, dobb_accumulate_moments
 *   takes output gradients (N x n), and the update is C_b = Q_b^T M_b,
 *   U_b = S_b' Q_b applied from the left (S_b' the normalised C_b, a sign
 *   or, with DOBB_NORM_L2, each ROW of C_b scaled to l2 norm sqrt(m)).  The
 *   momentum buffer (dobb_state_tensor) keeps the registered m x n layout,
 *   i.e. the transpose of the caller's momentum.  The update kernels read
 *   and write the caller's buffers through the transposed index.
 * Copies the per-matrix table on `stream` and waits for it.  The side is
 * configuration, like the normalisation and the refresh method: the state
 * that dobb_get_state / dobb_set_state carry does not include it.
 * DOBB_ERR_INVALID_ARG for another side or a matrix out of range;
 * DOBB_ERR_UNSUPPORTED for a block too wide for the FP32 update kernel. */
enum { DOBB_SIDE_INPUT = 0, DOBB_SIDE_OUTPUT = 1 };
dobb_status dobb_set_side(dobb_handle h, int matrix, int side, void* stream);

/* Refresh method ("Dobb", Table 15).
 * DOBB_REFRESH_EIGH (default): complete eigendecomposition of every block,
 *   Q_b with A_b = Q_b Lambda_b Q_b^T (two-sided Jacobi), columns by
 *   descending eigenvalue.
 * DOBB_REFRESH_ORTH: `steps` orthogonal-iteration steps from the current
 *   basis (one step is the pages' principal setting): Q_b <- T R^{-1} with
 *   T = A_b Q_b and R = chol(T^T T) (Table 16: Cholesky QR; computed as
 *   CholeskyQR2 in fp32, with a shifted first pass when T^T T is not
 *   numerically positive definite); Lambda_b holds the Rayleigh quotients
 *   diag(Q_b^T A_b Q_b).  Blocks at least as wide as dobb_set_eig_grid's
 *   min_k run on the grid (batched products, a Cholesky factorisation per
 *   block, the triangular solve by 64-row panels); a block whose Gram
 *   matrix is not numerically positive definite there is redone from its
 *   old basis with the shifted passes, one CTA per block, like the narrower
 *   blocks.  A block whose QR fails keeps its basis and gets
 *   DOBB_FLAG_NOT_CONVERGED.
 * DOBB_ERR_INVALID_ARG for another method or steps < 1.  Takes effect at the
 * next refresh. */
enum { DOBB_REFRESH_EIGH = 0, DOBB_REFRESH_ORTH = 1 };
dobb_status dobb_set_refresh(dobb_handle h, int method, int steps);

/* Precision of the basis the update multiplies with ("Dobb", Table 18:
 * fp32 moment accumulation with a bf16 basis is the principal setting).
 * DOBB_F32 (default): C_b = M_b Q_b and U_b = S_b Q_b^T with the fp32 basis.
 * DOBB_BF16: every entry of Q_b is rounded once to bf16 (nearest, ties to
 * even) and the products use that basis at fp32 accuracy.  The eigensolver
 * keeps the fp32 basis as its warm start either way.  Re-packs the
 * tensor-core operand images on `stream`; DOBB_ERR_INVALID_ARG for another
 * dtype. */
dobb_status dobb_set_basis_dtype(dobb_handle h, dobb_dtype basis_dtype, void* stream);

/* Change the refresh period T of dobb_step (0 = never); the step counter is
 * kept.  DOBB_ERR_INVALID_ARG for T < 0. */
dobb_status dobb_set_refresh_period(dobb_handle h, int refresh_period);

/* Which eigensolver refreshes a block: blocks at least `min_k` wide use the
 * grid solver (every table, tile pair and panel of a sweep its own CTA, a
 * launch per phase over a batch of blocks of one width; the call then
 * synchronises `stream` once per sweep), narrower ones one CTA per block.
 * Both run the same restarted Rayleigh-Ritz two-sided Jacobi.  The same
 * threshold and batches apply to the orthogonal-iteration refresh (no
 * synchronisation there).  0 = never the grid solver; otherwise min_k >= 64.  A batch holds the blocks of one width
 * whose scratch (12 k^2 bytes each) fits `batch_bytes` (at least one block;
 * 0 = all blocks of that width).  Defaults: 64, 0.  DOBB_ERR_INVALID_ARG for
 * other values. */
dobb_status dobb_set_eig_grid(dobb_handle h, int min_k, int64_t batch_bytes);

/* Eigensolver controls: sweep cap (default 40) and the convergence
 * threshold, the relative off-diagonal norm ||off(B)||_F / ||B||_F that the
 * last sweep of B = V^T A V may leave (0 = default 2e-6). */
dobb_status dobb_set_jacobi(dobb_handle h, int max_sweeps, float tol);

/* Device pointer and byte size of a state tensor of one matrix
 * (matrix >= 0) or of the whole region over all matrices (matrix == -1). */
dobb_status dobb_state_tensor(dobb_handle h, dobb_tensor which, int matrix,
                              void** dev_ptr, size_t* bytes);

/* Number of blocks over all matrices and the index of matrix i's first block
 * (blocks are numbered matrix by matrix). */
int64_t dobb_num_blocks(dobb_handle h);
int64_t dobb_block_offset(dobb_handle h, int matrix);

/* Copy the per-block flags / stats to host memory (num_blocks entries of
 * uint32, or 4 * num_blocks floats).  Synchronises `stream`. */
dobb_status dobb_get_block_flags(dobb_handle h, uint32_t* host_out, void* stream);
dobb_status dobb_clear_block_flags(dobb_handle h, void* stream);
dobb_status dobb_get_block_stats(dobb_handle h, float* host_out, void* stream);

/* Invariant check of the current bases (one grouped launch, fp64 sums):
 * per block 3 floats ||A Q - Q Lambda||_F / ||A||_F, ||Q^T Q - I||_F,
 * ||Q Lambda Q^T - A||_F / ||A||_F written to host_out (3 * num_blocks).
 * Synchronises `stream`. */
dobb_status dobb_check_bases(dobb_handle h, float* host_out, void* stream);

/* Checkpoint: bytes of the persistent state (A, Q, Lambda, M, flags), copy
 * it to / from a caller device buffer, together with the step counter. */
size_t dobb_checkpoint_bytes(dobb_handle h);
dobb_status dobb_get_state(dobb_handle h, void* dst_dev, size_t dst_bytes,
                           int64_t* t_out, void* stream);
dobb_status dobb_set_state(dobb_handle h, const void* src_dev, size_t src_bytes,
                           int64_t t, void* stream);

/* Number of kernel launches issued by this handle since creation (host count). */
int64_t dobb_launch_count(dobb_handle h);

/* Host-side view of the grouped work lists (the scheduler) of a handle over
 * this matrix set; needs no device.  phase 0: the update tiles of a step on
 * the default path (tensor-core launches, then the FFMA rest); 1: the moment
 * units of an accumulate with bf16 activations; 2: the eigen items of a
 * refresh.  Writes min(count, cap) entries of 7 int64 to `out` (may be NULL):
 *   (launch, kind, mat_base, matrix, block, a, b)
 * launch = index of the launch in the phase's sequence, kind = 0 for the
 * tensor-core kernel (phase 0, 1) or the eigensolver (2) and 1 for the FFMA
 * kernel, mat_base = the matrix in slot 0 of that launch's pointer table;
 * (a, b) = (first row, rows) for update tiles, (first, end) 128-row slice of
 * a tensor-core moment unit, (row, column) 64-tile of an FFMA moment tile,
 * (0, 0) for eigen items.  Returns the number of entries, -1 on bad
 * arguments (see dobb_last_error). */
int64_t dobb_describe_work(int num_matrices, const int64_t* m, const int64_t* n, int B,
                           int phase, int64_t* out, int64_t cap);

/* Update-kernel selection: 0 (default) runs the tcgen05 tensor-core kernel for
 * every matrix with k % 4 == 0 and k <= 448 (and 16-byte aligned W, G) and the
 * FP32 FFMA kernel for the rest; 1 runs the FFMA kernel for all matrices.
 * Both compute the same update within the documented tolerance. */
dobb_status dobb_set_step_path(dobb_handle h, int path);

/* Re-derive the tensor-core operand images of the bases after the caller
 * wrote Q directly through dobb_state_tensor(DOBB_T_BASES).  Refresh, create
 * and dobb_set_state do this themselves. */
dobb_status dobb_sync_bases(dobb_handle h, void* stream);

/* Throughput probe for the roofline denominators (the pages have no
 * counterpart): one launch of one instruction stream on every SM,
 *   which 0: FP32 FFMA, 1: TF32 mma.sync (m16n8k8), 2: TF32 tcgen05.mma
 *   (128 x 256 x 8), 3: BF16 tcgen05.mma (128 x 256 x 16);
 * `iters` scales the work.  scratch_dev: caller device memory of at least
 * 4 * (sms * 2048) + 256 bytes for the results (which mean nothing).
 * Synchronises `stream`; returns the launch's event time in ms and its exact
 * flop count (2 per multiply-add). */
dobb_status dobb_peak_probe(int which, void* scratch_dev, size_t scratch_bytes, int iters,
                            float* ms_out, double* flops_out, void* stream);

/* Failure-detection self-test (the pages have no counterpart): one launch of
 * the bounded mbarrier wait the tensor-core kernels use, on a barrier that
 * nothing arrives on.  After timeout_ns (1 ns ... 5 s) the wait gives up, the
 * kernel ORs 0x100 into *err_dev (device memory) and returns; asynchronous on
 * `stream`.  DOBB_ERR_INVALID_ARG for a NULL pointer or a timeout out of
 * range. */
dobb_status dobb_selftest_wait_timeout(uint32_t* err_dev, uint64_t timeout_ns, void* stream);

/* ------------------------------------------------------------------------
 * Allocation-free block eigendecomposition.
 *
 * The pages have no counterpart of this call.  It exists for callers of
 * this library that cannot call cudaMalloc: runtimes whose device memory is
 * reserved up front by an arena they do not control, and plugins of
 * frameworks that forbid allocations outside their own allocator.  It runs
 * the refresh eigensolver (the restarted Rayleigh-Ritz two-sided Jacobi of
 * dobb_refresh_bases, started from the identity) on caller buffers and
 * allocates nothing: its working memory is a file-scope device array of
 * DOBB_NOALLOC_SCRATCH_FLOATS floats (16 MiB) plus small fixed work-list
 * arrays, which every GPU that loads the library holds until the process
 * exits.
 *
 *   A_dev    count symmetric k x k fp32 matrices, row-major, back to back (in)
 *   Q_dev    count k x k fp32 outputs, row-major, column j = eigenvector of
 *            the j-th largest eigenvalue (out; its contents are overwritten)
 *   lam_dev  count x k fp32 eigenvalues, descending (out)
 *            Q_dev and lam_dev must not overlap A_dev (the basis is set to
 *            the identity before A is read): DOBB_ERR_INVALID_ARG otherwise
 *   k        1 <= k <= 1024;  count 0 <= count <= 4096 and
 *            count * 3 * k * k <= DOBB_NOALLOC_SCRATCH_FLOATS, otherwise the
 *            call returns DOBB_ERR_INVALID_ARG without touching the device
 *   max_sweeps  sweep cap of the Jacobi iteration (e.g. 40)
 *   flags_host  optional host array of count uint32 (DOBB_FLAG_* bits); when
 *               non-NULL the call synchronises `stream` and fills it
 * Asynchronous on `stream` otherwise.  The first call on a device resolves
 * the device addresses of the arrays (cudaGetSymbolAddress) and configures
 * the kernel; later calls only enqueue work.  All calls share the arrays,
 * which keep the last call's contents (the call clears what must start at
 * zero): calls that overlap on the GPU race.  Errors are reported by
 * dobb_eigh_noalloc_last_error() (thread-local). */
#define DOBB_NOALLOC_SCRATCH_FLOATS (4u << 20)
dobb_status dobb_eigh_noalloc(const float* A_dev, float* Q_dev, float* lam_dev, int k, int count,
                              int max_sweeps, uint32_t* flags_host, void* stream);
const char* dobb_eigh_noalloc_last_error(void);

/* ------------------------------------------------------------------------
 * The two ends of a language model, and its gradients before a step.
 *
 * The pages have no counterpart of these calls.  They make and prepare what
 * dobb_step consumes for the token embedding and the output head: the log
 * probabilities of given tokens and their gradient with respect to the
 * logits, the embedding lookup and its gradient, and the clipping of all
 * gradients by their global norm (written in the parameter dtype that
 * dobb_step reads).  They take no handle: every call works on the current
 * device, is asynchronous on `stream`, allocates nothing, synchronises
 * nothing and keeps nothing for the next call.  Rows and tensors may start at
 * any multiple of their element size.  Sums, maxima, norms and softmax
 * statistics are held in 32 bits or more; a result of fewer bits is rounded
 * once (nearest, ties to even).  Results do not depend on the order in which
 * the GPU runs the work: the same call on the same data gives the same bits.
 * Token indices are int32 or int64 (token_bytes 4 or 8).  `flags_dev` is an
 * optional device uint32 that condition bits are OR-ed into. */
#define DOBB_FLAG_BAD_TOKEN 16u /* a token index >= vocab                       */
#define DOBB_FLAG_TIMEOUT 32u   /* a device-side wait gave up: the call's results are not valid */

/* Largest number of alternatives dobb_log_probs returns per row. */
#define DOBB_MAX_TOP_K 32

/* Log probabilities of given tokens, entropies and the most likely
 * alternatives.  With y_j = scale * logits[r][j], j < vocab:
 *   row_max[r] = max_j logits[r][j] (NaN are passed over)
 *   log_sum[r] = log sum_j exp(scale * (logits[r][j] - row_max[r]))
 *   lse[r]     = scale * row_max[r] + log_sum[r]
 *   logp[r]    = y_t - lse[r],  t = tokens[r]
 *   entropy[r] = - sum_j p_j log p_j,  p_j = exp(y_j - lse[r])
 *   top_ids[r][0 .. top_k): the indices of the top_k largest logits, largest
 *     first, ties by the lowest index (-0 equals 0, a NaN counts as larger
 *     than every number); top_logp: their log probabilities.
 * -inf logits are tokens that cannot occur.  A row of -inf alone has row_max
 * = log_sum = lse = -inf, logp -inf and entropy 0, its alternatives are
 * 0, 1, ... with -inf.  A row with a NaN or +inf logit has NaN for log_sum,
 * lse, logp, entropy and top_logp.  A token < 0 stands for none: logp 0.  A
 * token >= vocab has logp NaN and sets DOBB_FLAG_BAD_TOKEN.
 *   logits_dev  rows x vocab, row r at r * row_stride elements
 *   scale       in (0, 2^127] (the inverse temperature)
 *   top_k       0 ... min(DOBB_MAX_TOP_K, vocab)
 *   logp, lse, row_max, log_sum, entropy  rows floats each; entropy and lse
 *               may be NULL (not computed)
 *   top_ids, top_logp  rows x top_k, NULL when top_k is 0
 * rows may be 0 (nothing is done); vocab is 1 ... 2^31 - 1.
 * Many long rows are copied in ahead of the arithmetic, and the waits for those
 * copies are bounded (2 s): a row that a wait gave up on reads as a row of NaN
 * with NaN for row_max and -1 for top_ids, whether or not there are flags for
 * DOBB_FLAG_TIMEOUT, and its gradient is NaN. */
dobb_status dobb_log_probs(const void* logits_dev, dobb_dtype logits_dtype, int64_t rows,
                           int64_t vocab, int64_t row_stride, const void* tokens_dev,
                           int token_bytes, float scale, int top_k, float* logp_dev,
                           float* lse_dev, float* row_max_dev, float* log_sum_dev,
                           float* entropy_dev, int32_t* top_ids_dev, float* top_logp_dev,
                           uint32_t* flags_dev, void* stream);

/* Self-test of those bounded waits: dobb_log_probs with a limit of timeout_ns
 * (1 ns ... 5 s) and only the first loaded_rows rows copied in, so that the waits
 * for the others run out.  Unlike the call itself it may leave earlier rows
 * unfinished, too, where the limit is short.  DOBB_ERR_UNSUPPORTED for sizes that
 * are computed without such waits. */
dobb_status dobb_selftest_log_probs_timeout(const void* logits_dev, dobb_dtype logits_dtype,
                                            int64_t rows, int64_t vocab, int64_t row_stride,
                                            const void* tokens_dev, int token_bytes, float scale,
                                            int top_k, float* logp_dev, float* lse_dev,
                                            float* row_max_dev, float* log_sum_dev,
                                            float* entropy_dev, int32_t* top_ids_dev,
                                            float* top_logp_dev, uint32_t* flags_dev, void* stream,
                                            int64_t loaded_rows, uint64_t timeout_ns);

/* Gradient of dobb_log_probs with respect to the logits, for the gradients g
 * of logp, h of entropy and l of lse (rows floats each; h and l may be NULL,
 * h needs entropy_dev):
 *   dlogits[r][j] = scale * (g (1[j = t] - p_j) + l p_j
 *                            - h p_j (log p_j + entropy[r]))
 * with p_j log p_j = 0 where p_j = 0.  A row of -inf alone and, for g, a row
 * whose token is not in [0, vocab) contribute nothing (zeros); a row whose
 * log_sum is NaN gets NaN.  row_max, log_sum and entropy are those of the
 * forward call with the same scale.  dlogits_dev has the logits' dtype, row r
 * at r * out_stride elements, and may be logits_dev itself (with the same
 * stride); any other overlap with the logits is refused. */
dobb_status dobb_log_probs_backward(const void* logits_dev, dobb_dtype logits_dtype, int64_t rows,
                                    int64_t vocab, int64_t row_stride, const void* tokens_dev,
                                    int token_bytes, float scale, const float* row_max_dev,
                                    const float* log_sum_dev, const float* entropy_dev,
                                    const float* grad_logp_dev, const float* grad_entropy_dev,
                                    const float* grad_lse_dev, void* dlogits_dev,
                                    int64_t out_stride, void* stream);

/* Embedding lookup: out[t][:] = scale * weight[tokens[t]][:], computed in
 * fp32 and rounded once to out_dtype.  A token < 0 (padding) and a token >=
 * vocab give a row of zeros; the latter sets DOBB_FLAG_BAD_TOKEN.
 *   weight_dev  vocab x dim, row v at v * weight_stride elements
 *   out_dev     count x dim, row t at t * out_stride elements; it shares no
 *               memory with the weight (refused) */
dobb_status dobb_embedding(const void* weight_dev, dobb_dtype weight_dtype, int64_t vocab,
                           int64_t dim, int64_t weight_stride, const void* tokens_dev,
                           int token_bytes, int64_t count, float scale, void* out_dev,
                           dobb_dtype out_dtype, int64_t out_stride, uint32_t* flags_dev,
                           void* stream);

/* Bytes of device workspace dobb_embedding_backward needs for `count` tokens
 * (0 with a message when the sizes are invalid). */
size_t dobb_embedding_backward_bytes(int64_t count, int64_t vocab, int64_t dim);

/* Gradient of dobb_embedding with respect to the weight:
 *   dweight[v][:] = scale * sum over t with tokens[t] = v of grad[t][:]
 * (accumulate 0: every row of dweight is written, zeros for tokens that do not
 * occur) or added to dweight (accumulate 1: rows of tokens that do not occur
 * are neither read nor written; the tied embedding adds to the head's
 * gradient).  The tokens are sorted (stable) and each row's gradients summed
 * in fp32 in a fixed order that depends only on the tokens; the sum is
 * rounded once.  Tokens outside [0, vocab) contribute nothing; those >= vocab
 * set DOBB_FLAG_BAD_TOKEN.  workspace_dev is caller memory of at least
 * dobb_embedding_backward_bytes(), 256-byte aligned; it holds nothing between
 * calls.  dweight shares no memory with grad (refused).  count is 0 ... 2^31 - 1, vocab 1 ... 2^30. */
dobb_status dobb_embedding_backward(const void* grad_dev, dobb_dtype grad_dtype, int64_t count,
                                    int64_t dim, int64_t grad_stride, const void* tokens_dev,
                                    int token_bytes, int64_t vocab, float scale,
                                    void* dweight_dev, dobb_dtype dweight_dtype,
                                    int64_t dweight_stride, int accumulate, uint32_t* flags_dev,
                                    void* workspace_dev, size_t workspace_bytes, void* stream);

/* Bytes of device workspace dobb_clip_grads needs for these tensors (0 with
 * a message when the sizes are invalid). */
size_t dobb_clip_grads_bytes(int num_tensors, const int64_t* numel);

/* Global l2 norm of a set of gradients, and clipping by it:
 *   stats[2 + i] = ||G_i||,  stats[0] = norm = sqrt(sum_i ||G_i||^2)
 *   stats[1] = c = max_norm / norm if norm > max_norm, else 1
 *   out_i = c * G_i, rounded once to out_dtype[i]
 * stats_dev is 2 + num_tensors floats.  No square overflows or underflows on
 * the way: c is right wherever the norm is finite in 64 bits, below the normal
 * range of fp32, too (stats hold both rounded to fp32: a norm beyond its range
 * reads Inf, a factor below it is a subnormal number or 0).  When an entry is NaN or Inf, norm is
 * NaN or Inf, DOBB_FLAG_NONFINITE_G is set and c = 1: the gradients are passed
 * on as they are, and the caller decides.
 *   G, out     host arrays of device pointers; `out` may be NULL (norms only,
 *              max_norm is ignored and c = 1); out[i] may be G[i] (in place:
 *              nothing is written when c = 1) but no output may share memory with
 *              another gradient or output (refused; without `out` a tensor that
 *              is listed twice counts twice); an entry with numel 0 may be NULL
 *   grad_dtype, out_dtype  host arrays of num_tensors dobb_dtype values
 *   numel      host array of entry counts (0 is allowed), dense tensors
 *   max_norm   >= 0, not NaN
 * workspace_dev: at least dobb_clip_grads_bytes(), 256-byte aligned. */
dobb_status dobb_clip_grads(int num_tensors, const void* const* G, const int32_t* grad_dtype,
                            const int64_t* numel, float max_norm, void* const* out,
                            const int32_t* out_dtype, float* stats_dev, uint32_t* flags_dev,
                            void* workspace_dev, size_t workspace_bytes, void* stream);

/* Layer norm of every row, with the optional gain `weight` and offset `bias`
 * (dim entries each, param_dtype; NULL: ones, zeros):
 *   mean[r] = sum_j x[r][j] / dim,  var = sum_j (x[r][j] - mean)^2 / dim
 *   rstd[r] = 1 / sqrt(var + eps),  xh = (x - mean) rstd
 *   out[r][j] = xh weight[j] + bias[j], rounded once to out_dtype
 * Rows whose squares leave fp32 are summed scaled down: finite rows have finite
 * results.  A row with a NaN or an infinity has NaN for rstd and out.
 *   x_dev    rows x dim, row r at r * x_stride elements
 *   out_dev  rows x dim, row r at r * out_stride elements; may be x_dev itself
 *            (same dtype and stride)
 *   mean, rstd  rows floats each (what the gradient needs)
 *   eps      a positive normal number
 * Outputs share no memory with each other or with what is read (refused), but
 * for out_dev in place of x_dev.  rows may be 0; dim is 1 ... 2^30 - 1.
 * The waits for copies are bounded as dobb_log_probs' are: a row that a wait gave up on
 * has NaN for mean, rstd and out (there is no flag). */
dobb_status dobb_layer_norm(const void* x_dev, dobb_dtype x_dtype, int64_t rows, int64_t dim,
                            int64_t x_stride, const void* weight_dev, const void* bias_dev,
                            dobb_dtype param_dtype, float eps, void* out_dev,
                            dobb_dtype out_dtype, int64_t out_stride, float* mean_dev,
                            float* rstd_dev, void* stream);

/* Bytes of device workspace dobb_layer_norm_backward needs (0 with a message
 * when the sizes are invalid). */
size_t dobb_layer_norm_backward_bytes(int64_t rows, int64_t dim);

/* Gradients of dobb_layer_norm for the gradient G of out (u = G weight; mean
 * and rstd are the forward call's, x is what it read):
 *   dx[r][j] = rstd (u_j - mean(u) - xh_j mean(u xh)), in x's dtype
 *   dweight[j] = sum_r G[r][j] xh[r][j],  dbias[j] = sum_r G[r][j]
 * summed in fp32 in a fixed order, rounded once to dparam_dtype; with accumulate
 * 1 added to what dweight and dbias hold.  dx, dweight and dbias may each be
 * NULL (not computed).  dx_dev may be grad_dev or x_dev itself (same dtype and
 * stride); any other overlap of an output is refused.  workspace_dev is
 * caller memory of at least dobb_layer_norm_backward_bytes(), 256-byte aligned;
 * it holds nothing between calls.  With no rows dweight and dbias are zeros
 * (accumulate 0).  A row that a wait for its copies gave up on has NaN for dx, and
 * dweight and dbias are NaN. */
dobb_status dobb_layer_norm_backward(const void* grad_dev, dobb_dtype grad_dtype,
                                     int64_t grad_stride, const void* x_dev, dobb_dtype x_dtype,
                                     int64_t rows, int64_t dim, int64_t x_stride,
                                     const void* weight_dev, dobb_dtype param_dtype,
                                     const float* mean_dev, const float* rstd_dev, void* dx_dev,
                                     int64_t dx_stride, void* dweight_dev, void* dbias_dev,
                                     dobb_dtype dparam_dtype, int accumulate, void* workspace_dev,
                                     size_t workspace_bytes, void* stream);

/* Self-test: the dynamic shared memory in bytes that a layer norm call (backward 0)
 * or its gradients (1) launch with, 0 where they go over the rows in memory, -1
 * for sizes that are refused; *most (may be NULL): the largest that a launch may ask
 * for.  No GPU is needed. */
int64_t dobb_selftest_layer_norm_smem(int64_t rows, int64_t dim, dobb_dtype x_dtype, int64_t x_stride,
                                      dobb_dtype grad_dtype, int64_t grad_stride, int backward,
                                      int64_t* most);

/* Self-tests of the bounded waits of dobb_layer_norm and dobb_layer_norm_backward, with a
 * limit of timeout_ns (1 ns ... 5 s): rows from loaded_rows on are not copied in (but for
 * those that share a copy with an earlier one), so that the waits for them run out.
 * DOBB_ERR_UNSUPPORTED for sizes that are computed without such waits. */
dobb_status dobb_selftest_layer_norm_timeout(const void* x_dev, dobb_dtype x_dtype, int64_t rows,
                                             int64_t dim, int64_t x_stride, const void* weight_dev,
                                             const void* bias_dev, dobb_dtype param_dtype, float eps,
                                             void* out_dev, dobb_dtype out_dtype, int64_t out_stride,
                                             float* mean_dev, float* rstd_dev, void* stream,
                                             int64_t loaded_rows, uint64_t timeout_ns);
dobb_status dobb_selftest_layer_norm_backward_timeout(
    const void* grad_dev, dobb_dtype grad_dtype, int64_t grad_stride, const void* x_dev,
    dobb_dtype x_dtype, int64_t rows, int64_t dim, int64_t x_stride, const void* weight_dev,
    dobb_dtype param_dtype, const float* mean_dev, const float* rstd_dev, void* dx_dev,
    int64_t dx_stride, void* dweight_dev, void* dbias_dev, dobb_dtype dparam_dtype, int accumulate,
    void* workspace_dev, size_t workspace_bytes, void* stream, int64_t loaded_rows,
    uint64_t timeout_ns);

/* Largest number of a teacher's entries per row. */
#define DOBB_MAX_TEACHER 256

/* Distillation from a teacher's top logits.  Row r has k entries: the token
 * ids[r][i] (below 0: none) and the teacher's logit teacher[r][i] of it (logits or
 * log probabilities: only their differences count; log_probs' alternatives of
 * the teacher fit).  With p = softmax(scale * logits[r]) over the vocabulary and
 * q = softmax(teacher_scale * teacher[r]) over the row's entries:
 *   loss[r] = sum_i q_i (log q_i - log p[ids[r][i]])
 * terms with q_i = 0 (a teacher of -inf among them) are 0.  A row without
 * entries, or whose entries are all -inf, has loss 0.  An entry with q_i > 0 whose
 * logit is -inf gives a loss of +inf.  A token that occurs twice counts twice.  An
 * id >= vocab gives NaN and sets DOBB_FLAG_BAD_TOKEN.  NaN or +inf among a
 * row's logits, or the teacher's of its entries, give NaN (a row without
 * entries: 0).
 * With grad_loss (g, rows floats) and dlogits also the gradient of sum_r g loss:
 *   dlogits[r][j] = scale * g (p_j - sum_{i: ids[r][i] = j} q_i)
 * zeros in rows without entries, with an id >= vocab or with logits of -inf alone.  A
 * p_j below 2^-126 counts as 0.
 *   logits_dev  rows x vocab, row r at r * row_stride elements
 *   ids_dev     rows x k, int32 or int64 (id_bytes 4 or 8); teacher_dev rows x k
 *   k           1 ... DOBB_MAX_TEACHER
 *   scale, teacher_scale  in (0, 2^127] (inverse temperatures)
 *   loss, row_max, log_sum  rows floats each; the latter two as dobb_log_probs
 *               gives them, for dobb_distill_backward
 *   dlogits_dev rows x vocab in the logits' dtype, row r at r * out_stride
 *               elements, or NULL (then grad_loss is NULL, too); may be logits_dev
 *               itself with the same stride; any other overlap of an output is
 *               refused
 * The waits for copies are bounded as dobb_log_probs' are: a row that a wait
 * gave up on has NaN for its results, and sets DOBB_FLAG_TIMEOUT. */
dobb_status dobb_distill(const void* logits_dev, dobb_dtype logits_dtype, int64_t rows,
                         int64_t vocab, int64_t row_stride, const void* ids_dev, int id_bytes,
                         const void* teacher_dev, dobb_dtype teacher_dtype, int k, float scale,
                         float teacher_scale, float* loss_dev, float* row_max_dev,
                         float* log_sum_dev, const float* grad_loss_dev, void* dlogits_dev,
                         int64_t out_stride, uint32_t* flags_dev, void* stream);

/* Self-test of those bounded waits: dobb_distill with the gradient, a limit of
 * timeout_ns (1 ns ... 5 s), and in every group of blocks that share a row the block
 * late_part (0 for the first) copying in only the first loaded_rows rows, so that the waits
 * for the others run out.  DOBB_ERR_UNSUPPORTED for sizes that are computed without
 * such waits, DOBB_ERR_INVALID_ARG where there is no such block. */
dobb_status dobb_selftest_distill_timeout(const void* logits_dev, dobb_dtype logits_dtype,
                                          int64_t rows, int64_t vocab, int64_t row_stride,
                                          const void* ids_dev, int id_bytes, const void* teacher_dev,
                                          dobb_dtype teacher_dtype, int k, float scale,
                                          float teacher_scale, float* loss_dev, float* row_max_dev,
                                          float* log_sum_dev, const float* grad_loss_dev,
                                          void* dlogits_dev, int64_t out_stride,
                                          uint32_t* flags_dev, void* stream, int64_t loaded_rows,
                                          int late_part, uint64_t timeout_ns);

/* The gradient alone, given the row_max and log_sum of a dobb_distill call (or
 * of dobb_log_probs with the same scale) on the same logits. */
dobb_status dobb_distill_backward(const void* logits_dev, dobb_dtype logits_dtype, int64_t rows,
                                  int64_t vocab, int64_t row_stride, const void* ids_dev,
                                  int id_bytes, const void* teacher_dev, dobb_dtype teacher_dtype,
                                  int k, float scale, float teacher_scale,
                                  const float* row_max_dev, const float* log_sum_dev,
                                  const float* grad_loss_dev, void* dlogits_dev,
                                  int64_t out_stride, void* stream);

/* Sampling from rows of logits with given random numbers.  With y_j = scale *
 * logits[r][j], ordered from the largest, equal ones by the lowest index (-0
 * equals 0), the filters keep, one after the other,
 *   top_k   the first top_k entries of that order (0, or vocab and more: all)
 *   top_p   of those the entries before which less than top_p of their mass
 *           sum e^y lies (1: all)
 *   min_p   of those the entries with y >= max y + log min_p (0: all)
 * and always the first one; -inf logits (tokens that cannot occur) never.
 *   tokens[r] = the kept j with the largest y_j - log noise[r][j], equal ones
 *     by the lowest index
 *   logp[r]   = y_token - log sum_{kept} e^y
 * For noise drawn independently from the exponential distribution with mean 1
 * token j comes out with probability e^{logp}.  The comparison is made in
 * 64 bits where fp32 might decide otherwise.  top_p's sums are good to (3 W + 32) 2^-24
 * of the mass, W the mean of |y - max y| over it (2^-18 for ordinary rows; an entry whose
 * border is nearer falls on either side), and taken in a fixed order or in whole numbers: the
 * same call on the same data gives the same tokens.  Noise is a positive
 * number for each logit; 0 wins over every other, NaN and negative numbers lose
 * like +inf.  Noise of entries that are not kept is not looked at.
 *   scale   in (0, 2^127] (the inverse temperature); greedy choice is top_k 1
 *   scales, top_ks, top_ps, min_ps  rows values each, or NULL: then the one
 *           value is every row's.  In them a top_k <= 0 or a top_p that is not
 *           below 1 keeps all, a top_p <= 0 the first entry, a min_p that is not
 *           above 0 all, a min_p above 1 counts as 1.
 * A row of -inf alone has token -1 and logp -inf; a row with NaN or +inf, or a
 * scale outside (0, 2^127], token -1 and logp NaN.
 *   logits_dev  rows x vocab, row r at r * row_stride elements; noise_dev fp32,
 *               row r at r * noise_stride
 * tokens (int32) and logp (fp32), rows each, share no memory with anything else
 * (refused). */
dobb_status dobb_sample(const void* logits_dev, dobb_dtype logits_dtype, int64_t rows,
                        int64_t vocab, int64_t row_stride, const float* noise_dev,
                        int64_t noise_stride, float scale, int top_k, float top_p, float min_p,
                        const float* scales_dev, const int32_t* top_ks_dev,
                        const float* top_ps_dev, const float* min_ps_dev, int32_t* tokens_dev,
                        float* logp_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DOBB_H */
