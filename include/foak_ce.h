/*
 * foak_ce.h -- C ABI of the GB300 (sm_103a) fused cross-entropy library.
 *
 * The operation is the loss the fms-acceleration FOAK plugin swaps into a causal
 * LM head: "Fast Cross Entropy Triton Kernels" on the fms-acceleration-foak 0.7.4
 * page (list of fused operations and kernels), called FastCrossEntropyLoss in
 * fms-acceleration PR #79 "Allow Kernels for Full FT and Non-Quantized PEFT"
 * (Description, items 4 and 5).  The pages name the kernel but print no formula;
 * this library computes the textbook softmax cross-entropy over the rows of an
 * N x V logits matrix with mean reduction over rows whose label is not
 * ignore_index:
 *
 *     lse_i = log sum_j exp(x_ij)          l_i = lse_i - x_{i, y_i}
 *     loss  = sum_{valid i} l_i / D        D = denom > 0 ? denom : n_valid
 *     dx_ij = (g / D) * (exp(x_ij - lse_i) - [j == y_i])   (0 on ignored rows)
 *
 * The chunked linear + CE call is the fused-linear form the pages name as
 * LigerFusedLinearCrossEntropy ("Running Liger Kernel Benchmarks", foak page),
 * "chunked loss" (PR #79, TODO) and FusedCrossEntropyLoss (fms-hf-tuning PR #280,
 * "Notes on FastKernels").  A caller-supplied denom is the per-token mean across
 * data-parallel ranks that PR #280 lists under LossAccelerationPlugin
 * ("--loss_across_gpus mean token"): the caller all-reduces n_valid and passes it.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Pointers marked (device) are device memory owned by the caller; the library
 *   never allocates or frees.  Host pointers are marked (host).
 * - Logits are row-major: element (i, j) is at logits[i * ld + j], ld >= V, in
 *   FOAK_BF16 (bfloat16) or FOAK_F32.  fp16 is not accepted.
 * - labels (device) are int64[N]; a label equal to ignore_index marks an ignored
 *   row.  A label outside [0, V) that is not ignore_index is an error found on the
 *   device: the row is treated as ignored and the error word gets
 *   FOAK_ERRBIT_LABEL_RANGE.  Nothing traps.
 * - stream is a cudaStream_t passed as void* (NULL = legacy default stream).  All
 *   work is enqueued asynchronously on it; nothing synchronises unless the
 *   environment variable FOAK_SYNC_CHECK=1 is set, in which case the call waits
 *   for its own work and turns a non-zero error word into FOAK_ERR_LABEL_RANGE,
 *   FOAK_ERR_TIMEOUT or FOAK_ERR_PAGE_RANGE.
 * - Problems checkable on the host return a status before anything is enqueued.
 *   A failed launch returns FOAK_ERR_CUDA.  No C++ exception crosses the ABI.
 * - Scalar outputs (loss, n_valid, err) are single device elements written by the
 *   last kernel of the call.  With n_valid == 0 and denom <= 0 the loss is 0/0 =
 *   NaN (as torch's mean reduction gives) and every gradient row is +0.0.
 * - The result is deterministic for a given input and device: the loss is the
 *   sum of the per-row float32 terms in a fixed order (each of 512 threads adds
 *   rows t, t + 512, ...; then a fixed tree) carried as a double-float (hi + lo,
 *   about 48 significant bits, Knuth's TwoSum), divided by D and rounded to float.
 */
#ifndef FOAK_CE_H
#define FOAK_CE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FOAK_CE_ABI_VERSION 1

typedef enum foak_status {
    FOAK_OK = 0,
    FOAK_ERR_INVALID_ARG = 1,   /* null/negative/misaligned argument, ld < V, ... */
    FOAK_ERR_UNSUPPORTED = 2,   /* dtype or size outside what the kernels handle */
    FOAK_ERR_LABEL_RANGE = 3,   /* (FOAK_SYNC_CHECK only) a label was out of range */
    FOAK_ERR_WORKSPACE = 4,     /* workspace missing, misaligned or too small */
    FOAK_ERR_CUDA = 5,          /* a CUDA runtime call or launch failed */
    FOAK_ERR_TIMEOUT = 6,       /* (FOAK_SYNC_CHECK only) a device wait gave up */
    FOAK_ERR_PAGE_RANGE = 7     /* (FOAK_SYNC_CHECK only) a page or slot was out of range */
} foak_status;

typedef enum foak_dtype { FOAK_F32 = 0, FOAK_BF16 = 1 } foak_dtype;

/* Bits of the device error word (int32) that calls write when err != NULL. */
#define FOAK_ERRBIT_LABEL_RANGE 1
#define FOAK_ERRBIT_TIMEOUT 2
#define FOAK_ERRBIT_PAGE_RANGE 4

/* Human-readable name of a status code (static string, never NULL). */
const char* foak_status_string(int32_t status);

/* ABI version of the loaded library (FOAK_CE_ABI_VERSION at build time). */
int32_t foak_abi_version(void);

/* Largest V the row calls accept for a dtype: 2^31 - 1 (rows past 8 CTAs x 64 KB,
 * the one-pass plans' reach, are streamed twice by one CTA).  The chunked linear +
 * CE calls take V <= 262144. */
int64_t foak_ce_max_vocab(int32_t dtype);

/*
 * Bytes of device workspace that foak_ce_forward / foak_ce_fwd_bwd need for N rows
 * (a 256-byte header plus N float32 per-row loss terms).  The workspace must be
 * 256-byte aligned and zero-filled before its first use; every call leaves the
 * header zeroed again when its work completes, so one buffer can serve any number
 * of stream-ordered calls.  Calls that share a workspace must not overlap on the
 * GPU (same stream, or ordered by events).
 */
size_t foak_ce_workspace_size(int64_t N);

/*
 * Forward: one read of each non-ignored row (an ignored row is never read).
 *   logits (device)   N x V, row stride ld (elements)
 *   dtype             FOAK_BF16 or FOAK_F32
 *   labels (device)   int64[N]
 *   ignore_index      label value of ignored rows (usually -100)
 *   denom             > 0: divide by denom (global valid-token count under data
 *                     parallelism); <= 0: divide by this call's n_valid
 *   loss (device)     float[1]: the mean loss
 *   lse (device)      float[N] or NULL: log-sum-exp per row (0 for ignored rows);
 *                     foak_ce_backward needs it
 *   row_loss (device) float[N] or NULL: per-row terms lse_i - x_{i,y_i} (0 for
 *                     ignored rows), i.e. reduction 'none'
 *   n_valid (device)  int32[1] or NULL: rows with a label in [0, V)
 *   err (device)      int32[1] or NULL: FOAK_ERRBIT_* of this call (0 = clean)
 *   workspace (device) foak_ce_workspace_size(N) bytes, see above
 */
foak_status foak_ce_forward(const void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                            int64_t N, int64_t V, int64_t ignore_index, float denom, float* loss,
                            float* lse, float* row_loss, int32_t* n_valid, int32_t* err,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward: dlogits = (exp(logits - lse) - onehot) * g / D, ignored rows +0.0.
 *   dlogits (device)  N x V with the same ld and dtype; may equal logits (in place)
 *   logits (device)   as in forward (not read on ignored rows)
 *   lse (device)      float[N] from foak_ce_forward
 *   grad_out (device) float[1]: g, the upstream gradient of the loss; NULL = 1.0
 *   denom             as in forward (<= 0: count n_valid again from labels)
 *   err (device)      int32[1] or NULL: FOAK_ERRBIT_LABEL_RANGE if a label is bad
 * Needs no workspace.
 */
foak_status foak_ce_backward(void* dlogits, const void* logits, int32_t dtype, int64_t ld,
                             const int64_t* labels, int64_t N, int64_t V, int64_t ignore_index,
                             const float* lse, const float* grad_out, float denom, int32_t* err,
                             void* stream);

/*
 * Fused forward + backward, in place: each non-ignored row is read once and its
 * gradient written over it; ignored rows are only written (+0.0).  The logits are
 * destroyed; a caller that still needs them calls forward + backward instead.
 *   g (host)          upstream gradient of the loss (1.0 for a plain mean loss,
 *                     or a loss-scale / accumulation factor)
 *   lse (device)      float[N] or NULL, as in forward
 *   other arguments   as in forward
 */
foak_status foak_ce_fwd_bwd(void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                            int64_t N, int64_t V, int64_t ignore_index, float g, float denom,
                            float* loss, float* lse, int32_t* n_valid, int32_t* err,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * The data-parallel per-token mean (fms-hf-tuning PR #280, "Early Version Of This
 * Plugin": LossAccelerationPlugin, --loss_across_gpus mean token) divides every
 * rank's share by the number of valid tokens of ALL ranks, which each rank knows
 * only after an all-reduce.  These two calls keep that exchange on the device:
 * a rank counts its valid labels into device memory, the caller sums the counts
 * across ranks in place (e.g. an NCCL all-reduce of one int64), and the fused
 * call reads the total from device memory, with no host synchronisation between.
 *
 * foak_ce_count_valid: number of rows whose label is not ignore_index and lies in
 * [0, V).
 *   labels (device)   int64[N] (may be NULL when N == 0)
 *   n_valid (device)  int64[1], 8-byte aligned: the count
 *   err (device)      int32[1] or NULL: FOAK_ERRBIT_LABEL_RANGE if a label is
 *                     neither ignore_index nor in [0, V), else 0
 * Errors: FOAK_ERR_INVALID_ARG for N < 0, V < 1, a null or misaligned pointer.
 */
foak_status foak_ce_count_valid(const int64_t* labels, int64_t N, int64_t V, int64_t ignore_index,
                                int64_t* n_valid, int32_t* err, void* stream);

/*
 * foak_ce_fwd_bwd with the denominator read from device memory: D = *denom_count
 * (int64, e.g. the all-reduced sum of every rank's foak_ce_count_valid), read by
 * the kernel when it runs, so the count may still be in flight on `stream` when
 * the call is made.  loss is then this rank's share sum_{valid i} l_i / D (the
 * ranks' losses add up to the global mean); n_valid is this call's own count.
 * With D == 0 the loss is NaN and every gradient row +0.0, as in foak_ce_fwd_bwd.
 *   denom_count (device)  int64[1], 8-byte aligned
 *   other arguments       as for foak_ce_fwd_bwd (there is no host denom)
 */
foak_status foak_ce_fwd_bwd_devdenom(void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                                     int64_t N, int64_t V, int64_t ignore_index, float g,
                                     const int64_t* denom_count, float* loss, float* lse, int32_t* n_valid,
                                     int32_t* err, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace foak_ce_fwd_bwd_host needs for N rows: a 256-byte
 * header, N float32 per-row loss terms and 256 bytes of per-chunk error words and
 * results.  256-byte aligned, zero-filled before first use, left reusable by every
 * call (the same rules as foak_ce_workspace_size).
 */
size_t foak_ce_host_workspace_size(int64_t N);

/*
 * Fused forward + backward on logits that live in HOST memory: the call copies
 * the labels and then the logits to the device in row chunks on a copy stream of
 * its own and runs the fused kernel of foak_ce_fwd_bwd on each chunk as soon as it
 * has landed (on `stream`), so the arithmetic hides under the host-to-device copy;
 * every chunk divides by the n_valid of all N rows (or denom), and one reduction
 * over all N rows in the same order as foak_ce_fwd_bwd's gives the loss.
 * This is the same mean-reduced cross-entropy and in-place gradient as the
 * FastCrossEntropyLoss kernel of the FOAK pages (fms-acceleration PR #79,
 * Description item 4); the pages fix no host interface, so this one is ours.
 *   host_logits (host)   N x V in dtype, row stride ld elements; pinned memory
 *                        (cudaHostAlloc / torch pin_memory) for a full-speed copy.
 *                        Only the first V elements of each row are copied.
 *   host_labels (host)   int64[N]
 *   dev_logits (device)  N x ld in dtype, 16-byte aligned: receives the logits and
 *                        ends holding dlogits (ignored rows +0.0)
 *   dev_labels (device)  int64[N], receives the labels
 *   host_loss (host)     float[1]; host_n_valid, host_err (host) int32[1] or NULL:
 *                        written by device-to-host copies at the end of the work on
 *                        `stream` (pinned memory keeps the call asynchronous;
 *                        read them after synchronising the stream)
 *   workspace (device)   foak_ce_host_workspace_size(N) bytes
 *   other arguments      as for foak_ce_fwd_bwd
 * Errors: as foak_ce_fwd_bwd for the arguments; FOAK_ERR_INVALID_ARG for a null
 * host or device buffer when N > 0.  Calls for the same device from several host
 * threads are serialised internally (they share the copy stream).
 */
foak_status foak_ce_fwd_bwd_host(const void* host_logits, int32_t dtype, int64_t ld, const int64_t* host_labels,
                                 int64_t N, int64_t V, int64_t ignore_index, float g, float denom,
                                 void* dev_logits, int64_t* dev_labels, float* host_loss, int32_t* host_n_valid,
                                 int32_t* host_err, void* workspace, size_t workspace_bytes, void* stream);

/*
 * RMSNorm, the "Fast RMS LayerNorm" kernel the FOAK pages list among their fused
 * operations (fms-acceleration-foak 0.7.4 page; its patch rule swaps a decoder's
 * RMSNorm module for fast_rms_layernorm).  The pages print no formula; the
 * operation is the Llama / Mistral / Granite RMSNorm, in fp32, rounded once:
 *     r_i = 1 / sqrt(mean_j X_ij^2 + eps),   Y_ij = X_ij * r_i * gamma_j
 *   X (device)      N x D in dtype (bf16 or fp32), row stride ldx elements
 *   gamma (device)  D in dtype
 *   Y (device)      N x D in dtype, row stride ldy (may equal X)
 *   rstd (device)   float[N] or NULL: r_i, needed by the backward
 * D % 8 == 0; X, Y, gamma 16-byte aligned with 16-byte row strides; eps >= 0.
 */
foak_status foak_rmsnorm_forward(const void* X, int32_t dtype, int64_t ldx, const void* gamma, int64_t N, int64_t D,
                                 float eps, void* Y, int64_t ldy, float* rstd, void* stream);

/* Bytes of device workspace foak_rmsnorm_backward needs for dgamma (512 x D floats of partial sums). */
size_t foak_rmsnorm_workspace_size(int64_t D);

/*
 * RMSNorm backward: with xh = X * r and u = gamma * dY (per row),
 *     dX = r * (u - xh * mean(xh * u)),    dgamma_j = sum_i dY_ij * xh_ij
 *   dY, X (device)  N x D in dtype (row strides lddy, ldx); rstd from the forward
 *   dX (device)     N x D in dtype, row stride lddx (may equal dY)
 *   dgamma (device) float32[D], overwritten, or NULL to skip it; it is summed in a
 *                   fixed order (deterministic) through `workspace`
 *                   (foak_rmsnorm_workspace_size(D) bytes, 256-byte aligned)
 * Alignment as for the forward.
 */
foak_status foak_rmsnorm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* gamma,
                                  const float* rstd, int32_t dtype, int64_t N, int64_t D, void* dX, int64_t lddx,
                                  float* dgamma, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace foak_rmsnorm_linear_ce_chunked needs: the chunked
 * linear + CE workspace, the normalised hidden states H and their gradient dH
 * (bf16 N x D each), r (float[N]) and the dgamma partials.
 */
size_t foak_rmsnorm_linear_ce_workspace_size(int64_t N, int64_t V, int64_t D, int64_t chunk);

/*
 * The decoder's tail: final RMSNorm -> LM head -> cross-entropy, the norm and the
 * chunked linear + CE of the FOAK pages composed on the device (the norm as the
 * chunked path's prologue and its backward as the epilogue; H and dH never leave
 * the device, the logits are never materialised):
 *     H = rmsnorm(X, gamma, eps) (bf16), loss / dH / dW as foak_linear_ce_chunked on
 *     H, then dX, dgamma through the norm (the rounding of H to bf16 is passed
 *     through as the identity).
 *   X (device)       bf16 [N][D] dense (row stride D), D % 8 == 0
 *   gamma (device)   bf16 [D]
 *   W, labels, chunk, g, denom, loss, dW, n_valid, err: as foak_linear_ce_chunked
 *   eps              >= 0 (1e-5 for Mistral and Llama-3)
 *   dX (device)      bf16 [N][D], overwritten
 *   dgamma (device)  float32 [D], overwritten
 * All pointers 16-byte aligned (loss, dgamma, n_valid, err: 4-byte).
 */
foak_status foak_rmsnorm_linear_ce_chunked(const void* X, const void* gamma, const void* W, const int64_t* labels,
                                           int64_t N, int64_t V, int64_t D, int64_t ignore_index, int64_t chunk,
                                           float eps, float g, float denom, float* loss, void* dX, float* dgamma,
                                           float* dW, int32_t* n_valid, int32_t* err, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * Rotary position embedding, the "Fast RoPE" kernel the FOAK pages list among
 * their fused operations (fms-acceleration-foak 0.7.4 page), with the explicit
 * position ids the pages note the FOAK version lacks (foak page, Known Issues;
 * fms-hf-tuning PR #280, Notes on FastKernels).  The pages print no formula; the
 * operation is the Llama / Mistral rotary embedding, "rotate half" pairing: for
 * head dimension d and i < d/2, elements i and i + d/2 of every head vector of
 * token t turn by theta = positions[t] * base^(-2i/d).
 *
 * Bytes of the cos/sin table for positions [0, max_pos) and head dimension d
 * (two fp32 planes of max_pos x d/2); 0 for an unsupported d (d % 16 != 0).
 */
size_t foak_rope_cache_size(int64_t max_pos, int64_t d);

/*
 * Build the table on the device: cos and sin of every (position, frequency),
 * the angle and its reduction in float64, stored as fp32.  base > 1 (10000 for
 * Llama-2 / Mistral, 500000 for Llama-3).  cache (device): 256-byte aligned,
 * foak_rope_cache_size(max_pos, d) bytes, owned by the caller; build it once per
 * (base, d, max_pos) and reuse it.
 */
foak_status foak_rope_build_cache(double base, int64_t d, int64_t max_pos, void* cache, size_t cache_bytes,
                                  void* stream);

/*
 * Apply the rotation in place (inverse != 0: turn by -theta, the backward: the
 * gradient of sum(G * rope(X)) is rope(G, inverse)).
 *   X (device)          T tokens x H heads x d in dtype (bf16 or fp32); heads of a
 *                       token contiguous, token stride ldt >= H*d elements (so Q
 *                       and K may be views into a fused QKV buffer); 16-byte
 *                       aligned, ldt * sizeof(dtype) % 16 == 0
 *   positions (device)  int64[T]: the token's position id (restarting at 0 per
 *                       sequence in a packed batch)
 *   cache (device)      the table of foak_rope_build_cache for max_pos, d
 *   err (device)        int32[1] or NULL: FOAK_ERRBIT_LABEL_RANGE when a position
 *                       is outside [0, max_pos); that token is left unchanged
 * d % 16 == 0 (FOAK_ERR_UNSUPPORTED otherwise).
 */
foak_status foak_rope_apply(void* X, int32_t dtype, int64_t T, int64_t H, int64_t ldt, int64_t d,
                            const int64_t* positions, const void* cache, int64_t max_pos, int32_t inverse,
                            int32_t* err, void* stream);

/*
 * foak_rope_apply on the Q and K of one layer in a single launch: Q is T x Hq x d
 * (token stride ldq), K is T x Hk x d (token stride ldk), both in dtype, same
 * positions and table; either may be empty (H = 0, pointer may be NULL).  Rules
 * and errors as foak_rope_apply.
 */
foak_status foak_rope_apply_qk(void* Q, int64_t Hq, int64_t ldq, void* K, int64_t Hk, int64_t ldk, int32_t dtype,
                               int64_t T, int64_t d, const int64_t* positions, const void* cache, int64_t max_pos,
                               int32_t inverse, int32_t* err, void* stream);

/*
 * The norms around a block with its gate and residual scale, in one pass over the rows:
 *     u_i = X_i,  or with post_gamma  X_i r1_i post_gamma,  r1_i = 1 / sqrt(mean_j X_ij^2 + post_eps)
 *     H_i = R_i + scale * g * u_i
 *     Y_i = H_i r_i gamma,  r_i = 1 / sqrt(mean_j H_ij^2 + eps)      (from the unrounded H_i)
 * in fp32, H and Y rounded once.  It is what stands between two blocks of a decoder beside
 * foak_rmsnorm_forward: X is a block's output, R the residual stream, Y the next block's input.
 *   X, R (device)       N x D in dtype, row strides ldx, ldr
 *   gate (device)       by gate_kind: FOAK_GATE_NONE (NULL); FOAK_GATE_CHANNEL: D values;
 *                       FOAK_GATE_ROW: N values, ldg elements apart; FOAK_GATE_FULL: N x D,
 *                       row stride ldg; all in dtype
 *   post_gamma (device) D in dtype (gains kept in fp32 beside bf16 rows are not taken), or NULL: no
 *                       norm after the block
 *   gamma (device)      D in dtype, or NULL: no norm before the next block (Y must be NULL)
 *   H, Y (device)       N x D in dtype, row strides ldh, ldy.  H may equal R or X; Y may equal X
 *                       or R, but not H; otherwise outputs overlap nothing
 *   post_rstd, rstd (device) float[N] or NULL: r1 and r, for the backward
 * D % 8 == 0, D <= FOAK_RESIDUAL_NORM_MAX_D; rows and vectors 16-byte aligned with 16-byte
 * strides (a FOAK_GATE_ROW gate: its elements' own alignment); scale finite; eps, post_eps >= 0.
 */
#define FOAK_GATE_NONE 0
#define FOAK_GATE_CHANNEL 1
#define FOAK_GATE_ROW 2
#define FOAK_GATE_FULL 3
#define FOAK_RESIDUAL_NORM_MAX_D 32768
foak_status foak_residual_norm_forward(const void* X, int64_t ldx, const void* R, int64_t ldr, int32_t dtype, int64_t N,
                                       int64_t D, const void* gate, int32_t gate_kind, int64_t ldg,
                                       const void* post_gamma, const void* gamma, float scale, float post_eps, float eps,
                                       void* H, int64_t ldh, void* Y, int64_t ldy, float* post_rstd, float* rstd,
                                       void* stream);

/*
 * Bytes of device workspace that foak_residual_norm_backward needs (partial sums over the
 * rows).  256-byte aligned; its contents need no initialisation, and calls that follow one
 * another on a stream may share it.
 */
size_t foak_residual_norm_workspace_size(int64_t N, int64_t D);

/*
 * Its backward, from H (as rounded), r and r1.  With t = gamma dY, hh = H r, xh = X r1:
 *     dR = dh = dH + r (t - hh mean_j(hh t)),     dgamma_j = sum_i dY hh
 *     du = scale g dh,     dgate = scale dh u, summed over the rows (channel) or a row (row)
 *     dX = du,  or with post_gamma  r1 (post_gamma du - xh mean_j(xh post_gamma du)),
 *     dpost_gamma_j = sum_i du xh
 *   dY (device)         N x D, or NULL: zero (H, gamma and rstd are not read; dgamma must be NULL
 *                       unless N is 0)
 *   dH (device)         N x D, the gradient that arrives along the residual stream, or NULL: zero;
 *                       not both NULL
 *   X (device)          N x D; may be NULL where neither post_gamma nor dgate is given
 *   gate, gate_kind, ldg, post_gamma, gamma, scale: as in the forward
 *   dR (device)         N x D; may equal dH or dY
 *   dX (device)         N x D or NULL: not wanted (without gate and post_gamma and with scale 1
 *                       it would be dR)
 *   dgamma, dpost_gamma (device) float[D] or NULL, overwritten
 *   dgate (device)      float[D] (channel), float[N] (row) or N x D in dtype with row stride lddg
 *                       (full), or NULL
 * The sums over the rows have a fixed order: results are the same from run to run.  Without rows
 * they are zeros, and N x D operands, statistics and gates of rows or elements may be NULL.  Sizes and
 * alignment as in the forward.  An output may be one of the N x D inputs (same stride), no two
 * outputs the same.
 */
foak_status foak_residual_norm_backward(const void* dY, int64_t lddy, const void* dH, int64_t lddh, const void* H,
                                        int64_t ldh, const void* X, int64_t ldx, int32_t dtype, int64_t N, int64_t D,
                                        const void* gate, int32_t gate_kind, int64_t ldg, const void* post_gamma,
                                        const void* gamma, const float* post_rstd, const float* rstd, float scale,
                                        void* dR, int64_t lddr, void* dX, int64_t lddx, float* dgamma, void* dgate,
                                        int64_t lddg, float* dpost_gamma, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * Rotary positions beyond foak_rope_*: both layouts, part of the head, contexts longer than the
 * trained one, out of place, and no table of positions.  Pair i < rotary_dim / 2 of a head --
 * elements (i, i + rotary_dim / 2), or (2i, 2i + 1) where interleaved -- turns by
 * positions[t] * inv_freq[i] and is multiplied by factor; the elements from rotary_dim on pass.
 *
 * foak_rotary_inv_freq (host): the frequencies base^(-2i / rotary_dim), scaled:
 *   FOAK_ROTARY_NONE    as they are
 *   FOAK_ROTARY_LINEAR  divided by scale (position interpolation)
 *   FOAK_ROTARY_NTK     of the base  base * scale^(rotary_dim / (rotary_dim - 2))
 *   FOAK_ROTARY_BANDS   by the turns n that a frequency makes over `original` positions: divided by
 *                       scale below `low` turns, kept above `high`, linear in n between
 *   FOAK_ROTARY_RAMP    the same, linear in the index i between the index of `high` turns, rounded
 *                       down, and that of `low` turns, rounded up
 *   inv_freq (host)     double[rotary_dim / 2]
 * rotary_dim even, 2 .. 65536 (NTK: above 2); base > 1; scale >= 1; BANDS and RAMP: 0 < low < high,
 * original >= 1.
 *
 * foak_rotary_turns (host): what the device calls take: turns[i] = inv_freq[i] / 2 pi as a
 * fraction of 2^64, whole turns dropped: within 2^-63 turn where |inv_freq[i]| <= 2^40 (above, its
 * 106 bits are not enough).  inv_freq finite.
 */
#define FOAK_ROTARY_NONE 0
#define FOAK_ROTARY_LINEAR 1
#define FOAK_ROTARY_NTK 2
#define FOAK_ROTARY_BANDS 3
#define FOAK_ROTARY_RAMP 4
foak_status foak_rotary_inv_freq(double base, int64_t rotary_dim, int32_t scaling, double scale, double low, double high,
                                 double original, double* inv_freq);
foak_status foak_rotary_turns(const double* inv_freq, int64_t n, uint64_t* turns);

/*
 * Rotate queries and keys in one launch (inverse != 0: back by the same angles, the backward pass).
 *   Q, K (device)       T x H x d in dtype, element (t, h, j) at t * ld + h * ldh + j; either may be
 *                       NULL.  Strides >= 0; what is 16-byte aligned moves 16 bytes at a time
 *   Qo, Ko (device)     where they go, with their own strides; Q and K themselves (same strides) to
 *                       rotate in place; otherwise they overlap nothing; heads d elements or more apart
 *   positions (device)  int64[T], any value: the angle modulo a turn is an integer product, off by
 *                       |positions[t]| times what the fraction is off (2^-63 turn at most)
 *   turns (device)      uint64[rotary_dim / 2] of foak_rotary_turns
 * Sine and cosine of that angle are within 4e-9 and a few fp32 roundings of themselves, and 2^-55
 * turn of the angle.
 * d >= rotary_dim >= 2, rotary_dim even; H * d <= 2^28.  Every element is computed the same way in every
 * call: it depends on its own pair, position and frequency alone.
 */
foak_status foak_rotary_apply(const void* Q, int64_t ldq, int64_t ldqh, void* Qo, int64_t ldqo, int64_t ldqoh, int64_t Hq,
                              const void* K, int64_t ldk, int64_t ldkh, void* Ko, int64_t ldko, int64_t ldkoh, int64_t Hk,
                              int32_t dtype, int64_t T, int64_t d, int64_t rotary_dim, int32_t interleaved,
                              const int64_t* positions, const uint64_t* turns, float factor, int32_t inverse,
                              void* stream);

/*
 * Where a serving step's tokens go in a paged cache: once a step, for the appends of all layers.
 * The T rows hold the step's tokens of B sequences one after another; sequence b has rows
 * seq_starts[b] .. seq_starts[b + 1] - 1 and cache_lens[b] tokens in the cache already.  With
 * pos = cache_lens[b] + t - seq_starts[b] its token goes to
 *     slots[t] = page_table[b][pos / page_size] * page_size + pos % page_size,   positions[t] = pos
 * Rows before the first sequence and behind the last one are padding: slot -1, position 0.
 *   page_table (device) int32[B][ld_table], max_pages <= ld_table entries a sequence
 *   cache_lens (device) int32[B];  seq_starts (device) int32[B + 1], ascending
 *   slots, positions (device) int64[T]
 *   err (device)        int32[1] or NULL: FOAK_ERRBIT_PAGE_RANGE is OR-ed in (the caller clears it)
 *                       for a page that is not in [0, num_pages), not in the table or of a negative
 *                       length; its tokens get slot -1
 * page_size and num_pages >= 1, their product below 2^62; T, B <= 2^31 - 1.
 */
foak_status foak_kv_slots(const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* cache_lens,
                          const int32_t* seq_starts, int64_t B, int64_t T, int64_t page_size, int64_t num_pages,
                          int64_t* slots, int64_t* positions, int32_t* err, void* stream);

/*
 * Append a step's keys and values to a layer's paged cache, the keys rotated on the way, and rotate
 * its queries, in one launch.  Token t goes to slot slots[t]: page slots[t] / page_size, place
 * slots[t] % page_size.  A token with a negative slot is padding: nothing of it is written.
 *   K, V (device)       T x Hk x d and T x Hk x dv in dtype, strides as for foak_rotary_apply
 *   k_cache, v_cache (device) element (page, place, h, j) at page * ld_page + place * ld_place +
 *                       h * ld_head + j, so either of (page, place, head) and (page, head, place)
 *   slots (device)      int64[T], distinct unless negative (of two equal ones, either token's
 *                       elements stay)
 *   Q, Qo (device)      T x Hq x d, as for foak_rotary_apply, or NULL
 *   rotary_dim          0: keys go as they are (positions and turns are not read, Q must be NULL)
 *   positions, turns, interleaved, factor: as for foak_rotary_apply
 *   err (device)        int32[1] or NULL: FOAK_ERRBIT_PAGE_RANGE is OR-ed in (the caller clears it)
 *                       for a slot of num_pages * page_size or more; nothing is written for it
 * Hk * max(d, dv) and Hq * d at most 2^28; page_size, num_pages as for foak_kv_slots.  The caches
 * overlap neither each other nor an input.
 */
foak_status foak_kv_append(const void* K, int64_t ldk, int64_t ldkh, const void* V, int64_t ldv, int64_t ldvh, int64_t Hk,
                           int32_t dtype, int64_t T, int64_t d, int64_t dv, const int64_t* slots, void* k_cache,
                           int64_t ldk_page, int64_t ldk_place, int64_t ldk_head, void* v_cache, int64_t ldv_page,
                           int64_t ldv_place, int64_t ldv_head, int64_t num_pages, int64_t page_size, const void* Q,
                           int64_t ldq, int64_t ldqh, void* Qo, int64_t ldqo, int64_t ldqoh, int64_t Hq,
                           int64_t rotary_dim, int32_t interleaved, const int64_t* positions, const uint64_t* turns,
                           float factor, int32_t* err, void* stream);

/*
 * Log probabilities, entropy and most likely tokens of the rows of a logits matrix:
 * what sits beside the loss once a model is served, trained by policy gradients or
 * used as a teacher.  The pages have no counterpart.  With z = x / temperature:
 *     lse_i = log sum_j exp(z_ij)          logp_i = z_{i,y_i} - lse_i
 *     H_i   = -sum_j p_ij log p_ij         p_ij = exp(z_ij - lse_i)
 * and the top_k largest logits of the row in descending order (equal logits: the
 * lower token id first) with their z_ij - lse_i.  One read of each row.
 *   logits, dtype, ld    as for foak_ce_forward
 *   labels (device)      int64[N], the given tokens, or NULL: every row is computed,
 *                        and logp must be NULL.  A row whose label is ignore_index, or
 *                        out of range (error bit FOAK_ERRBIT_LABEL_RANGE), is not read:
 *                        its outputs are 0 and its top ids -1
 *   temperature          in [1e-6, 1e6]
 *   top_k                0 .. min(V, FOAK_LOGPROBS_MAX_K); with top_k > 0, V <= 262144
 *   logp, entropy, lse (device)  float[N] each, or NULL
 *   stats (device)       float[N][2], 8-byte aligned, or NULL: (max_j x_ij, log sum_j
 *                        exp((x_ij - max) / temperature)), for foak_logprobs_backward
 *   top_logprobs (device) float[N][top_k];  top_ids (device) int32[N][top_k]
 *   err (device)         int32[1] or NULL
 *   workspace (device)   foak_logprobs_workspace_size() bytes, with the rules of
 *                        foak_ce_workspace_size (a buffer of that kind serves too)
 * Masked logits: an element of -inf has probability 0 and adds nothing to the entropy.
 * A row of nothing but -inf has lse -inf, log probabilities -inf, entropy 0 and top ids
 * 0 .. top_k - 1.  A row that holds NaN or +inf gives NaN, and top ids -1.
 */
#define FOAK_LOGPROBS_MAX_K 256
size_t foak_logprobs_workspace_size(void);
foak_status foak_logprobs_forward(const void* logits, int32_t dtype, int64_t ld, const int64_t* labels, int64_t N,
                                  int64_t V, int64_t ignore_index, float temperature, int64_t top_k, float* logp,
                                  float* entropy, float* lse, float* stats, float* top_logprobs, int32_t* top_ids,
                                  int32_t* err, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of sum_i (grad_logp_i logp_i + grad_entropy_i H_i) with respect to the logits:
 *     dx_ij = (grad_logp_i ([j == y_i] - p_ij) - grad_entropy_i p_ij (log p_ij + H_i)) / temperature
 * Rows that do not count get +0.0 and are not read; a row of nothing but -inf has p = 0.
 *   dlogits (device)     N x V, ld and dtype of the logits and the same offset modulo 16
 *                        bytes; may equal logits (in place)
 *   stats (device)       float[N][2] from the forward at the same temperature
 *   grad_logp (device)   float[N] or NULL (zero)
 *   entropy (device)     float[N] from the forward; needed with grad_entropy
 *   grad_entropy (device) float[N] or NULL (zero)
 *   err (device)         int32[1] or NULL
 */
foak_status foak_logprobs_backward(void* dlogits, const void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                                   int64_t N, int64_t V, int64_t ignore_index, float temperature, const float* stats,
                                   const float* grad_logp, const float* entropy, const float* grad_entropy,
                                   int32_t* err, void* stream);

/*
 * Distillation from a teacher's top tokens, mixed with the labels' cross-entropy.  The
 * teacher's row is K token ids with their log probabilities t (at the distillation
 * temperature: top_ids and top_logprobs of foak_logprobs_forward called with it).
 *     q_k  = exp(t_k) / sum_l exp(t_l)  (normalize != 0; t may then also be logits / temperature),  else exp(t_k)
 *     KD_i = sum_k q_k (log q_k - log p_{id_k}),  p = softmax(x_i / temperature)
 *     CE_i = log sum_j exp(x_ij) - x_{i,y_i}
 *     loss = sum_{valid i} (ce_weight CE_i + kd_weight KD_i) / D,   D = denom > 0 ? denom : n_valid
 *     dx_ij = (g / D) (ce_weight (softmax(x_i)_j - [j == y_i])
 *                      + kd_weight / temperature (p_ij sum_k q_k - sum_k q_k [j == id_k]))
 * (the customary factor temperature^2 is the caller's to put into kd_weight).
 *   logits, dtype, ld, ignore_index, denom, loss, n_valid, err, workspace: as for
 *                        foak_ce_forward (foak_ce_workspace_size(N) bytes)
 *   labels (device)      int64[N]; rows whose label is ignore_index do not count.  NULL:
 *                        every row counts, and ce_weight must be 0
 *   teacher_ids (device) int32[N][ld_teacher]: K ids a row.  A negative id is padding; an
 *                        id >= V counts as padding and sets FOAK_ERRBIT_LABEL_RANGE.  An
 *                        id may be listed more than once; its shares add up
 *   teacher_logprobs (device) float[N][ld_teacher]; -inf: no share
 *   K                    1 .. FOAK_DISTILL_MAX_K
 *   temperature          in [1e-6, 1e6]; ce_weight and kd_weight finite
 *   row_ce, row_kd (device) float[N] or NULL: the rows' terms (row_ce is 0 when
 *                        ce_weight is 0; 0 on rows that do not count)
 *   stats (device)       float[N][4], 16-byte aligned, or NULL: what foak_distill_backward
 *                        needs (max, log sum exp(x - max), log sum exp((x - max) / temperature),
 *                        sum of q)
 *   dlogits (device)     as for foak_logprobs_backward; may equal logits
 * foak_distill_fwd_bwd reads each logit once from device memory and writes its gradient;
 * foak_distill_backward recomputes it from stats, times *grad_out (device float[1], NULL = 1).
 * A student that gives a listed token probability 0 (a masked logit) has an infinite loss.
 */
#define FOAK_DISTILL_MAX_K 256
foak_status foak_distill_forward(const void* logits, int32_t dtype, int64_t ld, const int64_t* labels, int64_t N,
                                 int64_t V, int64_t ignore_index, const int32_t* teacher_ids,
                                 const float* teacher_logprobs, int64_t ld_teacher, int64_t K, int32_t normalize,
                                 float ce_weight, float kd_weight, float temperature, float denom, float* loss,
                                 float* row_ce, float* row_kd, float* stats, int32_t* n_valid, int32_t* err,
                                 void* workspace, size_t workspace_bytes, void* stream);
foak_status foak_distill_fwd_bwd(const void* logits, void* dlogits, int32_t dtype, int64_t ld, const int64_t* labels,
                                 int64_t N, int64_t V, int64_t ignore_index, const int32_t* teacher_ids,
                                 const float* teacher_logprobs, int64_t ld_teacher, int64_t K, int32_t normalize,
                                 float ce_weight, float kd_weight, float temperature, float g, float denom,
                                 float* loss, float* row_ce, float* row_kd, int32_t* n_valid, int32_t* err,
                                 void* workspace, size_t workspace_bytes, void* stream);
foak_status foak_distill_backward(void* dlogits, const void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                                  int64_t N, int64_t V, int64_t ignore_index, const int32_t* teacher_ids,
                                  const float* teacher_logprobs, int64_t ld_teacher, int64_t K, int32_t normalize,
                                  float ce_weight, float kd_weight, float temperature, const float* stats,
                                  const float* grad_out, float denom, int32_t* err, void* stream);

/*
 * Bytes of device workspace foak_linear_ce_chunked needs: the batch's label
 * count, N float32 per-row loss terms, a few error words, one chunk's per-tile
 * softmax statistics (chunk x ceil(V / 256) float pairs), its label logits and
 * log-sum-exps, and eight chunks of bf16 logits (min(8 chunk, N) x V, rows padded
 * to 64 elements: dW is updated once per group of four chunks, and one group is
 * computed while the last one is used).  256-byte aligned; its
 * contents need no initialisation and every call may reuse it.
 */
size_t foak_linear_ce_workspace_size(int64_t N, int64_t V, int64_t D, int64_t chunk);

/*
 * Chunked linear + cross-entropy: loss, dH and dW of CE(H W^T) computed chunk by
 * chunk (Z = H_c W^T, dZ = (softmax(Z) - onehot) g / D, dH_c = dZ W,
 * dW += dZ^T H_c) without materialising the N x V logits; the products run on the
 * tcgen05 tensor cores with fp32 accumulation, Z/dZ are kept in bf16.  The Z
 * product's epilogue reduces its fp32 accumulator to per-row, per-tile softmax
 * statistics and the label's logit, so the loss and log-sum-exp come from the
 * unrounded logits and dZ is one streaming pass over Z.
 *   H (device)        bf16 [N][D] row-major (hidden states), D % 8 == 0
 *   W (device)        bf16 [V][D] row-major (LM-head weight, no bias)
 *   labels (device)   int64[N]; ignore_index as for the CE calls
 *   chunk             rows per chunk (e.g. 1024), >= 1
 *   g (host), denom   as for foak_ce_fwd_bwd; D = denom > 0 ? denom : n_valid of
 *                     all N rows, the same for every chunk
 *   loss (device)     float[1]
 *   dH (device)       bf16 [N][D], overwritten
 *   dW (device)       float32 [V][D], overwritten (not accumulated into)
 *   n_valid, err      as for foak_ce_forward (err also reports GEMM wait timeouts)
 * All pointers 16-byte aligned.
 */
foak_status foak_linear_ce_chunked(const void* H, const void* W, const int64_t* labels, int64_t N, int64_t V,
                                   int64_t D, int64_t ignore_index, int64_t chunk, float g, float denom,
                                   float* loss, void* dH, float* dW, int32_t* n_valid, int32_t* err,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Building block of the chunked linear + CE: C[M x N] (+)= A[M x K] * B[N x K]^T on
 * the tcgen05 tensor cores, bf16 operands, fp32 accumulation (exposed so the
 * three products of the chunked call can be tested and timed alone).
 *   a, b (device)     bf16.  With *_mn_major = 0 the operand is stored row-major
 *                     as [rows][K] (K contiguous, row stride lda/ldb elements);
 *                     with 1 as [K][rows] (rows contiguous).  16-byte aligned
 *                     pointers and row strides; row strides >= the contiguous extent.
 *   out (device)      row-major [M][ldo]: bf16 for out_mode FOAK_GEMM_BF16, fp32 for
 *                     FOAK_GEMM_F32 (overwrite) and FOAK_GEMM_F32_ACC (add into it);
 *                     16-byte aligned pointer and row stride.
 *   err (device)      int32[1] or NULL: FOAK_ERRBIT_TIMEOUT is OR-ed in if a
 *                     device wait gave up (never set on a healthy GPU).
 */
#define FOAK_GEMM_BF16 0
#define FOAK_GEMM_F32 1
#define FOAK_GEMM_F32_ACC 2
foak_status foak_gemm_bf16(const void* a, int64_t lda, int32_t a_mn_major, const void* b, int64_t ldb,
                           int32_t b_mn_major, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                           int32_t out_mode, int32_t* err, void* stream);

/*
 * Up to FOAK_GEMM_GROUP_MAX independent products of foak_gemm_bf16's form in one
 * persistent launch: the SM pairs take a list of (product, 256 x 256 output unit)
 * entries balanced by estimated cost, longest units first, so a product with fewer
 * units than the GPU has SM pairs (dH of the chunked call: 4 x 16 units on 76 pairs)
 * shares the machine with another instead of leaving pairs idle.  This is how the
 * chunked call issues its dH products (with the next chunk's logits product).
 *   problems (host)   n descriptors, fields and rules as for foak_gemm_bf16; read
 *                     before the call returns.  No product may write memory that
 *                     another one reads or writes.
 *   n                 0 .. FOAK_GEMM_GROUP_MAX
 *   err (device)      as for foak_gemm_bf16, shared by the products
 * Products with M <= 128 (single-CTA tiles), or more than 8192 output units in all,
 * are launched one after another in the order given, with the same results.
 */
#define FOAK_GEMM_GROUP_MAX 3
typedef struct foak_gemm_problem {
    const void* a;
    int64_t lda;
    int32_t a_mn_major;
    const void* b;
    int64_t ldb;
    int32_t b_mn_major;
    int64_t M, N, K;
    void* out;
    int64_t ldo;
    int32_t out_mode;
} foak_gemm_problem;
foak_status foak_gemm_bf16_group(const foak_gemm_problem* problems, int32_t n, int32_t* err, void* stream);

/*
 * Largest N that foak_ce_fwd_bwd_noalloc accepts (its fixed scratch holds one
 * float per row: 1 MiB plus a 256-byte header on every device that loads the
 * library, kept until the process exits).
 */
#define FOAK_CE_NOALLOC_MAX_ROWS 262144

/*
 * Fused forward + backward without any workspace from the caller.  The pages
 * have no counterpart to this call; it exists for callers that must not allocate
 * device memory while they run -- e.g. code on a latency-critical path, where
 * cudaMalloc/cudaFree can synchronise the whole device, or a plugin inside a
 * runtime that owns all device memory and forbids allocations during execution.
 * It computes exactly what foak_ce_fwd_bwd computes, with the same arguments
 * minus the workspace, and allocates nothing: its scratch is a fixed array in the
 * library's device image.
 *   N                 at most FOAK_CE_NOALLOC_MAX_ROWS; larger N returns
 *                     FOAK_ERR_WORKSPACE before anything is enqueued
 *   stream            besides the kernel, the call enqueues a 256-byte
 *                     cudaMemsetAsync that clears the scratch header
 * The scratch used is the CURRENT device's: make the device that holds the
 * buffers and owns `stream` current before the call.  The first call on a device
 * looks up the scratch array's device address (once per device, with that device
 * current); make that first call before any stream capture begins.  Every call on a device shares the one scratch array, so calls
 * that overlap on the GPU (different streams without ordering) race and give
 * wrong results: serialise them.
 */
foak_status foak_ce_fwd_bwd_noalloc(void* logits, int32_t dtype, int64_t ld, const int64_t* labels,
                                    int64_t N, int64_t V, int64_t ignore_index, float g, float denom,
                                    float* loss, float* lse, int32_t* n_valid, int32_t* err,
                                    void* stream);

/*
 * Test hook: the next `count` launches made by this library fail with
 * FOAK_ERR_CUDA before anything is enqueued (host-side fault injection).
 */
void foak_test_fail_next_launches(int32_t count);

/*
 * Test hooks for the device-side failure path (no fault is involved): the row
 * kernels' shared-memory barrier waits give up after `ns` nanoseconds (0 restores
 * the default of 4 s), and the row kernels' producers never load row `row`'s data
 * (-1 disables), so the wait for that row is sure to run out.  A call that hits a
 * run-out wait stops loading, finishes its barriers, leaves the workspace reusable
 * and reports FOAK_ERRBIT_TIMEOUT in its error word (FOAK_ERR_TIMEOUT under
 * FOAK_SYNC_CHECK=1); its loss and gradient are then undefined.
 */
void foak_test_set_wait_limit_ns(uint64_t ns);
void foak_test_skip_row_load(int64_t row);

/*
 * Test hook: which row kernel the forward and fused calls use.  0 (default):
 * automatic -- aligned rows that fit one CTA's 64 KB slice go to the kernel whose
 * 16 warps each stream a 4 KB region of every row on their own, other rows of one
 * slice are swept once by one CTA in step, longer rows are streamed twice by one
 * CTA (log-sum-exp, then gradient); 1: one pass with the CTA in step, longer rows
 * split over a cluster of 2, 4 or 8 CTAs; 2: the two-pass streaming kernel for
 * every row length; 3: as 0 (the independent-warp kernel wherever it applies).
 * Results agree up to fp32 summation order.  Other values are treated as 0.
 */
void foak_test_set_row_path(int32_t path);

/*
 * Test hook (host only, no device work): the unit list foak_gemm_bf16_group would
 * give products of these shapes on `pairs` SM pairs.
 *   mnk      host int64[3 n]: M, N, K of each product (every M > 128), n in 1 .. 3
 *   start    host int32[pairs + 1]: cluster c takes entries start[c] .. start[c+1] - 1
 *   ent      host int32[ent_cap]: entries, product << 14 | output unit
 * Returns the number of clusters used (<= pairs), or -1 for bad arguments or when
 * ent_cap is too small.
 */
int32_t foak_test_gemm_group_schedule(const int64_t* mnk, int32_t n, int32_t pairs, int32_t* start, int32_t* ent,
                                      int32_t ent_cap);

#ifdef __cplusplus
}
#endif

#endif /* FOAK_CE_H */
