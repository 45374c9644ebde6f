/*
 * muon_adamw.h -- C ABI of the MI355X (gfx950) Muon + AdamW optimizer step.
 *
 * Two operations, both in place on caller-owned device memory, both
 * asynchronous on the caller's HIP stream:
 *
 *   ma_muon_step   one Muon step over groups of same-shape weight matrices
 *                  ("Chapter 4: The MuonAdamW Optimizer", sections "The Muon
 *                  Update Rule", "Polar Express: Newton-Schulz
 *                  Orthogonalization" and "The Full Muon Step"; nanochat
 *                  discussion "Stuck at the optimizer after figuring out
 *                  backward()", reply by mira687: per-step Polar Express
 *                  coefficients, cautious weight decay, MuonEq, the
 *                  max(1, rows/cols)^0.5 lr multiplier, stacked same-shape
 *                  matrices);
 *   ma_adamw_step  one AdamW step over flat buffers ("3.9 Optimizers: SGD,
 *                  Adam, Adafactor, Lion, Muon & Shampoo", section
 *                  "Implementing AdamW from scratch"; "Chapter 4", section
 *                  "The AdamW Step");
 *   ma_lion_step   one Lion step over flat buffers ("3.9 Optimizers",
 *                  section "Lion: Learning the Sign of the Update" and
 *                  exercise 5; "Muon vs AdamW, Lion and Sophia: a fair
 *                  race", section "Lion").
 *
 * and the operators that fill the gradients they read: ma_embedding_*,
 * ma_layernorm_*, ma_act_* (8-bit activation checkpoints and the weight
 * gradient of a linear layer out of one).
 *
 * Conventions for every entry point:
 *   - Pointers named "device" are HIP device pointers; "host" pointers are
 *     read during the call only and may be freed when it returns.
 *   - The library allocates no device memory and keeps no state between
 *     calls. Scratch memory is the caller's workspace.
 *   - Matrices are row-major, rows x cols, contiguous (leading dimension ==
 *     cols); rows are output features, cols input features.
 *   - Return value: MA_OK (0) or a negative MA_ERR_* code. Every argument is
 *     validated before the first launch, so a rejected call changes nothing.
 *     A kernel fault surfaces at the caller's next synchronisation.
 *     ma_last_error() returns a message for the calling thread's last
 *     failure.
 *   - `stream` is a hipStream_t passed as void* (NULL: the default stream).
 *   - Calls that overlap on one stream are ordered; concurrent calls on
 *     different streams must not share buffers or a workspace.
 */
#ifndef MUON_ADAMW_H
#define MUON_ADAMW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define MA_OK 0
#define MA_ERR_INVALID_ARG -1   /* null pointer, bad size, bad enum, aliasing */
#define MA_ERR_UNSUPPORTED -2   /* dtype combination not provided */
#define MA_ERR_WORKSPACE -3     /* workspace null, too small or misaligned */
#define MA_ERR_HIP -4           /* a HIP runtime call or launch failed */
#define MA_ERR_NONFINITE -5     /* ma_muon_nonfinite: a matrix of the last step had
                                   non-finite norms (check_finite == 1 only) */

typedef enum { MA_F32 = 0, MA_BF16 = 1 } ma_dtype;

/* Row scalings (rows are output features, in the parameter's own layout).
 * ROWS_PRE (MuonEq): each row of the Nesterov look-ahead is divided by its
 *   Euclidean norm (+eq_eps) before the Frobenius normalisation.
 * ROWS_POST (MuonEq after the iteration): each row of the orthogonalised
 *   update U is rescaled to the matrix's mean row norm, ||U||_F/sqrt(rows),
 *   over (||U_i|| + eq_eps).
 * ROWS_RMS (NorMuon, "Chapter 4: The MuonAdamW Optimizer", section "NorMuon:
 *   Normalized Muon"): each row of U is divided by its RMS,
 *   ||U_i||/sqrt(cols), plus eq_eps (the page uses 1e-8), so that with
 *   lr_scale NONE every row of the step has RMS lr. */
typedef enum { MA_EQ_OFF = 0, MA_EQ_ROWS_PRE = 1, MA_EQ_ROWS_POST = 2, MA_EQ_ROWS_RMS = 3 } ma_eq;

/* Per-matrix lr multiplier:
 *   NONE                1
 *   SQRT_MAX1_R_OVER_C  sqrt(max(1, rows/cols)) (nanochat discussion, reply by
 *                       mira687: x2 for c_fc, x1 for c_proj)
 *   MOONSHOT            0.2 * sqrt(max(rows, cols)) ("Muon vs AdamW, Lion and
 *                       Sophia: a fair race": entries about AdamW's size)
 *   SQRT_MAX            sqrt(max(rows, cols)) ("3.9 Optimizers ...", section
 *                       "Muon: Orthogonalizing the Update": update RMS about 1) */
typedef enum {
  MA_SCALE_NONE = 0,
  MA_SCALE_SQRT_MAX1_R_OVER_C = 1,
  MA_SCALE_MOONSHOT = 2,
  MA_SCALE_SQRT_MAX = 3
} ma_scale;

/* One group: `count` matrices of identical shape rows x cols.
 * params/grads/momentum are HOST arrays of `count` DEVICE pointers; matrix i
 * of the group is params[i] (rows*cols elements of param_dtype), grads[i]
 * (grad_dtype, read only) and momentum[i] (mom_dtype, updated in place).
 * Limits (MA_ERR_INVALID_ARG beyond them): rows, cols <= 2^24,
 * rows*cols <= 2^31, count*rows*cols <= 2^40. */
typedef struct {
  int64_t rows, cols;
  int32_t count;
  int32_t param_dtype, grad_dtype, mom_dtype; /* ma_dtype */
  void* const* params;
  const void* const* grads;
  void* const* momentum;
} ma_muon_group;

/* Muon hyperparameters ("Chapter 4", section "The Full Muon Step"; the
 * nanochat discussion for the coefficient table, cautious mask and MuonEq).
 *   lr            base learning rate (multiplied per matrix by lr_scale)
 *   momentum      beta of the sum-form buffer  m <- beta*m + G
 *   weight_decay  decoupled decay; the applied factor is lr_eff*weight_decay
 *   nesterov      1: orthogonalise G + beta*m (look-ahead), 0: orthogonalise m
 *   ns_steps      number T of quintic steps, 0..MA_MAX_NS_STEPS
 *   abc           HOST array of 3*ns_steps floats: (a_k, b_k, c_k) of step k,
 *                 X <- a_k X + (b_k A + c_k A A) X with A = X X^T
 *   cautious      1: decay only where update and weight agree in sign,
 *                 mask = (U * W >= 0)
 *   equilibrate   ma_eq
 *   ns_precision  MA_BF16: iterate in bf16 with fp32 accumulation;
 *                 MA_F32: iterate in fp32
 *   lr_scale      ma_scale
 *   norm_eps      added to the Frobenius norm (the pages use 1e-7)
 *   eq_eps        added to each row norm by MuonEq (1e-7), or to each row RMS
 *                 by ROWS_RMS
 *   check_finite  1: detect non-finite values, after the fast-fail rule of
 *                 "Chapter 4", section "Fast-Fail on NaN or Loss > 100".
 *                 A matrix whose look-ahead momentum has a non-finite sum of
 *                 squares (a NaN or Inf entry, or an overflowing square) --
 *                 or, with ROWS_POST / ROWS_RMS, whose orthogonalised update
 *                 has one -- keeps its weight unchanged (no decay, no
 *                 update); its momentum buffer is updated as usual and holds
 *                 the non-finite values. Every other matrix is stepped
 *                 exactly as without the check. ma_muon_nonfinite reports
 *                 which matrices were flagged. 0: no check (non-finite
 *                 values propagate into the weights). */
typedef struct {
  float lr, momentum, weight_decay;
  int32_t nesterov, ns_steps;
  const float* abc;
  int32_t cautious, equilibrate, ns_precision, lr_scale;
  float norm_eps, eq_eps;
  int32_t check_finite;
} ma_muon_hparams;

#define MA_MAX_NS_STEPS 16
#define MA_WORKSPACE_ALIGN 256

/* Bytes of device workspace ma_muon_step needs for these groups and
 * hyperparameters (0 on invalid arguments; see ma_last_error). The
 * workspace holds the normalised momentum and the Newton-Schulz iterates
 * and Gram matrices of every matrix, padded to multiples of 256, the
 * partial sums of ma_muon_step_stats and, for fp32 groups small enough that
 * their Gram product is split along K, its per-slice partial products. */
size_t ma_muon_workspace_size(const ma_muon_group* groups, int32_t n_groups,
                              const ma_muon_hparams* hp);

/* One Muon step for every matrix of every group. Per matrix W (R x C),
 * gradient G, momentum buffer M, in this order:
 *   m1 = beta*M + G (fp32); M <- m1 rounded to mom_dtype (RNE)
 *   Mt = G + beta*m1 if nesterov else m1                      (fp32)
 *   optional MuonEq PRE; X0 = Mt / (||Mt||_F + norm_eps)
 *     (with MuonEq PRE and T >= 1, groups for which ma_muon_row_pass is 1
 *     store the row-scaled Mt rounded to the iteration's precision and apply
 *     1 / (||.||_F + norm_eps) in the first Gram product and update: the same
 *     X0 with one rounding at a different point)
 *   if R > C the iteration runs on X0^T (layout, no extra copy)
 *   T quintic steps with the caller's coefficient table
 *   optional MuonEq POST; U = final iterate in W's layout
 *   lr_eff = lr * multiplier(R, C)  (fp64 on the host, then fp32)
 *   mask = cautious ? (U*W >= 0) : 1
 *   W <- RNE( (mask ? W - (lr_eff*wd)*W : W) - lr_eff*U )   (fp32, no FMA)
 * The decay term is skipped entirely when weight_decay == 0.
 * Supported storage: param/grad/mom each MA_BF16 or MA_F32.
 * workspace: DEVICE, >= ma_muon_workspace_size bytes, MA_WORKSPACE_ALIGN
 * aligned. Parameter, gradient and momentum buffers must not overlap each
 * other or the workspace (MA_ERR_INVALID_ARG is returned for overlaps among
 * the pointers passed).
 * Results are deterministic for given inputs. The kernels a call uses depend
 * on its total work (launches of few tile jobs run smaller tiles, and an fp32
 * Gram product of few jobs is split along K), so one matrix stepped alone
 * and the same matrix stepped with many others can differ at the rounding
 * level. */
int ma_muon_step(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ma_muon_step with no workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation). The step's scratch memory is a fixed
 * array of MA_NOALLOC_SCRATCH_BYTES inside the library's device code, one
 * per GPU, held until the process ends; the call allocates nothing. Same
 * arguments, kernels and results as ma_muon_step. A call whose
 * ma_muon_workspace_size exceeds MA_NOALLOC_SCRATCH_BYTES is rejected with
 * MA_ERR_WORKSPACE before any launch. Every call on one GPU uses that GPU's
 * one array: calls that may overlap on one GPU (on different streams, or
 * from different host threads) race and must be ordered by the caller. Each
 * call writes every byte of scratch it later reads, so nothing carries over
 * from an earlier call. With check_finite, ma_muon_nonfinite is not available
 * for this entry point (the flags live in the shared array). The array used
 * is the current device's: a stream of another device is rejected with
 * MA_ERR_INVALID_ARG. */
#define MA_NOALLOC_SCRATCH_BYTES (64u << 20)
int ma_muon_step_noalloc(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp, void* stream);

/* ma_muon_step that also reports, per matrix, the size of the step it took:
 * the per-layer ratio ||delta theta|| / ||theta|| that "3.9 Optimizers: SGD,
 * Adam, Adafactor, Lion, Muon & Shampoo" (section "Large-batch training:
 * LARS, LAMB and the trust ratio") recommends logging. stats: DEVICE array of
 * 2 floats per matrix, groups in order and matrices in order within a group:
 *   stats[2k]   = ||W_new - W_old||_F, W_new as stored (after rounding to
 *                 param_dtype), W_old the weight before the step
 *   stats[2k+1] = ||W_old||_F
 * Per-element squares are summed in fp32 per block and the block sums in
 * fp64 in a fixed order, so the result is deterministic. stats must be
 * 4-byte aligned and must not overlap any other buffer (MA_ERR_INVALID_ARG).
 * The update itself is identical to ma_muon_step's. */
int ma_muon_step_stats(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp,
                       void* workspace, size_t workspace_bytes, float* stats, void* stream);

/* After a ma_muon_step / ma_muon_step_stats / ma_muon_adamw_step with
 * check_finite == 1 has completed (the caller has synchronised its stream),
 * the matrices it flagged: flags (HOST array of the total matrix count,
 * groups in order, or null) receives 1 for a flagged matrix and 0 otherwise.
 * groups, n_groups, hp and workspace must be those of the step. Returns MA_OK
 * when no matrix was flagged, MA_ERR_NONFINITE when one was, or
 * MA_ERR_INVALID_ARG when hp->check_finite is 0 (the step wrote no flags).
 * Synchronous: it copies the flags from device memory. */
int ma_muon_nonfinite(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp,
                      const void* workspace, int32_t* flags);

/* Whether ma_muon_step treats group `group` in one pass over G and M: the
 * momentum update, MuonEq PRE's row sums and the row-scaled X0 together, the
 * Frobenius factor of "Chapter 4: The MuonAdamW Optimizer" (section "Polar
 * Express: Newton-Schulz Orthogonalization") then applied by the first
 * Newton-Schulz products. That is the case for MuonEq PRE with T >= 1, a bf16
 * iteration, rows <= cols, cols a multiple of 8 and at most 4096 (after
 * padding to 256), 16-byte aligned buffers, unless the environment sets
 * MA_PRE_ROWS=0. Returns 1 or 0, or a negative MA_ERR_* for invalid
 * arguments (as ma_muon_workspace_size validates them). Host-only. */
int ma_muon_row_pass(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp, int32_t group);

/* Where matrix `index` of group `group` keeps the result of its Newton-Schulz
 * iteration inside a workspace after ma_muon_step (for inspection; valid
 * until the workspace is reused; with MA_EQ_ROWS_POST or MA_EQ_ROWS_RMS the
 * row scaling is applied later, in the update, and is not included). *u receives a DEVICE
 * pointer into `workspace`, in the parameter's layout (rows x cols, row pitch
 * *ld elements); *transposed (may be null) is set to 0; *elem_bytes is 2
 * (bf16 iteration) or 4 (fp32). */
int ma_muon_workspace_update(const ma_muon_group* groups, int32_t n_groups,
                             const ma_muon_hparams* hp, void* workspace, int32_t group,
                             int32_t index, void** u, int64_t* ld, int32_t* transposed,
                             int32_t* elem_bytes);

/* One flat AdamW buffer. param, grad, exp_avg, exp_avg_sq: DEVICE pointers to
 * n elements each (fp32; param_dtype and grad_dtype must be MA_F32). `step` is
 * the 1-based step count after increment (1 on the first call). */
typedef struct {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  int64_t n;
  int32_t param_dtype, grad_dtype;
  float lr, beta1, beta2, eps, weight_decay;
  int64_t step;
} ma_adamw_segment;

/* One AdamW step over every segment (fp32 throughout), per element:
 *   p = p*(1 - lr*wd)            (only when wd != 0)
 *   m = beta1*m + (1-beta1)*g
 *   v = beta2*v + (1-beta2)*(g*g)
 *   p = p - (lr/(1-beta1^t)) * (m / (sqrt(v)/sqrt(1-beta2^t) + eps))
 * Step-dependent scalars are formed in fp64 on the host and rounded to fp32
 * once; each per-element operation is one correctly rounded fp32 operation
 * (no fused multiply-add). Segments may be in any order and of any length
 * (0 <= n <= 2^40); buffers of different segments must not overlap.
 * `segments` is a HOST array. */
int ma_adamw_step(const ma_adamw_segment* segments, int32_t n_segments, void* stream);

/* ma_adamw_step with identical results, run by at most `workgroups`
 * persistent workgroups that each keep one 16-byte chunk per buffer in
 * flight per thread: a register footprint small enough for a workgroup to
 * share a CU with a Newton-Schulz GEMM workgroup. For issuing the AdamW part
 * of a step on a second stream while ma_muon_step runs on another (the two
 * touch disjoint buffers); alone it is slower than ma_adamw_step. workgroups
 * >= 1 (MA_ERR_INVALID_ARG otherwise); 256, one per CU, suits MI355X. */
int ma_adamw_step_background(const ma_adamw_segment* segments, int32_t n_segments, int32_t workgroups,
                             void* stream);

/* One MuonAdamW step: ma_muon_step on `stream` and, on `side_stream`, the
 * AdamW update of ma_adamw_step_background (`workgroups` workgroups), which
 * starts once the Muon step's elementwise passes and first Gram and
 * polynomial products are done ("Chapter 4: The MuonAdamW Optimizer",
 * section "The Full Muon Step": the two optimizers update disjoint parameter
 * sets) and runs beside its remaining products; `stream` waits for it before
 * any later work. Results are those of ma_muon_step followed by
 * ma_adamw_step. side_stream must differ from stream (both may be captured
 * into one HIP graph: the fork and join are event records and waits on
 * events the library creates once per device and host thread; both streams
 * must belong to the current device, MA_ERR_INVALID_ARG otherwise). Every
 * argument is validated before the first launch, and no two buffers of the
 * two steps (Muon parameters, gradients, momentum, the workspace, AdamW
 * buffers) may overlap (MA_ERR_INVALID_ARG). If a launch fails after the
 * fork, `stream` still waits for what was queued on side_stream before the
 * error is returned. */
int ma_muon_adamw_step(const ma_muon_group* groups, int32_t n_groups, const ma_muon_hparams* hp,
                       void* workspace, size_t workspace_bytes, const ma_adamw_segment* segments,
                       int32_t n_segments, int32_t workgroups, void* stream, void* side_stream);

/* One flat Lion buffer. param, grad, exp_avg (the momentum, Lion's only
 * state): DEVICE pointers to n elements each, fp32 (param_dtype and
 * grad_dtype must be MA_F32), 4-byte aligned. */
typedef struct {
  void* param;
  const void* grad;
  void* exp_avg;
  int64_t n;
  int32_t param_dtype, grad_dtype;
  float lr, beta1, beta2, weight_decay;
} ma_lion_segment;

/* One Lion step over every segment (fp32 throughout), per element:
 *   p = p*(1 - lr*wd)            (only when wd != 0)
 *   c = beta1*m + (1-beta1)*g    (not stored)
 *   p = p - lr*sign(c)           sign: +1, -1, +0 for either zero, NaN for NaN
 *   m = beta2*m + (1-beta2)*g    (after the step, with the raw gradient)
 * 1 - lr*wd, 1 - beta1 and 1 - beta2 are formed in fp64 on the host and
 * rounded to fp32 once; each per-element operation is one correctly rounded
 * fp32 operation (no fused multiply-add). Requirements: finite lr and
 * weight_decay, 0 <= beta1, beta2 < 1. Segments may be in any order and of
 * any length (0 <= n <= 2^40); no two buffers, of one segment or of different
 * segments, may overlap. `segments` is a HOST array. Returns
 * MA_ERR_INVALID_ARG / MA_ERR_UNSUPPORTED before any launch on a bad
 * segment. */
int ma_lion_step(const ma_lion_segment* segments, int32_t n_segments, void* stream);

/* ---------------------------------------------------------------------------
 * The operators around the step: what fills the gradient buffers that the
 * steps above read. The embedding's and the norms' gradients are flat fp32
 * buffers (AdamW and Lion segments), the weight gradient is a row-major
 * outs x ins matrix of either storage type (a Muon group's grads[i]). All
 * tensors are dense and row-major and start at any multiple of their element
 * size; outputs may not overlap any other buffer of the call
 * (MA_ERR_INVALID_ARG). Sums are fp32, in an order that depends on the sizes
 * and types (and the tokens) alone, and each output is rounded once to its
 * type: a call repeated on the same inputs gives the same bits. accumulate = 1 adds to the gradient that is
 * already there (in fp32, before the one rounding); 0 writes it whole. `stream`
 * must belong to the current device (MA_ERR_INVALID_ARG). Every call may be
 * captured in a HIP graph; a graph keeps the workspace it was captured with,
 * and graphs or calls that may overlap need one each.
 * ------------------------------------------------------------------------- */

/* out[i,:] = scale * table[tokens[i],:] for i < n_tokens. table: rows x cols;
 * tokens: n_tokens integers of token_bytes (4 or 8, signed); out: n_tokens x
 * cols. A token outside 0..rows-1 is ignored: its output row is zero, and it
 * takes no part in the gradient (a row of another rank's shard, a masked
 * position). Limits: rows <= 2^24, cols <= 2^20, n_tokens <= 2^25, rows * cols
 * <= 2^35, n_tokens * cols <= 2^36; scale finite. */
int ma_embedding_forward(const void* table, int32_t table_dtype, int64_t rows, int64_t cols, const void* tokens,
                         int32_t token_bytes, int64_t n_tokens, float scale, void* out, int32_t out_dtype, void* stream);

/* grad[v,:] = scale * sum of dout[i,:] over the i with tokens[i] == v, for
 * every row v < rows (zero where there is none). With accumulate the rows that
 * occur are added to and no other row is touched. dout: n_tokens x cols; grad:
 * rows x cols, fp32. Up to 1024 tokens a row's positions are found by
 * comparison, up to 16 of them summed in ascending i, more in 8 contiguous
 * shares that are added in order. More tokens are sorted first (stable, by
 * kernels of this call): runs of up to 16 positions (32 above 16384 tokens) are
 * summed in ascending i, longer ones in pieces of as many sorted positions,
 * whose sums are added up in 8 contiguous shares, in order. workspace: at
 * least ma_embedding_workspace_size bytes (0 from that function: invalid
 * sizes), MA_WORKSPACE_ALIGN aligned; that of more tokens serves fewer too. */
size_t ma_embedding_workspace_size(int64_t rows, int64_t cols, int64_t n_tokens);
int ma_embedding_backward(const void* dout, int32_t dout_dtype, const void* tokens, int32_t token_bytes, int64_t n_tokens,
                          int64_t rows, int64_t cols, float scale, int32_t accumulate, float* grad, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Layer norm over the last dimension, per row of x (rows x cols; rows <= 2^24,
 * cols <= 16384, rows * cols <= 2^36):
 *   mean = sum x / cols;  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps)
 *   y = (x - mean) * rstd * gain + bias        gain, bias: cols fp32 values, either may be null
 * A mean of more than 4 deviations is corrected by the sum of the differences
 * from it, so that a row of equal values has no variance. Sums are fp32: a row
 * whose sum of squares passes its range has rstd 0, one whose sum does NaN.
 * stats (rows x 2 fp32, 8-byte aligned) receives mean and rstd for the backward
 * pass. With ckpt_q and ckpt_scale (both or neither) the same pass also writes
 * the 8-bit checkpoint of x, as ma_act_pack would. */
int ma_layernorm_forward(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, const float* gain, const float* bias,
                         float eps, void* y, int32_t y_dtype, float* stats, uint8_t* ckpt_q, uint8_t* ckpt_scale,
                         void* stream);

/* Its backward pass from dy, stats and either x or x's checkpoint (the other
 * null): with xh = (x - mean) * rstd and g = dy * gain (gain may be null),
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh))
 *   dgain (+)= sum over rows of dy * xh;  dbias (+)= sum over rows of dy
 * dx has x's type, or dy's where x is a checkpoint. dgain and dbias (cols fp32
 * values) may each be null; with both null no workspace is needed, else at
 * least ma_layernorm_workspace_size bytes, which may be 0 (few rows); that of
 * more rows serves fewer too. accumulate applies to dgain and dbias. */
size_t ma_layernorm_workspace_size(int64_t rows, int64_t cols);
int ma_layernorm_backward(const void* dy, int32_t dy_dtype, const void* x, int32_t x_dtype, const uint8_t* ckpt_q,
                          const uint8_t* ckpt_scale, int64_t rows, int64_t cols, const float* stats, const float* gain,
                          void* dx, int32_t dx_dtype, float* dgain, float* dbias, int32_t accumulate, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Root-mean-square norm with the residual's addition, per row (rows <= 2^24,
 * cols <= 16384, rows * cols <= 2^36):
 *   t = x + residual, added in fp32 and rounded to the residual's type, written to `total`;
 *       without a residual t = x, and `total` must be null
 *   rstd = 1 / sqrt(sum t^2 / cols + eps)
 *   y = t * rstd * gain                        gain: cols fp32 values, may be null
 * The norm reads t as it is stored. rstd (rows fp32) and t are what the backward
 * pass reads. y may be null where held_q and held_scale (both or neither) are
 * given: they receive y as an 8-bit checkpoint (ma_act_pack), rounded from fp32
 * once; with y given too, both are written. Sums are fp32: a row whose sum of
 * squares passes its range has rstd 0. With eps 0 a row of zeros has y NaN, one whose
 * squares all vanish in fp32 rstd infinite, and squares below 2^-126 lose bits. */
int ma_rmsnorm_forward(const void* x, int32_t x_dtype, const void* residual, int32_t residual_dtype, int64_t rows, int64_t cols,
                       const float* gain, float eps, void* total, void* y, int32_t y_dtype, float* rstd, uint8_t* held_q,
                       uint8_t* held_scale, void* stream);

/* Its backward pass from dy, rstd and either t or t's 8-bit checkpoint (the other
 * null): with xh = t * rstd and g = dy * gain (gain may be null),
 *   dx = dtotal + rstd * (g - xh * mean(g * xh));  dgain (+)= sum over rows of dy * xh
 * dtotal is the gradient that reaches t on other ways (the residual stream's; may
 * be null), so dx is the gradient of x and of the residual alike. dx and dtotal
 * have t's type, or dy's where t is held in 8 bits. dgain (cols fp32 values) may be
 * null; else at least ma_rmsnorm_workspace_size bytes of workspace are needed, which
 * may be 0 (few rows); that of more rows serves fewer too. accumulate applies to
 * dgain. */
size_t ma_rmsnorm_workspace_size(int64_t rows, int64_t cols);
int ma_rmsnorm_backward(const void* dy, int32_t dy_dtype, const void* t, int32_t t_dtype, const uint8_t* held_q,
                        const uint8_t* held_scale, int64_t rows, int64_t cols, const float* rstd, const float* gain,
                        const void* dtotal, void* dx, int32_t dx_dtype, float* dgain, int32_t accumulate, void* workspace,
                        size_t workspace_bytes, void* stream);

/* 8-bit activation checkpoints. q (rows x P bytes, P = cols rounded up to a
 * multiple of MA_ACT_BLOCK, 16-byte aligned, zero beyond cols) holds e4m3 (OCP)
 * values, scale (rows x P / MA_ACT_BLOCK bytes) a power of two for each block of
 * MA_ACT_BLOCK columns: the byte s stands for 2^(s - 127). Packing takes the
 * least exponent in -117..120 with amax <= 448 * 2^e over the block's finite
 * values and rounds x / 2^e to nearest even, within 448 (240 at e = 120, so that
 * every value held is finite in bf16 and fp32). NaN and infinities are held as
 * NaN. Every held value is exact in bf16: unpacking rounds nothing, and the
 * error against x is at most 2^-4 |x|, or 2^-10 * 2^e for values below the
 * block's e4m3 normal range (2^-6 * 2^e). Limits: rows, cols <= 2^24, rows * P
 * <= 2^36 (2^35 where x or out is fp32). */
#define MA_ACT_BLOCK 128
int ma_act_pack(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, uint8_t* q, uint8_t* scale, void* stream);
int ma_act_unpack(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, void* out, int32_t out_dtype,
                  void* stream);

/* The weight gradient of a linear layer y = x W^T out of x's checkpoint:
 *   grad[n,k] (+)= sum over tokens t of dy[t,n] * x[t,k]
 * dy: tokens x outs; q, scale: the checkpoint of x (tokens x ins) as written by
 * ma_act_pack; grad: outs x ins. The held values are used as they are (no
 * second rounding) and dy at its full precision, but for what of a fp32 value
 * lies below 2^-133, the last bit of bf16 (so all of it from 2^-110 up);
 * products are summed in fp32.
 * Limits: tokens <= 2^25, outs, ins <= 2^23, outs * ins <= 2^31, tokens * outs and
 * tokens * P <= 2^36. workspace: at
 * least ma_act_weight_grad_workspace_size bytes, which may be 0. That is the
 * need of exactly these sizes: fewer tokens can need more (they may be shared
 * out among more blocks), so a workspace for calls of several sizes takes the
 * largest of theirs. */
size_t ma_act_weight_grad_workspace_size(int64_t tokens, int64_t outs, int64_t ins, int32_t dy_dtype);
int ma_act_weight_grad(const void* dy, int32_t dy_dtype, const uint8_t* q, const uint8_t* scale, int64_t tokens,
                       int64_t outs, int64_t ins, void* grad, int32_t grad_dtype, int32_t accumulate, void* workspace,
                       size_t workspace_bytes, void* stream);

/* 4-bit matrices: blocks of MA_MX4_BLOCK columns of a row with one power of two
 * each, and e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives). With
 * P = cols rounded up to a multiple of MA_MX4_TILE:
 *   q      rows x P/2 bytes, 16-byte aligned; two values a byte, the even column in
 *          the lower half; zero beyond cols
 *   scale  P/MA_MX4_TILE x rows x 4 bytes, 4-byte aligned: for every tile of columns
 *          and row the bytes of its 4 blocks; the byte s stands for 2^(s - 127), 255
 *          for NaN (E8M0), also in a block beyond cols, where packing writes 1
 * Packing takes the least exponent e in -126..125 for which the block's largest
 * magnitude over 2^e rounds to at most 6, and rounds x / 2^e to nearest even: every
 * value is off by half a step at most (|x| / 5 from 2^e up, 2^e / 4 below). At
 * e = 125 values stop at 6 * 2^125. A block with a NaN or an infinity is held as NaN.
 * Every held value is exact in bf16. transpose = 1 packs x^T: q and scale then
 * describe a cols x rows matrix, whose blocks go along x's rows. Unpacking rounds
 * nothing; under the scale bytes 253 and 254, which packing does not write, values from
 * 4 and from 2 are beyond either type and come out infinite. Limits: rows, cols <=
 * 2^24, and padded rows of at most 2^36 values in all (2^35 where x or out is fp32). */
#define MA_MX4_BLOCK 32
#define MA_MX4_TILE 128
int ma_mx4_pack(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int32_t transpose, uint8_t* q, uint8_t* scale,
                void* stream);
int ma_mx4_unpack(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, void* out, int32_t out_dtype,
                  void* stream);

/* A linear layer on held values: y[m,n] (+)= sum over k of x[m,k] * w[n,k].
 * wq, wscale: a 4-bit outs x ins matrix; xq, xscale: rows x ins held in 4 bits
 * (x_bits 4) or as an 8-bit checkpoint (x_bits 8). The held values are multiplied as
 * they are and summed in fp32, and y (rows x outs) is rounded once. A NaN that is held
 * reaches every output of its row (of w: of its column).
 * Limits: rows <= 2^24, outs, ins <= 2^23, rows * outs, rows * P and outs * P <= 2^36
 * (P = ins rounded up to a multiple of MA_MX4_TILE). workspace: at least ma_mx4_matmul_workspace_size
 * bytes, which may be 0; that is the need of exactly these sizes. */
size_t ma_mx4_matmul_workspace_size(int64_t rows, int64_t outs, int64_t ins, int32_t x_bits);
int ma_mx4_matmul(const uint8_t* xq, const uint8_t* xscale, int32_t x_bits, int64_t rows, const uint8_t* wq,
                  const uint8_t* wscale, int64_t outs, int64_t ins, void* y, int32_t y_dtype, int32_t accumulate,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Status text for a code, and the calling thread's last error message. */
const char* ma_status_string(int status);
const char* ma_last_error(void);

/* Library version string, and the GPU architecture it was built for. */
const char* ma_version(void);

/* ---------------------------------------------------------------------------
 * Kernel timing. Between ma_profile_begin and ma_profile_end every kernel the
 * library launches is bracketed by two HIP events recorded on its stream
 * (host-side objects from a pool of 2*max_launches events created by
 * ma_profile_begin; no device memory). ma_profile_read synchronises on the
 * recorded events and returns, for one kernel kind, the summed duration in
 * milliseconds and the number of launches. Launches beyond max_launches are
 * not timed. Not thread-safe with concurrent library calls.
 * ------------------------------------------------------------------------- */
typedef enum {
  MA_K_ROWNORM = 0,   /* row sums of squares (momentum look-ahead or update) */
  MA_K_FINALIZE = 1,  /* per-matrix Frobenius / MuonEq factors */
  MA_K_PRE = 2,       /* momentum update and X0 in both layouts */
  MA_K_GRAM = 3,      /* A = X X^T */
  MA_K_POLY = 4,      /* B = b A + c A A */
  MA_K_AXPY = 5,      /* X' = a X + B X */
  MA_K_POST = 6,      /* cautious decay and the update */
  MA_K_ADAMW = 7,
  MA_K_LION = 8,
  MA_K_AXPY_UPDATE = 9, /* the last AXPY of a step with the update fused into it */
  MA_K_EMBEDDING = 10,  /* one ma_embedding_* call, all its launches */
  MA_K_LAYERNORM = 11,  /* one ma_layernorm_* call */
  MA_K_ACT = 12,        /* ma_act_pack, ma_act_unpack */
  MA_K_WEIGHT_GRAD = 13, /* one ma_act_weight_grad call */
  MA_K_RMSNORM = 14,    /* one ma_rmsnorm_* call */
  MA_K_MX4 = 15,        /* ma_mx4_pack, ma_mx4_unpack */
  MA_K_MX4_MATMUL = 16, /* one ma_mx4_matmul call */
  MA_K_COUNT = 17
} ma_kernel_kind;

int ma_profile_begin(int32_t max_launches);
int ma_profile_end(void);
int ma_profile_read(int32_t kind, double* total_ms, int64_t* launches);

/* ---------------------------------------------------------------------------
 * Calibration (not part of the optimizer step): the bf16 MFMA rate the part
 * sustains without memory traffic, the practical ceiling the Newton-Schulz
 * GEMMs are compared with. Launches `blocks` workgroups of 4 waves; each
 * wave issues iters x 16 independent 32x32x16 bf16 MFMAs (32768 flops each)
 * on register operands and stores one float per lane into sink (DEVICE,
 * blocks x 256 floats, 4-byte aligned). changing = 0: near-constant
 * operands; 1: random operands that change from one MFMA to the next, as a
 * real product's do (more switching, more power, and under the part's power
 * limit a lower clock). Time it with events on `stream`.
 * ------------------------------------------------------------------------- */
int ma_calib_mfma(int32_t blocks, int32_t iters, int32_t changing, float* sink, void* stream);

/* ---------------------------------------------------------------------------
 * Stage entry points, used by the test suite to check single stages with
 * identical inputs on both sides. Same conventions as above.
 * ------------------------------------------------------------------------- */

/* out[i] = bf16 bits of in[i], round to nearest even (DEVICE buffers). */
int ma_test_bf16_round(const float* in, uint16_t* out, int64_t n, void* stream);

/* Momentum stage alone for one group: M <- RNE(beta*M + G) and, in
 * mt_out (DEVICE, count*rows*cols fp32, W's layout), the look-ahead
 * G + beta*m1 (or m1 when nesterov == 0), exactly as ma_muon_step forms it. */
int ma_test_muon_momentum(const ma_muon_group* group, float beta, int32_t nesterov,
                          float* mt_out, void* stream);

/* Decay-and-update stage alone for one group: W <- RNE(post(W, U)) with
 * U (DEVICE, count dense rows x cols matrices of u_dtype, W's layout) and the
 * scalars c_lr = lr_eff, c_wd = lr_eff*wd passed as they are. Only params[]
 * of the group is used. decay == 0 skips the decay term. */
int ma_test_muon_update(const ma_muon_group* group, const void* u, int32_t u_dtype,
                        float c_lr, float c_wd, int32_t cautious, int32_t decay, void* stream);

/* Makes the calling thread's next ma_muon_adamw_step fail with MA_ERR_HIP
 * right after its fork (AdamW already queued on the side stream), as a launch
 * failure there would: for testing that the join is still enqueued. */
int ma_test_fail_after_fork(void);

/* What ma_act_weight_grad does with these sizes: the edge of its square output
 * tile (128 or 256) and the number of contiguous shares of the tokens that
 * are summed apart. Host only. */
int ma_test_act_weight_grad_plan(int64_t tokens, int64_t outs, int64_t ins, int32_t dy_dtype,
                                 int32_t* edge, int32_t* splits);

/* What ma_mx4_matmul does with these sizes: the edge of its square output tile
 * (128 or 256; 0: 16 outputs of few rows at a time) and the number of contiguous
 * shares of the columns that are summed apart. Host only. */
int ma_test_mx4_matmul_plan(int64_t rows, int64_t outs, int64_t ins, int32_t x_bits, int32_t* edge, int32_t* splits);

/* Newton-Schulz iteration alone: `count` dense m x n matrices (m <= n) in
 * x0 (DEVICE, dtype `precision`), result in u (DEVICE, same layout). */
size_t ma_test_ns_workspace_size(int64_t m, int64_t n, int32_t count, int32_t precision);
int ma_test_ns(int64_t m, int64_t n, int32_t count, int32_t precision, const void* x0, void* u,
               const float* abc, int32_t ns_steps, void* workspace, size_t workspace_bytes,
               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_ADAMW_H */
