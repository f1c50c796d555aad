/*
 * grpo.h -- C ABI of the fused, chunked GRPO policy loss for AMD MI355X (gfx950).
 *
 * What it computes (sources: Unsloth "Long-context GRPO" blog, Chinese
 * translation at zjt100.com, section on the GRPO maths; Unsloth docs "GRPO
 * with 7x longer context", sections "Flattened sequence length chunking" and
 * "Offloading activations for log softmax"; aibit.im "Mastering GRPO",
 * section "From RLHF and PPO to the efficiency of GRPO"):
 *
 *   tokens   t = b*L + j over B sequences of padded length L (N = B*L)
 *   logits   z_t = W h_t              W: [V, d] LM head, h_t: row t of H [N, d]
 *   lse_t    = log sum_v exp(z_tv)     (max-shifted, float32 or better)
 *   lp_t     = z_{t, y_t} - lse_t      selective log-softmax at the target id
 *   x_t      = ref_lp_t - lp_t
 *   kl_t     = exp(x_t) - x_t - 1      reverse KL, no extra policy factor
 *   l_t      = -(exp(lp_t - stopgrad(lp_t)) * A_{b(t)} - beta * kl_t)
 *              (the ratio's value is 1; its gradient is that of lp_t)
 *   loss     = sum_t m_t l_t / max(sum_t m_t, 1)   masked token mean
 *
 * and the backward of that loss, which recomputes every logit tile instead
 * of keeping a (tokens x vocab) tensor:
 *   c_t  = g * m_t / max(sum m, 1) * (-A_{b(t)} + beta * (1 - exp(x_t)))
 *   dZ_t = c_t * (onehot(y_t) - softmax(z_t))
 *   dH_t = dZ_t W            dW += sum_t dZ_t^T h_t
 *
 * Conventions shared by every call:
 *  - Every pointer argument is a DEVICE pointer unless stated otherwise, to a
 *    dense row-major array owned by the caller.  The library allocates no
 *    memory and keeps no state between calls beyond its loaded code objects.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls only
 *    enqueue work and return; nothing is synchronised on the host.
 *  - `dtype` (grpo_dtype) gives the element type of H, H_ref, W and dH
 *    together: GRPO_F32 (float) or GRPO_BF16 (bfloat16).  Logits, log-sum-exp
 *    and every per-token output are float32; dW is always float32.
 *  - Return value: GRPO_OK or a negative grpo_status.  Argument errors are
 *    detected on the host before anything is enqueued; no output is touched
 *    then.  GRPO_ERR_HIP means a launch failed and the outputs are undefined.
 *    grpo_last_error() returns a thread-local text describing the last
 *    failure.
 *  - Device-side preconditions not checked on the host: targets y in
 *    [0, V) (an out-of-range target gives lp = NaN in the forward and an
 *    undefined gradient), mask values in {0, 1}, and no aliasing between
 *    inputs and outputs.
 *  - Shape limits: d must be a multiple of 8 (bf16) or 4 (f32) so that rows
 *    load as 16-byte vectors; N, d, V, chunk >= 1.
 */
#ifndef GRPO_H
#define GRPO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GRPO_F32 = 0, GRPO_BF16 = 1, GRPO_FP8_E4M3 = 2 } grpo_dtype;

typedef enum {
  GRPO_OK = 0,
  GRPO_ERR_INVALID_ARG = -1, /* null pointer, size <= 0, N != B*L, bad dtype, non-finite beta */
  GRPO_ERR_WORKSPACE = -2,   /* workspace pointer null or smaller than grpo_workspace_bytes() */
  GRPO_ERR_UNSUPPORTED = -3, /* shape outside the limits above */
  GRPO_ERR_HIP = -4          /* a HIP launch or runtime call failed */
} grpo_status;

typedef enum {
  GRPO_OP_REF = 0,     /* grpo_ref_logprobs */
  GRPO_OP_FWD = 1,     /* grpo_loss_fwd */
  GRPO_OP_BWD = 2,     /* grpo_loss_bwd, default (fastest) dZ slab */
  GRPO_OP_BWD_MIN = 3, /* grpo_loss_bwd, the least workspace it accepts */
  GRPO_OP_LOGPROBS_FWD = 16, /* grpo_logprobs_fwd */
  GRPO_OP_LOGPROBS_BWD = 17  /* grpo_logprobs_bwd */
} grpo_op;

/*
 * Workspace bytes that grpo_ref_logprobs (op = GRPO_OP_REF), grpo_loss_fwd
 * (GRPO_OP_FWD) or grpo_loss_bwd (GRPO_OP_BWD, GRPO_OP_BWD_MIN) needs for
 * these sizes.  The workspace is caller-owned device memory with 256-byte
 * alignment; its contents on entry do not matter and are clobbered.  Returns
 * 0 for invalid arguments.  It never scales with N*V: the forward keeps only
 * per-token split partials of one chunk; the backward one chunk of hidden
 * states (and its transpose), per-token scalars, float32 dH partials of one
 * chunk, 8 bytes per token (active-token list, per-sequence counts) and one
 * dZ slab: the gradient of V_s vocabulary columns of the chunk's logits, in
 * H's dtype (bf16 for fp8), stored once, in strips of 256 columns that each
 * hold every active token's 256 values contiguously.
 * The backward plans V_s from the workspace_bytes it is passed: a multiple of
 * 256 columns (up to the whole vocabulary) that fits, the widest one or a
 * narrower one down to half of it where that wastes fewer waves of
 * workgroups, so a caller trades speed for memory by passing any size from
 * grpo_workspace_bytes(GRPO_OP_BWD_MIN, ...) (one 256-column slab) up.
 * GRPO_OP_BWD sizes a slab of at most 1.25 GiB (the whole vocabulary of a
 * 4096-token chunk at the usual LM-head shapes; a wider slab is not faster).
 * The slab's bytes (chunk x V_s) and V_s x d elements of W are each read
 * through one buffer resource, so V_s is also capped below 2^31 bytes for both.
 */
size_t grpo_workspace_bytes(int op, int64_t N, int64_t d, int64_t V, int dtype, int64_t chunk);

/*
 * Automatic chunk size (Unsloth docs, "Flattened sequence length chunking"
 * and "Configuring the parameters": left unset, the chunk multiplier and the
 * hidden-state mini-batch are tuned from the free VRAM and the context
 * length; the multiplier defaults to max(4, context_length // 4096)).  There
 * the chunk's float32 logits are materialised, so memory sets the chunk; here
 * the forward never holds chunk x V logits and the backward's dZ slab has its
 * own bound, so the chunk is chosen for speed within the memory given.
 * Returns the largest multiple of 256 tokens that is at most 8192 (the best
 * measured size at d = 1536 and d = 4096; at 16384 the backward slows down)
 * and at most N = B * L rounded up to 256, for which
 *   grpo_workspace_bytes(GRPO_OP_FWD, ...) + grpo_workspace_bytes(GRPO_OP_BWD, ...)
 * is at most budget_bytes; 256 if no candidate fits.  Pure host arithmetic:
 * no device call, deterministic for given arguments.
 * The caller passes its own budget (for example part of the free HBM) and
 * then uses the result for the workspace query and every call.  Returns 0
 * for invalid arguments.
 */
int64_t grpo_auto_chunk(int64_t B, int64_t L, int64_t d, int64_t V, int dtype, size_t budget_bytes);

/*
 * Group-relative advantages (aibit.im "Mastering GRPO", section "From RLHF
 * and PPO to the efficiency of GRPO": several completions per prompt are
 * scored and the advantage is derived from the group's rewards).
 *   rewards [num_groups * group_size] float32, group-major (group p holds
 *           entries p*group_size .. p*group_size + group_size - 1)
 *   adv     [num_groups * group_size] float32, written:
 *           adv = (r - mean_p) / (std_p + eps), std with divisor n - 1;
 *           a group of one has std 0 (so adv = 0).  NaN rewards propagate
 *           to their own group only.
 */
int grpo_advantages(const float* rewards, int64_t num_groups, int64_t group_size, float eps,
                    float* adv, void* stream);

/*
 * Reference-policy log-probabilities, no gradient (Unsloth blog, GRPO maths:
 * P is the frozen reference model in the reverse-KL term).
 *   H_ref [N, d] dtype; W [V, d] dtype; y [N] int32 target ids.
 *   ref_lp [N] float32, written: log softmax(W h_t)[y_t] for every token.
 *   chunk: flattened tokens per launch (>= 1); the result does not depend on it.
 * Uses exactly the same kernels as grpo_loss_fwd, so H_ref == H gives
 * ref_lp bitwise equal to lp, hence kl == 0 exactly.
 */
int grpo_ref_logprobs(const void* H_ref, const void* W, const int32_t* y, int64_t N, int64_t d,
                      int64_t V, int dtype, int64_t chunk, float* ref_lp, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Forward of the masked token-mean GRPO loss over N = B*L flattened tokens
 * (Unsloth docs, "Flattened sequence length chunking": the (batch x context)
 * axis is flattened and processed `chunk` tokens at a time; no logits are
 * ever written to memory, each vocabulary tile is folded into an online
 * log-sum-exp in registers).
 *   H [N, d] dtype; W [V, d] dtype; y [N] int32; mask [N] uint8 (0/1);
 *   adv [B] float32 (one advantage per sequence); ref_lp [N] float32.
 *   beta: KL weight (0.04 in the pages' setting), finite.
 *   loss [1] float32, written.
 *   lp, kl, lse [N] float32, written for every token, masked or not
 *   (kl unscaled by beta; lse is what grpo_loss_bwd needs back).
 */
int grpo_loss_fwd(const void* H, const void* W, const int32_t* y, const uint8_t* mask,
                  const float* adv, const float* ref_lp, int64_t B, int64_t L, int64_t d,
                  int64_t V, int dtype, float beta, int64_t chunk, float* loss, float* lp,
                  float* kl, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of grpo_loss_fwd's loss with upstream gradient grad_loss (Unsloth
 * docs, "Offloading activations for log softmax": the backward recomputes
 * the chunk's logits rather than keeping them from the forward).  Only
 * unmasked tokens are visited (masked tokens have zero gradient).
 *   H, W, y, mask, adv, ref_lp as in grpo_loss_fwd; lp and lse [N] float32
 *   are the forward's outputs for the same inputs.
 *   dH [N, d] dtype, OVERWRITTEN (rows of masked tokens become 0).
 *   dW [V, d] float32, ACCUMULATED (+=): the caller zeroes it first for a
 *   plain gradient.
 *   workspace_bytes: at least grpo_workspace_bytes(GRPO_OP_BWD_MIN, ...)
 *   (GRPO_ERR_WORKSPACE otherwise); the dZ slab is planned from it (see
 *   grpo_workspace_bytes), so results depend on it only through the
 *   summation order of dH over slabs.
 */
int grpo_loss_bwd(const void* H, const void* W, const int32_t* y, const uint8_t* mask,
                  const float* adv, const float* ref_lp, const float* lp, const float* lse,
                  int64_t B, int64_t L, int64_t d, int64_t V, int dtype, float beta,
                  float grad_loss, int64_t chunk, void* dH, float* dW, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * Options of the _ex calls.  A zero-initialised struct (or a NULL pointer)
 * gives exactly the plain calls.
 *
 * Logit transform (Unsloth docs, "Flattened sequence length chunking": the
 * chunked log-softmax takes logit_scale_multiply, logit_scale_divide,
 * logit_softcapping and temperature, and supports softcapping and
 * temperature).  The pages give no formulas; applied here in the order of
 * those arguments to every logit z = h . w before the log-softmax:
 *   z * multiply, / divide, cap * tanh(z / cap), / temperature.
 * A zero multiply, divide or cap is "off"; a zero temperature means 1.  Every
 * float field must be finite and >= 0 (GRPO_ERR_INVALID_ARG otherwise).  lp,
 * lse, kl and the gradients are those of the transformed logits.
 *
 * Loss variants (Unsloth blog, GRPO maths: the four-run ablation trains the
 * reference loss, the loss with the detach removed, a "full" reverse KL with
 * the extra factor Q and a forward KL; the formulas are lost, so these are
 * the plainest readings), with x = ref_lp - lp and r = exp(x):
 *   kl_estimator  GRPO_KL_REVERSE    kl = r - x - 1 (k3; the default)
 *                 GRPO_KL_FORWARD    kl = r x - (r - 1), the estimator of
 *                                    KL(ref || policy) from policy samples
 *                 GRPO_KL_REVERSE_Q  kl = exp(lp) (r - x - 1), the factor
 *                                    differentiated with the term
 *   no_detach     1: the ratio is exp(lp - lp) -- still 1 in value, but the
 *                 advantage term then carries no gradient
 *   aggregation   GRPO_AGG_TOKEN_MEAN     sum_t m_t l_t / max(sum m, 1)
 *                 GRPO_AGG_SEQUENCE_MEAN  (1/B) sum_b sum_j m l / max(n_b, 1),
 *                                         n_b = sum_j m_{b,j}; an empty
 *                                         sequence adds 0 and counts in B
 * The backward coefficient follows: c_t = g w_t (-[no_detach = 0] A +
 * beta dkl/dlp) with w_t the aggregation weight and dkl/dlp = 1 - r, -x r,
 * -x exp(lp) for the three estimators.  Values outside these sets:
 * GRPO_ERR_INVALID_ARG.  grpo_ref_logprobs_ex uses only the logit transform.
 */
typedef enum { GRPO_KL_REVERSE = 0, GRPO_KL_FORWARD = 1, GRPO_KL_REVERSE_Q = 2 } grpo_kl_estimator;
typedef enum { GRPO_AGG_TOKEN_MEAN = 0, GRPO_AGG_SEQUENCE_MEAN = 1 } grpo_aggregation;

typedef struct grpo_opts {
  float logit_scale_multiply;
  float logit_scale_divide;
  float logit_softcapping;
  float temperature;
  int32_t kl_estimator;   /* grpo_kl_estimator */
  int32_t no_detach;      /* 0 or 1 */
  int32_t aggregation;    /* grpo_aggregation */
} grpo_opts;

/*
 * grpo_ref_logprobs, grpo_loss_fwd and grpo_loss_bwd with options (`opts`
 * may be NULL: exactly the calls above).  Arguments and outputs are otherwise
 * those of the plain calls; grpo_loss_bwd_ex must get the opts of the
 * grpo_loss_fwd_ex call that produced lp and lse, and the reference
 * log-probs are taken with the same logit transform.  kl holds the selected
 * estimator's per-token value.
 */
int grpo_ref_logprobs_ex(const void* H_ref, const void* W, const int32_t* y, int64_t N, int64_t d,
                         int64_t V, int dtype, int64_t chunk, const grpo_opts* opts,
                         float* ref_lp, void* workspace, size_t workspace_bytes, void* stream);
int grpo_loss_fwd_ex(const void* H, const void* W, const int32_t* y, const uint8_t* mask,
                     const float* adv, const float* ref_lp, int64_t B, int64_t L, int64_t d,
                     int64_t V, int dtype, float beta, int64_t chunk, const grpo_opts* opts,
                     float* loss, float* lp, float* kl, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream);
int grpo_loss_bwd_ex(const void* H, const void* W, const int32_t* y, const uint8_t* mask,
                     const float* adv, const float* ref_lp, const float* lp, const float* lse,
                     int64_t B, int64_t L, int64_t d, int64_t V, int dtype, float beta,
                     float grad_loss, int64_t chunk, const grpo_opts* opts, void* dH,
                     float* dW, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fp8 path (Unsloth docs: FP8 RL training is offered; Unsloth blog, "Unsloth
 * efficient GRPO algorithm": a naive float8 linear cross-entropy breaks loss
 * scaling).  The pages give no recipe; here the LM-head GEMM takes OCP float8
 * e4m3 ("fn": bias 7, 3 mantissa bits, no infinities, largest 448) codes with
 * float32 accumulation (v_mfma_f32_16x16x128_f8f6f4, twice the bf16 rate) and
 * float32 log-sum-exp.  Each hidden-state row (token) has its own scale and
 * the head one scale; the logit is z = (sum_k h8 w8) * w_scale * h_scale[t].
 * Scales are powers of two, so dequantised values are exact.
 *
 * grpo_quantize_fp8: X [rows, cols] (GRPO_F32 or GRPO_BF16, device) ->
 *   codes [rows, cols] uint8 and scales (float32, device): per_row = 1 gives
 *   scales[rows], per_row = 0 one scales[0] for the tensor.  The scale of a
 *   row (or tensor) is 2^e with e the smallest integer such that its largest
 *   |x| <= 448 * 2^e (e = 0 for an all-zero block); codes are x / 2^e rounded
 *   to the nearest e4m3 value, ties to even (the division is exact).  cols must
 *   be a multiple of 16.  per_row = 0 needs grpo_quantize_fp8_workspace_bytes()
 *   of workspace (partial maxima); per_row = 1 needs none (NULL allowed).
 * grpo_dequantize_fp8: out [rows, cols] bfloat16 = codes * scale, exact.
 * grpo_ref_logprobs_fp8, grpo_loss_fwd_fp8: grpo_ref_logprobs_ex and
 *   grpo_loss_fwd_ex on fp8 codes H8 [N, d] (h_scale [N]) and W8 [V, d]
 *   (w_scale [1]); outputs and workspace (grpo_workspace_bytes with dtype
 *   GRPO_FP8_E4M3) as there.  d must be a multiple of 16.
 * grpo_loss_bwd_fp8: the backward of that loss with respect to the dequantised
 *   H and W.  The logits are recomputed from the fp8 codes through the same
 *   MFMA loop as the forward (so they equal the forward's), and dH = dZ W,
 *   dW += dZ^T H run in bfloat16 on exact bfloat16 copies of H and W that it
 *   writes into its workspace (grpo_workspace_bytes(GRPO_OP_BWD, ...,
 *   GRPO_FP8_E4M3, chunk) includes them and one chunk of gathered fp8 rows);
 *   dH [N, d] is bfloat16.
 */
size_t grpo_quantize_fp8_workspace_bytes(void);
int grpo_quantize_fp8(const void* X, int dtype, int64_t rows, int64_t cols, int per_row,
                      uint8_t* codes, float* scales, void* workspace, size_t workspace_bytes,
                      void* stream);
int grpo_dequantize_fp8(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols,
                        int per_row, void* out, void* stream);
int grpo_ref_logprobs_fp8(const uint8_t* H8, const float* h_scale, const uint8_t* W8,
                          const float* w_scale, const int32_t* y, int64_t N, int64_t d, int64_t V,
                          int64_t chunk, const grpo_opts* opts, float* ref_lp, void* workspace,
                          size_t workspace_bytes, void* stream);
int grpo_loss_fwd_fp8(const uint8_t* H8, const float* h_scale, const uint8_t* W8,
                      const float* w_scale, const int32_t* y, const uint8_t* mask,
                      const float* adv, const float* ref_lp, int64_t B, int64_t L, int64_t d,
                      int64_t V, float beta, int64_t chunk, const grpo_opts* opts, float* loss,
                      float* lp, float* kl, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream);
int grpo_loss_bwd_fp8(const uint8_t* H8, const float* h_scale, const uint8_t* W8,
                      const float* w_scale, const int32_t* y, const uint8_t* mask,
                      const float* adv, const float* ref_lp, const float* lp, const float* lse,
                      int64_t B, int64_t L, int64_t d, int64_t V, float beta, float grad_loss,
                      int64_t chunk, const grpo_opts* opts, void* dH, float* dW, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc):
 * grpo_loss_fwd_ex without a workspace argument.  Its scratch is a static
 * device array of grpo_noalloc_scratch_bytes() (64 MiB) that each GPU holds
 * for the life of the process; it is located once per device (on the first
 * call there, with that device current) and nothing is allocated, by the
 * library or on its behalf, in any call.  Shapes whose forward workspace
 * (grpo_workspace_bytes(GRPO_OP_FWD, ...)) exceeds it are rejected with
 * GRPO_ERR_WORKSPACE before anything is enqueued; that allows chunks of up
 * to 13 824 tokens at a 151 936-token vocabulary (10 496 at 201 088) for up to
 * 163 840 flattened tokens.  Every call on one GPU
 * shares that GPU's array: calls that overlap on one GPU (other streams, other
 * threads) race and give undefined results.  Nothing in the scratch needs to
 * start at zero.  Arguments and results are otherwise exactly those of
 * grpo_loss_fwd_ex, whose kernels it runs.
 */
size_t grpo_noalloc_scratch_bytes(void);
int grpo_loss_fwd_noalloc(const void* H, const void* W, const int32_t* y, const uint8_t* mask,
                          const float* adv, const float* ref_lp, int64_t B, int64_t L, int64_t d,
                          int64_t V, int dtype, float beta, int64_t chunk, const grpo_opts* opts,
                          float* loss, float* lp, float* kl, float* lse, void* stream);

/*
 * The log-probabilities of the targets and their gradient, for a loss of the caller's own over
 * them (grpo_clip_loss_*, grpo_pref_loss_*):
 *   lp_t = z_{t, y_t} - lse_t,  dZ_t = g_t (onehot(y_t) - softmax(z_t)) dz/d(w h)
 *   dH_t = dZ_t W               dW += sum_t dZ_t^T h_t
 * with z the transformed logits of the opts (NULL: plain) and g = grad_lp, the loss's gradient
 * with respect to lp.
 * grpo_logprobs_fwd: lp [N] and lse, float32, written.  With GRPO_BF16 lse has N elements, and both
 *   are bitwise grpo_ref_logprobs's and grpo_loss_fwd's.  With GRPO_F32 lse has 2 N, behind each
 *   token's value what its rounding to float32 left, N elements on; lp is formed without that rounding,
 *   and equals theirs within it.
 * grpo_logprobs_bwd: lp and lse as the forward of the same inputs and opts wrote them.  A token with
 *   g_t = 0 has no part in it, whatever its other values are: its row of dH is 0.  dH [N, d] dtype,
 *   OVERWRITTEN; dW [V, d] dw_dtype, ACCUMULATED if accumulate is 1, OVERWRITTEN if it is 0; either
 *   may be NULL and is then not formed.  dw_dtype is GRPO_F32, or with a bfloat16 head, accumulate 0
 *   and chunk >= N also GRPO_BF16: then each sum is rounded once.
 * workspace: grpo_workspace_bytes(GRPO_OP_LOGPROBS_FWD or GRPO_OP_LOGPROBS_BWD, ...), 256-byte aligned.  A smaller chunk
 *   needs less; results depend on it through the order in which dW's and, in bfloat16, dH's parts are summed.
 * dtype GRPO_F32 or GRPO_BF16.  H, W, dH and dW 16-byte aligned.  Outputs and workspace lie apart from the
 * inputs and from each other (others are refused).  Only the logit transform of the opts is used.
 */
int grpo_logprobs_fwd(const void* H, const void* W, const int32_t* y, int64_t N, int64_t d,
                      int64_t V, int dtype, int64_t chunk, const grpo_opts* opts, float* lp,
                      float* lse, void* workspace, size_t workspace_bytes, void* stream);
int grpo_logprobs_bwd(const void* H, const void* W, const int32_t* y, const float* lp,
                      const float* lse, const float* grad_lp, int64_t N, int64_t d, int64_t V,
                      int dtype, int64_t chunk, const grpo_opts* opts, int accumulate,
                      int dw_dtype, void* dH, void* dW, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * The clipped policy loss over given log-probabilities, for steps in which the policy is no longer
 * the one that sampled.  For the unmasked tokens t = b L + j of B sequences, n_b of them in b, n in
 * all, with D = lp - old_lp (0 where old_lp is NULL):
 *   r = exp(D_t)                              (GRPO_RATIO_TOKEN)
 *   r = exp(sum_j m D / n_b)                  (GRPO_RATIO_SEQUENCE: the same for all tokens of b)
 *   s = min(r, 1 + clip_high) where A >= 0, min(max(r, 1 - clip_low), clip_dual) where A < 0
 *   l = -A s + beta kl(ref_lp - lp, lp)       kl as in grpo_opts; no term where ref_lp is NULL
 *   loss = sum_t m_t l_t / max(n, 1), or (1/B) sum_b sum_j m l / max(n_b, 1)
 * and its gradient with respect to lp (with w_t the weight of l_t in the loss):
 *   g_t = w_t ((s = r ? -A r : 0) + beta dkl/dlp)
 * What masked places hold (NaN, infinities) plays no part.  Which side of a border a ratio is on is
 * decided in float64 by its logarithm.  Sums are float64, in a fixed order, but that four adjacent tokens' kl, and
 * r - 1 - log r, which are not negative, first join in float32.
 *   lp, old_lp (NULL), ref_lp (NULL) [N] float32; mask [N] uint8; adv float32 [B], or [N] if
 *   adv_per_token is 1 (GRPO_RATIO_TOKEN only).  lp, old_lp and ref_lp under the same logit transform.
 * grpo_clip_loss_fwd: loss [1] and stats [4] float32, written: over the unmasked tokens the mean of kl
 *   (0 without ref_lp), the share of tokens with s > r, the share with s < r, and the mean of
 *   r - 1 - log r (an estimate of the divergence from the old policy).  weights [2 B + 1] float32, written, for
 *   the backward: for each sequence the factor of its terms (1, or 1 / max(n_b, 1) for the mean over sequences) and
 *   the slope of its ratio (0 for a ratio a token), then the weight of all.  workspace: grpo_clip_loss_workspace_bytes(B, L), 256-byte aligned.
 * grpo_clip_loss_bwd: grad_lp [N] float32, OVERWRITTEN (0 where masked) = g times *grad_loss (a device
 *   scalar; NULL: 1).  Other arguments and opts are the forward's.
 * Outputs and workspace lie apart from the inputs and from each other (others are refused).
 * opts (NULL: all zeros): zeros are "off": no clipping on that side, no KL term.  clip_low, clip_high
 * finite and >= 0, clip_dual 0 or finite and > 1, beta finite.  beta != 0 needs ref_lp.
 * B * L must fit int32.
 */
typedef enum { GRPO_RATIO_TOKEN = 0, GRPO_RATIO_SEQUENCE = 1 } grpo_ratio;

typedef struct grpo_clip_opts {
  double clip_low;
  double clip_high;
  double clip_dual;
  double beta;
  int32_t ratio;          /* grpo_ratio */
  int32_t kl_estimator;   /* grpo_kl_estimator */
  int32_t aggregation;    /* grpo_aggregation */
  int32_t adv_per_token;  /* 0 or 1 */
} grpo_clip_opts;

size_t grpo_clip_loss_workspace_bytes(int64_t B, int64_t L);
int grpo_clip_loss_fwd(const float* lp, const float* old_lp, const float* ref_lp,
                       const uint8_t* mask, const float* adv, int64_t B, int64_t L,
                       const grpo_clip_opts* opts, float* loss, float* stats, float* weights,
                       void* workspace, size_t workspace_bytes, void* stream);
int grpo_clip_loss_bwd(const float* lp, const float* old_lp, const float* ref_lp,
                       const uint8_t* mask, const float* adv, const float* weights,
                       const float* grad_loss, int64_t B, int64_t L, const grpo_clip_opts* opts,
                       float* grad_lp, void* stream);

/*
 * The preference loss over P pairs of sequences of padded length L: sequence 2p is the chosen one of
 * pair p, 2p + 1 the rejected one (N = 2 P L tokens).  For sequence b with n_b unmasked tokens:
 *   s_b = sum_j m (lp - ref_lp)     (without ref_lp, which may be NULL: sum_j m lp)
 *         divided by max(n_b, 1) if length_mean is 1
 *   h = s_{2p} - s_{2p+1},  x = beta h - margin
 *   l = -(1 - label_smoothing) log sigmoid(x) - label_smoothing log sigmoid(-x)   GRPO_PREF_SIGMOID
 *       max(0, 1 - x)                                                            GRPO_PREF_HINGE
 *       (h - margin - 1 / (2 beta))^2                                            GRPO_PREF_SQUARE
 *   l += nll_weight (-sum_j m lp_{2p} / max(n_{2p}, 1))
 *   loss = (1/P) sum_p l
 * grpo_pref_loss_fwd: loss [1], rewards [2 P] = beta s_b and weights [2 P] (the loss's gradient with
 *   respect to each unmasked lp of a sequence) float32, written.  workspace:
 *   grpo_pref_loss_workspace_bytes(P, L), 256-byte aligned.
 * grpo_pref_loss_bwd: grad_lp [N] float32, OVERWRITTEN (0 where masked): the sequence's weight times
 *   *grad_loss (a device scalar; NULL: 1).
 * Outputs and workspace lie apart from the inputs and from each other (others are refused).
 * What masked places hold plays no part.  beta finite and > 0, margin and nll_weight finite,
 * nll_weight >= 0, label_smoothing in [0, 1) and, but for GRPO_PREF_SIGMOID, 0.  2 P L must fit int32.
 */
typedef enum { GRPO_PREF_SIGMOID = 0, GRPO_PREF_HINGE = 1, GRPO_PREF_SQUARE = 2 } grpo_pref_kind;

typedef struct grpo_pref_opts {
  double beta;
  double label_smoothing;
  double margin;
  double nll_weight;
  int32_t kind;         /* grpo_pref_kind */
  int32_t length_mean;  /* 0 or 1 */
} grpo_pref_opts;

size_t grpo_pref_loss_workspace_bytes(int64_t P, int64_t L);
int grpo_pref_loss_fwd(const float* lp, const float* ref_lp, const uint8_t* mask, int64_t P,
                       int64_t L, const grpo_pref_opts* opts, float* loss, float* rewards,
                       float* weights, void* workspace, size_t workspace_bytes, void* stream);
int grpo_pref_loss_bwd(const uint8_t* mask, const float* weights, const float* grad_loss,
                       int64_t P, int64_t L, float* grad_lp, void* stream);

/*
 * The norm of many gradients as one vector, and the factor that clips it: what grpo_adamw takes as
 * grad_scale.
 *   norm  = sqrt(sum g^2) (GRPO_GRAD_NORM_L2) or max |g| (GRPO_GRAD_NORM_MAX)
 *   scale = min(1, max_norm / (norm + 1e-6)), or 1 if max_norm is 0
 * A NaN makes both NaN (scale 1 if max_norm is 0); infinities make norm inf and scale 0.
 * grpo_grad_plan (host only) checks the tensors and writes the table into the HOST buffer `image`
 *   of grpo_grad_plan_bytes(count) bytes, to be copied to device memory once (8-byte aligned) and
 *   passed along with it, as in grpo_adamw_plan.  Types may be mixed; n = 0 is allowed; tensors that
 *   share memory are refused.  At most 2^24 tensors, and 2^22 - 1 chunks of 8192 elements (3.4e10).
 * grpo_grad_norm: norm [1] and scale [1] float32, written.  Squares and sums are float64, in a fixed
 *   order: nothing overflows, and results are bitwise reproducible.  max_norm finite and >= 0.  workspace:
 *   grpo_grad_norm_workspace_bytes(), 256-byte aligned.
 * grpo_grad_clip: every gradient times *scale (a device scalar), in place, rounded to its type;
 *   nothing is touched where it is 1.
 * norm, scale and workspace lie apart from every gradient and from each other (others are refused).
 */
typedef enum { GRPO_GRAD_NORM_L2 = 0, GRPO_GRAD_NORM_MAX = 1 } grpo_grad_norm_kind;

typedef struct grpo_grad_tensor {
  void* grad;
  int64_t n;
  int32_t dtype;     /* GRPO_F32 or GRPO_BF16 */
  int32_t reserved;  /* not read */
} grpo_grad_tensor;

size_t grpo_grad_plan_bytes(int64_t count);
int grpo_grad_plan(const grpo_grad_tensor* tensors, int64_t count, void* image,
                   size_t image_bytes);
size_t grpo_grad_norm_workspace_bytes(void);
int grpo_grad_norm(const void* image, const void* plan, int kind, double max_norm, float* norm,
                   float* scale, void* workspace, size_t workspace_bytes, void* stream);
int grpo_grad_clip(const void* image, const void* plan, const float* scale, void* stream);

/*
 * The norm in front of the LM head, whose output is H and whose backward takes
 * dH.  For each row x of X [rows, cols]:
 *   mu = mean(x) (GRPO_NORM_LAYER; 0 for GRPO_NORM_RMS)
 *   r  = 1 / sqrt(mean((x - mu)^2) + eps)
 *   y  = (x - mu) r weight + bias
 * grpo_norm_fwd: X, weight [cols], bias [cols] (NULL: none) and Y [rows, cols]
 *   are `dtype` (GRPO_F32 or GRPO_BF16); mean and rstd [rows] are float32,
 *   written (mean is not used for GRPO_NORM_RMS and may be NULL).  eps finite
 *   and >= 0.
 * grpo_norm_bwd: dY [rows, cols] the gradient of Y; X, weight, mean and rstd
 *   as in the forward.  dX [rows, cols] dtype, OVERWRITTEN; dweight [cols] and
 *   dbias [cols] (NULL: not formed) float32, ACCUMULATED (+=, as dW is in
 *   grpo_loss_bwd) if accumulate is 1, OVERWRITTEN if it is 0.  workspace:
 *   grpo_norm_workspace_bytes(rows, cols, dtype), 256-byte aligned.
 * Y is not X, nor dX dY or X (refused), and outputs overlap no input.
 * Any cols from 1 to 2^24 and any element alignment.  Sums are float32, in a
 * fixed order: results are bitwise reproducible.  Squares are float32 too:
 * where a row's sum of them passes its range (|x - mu| of about 1e19 /
 * sqrt(cols)), r is 0 and y the bias.
 */
typedef enum { GRPO_NORM_LAYER = 0, GRPO_NORM_RMS = 1 } grpo_norm_kind;

size_t grpo_norm_workspace_bytes(int64_t rows, int64_t cols, int dtype);
int grpo_norm_fwd(const void* X, const void* weight, const void* bias, int64_t rows, int64_t cols,
                  int dtype, int kind, float eps, void* Y, float* mean, float* rstd, void* stream);
int grpo_norm_bwd(const void* dY, const void* X, const void* weight, const float* mean,
                  const float* rstd, int64_t rows, int64_t cols, int dtype, int kind,
                  int accumulate, void* dX, float* dweight, float* dbias, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * One AdamW step over many tensors in one launch; the consumer of
 * grpo_loss_bwd's dW and grpo_norm_bwd's dweight.  For every element, with
 * g = grad * grad_scale and step t >= 1:
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   w = w - lr weight_decay w - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * w is the float32 master where there is one (all tensors have one, or none),
 * and param its rounding; else w is param itself.
 *
 * grpo_adamw_plan (host only) checks the tensors and writes the step's table
 *   into the HOST buffer `image` of grpo_adamw_plan_bytes(count) bytes.  The
 *   caller copies image to device memory once (8-byte aligned) and passes
 *   both to every grpo_adamw: image is read on the host during the call, plan
 *   (the device copy) by the kernel.  Both hold the tensors' addresses: a tensor that
 *   moves needs a new plan.  Tensors that share memory (one twice) are
 *   refused; n = 0 is allowed.  At most 2^24 tensors, and 2^24 - 1 chunks of
 *   2048 elements (3.4e10 elements).
 *   param_dtype, grad_dtype: GRPO_F32 or GRPO_BF16, the same for all tensors;
 *   a master goes with bfloat16 parameters only.
 *   state_bits 32: exp_avg and exp_avg_sq are float32 [n] (scales unused).
 *   state_bits 8: exp_avg is int8 [n], exp_avg_sq uint8 [n], with one float32
 *   scale a per 256 elements of the tensor (scales [ceil(n / 256)]), the
 *   largest |value| of the block (NaN if one is not finite):
 *     exp_avg    = sign(c) (c / 127)^2 a,  c rounded from 127 sqrt(|m| / a)
 *     exp_avg_sq = (c / 255)^4 a,          c rounded from 255 (v / a)^(1/4),
 *                                          at least 1 where v > 0
 *   All zeros is the state before the first step.  The new codes are those of
 *   the moments in float64, beta m + (1 - beta) g with each product and sum
 *   rounded; the weights use the moments before their rounding to codes.
 * grpo_adamw: betas in [0, 1); lr, eps and weight_decay finite in
 *   float32 and >= 0; step the number of this step, from 1.  Device-side values,
 *   each read when the kernel runs if non-NULL (for a step under graph capture):
 *   step_dev [1] int64
 *   in place of step (below 1 counts as 1), lr_dev [1] float32 in place of lr,
 *   grad_scale [1] float32 (NULL: 1).
 * grpo_moment_values: the float32 values of 8-bit codes (squared = 0: exp_avg's
 *   int8, 1: exp_avg_sq's uint8).
 */
typedef struct grpo_adamw_tensor {
  void* param;
  const void* grad;
  float* master;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scales;
  float* exp_avg_sq_scales;
  int64_t n;
} grpo_adamw_tensor;

typedef struct grpo_adamw_opts {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
} grpo_adamw_opts;

size_t grpo_adamw_plan_bytes(int64_t count);
int grpo_adamw_plan(const grpo_adamw_tensor* tensors, int64_t count, int param_dtype,
                    int grad_dtype, int state_bits, void* image, size_t image_bytes);
int grpo_adamw(const void* image, const void* plan, const grpo_adamw_opts* opts, void* stream);
int grpo_moment_values(const void* codes, const float* scales, int64_t n, int squared, float* out,
                       void* stream);

/*
 * One token for each row of logits [B, V] (GRPO_F32 or GRPO_BF16; row b starts at
 * logits + b * row_stride elements, row_stride >= V), from u [B] float32, one
 * uniform number in [0, 1) per row (a value outside counts as the nearest
 * bound, a NaN as 0).  The rollout's last step: token [B] int32 becomes y, lp [B] float32
 * the behaviour policy's log-probability.
 *   z = x / temperature, e = exp(z - max z); the tokens in the order (x down,
 *   index up).  top_k keeps the first top_k; top_p, of those, the ones whose
 *   mass before them is below top_p times the mass of those; min_p, of those,
 *   the ones with e >= min_p.
 *   token: the lowest index whose running kept mass, in index order, exceeds u
 *   times the kept mass.
 *   lp: z[token] - log sum exp z over the whole row, filters or not: what
 *   grpo_loss_fwd_ex gives as lp for that token and temperature.
 * Zeros in opts (or opts = NULL) are "off": temperature 1, no filter; top_k >= V
 * and top_p = 1 are off too, and top_k = 1 takes the largest logit (temperature
 * 0 does not: it samples at temperature 1).  The scalars
 * hold for all rows; a non-NULL ..._rows device array [B] gives each row its own
 * instead (there, values out of range are off for the filters; min_p above 1
 * counts as 1).
 * -inf logits are tokens that cannot be drawn.  A row with a NaN or +inf, with
 * nothing above -inf, or with a device-side temperature that is negative or
 * not finite has token -1 and lp NaN.
 * Whatever decides a token is computed in 64 bits.  Tokens lighter than 2^-1000
 * of the heaviest (of a row with a filter: than 2^-43, since its weights are
 * whole multiples of 2^-42) have no mass and are not drawn, whatever u is.
 * V and B at most 2^20.
 * workspace: grpo_sample_workspace_bytes(B, V), 256-byte aligned.
 */
typedef struct grpo_sample_opts {
  double temperature;
  double top_p;
  double min_p;
  int32_t top_k;
  int32_t reserved; /* not read */
  const float* temperature_rows;
  const float* top_p_rows;
  const float* min_p_rows;
  const int32_t* top_k_rows;
} grpo_sample_opts;

size_t grpo_sample_workspace_bytes(int64_t B, int64_t V);
int grpo_sample(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                const float* u, const grpo_sample_opts* opts, int32_t* token, float* lp,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Diagnostic: C[M, N] (float32, row-major, written) = A[M, K] . B[N, K]^T,
 * through the same MFMA tile main loop the loss kernels use (A, B dtype
 * elements, both rows contiguous along K).  K times the element size must be
 * a multiple of 16 bytes.  Used by the parity tests to check that loop on
 * its own; not part of the loss itself.
 */
int grpo_gemm_nt(const void* A, const void* B, int64_t M, int64_t N, int64_t K, int dtype,
                 float* C, void* stream);

/*
 * Diagnostics: per-kernel timing with HIP events, off by default.  After
 * grpo_timing_begin(), every kernel launch that this thread's library calls
 * enqueue is bracketed by two HIP events recorded on the launch's own stream.
 * grpo_timing_end() waits for those events and writes, for each kernel that
 * ran, its name (static string), launch count and summed elapsed time in
 * milliseconds into the caller's HOST arrays of max_entries; it returns the
 * number of kernels that ran (entries past max_entries are dropped) and
 * switches timing off.  Used by the benchmark for its roofline figure.
 */
int grpo_timing_begin(void);
int grpo_timing_end(const char** names, int* launches, double* total_ms, int max_entries);

/* Static text for a grpo_status code. */
const char* grpo_strerror(int code);

/* Thread-local text describing the most recent failure on this thread ("" if none). */
const char* grpo_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GRPO_H */
