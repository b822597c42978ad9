/*
 * hylo_ops.h — C ABI of the operators that stand beside the distillation losses of hylo_kl.h
 * (GB300, sm_103a): log-probabilities of given tokens, the AdamW and Muon steps that apply the
 * gradients, orthogonalised matrices, and the norms of the hidden states.
 *
 * Conventions are those of hylo_kl.h: device pointers owned by the caller unless a parameter
 * says otherwise, no allocation by the library, calls asynchronous on `stream`, a status code
 * for argument, architecture and launch errors (hylo_kl_last_error() has the text), no
 * fallback. Calls may be captured into a CUDA graph once one call has run eagerly on the device, all
 * but hylo_adamw_step and hylo_muon_step.
 */
#ifndef HYLO_OPS_H
#define HYLO_OPS_H

#include "hylo_kl.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { HYLO_F32 = 0, HYLO_BF16 = 1, HYLO_F16 = 2 } hylo_dtype;

#define HYLO_TOP_MAX 64 /* largest number of alternatives per row */

/* Log-probabilities of given tokens from logits, with entropy and top alternatives. Per row n:
 *     y = z[n] / tau,  m = max_v y_v,  s = sum_v exp(y_v - m),  lp_v = y_v - m - log s
 *     logp[n] = lp_tokens[n],  entropy[n] = -sum_v exp(lp_v) lp_v,  lse[n] = m + log s
 *     top_ids[n, j], top_logp[n, j]: the k words of largest logit, largest first, and their lp.
 * z: [N, V] of `dtype`, row stride ld elements (ld >= V; any ld and any element-aligned start).
 * tokens [N]: a negative token is ignored (logp 0); a token >= V gives logp NaN. Any int64 value
 * is safe. entropy, lse, stats may be NULL; top_logp and top_ids only if k = 0.
 * stats [N, 2] receives (max_v z_v, log s), which the backward reads.
 * Logits may be -inf (masked words): such a word has probability 0, and a row of only -inf has
 * logp, lse and top_logp -inf, entropy 0, and a zero gradient. A NaN or +inf anywhere in a row makes
 * logp, entropy, lse and top_logp of that row NaN (an ignored token's logp is 0 all the same); for the order of
 * alternatives NaN counts as larger than any number. Equal logits (also -0 and +0) go to the lowest index first.
 * 1 <= N, V <= 2^31 - 1; 0 <= k <= min(V, HYLO_TOP_MAX); tau and log2(e) / tau finite and > 0. Statistics are
 * fp32. Results are deterministic. Needs no workspace. */
hylo_status hylo_token_logprobs(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau,
                                const int64_t* tokens, int k, float* logp, float* entropy, float* lse,
                                float* stats, float* top_logp, int64_t* top_ids, cudaStream_t stream);

/* Gradient of sum_n g_logp[n] logp[n] + g_entropy[n] entropy[n] with respect to z:
 *     dz[n, v] = ( g_logp[n] (1[v = tokens[n]] - p_v) - g_entropy[n] p_v (lp_v + entropy[n]) ) / tau
 * (no g_logp term for an ignored token), as `dtype` in rows of stride ldd (columns v >= V
 * untouched). stats and entropy are the forward's. g_logp or g_entropy may be NULL (zero; both
 * NULL: dz = 0); entropy may be NULL if g_entropy is. dz may not overlap z unless it is z itself
 * with ldd = ld. */
hylo_status hylo_token_logprobs_backward(const void* z, int dtype, int64_t N, int64_t V, int64_t ld, float tau,
                                         const int64_t* tokens, const float* stats, const float* entropy,
                                         const float* g_logp, const float* g_entropy, void* dz, int64_t ldd,
                                         cudaStream_t stream);

/* The same log-probabilities and entropies for z = h W^T, without storing z: h [N, d] final hidden
 * states, W [V, d] LM head, bf16 bit patterns, row-major and contiguous, 16-byte aligned, d a multiple
 * of 8 in 8..65536. Inputs are meant finite (where they are not, the results of the tokens
 * concerned are NaN or infinite). tokens as above. entropy and lse may be NULL; the backward needs lse
 * (and entropy, if g_entropy is given). workspace: 256-byte aligned, not shared with a call still running
 * on another stream, and at least as long as the query says. ..._forward_workspace_bytes() is what the
 * forward needs: O(N), and up to 640 KiB for copies of few hidden states. ..._backward_workspace_bytes() is
 * what the backward needs for the gradients that are wanted (want_dh: dh is not NULL; want_dW the same):
 * the G ring of hylo_kl_backward (at most 128 MiB, twice that with split_g), the fp32 parts
 * that dh is joined from where N <= 1024 (at most 128 MiB) and, for bf16 gradients, the fp32 sums
 * behind them: N d of dh, and V d of dW if N is more than one token block.
 * hylo_head_logprobs_workspace_bytes() is enough for both directions with both gradients.
 * Accuracy: a logit is accumulated by the tensor cores in fp32 over at most 64 steps of 16 products, and these sums
 * are added up rounded to nearest, which can drift by up to 2^-18 of the logits' scale in one direction whatever d is
 * (measured 3e-7 of it). Without lse, those of one or two tokens are fp32 multiply-adds. Where lse is asked for,
 * they are accumulated as the backward will accumulate them again, so that its probabilities
 * exp(z - lse) are those of the forward to a few fp32 roundings of lse.
 * Each returns 0 for invalid sizes; token_chunk <= 0 means 4096; grad_dtype as in the backward. */
size_t hylo_head_logprobs_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t token_chunk, int split_g,
                                          int grad_dtype);
size_t hylo_head_logprobs_forward_workspace_bytes(int64_t N, int64_t d, int64_t V);
size_t hylo_head_logprobs_backward_workspace_bytes(int64_t N, int64_t d, int64_t V, int64_t token_chunk, int split_g,
                                                   int grad_dtype, int want_dh, int want_dW);
hylo_status hylo_head_logprobs(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V, float tau,
                               const int64_t* tokens, float* logp, float* entropy, float* lse, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/* Gradients of sum_n g_logp[n] logp[n] + g_entropy[n] entropy[n]: with G = dL/dz as in
 * hylo_token_logprobs_backward (recomputed tile by tile, rounded to bf16 once, or with split_g != 0
 * kept as two bf16 terms), dh = G W [N, d] and dW = G^T h [V, d], summed in fp32 and OVERWRITTEN as
 * grad_dtype (HYLO_F32 or HYLO_BF16, rounded once). Either may be NULL: that product is then left
 * out (frozen hidden states or LM head). lse and entropy are the forward's for the same inputs.
 * token_chunk as in hylo_kl_backward. Deterministic. */
hylo_status hylo_head_logprobs_backward(const uint16_t* h, const uint16_t* W, int64_t N, int64_t d, int64_t V,
                                        float tau, int64_t token_chunk, const int64_t* tokens, const float* lse,
                                        const float* entropy, const float* g_logp, const float* g_entropy, int split_g,
                                        int grad_dtype, void* dh, void* dW, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

/* One tensor of an optimizer step. All arrays have `n` elements and start element-aligned. No array that
 * the step writes may overlap another array of the step (a tensor given twice, a gradient that is the
 * parameter): HYLO_ERR_DIM. Tensors may share a gradient, which is only read. */
typedef struct {
  void* param;        /* fp32, or bf16 (see hylo_adamw_step) */
  const void* grad;   /* fp32 or bf16 */
  float* master;      /* fp32 copy of a bf16 param that the step is taken on, or NULL */
  void* m;            /* first moment: fp32, or e4m3 codes (uint8) */
  void* v;            /* second moment: fp32, or e4m3 codes (uint8) of its square root */
  int8_t* m_exp;      /* 8-bit states: one exponent per 256 elements, [ceil(n / 256)]; else NULL */
  int8_t* v_exp;
  int64_t n;          /* 0 <= n <= 2^40 */
  double lr;
  double weight_decay;
} hylo_adamw_tensor;

/* Global norm of a list of gradients: norm[0] = sqrt(sum over tensors, elements of g^2), fp32.
 * grads, sizes: HOST arrays of `count` device pointers and element counts; `dtype` HYLO_F32 or
 * HYLO_BF16 for all. workspace: hylo_grad_norm_workspace_bytes() bytes, 16-byte aligned, not
 * shared with a call still running on another stream. Summed in a fixed order (deterministic
 * on one kind of device); partial sums are fp32, their total fp64. count may be 0 (norm 0). */
size_t hylo_grad_norm_workspace_bytes(void);
hylo_status hylo_grad_norm(const void* const* grads, const int64_t* sizes, int count, int dtype, float* norm,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* One AdamW step (decoupled weight decay) over `count` tensors (HOST array, not kept):
 *     g' = g * grad_scale * c,  c = min(1, max_norm / (norm[0] * |grad_scale| + 1e-6))  (1 without norm)
 *     m <- beta1 m + (1 - beta1) g',   v <- beta2 v + (1 - beta2) g'^2
 *     w <- w (1 - lr weight_decay) - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 * norm (device, may be NULL) is the fp32 norm of the gradients as given (hylo_grad_norm). If it
 * is not finite the whole step is skipped: nothing is written.
 * All tensors of a call share param_dtype (HYLO_F32 or HYLO_BF16), grad_dtype (the same two) and
 * state_bits (32 or 8). fp32 parameters take master = NULL. bf16 parameters either all have
 * a master (w is the master; the param receives it rounded to nearest) or none (w is the param,
 * rounded stochastically).
 *
 * 8-bit states. m, and r = sqrt(v) for the second moment, are kept as e4m3 codes q with one power of two
 * per 256 consecutive elements of the tensor: value = q 2^e. After the update e is chosen so
 * that the block's largest finite magnitude lies in [128, 256) 2^e (e within [-120, 120]; -120 for a
 * block of zeros) and each magnitude x 2^-e is rounded to a neighbouring e4m3 value, up with
 * the probability of the part cut off, so that small steady changes are not lost (to nearest,
 * 0.999 v would round back to v for ever). A non-zero r is never stored as 0. eps must be >= 2^-126. A value that is not finite is
 * stored as NaN and leaves the other elements of its block alone.
 * Order of rounding. The last bit of a moment can decide its code, and the next step takes the whole code's
 * difference into the parameter, so m, v and r are defined to the last bit. With fl the rounding to fp32 (to nearest) of each
 * single operation, b1, b2, 1 - b1, 1 - b2 rounded from the double arguments, and c from the norm as given:
 *     c  = min(1, fl(max_norm / fl(norm[0] |grad_scale| + 1e-6))),  s = fl(grad_scale c),  g' = fl(g s)
 *     m <- fl(fl(b1 m) + fl((1 - b1) g'))
 *     v <- fl(fl(b2 (r r)) + fl((1 - b2) fl(g' g'))), taken as 0 below 2^-126,  r <- fl(sqrt(v))
 *     code of x: y = fl(|x| 2^-e), below 2^-6 rounded to a multiple of 2^-29; q = the multiple of the e4m3 step below
 *     y / step + (16 random bits) 2^-16, exactly
 * (fl(norm |grad_scale| + 1e-6) is one rounding.) The parameter's own update has no such order; it is within a few fp32
 * roundings of the formula.
 * The random bits: element j of tensor i has position c = B_i + j, B_i = the sum of the sizes
 * of the tensors before it, each rounded up to 256; with mix = the 32-bit finaliser of
 * MurmurHash3 (public domain), low/high the halves of c,
 *     bits = mix(low(c) + mix(seed + 0x9E3779B9 (high(c) + 1)))   (all modulo 2^32)
 * m takes the low 16 bits, r the high 16, and a bf16 param without master the high 16 of
 * bits * 0x9E3779B1. Pass another seed each step. The same seed and inputs give the same result.
 * A step may not be captured into a CUDA graph (HYLO_ERR_CAPTURE): step, the learning rates and seed are the host's, and
 * every replay would repeat one step's bias corrections and one step's random bits. */
hylo_status hylo_adamw_step(const hylo_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype,
                            int state_bits, double beta1, double beta2, double eps, int64_t step,
                            float grad_scale, const float* norm, float max_norm, uint32_t seed,
                            cudaStream_t stream);

/* Layer norm (rms = 0) or RMS norm (rms != 0) of rows, with the sum of two streams in front. Per row:
 *     s = x + residual, rounded to `dtype` (s = x if residual is NULL);  mu = mean(s) (RMS: 0)
 *     r = 1 / sqrt(mean((s - mu)^2) + eps),  y = (s - mu) r weight + bias
 * x, residual: [N, d] of `dtype` (HYLO_F32, HYLO_BF16, HYLO_F16), row strides ldx, ldr >= d elements; y, sum: [N, d],
 * contiguous. weight, bias: [d] or NULL (1 and 0), both of gain_dtype, which is dtype or HYLO_F32. All element-aligned; rows of
 * 16-byte vectors are fastest. sum receives s and is required with a residual (NULL without). stats [N, 2] receives (mu, r),
 * which the backward reads, or is NULL. y and sum may not overlap the inputs or each other. 1 <= N <= 2^31 - 1,
 * 1 <= d <= 2^20, eps finite and >= 0. Statistics are fp32: where mean((s - mu)^2) exceeds fp32's range the row's y is that of r = 0
 * (RMS norm of a row with infinite elements: NaN there, 0 elsewhere; a NaN makes the row NaN).
 * With eps = 0 a row without deviation has r infinite, and NaN. Deterministic. */
hylo_status hylo_norm(const void* x, const void* residual, int dtype, int64_t N, int64_t d, int64_t ldx, int64_t ldr,
                      const void* weight, const void* bias, int gain_dtype, int rms, double eps, void* sum, void* y,
                      float* stats, cudaStream_t stream);

/* Its gradients. s is the forward's sum, or x without a residual (row stride lds); stats the forward's; dy [N, d] (row stride
 * lddy) the gradient of y, dsum [N, d] (row stride ldds) that of sum, or NULL:
 *     g = dy weight,  xh = (s - mu) r,  dx = r (g - mean(g) - xh mean(g xh)) + dsum   (RMS: without mean(g))
 *     dweight = sum over rows of dy xh,  dbias = sum over rows of dy
 * dx [N, d] contiguous, of `dtype` (x and residual have the same gradient); dweight, dbias [d] of gain_dtype (summed in fp32,
 * rounded once). Any of the three may be NULL: it is left out. They are OVERWRITTEN and may not overlap the inputs or each
 * other. workspace: 16-byte aligned, at least hylo_norm_backward_workspace_bytes() (0 for invalid sizes), not shared
 * with a call still running on another stream; may be NULL without dweight and dbias. Deterministic: sums in a fixed order. */
size_t hylo_norm_backward_workspace_bytes(int64_t N, int64_t d);
hylo_status hylo_norm_backward(const void* s, int dtype, int64_t N, int64_t d, int64_t lds, const void* weight,
                               int gain_dtype, int rms, const float* stats, const void* dy, int64_t lddy,
                               const void* dsum, int64_t ldds, void* dx, void* dweight, void* dbias, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/* Orthogonalised matrices. Each matrix M of the list (HOST array, not kept) is scaled to X = M / (|M| + eps), |M| its Frobenius
 * norm, and `steps` Newton-Schulz steps with coefficients[3 k ..] = (a, b, c) of step k (HOST array [steps][3]) follow:
 *     A = X X^T,  X <- a X + (b A + c A^2) X
 * which leaves M's singular vectors and takes each singular value s to a s + b s^3 + c s^5, step by step (of a matrix with
 * more rows than columns X is the transpose). x: [rows, cols] of `dtype` (fp32, bf16 or fp16), row stride ld >= cols; out:
 * [rows, cols] contiguous, of out_dtype (HYLO_BF16 or HYLO_F16). rows, cols <= 2^20, the shorter at most 16384; a
 * matrix without elements is skipped. 1 <= steps <= 32. Coefficients with which singular values could pass 2^20 are refused.
 * A matrix of zeros gives zeros; NaN or infinity anywhere in a matrix makes that whole result NaN, and leaves the others alone. No
 * output may overlap anything else. workspace: 256-byte aligned, hylo_orthogonalize_workspace_bytes() of the same list
 * (0 for invalid sizes; 6 bytes per element and 4 per element of A, padded, for matrices of together 1 GiB or one larger
 * one, and parts of long sums), not shared with a call still running on another stream.
 * Accuracy: products of fp16 numbers scaled by powers of two, fp32 sums, X as two fp16 terms where it is added: 1e-3 to 2e-3 of
 * the result's norm after five steps with the usual coefficients, up to 4e-3 where few singular values share it (one row).
 * Deterministic: the same list gives the same bits (with other matrices in the list, the sums of a matrix with a side of more
 * than 8128 may be added up in another order). */
typedef struct {
  const void* x;
  void* out;
  int64_t rows, cols, ld;
} hylo_orth_matrix;
size_t hylo_orthogonalize_workspace_bytes(const hylo_orth_matrix* matrices, int count);
hylo_status hylo_orthogonalize(const hylo_orth_matrix* matrices, int count, int dtype, int out_dtype, int steps,
                               const double* coefficients, double eps, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/* One Muon step over `count` matrices (HOST array, not kept), all contiguous:
 *     g' = g * grad_scale * c,  c = min(1, max_norm / (norm[0] * |grad_scale| + 1e-6))  (1 without norm)
 *     m <- momentum m + (1 - momentum) g',   u = momentum m + (1 - momentum) g' (nesterov != 0) or m
 *     w <- w (1 - lr weight_decay) - lr scale O(u),   O as in hylo_orthogonalize, in fp16 (its accuracy is that of the step)
 * param, grad, master, momentum: as param, grad, master and m of hylo_adamw_step with 32-bit states, with the same rules for
 * masters, for overlaps (HYLO_ERR_DIM), for a norm that is not finite (nothing is written) and for capture (HYLO_ERR_CAPTURE),
 * and the same random bits where a bf16 param without master is rounded. Sizes, steps, coefficients, eps and workspace
 * as in hylo_orthogonalize. momentum in [0, 1). */
typedef struct {
  void* param;
  const void* grad;
  float* master;
  float* momentum;
  int64_t rows, cols;
  double lr;
  double weight_decay;
  double scale;
} hylo_muon_tensor;
size_t hylo_muon_workspace_bytes(const hylo_muon_tensor* tensors, int count);
hylo_status hylo_muon_step(const hylo_muon_tensor* tensors, int count, int param_dtype, int grad_dtype, double momentum,
                           int nesterov, int steps, const double* coefficients, double eps, float grad_scale, const float* norm,
                           float max_norm, uint32_t seed, void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HYLO_OPS_H */
