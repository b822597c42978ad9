// Internal launch interface of the operators declared in include/hylo_ops.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/hylo_ops.h"
#include "hylo_internal.h"

namespace hylo {

struct TokenRows {
  const void* z;  // logits [N, V], row stride ld elements
  int64_t ld;
  int N, V;
  float inv_tau;
  float c;        // log2(e) / tau
  const int64_t* tokens;
};

struct TokenOut {
  int k;
  float* logp;
  float* entropy;  // or null
  float* lse;      // or null
  float2* stats;   // (max, log sum), or null
  float* top_logp;
  int64_t* top_ids;
};

struct TokenGrad {
  const float2* stats;
  const float* entropy;
  const float* g_logp;     // or null
  const float* g_entropy;  // or null
  void* dz;
  int64_t ldd;
};

// What fits on the device at once: clusters of 1, 2, 4, 8 and 16 CTAs of the kernels that split rows.
struct TokenOccupancy {
  int sms = 0;
  int clusters[5] = {};
};
cudaError_t token_logprobs_prepare(int sms, TokenOccupancy* occ);  // once per device
cudaError_t launch_token_logprobs(const TokenRows& in, const TokenOut& out, int dtype, const TokenOccupancy& occ,
                                  cudaStream_t stream);
cudaError_t launch_token_logprobs_bwd(const TokenRows& in, const TokenGrad& g, int dtype, int sms, cudaStream_t stream);

// The tensor cores cut the sum off at fp32's last bit after every 16 products, which carries a logit towards 0 by up to
// 2^-24 of it per step. So the logits of the log-probabilities from hidden states are accumulated over at most this many
// 64-wide k-blocks at a time, and these partial sums added up in registers, rounded to nearest. Log-probabilities of 8
// tokens, d = 4096, V = 32000: in one go 1.5e-5 off, so 4e-6; with half the depth 2e-6, but the reads of TMEM then hold up the
// tensor cores (8192 tokens, d = 2048 2107 us in one go, 2102 to 2152 so, 2150 to 2209 with half the depth; 3 tokens, d = 4096
// 182, 180 and 200).
constexpr int kLogitDepth = 16;

// Forward of the log-probabilities from hidden states (head_logprobs.cu).
struct HeadParams {
  int N, V;
  int kb;           // 64-wide k-blocks of d
  int depths;       // ceil(kb / kLogitDepth)
  int token_tiles;  // ceil(N / 256)
  int vtiles;       // ceil(V / 256)
  int nseg;         // vocabulary segments per token tile
  int units;        // token_tiles * nseg
  int copies;       // of h, which the clusters share out
  float c;          // log2(e) / tau
  float inv_tau;
  const int64_t* tokens;
  int slots;        // partial sums per token
  float4* part;     // partial sums [N][slots]
  float* z_token;   // the tokens' logits [N]
  WaitCtl ctl;
};
cudaError_t head_prepare(int* max_clusters);
cudaError_t launch_head_logprobs(const CUtensorMap& h, const CUtensorMap& W, const HeadParams& p, float* logp,
                                 float* entropy, float* lse, int clusters, cudaStream_t stream);

cudaError_t launch_head_copy(const uint16_t* h, void* copies, int64_t n, int count, cudaStream_t stream);

// The forward of few tokens, without the tensor cores; p.slots CTAs.
bool head_few_fits(int64_t N, int64_t d);
cudaError_t launch_head_few(const uint16_t* h, const uint16_t* W, int d, const HeadParams& p, float* logp, float* entropy,
                            float* lse, cudaStream_t stream);

// Backward of the same: the pipelined backward (kl_bwd_pipe.cu) with
//   G[n, v] = dL/dz = p (A + B log2 p) + 1[v = tokens[n]] g_logp / tau,
//   A = -(g_logp + g_entropy entropy) / tau, B = -g_entropy ln 2 / tau, log2 p = c z - log2(e) lse.
struct HeadGrad {
  const int64_t* tokens;
  const float* lse;
  const float* entropy;
  const float* g_logp;     // or null
  const float* g_entropy;  // or null
  float inv_tau;
  int dw_bf16;             // one token block: map kMapDW is a bf16 tensor of 32 x 32 tiles with 64-byte swizzle
  int order;               // see below
  int want_dh, want_dw;    // which gradients there are
  int dh_words;            // kOrderParts: words of a block whose products go into one part (a multiple of 64); else INT_MAX
};
// How the items of one block wait for those of others (M(b): products of block b, F(b): its G).
//   kOrderChain: M(b) needs all of M(b - 1), as the distillation loss.
//   kOrderDh: only the dh items of block b - 1 (which come first), as dh is what one block after another adds to; dW's
//     items of one block then do not hold up the next. With several token blocks dW is added to as well. Its items of the same
//     words, VB blocks before, are complete if VB >= 3 and there are dh items: those of block b wait for those of b - 1, so
//     for F(b - 1), F(b - 2), ..., which had to wait for all of M(b - 4), M(b - 5), ... to take their ring slots; and F(b)
//     for M(b - 3).
//   kOrderParts: nothing of M(b - 1). Map kMapDh is [vocabulary blocks][N][d]: every block's part of dh apart (one token
//     block).
enum : int { kOrderChain = 0, kOrderDh = 1, kOrderParts = 2 };
// y = the sum over `parts` of x [parts][n] in ascending order, as fp32 or rounded to bf16 (n a multiple of 8, 16-byte aligned).
cudaError_t launch_join_parts(const float* x, int parts, void* y, bool bf16, int64_t n, int sms, cudaStream_t stream);
cudaError_t launch_bwd_pipe_head(const CUtensorMap* maps, const BwdPipeParams& p, const HeadGrad& g, int clusters,
                                 cudaStream_t stream);

// Gradient-norm partial sums: one per block of the norm kernel.
constexpr int kNormPartials = 2048;
cudaError_t launch_grad_norm(const void* const* grads, const int64_t* sizes, int count, int dtype, float* norm,
                             float* partials, int sms, cudaStream_t stream);

struct AdamWHyper {
  float beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
  float rbc2;        // 1 / sqrt(1 - beta2^step)
  float grad_scale;
  const float* norm;  // or null
  float max_norm;
  uint32_t seed;
};
cudaError_t launch_adamw(const hylo_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype, int state_bits,
                         bool masters, double bias1, const AdamWHyper& h, int sms, cudaStream_t stream);

// Layer norm and RMS norm (norm.cu).
struct NormParams {
  const void* x;         // [N, d], row stride ldx: the forward's input, the backward's normalised rows
  const void* residual;  // [N, d], row stride ldr, or null
  int64_t ldx, ldr;
  int64_t N;
  int d;
  int rms;
  float eps;
  const void* weight;    // [d] or null
  const void* bias;      // [d] or null
  int gain_f32;          // weight and bias are fp32, not of the type of x
  void* sum;             // [N, d], with a residual
  void* y;               // [N, d]
  float2* stats;         // (mean, 1 / deviation) [N], or null in a forward
  int threads;           // threads that share a row, set by the launch
};
struct NormGrad {
  const void* dy;    // [N, d], row stride lddy
  const void* dsum;  // [N, d], row stride ldds, or null
  int64_t lddy, ldds;
  void* dx;          // [N, d] or null
  float* part;       // [2][parts][d], or null: no column sums are wanted
  int want_dw, want_db;
  void* dw;
  void* db;
  int cta_cols;      // columns of a CTA of a cluster, set by the launch
  WaitCtl ctl;
};
// Widest rows (fp32: half of it) whose gradients are formed in one reading, and how many rows of `part` there may be.
constexpr int kNormFusedCols = 65536;
int norm_parts(int64_t N, int d);
cudaError_t launch_norm(const NormParams& p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormParams& p, const NormGrad& q, int dtype, int parts, int sms, cudaStream_t stream);

}  // namespace hylo
