// Internal launch interface of the operators declared in include/hylo_ops.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/hylo_ops.h"

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

cudaError_t launch_token_logprobs(const TokenRows& in, const TokenOut& out, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_token_logprobs_bwd(const TokenRows& in, const TokenGrad& g, int dtype, int sms, cudaStream_t stream);

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
                         bool masters, double bias1, const AdamWHyper& h, cudaStream_t stream);

}  // namespace hylo
