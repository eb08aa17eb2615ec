// The AdamW step over many tensors and the norm of their gradients: what the
// host hands to the kernels.
#pragma once

#include "vpce_rows.cuh"

namespace vpce {

constexpr int kAdamBlock = 256;       // elements that share a scale of 8-bit states
constexpr int kAdamTensors = 440;     // of one launch: what 32 KB of kernel parameters hold
constexpr int kAdamFewTensors = 24;   // of the short forms: a launch copies its parameters
constexpr int kAdamSomeTensors = 100;
constexpr int kNormThreads = 512;
constexpr int kNormMaxCtas = 1024;    // of one launch: partial sums that the workspace holds

struct AdamHyper {
  const long long* step;
  const float* lr_dev;
  const float* grad_scale;
  const unsigned long long* rng;
  float lr, eps;
  float b1, a1, b2, a2;        // beta and 1 - beta
  float ln_b1, ln_b2;          // log of beta, rounded once from fp64
};

void launch_adamw(const vpce_adamw_tensor* tensors, long long n_tensors, bool param_bf16, bool grad_bf16, int bits,
                  const AdamHyper& hy, int sms, cudaStream_t st);
size_t grad_norm_workspace_bytes(long long n_tensors);
cudaError_t launch_grad_norm(const vpce_adamw_tensor* tensors, long long n_tensors, bool grad_bf16, float max_norm,
                             float* norm_out, float* scale_out, void* ws, int sms, cudaStream_t st);

}  // namespace vpce
