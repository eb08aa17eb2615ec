// Parameter blocks of the token scores: log probabilities of given tokens,
// entropy and top alternatives over vocabulary shards, and their gradient.
#pragma once

#include "vpce_device.cuh"

namespace vpce {

struct LogprobParams {
  ShardSet sh;
  int t;
  long long s;
  long long V;
  const long long* targets;  // null: every row is scored, no logp
  long long ignore_index;
  float inv_t;               // 1 / temperature
  int top;                   // 0..VPCE_MAX_TOP
  float* logp;               // each output may be null
  float* entropy;
  long long* top_ids;        // [s][top]
  float* top_logp;           // [s][top]
  float4* stats;             // [s]: largest logit, ln sum exp((z - max) / T), entropy, 0
  int* flag;
  // set by the launch: pieces of a row, vectors in each, rows held at a time,
  // warps that finish rows
  int pieces, len, slots, team;
};

struct LogprobBwdParams {
  ShardSet sh;
  unsigned char* grad[VPCE_MAX_SHARDS];
  long long ld_grad_bytes[VPCE_MAX_SHARDS];
  int t;
  long long s;
  long long V;
  const long long* targets;
  long long ignore_index;
  float inv_t;
  const float4* stats;
  const float* g_logp;       // [s] or null
  const float* g_entropy;    // [s] or null
  int top;
  const long long* top_ids;  // [s][top]
  const float* g_top;        // [s][top]
  int chunks;                // set by the launch: chunks of a row,
  int first[VPCE_MAX_SHARDS + 1];  // and the first one of each shard
};

// Order-preserving keys of fp32 values: a NaN of either sign is the largest
// key, -0 equals +0, and key order is value order everywhere else.
__device__ __forceinline__ unsigned value_key(float x) {
  const unsigned b = __float_as_uint(x);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (b == 0x80000000u) return 0x80000000u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <typename T>
void launch_logprob_forward(LogprobParams p, int sms, cudaStream_t st);
template <typename T>
void launch_logprob_backward(LogprobBwdParams p, int sms, cudaStream_t st);

}  // namespace vpce
