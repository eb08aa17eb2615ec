// Scaled embedding lookup with counter-based dropout: parameter blocks and the
// generator shared by the lookup and its gradient.
#pragma once

#include "vpce_device.cuh"

namespace vpce {

struct EmbedDropParams {
  ShardSet sh;               // table shards [w_i, h] (backward: fp32 gradient shards)
  int t;
  long long V;
  long long h;
  const long long* ids;
  long long s;
  long long padding_id;
  float factor;              // scale * 65536 / (65536 - drop)
  unsigned drop;             // 0..65535: a 16-bit value below it drops its element
  const unsigned long long* rng;  // device {seed, offset}; null when drop = 0
  unsigned char* out;        // forward: [s][h]; backward: the gradient rows read
  long long ld_out_bytes;
  int* flag;                 // may be null
  int accumulate;            // backward
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter, the key stepped by a constant between rounds.
struct DropKey {
  uint2 k[10];  // the rounds' keys
  unsigned lo, hi;  // offset
  __device__ __forceinline__ void set(const unsigned long long* rng) {
    const unsigned long long seed = rng != nullptr ? rng[0] : 0, offset = rng != nullptr ? rng[1] : 0;
    lo = unsigned(offset);
    hi = unsigned(offset >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i)
      k[i] = make_uint2(unsigned(seed) + i * 0x9E3779B9u, unsigned(seed >> 32) + i * 0xBB67AE85u);
  }
};

// The 8 random 16-bit values of columns [8 cb, 8 cb + 8) of row r: value j is
// half j of the block, low halves first.
__device__ __forceinline__ uint4 drop_block(const DropKey& key, long long r, unsigned cb) {
  uint4 c = make_uint4(cb, unsigned(r), key.lo, key.hi);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long a = (unsigned long long)c.x * 0xD2511F53u, b = (unsigned long long)c.z * 0xCD9E8D57u;
    c = make_uint4(unsigned(b >> 32) ^ c.y ^ key.k[i].x, unsigned(b), unsigned(a >> 32) ^ c.w ^ key.k[i].y,
                   unsigned(a));
  }
  return c;
}

// Rows of the table gradient: positions in the sorted order, with a task's or a
// CTA's stride past the last one, are 32-bit.
constexpr long long kEmbedDropMaxRows = (1ll << 31) - 4096;

// CTAs of the lookup
long long embed_dropout_forward_blocks(long long s, long long h);
void launch_embed_dropout_forward(const EmbedDropParams& p, bool table_bf16, bool out_bf16, cudaStream_t st);
size_t embed_dropout_workspace_bytes(long long s, long long V, long long h);
cudaError_t launch_embed_dropout_backward(const EmbedDropParams& p, bool grad_bf16, void* ws, int sms,
                                          cudaStream_t st);

}  // namespace vpce
