// Log probabilities of given tokens, entropy and top alternatives of rows of
// vocabulary-sharded logits.
//
// With x_k = z_k / T, m the row's largest z and u_k = (z_k - m) / T,
//     S = sum_k exp(u_k),  U = sum_k u_k exp(u_k),
//     logp_y = u_y - ln S,  entropy = ln S - U / S,
// so a column at -inf adds nothing to S or U (its 0 * inf is skipped), and a
// row whose logits are all the type's lowest finite value is a uniform one.
// The top alternatives are the columns of largest z; equal values rank by
// column, lowest first.
#include "vpce_logprob.cuh"

namespace vpce {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;

// (m, S, U) of a running maximum, sum exp(u) and sum u exp(u): merge two.
// Moving the maximum by d multiplies S by exp(d) and gives U' = (U + S d) exp(d).
struct Msu {
  float m, s, u;
};
__device__ __forceinline__ Msu merge(const Msu& a, const Msu& b, float inv_t) {
  Msu r;
  r.m = max_nan(a.m, b.m);
  const float da = a.m == r.m ? 0.f : (a.m - r.m) * inv_t, db = b.m == r.m ? 0.f : (b.m - r.m) * inv_t;
  const float ea = a.s == 0.f ? 0.f : expf(da), eb = b.s == 0.f ? 0.f : expf(db);
  r.s = a.s * ea + b.s * eb;
  r.u = (ea == 0.f ? 0.f : (a.u + a.s * da) * ea) + (eb == 0.f ? 0.f : (b.u + b.s * db) * eb);
  return r;
}

__device__ __forceinline__ void add_value(Msu& a, float z, float inv_t) {
  if (z == -INFINITY) return;
  Msu b;
  b.m = z;
  b.s = 1.f;
  b.u = 0.f;
  a = merge(a, b, inv_t);
}

// One CTA per row: a pass for (m, S, U), then one pass per alternative that
// finds the best column after the previous one.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprob_forward_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int EB = Elem<T>::kBytes;
  __shared__ Msu part[kLpWarps];
  __shared__ unsigned long long best[kLpWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (long long r = blockIdx.x; r < p.s; r += gridDim.x) {
    const long long y = p.targets != nullptr ? p.targets[r] : 0;
    if (p.targets != nullptr && y == p.ignore_index) {
      if (tid == 0) {
        if (p.logp) p.logp[r] = 0.f;
        if (p.entropy) p.entropy[r] = 0.f;
        if (p.stats) p.stats[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (tid < p.top) {
        p.top_ids[r * p.top + tid] = -1;
        if (p.top_logp) p.top_logp[r * p.top + tid] = 0.f;
      }
      continue;
    }
    Msu a{-INFINITY, 0.f, 0.f};
    for (int i = 0; i < p.t; ++i) {
      const unsigned char* row = p.sh.ptr[i] + r * p.sh.ld_bytes[i];
      const int w = int(p.sh.start[i + 1] - p.sh.start[i]);
      for (int c = tid; c < w; c += kLpThreads) add_value(a, Elem<T>::load(row + (long long)c * EB), p.inv_t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Msu b;
      b.m = __shfl_xor_sync(kFull, a.m, o);
      b.s = __shfl_xor_sync(kFull, a.s, o);
      b.u = __shfl_xor_sync(kFull, a.u, o);
      a = merge(a, b, p.inv_t);
    }
    __syncthreads();
    if (lane == 0) part[warp] = a;
    __syncthreads();
    a = part[0];
    for (int w = 1; w < kLpWarps; ++w) a = merge(a, part[w], p.inv_t);
    // no finite largest logit (nothing unmasked, +inf or NaN): no distribution
    const bool ok = isfinite(a.m) && a.s > 0.f;
    const float nan = __int_as_float(0x7fc00000);
    const float ls = ok ? logf(a.s) : nan;
    const float ent = ok ? ls - a.u / a.s : nan;
    if (tid == 0) {
      if (p.entropy) p.entropy[r] = ent;
      if (p.stats) p.stats[r] = make_float4(a.m, ls, ent, 0.f);
      if (p.targets != nullptr) {
        float lp = nan;
        if (y >= 0 && y < p.V) {
          int i = 0;
          while (y >= p.sh.start[i + 1]) ++i;
          const float z = Elem<T>::load(p.sh.ptr[i] + r * p.sh.ld_bytes[i] + (y - p.sh.start[i]) * EB);
          lp = (z - a.m) * p.inv_t - ls;
        } else if (p.flag != nullptr) {
          atomicOr(p.flag, VPCE_FLAG_BAD_TARGET);
        }
        if (p.logp) p.logp[r] = lp;
      }
    }
    unsigned long long prev = ~0ull;
    for (int j = 0; j < p.top; ++j) {
      unsigned long long b = 0;
      for (int i = 0; i < p.t; ++i) {
        const unsigned char* row = p.sh.ptr[i] + r * p.sh.ld_bytes[i];
        const int w = int(p.sh.start[i + 1] - p.sh.start[i]);
        for (int c = tid; c < w; c += kLpThreads) {
          const unsigned key = value_key(Elem<T>::load(row + (long long)c * EB));
          const unsigned long long k = ((unsigned long long)key << 32) | unsigned(~unsigned(p.sh.start[i] + c));
          if (k < prev && k > b) b = k;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long q = __shfl_xor_sync(kFull, b, o);
        b = q > b ? q : b;
      }
      __syncthreads();
      if (lane == 0) best[warp] = b;
      __syncthreads();
      for (int w = 0; w < kLpWarps; ++w) b = best[w] > b ? best[w] : b;
      prev = b;
      if (tid == 0) {
        const long long c = (long long)unsigned(~unsigned(b));
        p.top_ids[r * p.top + j] = c;
        if (p.top_logp) {
          int i = 0;
          while (c >= p.sh.start[i + 1]) ++i;
          const float z = Elem<T>::load(p.sh.ptr[i] + r * p.sh.ld_bytes[i] + (c - p.sh.start[i]) * EB);
          p.top_logp[r * p.top + j] = (z - a.m) * p.inv_t - ls;
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

template <typename T>
void launch_logprob_forward(const LogprobParams& p, int sms, cudaStream_t st) {
  const long long cap = (long long)sms * 8;
  logprob_forward_kernel<T><<<int(p.s < cap ? p.s : cap), kLpThreads, 0, st>>>(p);
}
template void launch_logprob_forward<float>(const LogprobParams&, int, cudaStream_t);
template void launch_logprob_forward<__nv_bfloat16>(const LogprobParams&, int, cudaStream_t);

}  // namespace vpce
