// Gradient of the token scores with respect to the logits.
//
// With p_k = exp(u_k - ln S) from the forward's row statistics,
//     dz_k = (g_l [k = y] + sum_j g_j [k = id_j]
//             - p_k (g_l + sum_j g_j + g_H (ln p_k + H))) / T,
// since d logp_c / dx_k = [k = c] - p_k and dH / dx_k = -p_k (ln p_k + H).
// A column at -inf has p = 0 and gradient 0; a row without a distribution
// (statistics NaN) has a NaN gradient.
#include "vpce_logprob.cuh"

namespace vpce {

namespace {

constexpr int kLbThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kLbThreads) logprob_backward_kernel(const __grid_constant__ LogprobBwdParams p) {
  constexpr int EB = Elem<T>::kBytes;
  __shared__ long long ids[VPCE_MAX_TOP];
  __shared__ float gt[VPCE_MAX_TOP];
  const int tid = threadIdx.x;
  for (long long r = blockIdx.x; r < p.s; r += gridDim.x) {
    const long long y = p.targets != nullptr ? p.targets[r] : -1;
    const bool ignored = p.targets != nullptr && y == p.ignore_index;
    __syncthreads();
    if (tid < p.top) {
      ids[tid] = p.top_ids[r * p.top + tid];
      gt[tid] = p.g_top[r * p.top + tid];
    }
    __syncthreads();
    const float4 st = p.stats[r];
    const float gl = p.g_logp != nullptr ? p.g_logp[r] : 0.f, gh = p.g_entropy != nullptr ? p.g_entropy[r] : 0.f;
    float w = gl;
    for (int j = 0; j < p.top; ++j)
      if (ids[j] >= 0 && ids[j] < p.V) w += gt[j];
    if (p.g_logp != nullptr && (y < 0 || y >= p.V)) w = __int_as_float(0x7fc00000);
    if (isnan(st.y)) w = st.y;
    for (int i = 0; i < p.t; ++i) {
      const unsigned char* row = p.sh.ptr[i] + r * p.sh.ld_bytes[i];
      unsigned char* out = p.grad[i] + r * p.ld_grad_bytes[i];
      const int n = int(p.sh.start[i + 1] - p.sh.start[i]);
      for (int c = tid; c < n; c += kLbThreads) {
        float d = 0.f;
        if (!ignored) {
          const float lp = fmaxf((Elem<T>::load(row + (long long)c * EB) - st.x) * p.inv_t - st.y, -200.f);
          d = -expf(lp) * (w + gh * (lp + st.z));
          const long long k = p.sh.start[i] + c;
          if (k == y) d += gl;
          for (int j = 0; j < p.top; ++j)
            if (ids[j] == k) d += gt[j];
          d *= p.inv_t;
        }
        Elem<T>::store(out + (long long)c * EB, d);
      }
    }
  }
}

}  // namespace

template <typename T>
void launch_logprob_backward(const LogprobBwdParams& p, int sms, cudaStream_t st) {
  const long long cap = (long long)sms * 8;
  logprob_backward_kernel<T><<<int(p.s < cap ? p.s : cap), kLbThreads, 0, st>>>(p);
}
template void launch_logprob_backward<float>(const LogprobBwdParams&, int, cudaStream_t);
template void launch_logprob_backward<__nv_bfloat16>(const LogprobBwdParams&, int, cudaStream_t);

}  // namespace vpce
