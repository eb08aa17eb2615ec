// Scaled embedding lookup with dropout, and its gradient by sorted tokens.
//
//     out[r, c] = f m(r, c) E[id_r, c],   f = scale * 65536 / (65536 - D),
// with m(r, c) = 0 where the 16 random bits of (r, c) are below D and 1
// elsewhere.  The bits come from a counter-based generator keyed by the call's
// (seed, offset), so the gradient forms the same mask again and no mask is
// stored.  The gradient of a table row is the sum of f m(r, c) g[r, c] over
// its tokens' rows in ascending order.
#include "vpce_embed_dropout.cuh"

namespace vpce {

namespace {

constexpr int kEdThreads = 256;

__device__ __forceinline__ int shard_holding(const ShardSet& sh, int t, long long id) {
  int lo = 0, hi = t;  // start[lo] <= id < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.start[mid] <= id) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kEdThreads) embed_dropout_forward_kernel(const __grid_constant__ EmbedDropParams p) {
  const long long blocks = (p.h + 7) / 8;
  const unsigned long long seed = p.drop ? p.rng[0] : 0, offset = p.drop ? p.rng[1] : 0;
  for (long long r = blockIdx.x; r < p.s; r += gridDim.x) {
    const long long id = p.ids[r];
    const bool in = id >= 0 && id < p.V, live = in && id != p.padding_id;
    if (!in && id != p.padding_id && threadIdx.x == 0 && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_BAD_TARGET);
    const int i = in ? shard_holding(p.sh, p.t, id) : 0;
    const unsigned char* src = in ? p.sh.ptr[i] + (id - p.sh.start[i]) * p.sh.ld_bytes[i] : nullptr;
    unsigned char* dst = p.out + r * p.ld_out_bytes;
    for (long long b = threadIdx.x; b < blocks; b += kEdThreads) {
      uint4 bits = make_uint4(0u, 0u, 0u, 0u);
      if (p.drop && live) bits = drop_block(seed, offset, r, unsigned(b));
      for (int j = 0; j < 8; ++j) {
        const long long c = b * 8 + j;
        if (c >= p.h) break;
        float v = 0.f;
        if (live && drop_keeps(bits, j, p.drop)) v = Elem<TI>::load(src + c * Elem<TI>::kBytes) * p.factor;
        Elem<TO>::store(dst + c * Elem<TO>::kBytes, v);
      }
    }
  }
}

// One CTA per table row: finds the row's tokens in order and adds their
// gradient rows.
template <typename T>
__global__ void __launch_bounds__(kEdThreads) embed_dropout_backward_kernel(const __grid_constant__ EmbedDropParams p) {
  __shared__ int list[kEdThreads];
  __shared__ int wcount[kEdThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned long long seed = p.drop ? p.rng[0] : 0, offset = p.drop ? p.rng[1] : 0;
  for (long long v = blockIdx.x; v < p.V; v += gridDim.x) {
    const int i = shard_holding(p.sh, p.t, v);
    float* row = reinterpret_cast<float*>(const_cast<unsigned char*>(p.sh.ptr[i]) + (v - p.sh.start[i]) * p.sh.ld_bytes[i]);
    if (!p.accumulate)
      for (long long c = tid; c < p.h; c += kEdThreads) row[c] = 0.f;
    if (v == p.padding_id) continue;
    for (long long r0 = 0; r0 < p.s; r0 += kEdThreads) {
      const bool mine = r0 + tid < p.s && p.ids[r0 + tid] == v;
      const unsigned m = __ballot_sync(kFull, mine);
      __syncthreads();
      if (lane == 0) wcount[warp] = __popc(m);
      __syncthreads();
      int before = 0, n = 0;
      for (int w = 0; w < kEdThreads / 32; ++w) {
        before += w < warp ? wcount[w] : 0;
        n += wcount[w];
      }
      if (n == 0) continue;
      if (mine) list[before + __popc(m & ((1u << lane) - 1u))] = int(r0) + tid;
      __syncthreads();
      for (long long b = tid; b < (p.h + 7) / 8; b += kEdThreads) {
        float acc[8] = {};
        for (int k = 0; k < n; ++k) {
          const long long r = list[k];
          uint4 bits = make_uint4(0u, 0u, 0u, 0u);
          if (p.drop) bits = drop_block(seed, offset, r, unsigned(b));
          for (int j = 0; j < 8; ++j)
            if (b * 8 + j < p.h && drop_keeps(bits, j, p.drop))
              acc[j] += Elem<T>::load(p.out + r * p.ld_out_bytes + (b * 8 + j) * Elem<T>::kBytes);
        }
        for (int j = 0; j < 8; ++j)
          if (b * 8 + j < p.h) row[b * 8 + j] += acc[j] * p.factor;
      }
    }
  }
}

}  // namespace

void launch_embed_dropout_forward(const EmbedDropParams& p, bool table_bf16, bool out_bf16, int sms,
                                  cudaStream_t st) {
  const long long cap = (long long)sms * 8;
  const int grid = int(p.s < cap ? p.s : cap);
  if (table_bf16 && out_bf16) embed_dropout_forward_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kEdThreads, 0, st>>>(p);
  else if (table_bf16) embed_dropout_forward_kernel<__nv_bfloat16, float><<<grid, kEdThreads, 0, st>>>(p);
  else if (out_bf16) embed_dropout_forward_kernel<float, __nv_bfloat16><<<grid, kEdThreads, 0, st>>>(p);
  else embed_dropout_forward_kernel<float, float><<<grid, kEdThreads, 0, st>>>(p);
}

size_t embed_dropout_workspace_bytes(long long, long long, long long) { return 256; }

cudaError_t launch_embed_dropout_backward(const EmbedDropParams& p, bool grad_bf16, void*, int sms, cudaStream_t st) {
  const long long cap = (long long)sms * 8;
  const int grid = int(p.V < cap ? p.V : cap);
  if (grad_bf16) embed_dropout_backward_kernel<__nv_bfloat16><<<grid, kEdThreads, 0, st>>>(p);
  else embed_dropout_backward_kernel<float><<<grid, kEdThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace vpce
