// Gradient of the token scores with respect to the logits.
//
// With p_k = exp(u_k - ln S) from the forward's row statistics,
//     dz_k = (g_l [k = y] + sum_j g_j [k = id_j]
//             - p_k (g_l + sum_j g_j + g_H (ln p_k + H))) / T,
// since d logp_c / dx_k = [k = c] - p_k and dH / dx_k = -p_k (ln p_k + H).
// Per element that is v = log2 p (a subtraction and a fused multiply-add),
// 2^v, and a factor linear in v: e (a + b v).  The subtraction of the row's
// largest logit comes first, so that rows filled with the type's lowest value
// stay finite; v is clamped at -256, where 2^v is 0, so that a column at -inf
// gets 0 and not 0 * inf.
//
// Bound by HBM: one read and one write of the logits.  A row's shard segments
// are cut into chunks; a warp loads a chunk into registers, turns it into
// gradients and stores it with 16-byte stores, three blocks of warps per SM
// keeping loads and stores in flight.  Measured at s = 8192, V = 128256 bf16:
// 0.636 ms, 6.6 TB/s (8 vectors a lane; 4: 0.640, 16: 0.648); s = 4096,
// V = 152064 fp32: 0.737 ms, 6.76 TB/s.  The shared-memory ring of bulk copies
// that the loss's in-place backward uses takes 0.655 and 0.783 ms for the same
// bytes.
#include "vpce_logprob.cuh"

namespace vpce {

namespace {

constexpr int kLbThreads = 256;
constexpr int kLbWarps = kLbThreads / 32;
constexpr int kLbVecs = 8;                    // vectors per lane and chunk
constexpr int kLbChunk = 32 * kLbVecs;        // vectors per chunk

// What a row's gradient needs besides the logits.
struct RowGrad {
  float m, lse2, a, b;  // largest logit; log2 S; the factor a + b v
  float gl;             // g_l / T
};

__device__ __forceinline__ float top_weight(const LogprobBwdParams& p, long long row, int lane, long long& id,
                                            float& g) {
  id = -1;
  g = 0.f;
  if (lane < p.top) {
    id = __ldg(p.top_ids + row * p.top + lane);
    g = __ldg(p.g_top + row * p.top + lane);
    if (id < 0 || id >= p.V) {
      id = -1;
      g = 0.f;
    }
  }
  float w = g;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(kFull, w, o);
  return w;
}

__device__ __forceinline__ RowGrad row_grad(const LogprobBwdParams& p, long long row, long long y, float tops) {
  const float4 st = __ldg(p.stats + row);
  RowGrad r;
  const float gl = p.g_logp != nullptr ? __ldg(p.g_logp + row) : 0.f;
  const float gh = p.g_entropy != nullptr ? __ldg(p.g_entropy + row) : 0.f;
  float w = gl + tops;
  // a target out of range, or a row without a distribution: NaN
  if ((p.g_logp != nullptr && (y < 0 || y >= p.V)) || isnan(st.y)) w = __int_as_float(0x7fc00000);
  r.m = st.x;
  r.lse2 = st.y * kLog2e;
  r.a = -p.inv_t * (w + gh * st.z);
  r.b = -p.inv_t * gh * 0.6931471806f;
  r.gl = gl * p.inv_t;
  return r;
}

__device__ __forceinline__ float grad_of(float x, const RowGrad& r, float c) {
  const float v = fmaxf(fmaf(x - r.m, c, -r.lse2), -256.f);
  return ex2(v) * fmaf(v, r.b, r.a);
}

__device__ __forceinline__ f32x2 grad_pair(float x0, float x1, f32x2 nm, f32x2 c, f32x2 nl, f32x2 a, f32x2 b) {
  float v0, v1;
  f2_unpack(f2_fma(f2_add(f2_pack(x0, x1), nm), c, nl), v0, v1);
  v0 = fmaxf(v0, -256.f);
  v1 = fmaxf(v1, -256.f);
  return f2_mul(f2_pack(ex2(v0), ex2(v1)), f2_fma(f2_pack(v0, v1), b, a));
}

struct PackedRow {
  f32x2 nm, c, nl, a, b;
};

__device__ __forceinline__ uint4 grad_vector(const uint4& q, const PackedRow& r, __nv_bfloat16) {
  const unsigned w[4] = {q.x, q.y, q.z, q.w};
  unsigned o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float d0, d1;
    f2_unpack(grad_pair(bf16_lo(w[i]), bf16_hi(w[i]), r.nm, r.c, r.nl, r.a, r.b), d0, d1);
    o[i] = pack_bf16x2(d0, d1);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 grad_vector(const uint4& q, const PackedRow& r, float) {
  float d0, d1, d2, d3;
  f2_unpack(grad_pair(__uint_as_float(q.x), __uint_as_float(q.y), r.nm, r.c, r.nl, r.a, r.b), d0, d1);
  f2_unpack(grad_pair(__uint_as_float(q.z), __uint_as_float(q.w), r.nm, r.c, r.nl, r.a, r.b), d2, d3);
  return make_uint4(__float_as_uint(d0), __float_as_uint(d1), __float_as_uint(d2), __float_as_uint(d3));
}

// One unit per warp at a time: chunk `ch` of (row, shard), kLbChunk vectors of
// the segment's 16-byte aligned body; a shard's chunk 0 also takes the elements
// before and after the body.  The gradient is stored in vectors where its row
// has the logits' alignment, by element otherwise.
template <typename T>
__global__ void __launch_bounds__(kLbThreads) logprob_backward_kernel(const __grid_constant__ LogprobBwdParams p) {
  constexpr int EB = Elem<T>::kBytes, EPV = Elem<T>::kPerVec;
  const int lane = threadIdx.x & 31;
  const float c = p.inv_t * kLog2e;
  const long long nw = (long long)gridDim.x * kLbWarps;
  const long long w0 = (long long)blockIdx.x * kLbWarps + (threadIdx.x >> 5);
  const long long step_row = nw / p.chunks;
  const int step_ch = int(nw - step_row * p.chunks);
  long long row = w0 / p.chunks;
  int at = int(w0 - row * p.chunks);
#pragma unroll 1
  for (; row < p.s; row += step_row, at += step_ch) {
    if (at >= p.chunks) {
      at -= p.chunks;
      if (++row >= p.s) break;
    }
    int shard = 0;
    while (at >= p.first[shard + 1]) ++shard;
    const int ch = at - p.first[shard];
    const Unit g = make_unit_at(p.sh, shard, row, EB);
    const int nv = int(g.body >> 4), head = int(g.head) / EB, tail = int(g.tail) / EB;
    const int base = ch * kLbChunk, n = min(kLbChunk, nv - base);
    const uint4* src = reinterpret_cast<const uint4*>(g.addr + g.head) + base;
    const long long y = p.targets != nullptr ? __ldg(p.targets + row) : -1;
    const bool ignored = p.targets != nullptr && y == p.ignore_index;
    uint4 q[kLbVecs];
    if (!ignored) {
#pragma unroll
      for (int j = 0; j < kLbVecs; ++j) {
        const int i = lane + 32 * j;
        q[j] = i < n ? __ldcs(src + i) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    unsigned char* out = p.grad[shard] + row * p.ld_grad_bytes[shard];
    unsigned char* dst = out + g.head + (long long)base * 16;
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
    int rag = -1;  // the ragged element this lane takes
    if (ch == 0) {
      if (lane < head) rag = lane;
      else if (lane >= 16 && lane - 16 < tail) rag = head + nv * EPV + lane - 16;
    }
    if (ignored) {
      for (int i = lane; i < n; i += 32) {
        if (vec) __stcs(reinterpret_cast<uint4*>(dst) + i, make_uint4(0u, 0u, 0u, 0u));
        else
          for (int e = 0; e < EPV; ++e) Elem<T>::store(dst + (i * EPV + e) * EB, 0.f);
      }
      if (rag >= 0) Elem<T>::store(out + (long long)rag * EB, 0.f);
      continue;
    }
    long long id = -1;  // lane j's alternative and its weight
    float gt = 0.f, tops = 0.f;
    if (p.top > 0) tops = top_weight(p, row, lane, id, gt);
    const RowGrad r = row_grad(p, row, y, tops);
    // The columns of this chunk with onehot terms (the lane's alternative, and
    // the target as lane 0's second): their gradients from the logits as they
    // were, formed before any lane stores.  Equal columns get equal values.
    const long long c0 = p.sh.start[shard];
    const long long lo = c0 + head + (long long)base * EPV, hi = lo + (long long)n * EPV;
    auto whole = [&](long long col, float x) -> float {
      float d = grad_of(x, r, c);
      if (p.g_logp != nullptr && col == y) d += r.gl;
      for (int j = 0; j < p.top; ++j)
        if (__ldg(p.top_ids + row * p.top + j) == col) d += __ldg(p.g_top + row * p.top + j) * p.inv_t;
      return d;
    };
    const bool s1 = id >= lo && id < hi, s2 = p.g_logp != nullptr && lane == 0 && y >= lo && y < hi;
    float d1 = 0.f, d2 = 0.f, dr = 0.f;
    if (s1) d1 = whole(id, Elem<T>::load(g.addr + (id - c0) * EB));
    if (s2) d2 = whole(y, Elem<T>::load(g.addr + (y - c0) * EB));
    if (rag >= 0) dr = whole(c0 + rag, Elem<T>::load(g.addr + (long long)rag * EB));
    __syncwarp();
    const PackedRow pr{f2_pack(-r.m, -r.m), f2_pack(c, c), f2_pack(-r.lse2, -r.lse2), f2_pack(r.a, r.a),
                       f2_pack(r.b, r.b)};
    if (vec) {
#pragma unroll
      for (int j = 0; j < kLbVecs; ++j) {
        const int i = lane + 32 * j;
        if (i < n) __stcs(reinterpret_cast<uint4*>(dst) + i, grad_vector(q[j], pr, T()));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kLbVecs; ++j) {
        const int i = lane + 32 * j;
        float x[EPV];
        unpack(q[j], x, T());
        if (i < n) {
#pragma unroll
          for (int e = 0; e < EPV; ++e) Elem<T>::store(dst + (i * EPV + e) * EB, grad_of(x[e], r, c));
        }
      }
    }
    if (rag >= 0) Elem<T>::store(out + (long long)rag * EB, dr);
    __syncwarp();
    if (s1) Elem<T>::store(out + (id - c0) * EB, d1);
    if (s2) Elem<T>::store(out + (y - c0) * EB, d2);
  }
}

}  // namespace

template <typename T>
void launch_logprob_backward(LogprobBwdParams p, int sms, cudaStream_t st) {
  p.chunks = 0;
  for (int i = 0; i < p.t; ++i) {
    p.first[i] = p.chunks;
    const long long nv = (p.sh.start[i + 1] - p.sh.start[i]) / Elem<T>::kPerVec;
    p.chunks += int(nv > kLbChunk ? (nv + kLbChunk - 1) / kLbChunk : 1);
  }
  for (int i = p.t; i <= VPCE_MAX_SHARDS; ++i) p.first[i] = p.chunks;
  const long long want = (p.s * p.chunks + kLbWarps - 1) / kLbWarps, cap = (long long)sms * 8;
  logprob_backward_kernel<T><<<int(want < cap ? want : cap), kLbThreads, 0, st>>>(p);
}
template void launch_logprob_backward<float>(LogprobBwdParams, int, cudaStream_t);
template void launch_logprob_backward<__nv_bfloat16>(LogprobBwdParams, int, cudaStream_t);

}  // namespace vpce
