// AdamW over many tensors in one launch, states in fp32 or in e4m3 with a
// scale per 256 elements, and the norm of all gradients.
//
// The tensors' addresses travel in the kernels' parameters (32 KB hold 440),
// so that a step is one launch, captured graphs carry them by value, and
// nothing is copied to the device.  A CTA takes a run of consecutive elements
// of one tensor, found by bisection over the runs' numbers.  Both kernels are
// bound by HBM: 30 bytes an element move for some 16 operations with fp32
// states, 18 bytes for some 50 with 8-bit ones.
#include <cmath>

#include <cuda_fp8.h>

#include "vpce_adamw.cuh"
#include "vpce_embed_dropout.cuh"

namespace vpce {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                       // consecutive elements of a thread
constexpr int kTile = kThreads * kPer;        // elements of a CTA's turn
constexpr float kTiny = 1.17549435e-38f;      // 2^-126: the least scale, so that 1 / scale is finite

struct AdamTensor {
  unsigned char *p, *m, *v, *copy;
  const unsigned char* g;
  float *ms, *vs;
  long long n;
  float wd;
  int run0;  // number of its first run
};

template <int kCap> struct AdamArgs {
  AdamHyper hy;
  int n, base;     // tensors here, and position of the first in the caller's list
  int run;         // elements of a run
  AdamTensor t[kCap];
};
static_assert(sizeof(AdamArgs<kAdamTensors>) <= 32764, "kernel parameters");

template <int kCap> struct NormArgs {
  int n, runs;
  float* part;
  const unsigned char* g[kCap];
  long long count[kCap];
  int run0[kCap];
};
static_assert(sizeof(NormArgs<kAdamTensors>) <= 32764, "kernel parameters");

// Eight consecutive elements: one or two vectors where `vec`, else one by one,
// `left` of them (the others 0).
__device__ __forceinline__ void load8(const unsigned char* base, long long e, int left, bool vec, float (&x)[8], float) {
  const float* p = reinterpret_cast<const float*>(base) + e;
  if (vec && left >= 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < left ? p[j] : 0.f;
  }
}
__device__ __forceinline__ void load8(const unsigned char* base, long long e, int left, bool vec, float (&x)[8],
                                      __nv_bfloat16 t) {
  const unsigned char* p = base + e * 2;
  if (vec && left >= 8) {
    unpack(*reinterpret_cast<const uint4*>(p), x, t);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < left ? Elem<__nv_bfloat16>::load(p + j * 2) : 0.f;
  }
}
__device__ __forceinline__ void store8(unsigned char* base, long long e, int left, bool vec, const float (&x)[8], float) {
  float* p = reinterpret_cast<float*>(base) + e;
  if (vec && left >= 8) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = x[j];
  }
}
__device__ __forceinline__ void store8(unsigned char* base, long long e, int left, bool vec, const float (&x)[8],
                                       __nv_bfloat16 t) {
  unsigned char* p = base + e * 2;
  if (vec && left >= 8) {
    *reinterpret_cast<uint4*>(p) = pack(x, t);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) Elem<__nv_bfloat16>::store(p + j * 2, x[j]);
  }
}
__device__ __forceinline__ uint2 load_codes(const unsigned char* p, int left, bool vec) {
  if (vec && left >= 8) return *reinterpret_cast<const uint2*>(p);
  uint2 c = make_uint2(0, 0);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) (j < 4 ? c.x : c.y) |= unsigned(p[j]) << (8 * (j & 3));
  return c;
}
__device__ __forceinline__ void store_codes(unsigned char* p, int left, bool vec, uint2 c) {
  if (vec && left >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = (unsigned char)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// values of four e4m3 codes
__device__ __forceinline__ void decode4(unsigned c, float (&x)[8], int at) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((c >> (16 * i)) & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[at + 2 * i] = f.x;
    x[at + 2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float approx_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float block_scale(unsigned top) {
  const float s = __fmul_rn(__uint_as_float(top), 1.f / 448.f);
  return s < kTiny ? kTiny : s;  // a NaN stays
}

// x / s correctly rounded, for inv = 1 / s correctly rounded and x <= 448 s
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990: one residual step).
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, s, x), inv, q);
}

// Stochastic rounding to e4m3.  A value a takes the e4m3 neighbour above it
// where c = (u + 1/2) / 2^16, u a random half, is below a's place between its
// neighbours lo and hi: fl((a - lo) / (hi - lo)) > c, and for kSquares
// fl((fl(a^2) - lo^2) / (hi^2 - lo^2)) > c.
//
// For e4m3's normal values (2^-6 <= |a|, up to 448 or what rounds past it; the
// conversion saturates) both are decided without a quotient:
// * the place is the 20 bits of the fp32 word below e4m3's, so adding
//   2^20 - 1 - 2^20 c to the word carries exactly where it is above c;
// * counted in steps hi - lo, A = a and L = lo (8 to 15), the squares' test is
//   fl(A^2) > L^2 + (2 L + 1) c.  The quotient's rounding cannot matter: c has
//   17 bits, so it would have to lie within (2 L + 1) 2^-25 above the right
//   side, nearer than the last place (2^-17 or 2^-16) of A^2; and the right
//   side, of at most 25 bits, is rounded down, which no A^2 lies between.
// Smaller values and what is not finite take the formulas as they stand.
struct RoundWord {
  unsigned carry;  // 2^20 - 1 - 2^20 c
  float c1;        // 1 + c
  template <bool kHigh> __device__ __forceinline__ void set(unsigned word) {
    carry = (~(kHigh ? word >> 12 : word << 4) & 0xffff0u) | 7u;
    c1 = __uint_as_float(((kHigh ? word >> 9 : word << 7) & 0x7fff80u) | 0x3f800040u);
  }
};

__device__ __forceinline__ float round_linear(float a, const RoundWord& u) {  // either sign
  return __uint_as_float((__float_as_uint(a) + u.carry) & 0xfff00000u);
}

__device__ __forceinline__ float round_squares(float a, const RoundWord& u) {
  const unsigned bits = __float_as_uint(a);
  const float A = __uint_as_float((bits & 0x7fffffu) | 0x41000000u);
  const float L = __uint_as_float(__float_as_uint(A) & 0xfff00000u), D = fmaf(2.f, L, 1.f);
  // (L^2 - D) + D (1 + c)
  const bool up = __fmul_rn(A, A) > __fmaf_rd(D, u.c1, fmaf(L, L, -D));
  return __uint_as_float((bits & 0xfff00000u) + (up ? 0x100000u : 0u));
}

// Any value: e4m3's subnormal ones are steps of 2^-9 from 0; a NaN stays one,
// and for kSquares what is above 0 stays above it.
template <bool kSquares> __device__ __noinline__ float round_any(float a, RoundWord u) {
  const float x = fabsf(a), c = u.c1 - 1.f;
  if (x >= 0.015625f || a != a) {
    if (a != a || x > 480.f) return a;
    return kSquares ? round_squares(a, u) : round_linear(a, u);
  }
  const float A = x * 512.f, L = truncf(A);
  const bool up = kSquares ? __fdiv_rn(__fsub_rn(__fmul_rn(A, A), L * L), fmaf(2.f, L, 1.f)) > c : A - L > c;
  const float r = (L + (up ? 1.f : 0.f)) * 0x1p-9f;
  return kSquares && x > 0.f ? fmaxf(r, 0x1p-9f) : copysignf(r, a);
}

// two values that are e4m3 values already (or past 448) as codes
__device__ __forceinline__ unsigned pack_codes(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int kCap> __device__ __forceinline__ int find_tensor(const AdamArgs<kCap>& a, int run) {
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.t[mid].run0 <= run) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename PT, typename GT, int kBits, int kCap>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs<kCap> a) {
  const AdamHyper& hy = a.hy;
  const float gs = hy.grad_scale != nullptr ? __ldg(hy.grad_scale) : 1.f;
  if (gs == 0.f) return;  // the step is skipped
  const int i = find_tensor(a, blockIdx.x);
  const AdamTensor& t = a.t[i];
  const float lr = hy.lr_dev != nullptr ? __ldg(hy.lr_dev) : hy.lr;
  const long long step = __ldg(hy.step);
  const float ft = float(step > 1 ? step : 1);
  // 1 - beta^t without cancellation
  const float rate = lr / -expm1f(ft * hy.ln_b1), inv2 = rsqrtf(-expm1f(ft * hy.ln_b2));
  const float keep = 1.f - lr * t.wd;
  unsigned char *const p = t.p, *const m = t.m, *const v = t.v, *const copy = t.copy;
  const unsigned char* const g = t.g;
  const long long n = t.n, e0 = (long long)(blockIdx.x - t.run0) * a.run;
  const long long e1 = e0 + a.run < n ? e0 + a.run : n;
  const uintptr_t where = uintptr_t(p) | uintptr_t(g) | uintptr_t(copy);
  const bool vec = kBits == 32 ? ((where | uintptr_t(m) | uintptr_t(v)) & 15) == 0
                               : (where & 15) == 0 && ((uintptr_t(m) | uintptr_t(v)) & 7) == 0;
  DropKey key;
  if constexpr (kBits == 8) key.set(hy.rng);
  // (8-bit states: a warp's 32 threads hold one block of 256 elements)
  for (long long e = e0 + (long long)threadIdx.x * kPer; e - (threadIdx.x & 31) * kPer < e1; e += kTile) {
    const int left = e1 > e ? int(e1 - e < kPer ? e1 - e : kPer) : 0;
    float xp[8], xg[8], xm[8], xv[8];
    load8(p, e, left, vec, xp, PT());
    load8(g, e, left, vec, xg, GT());
    if constexpr (kBits == 32) {
      load8(m, e, left, vec, xm, 0.f);
      load8(v, e, left, vec, xv, 0.f);
    } else {
      const uint2 cm = load_codes(m + e, left, vec), cv = load_codes(v + e, left, vec);
      const float sm = t.ms[e / kAdamBlock], sv = t.vs[e / kAdamBlock];
      decode4(cm.x, xm, 0);
      decode4(cm.y, xm, 4);
      decode4(cv.x, xv, 0);
      decode4(cv.y, xv, 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xm[j] = __fmul_rn(xm[j], sm);
        xv[j] = __fmul_rn(xv[j], sv);
        xv[j] = __fmul_rn(xv[j], xv[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // each operation rounded by itself: the states, and so their codes, are
      // those of the formula as it stands, in fp32 on any machine
      const float gj = __fmul_rn(xg[j], gs);
      xm[j] = __fadd_rn(__fmul_rn(hy.b1, xm[j]), __fmul_rn(hy.a1, gj));
      xv[j] = __fadd_rn(__fmul_rn(hy.b2, xv[j]), __fmul_rn(__fmul_rn(hy.a2, gj), gj));
      const float root = __fsqrt_rn(xv[j]);
      xp[j] = fmaf(-rate, xm[j] * approx_rcp(fmaf(root, inv2, hy.eps)), xp[j] * keep);
      if constexpr (kBits == 8) xv[j] = root;
    }
    store8(p, e, left, vec, xp, PT());
    if (copy != nullptr) store8(copy, e, left, vec, xp, __nv_bfloat16());
    if constexpr (kBits == 32) {
      store8(m, e, left, vec, xm, 0.f);
      store8(v, e, left, vec, xv, 0.f);
    } else {
      unsigned tm = 0, tv = 0, lm = 0x7f800000u, lv = 0x7f800000u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned a = __float_as_uint(xm[j]) & 0x7fffffffu, b = __float_as_uint(xv[j]);
        tm = max(tm, a), lm = min(lm, a);
        tv = max(tv, b), lv = min(lv, b);
      }
      tm = __reduce_max_sync(kFull, tm), tv = __reduce_max_sync(kFull, tv);
      const float sm = block_scale(tm), sv = block_scale(tv);
      const float im = __fdiv_rn(1.f, sm), iv = __fdiv_rn(1.f, sv);
      const bool normal = __uint_as_float(lm) >= sm * 0x1.1p-6f && __uint_as_float(lv) >= sv * 0x1.1p-6f &&
                          tm < 0x7f800000u && tv < 0x7f800000u;  // of e4m3, with some room
      const uint4 u = drop_block(key, a.base + i, unsigned(e >> 3));
      const unsigned word[4] = {u.x, u.y, u.z, u.w};
      unsigned cm2[4], cv2[4];
      // (about one block in 50 of normally distributed gradients has an element
      // that is not; a ragged block always)
      if (__all_sync(kFull, normal || left == 0)) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          RoundWord u0, u1;
          u0.set<false>(word[j / 2]);
          u1.set<true>(word[j / 2]);
          cm2[j / 2] = pack_codes(round_linear(quotient(xm[j], sm, im), u0), round_linear(quotient(xm[j + 1], sm, im), u1));
          cv2[j / 2] = pack_codes(round_squares(quotient(xv[j], sv, iv), u0), round_squares(quotient(xv[j + 1], sv, iv), u1));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          RoundWord u0, u1;
          u0.set<false>(word[j / 2]);
          u1.set<true>(word[j / 2]);
          cm2[j / 2] = pack_codes(round_any<false>(quotient(xm[j], sm, im), u0), round_any<false>(quotient(xm[j + 1], sm, im), u1));
          cv2[j / 2] = pack_codes(round_any<true>(quotient(xv[j], sv, iv), u0), round_any<true>(quotient(xv[j + 1], sv, iv), u1));
        }
      }
      const uint2 cm = make_uint2(cm2[0] | cm2[1] << 16, cm2[2] | cm2[3] << 16);
      const uint2 cv = make_uint2(cv2[0] | cv2[1] << 16, cv2[2] | cv2[3] << 16);
      store_codes(m + e, left, vec, cm);
      store_codes(v + e, left, vec, cv);
      if ((threadIdx.x & 31) == 0) {
        t.ms[e / kAdamBlock] = sm;
        t.vs[e / kAdamBlock] = sv;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// norm of all gradients
// ---------------------------------------------------------------------------
// sum over a CTA of kNormThreads threads, in a fixed order; thread 0 has it
__device__ __forceinline__ float cta_sum(float v, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kNormThreads / 32 ? sm[threadIdx.x] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  }
  return v;
}

constexpr int kNormRun = kNormThreads * kPer * 4;  // elements of a CTA's turn

// Squares of the runs blockIdx.x, blockIdx.x + gridDim.x, ...: eight sums a
// thread, joined by a tree.
template <typename GT, int kCap>
__global__ void __launch_bounds__(kNormThreads) grad_norm_kernel(const __grid_constant__ NormArgs<kCap> a) {
  __shared__ float sm[kNormThreads / 32];
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int run = blockIdx.x; run < a.runs; run += gridDim.x) {
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.run0[mid] <= run) lo = mid;
      else hi = mid;
    }
    const unsigned char* g = a.g[lo];
    const long long e0 = (long long)(run - a.run0[lo]) * kNormRun, n = a.count[lo];
    const bool vec = (uintptr_t(g) & 15) == 0;
    if (vec && e0 + kNormRun <= n) {
      float x[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k) load8(g, e0 + (k * kNormThreads + threadIdx.x) * kPer, 8, true, x[k], GT());
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(x[k][j], x[k][j], s[j]);
    } else {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const long long e = e0 + (k * kNormThreads + threadIdx.x) * kPer;
        const int left = n > e ? int(n - e < kPer ? n - e : kPer) : 0;
        float x[8];
        load8(g, e, left, vec, x, GT());
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(x[j], x[j], s[j]);
      }
    }
  }
  grid_launch_dependents();
  const float v = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  const float total = cta_sum(v, sm);
  if (threadIdx.x == 0) a.part[blockIdx.x] = total;
}

// The CTAs' sums in fp64, in a fixed order: thread i takes every 256th.
__global__ void __launch_bounds__(256) grad_norm_finish(const float* part, int parts, float max_norm, float* norm_out,
                                                        float* scale_out) {
  __shared__ double sm[256];
  grid_dependency_wait();
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) v += double(__ldcg(part + i));
  sm[threadIdx.x] = v;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) sm[threadIdx.x] += sm[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float norm = float(sqrt(sm[0]));
    if (norm_out != nullptr) *norm_out = norm;
    if (scale_out != nullptr) {
      const float scale = norm > max_norm ? float(double(max_norm) / sqrt(sm[0])) : 1.f;
      *scale_out = isfinite(norm) ? scale : 0.f;
    }
  }
}

template <typename PT, typename GT, int kBits, int kCap>
void step_launch(const vpce_adamw_tensor* tensors, long long first, long long count, const AdamHyper& hy, int sms,
                 cudaStream_t st) {
  AdamArgs<kCap> a;
  a.hy = hy;
  a.base = int(first);
  a.n = 0;
  long long total = 0;
  for (long long i = 0; i < count; ++i) total += tensors[first + i].n;
  // a run: long enough to spread a CTA's start over several turns, short
  // enough that every SM has some
  long long turns = total / ((long long)kTile * sms * 8);
  turns = turns < 1 ? 1 : turns > 8 ? 8 : turns;
  a.run = int(turns) * kTile;
  long long runs = 0;
  for (long long i = 0; i < count; ++i) {
    const vpce_adamw_tensor& t = tensors[first + i];
    AdamTensor& d = a.t[a.n++];
    d.p = static_cast<unsigned char*>(t.param);
    d.g = static_cast<const unsigned char*>(t.grad);
    d.copy = static_cast<unsigned char*>(t.copy);
    d.m = static_cast<unsigned char*>(t.exp_avg);
    d.v = static_cast<unsigned char*>(t.exp_avg_sq);
    d.ms = t.exp_avg_scale;
    d.vs = t.exp_avg_sq_scale;
    d.n = t.n;
    d.wd = t.weight_decay;
    d.run0 = int(runs);
    runs += (t.n + a.run - 1) / a.run;
  }
  if (runs > 0) adamw_kernel<PT, GT, kBits, kCap><<<int(runs), kThreads, 0, st>>>(a);
}

template <typename PT, typename GT, int kBits>
void step_all(const vpce_adamw_tensor* tensors, long long n, const AdamHyper& hy, int sms, cudaStream_t st) {
  for (long long i = 0; i < n; i += kAdamTensors) {
    const long long count = n - i < kAdamTensors ? n - i : kAdamTensors;
    if (count <= kAdamFewTensors) step_launch<PT, GT, kBits, kAdamFewTensors>(tensors, i, count, hy, sms, st);
    else step_launch<PT, GT, kBits, kAdamTensors>(tensors, i, count, hy, sms, st);
  }
}

template <typename PT, typename GT>
void step_bits(const vpce_adamw_tensor* tensors, long long n, int bits, const AdamHyper& hy, int sms, cudaStream_t st) {
  if (bits == 32) step_all<PT, GT, 32>(tensors, n, hy, sms, st);
  else step_all<PT, GT, 8>(tensors, n, hy, sms, st);
}

template <typename GT, int kCap>
int norm_launch(const vpce_adamw_tensor* tensors, long long count, float* part, int sms, cudaStream_t st) {
  NormArgs<kCap> a;
  a.n = int(count);
  a.part = part;
  long long runs = 0;
  for (long long i = 0; i < count; ++i) {
    a.g[i] = static_cast<const unsigned char*>(tensors[i].grad);
    a.count[i] = tensors[i].n;
    a.run0[i] = int(runs);
    runs += (tensors[i].n + kNormRun - 1) / kNormRun;
  }
  if (runs == 0) return 0;
  a.runs = int(runs);
  const int most = sms * 4 < kNormMaxCtas ? sms * 4 : kNormMaxCtas;
  const int grid = int(runs < most ? runs : most);
  grad_norm_kernel<GT, kCap><<<grid, kNormThreads, 0, st>>>(a);
  return grid;
}

template <typename GT>
int norm_all(const vpce_adamw_tensor* tensors, long long n, float* part, int sms, cudaStream_t st) {
  int parts = 0;
  for (long long i = 0; i < n; i += kAdamTensors) {
    const long long count = n - i < kAdamTensors ? n - i : kAdamTensors;
    parts += count <= kAdamFewTensors ? norm_launch<GT, kAdamFewTensors>(tensors + i, count, part + parts, sms, st)
                                      : norm_launch<GT, kAdamTensors>(tensors + i, count, part + parts, sms, st);
  }
  return parts;
}

}  // namespace

void launch_adamw(const vpce_adamw_tensor* tensors, long long n, bool param_bf16, bool grad_bf16, int bits,
                  const AdamHyper& hy, int sms, cudaStream_t st) {
  if (param_bf16) {
    if (grad_bf16) step_bits<__nv_bfloat16, __nv_bfloat16>(tensors, n, bits, hy, sms, st);
    else step_bits<__nv_bfloat16, float>(tensors, n, bits, hy, sms, st);
  } else {
    if (grad_bf16) step_bits<float, __nv_bfloat16>(tensors, n, bits, hy, sms, st);
    else step_bits<float, float>(tensors, n, bits, hy, sms, st);
  }
}

size_t grad_norm_workspace_bytes(long long n) {
  return round256(size_t((n + kAdamTensors - 1) / kAdamTensors) * kNormMaxCtas * sizeof(float) + 256);
}

cudaError_t launch_grad_norm(const vpce_adamw_tensor* tensors, long long n, bool grad_bf16, float max_norm,
                             float* norm_out, float* scale_out, void* ws, int sms, cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  const int parts = grad_bf16 ? norm_all<__nv_bfloat16>(tensors, n, part, sms, st) : norm_all<float>(tensors, n, part, sms, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a programmatic dependent: its launch is hidden behind the last runs
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, grad_norm_finish, (const float*)part, parts, max_norm, norm_out, scale_out);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace vpce
