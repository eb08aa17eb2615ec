// AdamW over many tensors in one launch, states in fp32 or in e4m3 with a
// scale per 256 elements, and the norm of all gradients.
//
// The tensors' addresses travel in the kernels' parameters (32 KB hold 440),
// so that a step is one launch, captured graphs carry them by value, and
// nothing is copied to the device.  A CTA takes a run of consecutive elements
// of one tensor, found by bisection over the runs' numbers.
//
// With fp32 states HBM bounds the step: 30 bytes an element (weights and
// gradients fp32, bf16 copies), 128256 x 4096 2287 us, 6.9 TB/s.  With 8-bit
// states 18 bytes an element come with 79 instructions (32 on the integer and
// logic pipe, 30 on those of multiplications): 50304 x 4096 642 us, 5.8 TB/s, the
// issue slots 68% busy.  The gradients' norm reads 128256 x 4096 fp32 in 307 us,
// 6.8 TB/s.
#include <cmath>

#include <cuda_fp8.h>

#include "vpce_adamw.cuh"
#include "vpce_embed_dropout.cuh"

namespace vpce {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                       // consecutive elements of a thread
constexpr int kTile = kThreads * kPer;        // elements of a CTA's turn

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

// Stochastic rounding to e4m3.  A value a takes the e4m3 neighbour above it
// where c = (u + 1/2) / 2^16, u a random half, is below a's place between its
// neighbours lo and hi: fl((a - lo) / (hi - lo)) > c, and for kSquares
// fl((fl(a^2) - lo^2) / (hi^2 - lo^2)) > c.
//
// For e4m3's normal values (2^-6 <= |a|, up to 448 or what rounds past it; the
// conversion saturates) both are decided without a quotient:
// * the place is the 20 bits of the fp32 word below e4m3's, so adding
//   2^20 - 1 - 2^20 c to the word carries exactly where it is above c (c1 >> 3
//   is 2^20 c + 0x17f00000);
// * counted in steps hi - lo, A = a and L = lo (8 to 15), the squares' test is
//   fl(A^2) > L^2 + (2 L + 1) c.  The quotient's rounding cannot matter: c has
//   17 bits, so it would have to lie within (2 L + 1) 2^-25 above the right
//   side, nearer than the last place (2^-17 or 2^-16) of A^2; and the right
//   side, of at most 25 bits, is rounded down, which no A^2 lies between.
// Smaller values and what is not finite take the formulas as they stand.
struct RoundWord {
  unsigned c1;  // bits of -(1 + c)
  template <bool kHigh> __device__ __forceinline__ void set(unsigned word) {
    c1 = ((kHigh ? word >> 9 : word << 7) & 0x7fff80u) | 0xbf800040u;
  }
  __device__ __forceinline__ float minus() const { return __uint_as_float(c1); }
};

__device__ __forceinline__ float round_linear(float a, const RoundWord& u) {  // either sign
  // (2^20 c is c1's mantissa, an eighth of it)
  return __uint_as_float((__float_as_uint(a) + 0x17ffffffu - (u.c1 >> 3)) & 0xfff00000u);
}

// The same for any finite value: below 2^-6, adding 2^-6 gives the word whose
// 20 lower bits are the place (rounded up, which no c lies between).
__device__ __forceinline__ float round_linear_small(float a, const RoundWord& u) {
  const float x = fabsf(a), by = x < 0x1p-6f ? 0x1p-6f : 0.f;
  return copysignf(round_linear(__fadd_ru(x, by), u) - by, a);
}

__device__ __forceinline__ float round_squares(float a, const RoundWord& u) {
  const unsigned bits = __float_as_uint(a);
  const float A = __uint_as_float((bits & 0x7fffffu) | 0x41000000u);
  const float L = __uint_as_float(__float_as_uint(A) & 0xfff00000u), minus_d = fmaf(-2.f, L, -1.f);
  // (L^2 - D) + D (1 + c), D = 2 L + 1
  const bool up = __fmul_rn(A, A) > __fmaf_rd(minus_d, u.minus(), fmaf(L, L, minus_d));
  return __uint_as_float((bits & 0xfff00000u) + (up ? 0x100000u : 0u));
}

// Any value: e4m3's subnormal ones are steps of 2^-9 from 0; a NaN stays one,
// and for kSquares what is above 0 stays above it.
template <bool kSquares> __device__ __noinline__ float round_any(float a, RoundWord u) {
  const float x = fabsf(a), c = -u.minus() - 1.f;
  if (x >= 0.015625f || a != a) {
    if (a != a || x > 480.f) return a;
    return kSquares ? round_squares(a, u) : round_linear(a, u);
  }
  if (!kSquares) return round_linear_small(a, u);
  const float A = x * 512.f, L = truncf(A);
  const bool up = __fdiv_rn(__fsub_rn(__fmul_rn(A, A), L * L), fmaf(2.f, L, 1.f)) > c;
  return x > 0.f ? fmaxf((L + (up ? 1.f : 0.f)) * 0x1p-9f, 0x1p-9f) : 0.f;
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

// What one step's arithmetic needs besides the elements.
struct StepScalars {
  float gs, b1, a1, b2, a2, rate, inv2, eps, keep;
};

// p of one element from its new m and v; v becomes its root.
__device__ __forceinline__ void apply(const StepScalars& c, float& p, float m, float& v) {
  v = __fsqrt_rn(v);
  p = fmaf(-c.rate, m * approx_rcp(fmaf(v, c.inv2, c.eps)), p * c.keep);
}

// m, v and p of eight elements; xv becomes v, or its root for kRoot.  Each
// operation on m and v is rounded by itself: the states, and so their codes,
// are those of the formula as it stands, in fp32 on any machine.
template <bool kRoot>
__device__ __forceinline__ void update8(const StepScalars& c, float (&xp)[8], const float (&xg)[8], float (&xm)[8],
                                        float (&xv)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float g = __fmul_rn(xg[j], c.gs);
    xm[j] = __fadd_rn(__fmul_rn(c.b1, xm[j]), __fmul_rn(c.a1, g));
    xv[j] = __fadd_rn(__fmul_rn(c.b2, xv[j]), __fmul_rn(__fmul_rn(c.a2, g), g));
    float root = xv[j];
    apply(c, xp[j], xm[j], root);
    if constexpr (kRoot) xv[j] = root;
  }
}

__device__ __forceinline__ void decode8(uint2 cm, uint2 cv, float sm, float sv, float (&xm)[8], float (&xv)[8]) {
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

// quotient() is correctly rounded for scales from 2^-95 up; below, its residual
// passes fp32's smallest number.  m's scale may lie there (rows of a table that
// have had no gradient for long), the root of v's not: v is 0 or 2^-149 at least.
constexpr float kExactScale = 0x1p-94f;
// What both sides of such a quotient are multiplied by, and the reciprocal
// divided by, without rounding.
struct ExactScale {
  float up, down;
  __device__ __forceinline__ explicit ExactScale(float s)
      : up(s < kExactScale ? 0x1p64f : 1.f), down(s < kExactScale ? 0x1p-64f : 1.f) {}
};

// New codes and scales of a block of 256 elements, eight a lane: m in xm, the
// root of v in xv, `inside` false on lanes past the block's end.
__device__ __forceinline__ void encode8(const float (&xm)[8], const float (&xv)[8], uint4 random, bool inside, uint2& cm,
                                        uint2& cv, float& sm, float& sv) {
  unsigned tm = 0, tv = 0, lm = 0x7f800000u, lv = 0x7f800000u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned a = __float_as_uint(xm[j]) & 0x7fffffffu, b = __float_as_uint(xv[j]);
    tm = max(tm, a), lm = min(lm, a);
    tv = max(tv, b), lv = min(lv, b);
  }
  tm = __reduce_max_sync(kFull, tm), tv = __reduce_max_sync(kFull, tv);
  sm = e4m3_scale(tm), sv = e4m3_scale(tv);
  const float im = __fdiv_rn(1.f, sm), iv = __fdiv_rn(1.f, sv);
  const bool normal = __uint_as_float(lm) >= sm * 0x1.1p-6f && __uint_as_float(lv) >= sv * 0x1.1p-6f &&
                      tm < 0x7f800000u && tv < 0x7f800000u && sm >= kExactScale;  // of e4m3, with some room
  const unsigned word[4] = {random.x, random.y, random.z, random.w};
  unsigned m2[4], v2[4];
  // (about one block in 50 of normally distributed gradients has an element
  // that is not; a ragged block always)
  if (__all_sync(kFull, normal || !inside)) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      RoundWord u0, u1;
      u0.set<false>(word[j / 2]);
      u1.set<true>(word[j / 2]);
      m2[j / 2] = pack_codes(round_linear(quotient(xm[j], sm, im), u0), round_linear(quotient(xm[j + 1], sm, im), u1));
      v2[j / 2] = pack_codes(round_squares(quotient(xv[j], sv, iv), u0), round_squares(quotient(xv[j + 1], sv, iv), u1));
    }
  } else {
    const ExactScale by(sm);
    const float s = sm * by.up, inv = im * by.down;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      RoundWord u0, u1;
      u0.set<false>(word[j / 2]);
      u1.set<true>(word[j / 2]);
      m2[j / 2] = pack_codes(round_any<false>(quotient(xm[j] * by.up, s, inv), u0),
                             round_any<false>(quotient(xm[j + 1] * by.up, s, inv), u1));
      v2[j / 2] = pack_codes(round_any<true>(quotient(xv[j], sv, iv), u0), round_any<true>(quotient(xv[j + 1], sv, iv), u1));
    }
  }
  cm = make_uint2(m2[0] | m2[1] << 16, m2[2] | m2[3] << 16);
  cv = make_uint2(v2[0] | v2[1] << 16, v2[2] | v2[3] << 16);
}

// ---------------------------------------------------------------------------
// The same on pairs of fp32 values (one instruction for two), for blocks whose
// values are all ordinary: no quotient by a division, no special case, 79
// instructions an element (118 on single values).  m, v and the codes are the
// same bits.
// ---------------------------------------------------------------------------
__device__ __forceinline__ f32x2 f2_fma_down(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The sums of two pairs of products, which a packed sum would fuse with one of
// them (measured: the packed forms are contracted where the single ones, with
// their rounding named, are not).
__device__ __forceinline__ f32x2 sum2(f32x2 a, f32x2 b) {
  float a0, a1, b0, b1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  return f2_pack(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

struct StepPairs {
  f32x2 gs, b1, a1, b2, a2, rate, inv2, eps, keep;
  __device__ __forceinline__ explicit StepPairs(const StepScalars& c)
      : gs(both(c.gs)), b1(both(c.b1)), a1(both(c.a1)), b2(both(c.b2)), a2(both(c.a2)), rate(both(-c.rate)),
        inv2(both(c.inv2)), eps(both(c.eps)), keep(both(c.keep)) {}
};

// round_linear of two quotients x / s (with `small`: round_linear_small, and x
// and s as ExactScale has them), and round_squares of two values
__device__ __forceinline__ unsigned linear_codes2(f32x2 x, float s, float inv, const RoundWord& u0, const RoundWord& u1,
                                                  bool small) {
  float a, b;
  if (small) {
    const ExactScale by(s);
    f2_unpack(quotient2(f2_mul(x, both(by.up)), both(-s * by.up), both(inv * by.down)), a, b);
    return pack_codes(round_linear_small(a, u0), round_linear_small(b, u1));
  }
  f2_unpack(quotient2(x, both(-s), both(inv)), a, b);
  return pack_codes(round_linear(a, u0), round_linear(b, u1));
}
__device__ __forceinline__ unsigned square_codes2(f32x2 a, const RoundWord& u0, const RoundWord& u1) {
  float x, y, ax, ay, tx, ty;
  f2_unpack(a, x, y);
  const unsigned bx = __float_as_uint(x), by = __float_as_uint(y);
  const unsigned Ax = (bx & 0x7fffffu) | 0x41000000u, Ay = (by & 0x7fffffu) | 0x41000000u;
  const f32x2 A = f2_pack(__uint_as_float(Ax), __uint_as_float(Ay));
  const f32x2 L = f2_pack(__uint_as_float(Ax & 0xfff00000u), __uint_as_float(Ay & 0xfff00000u));
  const f32x2 minus_d = f2_fma(L, both(-2.f), both(-1.f));
  f2_unpack(f2_mul(A, A), ax, ay);
  f2_unpack(f2_fma_down(minus_d, f2_pack(u0.minus(), u1.minus()), f2_fma(L, L, minus_d)), tx, ty);
  return pack_codes(__uint_as_float((bx & 0xfff00000u) + (ax > tx ? 0x100000u : 0u)),
                    __uint_as_float((by & 0xfff00000u) + (ay > ty ? 0x100000u : 0u)));
}

// One element type's part of the ring: eight elements a thread, in one or two
// vectors of shared memory kThreads apart.
template <typename T> struct Ahead {
  uint4 v[sizeof(T) / 2][kThreads];
  __device__ __forceinline__ void copy(const unsigned char* src) {
    copy_async<16, sizeof(T) == 4>(&v[0][threadIdx.x], src);  // (two vectors share sectors: through L1)
    if constexpr (sizeof(T) == 4) copy_async<16, true>(&v[1][threadIdx.x], src + 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      unpack(v[0][threadIdx.x], x, T());
    } else {
      const float4 a = *reinterpret_cast<const float4*>(&v[0][threadIdx.x]),
                   b = *reinterpret_cast<const float4*>(&v[1][threadIdx.x]);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  }
};

template <typename PT, typename GT, int kBits, int kCap>
__global__ void __launch_bounds__(kThreads, kBits == 8 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamArgs<kCap> a) {
  const AdamHyper& hy = a.hy;
  const int i = find_tensor(a, blockIdx.x);
  const AdamTensor& t = a.t[i];
  unsigned char *const p = t.p, *const m = t.m, *const v = t.v, *const copy = t.copy;
  const unsigned char* const g = t.g;
  const long long n = t.n, e0 = (long long)(blockIdx.x - t.run0) * a.run;
  const long long e1 = e0 + a.run < n ? e0 + a.run : n;
  const uintptr_t where = uintptr_t(p) | uintptr_t(g) | uintptr_t(copy);
  const bool vec = kBits == 32 ? ((where | uintptr_t(m) | uintptr_t(v)) & 15) == 0
                               : (where & 15) == 0 && ((uintptr_t(m) | uintptr_t(v)) & 7) == 0;
  // Whole runs of 8-bit states in vectors come through a ring of two turns that
  // each thread fills for itself, the first of them before anything else is
  // read: the codes' arithmetic takes about 70% of the SM's issue slots, so
  // loads have to be under way meanwhile.
  constexpr bool kRing = kBits == 8;
  __shared__ Ahead<PT> rp[kRing ? 2 : 1];
  __shared__ Ahead<GT> rg[kRing ? 2 : 1];
  __shared__ uint2 rm[kRing ? 2 : 1][kThreads], rv[kRing ? 2 : 1][kThreads];
  const auto fetch = [&](long long at, int stage) {
    rp[stage].copy(p + at * sizeof(PT));
    rg[stage].copy(g + at * sizeof(GT));
    copy_async<8>(&rm[stage][threadIdx.x], m + at);
    copy_async<8>(&rv[stage][threadIdx.x], v + at);
  };
  const bool ring = kRing && vec && e1 - e0 == a.run;
  const int turns = a.run / kTile;
  long long e = e0 + (long long)threadIdx.x * kPer;
  float sm = 0.f, sv = 0.f;
  if (ring) {
    fetch(e, 0);
    copy_commit();
    if (turns > 1) fetch(e + kTile, 1);
    copy_commit();
    sm = t.ms[e / kAdamBlock], sv = t.vs[e / kAdamBlock];
  }
  const float gs = hy.grad_scale != nullptr ? __ldg(hy.grad_scale) : 1.f;
  const float lr = hy.lr_dev != nullptr ? __ldg(hy.lr_dev) : hy.lr;
  const long long step = __ldg(hy.step);
  [[maybe_unused]] DropKey key;
  if constexpr (kBits == 8) key.set(hy.rng);
  if (gs == 0.f) {  // the step is skipped
    copy_wait<0>();
    return;
  }
  const float ft = float(step > 1 ? step : 1);
  // 1 - beta^t without cancellation
  const StepScalars c = {gs, hy.b1, hy.a1, hy.b2, hy.a2, lr / -expm1f(ft * hy.ln_b1), rsqrtf(-expm1f(ft * hy.ln_b2)),
                         hy.eps, 1.f - lr * t.wd};

  if constexpr (kRing) {
    if (ring) {
      const StepPairs c2(c);
      for (int turn = 0; turn < turns; ++turn, e += kTile) {
        const int stage = turn & 1;
        float next_sm = 0.f, next_sv = 0.f;
        if (turn + 1 < turns) {
          next_sm = t.ms[(e + kTile) / kAdamBlock];
          next_sv = t.vs[(e + kTile) / kAdamBlock];
        }
        const uint4 random = drop_block(key, a.base + i, unsigned(e >> 3));
        copy_wait<1>();
        f32x2 xp[4], xm[4], xv[4];
        {
          float p8[8], g8[8], m8[8], v8[8];
          rp[stage].get(p8);
          rg[stage].get(g8);
          const uint2 cm = rm[stage][threadIdx.x], cv = rv[stage][threadIdx.x];
          decode4(cm.x, m8, 0);
          decode4(cm.y, m8, 4);
          decode4(cv.x, v8, 0);
          decode4(cv.y, v8, 4);
          const f32x2 sm2 = both(sm), sv2 = both(sv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2 g = f2_mul(f2_pack(g8[2 * j], g8[2 * j + 1]), c2.gs);
            const f32x2 m0 = f2_mul(f2_pack(m8[2 * j], m8[2 * j + 1]), sm2);
            f32x2 v0 = f2_mul(f2_pack(v8[2 * j], v8[2 * j + 1]), sv2);
            v0 = f2_mul(v0, v0);
            xm[j] = sum2(f2_mul(c2.b1, m0), f2_mul(c2.a1, g));
            xv[j] = sum2(f2_mul(c2.b2, v0), f2_mul(f2_mul(c2.a2, g), g));
            xp[j] = f2_pack(p8[2 * j], p8[2 * j + 1]);
          }
        }
        if (turn + 2 < turns) fetch(e + 2 * kTile, stage);  // (the stage's values are in registers)
        copy_commit();
        float m8[8], v8[8], p8[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f2_unpack(xm[j], m8[2 * j], m8[2 * j + 1]);
          f2_unpack(xv[j], v8[2 * j], v8[2 * j + 1]);
        }
        const float lm = least_magnitude(m8), lv = least_magnitude(v8);
        const unsigned tm = __reduce_max_sync(kFull, __float_as_uint(most_magnitude(m8)));
        const unsigned tv = __reduce_max_sync(kFull, __float_as_uint(most_magnitude(v8)));
        // half of the warp finds m's scale and its reciprocal, half sqrt(v)'s
        // (the root is monotone: the largest v's is the largest)
        const bool second = (threadIdx.x & 16) != 0;
        const float root_top = __fsqrt_rn(__uint_as_float(tv));
        const float scale = e4m3_scale(second ? __float_as_uint(root_top) : tm), inv = __frcp_rn(scale);
        sm = __shfl_sync(kFull, scale, 0), sv = __shfl_sync(kFull, scale, 16);
        // v: of e4m3's normal values, with some room, and of root2's range
        // (2.8e-4 > (2^-6)^2: v is compared with the scale's square).  About
        // one block in 50 of normally distributed gradients has an m below them.
        const bool ordinary = lv >= fmaxf(sv * sv * 2.8e-4f, 0x1p-100f) && tm < 0x7f800000u && tv < 0x7f000000u;
        const bool small = !__all_sync(kFull, lm >= sm * 0x1.1p-6f) || sm < kExactScale;
        uint2 cm, cv;
        if (__all_sync(kFull, ordinary)) {
          const float im = __shfl_sync(kFull, inv, 0), iv = __shfl_sync(kFull, inv, 16);
          const f32x2 iv2 = both(iv), nsv = both(-sv);
          const unsigned word[4] = {random.x, random.y, random.z, random.w};
          unsigned mc[4], vc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2 root = root2(xv[j]);
            float d0, d1;
            f2_unpack(f2_fma(root, c2.inv2, c2.eps), d0, d1);
            xp[j] = f2_fma(c2.rate, f2_mul(xm[j], f2_pack(approx_rcp(d0), approx_rcp(d1))), f2_mul(xp[j], c2.keep));
            RoundWord u0, u1;
            u0.set<false>(word[j]);
            u1.set<true>(word[j]);
            mc[j] = linear_codes2(xm[j], sm, im, u0, u1, small);
            vc[j] = square_codes2(quotient2(root, nsv, iv2), u0, u1);
          }
          cm = make_uint2(mc[0] | mc[1] << 16, mc[2] | mc[3] << 16);
          cv = make_uint2(vc[0] | vc[1] << 16, vc[2] | vc[3] << 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) f2_unpack(xp[j], p8[2 * j], p8[2 * j + 1]);
        } else if (tm == 0 && tv == 0 && c.eps > 0.f) {
          // a block that has had no gradient yet, as rows of a table do
          cm = cv = make_uint2(0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) f2_unpack(f2_mul(xp[j], c2.keep), p8[2 * j], p8[2 * j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) f2_unpack(xp[j], p8[2 * j], p8[2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) apply(c, p8[j], m8[j], v8[j]);
          encode8(m8, v8, random, true, cm, cv, sm, sv);
        }
        store8(p, e, 8, true, p8, PT());
        if (copy != nullptr) store8(copy, e, 8, true, p8, __nv_bfloat16());
        *reinterpret_cast<uint2*>(m + e) = cm;
        *reinterpret_cast<uint2*>(v + e) = cv;
        if ((threadIdx.x & 31) == 0) {
          t.ms[e / kAdamBlock] = sm;
          t.vs[e / kAdamBlock] = sv;
        }
        sm = next_sm;
        sv = next_sv;
      }
      return;
    }
  }
  // (8-bit states: a warp's 32 threads hold one block of 256 elements)
  for (; e - (threadIdx.x & 31) * kPer < e1; e += kTile) {
    const int left = e1 > e ? int(e1 - e < kPer ? e1 - e : kPer) : 0;
    float xp[8], xg[8], xm[8], xv[8];
    load8(p, e, left, vec, xp, PT());
    load8(g, e, left, vec, xg, GT());
    if constexpr (kBits == 32) {
      load8(m, e, left, vec, xm, 0.f);
      load8(v, e, left, vec, xv, 0.f);
      update8<false>(c, xp, xg, xm, xv);
    } else {
      const uint2 cm = load_codes(m + e, left, vec), cv = load_codes(v + e, left, vec);
      decode8(cm, cv, t.ms[e / kAdamBlock], t.vs[e / kAdamBlock], xm, xv);
      update8<true>(c, xp, xg, xm, xv);
    }
    store8(p, e, left, vec, xp, PT());
    if (copy != nullptr) store8(copy, e, left, vec, xp, __nv_bfloat16());
    if constexpr (kBits == 32) {
      store8(m, e, left, vec, xm, 0.f);
      store8(v, e, left, vec, xv, 0.f);
    } else {
      uint2 cm, cv;
      encode8(xm, xv, drop_block(key, a.base + i, unsigned(e >> 3)), left > 0, cm, cv, sm, sv);
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
  // a run: long enough to spread a CTA's start over several turns, and some 32
  // runs an SM, of which three or four are resident, so that the last ones do
  // not leave SMs idle (12 layers of 512, 8-bit states: 8 runs an SM 119 us, 32
  // 110; 50304 x 4096: turns up to 16 667 us, up to 10 638)
  long long turns = total / ((long long)kTile * sms * 32);
  turns = turns < 1 ? 1 : turns > 10 ? 10 : turns;
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
    else if (count <= kAdamSomeTensors) step_launch<PT, GT, kBits, kAdamSomeTensors>(tensors, i, count, hy, sms, st);
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
    parts += count <= kAdamFewTensors    ? norm_launch<GT, kAdamFewTensors>(tensors + i, count, part + parts, sms, st)
             : count <= kAdamSomeTensors ? norm_launch<GT, kAdamSomeTensors>(tensors + i, count, part + parts, sms, st)
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
