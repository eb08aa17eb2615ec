// Device-side pieces of the norm and of the AdamW step: copies that every thread
// makes for itself, magnitudes of eight values, and scales of e4m3 codes.
#pragma once

#include "vpce_device.cuh"

namespace vpce {

// global -> shared copies of 4, 8 or 16 bytes that every thread makes for
// itself (cp.async).  kThroughL1: also for 16 bytes (the others always do).
template <int kBytes, bool kThroughL1 = kBytes != 16>
__device__ __forceinline__ void copy_async(void* dst_smem, const void* src) {
  if constexpr (kThroughL1)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst_smem)), "l"(src), "n"(kBytes) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst_smem)), "l"(src), "n"(kBytes) : "memory");
}
// 16 bytes to shared memory of which `bytes` are read and the others set to 0
__device__ __forceinline__ void copy_async_part(void* dst_smem, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst_smem)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's groups of them are incomplete.
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The largest (a NaN if there is one) and the least magnitude of eight.
__device__ __forceinline__ float most_magnitude(const float (&x)[8]) {
  float a, b, c;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(x[6]), "f"(x[7]), "f"(a));
  asm("max.NaN.abs.f32 %0, %1, %2, %2;" : "=f"(a) : "f"(b), "f"(c));
  return a;
}
__device__ __forceinline__ float least_magnitude(const float (&x)[8]) {
  float a, b, c;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(x[6]), "f"(x[7]), "f"(a));
  asm("min.abs.f32 %0, %1, %2, %2;" : "=f"(a) : "f"(b), "f"(c));
  return a;
}

// Scale of values whose largest magnitude has the bits `top`: that over e4m3's
// largest value, at least 2^-126, so that its reciprocal is finite.  A NaN stays.
__device__ __forceinline__ float e4m3_scale(unsigned top) {
  const float s = __fmul_rn(__uint_as_float(top), 1.f / 448.f);
  return s < 0x1p-126f ? 0x1p-126f : s;
}

// x / s correctly rounded, for inv = 1 / s correctly rounded, s from 2^-95 up and
// |x| at most 448 s or so (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990: one residual step).  Below 2^-95 the
// residual passes fp32's smallest number: the result is within two ulps.  For an
// infinite scale, s is given as 0: the result is x inv, 0 or, of an infinity, NaN.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, s, x), inv, q);
}

// The same of two values (minus_s = -s).
__device__ __forceinline__ f32x2 both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ f32x2 quotient2(f32x2 x, f32x2 minus_s, f32x2 inv) {
  const f32x2 q = f2_mul(x, inv);
  return f2_fma(f2_fma(q, minus_s, x), inv, q);
}

// Roots of two values from 2^-100 to 2^127 by the same paper's residual step on
// v rsqrt(v): correctly rounded.  No bound of rsqrt.approx's error implies it, so
// a test compares every value of the range with CUDA's correctly rounded root.
__device__ __forceinline__ f32x2 root2(f32x2 v) {
  float a, b, ya, yb;
  f2_unpack(v, a, b);
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(ya) : "f"(a));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(yb) : "f"(b));
  const f32x2 y = f2_pack(ya, yb), r = f2_mul(v, y), h = f2_mul(y, both(0.5f));
  return f2_fma(f2_fma(f2_mul(r, both(-1.f)), r, v), h, r);
}

}  // namespace vpce
