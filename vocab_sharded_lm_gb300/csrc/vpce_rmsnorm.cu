// Root-mean-square norm with the residual's addition, its output as it is or
// as e4m3 codes with scales per group of columns.
//
// One pass: a row is read once into registers as fp32 (r = x + residual), its
// squares are summed over the row's threads, and the same registers give the
// output, so the only traffic is the operands'.  It is bound by HBM: at
// h = 8192 bf16 a row moves 64 KB for some 5 operations an element.
#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126: the least scale, so that 1 / scale is finite

__device__ __forceinline__ unsigned short e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store_codes(unsigned char* p, const float (&v)[8]) {
  const uint32_t a = e4m3x2(v[0], v[1]) | uint32_t(e4m3x2(v[2], v[3])) << 16;
  const uint32_t b = e4m3x2(v[4], v[5]) | uint32_t(e4m3x2(v[6], v[7])) << 16;
  *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
}
__device__ __forceinline__ void store_codes(unsigned char* p, const float (&v)[1]) {
  *p = (unsigned char)(e4m3x2(v[0], 0.f) & 0xff);
}

// |v| as ordered bits: infinities above every number, NaN above them, so that
// a maximum of these bits carries a NaN on.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ float group_scale(unsigned top) {
  const float s = __fdiv_rn(__uint_as_float(top), 448.f);
  return s < kTiny ? kTiny : s;  // a NaN stays
}

template <typename XT, typename RT, bool kCodes, int U, int NU, bool kWarp, int kMaxT>
__global__ void __launch_bounds__(kMaxT) rmsnorm_forward_kernel(const __grid_constant__ RmsNormParams p) {
  extern __shared__ unsigned top_sm[];  // [teams][2][groups], codes only
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31;
  const int team = kWarp ? int(threadIdx.x >> 5) : 0, teams = kWarp ? int(blockDim.x >> 5) : 1;
  const int tid = kWarp ? lane : int(threadIdx.x), T = kWarp ? 32 : int(blockDim.x);
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + team; row < p.s; row += (long long)gridDim.x * teams) {
    const unsigned char* xr = p.x + row * p.ld_x;
    RawUnit<XT, U> a[NU];
    RawUnit<RT, U> b[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      a[k].zero();
      if (c < p.h) a[k].load(xr, c);
    }
    if (p.res != nullptr) {
      const unsigned char* rr = p.res + row * p.ld_res;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        b[k].zero();
        if (c < p.h) b[k].load(rr, c);
      }
    }
    float r[NU][U], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      a[k].get(r[k]);
      if (p.res != nullptr) {
        float q[U];
        b[k].get(q);
#pragma unroll
        for (int j = 0; j < U; ++j) r[k][j] += q[j];
        if (c < p.h) store_unit(p.res_out + row * p.ld_res_out, c, r[k], RT());
      }
#pragma unroll
      for (int j = 0; j < U; ++j) ss = fmaf(r[k][j], r[k][j], ss);
    }
    // the two buffers alternate: who still reads one row's is at most a
    // barrier behind whoever writes the next row's
    unsigned* top = kCodes ? top_sm + (team * 2 + parity) * p.groups : nullptr;
    if constexpr (kCodes) {
      for (int g = tid; g < p.groups; g += T) top[g] = 0;
      if constexpr (kWarp) __syncwarp();
    }
    ss = team_sum<kWarp>(ss, red[parity]);
    parity ^= 1;
    const float rstd = rsqrtf(ss / float(p.h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      if (c < p.h) {
        float w[U];
        load_weight(p.w, p.w_bf16, c, w);
#pragma unroll
        for (int j = 0; j < U; ++j) r[k][j] = r[k][j] * rstd * w[j];
        if constexpr (!kCodes) {
          store_unit(p.out + row * p.ld_out, c, r[k], XT());
        } else {
          unsigned m = 0;
#pragma unroll
          for (int j = 0; j < U; ++j) m = max(m, mag(r[k][j]));
          atomicMax(top + c / p.group, m);  // shared memory; the order does not matter
        }
      }
    }
    if constexpr (kCodes) {
      if constexpr (kWarp) __syncwarp();
      else __syncthreads();
      for (int g = tid; g < p.groups; g += T) p.scale[row * p.groups + g] = group_scale(top[g]);
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (c < p.h) {
          const float inv = __fdiv_rn(1.f, group_scale(top[c / p.group]));
#pragma unroll
          for (int j = 0; j < U; ++j) r[k][j] *= inv;
          store_codes(p.out + row * p.ld_out + c, r[k]);
        }
      }
    }
  }
}

template <typename XT, typename RT, bool kCodes, int U, int NU, bool kWarp, int kMaxT = 128>
void launch(const RmsNormParams& p, int threads, int sms, cudaStream_t st) {
  const int teams = kWarp ? 4 : 1;
  const long long rows = (p.s + teams - 1) / teams, most = (long long)sms * 64;
  const size_t smem = kCodes ? size_t(teams) * 2 * p.groups * sizeof(unsigned) : 0;
  rmsnorm_forward_kernel<XT, RT, kCodes, U, NU, kWarp, kMaxT>
      <<<int(rows < most ? rows : most), kWarp ? 128 : threads, smem, st>>>(p);
}

template <typename XT, typename RT, bool kCodes> void pick(const RmsNormParams& p, bool vectors, int sms, cudaStream_t st) {
  const int h = p.h;
  if (vectors) {
    const int units = h / 8;
    if (units <= 32) return launch<XT, RT, kCodes, 8, 1, true>(p, 32, sms, st);
    if (units <= 128) return launch<XT, RT, kCodes, 8, 4, true>(p, 32, sms, st);
    const int threads = ((units + 3) / 4 + 31) / 32 * 32;
    if (threads <= 512) return launch<XT, RT, kCodes, 8, 4, false, 512>(p, threads, sms, st);
    return launch<XT, RT, kCodes, 8, 4, false, 1024>(p, threads, sms, st);
  }
  if (h <= 256) return launch<XT, RT, kCodes, 1, 8, true>(p, 32, sms, st);
  if (h <= 1024) return launch<XT, RT, kCodes, 1, 32, true>(p, 32, sms, st);
  const int threads = ((h + 31) / 32 + 31) / 32 * 32;
  if (threads <= 512) return launch<XT, RT, kCodes, 1, 32, false, 512>(p, threads, sms, st);
  launch<XT, RT, kCodes, 1, 32, false, 1024>(p, threads, sms, st);
}

template <typename XT, typename RT> void pick(const RmsNormParams& p, bool codes, bool vectors, int sms, cudaStream_t st) {
  if (codes) pick<XT, RT, true>(p, vectors, sms, st);
  else pick<XT, RT, false>(p, vectors, sms, st);
}

}  // namespace

void launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                            cudaStream_t st) {
  if (!x_bf16) pick<float, float>(p, codes, vectors, sms, st);
  else if (res_bf16) pick<__nv_bfloat16, __nv_bfloat16>(p, codes, vectors, sms, st);
  else pick<__nv_bfloat16, float>(p, codes, vectors, sms, st);
}

}  // namespace vpce
