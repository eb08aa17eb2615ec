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

// y / s correctly rounded, for inv = 1 / s (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990: one
// residual step); where s is infinite, y inv.
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  const float q = __fmul_rn(y, inv);
  return __fmaf_rn(__fmaf_rn(-q, s, y), inv, q);
}

__device__ __forceinline__ float group_scale(unsigned top) {
  const float s = __fmul_rn(__uint_as_float(top), 1.f / 448.f);
  return s < kTiny ? kTiny : s;  // a NaN stays
}

// Where a group's largest magnitude is found: in the lanes of a warp that hold
// the group (16, 32, .. 256 columns in vectors), by the whole team (one group a
// row), or through shared memory.
enum GroupKind { kNoCodes, kLanes, kRow, kShared };

// kT: threads of a team, known when compiled (single elements: their addresses
// are then one register and constants), or 0.
template <typename XT, typename RT, GroupKind kGroups, int U, int NU, bool kWarp, int kMaxT, int kT>
__global__ void __launch_bounds__(kMaxT, U == 1 ? (kMaxT < 512 ? 512 / kMaxT : 1) : kMaxT == 256 ? 3 : 1) rmsnorm_forward_kernel(const __grid_constant__ RmsNormParams p) {
  extern __shared__ unsigned top_sm[];  // [teams][2][2][groups], kShared only
  __shared__ float red[2][32];
  [[maybe_unused]] __shared__ unsigned top_row[2][32];
  const int lane = threadIdx.x & 31;
  const int team = kWarp ? int(threadIdx.x >> 5) : 0, teams = kWarp ? int(blockDim.x >> 5) : 1;
  const int tid = kWarp ? lane : int(threadIdx.x), T = kT > 0 ? kT : int(blockDim.x);
  // (elements past the row are skipped by all of a team's threads)
  const auto past = [&](int k) { return U == 1 && k * T >= p.h; };
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + team; row < p.s; row += (long long)gridDim.x * teams) {
    const unsigned char* xr = p.x + row * p.ld_x;
    RawUnit<XT, U> a[NU];
    RawUnit<RT, U> b[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      if (past(k)) break;
      const int c = (k * T + tid) * U;
      a[k].zero();
      if (c < p.h) a[k].load(xr, c);
    }
    if (p.res != nullptr) {
      const unsigned char* rr = p.res + row * p.ld_res;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (past(k)) break;
        const int c = (k * T + tid) * U;
        b[k].zero();
        if (c < p.h) b[k].load(rr, c);
      }
    }
    float r[NU][U], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      if (past(k)) break;
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
    [[maybe_unused]] unsigned* top = nullptr;
    [[maybe_unused]] float* inverse = nullptr;
    if constexpr (kGroups == kShared) {
      top = top_sm + (team * 2 + parity) * 2 * p.groups;
      inverse = reinterpret_cast<float*>(top + p.groups);
      for (int g = tid; g < p.groups; g += T) top[g] = 0;
      if constexpr (kWarp) __syncwarp();
    }
    ss = team_sum<kWarp>(ss, red[parity]);
    const float rstd = rsqrtf(ss / float(p.h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    [[maybe_unused]] unsigned m[NU], all = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      if (past(k)) break;
      const int c = (k * T + tid) * U;
      m[k] = 0;
      const int group = kGroups == kShared || kGroups == kLanes ? int(__umulhi(unsigned(c), p.group_inverse)) : 0;
      if (c < p.h) {
        float w[U];
        load_weight(p.w, p.w_bf16, c, w);
#pragma unroll
        for (int j = 0; j < U; ++j) r[k][j] = r[k][j] * rstd * w[j];
        if constexpr (kGroups == kNoCodes) {
          store_unit(p.out + row * p.ld_out, c, r[k], XT());
        } else {
#pragma unroll
          for (int j = 0; j < U; ++j) m[k] = max(m[k], mag(r[k][j]));
          if constexpr (kGroups == kRow) all = max(all, m[k]);
        }
      }
      if constexpr (kGroups == kShared) {
        // (atomics on shared memory; their order does not matter)
        if (U == 1) {
          // 32 consecutive columns: of one group, or 16 and 16 of one each
          const unsigned half = p.group % 32 == 0 ? kFull : lane < 16 ? 0xffffu : 0xffff0000u;
          const unsigned t = __reduce_max_sync(half, m[k]);
          if ((lane == 0 || (lane == 16 && half != kFull)) && c < p.h) atomicMax(top + group, t);
        } else if (c < p.h) {
          atomicMax(top + group, m[k]);
        }
      }
    }
    if constexpr (kGroups == kLanes) {
      const int lanes = p.group / U;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (o < lanes) {
#pragma unroll
          for (int k = 0; k < NU; ++k) m[k] = max(m[k], __shfl_xor_sync(kFull, m[k], o));
        }
      }
    } else if constexpr (kGroups == kRow) {
      all = __reduce_max_sync(kFull, all);
      if constexpr (!kWarp) {
        const int warps = T >> 5;
        if (lane == 0) top_row[parity][threadIdx.x >> 5] = all;
        __syncthreads();
        all = __reduce_max_sync(kFull, lane < warps ? top_row[parity][lane] : 0u);
      }
    } else if constexpr (kGroups == kShared) {
      // each group's scale and its reciprocal, in the maximum's place
      if constexpr (kWarp) __syncwarp();
      else __syncthreads();
      for (int g = tid; g < p.groups; g += T) {
        const float scale = group_scale(top[g]);
        p.scale[row * p.groups + g] = scale;
        top[g] = __float_as_uint(scale);
        inverse[g] = __fdiv_rn(1.f, scale);
      }
      if constexpr (kWarp) __syncwarp();
      else __syncthreads();
    }
    if constexpr (kGroups != kNoCodes) {
      [[maybe_unused]] float row_scale = 0.f, row_inv = 0.f;
      if constexpr (kGroups == kRow) {
        row_scale = group_scale(all);
        row_inv = __fdiv_rn(1.f, row_scale);
        if (tid == 0) p.scale[row] = row_scale;
      }
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (past(k)) break;
        const int c = (k * T + tid) * U;
        if (c < p.h) {
          float scale, inv;
          if constexpr (kGroups == kRow) {
            scale = row_scale, inv = row_inv;
          } else {
            const int g = int(__umulhi(unsigned(c), p.group_inverse));
            if constexpr (kGroups == kShared) {
              scale = __uint_as_float(top[g]), inv = inverse[g];
            } else {
              scale = group_scale(m[k]), inv = __fdiv_rn(1.f, scale);
              if (c == g * p.group) p.scale[row * p.groups + g] = scale;
            }
          }
#pragma unroll
          for (int j = 0; j < U; ++j) r[k][j] = quotient(r[k][j], isinf(scale) ? 0.f : scale, inv);
          store_codes(p.out + row * p.ld_out + c, r[k]);
        }
      }
    }
    parity ^= 1;
  }
}

template <typename XT, typename RT, GroupKind kGroups, int U, int NU, bool kWarp, int kMaxT = 128, int kT = kWarp ? 32 : 0>
void launch(const RmsNormParams& p, int threads, int sms, cudaStream_t st) {
  const int teams = kWarp ? 4 : 1;
  const long long rows = (p.s + teams - 1) / teams, most = (long long)sms * 64;
  const size_t smem = kGroups == kShared ? size_t(teams) * 4 * p.groups * sizeof(unsigned) : 0;
  rmsnorm_forward_kernel<XT, RT, kGroups, U, NU, kWarp, kMaxT, kT>
      <<<int(rows < most ? rows : most), kWarp ? 128 : threads, smem, st>>>(p);
}

template <typename XT, typename RT, GroupKind kGroups>
void pick(const RmsNormParams& p, bool vectors, int sms, cudaStream_t st) {
  const int h = p.h;
  if (vectors) {
    const int units = h / 8;
    if (units <= 32) return launch<XT, RT, kGroups, 8, 1, true>(p, 32, sms, st);
    if (units <= 128) return launch<XT, RT, kGroups, 8, 4, true>(p, 32, sms, st);
    const int threads = ((units + 3) / 4 + 31) / 32 * 32;
    // (at most 85 registers a thread: three CTAs of 256 on an SM)
    if (threads <= 256) return launch<XT, RT, kGroups, 8, 4, false, 256>(p, threads, sms, st);
    if (threads <= 512) return launch<XT, RT, kGroups, 8, 4, false, 512>(p, threads, sms, st);
    return launch<XT, RT, kGroups, 8, 4, false, 1024>(p, threads, sms, st);
  }
  if constexpr (kGroups != kLanes) {
    // few warps a row: what a row costs besides its elements (sums, addresses)
    // is paid by every one of them
    if (h <= 1024) return launch<XT, RT, kGroups, 1, 32, true>(p, 32, sms, st);
    if (h <= 2048) return launch<XT, RT, kGroups, 1, 32, false, 64, 64>(p, 64, sms, st);
    if (h <= 4096) return launch<XT, RT, kGroups, 1, 32, false, 128, 128>(p, 128, sms, st);
    if (h <= 8192) return launch<XT, RT, kGroups, 1, 32, false, 256, 256>(p, 256, sms, st);
    if (h <= 16384) return launch<XT, RT, kGroups, 1, 32, false, 512, 512>(p, 512, sms, st);
    launch<XT, RT, kGroups, 1, 32, false, 1024, 1024>(p, 1024, sms, st);
  }
}

template <typename XT, typename RT>
void pick(const RmsNormParams& p, bool codes, bool vectors, int sms, cudaStream_t st) {
  const bool lanes = p.group <= 256 && (p.group & (p.group - 1)) == 0;
  if (!codes) pick<XT, RT, kNoCodes>(p, vectors, sms, st);
  else if (p.groups == 1) pick<XT, RT, kRow>(p, vectors, sms, st);
  else if (vectors && lanes) pick<XT, RT, kLanes>(p, vectors, sms, st);
  else pick<XT, RT, kShared>(p, vectors, sms, st);
}

}  // namespace

void launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                            cudaStream_t st) {
  if (!x_bf16) pick<float, float>(p, codes, vectors, sms, st);
  else if (res_bf16) pick<__nv_bfloat16, __nv_bfloat16>(p, codes, vectors, sms, st);
  else pick<__nv_bfloat16, float>(p, codes, vectors, sms, st);
}

}  // namespace vpce
