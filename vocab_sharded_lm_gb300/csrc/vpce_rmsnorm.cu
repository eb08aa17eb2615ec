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
__device__ __forceinline__ void store_code(unsigned char* p, float v) { *p = (unsigned char)(e4m3x2(v, 0.f) & 0xff); }

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

// Per team, twice (the rows alternate: who still reads one row's is at most a
// barrier behind whoever writes the next row's): the groups' maxima, then their
// scales, and the reciprocals of those.
struct SharedGroups {
  unsigned* top;
  float* inverse;
  __device__ __forceinline__ SharedGroups(unsigned* sm, int team, int parity, int groups)
      : top(sm + (team * 2 + parity) * 2 * groups), inverse(reinterpret_cast<float*>(top + groups)) {}
  __device__ __forceinline__ void clear(int groups, int tid, int T) const {
    for (int g = tid; g < groups; g += T) top[g] = 0;
  }
  __device__ __forceinline__ void scales(int groups, int tid, int T, float* out) const {
    for (int g = tid; g < groups; g += T) {
      const float scale = group_scale(top[g]);
      out[g] = scale;
      top[g] = __float_as_uint(scale);
      inverse[g] = __fdiv_rn(1.f, scale);
    }
  }
};

template <bool kWarp> __device__ __forceinline__ void team_sync() {
  if constexpr (kWarp) __syncwarp();
  else __syncthreads();
}

// Largest of a team's values; every thread gets it.
template <bool kWarp> __device__ __forceinline__ unsigned team_max(unsigned v, unsigned* sm) {
  v = __reduce_max_sync(kFull, v);
  if constexpr (!kWarp) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = __reduce_max_sync(kFull, lane < warps ? sm[lane] : 0u);
  }
  return v;
}

__device__ __forceinline__ int group_of(const RmsNormParams& p, int c) { return int(__umulhi(unsigned(c), p.group_inverse)); }

// Rows of 16-byte vectors: a warp (four a CTA) or a CTA a row, NU units of eight
// columns a thread.
template <typename XT, typename RT, GroupKind kGroups, int NU, bool kWarp, int kMaxT>
__global__ void __launch_bounds__(kMaxT, kMaxT == 256 ? 3 : 1) rmsnorm_forward_kernel(const __grid_constant__ RmsNormParams p) {
  extern __shared__ unsigned group_sm[];  // [teams][2][2][groups], kShared only
  __shared__ float red[2][32];
  [[maybe_unused]] __shared__ unsigned top_row[2][32];
  constexpr int U = 8;
  const int lane = threadIdx.x & 31;
  const int team = kWarp ? int(threadIdx.x >> 5) : 0, teams = kWarp ? int(blockDim.x >> 5) : 1;
  const int tid = kWarp ? lane : int(threadIdx.x), T = kWarp ? 32 : int(blockDim.x);
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + team; row < p.s; row += (long long)gridDim.x * teams, parity ^= 1) {
    const unsigned char* xr = p.x + row * p.ld_x;
    RawUnit<XT> a[NU];
    RawUnit<RT> b[NU];
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
    const SharedGroups shared(group_sm, team, parity, p.groups);
    if constexpr (kGroups == kShared) {
      shared.clear(p.groups, tid, T);
      if constexpr (kWarp) __syncwarp();
    }
    ss = team_sum<kWarp>(ss, red[parity]);
    const float rstd = rsqrtf(ss / float(p.h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    [[maybe_unused]] unsigned m[NU], all = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      m[k] = 0;
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
          if constexpr (kGroups == kShared) atomicMax(shared.top + group_of(p, c), m[k]);  // (the order does not matter)
          all = max(all, m[k]);
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
    } else if constexpr (kGroups == kShared) {
      team_sync<kWarp>();
      shared.scales(p.groups, tid, T, p.scale + row * p.groups);
      team_sync<kWarp>();
    }
    if constexpr (kGroups != kNoCodes) {
      [[maybe_unused]] float row_scale = 0.f, row_inv = 0.f;
      if constexpr (kGroups == kRow) {
        row_scale = group_scale(team_max<kWarp>(all, top_row[parity]));
        row_inv = __fdiv_rn(1.f, row_scale);
        if (tid == 0) p.scale[row] = row_scale;
      }
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (c < p.h) {
          float scale = row_scale, inv = row_inv;
          if constexpr (kGroups == kShared) {
            const int g = group_of(p, c);
            scale = __uint_as_float(shared.top[g]), inv = shared.inverse[g];
          } else if constexpr (kGroups == kLanes) {
            const int g = group_of(p, c);
            scale = group_scale(m[k]), inv = __fdiv_rn(1.f, scale);
            if (c == g * p.group) p.scale[row * p.groups + g] = scale;
          }
#pragma unroll
          for (int j = 0; j < U; ++j) r[k][j] = quotient(r[k][j], isinf(scale) ? 0.f : scale, inv);
          store_codes(p.out + row * p.ld_out + c, r[k]);
        }
      }
    }
  }
}

// Rows off 16 bytes, element by element: kT threads a row, few of them, since
// what a row costs besides its elements (sums, addresses) is paid by every warp.
template <typename XT, typename RT, GroupKind kGroups, int kT>
__global__ void __launch_bounds__(kT == 32 ? 128 : kT, kT >= 512 ? 1 : kT == 32 ? 4 : 512 / kT)
    rmsnorm_forward_odd_kernel(const __grid_constant__ RmsNormParams p) {
  extern __shared__ unsigned group_sm[];
  __shared__ float red[2][32];
  [[maybe_unused]] __shared__ unsigned top_row[2][32];
  constexpr bool kWarp = kT == 32;
  constexpr int XB = Elem<XT>::kBytes, RB = Elem<RT>::kBytes;
  const int lane = threadIdx.x & 31, h = p.h;
  const int team = kWarp ? int(threadIdx.x >> 5) : 0, teams = kWarp ? 4 : 1;
  const int tid = kWarp ? lane : int(threadIdx.x);
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + team; row < p.s; row += (long long)gridDim.x * teams, parity ^= 1) {
    const unsigned char* const xr = p.x + row * p.ld_x;
    float r[kOddColumns], ss = 0.f;
    odd_columns<kT>(h, tid, [&](int k, int c, bool) { r[k] = Elem<XT>::load(xr + c * XB); });
    if (p.res != nullptr) {
      const unsigned char* const rr = p.res + row * p.ld_res;
      unsigned char* const to = p.res_out + row * p.ld_res_out;
      odd_columns<kT>(h, tid, [&](int k, int c, bool) { r[k] += Elem<RT>::load(rr + c * RB); });
      // (in place, column 0 is written only after every lane has read it)
      team_sync<kWarp>();
      odd_columns<kT>(h, tid, [&](int k, int c, bool inside) {
        if (inside) Elem<RT>::store(to + c * RB, r[k]);
      });
    }
    odd_columns<kT>(h, tid, [&](int k, int, bool inside) { ss = inside ? fmaf(r[k], r[k], ss) : ss; });
    const SharedGroups shared(group_sm, team, parity, p.groups);
    if constexpr (kGroups == kShared) {
      shared.clear(p.groups, tid, kT);
      if constexpr (kWarp) __syncwarp();
    }
    ss = team_sum<kWarp>(ss, red[parity]);
    const float rstd = rsqrtf(ss / float(h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    unsigned char* const out = p.out + row * p.ld_out;
    [[maybe_unused]] unsigned all = 0;
    odd_columns<kT>(h, tid, [&](int k, int c, bool inside) {
      r[k] = r[k] * rstd * load_weight(p.w, p.w_bf16, c);
      if constexpr (kGroups == kNoCodes) {
        if (inside) Elem<XT>::store(out + c * XB, r[k]);
      } else if constexpr (kGroups == kRow) {
        all = max(all, inside ? mag(r[k]) : 0u);
      } else {
        // 32 consecutive columns: of one group, or 16 and 16 of one each
        // (atomics on shared memory; their order does not matter)
        const unsigned half = p.group % 32 == 0 ? kFull : lane < 16 ? 0xffffu : 0xffff0000u;
        const unsigned t = __reduce_max_sync(half, inside ? mag(r[k]) : 0u);
        if (inside && (lane == 0 || (lane == 16 && half != kFull))) atomicMax(shared.top + group_of(p, c), t);
      }
    });
    if constexpr (kGroups == kRow) {
      const float scale = group_scale(team_max<kWarp>(all, top_row[parity])), inv = __fdiv_rn(1.f, scale);
      const float s = isinf(scale) ? 0.f : scale;
      if (tid == 0) p.scale[row] = scale;
      odd_columns<kT>(h, tid, [&](int k, int c, bool inside) {
        if (inside) store_code(out + c, quotient(r[k], s, inv));
      });
    } else if constexpr (kGroups == kShared) {
      team_sync<kWarp>();
      shared.scales(p.groups, tid, kT, p.scale + row * p.groups);
      team_sync<kWarp>();
      odd_columns<kT>(h, tid, [&](int k, int c, bool inside) {
        const int g = group_of(p, c);
        const float scale = __uint_as_float(shared.top[g]);
        if (inside) store_code(out + c, quotient(r[k], isinf(scale) ? 0.f : scale, shared.inverse[g]));
      });
    }
  }
}

template <typename P> size_t group_bytes(GroupKind kind, int teams, const P& p) {
  return kind == kShared ? size_t(teams) * 4 * p.groups * sizeof(unsigned) : 0;
}

int row_grid(const RmsNormParams& p, int teams, int sms) {
  const long long rows = (p.s + teams - 1) / teams, most = (long long)sms * 64;
  return int(rows < most ? rows : most);
}

template <typename XT, typename RT, GroupKind kGroups, int NU, bool kWarp, int kMaxT = 128>
void launch(const RmsNormParams& p, int threads, int sms, cudaStream_t st) {
  constexpr int kTeams = kWarp ? 4 : 1;
  rmsnorm_forward_kernel<XT, RT, kGroups, NU, kWarp, kMaxT>
      <<<row_grid(p, kTeams, sms), kWarp ? 128 : threads, group_bytes(kGroups, kTeams, p), st>>>(p);
}

template <typename XT, typename RT, GroupKind kGroups, int kT>
void launch_odd(const RmsNormParams& p, int sms, cudaStream_t st) {
  constexpr int kTeams = kT == 32 ? 4 : 1;
  rmsnorm_forward_odd_kernel<XT, RT, kGroups, kT>
      <<<row_grid(p, kTeams, sms), kT == 32 ? 128 : kT, group_bytes(kGroups, kTeams, p), st>>>(p);
}

template <typename XT, typename RT, GroupKind kGroups>
void pick(const RmsNormParams& p, bool vectors, int sms, cudaStream_t st) {
  const int h = p.h;
  if (vectors) {
    const int units = h / 8;
    if (units <= 32) return launch<XT, RT, kGroups, 1, true>(p, 32, sms, st);
    if (units <= 128) return launch<XT, RT, kGroups, 4, true>(p, 32, sms, st);
    const int threads = ((units + 3) / 4 + 31) / 32 * 32;
    // (at most 85 registers a thread: three CTAs of 256 on an SM)
    if (threads <= 256) return launch<XT, RT, kGroups, 4, false, 256>(p, threads, sms, st);
    if (threads <= 512) return launch<XT, RT, kGroups, 4, false, 512>(p, threads, sms, st);
    return launch<XT, RT, kGroups, 4, false, 1024>(p, threads, sms, st);
  }
  if constexpr (kGroups != kLanes) {
    if (h <= 1024) return launch_odd<XT, RT, kGroups, 32>(p, sms, st);
    if (h <= 2048) return launch_odd<XT, RT, kGroups, 64>(p, sms, st);
    if (h <= 4096) return launch_odd<XT, RT, kGroups, 128>(p, sms, st);
    if (h <= 8192) return launch_odd<XT, RT, kGroups, 256>(p, sms, st);
    if (h <= 16384) return launch_odd<XT, RT, kGroups, 512>(p, sms, st);
    launch_odd<XT, RT, kGroups, 1024>(p, sms, st);
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
