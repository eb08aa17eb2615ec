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

// Sum over a team: one warp, or the CTA's warps through `red` (32 floats).
// The order is fixed, and every thread gets the same bits.
template <bool kWarp> __device__ __forceinline__ float team_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if constexpr (!kWarp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  }
  return v;
}

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

template <typename XT, typename RT, GroupKind kGroups>
void pick_vectors(const RmsNormParams& p, int sms, cudaStream_t st) {
  const int units = p.h / 8;
  if (units <= 32) return launch<XT, RT, kGroups, 1, true>(p, 32, sms, st);
  if (units <= 128) return launch<XT, RT, kGroups, 4, true>(p, 32, sms, st);
  const int threads = ((units + 3) / 4 + 31) / 32 * 32;
  // (at most 85 registers a thread: three CTAs of 256 on an SM)
  if (threads <= 256) return launch<XT, RT, kGroups, 4, false, 256>(p, threads, sms, st);
  if (threads <= 512) return launch<XT, RT, kGroups, 4, false, 512>(p, threads, sms, st);
  launch<XT, RT, kGroups, 4, false, 1024>(p, threads, sms, st);
}

template <typename XT, typename RT>
void pick(const RmsNormParams& p, bool codes, bool vectors, int sms, cudaStream_t st) {
  const GroupKind kind = !codes ? kNoCodes
                         : p.groups == 1 ? kRow
                         : vectors && p.group <= 256 && (p.group & (p.group - 1)) == 0 ? kLanes
                                                                                       : kShared;
  if (vectors) {
    if (kind == kNoCodes) pick_vectors<XT, RT, kNoCodes>(p, sms, st);
    else if (kind == kRow) pick_vectors<XT, RT, kRow>(p, sms, st);
    else if (kind == kLanes) pick_vectors<XT, RT, kLanes>(p, sms, st);
    else pick_vectors<XT, RT, kShared>(p, sms, st);
  } else {
    rmsnorm_forward_odd<XT, RT>(p, kind, sms, st);
  }
}

}  // namespace

cudaError_t set_rmsnorm_forward_smem() {
  cudaError_t e = set_rmsnorm_odd_smem<float, float>();
  if (e == cudaSuccess) e = set_rmsnorm_odd_smem<__nv_bfloat16, __nv_bfloat16>();
  return e == cudaSuccess ? set_rmsnorm_odd_smem<__nv_bfloat16, float>() : e;
}

void launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                            cudaStream_t st) {
  if (!x_bf16) pick<float, float>(p, codes, vectors, sms, st);
  else if (res_bf16) pick<__nv_bfloat16, __nv_bfloat16>(p, codes, vectors, sms, st);
  else pick<__nv_bfloat16, float>(p, codes, vectors, sms, st);
}

}  // namespace vpce
