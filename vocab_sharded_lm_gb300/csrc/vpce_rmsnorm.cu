// Root-mean-square norm with the residual's addition, its output as it is or
// as e4m3 codes with scales per group of columns: rows of 16-byte vectors.
//
// One pass: a row is read once into registers as fp32 (r = x + residual), its
// squares are summed over the row's threads, and the same registers give the
// output, so the only traffic is the operands'.  It is bound by HBM where there
// is a residual (64 KB a row at h = 8192 bf16): s = h = 8192 bf16 80 us, 6.7 TB/s
// of the copy rate's 6.8; with e4m3 output in groups of 128 74 us, 6.4 TB/s; the
// latter without a residual is bound by issue (53 us for 203 MB).  Up to 1024
// columns a warp takes a row (no barrier), up to 8192 a CTA of at most 256
// threads, three of which share an SM; above, the ring kernel.
#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

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

// Eight values as pairs (one instruction for two), their squares added to ss.
__device__ __forceinline__ void add_squares(const float (&v)[8], f32x2 (&r)[4], f32x2& ss) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = f2_pack(v[2 * j], v[2 * j + 1]);
    ss = f2_fma(r[j], r[j], ss);
  }
}

// Eight codes: quotient() of pairs.
__device__ __forceinline__ void store_quotients(unsigned char* to, const f32x2 (&r)[4], float scale, float inv) {
  const float minus = isinf(scale) ? 0.f : -scale;
  const f32x2 minus2 = f2_pack(minus, minus), inv2 = f2_pack(inv, inv);
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 q = f2_mul(r[j], inv2);
    f2_unpack(f2_fma(f2_fma(q, minus2, r[j]), inv2, q), v[2 * j], v[2 * j + 1]);
  }
  store_codes(to, v);
}

// Maxima of the 16 columns of each two lanes.
template <int NU>
__device__ __forceinline__ void segments16(const GroupWords& words, const unsigned (&m)[NU], int tid, int T, int h) {
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int c = (k * T + tid) * 8;
    const unsigned t = max(m[k], __shfl_xor_sync(kFull, m[k], 1));
    if (c < h && (tid & 1) == 0) words.tops[c / 16] = t;
  }
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
// columns a thread.  kWhole: every thread's columns are all of the row's, and
// there is no residual (1) or one (2).  Without a branch around each unit its
// loads go together: s = h = 8192 bf16 with a residual 80 us instead of 84, in
// e4m3 with groups of 128 74 instead of 80 (without a residual 53 instead of 62),
// of 48 76 instead of 95; s = 32768, h = 1024 in e4m3 41 instead of 52.
template <typename XT, typename RT, GroupKind kGroups, int NU, bool kWarp, int kMaxT, int kWhole>
__global__ void __launch_bounds__(kMaxT, kMaxT == 256 ? 3 : 1) rmsnorm_forward_kernel(const __grid_constant__ RmsNormParams p, const GroupPlan plan) {
  extern __shared__ uint4 smem[];  // [teams] GroupWords, kShared only
  __shared__ float red[2][32];
  [[maybe_unused]] __shared__ unsigned top_row[2][32];
  constexpr int U = 8;
  const auto inside = [&](int c) { return kWhole != 0 || c < p.h; };
  const bool with_res = kWhole != 0 ? kWhole == 2 : p.res != nullptr;
  const int lane = threadIdx.x & 31;
  const int team = kWarp ? int(threadIdx.x >> 5) : 0, teams = kWarp ? int(blockDim.x >> 5) : 1;
  const int tid = kWarp ? lane : int(threadIdx.x), T = kWarp ? 32 : int(blockDim.x);
  const GroupWords words(reinterpret_cast<unsigned char*>(smem) + team * plan.bytes(), plan);
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + team; row < p.s; row += (long long)gridDim.x * teams, parity ^= 1) {
    const unsigned char* xr = p.x + row * p.ld_x;
    RawUnit<XT> a[NU];
    RawUnit<RT> b[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      a[k].zero();
      if (inside(c)) a[k].load(xr, c);
    }
    if (with_res) {
      const unsigned char* rr = p.res + row * p.ld_res;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        b[k].zero();
        if (inside(c)) b[k].load(rr, c);
      }
    }
    f32x2 r[NU][4], ss = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      float v[U];
      a[k].get(v);
      if (with_res) {
        float q[U];
        b[k].get(q);
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] += q[j];
        if (inside(c)) store_unit(p.res_out + row * p.ld_res_out, c, v, RT());
      }
      add_squares(v, r[k], ss);
    }
    float s0, s1;
    f2_unpack(ss, s0, s1);
    const float rstd = rsqrtf(team_sum<kWarp>(s0 + s1, red[parity]) / float(p.h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    [[maybe_unused]] unsigned m[NU], all = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      m[k] = 0;
      if (inside(c)) {
        float w[U], v[U];
        load_weight(p.w, p.w_bf16, c, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[k][j] = f2_mul(f2_mul(r[k][j], f2_pack(rstd, rstd)), f2_pack(w[2 * j], w[2 * j + 1]));
          f2_unpack(r[k][j], v[2 * j], v[2 * j + 1]);
        }
        if constexpr (kGroups == kNoCodes) {
          store_unit(p.out + row * p.ld_out, c, v, XT());
        } else {
          m[k] = __float_as_uint(most_magnitude(v));
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
      segments16(words, m, tid, T, p.h);
      team_sync<kWarp>();
      words.join(plan, p.group, tid, T, p.scale + row * p.groups);
      team_sync<kWarp>();
    }
    if constexpr (kGroups != kNoCodes) {
      [[maybe_unused]] float row_scale = 0.f, row_inv = 0.f;
      if constexpr (kGroups == kRow) {
        row_scale = e4m3_scale(team_max<kWarp>(all, top_row[parity]));
        row_inv = __frcp_rn(row_scale);
        if (tid == 0) p.scale[row] = row_scale;
      }
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (inside(c)) {
          float scale = row_scale, inv = row_inv;
          if constexpr (kGroups == kShared) {
            const int g = group_of(p, c);
            scale = words.scales[g], inv = words.inverses[g];
          } else if constexpr (kGroups == kLanes) {
            const int g = group_of(p, c);
            scale = e4m3_scale(m[k]), inv = __frcp_rn(scale);
            if (c == g * p.group) p.scale[row * p.groups + g] = scale;
          }
          store_quotients(p.out + row * p.ld_out + c, r[k], scale, inv);
        }
      }
    }
  }
}

// The same for longer rows, which come through a ring that every thread fills
// for itself (cp.async: each reads only what it copied): kStages rows, one CTA
// of 288 to 512 threads an SM.  The weights stay in registers.
template <typename XT, typename RT, GroupKind kGroups, int NU, int kStages, int kWhole>
__global__ void __launch_bounds__(512, 1) rmsnorm_forward_ring_kernel(const __grid_constant__ RmsNormParams p, const GroupPlan plan) {
  extern __shared__ uint4 smem[];  // the ring, and GroupWords, kShared only
  constexpr int U = 8, kX = int(sizeof(XT)) / 2, kR = int(sizeof(RT)) / 2, kVecs = NU * (kX + kR);
  __shared__ float red[2][32];
  [[maybe_unused]] __shared__ unsigned top_row[2][32];
  const auto inside = [&](int c) { return kWhole != 0 || c < p.h; };
  const bool with_res = kWhole != 0 ? kWhole == 2 : p.res != nullptr;
  const int tid = int(threadIdx.x), T = int(blockDim.x);
  f32x2 w[NU][4];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int c = (k * T + tid) * U;
    float v[U] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (inside(c)) load_weight(p.w, p.w_bf16, c, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[k][j] = f2_pack(v[2 * j], v[2 * j + 1]);
  }
  const auto slot = [&](int stage, int v) {
    return reinterpret_cast<unsigned char*>(smem + (stage * kVecs + v) * 512 + tid);
  };
  const auto fetch = [&](long long row, int stage) {
    if (row < p.s) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (inside(c)) {
          const unsigned char* x = p.x + row * p.ld_x + size_t(c) * sizeof(XT);
#pragma unroll
          for (int i = 0; i < kX; ++i) copy_async<16, kX == 2>(slot(stage, k * kX + i), x + 16 * i);
          if (with_res) {
            const unsigned char* r = p.res + row * p.ld_res + size_t(c) * sizeof(RT);
#pragma unroll
            for (int i = 0; i < kR; ++i) copy_async<16, kR == 2>(slot(stage, NU * kX + k * kR + i), r + 16 * i);
          }
        }
      }
    }
    copy_commit();  // (an empty group past the end keeps the count)
  };
  const GroupWords words(smem + kStages * kVecs * 512, plan);
  const long long first = blockIdx.x, stride = gridDim.x;
#pragma unroll
  for (int i = 0; i < kStages; ++i) fetch(first + i * stride, i);
  int parity = 0, stage = 0;
  for (long long row = first; row < p.s; row += stride, parity ^= 1) {
    copy_wait<kStages - 1>();
    f32x2 r[NU][4], ss = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      RawUnit<XT> a;
      a.zero();
      if (inside(c)) a.take(slot(stage, k * kX), 512);
      float v[U];
      a.get(v);
      if (with_res) {
        RawUnit<RT> b;
        b.zero();
        if (inside(c)) b.take(slot(stage, NU * kX + k * kR), 512);
        float q[U];
        b.get(q);
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] += q[j];
        if (inside(c)) store_unit(p.res_out + row * p.ld_res_out, c, v, RT());
      }
      add_squares(v, r[k], ss);
    }
    float s0, s1;
    f2_unpack(ss, s0, s1);
    const float rstd = rsqrtf(team_sum<false>(s0 + s1, red[parity]) / float(p.h) + p.eps);
    fetch(row + kStages * stride, stage);  // (the stage's values are in registers)
    stage = stage + 1 == kStages ? 0 : stage + 1;
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    const f32x2 rstd2 = f2_pack(rstd, rstd);
    [[maybe_unused]] unsigned m[NU], all = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      float v[U];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[k][j] = f2_mul(f2_mul(r[k][j], rstd2), w[k][j]);
        f2_unpack(r[k][j], v[2 * j], v[2 * j + 1]);
      }
      if constexpr (kGroups == kNoCodes) {
        if (inside(c)) store_unit(p.out + row * p.ld_out, c, v, XT());
      } else {
        m[k] = __float_as_uint(most_magnitude(v));
        all = max(all, m[k]);
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
      segments16(words, m, tid, T, p.h);
      __syncthreads();
      words.join(plan, p.group, tid, T, p.scale + row * p.groups);
      __syncthreads();
    }
    if constexpr (kGroups != kNoCodes) {
      float scale = 0.f, inv = 0.f;
      if constexpr (kGroups == kRow) {
        scale = e4m3_scale(team_max<false>(all, top_row[parity]));
        inv = __frcp_rn(scale);
        if (tid == 0) p.scale[row] = scale;
      }
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (inside(c)) {
          if constexpr (kGroups == kLanes) {
            const int g = group_of(p, c);
            scale = e4m3_scale(m[k]), inv = __frcp_rn(scale);
            if (c == g * p.group) p.scale[row * p.groups + g] = scale;
          } else if constexpr (kGroups == kShared) {
            const int g = group_of(p, c);
            scale = words.scales[g], inv = words.inverses[g];
          }
          store_quotients(p.out + row * p.ld_out + c, r[k], scale, inv);
        }
      }
    }
  }
}

int row_grid(const RmsNormParams& p, int teams, int sms) {
  const long long rows = (p.s + teams - 1) / teams, most = (long long)sms * 64;
  return int(rows < most ? rows : most);
}

template <typename XT, typename RT, GroupKind kGroups, int NU, bool kWarp, int kMaxT = 128, int kWhole = 0>
cudaError_t launch(const RmsNormParams& p, int threads, int sms, cudaStream_t st) {
  if constexpr (kMaxT <= 256 && kWhole == 0) {
    if (p.h == NU * 8 * threads)
      return p.res != nullptr ? launch<XT, RT, kGroups, NU, kWarp, kMaxT, 2>(p, threads, sms, st)
                              : launch<XT, RT, kGroups, NU, kWarp, kMaxT, 1>(p, threads, sms, st);
  }
  constexpr int kTeams = kWarp ? 4 : 1;
  const GroupPlan plan(p, 16, 16);
  rmsnorm_forward_kernel<XT, RT, kGroups, NU, kWarp, kMaxT, kWhole>
      <<<row_grid(p, kTeams, sms), kWarp ? 128 : threads, kGroups == kShared ? kTeams * plan.bytes() : 0, st>>>(p, plan);
  return cudaGetLastError();
}

template <typename XT, typename RT, GroupKind kGroups, int kWhole = 0>
cudaError_t launch_ring(const RmsNormParams& p, int sms, cudaStream_t st) {
  constexpr int NU = 4, kVecs = NU * int(sizeof(XT) + sizeof(RT)) / 2, kStages = kMaxSmem / (kVecs * 16 * 512);
  const int T = (p.h / 8 + NU * 32 - 1) / (NU * 32) * 32;
  if constexpr (kWhole == 0) {
    if (p.h == NU * 8 * T)
      return p.res != nullptr ? launch_ring<XT, RT, kGroups, 2>(p, sms, st) : launch_ring<XT, RT, kGroups, 1>(p, sms, st);
  }
  const auto kernel = rmsnorm_forward_ring_kernel<XT, RT, kGroups, NU, kStages, kWhole>;
  const GroupPlan plan(p, 16, 16);
  // (GroupWords: three words for 16 columns, 12 KB)
  const int smem = kStages * kVecs * 16 * 512 + (kGroups == kShared ? plan.bytes() : 0);
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<int(p.s < sms ? p.s : sms), T, smem, st>>>(p, plan);
  return cudaGetLastError();
}

template <typename XT, typename RT, GroupKind kGroups>
cudaError_t pick_vectors(const RmsNormParams& p, int sms, cudaStream_t st) {
  const int units = p.h / 8;
  if (units <= 32) return launch<XT, RT, kGroups, 1, true>(p, 32, sms, st);
  if (units <= 128) return launch<XT, RT, kGroups, 4, true>(p, 32, sms, st);
  const int threads = ((units + 3) / 4 + 31) / 32 * 32;
  // (at most 85 registers a thread: three CTAs of 256 on an SM)
  if (threads <= 256) return launch<XT, RT, kGroups, 4, false, 256>(p, threads, sms, st);
  // a CTA of more has an SM for itself, and its row's loads, sum and stores would
  // follow one another: the ring keeps loads under way (s = 4096, h = 16384 bf16
  // with a residual 105 -> 90 us, without 71 -> 47, in 8 bits 121 -> 84; for
  // shorter rows three CTAs do that better: s = h = 8192 86 us against 94 when
  // neither had kWhole)
  if (threads <= 512) return launch_ring<XT, RT, kGroups>(p, sms, st);
  return launch<XT, RT, kGroups, 4, false, 1024>(p, threads, sms, st);
}

template <typename XT, typename RT>
cudaError_t pick(const RmsNormParams& p, bool codes, bool vectors, int sms, cudaStream_t st) {
  const GroupKind kind = !codes ? kNoCodes
                         : p.groups == 1 ? kRow
                         : vectors && p.group <= 256 && (p.group & (p.group - 1)) == 0 ? kLanes
                                                                                       : kShared;
  if (!vectors) return rmsnorm_forward_odd<XT, RT>(p, kind, sms, st);
  if (kind == kNoCodes) return pick_vectors<XT, RT, kNoCodes>(p, sms, st);
  if (kind == kRow) return pick_vectors<XT, RT, kRow>(p, sms, st);
  return kind == kLanes ? pick_vectors<XT, RT, kLanes>(p, sms, st) : pick_vectors<XT, RT, kShared>(p, sms, st);
}

}  // namespace

cudaError_t launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                                   cudaStream_t st) {
  if (!x_bf16) return pick<float, float>(p, codes, vectors, sms, st);
  if (res_bf16) return pick<__nv_bfloat16, __nv_bfloat16>(p, codes, vectors, sms, st);
  return pick<__nv_bfloat16, float>(p, codes, vectors, sms, st);
}

}  // namespace vpce
