// Gradient of the root-mean-square norm: with n = r rstd,
//     dr = dresidual + rstd (w dy - n mean(w dy n)),    dw = sum over rows dy n.
//
// One pass over dy, r and dresidual.  A thread keeps the same columns on every
// row that its team takes, so dw's terms add up in its registers; each CTA then
// leaves one partial row, and a second kernel adds those in a fixed order.
//
// The row's mean is a barrier in every row, so what keeps HBM busy is what a
// team has asked for ahead: rows in vectors come through a ring of shared
// memory that every thread fills for itself (cp.async: each reads only what it
// copied, so no barrier goes with it), a few rows deep; rows off 16 bytes through
// one that its team fills.
//
// s = h = 8192 bf16 with dresidual: 88 us, 6.1 TB/s over dy, r, dresidual and dr
// (one team of 512 threads an SM: its barrier and the two passes around it are
// not hidden by another row's; s = 16384, h = 4096 with two teams 84 us).
// s = 30001, h = 515 fp32: 40 us, 4.7 TB/s, about 2 us of it the second kernel.
#include <type_traits>

#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

constexpr int kColumns = 32, kRowLanes = 32;  // of the kernel that adds the partial rows

// Where a team puts its sums of the weight's gradient: the CTA's partial row,
// or a row of shared memory where the CTA has several teams (all its threads
// call this, and then join_sums).
__device__ __forceinline__ float* own_sums(const RmsNormBwdParams& p, uint4* smem, int teams, int team) {
  if (teams == 1) return p.part + (long long)blockIdx.x * p.h;
  __syncthreads();
  return reinterpret_cast<float*>(smem) + team * p.h;
}
__device__ __forceinline__ void join_sums(const RmsNormBwdParams& p, const uint4* smem, int teams) {
  if (teams == 1) return;
  __syncthreads();
  const float* sums = reinterpret_cast<const float*>(smem);
  float* part = p.part + (long long)blockIdx.x * p.h;
  for (int c = threadIdx.x; c < p.h; c += blockDim.x) {
    float v = sums[c];
    for (int i = 1; i < teams; ++i) v += sums[i * p.h + c];
    part[c] = v;
  }
}

// Rows of 16-byte vectors.  NU units of eight columns a thread; kStages: rows
// of the ring ahead (0: none, rows are loaded when they are due).  kKeep:
// products of a row's values stay in registers until its mean is known, and the
// weights for all rows; else (32 columns a thread) they are read a second time,
// from the ring or through L1.  kWhole: every thread's columns are all of the
// row's, and there is no dresidual (1) or one (2): without a branch around each
// unit and operand s = h = 8192 bf16 takes 88 us instead of 91, without dresidual
// 73 instead of 78, s = 8192, h = 4096 fp32 115 instead of 138.  (32 columns a
// thread would spill: s = 4096, h = 16384 bf16 111 us instead of 97.)
template <typename T> constexpr int kParts = int(sizeof(T)) / 2;  // vectors of a unit

template <typename GT, typename RT, int NU, int kStages, int kMaxT, bool kKeep, int kWhole>
__global__ void __launch_bounds__(kMaxT, 1) rmsnorm_backward_kernel(const __grid_constant__ RmsNormBwdParams p,
                                                                    int team_threads) {
  constexpr int U = 8;
  extern __shared__ uint4 smem[];  // the ring, and at the end sums [teams][h]
  __shared__ float red[kMaxT / 32][2][32];
  constexpr bool kRing = kStages > 0;
  const int T = team_threads;
  const auto inside = [&](int c) { return kWhole != 0 || c < p.h; };
  const bool with_dres = kWhole != 0 ? kWhole == 2 : p.dres != nullptr;
  // (a constant where an SM's shared memory is the ring's anyway)
  const int pitch = kMaxT == 512 ? kMaxT : int(blockDim.x);
  Team team;
  const int teams = blockDim.x / T;
  team.id = threadIdx.x / T;
  team.tid = threadIdx.x - team.id * T;
  team.threads = T;
  team.red = &red[team.id][0][0];
  const int tid = team.tid;
  // (pairs of fp32 values: one instruction for two)
  f32x2 acc[NU][4], w[kKeep ? NU : 1][4];
  const auto pairs = [](const float (&v)[U], f32x2 (&q)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f2_pack(v[2 * j], v[2 * j + 1]);
  };
  // bf16 weights are held as they are where fp32 pairs have no room (read through
  // L1, which the ring leaves too small for a row of them, s = 4096, h = 16384
  // bf16 took 140 us against 97)
  constexpr bool kHold16 = !kKeep && kMaxT == 512;
  [[maybe_unused]] uint4 w16[kHold16 ? NU : 1];
  const auto load_w = [&](int k, int c, f32x2 (&q)[4]) {
    float v[U] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (kHold16 && p.w_bf16) unpack(w16[kHold16 ? k : 0], v, __nv_bfloat16());
    else if (inside(c)) load_weight(p.w, p.w_bf16, c, v);
    pairs(v, q);
  };
#pragma unroll
  for (int k = 0; k < NU; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[k][j] = 0;
    const int c = (k * T + tid) * U;
    if constexpr (kKeep) {
      load_w(k, c, w[k]);
    } else if constexpr (kHold16) {
      w16[k] = make_uint4(0, 0, 0, 0);
      if (p.w_bf16 && inside(c)) w16[k] = __ldg(reinterpret_cast<const uint4*>(p.w + size_t(c) * 2));
    }
  }

  // ring slot of part v of a stage: this thread's own bytes
  constexpr int kG = kParts<GT>, kR = kParts<RT>, kVecs = NU * (kG + 2 * kR), kSlot = 16;
  const auto slot = [&](int stage, int v) {
    return reinterpret_cast<unsigned char*>(smem) + ((stage * kVecs + v) * pitch + int(threadIdx.x)) * kSlot;
  };
  // (the two vectors of eight fp32 values share sectors with each other: those go through L1)
  const auto copy = [&](int stage, int v, const unsigned char* src, auto fp32) {
    if constexpr (fp32) copy_async<16, true>(slot(stage, v), src);
    else copy_async<16>(slot(stage, v), src);
  };
  constexpr std::bool_constant<sizeof(GT) == 4> g32{};
  constexpr std::bool_constant<sizeof(RT) == 4> r32{};
  const auto fetch = [&](long long row, int stage) {
    if (row < p.s) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        if (inside(c)) {
          const unsigned char *g = p.dy + row * p.ld_dy + size_t(c) * sizeof(GT),
                              *x = p.x + row * p.ld_x + size_t(c) * sizeof(RT);
#pragma unroll
          for (int i = 0; i < kG; ++i) copy(stage, k * kG + i, g + 16 * i, g32);
#pragma unroll
          for (int i = 0; i < kR; ++i) copy(stage, NU * kG + k * kR + i, x + 16 * i, r32);
          if (with_dres) {
            const unsigned char* d = p.dres + row * p.ld_dres + size_t(c) * sizeof(RT);
#pragma unroll
            for (int i = 0; i < kR; ++i) copy(stage, NU * (kG + kR) + k * kR + i, d + 16 * i, r32);
          }
        }
      }
    }
    copy_commit();  // (an empty group past the end keeps the count)
  };

  const long long first = (long long)blockIdx.x * teams + team.id, stride = (long long)gridDim.x * teams;
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(first + i * stride, i);
  }
  int parity = 0, stage = 0;
  float next_rstd = first < p.s ? __ldg(p.rstd + first) : 0.f;
  for (long long row = first; row < p.s; row += stride) {
    const float rstd = next_rstd;
    if (row + stride < p.s) next_rstd = __ldg(p.rstd + row + stride);
    const auto load_g = [&](RawUnit<GT>& g, int k, int c) {
      if constexpr (kRing) g.take(slot(stage, k * kG), pitch);
      else g.load(p.dy + row * p.ld_dy, c);
    };
    const auto load_x = [&](RawUnit<RT>& x, int k, int c) {
      if constexpr (kRing) x.take(slot(stage, NU * kG + k * kR), pitch);
      else x.load(p.x + row * p.ld_x, c);
    };
    const auto load_d = [&](RawUnit<RT>& d, int k, int c) {
      if constexpr (kRing) d.take(slot(stage, NU * (kG + kR) + k * kR), pitch);
      else d.load(p.dres + row * p.ld_dres, c);
    };
    // dy, t = w dy and n = r rstd of a unit
    const f32x2 rstd2 = f2_pack(rstd, rstd);
    const auto terms = [&](int k, int c, const RawUnit<GT>& g, const RawUnit<RT>& x, f32x2 (&dy)[4], f32x2 (&t)[4],
                           f32x2 (&n)[4]) {
      if constexpr (!kKeep) load_w(k, c, w[0]);
      float v[U];
      g.get(v);
      pairs(v, dy);
      x.get(v);
      pairs(v, n);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[j] = f2_mul(n[j], rstd2);
        t[j] = f2_mul(w[kKeep ? k : 0][j], dy[j]);
      }
    };
    if constexpr (kRing) copy_wait<(kRing ? kStages - 1 : 0)>();
    constexpr int kKept = kKeep ? NU : 1;
    RawUnit<GT> g[kKept];
    RawUnit<RT> x[kKept], d[kKept];
    f32x2 t[kKept][4], n[kKept][4];
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int c = (k * T + tid) * U;
        d[k].zero();
        if (inside(c)) {
          load_g(g[k], k, c);
          load_x(x[k], k, c);
          if (with_dres) load_d(d[k], k, c);
        }
      }
    }
    f32x2 dot2 = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U, at = kKeep ? k : 0;
      if (inside(c)) {
        if constexpr (!kKeep) {
          load_g(g[0], k, c);
          load_x(x[0], k, c);
        }
        f32x2 dy[4];
        terms(k, c, g[at], x[at], dy, t[at], n[at]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[k][j] = f2_fma(dy[j], n[at][j], acc[k][j]);
          dot2 = f2_fma(t[at][j], n[at][j], dot2);
        }
      }
    }
    float d0, d1;
    f2_unpack(dot2, d0, d1);
    const float minus_dot = -team.sum(d0 + d1, parity) / float(p.h);
    const f32x2 minus_dot2 = f2_pack(minus_dot, minus_dot);
    parity ^= 1;
    if constexpr (kRing && kKeep) fetch(row + kStages * stride, stage);  // (the stage's values are in registers)
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U, at = kKeep ? k : 0;
      if (inside(c)) {
        if constexpr (!kKeep) {
          f32x2 dy[4];
          load_g(g[0], k, c);
          load_x(x[0], k, c);
          d[0].zero();
          if (with_dres) load_d(d[0], k, c);
          terms(k, c, g[0], x[0], dy, t[0], n[0]);
        }
        float o[U];
        d[at].get(o);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f2_unpack(f2_fma(rstd2, f2_fma(n[at][j], minus_dot2, t[at][j]), f2_pack(o[2 * j], o[2 * j + 1])), o[2 * j],
                    o[2 * j + 1]);
        store_unit(p.dx + row * p.ld_dx, c, o, RT());
      }
    }
    if constexpr (kRing) {
      if constexpr (!kKeep) fetch(row + kStages * stride, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  }
  grid_launch_dependents();
  if constexpr (kRing) copy_wait<0>();  // (what was copied past the last row is nothing)
  float* const mine = own_sums(p, smem, teams, team.id);
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int c = (k * T + tid) * U;
    if (inside(c)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_unpack(acc[k][j], mine[c + 2 * j], mine[c + 2 * j + 1]);
    }
  }
  join_sums(p, smem, teams);
}

// Rows off 16 bytes: dy, r and dresidual through an OddRing.  kStages: rows of
// it (0: none, rows are loaded when they are due).
template <typename GT, typename RT, int kT, int kStages>
__global__ void __launch_bounds__(kT > 512 ? kT : 512, 1) rmsnorm_backward_odd_kernel(const __grid_constant__ RmsNormBwdParams p,
                                                                                     const OddRing ring) {
  extern __shared__ uint4 smem[];  // the rings [teams][kStages], and at the end sums [teams][h]
  constexpr int kMaxTeams = kT > 512 ? 1 : 512 / kT, GB = Elem<GT>::kBytes, RB = Elem<RT>::kBytes;
  constexpr bool kRing = kStages > 0;
  __shared__ float red[kMaxTeams][2][32];
  Team team;
  const int teams = blockDim.x / kT;
  team.id = threadIdx.x / kT;
  team.tid = threadIdx.x % kT;
  team.threads = kT;
  team.red = &red[team.id][0][0];
  const int tid = team.tid, h = p.h;
  const OddColumns<kT> columns(h, tid);
  constexpr bool kHoldWeights = kT <= 512;  // (64 registers a thread otherwise)
  float acc[kOddColumns], weight[kHoldWeights ? kOddColumns : 1];
#pragma unroll
  for (int k = 0; k < kOddColumns; ++k) acc[k] = 0.f;
  if constexpr (kHoldWeights)
    columns.each([&](int k, int c, bool) { weight[k] = load_weight(p.w, p.w_bf16, c); });
  const auto weight_of = [&](int k, int c) { return kHoldWeights ? weight[kHoldWeights ? k : 0] : load_weight(p.w, p.w_bf16, c); };

  const int stage_bytes = ring.bytes(p.dres != nullptr ? 2 : 1);
  unsigned char* const mine = reinterpret_cast<unsigned char*>(smem) + team.id * kStages * stage_bytes;
  const auto fetch = [&](long long row, int stage) {
    if (row < p.s) {
      unsigned char* const dst = mine + stage * stage_bytes;
      copy_odd_row<GB, kT>(dst, p.dy, row, p.ld_dy, h, tid);
      copy_odd_row<RB, kT>(dst + ring.first, p.x, row, p.ld_x, h, tid);
      if (p.dres != nullptr) copy_odd_row<RB, kT>(dst + ring.first + ring.other, p.dres, row, p.ld_dres, h, tid);
    }
    copy_commit();  // (an empty group past the end keeps the count)
  };

  const long long first = (long long)blockIdx.x * teams + team.id, stride = (long long)gridDim.x * teams;
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) fetch(first + i * stride, i);
  }
  int parity = 0, stage = 0;
  float next_rstd = first < p.s ? __ldg(p.rstd + first) : 0.f;
  for (long long row = first; row < p.s; row += stride) {
    const float rstd = next_rstd;
    if (row + stride < p.s) next_rstd = __ldg(p.rstd + row + stride);
    const unsigned char *gr = p.dy + row * p.ld_dy, *xr = p.x + row * p.ld_x,
                        *dr = p.dres != nullptr ? p.dres + row * p.ld_dres : nullptr;
    if constexpr (kRing) {
      // this row's copies are in, everybody's; and everybody is done with the
      // stage of the row before, which is filled next
      copy_wait<(kRing ? kStages - 2 : 0)>();
      team.sync();
      fetch(row + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
      unsigned char* const at = mine + stage * stage_bytes;
      gr = at + (uintptr_t(gr) & 15);
      xr = at + ring.first + (uintptr_t(xr) & 15);
      if (dr != nullptr) dr = at + ring.first + ring.other + (uintptr_t(dr) & 15);
    }
    float dot = 0.f;
    columns.each([&](int k, int c, bool inside) {
      const float dy = inside ? Elem<GT>::load(gr + c * GB) : 0.f, n = Elem<RT>::load(xr + c * RB) * rstd;
      acc[k] = fmaf(dy, n, acc[k]);
      dot = inside ? fmaf(weight_of(k, c) * dy, n, dot) : dot;
    });
    dot = team.sum(dot, parity) / float(h);
    parity ^= 1;
    unsigned char* const out = p.dx + row * p.ld_dx;
    const auto second = [&](auto d_of) {
      columns.each([&](int k, int c, bool inside) {
        if (inside) {
          const float dy = Elem<GT>::load(gr + c * GB), n = Elem<RT>::load(xr + c * RB) * rstd;
          Elem<RT>::store(out + c * RB, fmaf(rstd, fmaf(-n, dot, weight_of(k, c) * dy), d_of(c)));
        }
      });
    };
    if (dr != nullptr) second([&](int c) { return Elem<RT>::load(dr + c * RB); });
    else second([](int) { return 0.f; });
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  grid_launch_dependents();
  if constexpr (kRing) copy_wait<0>();
  float* const sums = own_sums(p, smem, teams, team.id);
  columns.each([&](int k, int c, bool inside) {
    if (inside) sums[c] = acc[k];
  });
  join_sums(p, smem, teams);
}

// dw[c] (+)= sum over the partial rows, in a fixed order: kRowLanes threads
// take every kRowLanes-th row, then a warp adds their sums by a tree.
__global__ void __launch_bounds__(kColumns * kRowLanes) rmsnorm_weight_kernel(const float* part, int parts, int h,
                                                                            float* dw, int accumulate) {
  __shared__ float sm[kRowLanes][kColumns + 1];
  grid_dependency_wait();
  const int x = threadIdx.x % kColumns, y = threadIdx.x / kColumns, c = blockIdx.x * kColumns + x;
  float v = 0.f;
  if (c < h) {
    // (all of a thread's loads go together)
    float t[kRmsMaxParts / kRowLanes];
#pragma unroll
    for (int k = 0; k < kRmsMaxParts / kRowLanes; ++k) {
      const int i = k * kRowLanes + y;
      t[k] = i < parts ? __ldcg(part + (long long)i * h + c) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kRmsMaxParts / kRowLanes; ++k) v += t[k];
  }
  sm[y][x] = v;
  __syncthreads();
  // warp y holds column y
  v = sm[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  const int col = blockIdx.x * kColumns + y;
  if (x == 0 && col < h) dw[col] = accumulate ? dw[col] + v : v;
}

template <typename GT, typename RT, int NU, int kStages, int kMaxT, bool kKeep, int kWhole = 0>
cudaError_t launch(const RmsNormBwdParams& p, int team_threads, int sms, cudaStream_t st, int* parts) {
  if constexpr (kKeep && NU > 1 && kWhole == 0) {
    if (p.h == NU * 8 * team_threads)
      return p.dres != nullptr ? launch<GT, RT, NU, kStages, kMaxT, kKeep, 2>(p, team_threads, sms, st, parts)
                               : launch<GT, RT, NU, kStages, kMaxT, kKeep, 1>(p, team_threads, sms, st, parts);
  }
  const auto kernel = rmsnorm_backward_kernel<GT, RT, NU, kStages, kMaxT, kKeep, kWhole>;
  const int teams = team_threads < kMaxT ? kMaxT / team_threads : 1, threads = team_threads * teams;
  constexpr size_t kStageBytes = size_t(NU) * (kParts<GT> + 2 * kParts<RT>)*16;  // of a thread
  static_assert(kStages * kStageBytes * kMaxT <= kMaxSmem && NU * 8 * 4 * kMaxT <= kMaxSmem, "fits an SM");
  size_t smem = kStages * kStageBytes * (kMaxT == 512 ? kMaxT : threads);
  const size_t sums = teams > 1 ? size_t(teams) * p.h * sizeof(float) : 0;
  if (sums > smem) smem = sums;
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const long long rows = (p.s + teams - 1) / teams;
  const int most = sms < kRmsMaxParts ? sms : kRmsMaxParts;
  *parts = int(rows < most ? rows : most);
  kernel<<<*parts, threads, smem, st>>>(p, team_threads);
  return cudaGetLastError();
}

template <typename GT, typename RT, int kT, int kStages>
cudaError_t launch_odd(const RmsNormBwdParams& p, const OddRing& ring, int teams, int sms, cudaStream_t st, int* parts) {
  const auto kernel = rmsnorm_backward_odd_kernel<GT, RT, kT, kStages>;
  size_t smem = size_t(teams) * kStages * ring.bytes(p.dres != nullptr ? 2 : 1);
  const size_t sums = teams > 1 ? size_t(teams) * p.h * sizeof(float) : 0;
  if (sums > smem) smem = sums;
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const long long rows = (p.s + teams - 1) / teams;
  const int most = sms < kRmsMaxParts ? sms : kRmsMaxParts;
  *parts = int(rows < most ? rows : most);
  kernel<<<*parts, kT * teams, smem, st>>>(p, ring);
  return cudaGetLastError();
}

template <typename GT, typename RT, int kT>
cudaError_t pick_odd(const RmsNormBwdParams& p, int sms, cudaStream_t st, int* parts) {
  const OddRing ring(p.h, sizeof(GT), sizeof(RT));
  const OddPlan plan(ring.bytes(p.dres != nullptr ? 2 : 1), 0, kT);
  if constexpr (kT <= 512)
    if (plan.stages == 3) return launch_odd<GT, RT, kT, 3>(p, ring, plan.teams, sms, st, parts);
  if constexpr (kT >= 512)  // (shorter rows always have a ring)
    if (plan.stages == 0) return launch_odd<GT, RT, kT, 0>(p, ring, plan.teams, sms, st, parts);
  return launch_odd<GT, RT, kT, 2>(p, ring, plan.teams, sms, st, parts);
}

template <typename GT, typename RT>
cudaError_t pick(const RmsNormBwdParams& p, bool vectors, int sms, cudaStream_t st, int* parts) {
  const int h = p.h;
  if (vectors) {
    constexpr bool kSmall = sizeof(GT) + 2 * sizeof(RT) <= 6;  // a ring of bf16 rows holds twice as many
    const auto whole_warps = [](int n) { return (n + 31) / 32 * 32; };
    const int units = h / 8;
    if (units <= 32) return launch<GT, RT, 1, kSmall ? 8 : 4, 512, true>(p, 32, sms, st, parts);
    if (units <= 1024)
      return launch<GT, RT, 2, kSmall ? 4 : 2, 512, true>(p, whole_warps((units + 1) / 2), sms, st, parts);
    if (units <= 2048)
      return launch<GT, RT, 4, kSmall ? 2 : 1, 512, false>(p, whole_warps((units + 3) / 4), sms, st, parts);
    return launch<GT, RT, 4, kSmall ? 1 : 0, 1024, false>(p, whole_warps((units + 3) / 4), sms, st, parts);
  }
  if (h <= 1024) return pick_odd<GT, RT, 32>(p, sms, st, parts);
  if (h <= 4096) return pick_odd<GT, RT, 128>(p, sms, st, parts);
  if (h <= 16384) return pick_odd<GT, RT, 512>(p, sms, st, parts);
  return pick_odd<GT, RT, 1024>(p, sms, st, parts);
}

}  // namespace

size_t rmsnorm_backward_workspace_bytes(long long s, long long h) {
  return round256(size_t(s < kRmsMaxParts ? (s > 0 ? s : 1) : kRmsMaxParts) * size_t(h) * sizeof(float));
}

cudaError_t launch_rmsnorm_backward(const RmsNormBwdParams& p, bool dy_bf16, bool x_bf16, bool vectors, int sms,
                                    cudaStream_t st) {
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (p.s > 0) {
    e = !dy_bf16 ? pick<float, float>(p, vectors, sms, st, &parts)
        : x_bf16 ? pick<__nv_bfloat16, __nv_bfloat16>(p, vectors, sms, st, &parts)
                 : pick<__nv_bfloat16, float>(p, vectors, sms, st, &parts);
    if (e != cudaSuccess) return e;
  }
  // the partial rows are added by a programmatic dependent: its launch is
  // hidden behind the first kernel's last rows
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.h + kColumns - 1) / kColumns);
  cfg.blockDim = dim3(kColumns * kRowLanes);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.s > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, rmsnorm_weight_kernel, (const float*)p.part, parts, p.h, p.dw, p.accumulate);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace vpce
