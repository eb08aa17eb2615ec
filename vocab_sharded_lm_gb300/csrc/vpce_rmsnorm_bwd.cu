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
// copied, so no barrier goes with it), a few rows deep.  Rows off 16 bytes are
// read element by element by smaller teams, several in a CTA.
#include <type_traits>

#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

constexpr int kColumns = 32, kRowLanes = 32;  // of the kernel that adds the partial rows

// The threads of one team: whole warps, with a barrier of their own (not 0,
// which is the CTA's).
struct Team {
  int id, tid, threads;
  float* red;  // [2][32]
  __device__ __forceinline__ float sum(float v, int parity) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (threads > 32) {
      const int lane = tid & 31, warps = threads >> 5;
      float* r = red + parity * 32;
      if (lane == 0) r[tid >> 5] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
      v = lane < warps ? r[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    }
    return v;
  }
};

// What a thread copies ahead of a unit: vectors of 16 bytes, or one fp32 word.
template <typename T, int U> constexpr int kParts = U == 8 ? int(sizeof(T)) / 2 : 1;
template <int U> constexpr int kSlotBytes = U == 8 ? 16 : 4;

// kStages: rows of the ring ahead (0: none, rows are loaded when they are due).
// kT: threads of a team, known when compiled (addresses of single elements are
// then one register and constants), or 0.  kKeep: products of a row's values
// stay in registers until its mean is known, and the weights for all rows; else
// (32 columns a thread) they are read a second time, from the ring or through
// L1.
template <typename GT, typename RT, int U, int NU, int kStages, int kMaxT, int kCtas, int kT, bool kKeep>
__global__ void __launch_bounds__(kMaxT, kCtas) rmsnorm_backward_kernel(const __grid_constant__ RmsNormBwdParams p,
                                                                 int team_threads) {
  extern __shared__ uint4 smem[];  // the ring, and at the end sums [teams][h]
  __shared__ float red[kMaxT / 32][2][32];
  constexpr bool kRing = kStages > 0;
  const int T = kT > 0 ? kT : team_threads;
  Team team;
  const int teams = blockDim.x / T;
  team.id = threadIdx.x / T;
  team.tid = threadIdx.x - team.id * T;
  team.threads = T;
  team.red = &red[team.id][0][0];
  const int tid = team.tid;
  // (units past the row are skipped by all of a team's threads)
  const auto past = [&](int k) { return U == 1 && k * T >= p.h; };
  float acc[NU][U], w[kKeep ? NU : 1][U];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
#pragma unroll
    for (int j = 0; j < U; ++j) acc[k][j] = 0.f;
    if constexpr (kKeep) {
      const int c = (k * T + tid) * U;
      if (c < p.h) load_weight(p.w, p.w_bf16, c, w[k]);
    }
  }

  // ring slot of part v of a stage: this thread's own bytes
  constexpr int kG = kParts<GT, U>, kR = kParts<RT, U>, kVecs = NU * (kG + 2 * kR), kSlot = kSlotBytes<U>;
  const auto slot = [&](int stage, int v) {
    return reinterpret_cast<unsigned char*>(smem) + ((stage * kVecs + v) * int(blockDim.x) + int(threadIdx.x)) * kSlot;
  };
  // (the two vectors of eight fp32 values share sectors with each other: those go through L1)
  const auto copy = [&](int stage, int v, const unsigned char* src, auto fp32) {
    if constexpr (U == 1) copy_async<4>(slot(stage, v), src);
    else if constexpr (fp32) copy_async<16, true>(slot(stage, v), src);
    else copy_async<16>(slot(stage, v), src);
  };
  constexpr std::bool_constant<sizeof(GT) == 4> g32{};
  constexpr std::bool_constant<sizeof(RT) == 4> r32{};
  const auto fetch = [&](long long row, int stage) {
    if (row < p.s) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (past(k)) break;
        const int c = (k * T + tid) * U;
        if (c < p.h) {
          const unsigned char *g = p.dy + row * p.ld_dy + size_t(c) * sizeof(GT),
                              *x = p.x + row * p.ld_x + size_t(c) * sizeof(RT);
#pragma unroll
          for (int i = 0; i < kG; ++i) copy(stage, k * kG + i, g + 16 * i, g32);
#pragma unroll
          for (int i = 0; i < kR; ++i) copy(stage, NU * kG + k * kR + i, x + 16 * i, r32);
          if (p.dres != nullptr) {
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
    const auto load_g = [&](RawUnit<GT, U>& g, int k, int c) {
      if constexpr (kRing) g.take(slot(stage, k * kG), blockDim.x);
      else g.load(p.dy + row * p.ld_dy, c);
    };
    const auto load_x = [&](RawUnit<RT, U>& x, int k, int c) {
      if constexpr (kRing) x.take(slot(stage, NU * kG + k * kR), blockDim.x);
      else x.load(p.x + row * p.ld_x, c);
    };
    const auto load_d = [&](RawUnit<RT, U>& d, int k, int c) {
      if constexpr (kRing) d.take(slot(stage, NU * (kG + kR) + k * kR), blockDim.x);
      else d.load(p.dres + row * p.ld_dres, c);
    };
    // t = w dy and n = r rstd of a unit
    const auto terms = [&](int k, int c, const RawUnit<GT, U>& g, const RawUnit<RT, U>& x, float (&dy)[U], float (&t)[U],
                           float (&n)[U]) {
      if constexpr (!kKeep) load_weight(p.w, p.w_bf16, c, w[0]);
      g.get(dy);
      x.get(n);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        n[j] *= rstd;
        t[j] = w[kKeep ? k : 0][j] * dy[j];
      }
    };
    if constexpr (kRing) copy_wait<(kRing ? kStages - 1 : 0)>();
    constexpr int kKept = kKeep ? NU : 1;
    RawUnit<GT, U> g[kKept];
    RawUnit<RT, U> x[kKept], d[kKept];
    float t[kKept][U], n[kKept][U];
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (past(k)) break;
        const int c = (k * T + tid) * U;
        d[k].zero();
        if (c < p.h) {
          load_g(g[k], k, c);
          load_x(x[k], k, c);
          if (p.dres != nullptr) load_d(d[k], k, c);
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      if (past(k)) break;
      const int c = (k * T + tid) * U, at = kKeep ? k : 0;
      if (c < p.h) {
        if constexpr (!kKeep) {
          load_g(g[0], k, c);
          load_x(x[0], k, c);
        }
        float dy[U];
        terms(k, c, g[at], x[at], dy, t[at], n[at]);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          acc[k][j] = fmaf(dy[j], n[at][j], acc[k][j]);
          dot = fmaf(t[at][j], n[at][j], dot);
        }
      }
    }
    dot = team.sum(dot, parity) / float(p.h);
    parity ^= 1;
    if constexpr (kRing && kKeep) fetch(row + kStages * stride, stage);  // (the stage's values are in registers)
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      if (past(k)) break;
      const int c = (k * T + tid) * U, at = kKeep ? k : 0;
      if (c < p.h) {
        if constexpr (!kKeep) {
          float dy[U];
          load_g(g[0], k, c);
          load_x(x[0], k, c);
          d[0].zero();
          if (p.dres != nullptr) load_d(d[0], k, c);
          terms(k, c, g[0], x[0], dy, t[0], n[0]);
        }
        float o[U];
        d[at].get(o);
#pragma unroll
        for (int j = 0; j < U; ++j) o[j] = fmaf(rstd, fmaf(-n[at][j], dot, t[at][j]), o[j]);
        store_unit(p.dx + row * p.ld_dx, c, o, RT());
      }
    }
    if constexpr (kRing) {
      if constexpr (!kKeep) fetch(row + kStages * stride, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  }
  grid_launch_dependents();
  float* part = p.part + (long long)blockIdx.x * p.h;
  float* mine = part;
  if (teams > 1) {
    if constexpr (kRing) {  // (what was copied past the last row is nothing)
      copy_wait<0>();
      __syncthreads();
    }
    mine = reinterpret_cast<float*>(smem) + team.id * p.h;
  }
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int c = (k * T + tid) * U + j;
      if (c < p.h) mine[c] = acc[k][j];
    }
  if (teams > 1) {
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(smem);
    for (int c = threadIdx.x; c < p.h; c += blockDim.x) {
      float v = sums[c];
      for (int i = 1; i < teams; ++i) v += sums[i * p.h + c];
      part[c] = v;
    }
  }
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
#pragma unroll 8
    for (int i = y; i < parts; i += kRowLanes) v += __ldcg(part + (long long)i * h + c);
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

template <typename GT, typename RT, int U, int NU, int kStages, int kMaxT, int kCtas, int kT, bool kKeep>
cudaError_t launch(const RmsNormBwdParams& p, int team_threads, int sms, cudaStream_t st, int* parts) {
  const auto kernel = rmsnorm_backward_kernel<GT, RT, U, NU, kStages, kMaxT, kCtas, kT, kKeep>;
  const int teams = team_threads < kMaxT ? kMaxT / team_threads : 1, threads = team_threads * teams;
  constexpr size_t kStageBytes = size_t(NU) * (kParts<GT, U> + 2 * kParts<RT, U>)*kSlotBytes<U>;  // of a thread
  static_assert(kStages * kStageBytes * kMaxT * kCtas <= 227 * 1024 - kCtas * 8192, "the rings fit an SM");
  size_t smem = kStages * kStageBytes * threads;
  const size_t sums = teams > 1 ? size_t(teams) * p.h * sizeof(float) : 0;
  if (sums > smem) smem = sums;
  if (sms == 0) {  // device set-up: room for the ring, and for a row of sums a team
    const size_t ring = kStages * kStageBytes * kMaxT, most = size_t(kMaxT) * NU * U * sizeof(float);
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(ring > most ? ring : most));
  }
  const long long rows = (p.s + teams - 1) / teams;
  const int most = sms * kCtas < kRmsMaxParts ? sms * kCtas : kRmsMaxParts;
  *parts = int(rows < most ? rows : most);
  kernel<<<*parts, threads, smem, st>>>(p, team_threads);
  return cudaGetLastError();
}

template <typename GT, typename RT>
cudaError_t pick(const RmsNormBwdParams& p, bool vectors, int sms, cudaStream_t st, int* parts) {
  const int h = p.h;
  constexpr bool kSmall = sizeof(GT) + 2 * sizeof(RT) <= 6;  // a ring of bf16 rows holds twice as many
  const auto whole_warps = [](int n) { return (n + 31) / 32 * 32; };
  if (vectors) {
    const int units = h / 8;
    if (units <= 32) return launch<GT, RT, 8, 1, kSmall ? 8 : 4, 512, 1, 32, true>(p, 32, sms, st, parts);
    if (units <= 1024)
      return launch<GT, RT, 8, 2, kSmall ? 4 : 2, 512, 1, 0, true>(p, whole_warps((units + 1) / 2), sms, st, parts);
    if (units <= 2048)
      return launch<GT, RT, 8, 4, kSmall ? 2 : 1, 512, 1, 0, false>(p, whole_warps((units + 3) / 4), sms, st, parts);
    return launch<GT, RT, 8, 4, kSmall ? 1 : 0, 1024, 1, 0, false>(p, whole_warps((units + 3) / 4), sms, st, parts);
  }
  constexpr int kAhead = sizeof(GT) == 4 ? 2 : 0;  // cp.async has no 2-byte form
  if (h <= 256) return launch<GT, RT, 1, 8, kAhead, 512, 2, 32, true>(p, 32, sms, st, parts);
  if (h <= 1024) return launch<GT, RT, 1, 8, kAhead, 512, 2, 128, true>(p, 128, sms, st, parts);
  if (h <= 4096) return launch<GT, RT, 1, 8, kAhead, 512, 2, 512, true>(p, 512, sms, st, parts);
  return launch<GT, RT, 1, 32, 0, 1024, 1, 0, false>(p, whole_warps((h + 31) / 32), sms, st, parts);
}

// one call of each kind of row, with no SMs
template <typename GT, typename RT> cudaError_t set_up() {
  RmsNormBwdParams p = {};
  cudaError_t e = cudaSuccess;
  for (int h : {256, 1024, 4096, 8192, 16384, VPCE_MAX_NORM_COLUMNS}) {
    p.h = h;
    for (const bool vectors : {false, true})
      if (e == cudaSuccess) e = pick<GT, RT>(p, vectors, 0, nullptr, nullptr);
  }
  return e;
}

}  // namespace

cudaError_t set_rmsnorm_smem() {
  cudaError_t e = set_up<float, float>();
  if (e == cudaSuccess) e = set_up<__nv_bfloat16, __nv_bfloat16>();
  return e == cudaSuccess ? set_up<__nv_bfloat16, float>() : e;
}

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
