// Gradient of the root-mean-square norm: with n = r rstd,
//     dr = dresidual + rstd (w dy - n mean(w dy n)),    dw = sum over rows dy n.
//
// One pass over dy, r and dresidual.  A thread keeps the same columns on every
// row that its CTA takes, so dw's terms add up in its registers; each CTA then
// leaves one partial row, and a second kernel adds those in a fixed order.
#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

constexpr int kColumns = 32, kRowLanes = 16;  // of the kernel that adds the partial rows

template <typename GT, typename RT, int U, int NU, bool kWarp, int kMaxT>
__global__ void __launch_bounds__(kMaxT) rmsnorm_backward_kernel(const __grid_constant__ RmsNormBwdParams p) {
  extern __shared__ float sums[];  // [warps][h], one-warp teams only
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int teams = kWarp ? int(blockDim.x >> 5) : 1;
  const int tid = kWarp ? lane : int(threadIdx.x), T = kWarp ? 32 : int(blockDim.x);
  float acc[NU][U];
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int j = 0; j < U; ++j) acc[k][j] = 0.f;
  int parity = 0;
  for (long long row = (long long)blockIdx.x * teams + (kWarp ? warp : 0); row < p.s;
       row += (long long)gridDim.x * teams) {
    const unsigned char *gr = p.dy + row * p.ld_dy, *xr = p.x + row * p.ld_x;
    RawUnit<GT, U> g[NU];
    RawUnit<RT, U> x[NU], d[NU];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      g[k].zero();
      x[k].zero();
      d[k].zero();
      if (c < p.h) {
        g[k].load(gr, c);
        x[k].load(xr, c);
        if (p.dres != nullptr) d[k].load(p.dres + row * p.ld_dres, c);
      }
    }
    const float rstd = __ldg(p.rstd + row);
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      if (c < p.h) {
        float w[U], dy[U], n[U];
        load_weight(p.w, p.w_bf16, c, w);
        g[k].get(dy);
        x[k].get(n);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          n[j] *= rstd;
          acc[k][j] = fmaf(dy[j], n[j], acc[k][j]);
          dot = fmaf(w[j] * dy[j], n[j], dot);
        }
      }
    }
    dot = team_sum<kWarp>(dot, red[parity]) / float(p.h);
    parity ^= 1;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int c = (k * T + tid) * U;
      if (c < p.h) {
        float w[U], dy[U], n[U], o[U];
        load_weight(p.w, p.w_bf16, c, w);
        g[k].get(dy);
        x[k].get(n);
        d[k].get(o);
#pragma unroll
        for (int j = 0; j < U; ++j) o[j] = fmaf(rstd, w[j] * dy[j] - n[j] * rstd * dot, o[j]);
        store_unit(p.dx + row * p.ld_dx, c, o, RT());
      }
    }
  }
  grid_launch_dependents();
  float* part = p.part + (long long)blockIdx.x * p.h;
  if constexpr (kWarp) {
    float* mine = sums + warp * p.h;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int c = (k * T + tid) * U + j;
        if (c < p.h) mine[c] = acc[k][j];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < p.h; c += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < teams; ++i) v += sums[i * p.h + c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int c = (k * T + tid) * U + j;
        if (c < p.h) part[c] = acc[k][j];
      }
  }
}

// dw[c] (+)= sum over the partial rows, in a fixed order: kRowLanes threads
// take every kRowLanes-th row, then one adds their sums in turn.
__global__ void rmsnorm_weight_kernel(const float* part, int parts, int h, float* dw, int accumulate) {
  __shared__ float sm[kRowLanes][kColumns];
  grid_dependency_wait();
  const int x = threadIdx.x % kColumns, y = threadIdx.x / kColumns, c = blockIdx.x * kColumns + x;
  float v = 0.f;
  if (c < h) {
#pragma unroll 4
    for (int i = y; i < parts; i += kRowLanes) v += __ldcg(part + (long long)i * h + c);
  }
  sm[y][x] = v;
  __syncthreads();
  if (y == 0 && c < h) {
    v = sm[0][x];
#pragma unroll
    for (int i = 1; i < kRowLanes; ++i) v += sm[i][x];
    dw[c] = accumulate ? dw[c] + v : v;
  }
}

template <typename GT, typename RT, int U, int NU, bool kWarp, int kMaxT = 128>
int launch(const RmsNormBwdParams& p, int threads, int sms, cudaStream_t st) {
  const int warps = 4, teams = kWarp ? warps : 1;
  const long long rows = (p.s + teams - 1) / teams;
  const int per_sm = kWarp ? 6 : threads <= 256 ? 4 : threads <= 512 ? 2 : 1;
  const int most = sms * per_sm < kRmsMaxParts ? sms * per_sm : kRmsMaxParts;
  const int grid = int(rows < most ? rows : most);
  const size_t smem = kWarp ? size_t(warps) * p.h * sizeof(float) : 0;
  rmsnorm_backward_kernel<GT, RT, U, NU, kWarp, kMaxT><<<grid, kWarp ? warps * 32 : threads, smem, st>>>(p);
  return grid;
}

template <typename GT, typename RT> int pick(const RmsNormBwdParams& p, bool vectors, int sms, cudaStream_t st) {
  const int h = p.h;
  if (vectors) {
    const int units = h / 8;
    if (units <= 32) return launch<GT, RT, 8, 1, true>(p, 32, sms, st);
    if (units <= 128) return launch<GT, RT, 8, 4, true>(p, 32, sms, st);
    if (units <= 1024) return launch<GT, RT, 8, 2, false, 512>(p, ((units + 1) / 2 + 31) / 32 * 32, sms, st);
    return launch<GT, RT, 8, 4, false, 1024>(p, ((units + 3) / 4 + 31) / 32 * 32, sms, st);
  }
  if (h <= 256) return launch<GT, RT, 1, 8, true>(p, 32, sms, st);
  if (h <= 1024) return launch<GT, RT, 1, 32, true>(p, 32, sms, st);
  return launch<GT, RT, 1, 32, false, 1024>(p, ((h + 31) / 32 + 31) / 32 * 32, sms, st);
}

}  // namespace

size_t rmsnorm_backward_workspace_bytes(long long s, long long h) {
  return round256(size_t(s < kRmsMaxParts ? (s > 0 ? s : 1) : kRmsMaxParts) * size_t(h) * sizeof(float));
}

cudaError_t launch_rmsnorm_backward(const RmsNormBwdParams& p, bool dy_bf16, bool x_bf16, bool vectors, int sms,
                                    cudaStream_t st) {
  int parts = 0;
  if (p.s > 0) {
    parts = !dy_bf16 ? pick<float, float>(p, vectors, sms, st)
            : x_bf16 ? pick<__nv_bfloat16, __nv_bfloat16>(p, vectors, sms, st)
                     : pick<__nv_bfloat16, float>(p, vectors, sms, st);
    const cudaError_t e = cudaGetLastError();
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rmsnorm_weight_kernel, (const float*)p.part, parts, p.h, p.dw,
                                           p.accumulate);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace vpce
