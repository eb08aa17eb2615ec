// Root-mean-square norm with the residual's addition: parameter blocks and the
// element access shared by the forward and the gradient.
#pragma once

#include "vpce_device.cuh"

namespace vpce {

struct RmsNormParams {
  const unsigned char* x;
  long long ld_x;            // strides in bytes
  const unsigned char* res;  // null: no residual
  long long ld_res;
  const unsigned char* w;
  int w_bf16;
  float eps;
  long long s;
  int h;
  unsigned char* res_out;
  long long ld_res_out;
  unsigned char* out;        // rows of x's type, or e4m3 codes
  long long ld_out;
  float* scale;              // [s][groups], codes only
  int group, groups;
  unsigned group_inverse;    // ceil(2^32 / group): a column's group is the product's high word (columns < 2^15)
  float* rstd;               // may be null
};

struct RmsNormBwdParams {
  const unsigned char* dy;
  long long ld_dy;
  const unsigned char* x;
  long long ld_x;
  const unsigned char* w;
  int w_bf16;
  const float* rstd;
  const unsigned char* dres;  // may be null
  long long ld_dres;
  long long s;
  int h;
  unsigned char* dx;
  long long ld_dx;
  float* part;                // [CTAs][h]
  float* dw;
  int accumulate;
};

// CTAs whose sums of the weight's gradient the workspace holds.
constexpr int kRmsMaxParts = 1024;

// Eight consecutive elements of a row as they lie in memory, in 16-byte vectors.
template <typename T> struct RawUnit;
template <> struct RawUnit<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const unsigned char* row, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(row + size_t(c) * 4);
    a = p[0];
    b = p[1];
  }
  // from a thread's own slots in shared memory, `pitch` vectors apart
  __device__ __forceinline__ void take(const unsigned char* p, int pitch) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *(reinterpret_cast<const uint4*>(p) + pitch);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
};
template <> struct RawUnit<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const unsigned char* row, int c) {
    a = *reinterpret_cast<const uint4*>(row + size_t(c) * 2);
  }
  __device__ __forceinline__ void take(const unsigned char* p, int) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack(a, v, __nv_bfloat16()); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
};
__device__ __forceinline__ void store_unit(unsigned char* row, int c, const float (&v)[8], float) {
  uint4* p = reinterpret_cast<uint4*>(row + size_t(c) * 4);
  p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
}
__device__ __forceinline__ void store_unit(unsigned char* row, int c, const float (&v)[8], __nv_bfloat16 t) {
  *reinterpret_cast<uint4*>(row + size_t(c) * 2) = pack(v, t);
}
// The weights of eight columns, or one, through the read-only path (every row reads them).
__device__ __forceinline__ void load_weight(const unsigned char* w, int w_bf16, int c, float (&v)[8]) {
  if (w_bf16) {
    unpack(__ldg(reinterpret_cast<const uint4*>(w + size_t(c) * 2)), v, __nv_bfloat16());
  } else {
    const float4* p = reinterpret_cast<const float4*>(w + size_t(c) * 4);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ float load_weight(const unsigned char* w, int w_bf16, int c) {
  return w_bf16 ? __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short*>(w) + c)) << 16)
                : __ldg(reinterpret_cast<const float*>(w) + c);
}

// Rows off 16 bytes: kT threads take column k kT + tid, k < kOddColumns.  Calls
// f(k, c, inside) for every k that has columns, four at a time without a branch
// between them (so that their loads go together): for the last four, `inside`
// may be false, and c is then 0.
constexpr int kOddColumns = 32;
template <int kT, typename F> __device__ __forceinline__ void odd_columns(int h, int tid, F f) {
#pragma unroll
  for (int k = 0; k < kOddColumns; k += 4) {
    if (k * kT >= h) break;
    if ((k + 4) * kT <= h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f(k + i, (k + i) * kT + tid, true);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (k + i) * kT + tid;
        f(k + i, c < h ? c : 0, c < h);
      }
    }
  }
}

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

void launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                            cudaStream_t st);
cudaError_t launch_rmsnorm_backward(const RmsNormBwdParams& p, bool dy_bf16, bool x_bf16, bool vectors, int sms,
                                    cudaStream_t st);
size_t rmsnorm_backward_workspace_bytes(long long s, long long h);

}  // namespace vpce
