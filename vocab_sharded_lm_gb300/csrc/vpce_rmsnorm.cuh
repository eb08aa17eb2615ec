// Root-mean-square norm with the residual's addition: parameter blocks and the
// element access shared by the forward and the gradient.
#pragma once

#include "vpce_rows.cuh"

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

// CTAs (one an SM) whose sums of the weight's gradient the workspace holds.
constexpr int kRmsMaxParts = 256;

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

// Rows off 16 bytes: the columns of one thread of a team of kT.  A warp has a
// run of columns, up to eight times 128; a lane every 32nd of them.  (A run keeps
// a group's columns together, and the addresses of a lane's columns are one
// register and constants.)
constexpr int kOddColumns = 32;
template <int kT> struct OddColumns {
  int h, lane, start, quads;  // start: the warp's first column; quads: 128 columns each
  __device__ __forceinline__ OddColumns(int h_, int tid) : h(h_), lane(tid & 31) {
    constexpr int kWarps = kT / 32;
    quads = ((h + 127) / 128 + kWarps - 1) / kWarps;
    start = (tid >> 5) * quads * 128;
  }
  // f(q, first column, all): for every 128 columns; `all`: they are all of the row
  template <typename F> __device__ __forceinline__ void by_quads(F f) const {
#pragma unroll
    for (int q = 0; q < kOddColumns / 4; ++q) {
      const int c = start + q * 128;
      if (q >= quads || c >= h) break;
      if (c + 128 <= h) f(q, c, true);
      else f(q, c, false);
    }
  }
  // f(k, c, inside): for the thread's k-th column, four at a time without a
  // branch between them (so that their loads go together); in the row's last
  // 128, `inside` may be false, and c is then 0
  template <typename F> __device__ __forceinline__ void each(F f) const {
    by_quads([&](int q, int first, bool all) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = first + i * 32 + lane;
        f(q * 4 + i, all || c < h ? c : 0, all || c < h);
      }
    });
  }
};

// The threads of one team: whole warps, with a barrier of their own (not 0,
// which is the CTA's).
struct Team {
  int id, tid, threads;
  float* red;  // [2][32]
  __device__ __forceinline__ void sync() const {
    if (threads == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
  }
  // largest of the team's values, through 32 words of shared memory
  __device__ __forceinline__ unsigned max(unsigned v, unsigned* sm) const {
    v = __reduce_max_sync(kFull, v);
    if (threads > 32) {
      const int lane = tid & 31, warps = threads >> 5;
      if (lane == 0) sm[tid >> 5] = v;
      sync();
      v = __reduce_max_sync(kFull, lane < warps ? sm[lane] : 0u);
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v, int parity) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (threads > 32) {
      const int lane = tid & 31, warps = threads >> 5;
      float* r = red + parity * 32;
      if (lane == 0) r[tid >> 5] = v;
      sync();
      v = lane < warps ? r[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    }
    return v;
  }
};

// Rows off 16 bytes come through a ring of shared memory per team: a row's bytes
// are copied as the 16-byte vectors that hold them, the last cut to the row's
// end; the first may begin in the row before (where that is before the array's
// first element, it is copied by elements).
// Elements are then read from shared memory, where alignment costs nothing.
struct OddRing {
  int first, other;  // bytes of a row of the first array and of the others, with room for its offset
  __host__ __device__ OddRing(int h, int first_element, int other_element)
      : first((h * first_element + 30) / 16 * 16), other((h * other_element + 30) / 16 * 16) {}
  __host__ __device__ int bytes(int others) const { return first + others * other; }
};

template <int kElement, int kT>
__device__ __forceinline__ void copy_odd_row(unsigned char* dst, const unsigned char* base, long long row, long long ld, int h,
                                             int tid) {
  const unsigned char* const src = base + row * ld;
  const int off = int(uintptr_t(src) & 15), end = off + h * kElement;
  for (int v = tid * 16; v < end; v += kT * 16) {
    if (v == 0 && src - off < base) {
      for (int i = off; i < 16 && i < end; i += kElement) {
        if constexpr (kElement == 2) *reinterpret_cast<short*>(dst + i) = *reinterpret_cast<const short*>(src - off + i);
        else *reinterpret_cast<int*>(dst + i) = *reinterpret_cast<const int*>(src - off + i);
      }
    } else {
      copy_async_part(dst + v, src - off + v, end - v < 16 ? end - v : 16);
    }
  }
}

constexpr int kMaxSmem = 200 * 1024;  // a CTA's rings, where it has an SM for itself

// Lets a kernel have more shared memory than every launch may: 48 KB of static
// and dynamic memory together, and these kernels' own is 8 KB at most.  (Always
// the same bound, so that calls from several threads agree.  Done when a kernel
// is launched: for all of these kernels in a device's set-up it would load them all.)
template <typename K> cudaError_t allow_smem(K* kernel, size_t bytes) {
  return bytes > 40 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem + 16 * 1024)
                           : cudaSuccess;
}

// Teams of kT threads on an SM, 512 threads at most (or one team), and the rows
// of each ring: three where every team can have them, else two, else no ring.
// `more`: other shared memory of a team.
struct OddPlan {
  int teams, stages;
  OddPlan(int row_bytes, int more, int T) {
    const int most = T >= 512 ? 1 : 512 / T;
    for (stages = 3; stages >= 2; --stages) {
      teams = kMaxSmem / (stages * row_bytes + more);
      if (teams > most) teams = most;
      if ((stages == 3 && teams == most && T <= 512) || (stages == 2 && teams >= 1)) return;
    }
    stages = 0;
    teams = most;
  }
};

// ---------------------------------------------------------------------------
// e4m3 output
// ---------------------------------------------------------------------------
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

// Where a group's largest magnitude is found: in the lanes of a warp that hold
// the group (16, 32, .. 256 columns in vectors), by the whole team (one group a
// row), or through shared memory.
enum GroupKind { kNoCodes, kLanes, kRow, kShared };

__device__ __forceinline__ int group_of(const RmsNormParams& p, int c) { return int(__umulhi(unsigned(c), p.group_inverse)); }

// kShared: every `segment` columns leave their maximum in shared memory, and a
// team's first threads join those of a group.
struct GroupPlan {
  int segment, segments, groups;  // columns of a segment; segments (up to a multiple of `whole` columns) and groups of a row
  GroupPlan(const RmsNormParams& p, int segment_, int whole)
      : segment(segment_), segments((p.h + whole - 1) / whole * (whole / segment_)), groups(p.groups) {}
  __host__ __device__ int bytes() const { return (segments + 2 * groups + 3) / 4 * 16; }
};
struct GroupWords {
  unsigned* tops;            // [segments]
  float *scales, *inverses;  // [groups]; an infinite scale is held as 0 (see quotient)
  __device__ __forceinline__ GroupWords(void* sm, const GroupPlan& g)
      : tops(static_cast<unsigned*>(sm)), scales(reinterpret_cast<float*>(tops + g.segments)), inverses(scales + g.groups) {}
  __device__ __forceinline__ void join(const GroupPlan& g, int group, int tid, int T, float* out) const {
    const int per = group / g.segment;
    for (int i = tid; i < g.groups; i += T) {
      const int end = (i + 1) * per < g.segments ? (i + 1) * per : g.segments;
      unsigned t = 0;
      for (int j = i * per; j < end; ++j) t = max(t, tops[j]);
      const float scale = e4m3_scale(t);
      out[i] = scale;
      scales[i] = isinf(scale) ? 0.f : scale;
      inverses[i] = __frcp_rn(scale);
    }
  }
};

// Rows off 16 bytes: one translation unit for each pair of types (they are many
// kernels).
template <typename XT, typename RT> cudaError_t rmsnorm_forward_odd(const RmsNormParams& p, GroupKind kind, int sms, cudaStream_t st);

cudaError_t launch_rmsnorm_forward(const RmsNormParams& p, bool x_bf16, bool res_bf16, bool codes, bool vectors, int sms,
                            cudaStream_t st);
cudaError_t launch_rmsnorm_backward(const RmsNormBwdParams& p, bool dy_bf16, bool x_bf16, bool vectors, int sms,
                                    cudaStream_t st);
size_t rmsnorm_backward_workspace_bytes(long long s, long long h);

}  // namespace vpce
