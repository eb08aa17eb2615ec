// Log probabilities of given tokens, entropy and top alternatives of rows of
// vocabulary-sharded logits, in one pass.
//
// With m the row's largest z and v_k = (z_k - m) log2(e) / T,
//     S = sum_k 2^v_k,  U = sum_k v_k 2^v_k,
//     logp_y = (z_y - m) / T - ln S,  entropy = ln S - ln2 U / S.
// v is formed by subtracting first: bf16 logits subtract exactly, and rows
// filled with the type's lowest finite value stay finite.  v is clamped at
// -256, where 2^v is 0 in fp32, so a column at -inf adds 0 (not 0 * inf).
//
// A row is cut into pieces (part of one shard, 16-byte vectors).  The warp
// that takes a piece streams it into registers and leaves, per lane, (max, S,
// U) of the vectors that lane read.  The warp that completes a row folds these
// in a fixed order whatever warp made them, so results repeat bit for bit.
//
// Top alternatives without a second pass: a lane's maximum over its share of
// a piece (its batch) is in the partials already.  The top-th largest of 64
// batch-group maxima bounds the top-th largest logit from below, so every
// alternative lies in a batch whose maximum reaches the bound: some 20 to 45
// batches of a row's 1000, re-read while they are still in L2.  Candidates
// are 64-bit words (order-preserving key of the value, complement of the
// column), so one comparison ranks by value, then lowest column.
#include <cooperative_groups.h>

#include "vpce_logprob.cuh"

namespace vpce {

namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxPieces = 64;   // pieces per row
constexpr int kLpSlots = 3;        // rows with partials in shared memory at a time
constexpr int kLpCand = 128;       // candidate words per warp
constexpr int kLpList = 64;        // batches listed per warp before they are re-read
constexpr float kLpFloor = -256.f;

template <typename T> struct LpShape;
template <> struct LpShape<__nv_bfloat16> {
  static constexpr int kVecs = 16;
  static constexpr int kCtas = 2;
};
template <> struct LpShape<float> {
  static constexpr int kVecs = 12;
  static constexpr int kCtas = 2;
};

// How a row is cut: piece i covers vectors [off, off + len) of its shard's
// 16-byte aligned body; the shard's first piece also takes the elements
// before and after the body.
struct LpPlan {
  int pieces;      // per row
  int len;         // vectors per piece: a multiple of 32 U
};

struct Piece {
  int shard;
  int off;
};

struct LpSmem {
  float* m;            // [slots][pieces][32]
  float* s;
  float* u;
  unsigned long long (*cand)[kLpCand];
  unsigned short (*list)[kLpList];
};

__device__ __forceinline__ float lane_max(const uint4& v, __nv_bfloat16) {
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 x = __hmax2_nan(__hmax2_nan(b[0], b[1]), __hmax2_nan(b[2], b[3]));
  return max_nan(__low2float(x), __high2float(x));
}
__device__ __forceinline__ float lane_max(const uint4& v, float) {
  return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                 max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <int U>
__device__ __forceinline__ float vecs_max(const uint4 (&q)[U], __nv_bfloat16) {
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(q);
  __nv_bfloat162 x = b[0];
#pragma unroll
  for (int j = 1; j < 4 * U; ++j) x = __hmax2_nan(x, b[j]);
  return max_nan(__low2float(x), __high2float(x));
}
template <int U>
__device__ __forceinline__ float vecs_max(const uint4 (&q)[U], float) {
  float x = lane_max(q[0], 0.f);
#pragma unroll
  for (int j = 1; j < U; ++j) x = max_nan(x, lane_max(q[j], 0.f));
  return x;
}

__device__ __forceinline__ uint4 lp_pad(__nv_bfloat16) {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}
__device__ __forceinline__ uint4 lp_pad(float) {
  return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}

// A lane's running maximum and sums.
struct Acc {
  float m, s, u;
  // move the maximum up to nm: 2^v and v 2^v of every term change by the same
  // shift (v' = v + d).  fmaxf turns the NaN of (-inf) - (-inf) into the floor.
  __device__ __forceinline__ void raise(float nm, float c) {
    const float d = fmaxf((m - nm) * c, kLpFloor);
    const float e = ex2(d);
    u = fmaf(s, d, u) * e;
    s *= e;
    m = nm;
  }
};

__device__ __forceinline__ void add_pair(float x0, float x1, f32x2 nm, f32x2 c, f32x2& s, f32x2& u) {
  float a, b;
  f2_unpack(f2_mul(f2_add(f2_pack(x0, x1), nm), c), a, b);
  a = fmaxf(a, kLpFloor);
  b = fmaxf(b, kLpFloor);
  const f32x2 e = f2_pack(ex2(a), ex2(b));
  s = f2_add(s, e);
  u = f2_fma(f2_pack(a, b), e, u);
}
__device__ __forceinline__ void add_vec(const uint4& v, f32x2 nm, f32x2 c, f32x2 (&s)[2], f32x2 (&u)[2],
                                        __nv_bfloat16) {
  add_pair(bf16_lo(v.x), bf16_hi(v.x), nm, c, s[0], u[0]);
  add_pair(bf16_lo(v.y), bf16_hi(v.y), nm, c, s[1], u[1]);
  add_pair(bf16_lo(v.z), bf16_hi(v.z), nm, c, s[0], u[0]);
  add_pair(bf16_lo(v.w), bf16_hi(v.w), nm, c, s[1], u[1]);
}
__device__ __forceinline__ void add_vec(const uint4& v, f32x2 nm, f32x2 c, f32x2 (&s)[2], f32x2 (&u)[2], float) {
  add_pair(__uint_as_float(v.x), __uint_as_float(v.y), nm, c, s[0], u[0]);
  add_pair(__uint_as_float(v.z), __uint_as_float(v.w), nm, c, s[1], u[1]);
}

// The row segment of a shard: 16-byte aligned body and ragged ends.
struct Seg {
  const unsigned char* addr;
  int head, nv, tail;  // elements before the body, vectors in it, elements after
};
template <typename T>
__device__ __forceinline__ Seg segment(const LogprobParams& p, int shard, long long row) {
  const Unit g = make_unit_at(p.sh, shard, row, Elem<T>::kBytes);
  Seg q;
  q.addr = g.addr;
  q.head = int(g.head) / Elem<T>::kBytes;
  q.nv = int(g.body >> 4);
  q.tail = int(g.tail) / Elem<T>::kBytes;
  return q;
}
template <typename T>
__device__ __forceinline__ const uint4* body(const Seg& q) {
  return reinterpret_cast<const uint4*>(q.addr + q.head * Elem<T>::kBytes);
}
// the ragged element that lane l of a shard's first piece takes (column in
// the shard), or -1: lanes 0.. the ones before the body, 16.. those after
template <typename T>
__device__ __forceinline__ int ragged_column(const Seg& q, int l) {
  if (l < q.head) return l;
  if (l >= 16 && l - 16 < q.tail) return q.head + q.nv * Elem<T>::kPerVec + (l - 16);
  return -1;
}

// One piece by one warp: the lane's (max, S, U).
template <typename T, int U>
__device__ __forceinline__ Acc piece_stats(const LogprobParams& p, const Piece& pc, int len, long long row, float c,
                                           int lane) {
  const Seg g = segment<T>(p, pc.shard, row);
  const uint4* v = body<T>(g);
  Acc a{-INFINITY, 0.f, 0.f};
  const int end = min(pc.off + len, g.nv);
  const f32x2 cc = f2_pack(c, c);
#pragma unroll 1
  for (int base = pc.off; base < end; base += 32 * U) {
    uint4 q[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = base + lane + 32 * j;
      q[j] = i < end ? __ldcs(v + i) : lp_pad(T());
    }
    const float cm = vecs_max<U>(q, T());
    if (!(cm <= a.m)) a.raise(max_nan(a.m, cm), c);
    const f32x2 nm = f2_pack(-a.m, -a.m);
    f32x2 s[2] = {f2_pack(a.s, 0.f), f2_pack(0.f, 0.f)}, u[2] = {f2_pack(a.u, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < U; ++j) add_vec(q[j], nm, cc, s, u, T());
    float x0, x1;
    f2_unpack(f2_add(s[0], s[1]), x0, x1);
    a.s = x0 + x1;
    f2_unpack(f2_add(u[0], u[1]), x0, x1);
    a.u = x0 + x1;
  }
  if (pc.off == 0) {
    const int col = ragged_column<T>(g, lane);
    if (col >= 0) {
      const float x = Elem<T>::load(g.addr + (long long)col * Elem<T>::kBytes);
      if (!(x <= a.m)) a.raise(max_nan(a.m, x), c);
      const float w = fmaxf((x - a.m) * c, kLpFloor), e = ex2(w);
      a.s += e;
      a.u = fmaf(w, e, a.u);
    }
  }
  return a;
}

// ---------------------------------------------------------------------------
// top alternatives
// ---------------------------------------------------------------------------
__device__ __forceinline__ float key_value(unsigned k) {
  if (k == 0xffffffffu) return __int_as_float(0x7fc00000);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The candidates of one warp: cand[0 .. n) hold the words seen so far that
// beat `floor`; when full they are cut to the `top` best.
struct Best {
  unsigned long long* cand;
  unsigned long long floor;  // words must exceed it
  int n, top;

  // sorts cand[0 .. n) descending and keeps the first `top`
  __device__ __noinline__ void cut(int lane) {
    __syncwarp();
    unsigned long long w[kLpCand / 32];
    int rank[kLpCand / 32];
#pragma unroll
    for (int i = 0; i < kLpCand / 32; ++i) {
      w[i] = lane + 32 * i < n ? cand[lane + 32 * i] : 0ull;
      rank[i] = 0;
    }
    for (int j = 0; j < n; ++j) {
      const unsigned long long x = cand[j];
#pragma unroll
      for (int i = 0; i < kLpCand / 32; ++i) rank[i] += x > w[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLpCand / 32; ++i)
      if (lane + 32 * i < n && rank[i] < top) cand[rank[i]] = w[i];
    __syncwarp();
    if (n >= top) {
      n = top;
      floor = cand[top - 1];
    }
  }

  // offers one word per lane (0: none)
  __device__ __forceinline__ void offer(unsigned long long w, int lane) {
    unsigned m = __ballot_sync(kFull, w > floor);
    if (m == 0) return;
    if (n + __popc(m) > kLpCand) {
      cut(lane);
      m = __ballot_sync(kFull, w > floor);
    }
    if (w > floor) cand[n + __popc(m & ((1u << lane) - 1u))] = w;
    n += __popc(m);
  }
};

__device__ __forceinline__ unsigned long long word(unsigned key, unsigned col) {
  return ((unsigned long long)key << 32) | (unsigned)~col;
}

// The `top` best columns of a row, sorted, into best.cand[0 .. top).  m: the
// row's batch maxima [pieces][32].
template <typename T, int U>
__device__ __forceinline__ void find_top(const LogprobParams& p, const LpPlan& plan, const Piece* piece,
                                         const float* m, long long row, Best& best, unsigned short* list, int lane) {
  constexpr int EPV = Elem<T>::kPerVec;
  // lower bound: the top-th largest of the maxima of 64 groups of batches
  // (lane, piece parity)
  unsigned a = 0, b = 0;
  for (int i = 0; i < plan.pieces; i += 2) {
    a = max(a, value_key(m[i * 32 + lane]));
    if (i + 1 < plan.pieces) b = max(b, value_key(m[(i + 1) * 32 + lane]));
  }
  unsigned bound = 0;
  for (int seen = 0; seen < p.top;) {
    bound = __reduce_max_sync(kFull, max(a, b));
    seen += __popc(__ballot_sync(kFull, a == bound)) + __popc(__ballot_sync(kFull, b == bound));
    if (a == bound) a = 0;
    if (b == bound) b = 0;
    if (bound == 0) break;
  }
  best.n = 0;
  best.top = p.top;
  // a word beats the floor if its key is at least `bound`
  best.floor = ((unsigned long long)bound << 32) > 0 ? ((unsigned long long)bound << 32) - 1 : 0ull;

  int i = 0, listed = 0;
  while (true) {
    // list the batches that may hold a word above the floor
    while (i < plan.pieces && listed + 32 <= kLpList) {
      const bool in = word(value_key(m[i * 32 + lane]), 0) > best.floor;
      const unsigned mk = __ballot_sync(kFull, in);
      if (in) list[listed + __popc(mk & ((1u << lane) - 1u))] = (unsigned short)(i * 32 + lane);
      listed += __popc(mk);
      ++i;
    }
    __syncwarp();
    if (listed == 0) break;
    // re-read them: half a warp per batch, four batches per half in flight
    const int half = lane >> 4, hl = lane & 15;
    for (int l0 = 0; l0 < listed; l0 += 8) {
      const uint4* src[4];
      int left[4], col[4], rag[4];
      Seg seg[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int l = l0 + 2 * k + half;
        const int code = l < listed ? list[l] : -1;
        left[k] = 0;
        rag[k] = -1;
        col[k] = 0;
        src[k] = nullptr;
        if (code >= 0) {
          const Piece pc = piece[code >> 5];
          seg[k] = segment<T>(p, pc.shard, row);
          const int bl = code & 31, first = pc.off + bl + 32 * hl;
          const int end = min(pc.off + plan.len, seg[k].nv);
          left[k] = end > first ? (end - first + 511) / 512 : 0;
          src[k] = body<T>(seg[k]) + first;
          col[k] = int(p.sh.start[pc.shard]) + seg[k].head + first * EPV;
          if (pc.off == 0 && hl == 0) {
            const int rc = ragged_column<T>(seg[k], bl);
            if (rc >= 0) rag[k] = rc + int(p.sh.start[pc.shard]);
            if (rc >= 0) seg[k].addr += (long long)rc * Elem<T>::kBytes;
          }
        }
      }
      // the vectors of a batch are 32 apart; lane hl takes every 16th of them
      for (int step = 0;; ++step) {
        uint4 q[4];
        bool any = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[k] = step < left[k] ? src[k][step * 512] : lp_pad(T());
          any |= step < left[k];
        }
        if (!__any_sync(kFull, any)) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool has = step < left[k];
          const unsigned vk = has ? value_key(lane_max(q[k], T())) : 0;
          if (!__any_sync(kFull, has && word(vk, 0) > best.floor)) continue;
          float x[EPV];
          unpack(q[k], x, T());
#pragma unroll
          for (int e = 0; e < EPV; ++e)
            best.offer(has ? word(value_key(x[e]), unsigned(col[k] + step * 512 * EPV + e)) : 0ull, lane);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!__any_sync(kFull, rag[k] >= 0)) continue;
        best.offer(rag[k] >= 0 ? word(value_key(Elem<T>::load(seg[k].addr)), unsigned(rag[k])) : 0ull, lane);
      }
    }
    listed = 0;
    __syncwarp();
  }
  best.cut(lane);
}

// ---------------------------------------------------------------------------
// a complete row: fold the partials, write the outputs (one warp)
// ---------------------------------------------------------------------------
__device__ __forceinline__ void write_ignored(const LogprobParams& p, long long row, int lane) {
  if (lane == 0) {
    if (p.logp) p.logp[row] = 0.f;
    if (p.entropy) p.entropy[row] = 0.f;
    if (p.stats) p.stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (lane < p.top) {
    p.top_ids[row * p.top + lane] = -1;
    if (p.top_logp) p.top_logp[row * p.top + lane] = 0.f;
  }
}

template <typename T, int U>
__device__ __forceinline__ void finish_row(const LogprobParams& p, const LpPlan& plan, const Piece* piece,
                                           const float* m, const float* s, const float* u, long long row, long long y,
                                           unsigned long long* cand, unsigned short* list, int lane) {
  const float c = p.inv_t * kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  const bool in = p.targets != nullptr && y >= 0 && y < p.V;
  float zy = 0.f;
  if (in && lane == 0) {
    int i = 0;
    while (y >= p.sh.start[i + 1]) ++i;
    zy = Elem<T>::load(p.sh.ptr[i] + row * p.sh.ld_bytes[i] + (y - p.sh.start[i]) * Elem<T>::kBytes);
  }
  // lanes fold their own partials in piece order, then the warp in a fixed tree
  float M = -INFINITY;
  for (int i = 0; i < plan.pieces; ++i) M = max_nan(M, m[i * 32 + lane]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, o));
  float S = 0.f, W = 0.f;
  for (int i = 0; i < plan.pieces; ++i) {
    Acc a{m[i * 32 + lane], s[i * 32 + lane], u[i * 32 + lane]};
    a.raise(M, c);
    S += a.s;
    W += a.u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(kFull, S, o);
    W += __shfl_xor_sync(kFull, W, o);
  }
  // no finite largest logit (nothing unmasked, +inf or NaN): no distribution
  const bool ok = isfinite(M);
  const float ls = ok ? logf(S) : nan;
  const float ent = ok ? ls - 0.6931471806f * (W / S) : nan;
  if (lane == 0) {
    if (p.entropy) p.entropy[row] = ent;
    if (p.stats) p.stats[row] = make_float4(M, ls, ent, 0.f);
    if (p.logp) p.logp[row] = in ? (zy - M) * p.inv_t - ls : nan;
    if (p.targets != nullptr && !in && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_BAD_TARGET);
  }
  if (p.top > 0) {
    Best best;
    best.cand = cand;
    find_top<T, U>(p, plan, piece, m, row, best, list, lane);
    if (lane < p.top) {
      const unsigned long long w = best.cand[lane];
      p.top_ids[row * p.top + lane] = (long long)unsigned(~unsigned(w));
      if (p.top_logp) p.top_logp[row * p.top + lane] = (key_value(unsigned(w >> 32)) - M) * p.inv_t - ls;
    }
    __syncwarp();
  }
}

// The pieces of a row: every shard cut into ceil(vectors / len) of them, one
// at least.  Thread 0 writes the table.
template <typename T>
__device__ __forceinline__ void cut_row(const LogprobParams& p, const LpPlan& plan, Piece* piece) {
  int n = 0;
  for (int i = 0; i < p.t; ++i) {
    const int nv = int((p.sh.start[i + 1] - p.sh.start[i]) / Elem<T>::kPerVec);
    for (int off = 0; off == 0 || off < nv; off += plan.len) piece[n++] = Piece{i, off};
  }
}

// Persistent form: a CTA per row at a time, its warps taking pieces from a
// shared counter and running ahead into the next rows while one of them
// finishes a row.  A row's partials stay in one of kLpSlots places.
template <typename T>
__global__ void __launch_bounds__(kLpThreads, LpShape<T>::kCtas)
    logprob_forward_kernel(const __grid_constant__ LogprobParams p, const LpPlan plan) {
  constexpr int U = LpShape<T>::kVecs;
  extern __shared__ __align__(16) unsigned char lp_smem[];
  __shared__ Piece piece[kLpMaxPieces];
  __shared__ unsigned long long cand[kLpWarps][kLpCand];
  __shared__ unsigned short list[kLpWarps][kLpList];
  __shared__ int next;                      // pieces taken
  __shared__ int done[kLpSlots];            // pieces of the slot's row that are complete
  __shared__ volatile int finished[kLpSlots];  // rows finished in the slot
  __shared__ volatile int stop;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = plan.pieces * 32;
  float* sm = reinterpret_cast<float*>(lp_smem);
  float* ss = sm + kLpSlots * n;
  float* su = ss + kLpSlots * n;
  if (threadIdx.x == 0) {
    next = 0;
    stop = 0;
    for (int i = 0; i < kLpSlots; ++i) done[i] = finished[i] = 0;
    cut_row<T>(p, plan, piece);
  }
  __syncthreads();
  const float c = p.inv_t * kLog2e;
  const long long rows = (p.s - blockIdx.x + gridDim.x - 1) / gridDim.x;  // this CTA's rows
  while (true) {
    int it = 0;
    if (lane == 0) it = atomicAdd(&next, 1);
    it = __shfl_sync(kFull, it, 0);
    const long long k = it / plan.pieces;
    if (k >= rows) break;
    const int i = it - int(k) * plan.pieces;
    const int slot = int(k % kLpSlots);
    const long long row = blockIdx.x + k * gridDim.x;
    const long long y = p.targets != nullptr ? __ldg(p.targets + row) : 0;
    const bool ignored = p.targets != nullptr && y == p.ignore_index;
    Acc a;
    if (!ignored) a = piece_stats<T, U>(p, piece[i], plan.len, row, c, lane);
    // the slot's earlier row has to be finished
    const int turn = int(k / kLpSlots);
    int go = 1;
    if (lane == 0) {
      if (finished[slot] < turn) {
        const long long t0 = clock64();
        while (finished[slot] < turn && !stop) {
          if (clock64() - t0 > kWaitLimitCycles) stop = 1;
          __nanosleep(100);
        }
        go = !stop;
      }
      __threadfence_block();
    }
    if (!__shfl_sync(kFull, go, 0)) break;
    __syncwarp();
    if (!ignored) {
      const int at = slot * n + i * 32 + lane;
      sm[at] = a.m;
      ss[at] = a.s;
      su[at] = a.u;
    }
    __syncwarp();
    int last = 0;
    if (lane == 0) {
      __threadfence_block();
      last = atomicAdd(&done[slot], 1) == plan.pieces - 1;
      __threadfence_block();
    }
    if (!__shfl_sync(kFull, last, 0)) continue;
    __syncwarp();
    if (ignored) write_ignored(p, row, lane);
    else
      finish_row<T, U>(p, plan, piece, sm + slot * n, ss + slot * n, su + slot * n, row, y, cand[warp], list[warp],
                       lane);
    __syncwarp();
    if (lane == 0) {
      done[slot] = 0;
      __threadfence_block();
      finished[slot] = turn + 1;
    }
  }
  __syncthreads();
  if (stop) {  // a wait gave up: nothing of this CTA's rows is to be believed
    if (threadIdx.x == 0 && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_WAIT_TIMEOUT);
    const float nan = __int_as_float(0x7fc00000);
    for (long long k = threadIdx.x; k < rows; k += kLpThreads) {
      const long long row = blockIdx.x + k * gridDim.x;
      if (p.logp) p.logp[row] = nan;
      if (p.entropy) p.entropy[row] = nan;
      if (p.stats) p.stats[row] = make_float4(nan, nan, nan, 0.f);
      for (int j = 0; j < p.top; ++j) {
        p.top_ids[row * p.top + j] = -1;
        if (p.top_logp) p.top_logp[row * p.top + j] = nan;
      }
    }
  }
}

}  // namespace

template <typename T>
static LpPlan plan_pieces(const LogprobParams& p, int limit) {
  constexpr int kStep = 32 * LpShape<T>::kVecs;
  LpPlan plan;
  // one step per piece, more when the row would have too many pieces
  for (long long steps = 1;; steps *= 2) {
    const long long len = steps * kStep;
    long long n = 0;
    for (int i = 0; i < p.t; ++i) {
      const long long nv = (p.sh.start[i + 1] - p.sh.start[i]) / Elem<T>::kPerVec;
      n += nv > 0 ? (nv + len - 1) / len : 1;
    }
    if (n <= limit) {
      plan.pieces = int(n);
      plan.len = int(len);
      return plan;
    }
  }
}

template <typename T>
void launch_logprob_forward(const LogprobParams& p, int sms, cudaStream_t st) {
  const LpPlan plan = plan_pieces<T>(p, kLpMaxPieces);
  const long long cap = (long long)sms * LpShape<T>::kCtas;
  // equal numbers of rows per CTA: with one row more than CTAs, half the CTAs
  // and two rows each
  const long long turns = (p.s + cap - 1) / cap;
  const int grid = int((p.s + turns - 1) / turns);
  const size_t smem = size_t(kLpSlots) * plan.pieces * 32 * 3 * sizeof(float);
  logprob_forward_kernel<T><<<grid, kLpThreads, smem, st>>>(p, plan);
}
template void launch_logprob_forward<float>(const LogprobParams&, int, cudaStream_t);
template void launch_logprob_forward<__nv_bfloat16>(const LogprobParams&, int, cudaStream_t);

cudaError_t set_logprob_smem() {
  const int bytes = kLpSlots * kLpMaxPieces * 32 * 3 * int(sizeof(float));
  const cudaError_t e = cudaFuncSetAttribute(logprob_forward_kernel<float>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(logprob_forward_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              bytes);
}

}  // namespace vpce
