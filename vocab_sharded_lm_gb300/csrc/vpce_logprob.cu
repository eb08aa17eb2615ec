// Log probabilities of given tokens, entropy and top alternatives of rows of
// vocabulary-sharded logits, in one pass.
//
// With c = log2(e) / T and an offset K = c max_k z_k as rounded to fp32,
//     v_k = c z_k - K (one fused multiply-add, one rounding),
//     S = sum_k 2^v_k,  U = sum_k v_k 2^v_k,
//     entropy = ln S - ln2 U / S,   logp_y = (z_y - max) / T - ln S',
// where ln S' = ln S + ln2 (K - c max) is the sum relative to the largest
// logit itself.  Any offset gives the same entropy and probabilities, so K's
// own rounding costs nothing.  Logits below -2^21 / c enter at that floor,
// where 2^v is 0: a column at -inf adds 0 and not 0 * inf.  Rows whose largest
// logit is itself 2^20 / c or more from 0 (filled with the type's lowest value,
// say, or any ordinary row at T near 1e-5 or below) are summed again by
// subtraction, by one warp with single loads (sum_far: 6.5 ms instead of 0.38
// where all 8192 rows of V = 128256 are such ones).
//
// A row is cut into pieces (part of one shard, 16-byte vectors).  A streaming
// warp takes pieces from a shared counter and reads them through two 4 KB
// buffers of its own that the bulk-copy engine refills while it sums, so the
// bytes in flight do not depend on registers or on the arithmetic between
// loads.  It leaves the piece's (max, S, U); the warp that finishes the row
// folds these in a fixed order whatever warp made them, so results repeat bit
// for bit.
//
// Top alternatives without a second pass: the maxima of a lane's quarters of a
// piece (batches of 4 vectors a step) are kept with the partials.  The top-th
// largest of 128 group maxima bounds the top-th largest logit from below, so
// every alternative lies in a batch whose maximum reaches the bound: about
// `top` batches of a row's 4000, re-read in one round trip.  Candidates are
// 64-bit words (order-preserving key of the value, complement of the column),
// so one comparison ranks by value, then lowest column.
//
// Bound by HBM for fp32 logits (s = 4096, V = 152064, 32 alternatives: 0.376 ms
// for 2.49 GB, 6.6 TB/s; 0.343 ms without alternatives), by the issue of about
// 8 instructions per element for bf16 (s = 8192, V = 128256: 0.352 ms, 6.0 TB/s,
// 0.374 ms with 20 alternatives; the loss's statistics alone take 0.306 ms).
// Fewer streaming warps are better for fp32 (12: 0.376, 16: 0.404 ms), more are
// for bf16 until their registers run out (12: 0.416, 16: 0.374, 18: 0.47 ms).
// At 16 the 96 registers a thread are already short: the compiler reports 164
// bytes of spill stores and 276 of loads (none for fp32 at 12, 128 registers).
#include "vpce_logprob.cuh"

namespace vpce {

namespace {

// Warps that stream pieces and warps that finish rows, one CTA per SM.
template <typename T> struct LpShape;
template <> struct LpShape<__nv_bfloat16> { static constexpr int kStream = 16, kFinish = 4; };
template <> struct LpShape<float> { static constexpr int kStream = 12, kFinish = 4; };
template <typename T> constexpr int kLpThreads = 32 * (LpShape<T>::kStream + LpShape<T>::kFinish);
constexpr int kLpVecs = 8;         // vectors per lane and unit
constexpr int kLpUnit = 32 * kLpVecs;             // vectors per unit: one buffer
constexpr int kLpStep = 2 * kLpUnit;              // vectors per step: four batches of 4 vectors a lane
template <typename T> constexpr int kLpRing = LpShape<T>::kStream * 2 * kLpUnit * 16;  // bytes of all buffers
constexpr int kLpMaxPieces = 64;   // pieces per row (as many as shards can be)
constexpr int kLpPieces = 40;      // aimed at: as many as leave bf16 kLpSlots rows in kLpSmem, two for each finishing
                                   // warp (40 (16 + 256) 8 = 87 KB next to 128 KB of buffers; fp32: 4 rows, one each)
constexpr int kLpSlots = 8;        // rows with partials in shared memory at a time, where there is room
constexpr int kLpMaxSlots = 192;   // and where rows are short
constexpr int kLpSmem = 215 * 1024;     // room for the buffers and them: 227 KB less the static 11 KB
constexpr int kLpCand = 128;       // candidate words per warp
constexpr int kLpList = 128;       // batches listed per warp before they are re-read
constexpr float kLpFloor = -256.f;      // 2^v is 0 here
constexpr float kLpFar = 1048576.f;      // |K| from here on: K's rounding, up to 2^-5 below, is no longer small (sum_far)

// The maxima of a lane's four batches of a piece; bf16 ones are kept as they
// are (a maximum is one of its values).
template <typename T> struct BatchMax;
template <> struct BatchMax<float> {
  float4 v;
  __device__ __forceinline__ void set(const float4& x) { v = x; }
  __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct BatchMax<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void set(const float4& x) {
    v.x = __float_as_uint(x.x) >> 16 | (__float_as_uint(x.y) & 0xffff0000u);
    v.y = __float_as_uint(x.z) >> 16 | (__float_as_uint(x.w) & 0xffff0000u);
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
  }
};

// Part of a row: vectors [off, off + p.len) of its shard's 16-byte aligned
// body; the shard's first piece also takes the elements before and after the
// body.
struct __align__(16) Piece {
  const unsigned char* base;  // the shard
  long long ld;               // its row stride in bytes
  unsigned bytes;             // of a row
  int col;                    // its first column
  int off;
};

// A warp's room for finding a row's alternatives.
struct Scratch {
  unsigned long long cand[kLpCand];
  unsigned short list[kLpList];
  int n;
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
__device__ __forceinline__ float vecs_max(const uint4* q, __nv_bfloat16) {
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(q);
  __nv_bfloat162 x = b[0];
#pragma unroll
  for (int j = 1; j < 4 * U; ++j) x = __hmax2_nan(x, b[j]);
  return max_nan(__low2float(x), __high2float(x));
}
template <int U>
__device__ __forceinline__ float vecs_max(const uint4* q, float) {
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

// the value of a key
__device__ __forceinline__ float key_value(unsigned k) {
  if (k == 0xffffffffu) return __int_as_float(0x7fc00000);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The offset of a maximum: c m, never below -2^20 (which a NaN, or nothing
// unmasked, gives).  Rounded here: a product fused into a later difference
// would not be the offset that the sums were formed with.
__device__ __forceinline__ float offset_of(float m, float c) { return fmaxf(__fmul_rn(m, c), -kLpFar); }

// A lane's running offset and sums.
struct Acc {
  float k, s, u;
  // move the offset up to nk: every v changes by the same shift
  __device__ __forceinline__ void raise(float nk) {
    const float d = fmaxf(k - nk, kLpFloor);
    const float e = ex2(d);
    u = fmaf(s, d, u) * e;
    s *= e;
    k = nk;
  }
};

__device__ __forceinline__ void add_pair(float x0, float x1, f32x2 c, f32x2 nk, f32x2& s, f32x2& u) {
  const f32x2 v = f2_fma(f2_pack(x0, x1), c, nk);
  float a, b;
  f2_unpack(v, a, b);
  const f32x2 e = f2_pack(ex2(a), ex2(b));
  s = f2_add(s, e);
  u = f2_fma(v, e, u);
}
// logits are raised to `low` first (bf16: two at a time)
__device__ __forceinline__ void add_vec(const uint4& v, __nv_bfloat162 low, f32x2 c, f32x2 nk, f32x2 (&s)[2],
                                        f32x2 (&u)[2], __nv_bfloat16) {
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), low);
    const unsigned q = *reinterpret_cast<const unsigned*>(&h);
    add_pair(bf16_lo(q), bf16_hi(q), c, nk, s[i & 1], u[i & 1]);
  }
}
__device__ __forceinline__ void add_vec(const uint4& v, float low, f32x2 c, f32x2 nk, f32x2 (&s)[2], f32x2 (&u)[2],
                                        float) {
  add_pair(fmaxf(__uint_as_float(v.x), low), fmaxf(__uint_as_float(v.y), low), c, nk, s[0], u[0]);
  add_pair(fmaxf(__uint_as_float(v.z), low), fmaxf(__uint_as_float(v.w), low), c, nk, s[1], u[1]);
}
__device__ __forceinline__ __nv_bfloat162 packed_low(float floor, __nv_bfloat16) {
  return __float2bfloat162_rn(floor);
}
__device__ __forceinline__ float packed_low(float floor, float) { return floor; }

// The row segment of a shard: 16-byte aligned body and ragged ends.
struct Seg {
  const unsigned char* addr;
  int head, nv, tail;  // elements before the body, vectors in it, elements after
};
template <typename T>
__device__ __forceinline__ Seg segment(const Piece& pc, long long row) {
  Seg q;
  q.addr = pc.base + row * pc.ld;
  const unsigned off = unsigned(reinterpret_cast<uintptr_t>(q.addr)) & 15u;
  const unsigned head = min((16u - off) & 15u, pc.bytes), rest = pc.bytes - head;
  q.head = int(head) / Elem<T>::kBytes;
  q.nv = int(rest >> 4);
  q.tail = int(rest & 15u) / Elem<T>::kBytes;
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

// A unit's sums, its batches' maxima m0 and m1 known and the offset raised.
template <typename T>
__device__ __forceinline__ void unit_sums(const uint4 (&q)[kLpVecs], Acc& a, float c, float floor) {
  const f32x2 cc = f2_pack(c, c), off = f2_pack(-a.k, -a.k);
  const auto low = packed_low(floor, T());
  f32x2 s[2] = {f2_pack(a.s, 0.f), f2_pack(0.f, 0.f)}, u[2] = {f2_pack(a.u, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
  for (int j = 0; j < kLpVecs; ++j) add_vec(q[j], low, cc, off, s, u, T());
  float x0, x1;
  f2_unpack(f2_add(s[0], s[1]), x0, x1);
  a.s = x0 + x1;
  f2_unpack(f2_add(u[0], u[1]), x0, x1);
  a.u = x0 + x1;
}

// The ragged element a lane takes with a shard's first piece (-inf: none).
template <typename T>
__device__ __forceinline__ float ragged_value(const Seg& g, int lane) {
  const int col = ragged_column<T>(g, lane);
  return col >= 0 ? Elem<T>::load(g.addr + (long long)col * Elem<T>::kBytes) : -INFINITY;
}

// S and U of a row relative to its largest logit M, by subtraction, for rows
// whose logits are too large for the offset form (one warp; rare).
template <typename T>
__device__ __noinline__ float2 sum_far(const LogprobParams& p, long long row, float M, float c, int lane) {
  float S = 0.f, W = 0.f;
  for (int i = 0; i < p.t; ++i) {
    const unsigned char* at = p.sh.ptr[i] + row * p.sh.ld_bytes[i];
    const long long n = p.sh.start[i + 1] - p.sh.start[i];
    for (long long k = lane; k < n; k += 32) {
      const float v = fmaxf((Elem<T>::load(at + k * Elem<T>::kBytes) - M) * c, kLpFloor);
      const float e = ex2(v);
      S += e;
      W = fmaf(v, e, W);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(kFull, S, o);
    W += __shfl_xor_sync(kFull, W, o);
  }
  return make_float2(S, W);
}

// ---------------------------------------------------------------------------
// top alternatives
// ---------------------------------------------------------------------------
// Sorts n candidates (at most 32 W) and keeps the first `top`, in place.
template <int W>
__device__ __forceinline__ void rank_words(unsigned long long* cand, int n, int top, int lane) {
  unsigned long long w[W];
  int rank[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = lane + 32 * i < n ? cand[lane + 32 * i] : 0ull;
    rank[i] = 0;
  }
  for (int j = 0; j < n; ++j) {
    const unsigned long long x = cand[j];
#pragma unroll
    for (int i = 0; i < W; ++i) rank[i] += x > w[i];
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (lane + 32 * i < n && rank[i] < top) cand[rank[i]] = w[i];
  __syncwarp();
}

// The candidates of one warp: cand[0 .. n) hold the words seen so far that
// beat `floor`; when full they are cut to the `top` best.
struct Best {
  unsigned long long* cand;
  unsigned long long floor;  // words must exceed it
  int n, top;

  // sorts cand[0 .. n) descending and keeps the first `top`
  __device__ __forceinline__ void cut(int lane) {
    __syncwarp();
    rank_words<kLpCand / 32>(cand, n, top, lane);
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

// One batch of a row: number (piece, quarter, lane) as 128 piece + 32 quarter
// + lane.  Lane l (0..3) of the four that re-read it takes vector l of the
// batch's four in every step; lane 0 also takes the ragged element.
template <typename T>
struct Batch {
  const uint4* src;            // the lane's vector of step 0
  int left, col;               // steps it has a vector in; its first column
  const unsigned char* rag;    // ragged element or null
  int ragcol;
  __device__ __forceinline__ void at(const LogprobParams& p, const Piece* piece, long long row,
                                     int code, int l) {
    const Piece pc = piece[code >> 7];
    const Seg g = segment<T>(pc, row);
    const int quarter = (code >> 5) & 3;
    const int first = pc.off + (code & 31) + 32 * (4 * quarter + l);
    const int end = min(pc.off + p.len, g.nv);
    left = end > first ? (end - first + kLpStep - 1) / kLpStep : 0;
    src = body<T>(g) + first;
    col = pc.col + g.head + first * Elem<T>::kPerVec;
    if (pc.off == 0 && l == 0 && quarter == 0) {
      const int rc = ragged_column<T>(g, code & 31);
      if (rc >= 0) {
        rag = g.addr + (long long)rc * Elem<T>::kBytes;
        ragcol = rc + pc.col;
      }
    }
  }
};

__device__ __forceinline__ float quarter_max(const float4& b, int i) {
  return i < 2 ? (i == 0 ? b.x : b.y) : (i == 2 ? b.z : b.w);
}

// The `top` best columns of a row, sorted, into w.cand[0 .. top), for any row:
// batches that may beat the worst of the best so far are re-read in order, and
// a full candidate buffer is cut to the best.  Rows with many equal logits
// come here.
template <typename T>
__device__ __noinline__ void find_top_any(const LogprobParams& p, const Piece* piece, const BatchMax<T>* bm,
                                          long long row, unsigned bound, Scratch& w, int lane) {
  constexpr int EPV = Elem<T>::kPerVec;
  Best best;
  best.cand = w.cand;
  best.n = 0;
  best.top = p.top;
  // a word beats the floor if its key is at least `bound`
  best.floor = ((unsigned long long)bound << 32) > 0 ? ((unsigned long long)bound << 32) - 1 : 0ull;
  for (int i = 0; i < p.pieces; ++i) {
    const float4 b = bm[i * 32 + lane].get();
    for (int quarter = 0; quarter < 4; ++quarter) {
      // the columns of a batch are no lower than its first vector's
      const Piece pc = piece[i];
      const unsigned low = unsigned(pc.col) +
                           (pc.off == 0 ? 0u : unsigned(pc.off + 128 * quarter) * EPV);
      unsigned mk = __ballot_sync(kFull, word(value_key(quarter_max(b, quarter)), low) > best.floor);
      while (mk != 0) {
        // eight batches at a time, lowest lanes first
        int code = -1;
        for (int k = 0; k < 8 && mk != 0; ++k) {
          const int l = __ffs(mk) - 1;
          mk &= mk - 1;
          if ((lane >> 2) == k) code = i * 128 + quarter * 32 + l;
        }
        Batch<T> bt;
        bt.left = 0;
        bt.rag = nullptr;
        bt.src = nullptr;
        bt.col = bt.ragcol = 0;
        if (code >= 0) bt.at(p, piece, row, code, lane & 3);
        for (int step = 0; __any_sync(kFull, step < bt.left); ++step) {
          const bool has = step < bt.left;
          const uint4 q = has ? bt.src[step * kLpStep] : lp_pad(T());
          float x[EPV];
          unpack(q, x, T());
#pragma unroll 1
          for (int e = 0; e < EPV; ++e) {
            float xe = x[0];
#pragma unroll
            for (int f = 1; f < EPV; ++f) xe = e == f ? x[f] : xe;
            best.offer(has ? word(value_key(xe), unsigned(bt.col + step * kLpStep * EPV + e)) : 0ull, lane);
          }
        }
        const bool has = bt.rag != nullptr;
        best.offer(has ? word(value_key(Elem<T>::load(bt.rag)), unsigned(bt.ragcol)) : 0ull, lane);
      }
    }
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

// The top-th largest key among the lanes' four values (sorted here).
__device__ __forceinline__ unsigned bound_key(float4 x, int top) {
  unsigned a = value_key(x.x), b = value_key(x.y), c = value_key(x.z), d = value_key(x.w);
  auto order = [](unsigned& hi, unsigned& lo) {
    const unsigned h = max(hi, lo);
    lo = min(hi, lo);
    hi = h;
  };
  order(a, b);
  order(c, d);
  order(a, c);
  order(b, d);
  order(b, c);
  unsigned bound = 0;
  for (int seen = 0; seen < top;) {
    bound = __reduce_max_sync(kFull, a);
    const bool mine = a == bound;
    seen += __popc(__ballot_sync(kFull, mine));
    if (mine) {
      a = b;
      b = c;
      c = d;
      d = 0;
    }
  }
  return bound;
}

template <typename T>
__device__ __forceinline__ void finish_row(const LogprobParams& p, const Piece* piece, const BatchMax<T>* bm,
                                           const float4* sums, long long row, long long y, Scratch& w, int lane) {
  constexpr int EPV = Elem<T>::kPerVec;
  constexpr int kIn = 4;  // batches in flight per four lanes
  const float c = p.inv_t * kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  const bool in = p.targets != nullptr && y >= 0 && y < p.V;
  float zy = 0.f;
  if (in && lane == 0) {
    int i = 0;
    while (y >= p.sh.start[i + 1]) ++i;
    zy = Elem<T>::load(p.sh.ptr[i] + row * p.sh.ld_bytes[i] + (y - p.sh.start[i]) * Elem<T>::kBytes);
  }
  // the pieces' sums, two pieces a lane, added in a fixed tree
  const float4 none = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  const float4 s0 = lane < p.pieces ? sums[lane] : none, s1 = lane + 32 < p.pieces ? sums[lane + 32] : none;
  float M = max_nan(s0.x, s1.x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, o));
  const float K = offset_of(M, c);
  Acc a0{offset_of(s0.x, c), s0.y, s0.z}, a1{offset_of(s1.x, c), s1.y, s1.z};
  a0.raise(K);
  a1.raise(K);
  float S = a0.s + a1.s, W = a0.u + a1.u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(kFull, S, o);
    W += __shfl_xor_sync(kFull, W, o);
  }

  // list the batches that reach the bound
  unsigned bound = 0;
  float floor = 0.f;
  int listed = 0;
  if (p.top > 0) {
    // maxima of the lane's quarters over the pieces
    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll 4
    for (int i = 0; i < p.pieces; ++i) {
      const float4 b = bm[i * 32 + lane].get();
      x.x = max_nan(x.x, b.x);
      x.y = max_nan(x.y, b.y);
      x.z = max_nan(x.z, b.z);
      x.w = max_nan(x.w, b.w);
    }
    bound = bound_key(x, p.top);
    floor = key_value(bound);  // a NaN bound lists every batch
    if (lane == 0) w.n = 0;
    for (int i = 0; i < p.pieces; ++i) {
      const float4 b = bm[i * 32 + lane].get();
      const bool f[4] = {!(b.x < floor), !(b.y < floor), !(b.z < floor), !(b.w < floor)};
      if (!__any_sync(kFull, f[0] | f[1] | f[2] | f[3])) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned mk = __ballot_sync(kFull, f[k]);
        const int at = listed + __popc(mk & ((1u << lane) - 1u));
        if (f[k] && at < kLpList) w.list[at] = (unsigned short)(i * 128 + k * 32 + lane);
        listed += __popc(mk);
      }
    }
    __syncwarp();
  }
  const bool few = listed <= kLpList;
  Batch<T> bt[kIn];
  uint4 q[kIn];
  auto fetch = [&](int l0) {
#pragma unroll
    for (int k = 0; k < kIn; ++k) {
      const int l = l0 + 8 * k + (lane >> 2);
      bt[k].left = 0;
      if (l < listed) bt[k].at(p, piece, row, w.list[l], lane & 3);
      q[k] = bt[k].left > 0 ? *bt[k].src : lp_pad(T());
    }
  };
  if (p.top > 0 && few) fetch(0);

  // no finite largest logit (nothing unmasked, +inf or NaN): no distribution
  const bool ok = isfinite(M);
  float shift = fmaf(-M, c, K);  // K - c M, the rounding of K
  if (ok && !(fabsf(K) < kLpFar)) {
    const float2 far = sum_far<T>(p, row, M, c, lane);
    S = far.x;
    W = far.y;
    shift = 0.f;
  }
  const float ln2 = 0.6931471806f;
  const float ls = ok ? logf(S) + ln2 * shift : nan;
  const float ent = ok ? logf(S) - ln2 * (W / S) : nan;
  if (lane == 0) {
    if (p.entropy) p.entropy[row] = ent;
    if (p.stats) p.stats[row] = make_float4(M, ls, ent, 0.f);
    if (p.logp) p.logp[row] = in ? (zy - M) * p.inv_t - ls : nan;
    if (p.targets != nullptr && !in && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_BAD_TARGET);
  }
  if (p.top == 0) return;

  int n = kLpCand + 1;
  if (few) {
    auto offer = [&](float v, int col) {
      if (v < floor) return;
      const int at = atomicAdd(&w.n, 1);
      if (at < kLpCand) w.cand[at] = word(value_key(v), unsigned(col));
    };
    for (int l0 = 0;;) {
      for (int step = 0;;) {
#pragma unroll
        for (int k = 0; k < kIn; ++k) {
          if (step >= bt[k].left || lane_max(q[k], T()) < floor) continue;
          float v[EPV];
          unpack(q[k], v, T());
#pragma unroll
          for (int e = 0; e < EPV; ++e) offer(v[e], bt[k].col + step * kLpStep * EPV + e);
        }
        ++step;
        if (step * kLpStep >= p.len) break;
#pragma unroll
        for (int k = 0; k < kIn; ++k) q[k] = step < bt[k].left ? bt[k].src[step * kLpStep] : lp_pad(T());
      }
      l0 += 8 * kIn;
      if (l0 >= listed) break;
      fetch(l0);
    }
    // the ragged elements of the listed batches that have one
    for (int l = lane; l < listed; l += 32) {
      Batch<T> b;
      b.rag = nullptr;
      b.at(p, piece, row, w.list[l], 0);
      if (b.rag != nullptr) offer(Elem<T>::load(b.rag), b.ragcol);
    }
    __syncwarp();
    n = *(volatile int*)&w.n;
  }
  if (n <= 64) rank_words<2>(w.cand, n, p.top, lane);
  else if (n <= kLpCand) rank_words<kLpCand / 32>(w.cand, n, p.top, lane);
  else find_top_any<T>(p, piece, bm, row, bound, w, lane);
  if (lane < p.top) {
    const unsigned long long best = w.cand[lane];
    p.top_ids[row * p.top + lane] = (long long)unsigned(~unsigned(best));
    if (p.top_logp) p.top_logp[row * p.top + lane] = (key_value(unsigned(best >> 32)) - M) * p.inv_t - ls;
  }
  __syncwarp();
}

// The pieces of a row: every shard cut into ceil(vectors / len) of them, one
// at least.  One warp writes the table, a lane per shard.
template <typename T>
__device__ __forceinline__ void cut_row(const LogprobParams& p, Piece* piece, int lane) {
  int before = 0;
  for (int i0 = 0; i0 < p.t; i0 += 32) {
    const int i = i0 + lane;
    const int w = i < p.t ? int(p.sh.start[i + 1] - p.sh.start[i]) : 0;
    const int nv = w / Elem<T>::kPerVec;
    const int mine = i < p.t ? max(1, (nv + p.len - 1) / p.len) : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    for (int k = 0; k < mine; ++k)
      piece[before + upto - mine + k] = Piece{p.sh.ptr[i], p.sh.ld_bytes[i],
                                              unsigned(w) * unsigned(Elem<T>::kBytes), int(p.sh.start[i]), k * p.len};
    before += __shfl_sync(kFull, upto, 31);
  }
}

// Persistent form: a CTA per row at a time.  The streaming warps take pieces
// from a shared counter, run ahead into the next rows and leave partials in
// one of p.slots places; the finishing warps take the complete rows in turn.
// Finishing a row is a chain of dependent steps, longer than streaming one, so
// several rows are finished at a time; done by the streaming warps themselves,
// the same steps cost the stream its registers.
template <typename T>
__global__ void __launch_bounds__(kLpThreads<T>, 1)
    logprob_forward_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int kStream = LpShape<T>::kStream, kFinish = LpShape<T>::kFinish;
  extern __shared__ __align__(128) unsigned char lp_smem[];
  __shared__ Piece piece[kLpMaxPieces];
  __shared__ Scratch scratch[kFinish];
  __shared__ uint64_t full[kLpMaxSlots], empty[kLpMaxSlots], landed[kStream][2];
  __shared__ int next;  // pieces taken
  __shared__ volatile int stop;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // [ring | sums [slots][pieces] | batch maxima [slots][pieces][32]]
  float4* sums = reinterpret_cast<float4*>(lp_smem + kLpRing<T>);
  BatchMax<T>* maxima = reinterpret_cast<BatchMax<T>*>(sums + p.slots * p.pieces);
  if (threadIdx.x == 0) {
    next = 2 * kStream;
    stop = 0;
  }
  for (int i = threadIdx.x; i < p.slots; i += kLpThreads<T>) {
    mbar_init(&full[i], p.pieces);
    mbar_init(&empty[i], 1);
  }
  if (threadIdx.x < 2 * kStream) mbar_init(&landed[threadIdx.x / 2][threadIdx.x % 2], 1);
  fence_mbar_init();
  if (warp == kStream) cut_row<T>(p, piece, lane);
  __syncthreads();
  const int rows = int((p.s - blockIdx.x + gridDim.x - 1) / gridDim.x);  // this CTA's rows
  if (warp < kStream) {
    const float c = p.inv_t * kLog2e, floor = -2.f * kLpFar / c;
    const uint4* ring = reinterpret_cast<const uint4*>(lp_smem) + warp * kLpStep;
    uint64_t* bar = landed[warp];
    const uint64_t policy = policy_evict_first();
    const int units = p.len / kLpUnit;  // of a piece, an even number
    unsigned parity = 0;                // bit b: the phase of buffer b to wait for
    // piece i of the CTA's row k, and the one after it; a row's target is
    // loaded when the row is first taken, a piece ahead of its use
    struct Taken {
      int i, k;
      long long y;
    };
    auto settle = [&](Taken& x, int i, int k) {
      const int was = x.k;
      while (i >= p.pieces) {
        i -= p.pieces;
        ++k;
      }
      if (p.targets != nullptr && k != was && k < rows)
        x.y = __ldg(p.targets + blockIdx.x + (long long)k * gridDim.x);
      x.i = i;
      x.k = k;
    };
    // what a piece streams
    struct Stream {
      const uint4* v;  // its vectors
      int n;
      float ragged;
      bool live;       // a row of this CTA, not ignored
    };
    auto describe = [&](const Taken& x) {
      Stream q{nullptr, 0, -INFINITY, false};
      if (x.k >= rows || (p.targets != nullptr && x.y == p.ignore_index)) return q;
      const Piece pc = piece[x.i];
      const Seg g = segment<T>(pc, blockIdx.x + (long long)x.k * gridDim.x);
      q.v = body<T>(g) + pc.off;
      q.n = max(0, min(p.len, g.nv - pc.off));
      if (pc.off == 0 && (g.head | g.tail) != 0) q.ragged = ragged_value<T>(g, lane);
      q.live = true;
      return q;
    };
    // starts unit u of a piece into buffer u % 2 (an empty unit loads nothing)
    auto fetch = [&](const Stream& q, int u) {
      const int left = min(kLpUnit, q.n - u * kLpUnit);
      if (lane == 0 && left > 0) {
        uint64_t* b = &bar[u & 1];
        mbar_arrive_expect_tx(b, unsigned(left) * 16);
        bulk_load(const_cast<uint4*>(ring) + (u & 1) * kLpUnit, q.v + u * kLpUnit, unsigned(left) * 16, b, policy);
      }
    };
    Taken cur{0, -1, 0}, nxt;
    settle(cur, warp, 0);
    nxt = cur;
    settle(nxt, warp + kStream - cur.k * p.pieces, cur.k);
    Stream now = describe(cur);
    fetch(now, 0);
    fetch(now, 1);
    bool alive = true;
    while (cur.k < rows) {
      int taken = 0;
      if (lane == 0) taken = atomicAdd(&next, 1);
      const Stream then = describe(nxt);
      Acc a{-kLpFar, 0.f, 0.f};
      float4 bm = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      unsigned key = 0;  // of the piece's largest logit so far
      if (now.live) {
        float m0 = now.ragged, m1 = -INFINITY;  // the ragged element belongs to the first batch
#pragma unroll 1
        for (int u = 0; u < units; ++u) {
          const int n = now.n - u * kLpUnit, b = u & 1;
          uint4 q[kLpVecs];
          if (n > 0) {
            if (!mbar_wait_warp(&bar[b], parity >> b & 1)) {
              alive = false;
              break;
            }
            parity ^= 1u << b;
#pragma unroll
            for (int j = 0; j < kLpVecs; ++j) q[j] = ring[b * kLpUnit + lane + 32 * j];
            if (n < kLpUnit) {
#pragma unroll
              for (int j = 0; j < kLpVecs; ++j)
                if (lane + 32 * j >= n) q[j] = lp_pad(T());
            }
            m0 = max_nan(m0, vecs_max<kLpVecs / 2>(q, T()));
            m1 = max_nan(m1, vecs_max<kLpVecs / 2>(q + kLpVecs / 2, T()));
          }
          // every lane has its vectors once the warp has their maximum: only
          // then may the buffer be written again
          const unsigned was = key;
          key = max(key, __reduce_max_sync(kFull, value_key(max_nan(m0, m1))));
          if (key != 0u) {
            if (u + 2 < units) fetch(now, u + 2);
            else if (then.live) fetch(then, u + 2 - units);
          }
          if (key != was) {
            const float nk = offset_of(key_value(key), c);
            if (nk > a.k) a.raise(nk);
          }
          if (n > 0) unit_sums<T>(q, a, c, floor);
          if (u == 0 && now.ragged != -INFINITY) {
            const float v = fmaf(fmaxf(now.ragged, floor), c, -a.k), e = ex2(v);
            a.s += e;
            a.u = fmaf(v, e, a.u);
          }
          if (b == 0) {
            bm.x = max_nan(bm.x, m0);
            bm.y = max_nan(bm.y, m1);
          } else {
            bm.z = max_nan(bm.z, m0);
            bm.w = max_nan(bm.w, m1);
          }
          m0 = m1 = -INFINITY;
        }
        if (!alive) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          a.s += __shfl_xor_sync(kFull, a.s, o);
          a.u += __shfl_xor_sync(kFull, a.u, o);
        }
      } else if (then.live) {
        fetch(then, 0);
        fetch(then, 1);
      }
      const int slot = cur.k % p.slots, turn = cur.k / p.slots;
      if (turn > 0 && !mbar_wait_warp(&empty[slot], (turn - 1) & 1)) {
        alive = false;
        now = then;  // its copies are the ones in flight
        break;
      }
      if (now.live) {
        const int at = slot * p.pieces + cur.i;
        maxima[at * 32 + lane].set(bm);
        if (lane == 0) sums[at] = make_float4(key_value(key), a.s, a.u, 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&full[slot]);
      cur = nxt;
      now = then;
      settle(nxt, __shfl_sync(kFull, taken, 0) - cur.k * p.pieces, cur.k);
    }
    if (!alive) {
      stop = 1;
      // let this warp's copies land before the CTA leaves
      mbar_wait_warp(&bar[0], parity & 1);
      mbar_wait_warp(&bar[1], parity >> 1 & 1);
    }
  } else {
    for (int k = warp - kStream; k < rows && warp - kStream < p.team; k += p.team) {
      const long long row = blockIdx.x + (long long)k * gridDim.x;
      const long long y = p.targets != nullptr ? __ldg(p.targets + row) : 0;
      const int slot = k % p.slots;
      if (!mbar_wait_warp(&full[slot], (k / p.slots) & 1)) {
        stop = 1;
        break;
      }
      if (p.targets != nullptr && y == p.ignore_index) write_ignored(p, row, lane);
      else
        finish_row<T>(p, piece, maxima + slot * p.pieces * 32, sums + slot * p.pieces, row, y,
                      scratch[warp - kStream], lane);
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&empty[slot]);
    }
  }
  __syncthreads();
  if (stop) {  // a wait gave up: nothing of this CTA's rows is to be believed
    if (threadIdx.x == 0 && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_WAIT_TIMEOUT);
    const float nan = __int_as_float(0x7fc00000);
    for (int k = threadIdx.x; k < rows; k += kLpThreads<T>) {
      const long long row = blockIdx.x + (long long)k * gridDim.x;
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

// One step per piece, more when the row would have
// too many pieces.
template <typename T>
static void cut_plan(LogprobParams& p, int limit) {
  for (long long len = kLpStep;; len *= 2) {
    long long n = 0;
    for (int i = 0; i < p.t; ++i) {
      const long long nv = (p.sh.start[i + 1] - p.sh.start[i]) / Elem<T>::kPerVec;
      n += nv > 0 ? (nv + len - 1) / len : 1;
    }
    if (n <= limit || n == p.t) {
      p.pieces = int(n);
      p.len = int(len);
      return;
    }
  }
}

template <typename T>
void launch_logprob_forward(LogprobParams p, int sms, cudaStream_t st) {
  cut_plan<T>(p, kLpPieces);
  const int part = p.pieces * int(sizeof(float4) + 32 * sizeof(BatchMax<T>));
  // Slots.  Row k waits for row k - slots by a barrier's parity, which cannot
  // tell it from row k - 2 slots, so none may be two turns ahead of an
  // unfinished row r.  Rows r + slots, r + slots + team, .. are finished by
  // r's warp and block meanwhile (the others go on); all their pieces up to
  // row r + 2 slots are in the hands of streaming warps, which hold three at
  // most: (slots / team) * pieces >= 3 kStream rules it out.  And as slots is a
  // multiple of the team, a slot's rows are finished by one warp, in order.
  const int room = (kLpSmem - kLpRing<T>) / part;
  const int rows_each = (3 * LpShape<T>::kStream + p.pieces - 1) / p.pieces;  // slots per finishing warp
  p.team = LpShape<T>::kFinish;
  while (p.team > 1 && rows_each * p.team > room) --p.team;
  p.slots = rows_each * p.team;
  while (p.slots + p.team <= room && p.slots + p.team <= kLpSlots) p.slots += p.team;
  const int grid = int(p.s < sms ? p.s : sms);
  const size_t smem = kLpRing<T> + size_t(p.slots) * part;
  logprob_forward_kernel<T><<<grid, kLpThreads<T>, smem, st>>>(p);
}
template void launch_logprob_forward<float>(LogprobParams, int, cudaStream_t);
template void launch_logprob_forward<__nv_bfloat16>(LogprobParams, int, cudaStream_t);

cudaError_t set_logprob_smem() {
  const cudaError_t e = cudaFuncSetAttribute(logprob_forward_kernel<float>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kLpSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(logprob_forward_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kLpSmem);
}

}  // namespace vpce
