// Scaled embedding lookup with dropout, and its gradient by sorted tokens.
//
//     out[r, c] = f m(r, c) E[id_r, c],   f = scale * 65536 / (65536 - D),
// with m(r, c) = 0 where the 16 random bits of (r, c) are below D and 1
// elsewhere.  The bits come from a counter-based generator keyed by the call's
// (seed, offset), so the gradient forms the same mask again and no mask is
// stored.  One generator block serves 8 columns, the 16 bytes a lane moves.
//
// Gradient: dE[v, c] = f sum over the rows r of token v, ascending, of
// m(r, c) g[r, c].  Two launches.
//   sort   CTA b owns the ids congruent to b (so that frequent ids, which are
//          neighbours in most vocabularies, spread).  It reads all ids once to
//          count the tokens of the CTAs before it (its place in the sorted
//          order) and once to collect its own in row order, and sorts those by
//          a stable counting sort in shared memory: no passes over the whole
//          batch and no grid barrier.
//   sum    A warp per task of 256 columns: a segment of at most 64 rows of a
//          run longer than kLong (the last segment to finish adds a run's
//          partial sums in order), or the runs that start in 16 sorted rows, up
//          to 16 rows' loads in flight.  Then, when the table is overwritten,
//          the rows of ids that do not occur.
//
// Measured at s = 8192 Zipf ids, h = 8192, V = 128256, bf16, dropout 0.1: the
// lookup 0.055 ms and 0.042 without dropout, against 0.026 ms of HBM traffic
// (output and distinct rows): the generator adds 0.013, and the other 0.016 is a
// warp's chain of id, shard, loads and store, with nothing of another unit under
// way in it (how it divides is not measured).  The sort 0.012 ms; the gradient
// 0.62 ms written in full (4.2 GB of table, 6.9 TB/s) and 0.11 ms accumulated,
// against 0.046 ms for the gradient rows and the distinct table rows read and
// written: the SMs work 44% of the sum's time on average (h = 2048), the rest is
// waiting for the last of them.  Longer segments cost more (128 rows: 0.123 ms
// accumulated), and so did long runs summed by whole CTAs (0.142 ms).  Segment
// length and the sort's 128 CTAs were chosen on Zipf ids at this h.
#include <climits>

#include "vpce_embed_dropout.cuh"

namespace vpce {

namespace {

constexpr int kEdThreads = 256;
constexpr int kEdWarps = kEdThreads / 32;

__device__ __forceinline__ int shard_holding(const ShardSet& sh, int t, long long id) {
  int lo = 0, hi = t;  // start[lo] <= id < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.start[mid] <= id) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// eight columns at a time
// ---------------------------------------------------------------------------
template <typename T> struct Eight;  // as loaded
template <> struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack(v, x, __nv_bfloat16()); }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
__device__ __forceinline__ void clear(Eight<__nv_bfloat16>& e) { e.v = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void clear(Eight<float>& e) { e.a = e.b = make_float4(0.f, 0.f, 0.f, 0.f); }

// Columns [0, n) of eight at p (n <= 8; the others 0).  vec: p is 16-byte
// aligned.
__device__ __forceinline__ void load8(Eight<__nv_bfloat16>& e, const unsigned char* p, int n, bool vec) {
  if (vec && n == 8) {
    e.v = __ldcs(reinterpret_cast<const uint4*>(p));
    return;
  }
  const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
  unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 1] |= unsigned(__ldg(h + j)) << (16 * (j & 1));
  e.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(Eight<float>& e, const unsigned char* p, int n, bool vec) {
  const float4* q = reinterpret_cast<const float4*>(p);
  if (vec && n == 8) {
    e.a = __ldcs(q);
    e.b = __ldcs(q + 1);
    return;
  }
  const float* f = reinterpret_cast<const float*>(p);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = j < n ? __ldg(f + j) : 0.f;
  e.a = make_float4(x[0], x[1], x[2], x[3]);
  e.b = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(unsigned char* p, const float (&x)[8], int n, bool vec, __nv_bfloat16) {
  if (vec && n == 8) {
    __stcs(reinterpret_cast<uint4*>(p), pack(x, __nv_bfloat16()));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) Elem<__nv_bfloat16>::store(p + 2 * j, x[j]);
}
__device__ __forceinline__ void store8(unsigned char* p, const float (&x)[8], int n, bool vec, float) {
  if (vec && n == 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) reinterpret_cast<float*>(p)[j] = x[j];
}

// Zeroes the dropped ones of eight values.  A word's high half is below D
// where the word is below D << 16, its low half where the word shifted up is.
__device__ __forceinline__ void drop8(float (&x)[8], const uint4& bits, unsigned limit) {
  const unsigned w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = (w[i] << 16) < limit ? 0.f : x[2 * i];
    x[2 * i + 1] = w[i] < limit ? 0.f : x[2 * i + 1];
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
constexpr int kEfBlocks = 4;  // 8-column blocks per lane and unit

// One unit per warp: kEfBlocks * 256 columns of a row.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kEdThreads) embed_dropout_forward_kernel(const __grid_constant__ EmbedDropParams p) {
  constexpr int IB = Elem<TI>::kBytes, OB = Elem<TO>::kBytes;
  const int lane = threadIdx.x & 31;
  const long long per = (p.h + 256 * kEfBlocks - 1) / (256 * kEfBlocks);
  const long long w = (long long)blockIdx.x * kEdWarps + (threadIdx.x >> 5);
  const long long r = w / per;
  if (r >= p.s) return;
  const long long c0 = (w - r * per) * (256 * kEfBlocks) + lane * 8;
  const long long id = __ldg(p.ids + r);
  // INT64_MIN as padding id means none: an id of that value is out of range
  const bool pad = id == p.padding_id && id != LLONG_MIN, in = id >= 0 && id < p.V, live = in && !pad;
  if (!in && !pad && lane == 0 && p.flag != nullptr) atomicOr(p.flag, VPCE_FLAG_BAD_TARGET);
  const int i = live ? shard_holding(p.sh, p.t, id) : 0;
  const unsigned char* src = live ? p.sh.ptr[i] + (id - p.sh.start[i]) * p.sh.ld_bytes[i] : nullptr;
  unsigned char* dst = p.out + r * p.ld_out_bytes;
  const bool vi = (reinterpret_cast<uintptr_t>(src) & 15) == 0, vo = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
  Eight<TI> q[kEfBlocks];
#pragma unroll
  for (int k = 0; k < kEfBlocks; ++k) {
    const long long c = c0 + 256 * k;
    if (live && c < p.h) load8(q[k], src + c * IB, int(min(8LL, p.h - c)), vi);
    else clear(q[k]);
  }
  DropKey key;
  if (p.drop) key.set(p.rng);
  const unsigned limit = p.drop << 16;
#pragma unroll
  for (int k = 0; k < kEfBlocks; ++k) {
    const long long c = c0 + 256 * k;
    if (c >= p.h) break;
    uint4 bits = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (p.drop && live) bits = drop_block(key, r, unsigned(c >> 3));
    float x[8];
    q[k].get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= p.factor;
    drop8(x, bits, limit);
    store8(dst + c * OB, x, int(min(8LL, p.h - c)), vo, TO());
  }
}

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 1024;  // bins of one counting pass
constexpr int kLong = 64;      // runs with more rows are summed in segments
constexpr int kGroup = 16;     // sorted rows per warp task
constexpr int kSeg = 64;       // rows of a long run per warp task
constexpr int kSegShare = 32;  // n sorted tokens hold at most n / 32 segments: ceil(L / 64) <= L / 32 for L > 64
constexpr int kOwnBits = 7;    // the sort's CTAs: 2^kOwnBits
constexpr int kOwners = 1 << kOwnBits;
template <typename T> constexpr int kInFlight = sizeof(T) == 2 ? 16 : 8;  // rows' loads per lane

struct Segment {
  int at, rows;      // its first sorted position, its rows
  int first, count;  // the run's first segment and how many it has
};

struct SortHead {
  long long valid;           // tokens with a gradient
  unsigned long long taken;  // the zero rows' task counter
};

struct SortParams {
  const long long* ids;
  long long s;
  long long V;
  long long padding_id;
  int range;          // local ids (id / kOwners) of a CTA
  int words;          // of a CTA's part of `present`
  int blocks;         // column blocks of the sum
  int* row[2];        // [s] rows, before and after a pass
  int* key[2];        // [s] local ids
  int* sorted_id;     // [s]
  int* sorted_row;    // [s]
  unsigned* present;  // [kOwners][words], a bit per local id
  Segment* segs;      // of the long runs; a CTA's from its first position / kSegShare on
  int2* lists;        // per CTA: first of its segments, how many
  int* done;          // [segments][blocks], cleared at each run's first segment
  SortHead* head;
};

// Exclusive scan of one int per thread of the CTA, and the total.
__device__ __forceinline__ int cta_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kSortWarps; ++w) {
    before += w < warp ? tmp[w] : 0;
    total += tmp[w];
  }
  return before + x - v;
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ int count[];  // [warps][kDigits]
  __shared__ int nseg;
  __shared__ int tmp[kSortWarps], wmine[kSortWarps], wlow[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int own = blockIdx.x;
  auto owner = [&](long long id) {  // kOwners and more: no gradient
    return id >= 0 && id < p.V && id != p.padding_id ? int(id) & (kOwners - 1) : kOwners;
  };
  // this warp's slice of the ids
  const long long per = ((p.s + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const long long r0 = warp * per, r1 = min(p.s, r0 + per);
  int mine = 0, low = 0;
#pragma unroll 8
  for (long long r = r0 + lane; r < r1; r += 32) {
    const long long id = __ldg(p.ids + r);
    const int o = owner(id);
    mine += o == own;
    low += o < own;
  }
  mine = __reduce_add_sync(kFull, mine);
  low = __reduce_add_sync(kFull, low);
  if (lane == 0) {
    wmine[warp] = mine;
    wlow[warp] = low;
  }
  unsigned* present = p.present + (long long)own * p.words;
  for (int i = tid; i < p.words; i += kSortThreads) present[i] = 0u;
  if (own == 0 && tid == 0) p.head->taken = 0;
  if (tid == 0) nseg = 0;
  __syncthreads();
  int n = 0, at = 0;
  long long base = 0;
  for (int w = 0; w < kSortWarps; ++w) {
    at += w < warp ? wmine[w] : 0;
    n += wmine[w];
    base += wlow[w];
  }
  if (own == kOwners - 1 && tid == 0) p.head->valid = base + n;
  if (n == 0) {
    if (tid == 0) p.lists[own] = make_int2(0, 0);
    return;
  }
  const int first_seg = int(base / kSegShare);
  int *key = p.key[0] + base, *row = p.row[0] + base, *key2 = p.key[1] + base, *row2 = p.row[1] + base;
  if (mine > 0) {
    for (long long r = r0; r < r1; r += 256) {
      long long id[8];  // eight loads in flight
#pragma unroll
      for (int j = 0; j < 8; ++j) id[j] = r + 32 * j + lane < r1 ? __ldg(p.ids + r + 32 * j + lane) : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = owner(id[j]) == own;
        const unsigned m = __ballot_sync(kFull, in);
        if (in) {
          const int k = at + __popc(m & ((1u << lane) - 1u));
          key[k] = int(id[j] >> kOwnBits);
          row[k] = int(r) + 32 * j + lane;
        }
        at += __popc(m);
      }
    }
  }
  // stable counting passes, kDigits bins each; the warps take contiguous
  // slices of the list (fewer warps for short lists: less to clear and scan)
  const int warps = min(kSortWarps, (n + 127) / 128);
  const int slice = ((n + warps - 1) / warps + 31) / 32 * 32;
  for (int shift = 0; shift == 0 || ((p.range - 1) >> shift) > 0; shift += 10) {
    const int bins = min(kDigits, ((p.range - 1) >> shift) + 1);
    for (int i = tid; i < warps * kDigits; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const int k0 = min(n, warp * slice), k1 = warp < warps ? min(n, k0 + slice) : k0;
    int* mycount = count + warp * kDigits;
    for (int k = k0; k < k1; k += 32) {
      const bool in = k + lane < k1;
      const int d = in ? (key[k + lane] >> shift) & (kDigits - 1) : -1;
      const unsigned m = __match_any_sync(kFull, d);
      if (in && lane == __ffs(m) - 1) mycount[d] += __popc(m);
      __syncwarp();
    }
    __syncthreads();
    int sum = 0;
    if (tid < bins)
      for (int w = 0; w < warps; ++w) sum += count[w * kDigits + tid];
    int total;
    int pos = cta_scan(sum, tmp, total);
    if (tid < bins)
      for (int w = 0; w < warps; ++w) {
        const int x = count[w * kDigits + tid];
        count[w * kDigits + tid] = pos;
        pos += x;
      }
    __syncthreads();
    for (int k = k0; k < k1; k += 32) {
      const bool in = k + lane < k1;
      const int kk = in ? key[k + lane] : 0;
      const int d = in ? (kk >> shift) & (kDigits - 1) : -1;
      const unsigned m = __match_any_sync(kFull, d);
      if (in) {
        const int to = mycount[d] + __popc(m & ((1u << lane) - 1u));
        key2[to] = kk;
        row2[to] = row[k + lane];
      }
      __syncwarp();
      if (in && lane == __ffs(m) - 1) mycount[d] += __popc(m);
      __syncwarp();
    }
    __syncthreads();
    int* x = key;
    key = key2;
    key2 = x;
    x = row;
    row = row2;
    row2 = x;
  }
  // sorted ids and rows, the ids that occur, the long runs
  for (int k = tid; k < n; k += kSortThreads) {
    const int kk = key[k];
    p.sorted_id[base + k] = (kk << kOwnBits) + own;
    p.sorted_row[base + k] = row[k];
    if (k == 0 || key[k - 1] != kk) {
      atomicOr(present + kk / 32, 1u << (kk & 31));
      if (k + kLong < n && key[k + kLong] == kk) {
        int a = k + kLong, b = n;  // the run's end is in (a, b]
        while (b - a > 1) {
          const int mid = a + (b - a) / 2;
          if (key[mid] == kk) a = mid;
          else b = mid;
        }
        const int rows = b - k, count = (rows + kSeg - 1) / kSeg;
        const int first = first_seg + atomicAdd(&nseg, count);
        for (int i = 0; i < count; ++i)
          p.segs[first + i] = Segment{int(base) + k + i * kSeg, min(kSeg, rows - i * kSeg), first, count};
        for (int i = 0; i < p.blocks; ++i) p.done[(long long)first * p.blocks + i] = 0;
      }
    }
  }
  __syncthreads();
  if (tid == 0) p.lists[own] = make_int2(first_seg, nseg);
}

// ---------------------------------------------------------------------------
// sum
// ---------------------------------------------------------------------------
struct SumParams {
  EmbedDropParams e;  // e.sh: the gradient shards; e.out: the gradient rows
  const int* id;
  const int* row;
  const unsigned* present;
  int words;
  const Segment* segs;
  const int2* lists;
  int* done;
  float* part;        // [segments][blocks * 256] partial sums
  SortHead* head;
};

// a run's eight columns into the table: one store, or one addition that needs
// no answer (each element gets one, so the order cannot matter)
__device__ __forceinline__ void put8(float* p, const float (&x)[8], int n, bool vec, int accumulate) {
  if (vec && n == 8) {
    if (accumulate) {
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
                   : "memory");
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + 4), "f"(x[4]), "f"(x[5]), "f"(x[6]),
                   "f"(x[7])
                   : "memory");
    } else {
      __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (accumulate) p[j] += x[j];
      else p[j] = x[j];
    }
}

__device__ __forceinline__ float* table_row(const EmbedDropParams& e, int id) {
  const int i = shard_holding(e.sh, e.t, id);
  return reinterpret_cast<float*>(const_cast<unsigned char*>(e.sh.ptr[i]) + (id - e.sh.start[i]) * e.sh.ld_bytes[i]);
}

template <typename T>
struct RowSource {
  const EmbedDropParams& e;
  DropKey key;
  unsigned limit;
  long long c;  // the lane's first column
  int n;        // columns it has, 0..8
  bool vec;     // gradient rows are 16-byte aligned
  __device__ __forceinline__ void load(Eight<T>& q, int r) const {
    if (n > 0) load8(q, e.out + r * e.ld_out_bytes + c * Elem<T>::kBytes, n, vec);
    else clear(q);
  }
  __device__ __forceinline__ void add(float (&acc)[8], const Eight<T>& q, int r) const {
    float x[8];
    q.get(x);
    if (e.drop) drop8(x, drop_block(key, r, unsigned(c >> 3)), limit);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += x[j];
  }
};

template <typename T>
__global__ void __launch_bounds__(kEdThreads, 2) embed_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ int upto[kOwners];  // segments of the lists so far
  constexpr int kIn = kInFlight<T>;
  const EmbedDropParams& e = p.e;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = int((e.h + 255) / 256);  // column blocks of a warp
  RowSource<T> src{e, {}, e.drop << 16, 0, 0, ((reinterpret_cast<uintptr_t>(e.out) | e.ld_out_bytes) & 15) == 0};
  if (e.drop) src.key.set(e.rng);
  auto columns = [&](int block) {
    src.c = (long long)block * 256 + lane * 8;
    src.n = int(max(0LL, min(8LL, e.h - src.c)));
  };
  auto flush = [&](float* row, float (&acc)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= e.factor;
    float* at = row + src.c;
    if (src.n > 0) put8(at, acc, src.n, (reinterpret_cast<uintptr_t>(at) & 15) == 0, e.accumulate);
  };
  if (warp == 0) {
    int carry = 0;
#pragma unroll
    for (int i0 = 0; i0 < kOwners; i0 += 32) {
      int x = p.lists[i0 + lane].y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      upto[i0 + lane] = carry + x;
      carry += __shfl_sync(kFull, x, 31);
    }
  }
  __syncthreads();
  const int valid = int(p.head->valid);
  const long long groups = (valid + kGroup - 1) / kGroup;
  const long long nsegs = upto[kOwners - 1];
  const long long tasks = (nsegs + groups) * blocks, nw = (long long)gridDim.x * kEdWarps;
  // long tasks first; neighbouring warps take neighbouring columns
  for (long long tk = (long long)blockIdx.x * kEdWarps + warp; tk < tasks; tk += nw) {
    const long long unit = tk / blocks;
    const int block = int(tk - unit * blocks);
    columns(block);
    float acc[8] = {};
    if (unit < nsegs) {
      // a segment of a long run
      int l = 0;  // the list that holds it: the first with upto > unit
#pragma unroll
      for (int step = kOwners / 2; step > 0; step >>= 1)
        if (upto[l + step - 1] <= unit) l += step;
      const int slot = p.lists[l].x + int(unit) - (l > 0 ? upto[l - 1] : 0);
      const Segment sg = p.segs[slot];
      for (int k = 0; k < sg.rows; k += 32) {
        const int m = min(32, sg.rows - k);
        const int r32 = lane < m ? p.row[sg.at + k + lane] : 0;
        for (int b = 0; b < m; b += kIn) {
          Eight<T> q[kIn];
#pragma unroll
          for (int j = 0; j < kIn; ++j) {
            const int r = __shfl_sync(kFull, r32, b + j);
            if (b + j < m) src.load(q[j], r);
            else clear(q[j]);
          }
#pragma unroll
          for (int j = 0; j < kIn; ++j) {
            const int r = __shfl_sync(kFull, r32, b + j);
            if (b + j < m) src.add(acc, q[j], r);
          }
        }
      }
      if (sg.count > 1) {
        // leave the partial sum; the run's last segment to get here adds them
        const long long width = (long long)blocks * 256;
        float4* mine = reinterpret_cast<float4*>(p.part + slot * width + src.c);
        __stcg(mine, make_float4(acc[0], acc[1], acc[2], acc[3]));
        __stcg(mine + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
        __threadfence();
        __syncwarp();
        int arrived = 0;
        if (lane == 0) arrived = atomicAdd(p.done + (long long)sg.first * blocks + block, 1);
        if (__shfl_sync(kFull, arrived, 0) != sg.count - 1) continue;
        __threadfence();
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 4
        for (int i = 0; i < sg.count; ++i) {
          const float4* at = reinterpret_cast<const float4*>(p.part + (sg.first + i) * width + src.c);
          const float4 x = __ldcg(at), y = __ldcg(at + 1);
          acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
          acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
        }
      }
      flush(table_row(e, p.id[sg.at]), acc);
      continue;
    }
    // the runs that start in a group of 16 sorted rows
    const int g = int(unit - nsegs) * kGroup;
    float* cur = nullptr;  // table row of the run being summed
    bool done = false;
    for (int k = g; !done; k += kGroup) {
      // 16 positions; lane l holds position k + l
      const int pos = k + lane;
      const bool here = lane < kGroup && pos < valid;
      const int id = here ? p.id[pos] : -1;
      const int r16 = here ? p.row[pos] : 0;
      const int prev = here && pos > 0 ? p.id[pos - 1] : -1;
      const int far = here && pos + kLong < valid ? p.id[pos + kLong] : -1;
      const bool head = here && id != prev;
      const unsigned heads = __ballot_sync(kFull, head), longs = __ballot_sync(kFull, head && far == id),
                     heres = __ballot_sync(kFull, here);
      float* trow = head ? table_row(e, id) : nullptr;
      // the positions to sum: from the group's first head (past the group, from
      // the start) to the first head past the group or the first long run
      int a = 0, b = __popc(heres);
      if (k == g) {
        if (heads == 0) break;
        a = __ffs(heads) - 1;
      } else if (heads != 0) {
        b = __ffs(heads) - 1;
      }
      if (longs != 0) b = min(b, __ffs(longs) - 1);
      done = b < kGroup;
      for (int part = 0; part < kGroup; part += kIn) {
        if (part >= b) break;
        Eight<T> q[kIn];
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          const int j = part + i, r = __shfl_sync(kFull, r16, j);
          if (j >= a && j < b) src.load(q[i], r);
          else clear(q[i]);
        }
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          const int j = part + i, r = __shfl_sync(kFull, r16, j);
          const unsigned long long t = __shfl_sync(kFull, reinterpret_cast<unsigned long long>(trow), j);
          if (j < a || j >= b) continue;
          if (heads >> j & 1u) {
            if (cur != nullptr) flush(cur, acc);
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[x] = 0.f;
            cur = reinterpret_cast<float*>(t);
          }
          src.add(acc, q[i], r);
        }
      }
    }
    if (cur != nullptr) flush(cur, acc);
  }
  if (e.accumulate) return;

  // rows of ids that do not occur: about 64 KB per warp task
  const int each = int(max(1LL, min(32LL, 16384 / e.h)));
  const long long zero_tasks = (e.V + each - 1) / each;
  while (true) {
    unsigned long long got = 0;
    if (lane == 0) got = atomicAdd(&p.head->taken, 1ull);
    const long long tk = (long long)__shfl_sync(kFull, got, 0);
    if (tk >= zero_tasks) break;
    const long long mine = tk * each + lane;
    bool absent = false;
    if (lane < each && mine < e.V) {
      const int local = int(mine >> kOwnBits);
      absent = !(p.present[(mine & (kOwners - 1)) * p.words + local / 32] >> (local & 31) & 1u);
    }
    unsigned todo = __ballot_sync(kFull, absent);
    while (todo != 0) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      float* row = table_row(e, int(tk * each + l));
      // 16-byte stores between ragged ends
      const int head = min(int(e.h), int((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 4);
      const int nv = (int(e.h) - head) / 4, tail = int(e.h) - head - 4 * nv;
      float4* v = reinterpret_cast<float4*>(row + head);
#pragma unroll 4
      for (int i = lane; i < nv; i += 32) __stcs(v + i, make_float4(0.f, 0.f, 0.f, 0.f));
      if (lane < head) row[lane] = 0.f;
      if (lane < tail) row[head + 4 * nv + lane] = 0.f;
    }
  }
}

}  // namespace

long long embed_dropout_forward_blocks(long long s, long long h) {
  const long long units = s * ((h + 256 * kEfBlocks - 1) / (256 * kEfBlocks));
  return (units + kEdWarps - 1) / kEdWarps;
}

void launch_embed_dropout_forward(const EmbedDropParams& p, bool table_bf16, bool out_bf16, cudaStream_t st) {
  const unsigned grid = unsigned(embed_dropout_forward_blocks(p.s, p.h));
  if (table_bf16 && out_bf16) embed_dropout_forward_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kEdThreads, 0, st>>>(p);
  else if (table_bf16) embed_dropout_forward_kernel<__nv_bfloat16, float><<<grid, kEdThreads, 0, st>>>(p);
  else if (out_bf16) embed_dropout_forward_kernel<float, __nv_bfloat16><<<grid, kEdThreads, 0, st>>>(p);
  else embed_dropout_forward_kernel<float, float><<<grid, kEdThreads, 0, st>>>(p);
}

namespace {

struct EdLayout {
  size_t head, lists, row[2], key[2], sid, srow, present, segs, done, part, total;
  int range, words, blocks;
  EdLayout(long long s, long long V, long long h) {
    const size_t n = round256(sizeof(int) * size_t(s)), slots = size_t(s / kSegShare + 1);
    range = int((V + kOwners - 1) / kOwners);
    words = (range + 31) / 32;
    blocks = int((h + 255) / 256);
    head = 0;
    lists = 256;
    size_t at = lists + round256(sizeof(int2) * kOwners);
    for (int i = 0; i < 2; ++i) {
      row[i] = at;
      key[i] = at + n;
      at += 2 * n;
    }
    sid = at;
    srow = sid + n;
    present = srow + n;
    segs = present + round256(sizeof(unsigned) * size_t(kOwners) * size_t(words));
    done = segs + round256(sizeof(Segment) * slots);
    part = done + round256(sizeof(int) * slots * size_t(blocks));
    total = part + sizeof(float) * slots * size_t(blocks) * 256;
  }
};
constexpr size_t kSortSmem = sizeof(int) * kSortWarps * kDigits;

}  // namespace

size_t embed_dropout_workspace_bytes(long long s, long long V, long long h) { return EdLayout(s, V, h).total; }

cudaError_t launch_embed_dropout_backward(const EmbedDropParams& p, bool grad_bf16, void* ws, int sms,
                                          cudaStream_t st) {
  const EdLayout L(p.s, p.V, p.h);
  unsigned char* w = static_cast<unsigned char*>(ws);
  SortParams q;
  q.ids = p.ids;
  q.s = p.s;
  q.V = p.V;
  q.padding_id = p.padding_id;
  q.range = L.range;
  q.words = L.words;
  q.blocks = L.blocks;
  for (int i = 0; i < 2; ++i) {
    q.row[i] = reinterpret_cast<int*>(w + L.row[i]);
    q.key[i] = reinterpret_cast<int*>(w + L.key[i]);
  }
  q.sorted_id = reinterpret_cast<int*>(w + L.sid);
  q.sorted_row = reinterpret_cast<int*>(w + L.srow);
  q.present = reinterpret_cast<unsigned*>(w + L.present);
  q.segs = reinterpret_cast<Segment*>(w + L.segs);
  q.lists = reinterpret_cast<int2*>(w + L.lists);
  q.done = reinterpret_cast<int*>(w + L.done);
  q.head = reinterpret_cast<SortHead*>(w + L.head);
  embed_sort_kernel<<<kOwners, kSortThreads, kSortSmem, st>>>(q);
  SumParams u;
  u.e = p;
  u.id = q.sorted_id;
  u.row = q.sorted_row;
  u.present = q.present;
  u.words = L.words;
  u.segs = q.segs;
  u.lists = q.lists;
  u.done = q.done;
  u.part = reinterpret_cast<float*>(w + L.part);
  u.head = q.head;
  const int grid = sms * 2;
  if (grad_bf16) embed_sum_kernel<__nv_bfloat16><<<grid, kEdThreads, 0, st>>>(u);
  else embed_sum_kernel<float><<<grid, kEdThreads, 0, st>>>(u);
  return cudaGetLastError();
}

cudaError_t set_embed_dropout_smem() {
  return cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSortSmem));
}

}  // namespace vpce
