// The norm of rows off 16 bytes: h not a multiple of 8, or addresses or strides
// that are not whole vectors.  Read element by element from HBM these rows took
// twice the time (s = 30001, h = 515 fp32 52 us, with a residual 64); through the
// ring 25 and 44 us, 5.0 and 5.6 TB/s.  What bounds them now is a row's chain of
// steps (copies in, sum, output) with one CTA of 16 warps an SM; two CTAs with
// half the ring and half the registers each were slower (32 and 49 us).
#pragma once

#include "vpce_rmsnorm.cuh"

namespace vpce {
namespace {

// Rows off 16 bytes, through an OddRing (kStages rows of it; 0: none, rows are
// loaded when they are due).  For kShared, each 128, 64, 32 or 16 columns, the
// largest of these that a group is a multiple of, leave their maximum in shared
// memory, and the team's first threads join those of a group.
template <typename XT, typename RT, GroupKind kGroups, int kT, int kStages>
__global__ void __launch_bounds__(kT > 512 ? kT : 512, 1)
    rmsnorm_forward_odd_kernel(const __grid_constant__ RmsNormParams p, const OddRing ring, const GroupPlan og) {
  extern __shared__ uint4 smem[];  // [teams][groups' words, kStages rows]
  constexpr int kMaxTeams = kT > 512 ? 1 : 512 / kT, XB = Elem<XT>::kBytes, RB = Elem<RT>::kBytes;
  constexpr bool kRing = kStages > 0, kHoldWeights = kT <= 512;  // (64 registers a thread otherwise)
  __shared__ float red[kMaxTeams][2][32];
  [[maybe_unused]] __shared__ unsigned top_row[kMaxTeams][2][32];
  Team team;
  const int teams = blockDim.x / kT, lane = threadIdx.x & 31, h = p.h;
  team.id = threadIdx.x / kT;
  team.tid = threadIdx.x % kT;
  team.threads = kT;
  team.red = &red[team.id][0][0];
  const int tid = team.tid;
  const OddColumns<kT> columns(h, tid);
  float weight[kHoldWeights ? kOddColumns : 1];
  if constexpr (kHoldWeights)
    columns.each([&](int k, int c, bool) { weight[k] = load_weight(p.w, p.w_bf16, c); });
  const auto weight_of = [&](int k, int c) { return kHoldWeights ? weight[kHoldWeights ? k : 0] : load_weight(p.w, p.w_bf16, c); };

  const int stage_bytes = ring.bytes(p.res != nullptr ? 1 : 0);
  const int own = (kGroups == kShared ? og.bytes() : 0) + kStages * stage_bytes;
  unsigned char* const base = reinterpret_cast<unsigned char*>(smem) + team.id * own;
  const GroupWords words(base, og);
  unsigned char* const rows = base + (kGroups == kShared ? og.bytes() : 0);
  const auto fetch = [&](long long row, int stage) {
    if (row < p.s) {
      unsigned char* const dst = rows + stage * stage_bytes;
      copy_odd_row<XB, kT>(dst, p.x, row, p.ld_x, h, tid);
      if (p.res != nullptr) copy_odd_row<RB, kT>(dst + ring.first, p.res, row, p.ld_res, h, tid);
    }
    copy_commit();  // (an empty group past the end keeps the count)
  };

  const long long first = (long long)blockIdx.x * teams + team.id, stride = (long long)gridDim.x * teams;
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) fetch(first + i * stride, i);
  }
  int parity = 0, stage = 0;
  for (long long row = first; row < p.s; row += stride, parity ^= 1) {
    const unsigned char *xr = p.x + row * p.ld_x, *rr = p.res != nullptr ? p.res + row * p.ld_res : nullptr;
    if constexpr (kRing) {
      // this row's copies are in, everybody's; and everybody is done with the
      // stage of the row before, which is filled next
      copy_wait<(kRing ? kStages - 2 : 0)>();
      team.sync();
      fetch(row + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
      const unsigned char* const at = rows + stage * stage_bytes;
      xr = at + (uintptr_t(xr) & 15);
      if (rr != nullptr) rr = at + ring.first + (uintptr_t(rr) & 15);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    float r[kOddColumns], ss = 0.f;
    if (rr != nullptr) {
      unsigned char* const to = p.res_out + row * p.ld_res_out;
      // (lanes past the row read nothing that is written here: in place, without
      // a ring, column 0 may be)
      columns.each([&](int k, int c, bool inside) {
        r[k] = inside ? Elem<XT>::load(xr + c * XB) + Elem<RT>::load(rr + c * RB) : 0.f;
        ss = fmaf(r[k], r[k], ss);
        if (inside) Elem<RT>::store(to + c * RB, r[k]);
      });
    } else {
      columns.each([&](int k, int c, bool inside) {
        r[k] = inside ? Elem<XT>::load(xr + c * XB) : 0.f;
        ss = fmaf(r[k], r[k], ss);
      });
    }
    ss = team.sum(ss, parity);
    const float rstd = rsqrtf(ss / float(h) + p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
    unsigned char* const out = p.out + row * p.ld_out;
    [[maybe_unused]] unsigned all = 0;
    if constexpr (kGroups != kShared) {
      columns.each([&](int k, int c, bool inside) {
        r[k] = r[k] * rstd * weight_of(k, c);
        if constexpr (kGroups == kRow) all = max(all, inside ? mag(r[k]) : 0u);
        else if (inside) Elem<XT>::store(out + c * XB, r[k]);
      });
    } else {
      columns.by_quads([&](int q, int quad, bool whole) {
        unsigned m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = q * 4 + i, c = quad + i * 32 + lane;
          r[k] = r[k] * rstd * weight_of(k, whole || c < h ? c : 0);
          m[i] = whole || c < h ? mag(r[k]) : 0u;
        }
        unsigned* const to = words.tops + quad / og.segment;
        if (og.segment == 128) {
          const unsigned t = __reduce_max_sync(kFull, max(max(m[0], m[1]), max(m[2], m[3])));
          if (lane == 0) *to = t;
        } else if (og.segment == 64) {
          const unsigned t = __reduce_max_sync(kFull, max(m[0], m[1])), u = __reduce_max_sync(kFull, max(m[2], m[3]));
          if (lane < 2) to[lane] = lane == 0 ? t : u;
        } else if (og.segment == 32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned t = __reduce_max_sync(kFull, m[i]);
            if (lane == 0) to[i] = t;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(kFull, m[i], o));
            if ((lane & 15) == 0) to[2 * i + (lane >> 4)] = m[i];
          }
        }
      });
    }
    if constexpr (kGroups == kRow) {
      const float scale = e4m3_scale(team.max(all, top_row[team.id][parity])), inv = __frcp_rn(scale);
      const float s = isinf(scale) ? 0.f : scale;
      if (tid == 0) p.scale[row] = scale;
      columns.each([&](int k, int c, bool inside) {
        if (inside) store_code(out + c, quotient(r[k], s, inv));
      });
    } else if constexpr (kGroups == kShared) {
      team.sync();
      words.join(og, p.group, tid, kT, p.scale + row * og.groups);
      team.sync();
      columns.by_quads([&](int q, int quad, bool whole) {
        int g = group_of(p, quad);
        float scale = words.scales[g], inverse = words.inverses[g];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = q * 4 + i, c = quad + i * 32 + lane;
          if (og.segment < 128) {
            g = group_of(p, whole || c < h ? c : 0);
            scale = words.scales[g], inverse = words.inverses[g];
          }
          if (whole || c < h) store_code(out + c, quotient(r[k], scale, inverse));
        }
      });
    }
  }
  if constexpr (kRing) copy_wait<0>();  // (what was copied past the last row is nothing)
}

template <typename XT, typename RT, GroupKind kGroups, int kT, int kStages>
cudaError_t launch_odd(const RmsNormParams& p, int teams, const OddRing& ring, const GroupPlan& og, int sms, cudaStream_t st) {
  const auto kernel = rmsnorm_forward_odd_kernel<XT, RT, kGroups, kT, kStages>;
  const size_t smem = size_t(teams) * (kStages * ring.bytes(p.res != nullptr ? 1 : 0) + (kGroups == kShared ? og.bytes() : 0));
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const long long rows = (p.s + teams - 1) / teams;
  kernel<<<int(rows < sms ? rows : sms), kT * teams, smem, st>>>(p, ring, og);
  return cudaGetLastError();
}

template <typename XT, typename RT, GroupKind kGroups, int kT>
cudaError_t pick_odd(const RmsNormParams& p, int sms, cudaStream_t st) {
  const OddRing ring(p.h, sizeof(XT), sizeof(RT));
  const GroupPlan og(p, p.group % 128 == 0 ? 128 : p.group % 64 == 0 ? 64 : p.group % 32 == 0 ? 32 : 16, 128);
  const OddPlan plan(ring.bytes(p.res != nullptr ? 1 : 0), kGroups == kShared ? og.bytes() : 0, kT);
  if constexpr (kT <= 512)
    if (plan.stages == 3) return launch_odd<XT, RT, kGroups, kT, 3>(p, plan.teams, ring, og, sms, st);
  if constexpr (kT >= 512)  // (shorter rows always have a ring)
    if (plan.stages == 0) return launch_odd<XT, RT, kGroups, kT, 0>(p, plan.teams, ring, og, sms, st);
  return launch_odd<XT, RT, kGroups, kT, 2>(p, plan.teams, ring, og, sms, st);
}

template <typename XT, typename RT, GroupKind kGroups>
cudaError_t pick_odd(const RmsNormParams& p, int sms, cudaStream_t st) {
  // few warps a row: what a row costs besides its elements (sums, addresses) is
  // paid by every one of them
  if (p.h <= 1024) return pick_odd<XT, RT, kGroups, 32>(p, sms, st);
  if (p.h <= 4096) return pick_odd<XT, RT, kGroups, 128>(p, sms, st);
  if (p.h <= 16384) return pick_odd<XT, RT, kGroups, 512>(p, sms, st);
  return pick_odd<XT, RT, kGroups, 1024>(p, sms, st);
}

}  // namespace

template <typename XT, typename RT> cudaError_t rmsnorm_forward_odd(const RmsNormParams& p, GroupKind kind, int sms, cudaStream_t st) {
  if (kind == kNoCodes) return pick_odd<XT, RT, kNoCodes>(p, sms, st);
  return kind == kRow ? pick_odd<XT, RT, kRow>(p, sms, st) : pick_odd<XT, RT, kShared>(p, sms, st);
}

}  // namespace vpce
