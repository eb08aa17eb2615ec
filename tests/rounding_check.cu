// Counts where root2, quotient and quotient2 of vpce_rows.cuh differ from CUDA's
// correctly rounded root and quotient: every fp32 value from 2^-100 to 2^127,
// and quotients of 2^-17 to 2^8 by scales of each exponent.  Prints three counts
// for scales from 2^-95 up (roots, quotients, pairs), the largest difference in
// ulps below, and how many quotients were looked at.
#include <cstdio>

#include "vpce_rows.cuh"

using namespace vpce;

__device__ unsigned long long bad_roots, bad_quotients, bad_pairs, seen, ulps_below;

__global__ void roots() {
  const unsigned exponent = blockIdx.y + 27;
  for (unsigned m = blockIdx.x * blockDim.x + threadIdx.x; m < (1u << 23); m += gridDim.x * blockDim.x) {
    const float v = __uint_as_float(exponent << 23 | m);
    float a, b;
    f2_unpack(root2(both(v)), a, b);
    if (a != __fsqrt_rn(v) || b != a) atomicAdd(&bad_roots, 1ull);
  }
}

__device__ unsigned next(unsigned& s) {
  s ^= s << 13;
  s ^= s >> 17;
  s ^= s << 5;
  return s;
}

__global__ void quotients() {
  unsigned state = (blockIdx.x * blockDim.x + threadIdx.x) * 2654435761u + 12345u + blockIdx.y * 97u;
  if (state == 0) state = 1;
  const unsigned exponent = blockIdx.y + 1;
  for (int i = 0; i < 64; ++i) {
    const float s = __uint_as_float(exponent << 23 | (next(state) & 0x7fffffu));
    const float about = __uint_as_float((110u + next(state) % 25) << 23 | (next(state) & 0x7fffffu));
    const float x = __uint_as_float(__float_as_uint(s * about) + (next(state) & 3) - 1);
    if (!(x < 1e38f) || !(x > 0.f)) continue;
    const float inv = __frcp_rn(s), want = __fdiv_rn(x, s), got = quotient(x, s, inv);
    float a, b;
    f2_unpack(quotient2(f2_pack(x, -x), both(-s), both(inv)), a, b);
    if (exponent >= 127 - 95) {
      atomicAdd(&seen, 1ull);
      if (got != want) atomicAdd(&bad_quotients, 1ull);
      if (a != want || b != -want) atomicAdd(&bad_pairs, 1ull);
    } else {
      const int d = int(__float_as_uint(got)) - int(__float_as_uint(want));
      atomicMax(&ulps_below, (unsigned long long)(d < 0 ? -d : d));
    }
  }
}

int main() {
  roots<<<dim3(256, 227), 256>>>();
  quotients<<<dim3(64, 245), 256>>>();
  if (cudaDeviceSynchronize() != cudaSuccess) return 1;
  unsigned long long r = 0, q = 0, p = 0, n = 0, u = 0;
  cudaMemcpyFromSymbol(&r, bad_roots, sizeof(r));
  cudaMemcpyFromSymbol(&q, bad_quotients, sizeof(q));
  cudaMemcpyFromSymbol(&p, bad_pairs, sizeof(p));
  cudaMemcpyFromSymbol(&n, seen, sizeof(n));
  cudaMemcpyFromSymbol(&u, ulps_below, sizeof(u));
  printf("%llu %llu %llu %llu %llu\n", r, q, p, u, n);
  return 0;
}
