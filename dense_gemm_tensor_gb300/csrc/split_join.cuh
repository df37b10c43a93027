// What the kernels share whose tiles are split along K over a cluster of CTAs: each
// CTA leaves its sums in its shared memory, and adds up a share of the tile's rows
// from all of them, in the CTAs' order.
#pragma once

#include "gemm_kernel.cuh"

namespace dgt {

// Loads N (16 or 32) columns of the warp's 32 accumulator rows.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_wait_ld_into(r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}

// warp_wait_phase for kernels of a few microseconds: some tries come before the timed wait, whose first look at the
// clock takes 0.3 us (one tile, two slabs: 4.0 us without, 3.3 with).
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity) {
  for (int n = 0; n < 64; ++n)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ bool warp_wait_short(const GemmParams& p, uint32_t bar, uint32_t parity, uint32_t code) {
  uint32_t ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_short(bar, parity) || wait_phase(p, bar, parity, code) ? 1u : 0u;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Element `at` of the shared array `sums` of each of the cluster's `splits` CTAs, added in their order. (After a
// cluster barrier; another one keeps the CTAs until all have read.)
__device__ __forceinline__ float joined_sum(const float* sums, int at, int splits) {
  if (splits == 1) return sums[at];
  const uint32_t local = smem_u32(sums + at);
  float v[8];
#pragma unroll
  for (int z = 0; z < 8; ++z) v[z] = z < splits ? ld_cluster_f32(mapa_shared(local, z)) : 0.0f;
  float s = v[0];
#pragma unroll
  for (int z = 1; z < 8; ++z)
    if (z < splits) s += v[z];
  return s;
}

// CTAs of a tile's cluster, 1 to 8: as many as there are places for (`slots` CTAs), each with two slabs or more. (More
// of them, in turns, spend their time on starting and joining: 16 rows x 4096 -> 2 x 8192 BF16, 128 tiles on 152 SMs,
// 25.4 us with one CTA a tile and 38.6 us with seven.) Places are counted, not what a GPC can hold of clusters, so that
// at some tile counts the last clusters wait for a second round. Gated, 16 x 4096 -> 2 x F BF16, us at 15 tiles 7.3, 16
// to 21 (splits of 8 and 7) 12.5 to 12.8, 22 and 23 8.3 and 8.7, 24 and 25 14.0, 26 to 28 8.7 to 9.4, 29 and 30 15.0, 31
// to 36 9.4 to 10.1, 37 and 38 16.8; blocks, 16 rows, K = 8192: 33 tiles 10.5, 37 15.8, 41 17.2, 45 12.2, 49 18.9, 53 13.4.
inline int choose_splits(int64_t tiles, int64_t slabs, int64_t slots) {
  int64_t s = slots / tiles;
  if (s > slabs / 2) s = slabs / 2;
  return s < 1 ? 1 : s > 8 ? 8 : int(s);
}

}  // namespace dgt
