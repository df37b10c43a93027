// Internal interface between the grouped products' host code (group_host.cu)
// and their kernel units (group_<kind>_<rm|km|wgrad>.cu, which build in parallel).
#pragma once

#include "group_kernel.cuh"
#include "host.h"

namespace dgt {

struct GroupLaunch {
  CUtensorMap tmA, tmA2;  // the MMA's A operand: boxes; gathered rows (product) or the groups' ragged slabs (gradient)
  CUtensorMap tmB, tmB2;  // its B operand: boxes; ragged slabs (gradient)
  CUtensorMap tmC;        // valid when p.g.c_tma
  GroupParams p;
  bool pair, gated;
  int grid;  // CTAs
  int dev;
  cudaStream_t stream;
};

cudaError_t launch_group_bf16_rm(const GroupLaunch& L);
cudaError_t launch_group_bf16_km(const GroupLaunch& L);
cudaError_t launch_group_bf16_wgrad(const GroupLaunch& L);
cudaError_t launch_group_f16_rm(const GroupLaunch& L);
cudaError_t launch_group_f16_km(const GroupLaunch& L);
cudaError_t launch_group_f16_wgrad(const GroupLaunch& L);
cudaError_t launch_group_e4m3_km(const GroupLaunch& L);

// Sets the kernel's dynamic shared-memory limit once per device, then launches.
template <int KIND, int OPS, int BN, bool PAIR, bool GATED>
cudaError_t launch_group_variant(const GroupLaunch& L) {
  using Cf = GroupCfg<KIND, OPS, BN, PAIR, GATED>;
  static int configured[64] = {};
  auto kern = group_kernel<KIND, OPS, BN, PAIR, GATED>;
  if (L.dev >= 64 || !__atomic_load_n(&configured[L.dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (L.dev < 64) __atomic_store_n(&configured[L.dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, L.grid, kGroupThreads, Cf::SMEM_BYTES, L.stream, Cf::CTAS, L.tmA, L.tmA2, L.tmB, L.tmB2,
                          L.tmC, L.p);
}

// Accumulator columns of a tile: the CTA pair's, and one CTA's.
constexpr int kGroupPairN = 256;
constexpr int kGroupSingleN = 128;

#define DGT_DEFINE_GROUP(name, KIND, OPS)                                                            \
  cudaError_t launch_group_##name(const GroupLaunch& L) {                                            \
    if (L.pair)                                                                                      \
      return L.gated ? launch_group_variant<KIND, OPS, kGroupPairN, true, true>(L)                   \
                     : launch_group_variant<KIND, OPS, kGroupPairN, true, false>(L);                 \
    return L.gated ? launch_group_variant<KIND, OPS, kGroupSingleN, false, true>(L)                  \
                   : launch_group_variant<KIND, OPS, kGroupSingleN, false, false>(L);                \
  }

#define DGT_DEFINE_GROUP_WGRAD(name, KIND)                                                           \
  cudaError_t launch_group_##name(const GroupLaunch& L) {                                            \
    return launch_group_variant<KIND, GROUP_WGRAD, kGroupPairN, true, false>(L);                     \
  }

}  // namespace dgt
