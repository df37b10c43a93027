// Internal interface between the dense gated product's host code (gated.cu) and the
// units of its kernel for few rows (gated_few_<kind>.cu).
#pragma once

#include "gated_few.cuh"
#include "host.h"

namespace dgt {

struct GatedFewLaunch {
  CUtensorMap tmW, tmV, tmA;  // the weights; their value half; A
  GatedFewParams p;
  bool row_major;
  bool deep;  // one CTA to an SM
  int bn;    // 16, 32 or 64 rows of A
  int grid;  // CTAs
  int dev;
  cudaStream_t stream;
};

cudaError_t launch_gated_few_bf16(const GatedFewLaunch& L);
cudaError_t launch_gated_few_f16(const GatedFewLaunch& L);

// Sets the kernel's dynamic shared-memory limit once per device, then launches.
template <int KIND, bool MN, int BN, bool DEEP>
cudaError_t launch_gated_few(const GatedFewLaunch& L) {
  using Cf = GatedFewCfg<KIND, MN, BN, DEEP>;
  static int configured[64] = {};
  auto kern = gated_few_kernel<KIND, MN, BN, DEEP>;
  if (L.dev >= 64 || !__atomic_load_n(&configured[L.dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (L.dev < 64) __atomic_store_n(&configured[L.dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, L.grid, kFewThreads, Cf::SMEM_BYTES, L.stream, L.p.splits, L.tmW, L.tmV, L.tmA, L.p);
}

template <int KIND, bool MN, int BN>
cudaError_t launch_gated_few_bn(const GatedFewLaunch& L) {
  return L.deep ? launch_gated_few<KIND, MN, BN, true>(L) : launch_gated_few<KIND, MN, BN, false>(L);
}

#define DGT_DEFINE_GATED_FEW(name, KIND)                                                              \
  cudaError_t launch_gated_few_##name(const GatedFewLaunch& L) {                                      \
    if (L.row_major)                                                                                  \
      return L.bn == 16   ? launch_gated_few_bn<KIND, true, 16>(L)                                    \
             : L.bn == 32 ? launch_gated_few_bn<KIND, true, 32>(L)                                    \
                          : launch_gated_few_bn<KIND, true, 64>(L);                                   \
    return L.bn == 16   ? launch_gated_few_bn<KIND, false, 16>(L)                                     \
           : L.bn == 32 ? launch_gated_few_bn<KIND, false, 32>(L)                                     \
                        : launch_gated_few_bn<KIND, false, 64>(L);                                    \
  }

}  // namespace dgt
