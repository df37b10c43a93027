// Products with a scale for each block of 128 on CTA pairs.
#include "block_launch.h"
#include "block_pair.cuh"

namespace dgt {
namespace {

template <int BN, bool COLS>
cudaError_t launch(const BlockLaunch& L) {
  using Cf = BlockPairCfg<BN>;
  static int configured[64] = {};
  auto kern = block_pair_kernel<BN, COLS>;
  if (L.dev >= 64 || !__atomic_load_n(&configured[L.dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (L.dev < 64) __atomic_store_n(&configured[L.dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, L.grid, kPairThreads, Cf::SMEM_BYTES, L.stream, 2, L.tmP, L.tmQ, L.tmC, L.p);
}

}  // namespace

cudaError_t launch_block_pair(const BlockLaunch& L, int bn, bool cols) {
  return bn == 256 ? (cols ? launch<256, true>(L) : launch<256, false>(L))
                   : (cols ? launch<128, true>(L) : launch<128, false>(L));
}

}  // namespace dgt
