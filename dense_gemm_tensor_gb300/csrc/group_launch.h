// Internal interface between the grouped products' host code (group_host.cu)
// and their kernel units (group_<kind>_<rm|km|wgrad>.cu, which build in parallel).
#pragma once

#include "group_kernel.cuh"
#include "host.h"

namespace dgt {

struct GroupLaunch {
  // the MMA's A operand: boxes; gathered rows (product), the groups' ragged slabs (gradient) or W's value half (dense
  // gated product)
  CUtensorMap tmA, tmA2;
  CUtensorMap tmB, tmB2;  // its B operand: boxes; ragged slabs (gradient), or the kept halves (dense gated product)
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
cudaError_t launch_gated_bf16_rm(const GroupLaunch& L);
cudaError_t launch_gated_bf16_km(const GroupLaunch& L);
cudaError_t launch_gated_f16_rm(const GroupLaunch& L);
cudaError_t launch_gated_f16_km(const GroupLaunch& L);

// What a dense product adds to a grouped one: one group of all rows, without offsets on the device; and a gated one's
// activation (GEMM_GATE_*; -1: not gated) and kept halves.
struct DenseProduct {
  int gate;
  void* up;  // slots x N, or null
  int64_t ldup;
  // Where the value half of row-major weights goes that TMA cannot read in place (or null), and what copies it there.
  void* value;
  int64_t ldv;
  int (*copy)(const void* W, int64_t ldw, int64_t K, int64_t F, void* to, int64_t ld, cudaStream_t stream);
  // The kernel for few rows, taken by few_rows where TMA reads A and W in place, and the columns of C in its tile.
  int (*few)(int type, int64_t M, int64_t F, int64_t K, const void* A, int64_t lda, const void* W, int64_t ldw,
             bool row_major, const void* value, int64_t ldv, int gate, const void* bias, void* C, int64_t ldc, void* up,
             int64_t ldup, const CallContext& ctx, cudaStream_t stream);
  int few_columns;
};
// Whether a product of M rows and N columns, `per` of them a tile, takes the kernel for few rows: up to 64 rows, and
// beyond while its tiles are one an SM. Gated, BF16, us with it / with the grouped products' kernel, K = 4096: 65 x F
// 512 10.1 / 23.7, 128 x 4096 21.0 / 25.4, 256 x 2048 20.7 / 24.8, 256 x 4096 (beyond the limit) 25.1 / 25.4, 512 x
// 4096 48.0 / 26.9; K = 1024: 65 x 512 7.2 / 10.3, 128 x 4096 9.5 / 12.5.
inline bool few_rows(int64_t M, int64_t N, int per, int sms) {
  return M <= 64 || (M + 63) / 64 * ((N + per - 1) / per) <= sms;
}
// The grouped product and weight gradient behind the C entry points (group_host.cu). dense: null for groups on the
// device; offsets and rows are null where it is given.
int run_grouped(int kind, int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const void* A,
                int64_t a_rows, int64_t lda, const int32_t* rows, const void* W, int64_t ldw, int64_t stride_w, void* C,
                int64_t ldc, int layout, const gemm_grouped_epilogue_t* epi, void* workspace, int64_t workspace_bytes,
                void* stream, const DenseProduct* dense);
int run_wgrad(int kind, int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const void* A,
              int64_t a_rows, int64_t lda, const int32_t* rows, const void* dC, int64_t lddc, void* dW, int64_t lddw,
              int64_t stride_dw, int layout, void* workspace, int64_t workspace_bytes, void* stream, bool dense);
// Bytes of workspace that run_wgrad takes for a dense product: copies of rows whose pitch is not TMA's.
int64_t dense_wgrad_workspace(int64_t slots, int64_t N, int64_t K, int64_t lda, int64_t lddc);

// Sets the kernel's dynamic shared-memory limit once per device, then launches.
template <int KIND, int OPS, int BN, bool PAIR, int GATED>
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
      return L.gated ? launch_group_variant<KIND, OPS, kGroupPairN, true, GATED_SILU>(L)             \
                     : launch_group_variant<KIND, OPS, kGroupPairN, true, GATED_NONE>(L);            \
    return L.gated ? launch_group_variant<KIND, OPS, kGroupSingleN, false, GATED_SILU>(L)            \
                   : launch_group_variant<KIND, OPS, kGroupSingleN, false, GATED_NONE>(L);           \
  }

// The dense gated product.
#define DGT_DEFINE_GATED(name, KIND, OPS)                                                            \
  cudaError_t launch_gated_##name(const GroupLaunch& L) {                                            \
    return L.pair ? launch_group_variant<KIND, OPS, kGroupPairN, true, GATED_ANY>(L)                 \
                  : launch_group_variant<KIND, OPS, kGroupSingleN, false, GATED_ANY>(L);             \
  }

#define DGT_DEFINE_GROUP_WGRAD(name, KIND)                                                           \
  cudaError_t launch_group_##name(const GroupLaunch& L) {                                            \
    return launch_group_variant<KIND, GROUP_WGRAD, kGroupPairN, true, GATED_NONE>(L);                  \
  }

}  // namespace dgt
