// C entry point of the products with a scale for each block of 128
// (gemm_e4m3_blocks): argument checks, tensor maps, the choice of tile and split.
#include <cstring>

#include "block_kernel.cuh"
#include "host.h"

namespace dgt {
namespace {

constexpr int64_t kIntLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kLdLimit = int64_t(1) << 39;

bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }

struct Range {
  uintptr_t lo, hi;
};
Range range_of(const void* p, int64_t elems, int es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(elems * es)};
}
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Sets the kernel's dynamic shared-memory limit once per device, then launches.
template <int BN, bool COLS, bool SWAP>
cudaError_t launch_block(const CUtensorMap& tmP, const CUtensorMap& tmQ, const BlockParams& p, int dev, int grid,
                         cudaStream_t s) {
  using Cf = BlockCfg<BN>;
  static int configured[64] = {};
  auto kern = block_kernel<BN, COLS, SWAP>;
  if (dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, grid, kBlockThreads, Cf::SMEM_BYTES, s, p.splits, tmP, tmQ, p);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" int gemm_e4m3_blocks(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* a_scale,
                                int64_t as_row, int64_t as_block, const uint8_t* B, int64_t ldb, const float* b_scale,
                                int64_t bs_row, int64_t bs_block, int b_rows, uint16_t* C, int64_t ldc, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > kIntLimit - 256 || N > kIntLimit - 256 || K > kIntLimit - 256 ||
      (b_rows != 1 && b_rows != kBlockK))
    return GEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return GEMM_OK;
  if (C == nullptr || ldc < N || ldc > kLdLimit) return GEMM_ERR_INVALID_VALUE;
  if (misaligned(C, 2)) return GEMM_ERR_MISALIGNED;
  const int64_t blocks = (K + kBlockK - 1) / kBlockK, b_runs = b_rows == 1 ? N : (N + kBlockK - 1) / kBlockK;
  if (K > 0) {
    if (A == nullptr || B == nullptr || a_scale == nullptr || b_scale == nullptr || lda < K || ldb < K ||
        lda > kLdLimit || ldb > kLdLimit || as_row < 0 || as_block < 0 || bs_row < 0 || bs_block < 0 ||
        as_row > kLdLimit || as_block > kLdLimit || bs_row > kLdLimit || bs_block > kLdLimit)
      return GEMM_ERR_INVALID_VALUE;
    if (misaligned(A, 16) || misaligned(B, 16) || (M > 1 && lda % 16 != 0) || (N > 1 && ldb % 16 != 0) ||
        misaligned(a_scale, 4) || misaligned(b_scale, 4))
      return GEMM_ERR_MISALIGNED;
    const Range rc = range_of(C, (M - 1) * ldc + N, 2);
    if (meet(rc, range_of(A, (M - 1) * lda + K, 1)) || meet(rc, range_of(B, (N - 1) * ldb + K, 1)) ||
        meet(rc, range_of(a_scale, (M - 1) * as_row + (blocks - 1) * as_block + 1, 4)) ||
        meet(rc, range_of(b_scale, (b_runs - 1) * bs_row + (blocks - 1) * bs_block + 1, 4)))
      return GEMM_ERR_INVALID_VALUE;
  }
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  if (!on_device(C, ctx.dev) || (K > 0 && (!on_device(A, ctx.dev) || !on_device(B, ctx.dev) ||
                                           !on_device(a_scale, ctx.dev) || !on_device(b_scale, ctx.dev))))
    return GEMM_ERR_NOT_DEVICE_MEMORY;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return cudaMemset2DAsync(C, size_t(ldc) * 2, 0, size_t(N) * 2, size_t(M), s) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;

  // (the pitch of a matrix of one row says nothing)
  if (M == 1) lda = (K + 15) / 16 * 16;
  if (N == 1) ldb = (K + 15) / 16 * 16;
  const bool swap = M <= 64;
  BlockParams p;
  memset(&p, 0, sizeof(p));
  p.g.status = ctx.status;
  p.g.epoch = ctx.epoch;
  p.g.debug = ctx.debug;
  p.g.wait_limit_ns = ctx.wait_limit_ns;
  p.g.C = C;
  p.g.ldc = ldc;
  p.g.num_kb = int(blocks);
  const BlockScales sa = {a_scale, as_row, as_block, 0}, sb = {b_scale, bs_row, bs_block, b_rows == 1 ? 0 : 7};
  p.ps = swap ? sb : sa;
  p.qs = swap ? sa : sb;
  p.p_rows = int(swap ? N : M);
  p.q_rows = int(swap ? M : N);
  const int bn = !swap ? 128 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
  p.g.tiles_m = (p.p_rows + 127) / 128;
  p.g.tiles_n = (p.q_rows + bn - 1) / bn;
  p.g.raster = 8;
  const int64_t tiles = int64_t(p.g.tiles_m) * p.g.tiles_n;
  // a tile is split while the GPU (two CTAs to an SM) has room for twice the CTAs and each would keep four blocks
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= 2 * ctx.sm_count && blocks >= p.splits * 8) p.splits *= 2;
  if (tiles * p.splits > kIntLimit) return GEMM_ERR_INVALID_VALUE;
  const void* P = swap ? static_cast<const void*>(B) : A;
  const void* Q = swap ? static_cast<const void*>(A) : B;
  CUtensorMap tmP, tmQ;
  if (!encode_map_3d(&tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, P, K, p.p_rows, swap ? ldb : lda, 1, 0, kBlockK, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_3d(&tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, Q, K, p.q_rows, swap ? lda : ldb, 1, 0, kBlockK, bn,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  const int grid = int(tiles * p.splits);
  cudaError_t e;
  if (swap)
    e = bn == 16   ? launch_block<16, true, true>(tmP, tmQ, p, ctx.dev, grid, s)
        : bn == 32 ? launch_block<32, true, true>(tmP, tmQ, p, ctx.dev, grid, s)
                   : launch_block<64, true, true>(tmP, tmQ, p, ctx.dev, grid, s);
  else
    e = b_rows == 1 ? launch_block<128, true, false>(tmP, tmQ, p, ctx.dev, grid, s)
                    : launch_block<128, false, false>(tmP, tmQ, p, ctx.dev, grid, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
