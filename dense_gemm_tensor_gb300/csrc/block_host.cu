// C entry point of the products with a scale for each block of 128
// (gemm_e4m3_blocks): argument checks, tensor maps, the choice of tile and split.
#include <cstring>

#include "block_launch.h"

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
cudaError_t launch_block(const BlockLaunch& L) {
  using Cf = BlockCfg<BN>;
  static int configured[64] = {};
  auto kern = block_kernel<BN, COLS, SWAP>;
  if (L.dev >= 64 || !__atomic_load_n(&configured[L.dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (L.dev < 64) __atomic_store_n(&configured[L.dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, L.grid, kBlockThreads, Cf::SMEM_BYTES, L.stream, L.p.splits, L.tmP, L.tmQ, L.p);
}

// Columns of a CTA pair's tile, or 0 for single CTAs: the widest whose tiles give most pairs one.
int pair_width(int64_t M, int64_t N, int sms) {
  const int64_t rows = (M + 255) / 256, units = sms / 2;
  for (int bn : {256, 128})
    if (rows * ((N + bn - 1) / bn) * 4 >= units * 3) return bn;
  return 0;
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
  BlockLaunch L;
  memset(&L, 0, sizeof(L));
  BlockParams& p = L.p;
  p.g.status = ctx.status;
  p.g.epoch = ctx.epoch;
  p.g.debug = ctx.debug;
  p.g.wait_limit_ns = ctx.wait_limit_ns;
  p.g.C = C;
  p.g.ldc = ldc;
  p.g.num_kb = int(blocks);
  p.g.raster = 8;
  const BlockScales sa = {a_scale, as_row, as_block, 0}, sb = {b_scale, bs_row, bs_block, b_rows == 1 ? 0 : 7};
  p.ps = swap ? sb : sa;
  p.qs = swap ? sa : sb;
  p.p_rows = int(swap ? N : M);
  p.q_rows = int(swap ? M : N);
  L.dev = ctx.dev;
  L.stream = s;
  const int pair_bn = swap ? 0 : pair_width(M, N, ctx.sm_count);
  const int bn = pair_bn > 0 ? pair_bn : !swap ? 128 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int bm = pair_bn > 0 ? 256 : 128;
  p.g.tiles_m = (p.p_rows + bm - 1) / bm;
  p.g.tiles_n = (p.q_rows + bn - 1) / bn;
  const int64_t tiles = int64_t(p.g.tiles_m) * p.g.tiles_n;
  if (tiles > kIntLimit / 8) return GEMM_ERR_INVALID_VALUE;
  p.splits = 1;
  if (pair_bn > 0) {
    const int64_t units = ctx.sm_count / 2;
    L.grid = int(2 * (tiles < units ? tiles : units));
    const uint64_t v = uint64_t(reinterpret_cast<uintptr_t>(C)) | uint64_t(ldc * 2);
    p.g.c_gran = v % 16 == 0 ? 16 : v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
    p.g.c_tma = p.g.c_gran == 16;
    if (p.g.c_tma && !encode_map_3d(&L.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT16, C, N, M, ldc * 2, 1, 0, 64, 32,
                                    CU_TENSOR_MAP_SWIZZLE_128B))
      return GEMM_ERR_DRIVER;
  } else {
    // a tile is split while the GPU (two CTAs to an SM) has room for twice the CTAs and each would keep four blocks
    while (p.splits < 8 && tiles * p.splits * 2 <= 2 * ctx.sm_count && blocks >= p.splits * 8) p.splits *= 2;
    L.grid = int(tiles * p.splits);
  }
  const void* P = swap ? static_cast<const void*>(B) : A;
  const void* Q = swap ? static_cast<const void*>(A) : B;
  if (!encode_map_3d(&L.tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, P, K, p.p_rows, swap ? ldb : lda, 1, 0, kBlockK, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_3d(&L.tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, Q, K, p.q_rows, swap ? lda : ldb, 1, 0, kBlockK,
                     pair_bn > 0 ? bn / 2 : bn, CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  cudaError_t e;
  if (pair_bn > 0)
    e = launch_block_pair(L, bn, b_rows == 1);
  else if (swap)
    e = bn == 16 ? launch_block<16, true, true>(L) : bn == 32 ? launch_block<32, true, true>(L) : launch_block<64, true, true>(L);
  else
    e = b_rows == 1 ? launch_block<128, true, false>(L) : launch_block<128, false, false>(L);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
