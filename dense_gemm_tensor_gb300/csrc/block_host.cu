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
template <int BN>
cudaError_t launch_block(const BlockLaunch& L) {
  using Cf = BlockCfg<BN>;
  static int configured[64] = {};
  auto kern = block_kernel<BN>;
  if (L.dev >= 64 || !__atomic_load_n(&configured[L.dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (L.dev < 64) __atomic_store_n(&configured[L.dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, L.grid, kBlockThreads, Cf::SMEM_BYTES, L.stream, L.p.splits, L.tmP, L.tmQ, L.p);
}

constexpr int kFewRows = 64;  // up to here always the kernel for few rows

// Columns of a CTA pair's tile, or 0 for the kernel for few rows. Up to 64 rows, and where the tiles are so few that
// eight CTAs can share each and have work enough: us with it / with pairs, K = 4096: 65 x 512 6.4 / 10.6, 65 x 2048
// 8.7 / 10.7, 512 x 512 9.4 / 10.9, 1024 x 512 (beyond the limit) 12.0 / 11.2, 512 x 2048 18.0 / 13.5; K = 1024: 65 x
// 512 6.2 / 5.0. A pair's 256-wide tile takes about one and a half times a 128-wide one's time: 512 x 4096 x 4096
// (one round of either) 16.8 / 12.6 us, 2048 x 4096 x 4096 (two rounds or four) 30.6 / 37.7. With a scale for each row of
// B (`cols`) the columns weigh more, and it takes 1.8 times: 4096 x 4096 x 4096 (four or seven) 83.5 / 80.0, 4096 x 5120
// x 4096 (five or nine) 101.2 / 101.3, 8192 x 8192 x 8192 (14 or 27) 531 / 572.
int pair_width(int64_t M, int64_t N, int64_t blocks, bool cols, int sms) {
  const int64_t few = (M + 63) / 64 * ((N + 127) / 128);
  if (M <= kFewRows || (blocks >= 16 && few * 8 <= 2 * sms)) return 0;
  const int64_t rows = (M + 255) / 256, units = sms / 2;
  const int64_t wide = (rows * ((N + 255) / 256) + units - 1) / units, narrow = (rows * ((N + 127) / 128) + units - 1) / units;
  return (cols ? wide * 9 <= narrow * 5 : wide * 3 <= narrow * 2) ? 256 : 128;
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
  const int pair_bn = pair_width(M, N, blocks, b_rows == 1, ctx.sm_count);
  const bool few = pair_bn == 0;
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
  p.ps = few ? sb : sa;
  p.qs = few ? sa : sb;
  p.p_rows = int(few ? N : M);
  p.q_rows = int(few ? M : N);
  L.dev = ctx.dev;
  L.stream = s;
  const int bn = pair_bn > 0 ? pair_bn : !few ? 128 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int bm = pair_bn > 0 ? 256 : 128;
  p.g.tiles_m = (p.p_rows + bm - 1) / bm;
  p.g.tiles_n = (p.q_rows + bn - 1) / bn;
  const int64_t tiles = int64_t(p.g.tiles_m) * p.g.tiles_n;
  if (tiles > kIntLimit / 8) return GEMM_ERR_INVALID_VALUE;
  p.splits = 1;
  if (!few) {
    const int64_t units = ctx.sm_count / 2;
    L.grid = int(2 * (tiles < units ? tiles : units));
    const uint64_t v = uint64_t(reinterpret_cast<uintptr_t>(C)) | uint64_t(ldc * 2);
    p.g.c_gran = v % 16 == 0 ? 16 : v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
    p.g.c_tma = p.g.c_gran == 16;
    if (p.g.c_tma && !encode_map_3d(&L.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT16, C, N, M, ldc * 2, 1, 0, 64, 32,
                                    CU_TENSOR_MAP_SWIZZLE_128B))
      return GEMM_ERR_DRIVER;
  } else {
    p.splits = choose_splits(tiles, blocks, 2 * ctx.sm_count);
    L.grid = int(tiles * p.splits);
  }
  const void* P = few ? static_cast<const void*>(B) : A;
  const void* Q = few ? static_cast<const void*>(A) : B;
  if (!encode_map_3d(&L.tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, P, K, p.p_rows, few ? ldb : lda, 1, 0, kBlockK, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_3d(&L.tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, Q, K, p.q_rows, few ? lda : ldb, 1, 0, kBlockK,
                     few ? bn : bn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  cudaError_t e;
  if (!few)
    e = launch_block_pair(L, bn, b_rows == 1);
  else
    e = bn == 16 ? launch_block<16>(L) : bn == 32 ? launch_block<32>(L) : launch_block<64>(L);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
