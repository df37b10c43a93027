// 8-bit matrices with a scale for each block of 128 (gemm_quantize_blocks).
//
//   s = max(max |t| over the block, 1e-12) / 448,  q = e4m3(t (1 / s)),  t = x or x^T
//
// Bound by HBM: x is read once, into registers or shared memory, and q written
// once. Three kernels: blocks of 1 x 128 along x's rows (a part of a warp has a
// block), blocks of 128 x 128 or blocks along x's columns (a thread block has a
// 128 x 128 tile in shared memory), plain or transposed.
#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"

#include "dgt_feedforward.h"

namespace dgt {
namespace {

constexpr int kBlock = 128;
constexpr float kE4M3Max = 448.0f;

struct QuantParams {
  const void* x;
  uint8_t* q;
  float* scale;
  long long ldx, ldq, s_row, s_block;
  int rows, cols;      // of x
  int tall, transpose;
  int tiles_x;         // tiles across x's columns
};

// The scale of a block whose largest |t| has these bits (a NaN is above every number), and its reciprocal.
__device__ __forceinline__ float block_scale(uint32_t top, float& inv) {
  const float amax = __uint_as_float(top);
  const float scale = (amax < 1e-12f ? 1e-12f : amax) / kE4M3Max;
  inv = 1.0f / scale;
  return scale;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint8_t to_e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }

// Blocks along x's rows. A row's block is LANES lanes of VEC elements, 128 in all; rows by block row, blocks of a
// row next to each other. (VEC = 4 takes any row: elements one by one where the row does not allow more.)
template <int TYPE, int VEC, bool WIDE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  constexpr int LANES = kBlock / VEC;
  grid_dependency_wait();
  const int blocks = (p.cols + kBlock - 1) / kBlock;
  const long long tasks = static_cast<long long>(p.rows) * blocks;
  const int lane = threadIdx.x % LANES;
  const long long per_grid = static_cast<long long>(gridDim.x) * (256 / LANES);
  // (whole warps go round together: the shuffles below need all lanes)
  const long long first = static_cast<long long>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  const long long warp_first = first - (threadIdx.x % 32) / LANES;
  for (long long t0 = warp_first, t = first; t0 < tasks; t0 += per_grid, t += per_grid) {
    const bool in = t < tasks;
    const long long row = in ? t / blocks : 0;
    const int b = in ? static_cast<int>(t - row * blocks) : 0;
    const int c0 = b * kBlock + lane * VEC;
    float v[VEC];
    const T* src = static_cast<const T*>(p.x) + row * p.ldx + c0;
    if constexpr (WIDE) {
      Pack<TYPE, 16 / int(sizeof(T))> w[VEC * sizeof(T) / 16];
      constexpr int PER = 16 / sizeof(T);
#pragma unroll
      for (int i = 0; i < int(VEC * sizeof(T) / 16); ++i) {
        w[i].zero();
        if (in && c0 + i * PER < p.cols) w[i].stream(src + i * PER);
#pragma unroll
        for (int j = 0; j < PER; ++j) v[i * PER + j] = w[i].get(j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = in && c0 + j < p.cols ? E::get(src[j]) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = max(top, magnitude(v[j]));
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float inv;
    const float scale = block_scale(top, inv);
    if (!in) continue;
    if (lane == 0) p.scale[row * p.s_row + b * p.s_block] = scale;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] *= inv;
    uint8_t* dst = p.q + row * p.ldq + c0;
    if constexpr (WIDE) {
      if (c0 < p.cols) {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
          w[i] = lo | (hi << 16);
        }
        if constexpr (VEC == 16)
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        else
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c0 + j < p.cols) dst[j] = to_e4m3(v[j]);
    }
  }
  grid_launch_dependents();
}

// A 128 x 128 tile of x in shared memory: blocks of the whole tile (tall) or along x's columns (transposed, not
// tall), written as they lie or transposed. The tile's columns are one apart from a power of two, so that threads
// walking down a column meet other banks.
template <int TYPE, bool WIDE>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const QuantParams p) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  constexpr int PER = 16 / sizeof(T);
  constexpr int LD = kBlock + 4 / int(sizeof(T)) * 1;  // a word more than the tile's row
  extern __shared__ uint4 dynamic[];
  T* tile = reinterpret_cast<T*>(dynamic);
  __shared__ uint32_t tops[8];
  __shared__ uint32_t col_top[2][kBlock];
  __shared__ float col_inv[kBlock];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = static_cast<int>(blockIdx.x / p.tiles_x) * kBlock, c0 = static_cast<int>(blockIdx.x % p.tiles_x) * kBlock;
  const int nr = min(kBlock, p.rows - r0), nc = min(kBlock, p.cols - c0);
  const T* src = static_cast<const T*>(p.x) + static_cast<long long>(r0) * p.ldx + c0;
  grid_dependency_wait();
  uint32_t top = 0;
  if constexpr (WIDE) {
    constexpr int PIECES = kBlock / PER;
    for (int i = tid; i < kBlock * PIECES; i += 256) {
      const int r = i / PIECES, c = (i % PIECES) * PER;
      Pack<TYPE, PER> w;
      w.zero();
      if (r < nr && c < nc) w.stream(src + static_cast<long long>(r) * p.ldx + c);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        tile[r * LD + c + j] = w.v[j];
        top = max(top, magnitude(w.get(j)));
      }
    }
  } else {
    for (int i = tid; i < kBlock * kBlock; i += 256) {
      const int r = i / kBlock, c = i % kBlock;
      const T v = r < nr && c < nc ? src[static_cast<long long>(r) * p.ldx + c] : E::put(0.0f);
      tile[r * LD + c] = v;
      top = max(top, magnitude(E::get(v)));
    }
  }
  float inv = 0.0f;
  const int rb = r0 / kBlock, cb = c0 / kBlock;
  if (p.tall > 1) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, tops[lane & 7]);
    const float scale = block_scale(top, inv);
    if (tid == 0) p.scale[(p.transpose ? cb : rb) * p.s_row + (p.transpose ? rb : cb) * p.s_block] = scale;
  } else {
    // a column's block: two threads a column, half the rows each
    __syncthreads();
    const int c = tid & (kBlock - 1), half = tid / kBlock;
    top = 0;
#pragma unroll 8
    for (int r = half * (kBlock / 2); r < (half + 1) * (kBlock / 2); ++r) top = max(top, magnitude(E::get(tile[r * LD + c])));
    col_top[half][c] = top;
    __syncthreads();
    if (half == 0) {
      float one;
      const float scale = block_scale(max(col_top[0][c], col_top[1][c]), one);
      col_inv[c] = one;
      if (c < nc) p.scale[static_cast<long long>(c0 + c) * p.s_row + rb * p.s_block] = scale;
    }
    __syncthreads();
  }
  // four neighbouring elements of a row of q a thread
  const int out_rows = p.transpose ? nc : nr, out_cols = p.transpose ? nr : nc;
  const long long q0 = static_cast<long long>(p.transpose ? c0 : r0) * p.ldq + (p.transpose ? r0 : c0);
  for (int i = tid; i < kBlock * (kBlock / 4); i += 256) {
    const int r = i / (kBlock / 4), c = (i % (kBlock / 4)) * 4;
    if (r >= out_rows || c >= out_cols) continue;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = E::get(p.transpose ? tile[(c + j) * LD + r] : tile[r * LD + c + j]);
    const float f = p.tall > 1 ? inv : col_inv[r];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= f;
    uint8_t* dst = p.q + q0 + static_cast<long long>(r) * p.ldq + c;
    if (c + 4 <= out_cols && (reinterpret_cast<uintptr_t>(dst) & 3) == 0) {
      store_e4m3<4>(dst, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < out_cols) dst[j] = to_e4m3(v[j]);
    }
  }
  grid_launch_dependents();
}

template <int TYPE>
cudaError_t launch_quantize(const QuantParams& p, bool wide_x, bool wide_q, int dev, int sms, cudaStream_t s) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = 16;
  if (p.tall == 1 && !p.transpose) {
    const int64_t tasks = int64_t(p.rows) * ((p.cols + kBlock - 1) / kBlock);
    const int64_t per = wide_x && wide_q ? 256 / (kBlock / VEC) : 256 / (kBlock / 4);
    const int64_t need = (tasks + per - 1) / per, most = int64_t(sms) * 8;
    const int grid = int(need < most ? need : most);
    return wide_x && wide_q ? launch_dependent(quantize_rows_kernel<TYPE, VEC, true>, grid, 256, 0, s, 1, p)
                            : launch_dependent(quantize_rows_kernel<TYPE, 4, false>, grid, 256, 0, s, 1, p);
  }
  const int64_t tiles = int64_t(p.tiles_x) * ((p.rows + kBlock - 1) / kBlock);
  constexpr size_t smem = size_t(kBlock) * (kBlock + 4 / sizeof(T)) * sizeof(T);
  static int configured[64] = {};
  if (smem > 48 * 1024 && (dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE))) {
    cudaError_t e = cudaFuncSetAttribute(quantize_tile_kernel<TYPE, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(quantize_tile_kernel<TYPE, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  return wide_x ? launch_dependent(quantize_tile_kernel<TYPE, true>, int(tiles), 256, smem, s, 1, p)
                : launch_dependent(quantize_tile_kernel<TYPE, false>, int(tiles), 256, smem, s, 1, p);
}

bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }
constexpr int64_t kIntLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kLdLimit = int64_t(1) << 39;

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" int gemm_quantize_blocks(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, int block_rows,
                                    int transpose, uint8_t* q, int64_t ldq, float* scale, int64_t s_row,
                                    int64_t s_block, void* stream) {
  if ((type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F32) || rows < 0 || cols < 0 ||
      rows > kIntLimit - kBlock || cols > kIntLimit - kBlock || (block_rows != 1 && block_rows != kBlock) ||
      (transpose != 0 && transpose != 1))
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t out_rows = transpose ? cols : rows, out_cols = transpose ? rows : cols;
  const int64_t blocks = (out_cols + kBlock - 1) / kBlock, runs = block_rows == 1 ? out_rows : (out_rows + kBlock - 1) / kBlock;
  if (x == nullptr || q == nullptr || scale == nullptr || ldx < cols || ldq < out_cols || ldx > kLdLimit ||
      ldq > kLdLimit || s_row < 0 || s_block < 0 || s_row > kLdLimit || s_block > kLdLimit ||
      ((rows + kBlock - 1) / kBlock) * ((cols + kBlock - 1) / kBlock) > kIntLimit)
    return GEMM_ERR_INVALID_VALUE;
  // every scale has a place of its own: one stride spans what the other counts
  if (!((runs == 1 || s_row > (blocks - 1) * s_block) && (blocks == 1 || s_block >= 1)) &&
      !((blocks == 1 || s_block > (runs - 1) * s_row) && (runs == 1 || s_row >= 1)))
    return GEMM_ERR_INVALID_VALUE;
  const int es = type_bytes(type);
  if (misaligned(x, es) || misaligned(scale, 4)) return GEMM_ERR_MISALIGNED;
  struct Range {
    uintptr_t lo, hi;
  };
  auto range = [](const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + uintptr_t(bytes)};
  };
  auto meet = [](const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; };
  const Range rx = range(x, ((rows - 1) * ldx + cols) * es), rq = range(q, (out_rows - 1) * ldq + out_cols),
              rs = range(scale, ((runs - 1) * s_row + (blocks - 1) * s_block + 1) * 4);
  if (meet(rx, rq) || meet(rx, rs) || meet(rq, rs)) return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  if (!on_device(x, ctx.dev) || !on_device(q, ctx.dev) || !on_device(scale, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  // 16-byte pieces, where every row of x starts on one and is made of them; q's rows in pieces of 16 elements
  const bool wide_x = cols % (16 / es) == 0 && !misaligned(x, 16) && (rows == 1 || (ldx * es) % 16 == 0);
  const bool wide_q = cols % 16 == 0 && !misaligned(q, 16) && (rows == 1 || ldq % 16 == 0);
  QuantParams p = {x,          q,         scale,          (long long)ldx, (long long)ldq, (long long)s_row, (long long)s_block,
                   int(rows),  int(cols), block_rows,     transpose,      int((cols + kBlock - 1) / kBlock)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_quantize<GEMM_TYPE_F16>(p, wide_x, wide_q, ctx.dev, ctx.sm_count, s)
                        : type == GEMM_TYPE_BF16 ? launch_quantize<GEMM_TYPE_BF16>(p, wide_x, wide_q, ctx.dev, ctx.sm_count, s)
                                                 : launch_quantize<GEMM_TYPE_F32>(p, wide_x, wide_q, ctx.dev, ctx.sm_count, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
