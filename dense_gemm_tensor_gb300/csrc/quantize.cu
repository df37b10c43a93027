// 8-bit matrices with a scale for each block of 128 (gemm_quantize_blocks).
//
//   s = max(max |t| over the block, 1e-12) / 448,  q = e4m3(t (1 / s)),  t = x or x^T
//
// Bound by HBM: x is read once, into registers, and q written once. Two kernels:
// blocks of 1 x 128 along x's rows (a part of a warp has a block), and tiles of
// 128 x 128 (blocks of a whole tile, or along x's columns), plain or transposed.
// 8192 x 8192 BF16 32 us in every form (6.2 TB/s), FP32 54-57 (6.0), 4099 x 5120 BF16
// transposed 11.3 (5.6).
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
  int shares;          // thread blocks that share a group of rows
  int wide_q;          // q's rows start on 16-byte boundaries
};

// The scale of a block whose largest |t| has these bits (a NaN is above every number), and its reciprocal.
__device__ __forceinline__ float block_scale(uint32_t top, float& inv) {
  const float amax = __uint_as_float(top);
  const float scale = (amax < 1e-12f ? 1e-12f : amax) / kE4M3Max;
  inv = 1.0f / scale;
  return scale;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Four values to E4M3 bytes, the first lowest.
__device__ __forceinline__ uint32_t four_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ uint8_t to_e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }

// 16 bytes of a row from `src` on, of which `valid` elements are the row's; the others are zero. SHIFT: src is
// anywhere. 16-bit elements are then shifted together from the two aligned pieces that hold them (the second is read
// where it holds some of the row's: an aligned piece with a byte of the matrix is in its memory); FP32 ones are read
// one by one. (2048 x 4095 BF16 8.6 us shifted, 11.8 one by one; FP32 14.2 and 13.2.)
template <int TYPE, bool SHIFT>
__device__ __forceinline__ void load_piece(Pack<TYPE, 16 / int(sizeof(typename Elem<TYPE>::T))>& v,
                                           const typename Elem<TYPE>::T* src, int valid) {
  using T = typename Elem<TYPE>::T;
  constexpr int PER = 16 / sizeof(T);
  v.zero();
  if (valid <= 0) return;
  if constexpr (!SHIFT) {
    v.stream(src);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j < valid) v.v[j] = src[j];
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(src);
    const int m = static_cast<int>(at & 15);
    const uint4 lo = *reinterpret_cast<const uint4*>(at - m);
    uint4 hi = make_uint4(0u, 0u, 0u, 0u);
    if (m + valid * int(sizeof(T)) > 16) hi = *reinterpret_cast<const uint4*>(at - m + 16);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t a[6], b[5], o[4];
#pragma unroll
    for (int k = 0; k < 6; ++k) a[k] = m & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) b[k] = m & 4 ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(b[k], b[k + 1], (m & 3) * 8);
    *reinterpret_cast<uint4*>(v.v) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (valid < PER) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (j >= valid) v.v[j] = Elem<TYPE>::put(0.0f);
  }
}

// Blocks along x's rows. Eight lanes have a row's block, 16 elements each; a warp has neighbouring rows of the same
// block column, so that their scales, block by block, lie together; a thread block walks along its rows with the next
// block's elements in flight.
template <int TYPE, bool SHIFT>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  constexpr int VEC = 16, LANES = kBlock / VEC, ROWS = 256 / LANES;
  constexpr int PER = 16 / sizeof(T), PIECES = VEC / PER;
  const int blocks = (p.cols + kBlock - 1) / kBlock;
  const int lane = threadIdx.x % LANES;
  // blockIdx.x: a group of rows and a share of their blocks
  const long long group = blockIdx.x / p.shares;
  const int share = static_cast<int>(blockIdx.x % p.shares);
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * share / p.shares);
  const int b1 = static_cast<int>(static_cast<long long>(blocks) * (share + 1) / p.shares);
  const long long row = group * ROWS + threadIdx.x / LANES;
  const bool in = row < p.rows;
  const T* src = static_cast<const T*>(p.x) + row * p.ldx;
  grid_dependency_wait();
  Pack<TYPE, PER> next[PIECES];
  auto load = [&](int b) {
    const int c0 = b * kBlock + lane * VEC;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      load_piece<TYPE, SHIFT>(next[i], src + c0 + i * PER, in && b < b1 ? p.cols - c0 - i * PER : 0);
  };
  load(b0);
  for (int b = b0; b < b1; ++b) {
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = next[j / PER].get(j % PER);
    load(b + 1);
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
    const int c0 = b * kBlock + lane * VEC;
    uint8_t* dst = p.q + row * p.ldq + c0;
    if (p.wide_q && c0 + VEC <= p.cols) {
      uint32_t w[VEC / 4];
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) w[i] = four_e4m3(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c0 + j < p.cols) dst[j] = to_e4m3(v[j]);
    }
  }
  grid_launch_dependents();
}

// A 128 x 128 tile of x: blocks of the whole tile (tall) or along x's columns (transposed, not tall). A thread holds
// 8 x 8 elements in registers; the transposed q goes through shared memory, 8 rows of a column (8 bytes) at a time, in
// an order in which 16 threads meet 16 places: piece k of column c sits at k ^ (c / 8).
template <int TYPE, bool SHIFT>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const QuantParams p) {
  using E = Elem<TYPE>;
  using T = typename E::T;
  constexpr int PER = 16 / sizeof(T), PIECES = 8 / PER;
  using P = Pack<TYPE, PER>;
  __shared__ uint32_t tops[16][kBlock];
  __shared__ float col_inv[kBlock];
  __shared__ uint2 tile[kBlock][16];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int r0 = static_cast<int>(blockIdx.x / p.tiles_x) * kBlock, c0 = static_cast<int>(blockIdx.x % p.tiles_x) * kBlock;
  const int nr = min(kBlock, p.rows - r0), nc = min(kBlock, p.cols - c0);
  const T* src = static_cast<const T*>(p.x) + static_cast<long long>(r0 + rg * 8) * p.ldx + c0 + cg * 8;
  grid_dependency_wait();
  P x[8][PIECES];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < PIECES; ++k)
      load_piece<TYPE, SHIFT>(x[i][k], src + i * p.ldx + k * PER, rg * 8 + i < nr ? nc - cg * 8 - k * PER : 0);
  auto at = [&](int i, int j) { return x[i][j / PER].get(j % PER); };
  const int rb = r0 / kBlock, cb = c0 / kBlock;
  float inv[8];
  if (p.tall > 1) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, magnitude(at(i, j)));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((tid & 31) == 0) tops[0][tid >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, tops[0][tid & 7]);
    const float scale = block_scale(top, inv[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) inv[j] = inv[0];
    if (tid == 0) p.scale[(p.transpose ? cb : rb) * p.s_row + (p.transpose ? rb : cb) * p.s_block] = scale;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(at(i, j)));
      tops[rg][cg * 8 + j] = top;
    }
    __syncthreads();
    if (tid < kBlock) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, tops[i][tid]);
      float one;
      const float scale = block_scale(top, one);
      col_inv[tid] = one;
      if (tid < nc) p.scale[static_cast<long long>(c0 + tid) * p.s_row + rb * p.s_block] = scale;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = col_inv[cg * 8 + j];
  }
  if (!p.transpose) {
    // (tall) 8 neighbouring elements of a row of q a thread
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rg * 8 + i;
      if (r >= nr || cg * 8 >= nc) continue;
      uint8_t* dst = p.q + static_cast<long long>(r0 + r) * p.ldq + c0 + cg * 8;
      if (cg * 8 + 8 <= nc && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(four_e4m3(at(i, 0) * inv[0], at(i, 1) * inv[1], at(i, 2) * inv[2], at(i, 3) * inv[3]),
                       four_e4m3(at(i, 4) * inv[4], at(i, 5) * inv[5], at(i, 6) * inv[6], at(i, 7) * inv[7]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (cg * 8 + j < nc) dst[j] = to_e4m3(at(i, j) * inv[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[cg * 8 + j][rg ^ cg] =
          make_uint2(four_e4m3(at(0, j) * inv[j], at(1, j) * inv[j], at(2, j) * inv[j], at(3, j) * inv[j]),
                     four_e4m3(at(4, j) * inv[j], at(5, j) * inv[j], at(6, j) * inv[j], at(7, j) * inv[j]));
    __syncthreads();
    // 16 neighbouring elements of a row of q a thread, eight threads a row
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = k * 32 + (tid >> 3), r = (tid & 7) * 16;
      if (c >= nc || r >= nr) continue;
      const uint2 lo = tile[c][(2 * (tid & 7)) ^ (c >> 3)], hi = tile[c][(2 * (tid & 7) + 1) ^ (c >> 3)];
      uint8_t* dst = p.q + static_cast<long long>(c0 + c) * p.ldq + r0 + r;
      if (r + 16 <= nr && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (r + e < nr) dst[e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
  grid_launch_dependents();
}

template <int TYPE>
cudaError_t launch_quantize(QuantParams p, bool shift, cudaStream_t s) {
  if (p.tall == 1 && !p.transpose) {
    constexpr int rows = 256 / (kBlock / 16);  // of a thread block
    const int64_t groups = (int64_t(p.rows) + rows - 1) / rows, blocks = (p.cols + kBlock - 1) / kBlock;
    // about eight blocks of a row each, or as many thread blocks as keep the GPU busy. 8192 x 8192 BF16, shares of a
    // row's 64 blocks 2 / 4 / 8 / 16 / 64: 36.2 / 35.4 / 31.4 / 33.9 / 45.4 us; 8192 x 1024, 1 / 2 / 4 / 8: 6.8 / 5.3 /
    // 5.8 / 6.4; 1000 x 4096, 4 / 8 / 16 / 32: 6.2 / 3.9 / 3.3 / 3.7.
    const int64_t fill = (512 + groups - 1) / groups, want = fill > blocks / 8 ? fill : blocks / 8;
    p.shares = int(want < blocks ? want : blocks);
    const int grid = int(groups * p.shares);
    return shift ? launch_dependent(quantize_rows_kernel<TYPE, true>, grid, 256, 0, s, 1, p)
                 : launch_dependent(quantize_rows_kernel<TYPE, false>, grid, 256, 0, s, 1, p);
  }
  const int64_t tiles = int64_t(p.tiles_x) * ((p.rows + kBlock - 1) / kBlock);
  return shift ? launch_dependent(quantize_tile_kernel<TYPE, true>, int(tiles), 256, 0, s, 1, p)
               : launch_dependent(quantize_tile_kernel<TYPE, false>, int(tiles), 256, 0, s, 1, p);
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
  const bool shift = misaligned(x, 16) || (rows > 1 && (ldx * es) % 16 != 0);
  const bool wide_q = !misaligned(q, 16) && (rows == 1 || ldq % 16 == 0);
  QuantParams p = {x,          q,         scale,          (long long)ldx, (long long)ldq, (long long)s_row, (long long)s_block,
                   int(rows),  int(cols), block_rows,     transpose,      int((cols + kBlock - 1) / kBlock), 1, wide_q};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_quantize<GEMM_TYPE_F16>(p, shift, s)
                        : type == GEMM_TYPE_BF16 ? launch_quantize<GEMM_TYPE_BF16>(p, shift, s)
                                                 : launch_quantize<GEMM_TYPE_F32>(p, shift, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
