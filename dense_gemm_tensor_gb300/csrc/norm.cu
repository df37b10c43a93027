// Root-mean-square norm with the residual's addition and an optional 8-bit
// output, and its gradient (gemm_rmsnorm, gemm_rmsnorm_backward).
//
//   h = round(x + residual);  r = (mean(h^2) + eps)^-1/2;  y = h r w
//   dx = r (g - xhat mean(g xhat)) + dh,  g = dy w, xhat = h r;  dw = sum over rows of dy xhat
//
// Both are bound by HBM: each matrix is read or written once. A row stays in
// the registers of the `tpr` threads that own it (EPT elements each at most)
// between the reductions and the output, so nothing is read twice; a thread
// owns the same columns of every row it meets, so the weights are loaded once
// and dw accumulates in registers. 16-byte accesses where base, pitch and
// width allow, single elements otherwise.
#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kMaxThreads = 512;       // of a block whose threads hold more than 8 elements of a row
constexpr int64_t kMaxCols = 16384;    // 32 elements for each of them
constexpr float kE4M3Max = 448.0f;

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* h;
  void* y;
  float* scale;
  float* rstd;
  long long ldx, ldr, ldh, ldy;
  int rows, cols, tpr;
  float eps;
};

template <int TYPE, int VEC, int EPT, bool Q8>
__global__ void __launch_bounds__(EPT == 8 ? 1024 : kMaxThreads) rmsnorm_kernel(const NormParams p) {
  using P = Pack<TYPE, VEC>;
  using T = typename P::T;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][2][32];
  const int tid = threadIdx.x % p.tpr;
  const int per_block = blockDim.x / p.tpr;
  const int nvec = p.cols / VEC;
  grid_dependency_wait();
  P w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i].zero();
    if (i * p.tpr + tid < nvec) w[i].load(static_cast<const T*>(p.weight) + (i * p.tpr + tid) * VEC);
  }
  int turn = 0;
  for (long long r0 = static_cast<long long>(blockIdx.x) * per_block; r0 < p.rows;
       r0 += static_cast<long long>(gridDim.x) * per_block, turn ^= 1) {
    const long long row = r0 + threadIdx.x / p.tpr;
    const bool in = row < p.rows;
    P h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      h[i].zero();
      if (in && i * p.tpr + tid < nvec) h[i].load(static_cast<const T*>(p.x) + row * p.ldx + (i * p.tpr + tid) * VEC);
    }
    if (p.residual != nullptr) {
      P a[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        a[i].zero();
        if (in && i * p.tpr + tid < nvec)
          a[i].load(static_cast<const T*>(p.residual) + row * p.ldr + (i * p.tpr + tid) * VEC);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i].put(j, h[i].get(j) + a[i].get(j));
        if (p.h != nullptr && in && i * p.tpr + tid < nvec)
          h[i].store(static_cast<T*>(p.h) + row * p.ldh + (i * p.tpr + tid) * VEC);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += h[i].get(j) * h[i].get(j);
    ss = row_sum(ss, p.tpr, red[turn][0]);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.cols) + p.eps);
    if (p.rstd != nullptr && in && tid == 0) p.rstd[row] = rstd;
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        P o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.put(j, h[i].get(j) * rstd * w[i].get(j));
        if (in && i * p.tpr + tid < nvec) o.store(static_cast<T*>(p.y) + row * p.ldy + (i * p.tpr + tid) * VEC);
      }
    } else {
      // |y| compared by bit pattern: a NaN is above every number and reaches the scale
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          top = max(top, __float_as_uint(h[i].get(j) * rstd * w[i].get(j)) & 0x7FFFFFFFu);
      const float amax = __uint_as_float(row_max_bits(top, p.tpr, reinterpret_cast<uint32_t*>(red[turn][1])));
      const float scale = (amax < 1e-12f ? 1e-12f : amax) / kE4M3Max;
      const float inv = 1.0f / scale;
      if (in && tid == 0) p.scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = h[i].get(j) * rstd * w[i].get(j) * inv;
        if (in && i * p.tpr + tid < nvec)
          store_e4m3<VEC>(static_cast<uint8_t*>(p.y) + row * p.ldy + (i * p.tpr + tid) * VEC, o);
      }
    }
  }
  grid_launch_dependents();
}

struct NormGradParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;
  void* dx;
  float* partial;  // one row of `cols` per block
  long long lddy, ldh, lddh, lddx;
  int rows, cols, tpr;
};

template <int TYPE, int VEC, int EPT>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_grad_kernel(const NormGradParams p) {
  using P = Pack<TYPE, VEC>;
  using T = typename P::T;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][32];
  extern __shared__ float sums[];  // (rows of the block - 1) x cols
  const int tid = threadIdx.x % p.tpr, sub = threadIdx.x / p.tpr;
  const int per_block = blockDim.x / p.tpr;
  const int nvec = p.cols / VEC;
  grid_dependency_wait();
  P w[NV];
  float dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i].zero();
    if (i * p.tpr + tid < nvec) w[i].load(static_cast<const T*>(p.weight) + (i * p.tpr + tid) * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0;
  for (long long r0 = static_cast<long long>(blockIdx.x) * per_block; r0 < p.rows;
       r0 += static_cast<long long>(gridDim.x) * per_block, turn ^= 1) {
    const long long row = r0 + sub;
    const bool in = row < p.rows;
    P h[NV], dy[NV], dh[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      h[i].zero();
      dy[i].zero();
      dh[i].zero();
      const int at = (i * p.tpr + tid) * VEC;
      if (in && i * p.tpr + tid < nvec) {
        h[i].load(static_cast<const T*>(p.h) + row * p.ldh + at);
        dy[i].load(static_cast<const T*>(p.dy) + row * p.lddy + at);
        if (p.dh != nullptr) dh[i].load(static_cast<const T*>(p.dh) + row * p.lddh + at);
      }
    }
    const float rstd = in ? p.rstd[row] : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xhat = h[i].get(j) * rstd, d = dy[i].get(j);
        dot += d * w[i].get(j) * xhat;
        dw[i][j] += d * xhat;
      }
    const float mean = row_sum(dot, p.tpr, red[turn]) / static_cast<float>(p.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      P o;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        o.put(j, rstd * (dy[i].get(j) * w[i].get(j) - h[i].get(j) * rstd * mean) + dh[i].get(j));
      if (in && i * p.tpr + tid < nvec) o.store(static_cast<T*>(p.dx) + row * p.lddx + (i * p.tpr + tid) * VEC);
    }
  }
  // the block's sum over its rows, in row order
  if (per_block > 1) {
    __syncthreads();
    if (sub > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (i * p.tpr + tid < nvec) sums[(sub - 1) * p.cols + (i * p.tpr + tid) * VEC + j] = dw[i][j];
    }
    __syncthreads();
    if (sub == 0) {
      for (int s = 0; s + 1 < per_block; ++s)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (i * p.tpr + tid < nvec) dw[i][j] += sums[s * p.cols + (i * p.tpr + tid) * VEC + j];
    }
  }
  if (sub == 0) {
    float* out = p.partial + static_cast<long long>(blockIdx.x) * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * p.tpr + tid < nvec) {
        if constexpr (VEC == 1) {
          out[i * p.tpr + tid] = dw[i][0];
        } else {
#pragma unroll
          for (int j = 0; j < VEC; j += 4)
            *reinterpret_cast<float4*>(out + (i * p.tpr + tid) * VEC + j) =
                make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
        }
      }
  }
  grid_launch_dependents();
}

// dw[j] = sum of the blocks' partial rows: 32 columns a block, eight threads a
// column, each a fixed eighth of the rows.
template <int TYPE>
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const float* partial, int rows, int cols, void* dw) {
  using E = Elem<TYPE>;
  __shared__ float part[8][33];
  grid_dependency_wait();
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int r = g; r < rows; r += 8) s += __ldcg(partial + static_cast<long long>(r) * cols + col);
  }
  part[g][c] = s;
  __syncthreads();
  if (g == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][c];
    static_cast<typename E::T*>(dw)[col] = E::put(s);
  }
  grid_launch_dependents();
}

// Blocks of the gradient: each leaves one partial row of dw, so there are no
// more than two for each of a GB300's 152 SMs.
constexpr int kGradBlocks = 304;

bool aligned(const void* p, int64_t ld, int es, int to) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * es)) % to) == 0;
}

// Threads that own a row of `cols` elements, `ept` each: whole warps.
int threads_per_row(int64_t cols, int ept) { return int((cols + 32 * ept - 1) / (32 * ept) * 32); }

bool bad_type(int type) { return type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F32; }
bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 39); }

bool meet(const void* a, int64_t rows_a, int64_t cols_a, int64_t ld_a, int es_a, const void* b, int64_t rows_b,
          int64_t cols_b, int64_t ld_b, int es_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), a1 = a0 + uintptr_t(((rows_a - 1) * ld_a + cols_a) * es_a);
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(b), b1 = b0 + uintptr_t(((rows_b - 1) * ld_b + cols_b) * es_b);
  return a0 < b1 && b0 < a1;
}

template <int TYPE, int VEC, int EPT>
cudaError_t launch_norm_ept(const NormParams& p, bool q8, int grid, int block, cudaStream_t s) {
  return q8 ? launch_dependent(rmsnorm_kernel<TYPE, VEC, EPT, true>, grid, block, 0, s, 1, p)
            : launch_dependent(rmsnorm_kernel<TYPE, VEC, EPT, false>, grid, block, 0, s, 1, p);
}

template <int TYPE>
cudaError_t launch_norm(const NormParams& p, bool vec, int ept, bool q8, int grid, int block, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<TYPE>::T);
  if (vec) return ept == 8 ? launch_norm_ept<TYPE, V, 8>(p, q8, grid, block, s)
                           : launch_norm_ept<TYPE, V, 32>(p, q8, grid, block, s);
  return ept == 8 ? launch_norm_ept<TYPE, 1, 8>(p, q8, grid, block, s)
                  : launch_norm_ept<TYPE, 1, 32>(p, q8, grid, block, s);
}

template <int TYPE, int EPT>
cudaError_t launch_norm_grad(const NormGradParams& p, bool vec, int grid, int block, void* dw, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<TYPE>::T);
  const size_t smem = size_t(block / p.tpr - 1) * size_t(p.cols) * sizeof(float);
  cudaError_t e = vec ? launch_dependent(rmsnorm_grad_kernel<TYPE, V, EPT>, grid, block, smem, s, 1, p)
                      : launch_dependent(rmsnorm_grad_kernel<TYPE, 1, EPT>, grid, block, smem, s, 1, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_weight_sum_kernel<TYPE>, (p.cols + 31) / 32, 256, 0, s, 1, p.partial, grid, p.cols, dw);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_rmsnorm(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                 const void* weight, float eps, void* h, int64_t ldh, int y_type, void* y, int64_t ldy, float* y_scale,
                 float* rstd, void* stream) {
  if (bad_type(type) || (y_type != type && y_type != GEMM_TYPE_E4M3) || rows < 0 || cols < 0 || cols > kMaxCols ||
      rows >= (int64_t(1) << 31))
    return GEMM_ERR_INVALID_VALUE;
  const bool q8 = y_type == GEMM_TYPE_E4M3;
  if ((y_scale != nullptr) != q8 && rows > 0 && cols > 0) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (x == nullptr || weight == nullptr || y == nullptr || bad_ld(ldx, cols) || bad_ld(ldy, cols) ||
      (residual != nullptr && bad_ld(ldr, cols)))
    return GEMM_ERR_INVALID_VALUE;
  if (residual == nullptr) h = nullptr;  // h is x itself
  if (h != nullptr && bad_ld(ldh, cols)) return GEMM_ERR_INVALID_VALUE;
  const int es = type_bytes(type), eo = type_bytes(y_type);
  if (misaligned(x, es) || misaligned(residual, es) || misaligned(weight, es) || misaligned(h, es) ||
      misaligned(y, eo) || misaligned(y_scale, 4) || misaligned(rstd, 4))
    return GEMM_ERR_MISALIGNED;
  // an output may be an input's very buffer (each element is read, then written, by one thread), or apart from it
  auto clash = [&](const void* o, int64_t ldo, int e_o, const void* i, int64_t ldi) {
    if (o == nullptr || i == nullptr || (o == i && ldo == ldi && e_o == es)) return false;
    return meet(o, rows, cols, ldo, e_o, i, rows, cols, ldi, es);
  };
  if (clash(h, ldh, es, x, ldx) || clash(h, ldh, es, residual, ldr) || clash(y, ldy, eo, x, ldx) ||
      (residual != nullptr && meet(y, rows, cols, ldy, eo, residual, rows, cols, ldr, es)) ||
      (h != nullptr && meet(y, rows, cols, ldy, eo, h, rows, cols, ldh, es)) ||
      meet(y, rows, cols, ldy, eo, weight, 1, cols, cols, es) ||
      (h != nullptr && meet(h, rows, cols, ldh, es, weight, 1, cols, cols, es)))
    return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[7] = {x, weight, y, residual, h, y_scale, rstd};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  const int v = 16 / es;
  const bool vec = cols % v == 0 && aligned(x, ldx, es, 16) && aligned(weight, 0, es, 16) &&
                   (residual == nullptr || aligned(residual, ldr, es, 16)) && (h == nullptr || aligned(h, ldh, es, 16)) &&
                   aligned(y, ldy, eo, v * eo);
  NormParams p = {x,   residual, weight, h,   y,         y_scale,   rstd, (long long)ldx, (long long)ldr,
                  (long long)ldh, (long long)ldy, int(rows), int(cols), 0, eps};
  // Eight elements a thread while the rows leave threads to spare (a row's latency is then one load of each
  // matrix and two reductions), 32 once they fill the GPU (more loads in flight for each reduction).
  const int ept = cols <= 8192 && rows * cols <= int64_t(ctx.sm_count) * 8192 ? 8 : 32;
  p.tpr = threads_per_row(cols, ept);
  const int block = p.tpr < 128 ? 128 / p.tpr * p.tpr : p.tpr;
  const int64_t need = (rows + block / p.tpr - 1) / (block / p.tpr);
  const int64_t most = int64_t(ctx.sm_count) * (2048 / block);
  const int grid = int(need < most ? need : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_norm<GEMM_TYPE_F16>(p, vec, ept, q8, grid, block, s)
                        : type == GEMM_TYPE_BF16 ? launch_norm<GEMM_TYPE_BF16>(p, vec, ept, q8, grid, block, s)
                                                 : launch_norm<GEMM_TYPE_F32>(p, vec, ept, q8, grid, block, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int64_t gemm_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  return (rows < kGradBlocks ? rows : kGradBlocks) * cols * int64_t(sizeof(float));
}

int gemm_rmsnorm_backward(int type, int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* h,
                          int64_t ldh, const void* weight, const float* rstd, const void* dh, int64_t lddh, void* dx,
                          int64_t lddx, void* dw, void* workspace, int64_t workspace_bytes, void* stream) {
  if (bad_type(type) || rows < 0 || cols < 0 || cols > kMaxCols || rows >= (int64_t(1) << 31))
    return GEMM_ERR_INVALID_VALUE;
  if (cols == 0) return GEMM_OK;
  const int es = type_bytes(type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallContext ctx;
  if (dw == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (misaligned(dw, es)) return GEMM_ERR_MISALIGNED;
  if (rows == 0) {  // no rows: dw = 0
    const int st = begin_call(&ctx);
    if (st != GEMM_OK) return st;
    if (!on_device(dw, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
    return cudaMemsetAsync(dw, 0, size_t(cols) * es, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
  }
  if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr || workspace == nullptr ||
      bad_ld(lddy, cols) || bad_ld(ldh, cols) || bad_ld(lddx, cols) || (dh != nullptr && bad_ld(lddh, cols)) ||
      workspace_bytes < gemm_rmsnorm_backward_workspace(rows, cols))
    return GEMM_ERR_INVALID_VALUE;
  if (misaligned(dy, es) || misaligned(h, es) || misaligned(weight, es) || misaligned(rstd, 4) || misaligned(dh, es) ||
      misaligned(dx, es) || misaligned(workspace, 16))
    return GEMM_ERR_MISALIGNED;
  auto clash = [&](const void* i, int64_t ldi) {
    if (i == nullptr || (i == dx && ldi == lddx)) return false;
    return meet(dx, rows, cols, lddx, es, i, rows, cols, ldi, es);
  };
  if (clash(dy, lddy) || clash(dh, lddh) || clash(h, ldh) || meet(dx, rows, cols, lddx, es, weight, 1, cols, cols, es) ||
      meet(dx, rows, cols, lddx, es, dw, 1, cols, cols, es) || meet(dx, rows, cols, lddx, es, rstd, 1, rows, rows, 4))
    return GEMM_ERR_INVALID_VALUE;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[8] = {dy, h, weight, rstd, dx, dw, workspace, dh};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  const int v = 16 / es;
  const bool vec = cols % v == 0 && aligned(dy, lddy, es, 16) && aligned(h, ldh, es, 16) &&
                   aligned(weight, 0, es, 16) && aligned(dx, lddx, es, 16) && (dh == nullptr || aligned(dh, lddh, es, 16));
  NormGradParams p = {dy, h, weight, rstd, dh, dx, static_cast<float*>(workspace), (long long)lddy, (long long)ldh,
                      (long long)lddh, (long long)lddx, int(rows), int(cols), 0};
  const int ept = cols <= kMaxThreads * 16 ? 16 : 32;
  p.tpr = threads_per_row(cols, ept);
  const int block = p.tpr < 256 ? 256 / p.tpr * p.tpr : p.tpr;
  const int64_t need = (rows + block / p.tpr - 1) / (block / p.tpr);
  const int grid = int(need < kGradBlocks ? need : kGradBlocks);
  cudaError_t e;
  if (type == GEMM_TYPE_F16)
    e = ept == 16 ? launch_norm_grad<GEMM_TYPE_F16, 16>(p, vec, grid, block, dw, s)
                  : launch_norm_grad<GEMM_TYPE_F16, 32>(p, vec, grid, block, dw, s);
  else if (type == GEMM_TYPE_BF16)
    e = ept == 16 ? launch_norm_grad<GEMM_TYPE_BF16, 16>(p, vec, grid, block, dw, s)
                  : launch_norm_grad<GEMM_TYPE_BF16, 32>(p, vec, grid, block, dw, s);
  else
    e = ept == 16 ? launch_norm_grad<GEMM_TYPE_F32, 16>(p, vec, grid, block, dw, s)
                  : launch_norm_grad<GEMM_TYPE_F32, 32>(p, vec, grid, block, dw, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
