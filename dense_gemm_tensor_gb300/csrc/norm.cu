// Root-mean-square norm with the residual's addition and an optional 8-bit
// output, and its gradient (gemm_rmsnorm, gemm_rmsnorm_backward).
//
//   h = round(x + residual);  r = (mean(h^2) + eps)^-1/2;  y = h r w
//   dx = r (g - xhat mean(g xhat)) + dh,  g = dy w, xhat = h r;  dw = sum over rows of dy xhat
//
// Both are bound by HBM: each matrix is read or written once. A row stays in
// the registers of the `tpr` threads that own it (at most 64 bytes each)
// between the reductions and the output, so nothing is read twice. While a row
// is reduced and stored its threads load nothing, so several blocks share an SM:
// 64 registers a thread let 1024 threads keep two matrices' loads in flight.
//
// The three ways to reach memory (ALIGNED, FLAT, SINGLE) are in row.cuh.
#include "row.cuh"

namespace dgt {
namespace {

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

template <int TYPE, int MODE, int EPT, bool Q8>
__global__ void __launch_bounds__(kNormThreads<TYPE, EPT>, kNormThreads<TYPE, EPT> == 512 ? 2 : 1)
    rmsnorm_kernel(const NormParams p) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = MODE == SINGLE ? 1 : 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][2][32];
  extern __shared__ uint4 dynamic[];
  T* shared_w = reinterpret_cast<T*>(dynamic);
  const int per_block = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
  Row<MODE, VEC> r(threadIdx.x - sub * p.tpr, p.tpr, p.cols);
  const RowWarps row_warps(p.tpr, sub);
  grid_dependency_wait();
  if constexpr (MODE == FLAT) stage_weights<TYPE, VEC>(shared_w, p.weight, p.cols);
  int turn = 0;
  for (long long r0 = static_cast<long long>(blockIdx.x) * per_block; r0 < p.rows;
       r0 += static_cast<long long>(gridDim.x) * per_block, turn ^= 1) {
    const long long row = r0 + sub;
    const bool in = row < p.rows;
    r.at(row);
    P h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) r.load(h[i], p.x, row, p.ldx, i, in);
    if (p.residual != nullptr) {
      P a[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) r.load(a[i], p.residual, row, p.ldr, i, in);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = h[i].get(j) + a[i].get(j);
        h[i].set(x);
        if (p.h != nullptr) r.store(h[i], p.h, row, p.ldh, i, in);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += h[i].get(j) * h[i].get(j);
    ss = row_warps.sum(ss, red[turn][0]);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.cols) + p.eps);
    if (p.rstd != nullptr && in && r.tid == 0) p.rstd[row] = rstd;
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[VEC];
        load_weights<MODE, TYPE, VEC>(w, r, p.weight, shared_w, i);
        P o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = h[i].get(j) * rstd * w[j];
        o.set(w);
        r.store(o, p.y, row, p.ldy, i, in);
      }
    } else {
      // |y| compared by bit pattern: a NaN is above every number and reaches the scale
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[VEC];
        load_weights<MODE, TYPE, VEC>(w, r, p.weight, shared_w, i);
#pragma unroll
        for (int j = 0; j < VEC; ++j) top = max(top, __float_as_uint(h[i].get(j) * rstd * w[j]) & 0x7FFFFFFFu);
      }
      const float amax = __uint_as_float(row_warps.max_bits(top, red[turn][1]));
      const float scale = (amax < 1e-12f ? 1e-12f : amax) / kE4M3Max;
      const float inv = 1.0f / scale;
      if (in && r.tid == 0) p.scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float w[VEC];
        load_weights<MODE, TYPE, VEC>(w, r, p.weight, shared_w, i);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = h[i].get(j) * rstd * w[j] * inv;
        r.store_q8(w, p.y, row, p.ldy, i, in);
      }
    }
  }
  grid_launch_dependents();
}

constexpr int kGradEpt = 16;  // elements of a row per thread of the gradient

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

// A thread owns the same columns of every row (ALIGNED, SINGLE) and adds dw up
// in registers; FLAT rows move against the threads, and dw is in shared memory,
// where a column meets one thread a row and the rows' reductions separate them.
// ALIGNED with AHEAD: each thread copies its pieces of the next row to its own
// places in shared memory (cp.async) before it works on this one, so that loads
// are in flight during the reduction and the stores, and nothing but the thread
// itself waits for them (without: 8192 x 4096 BF16 took 60-73 us). It reads a
// piece from its place once for the sums and once for the output, so that
// registers hold one piece at a time, and has the next row's rstd loaded: with
// the row in registers the same took 58 us, 4097 x 5120 37.6 us. Now 51.7 us
// (5.2 TB/s) and 34.7 us (4.8 TB/s), of which the second launch is 4 us.
template <int TYPE, int MODE, bool AHEAD>
__global__ void __launch_bounds__(int(kMaxCols) / kGradEpt, 1) rmsnorm_grad_kernel(const NormGradParams p) {
  constexpr int EPT = kGradEpt;
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = MODE == SINGLE ? 1 : 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][32];
  extern __shared__ uint4 dynamic[];
  // ALIGNED, SINGLE: (rows of the block - 1) x cols partial sums; FLAT: dw of each row of the block, then the weights
  float* sums = reinterpret_cast<float*>(dynamic);
  const int places = (p.cols + VEC - 1) / VEC * VEC;
  const int per_block = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
  T* shared_w = reinterpret_cast<T*>(sums + per_block * places);
  Row<MODE, VEC> r(threadIdx.x - sub * p.tpr, p.tpr, p.cols);
  const RowWarps row_warps(p.tpr, sub);
  const long long step = static_cast<long long>(gridDim.x) * per_block;
  // AHEAD: piece i of h, dy or dh (m = 0, 1, 2) of stage s
  auto cell = [&](int s, int m, int i) { return dynamic + ((s * 3 + m) * NV + i) * blockDim.x + threadIdx.x; };
  auto fetch = [&](long long row, int s) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (r.whole(i)) {
        if (row < p.rows) {
          copy16(cell(s, 0, i), static_cast<const T*>(p.h) + row * p.ldh + r.lo(i));
          copy16(cell(s, 1, i), static_cast<const T*>(p.dy) + row * p.lddy + r.lo(i));
          if (p.dh != nullptr) copy16(cell(s, 2, i), static_cast<const T*>(p.dh) + row * p.lddh + r.lo(i));
        } else if (per_block > 1) {  // a row past the last one counts as zeros
          *cell(s, 0, i) = *cell(s, 1, i) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const long long start = static_cast<long long>(blockIdx.x) * per_block + sub;
  grid_dependency_wait();
  if constexpr (AHEAD) {
    // zeros where no copy lands: past the last column, and dh where there is none
#pragma unroll
    for (int i = 0; i < NV; ++i)
      for (int c = 0; c < 6; ++c)
        if (!r.whole(i) || (c % 3 == 2 && p.dh == nullptr)) *cell(c / 3, c % 3, i) = make_uint4(0u, 0u, 0u, 0u);
    fetch(start, 0);
  }
  float rstd_ahead = AHEAD && start < p.rows ? p.rstd[start] : 0.0f;
  float2 dw[MODE == FLAT ? 1 : EPT / 2];  // element e of the thread's EPT: half e & 1 of dw[e / 2]
  if constexpr (MODE == FLAT) {
    for (int i = threadIdx.x; i < per_block * places; i += blockDim.x) sums[i] = 0.0f;
    stage_weights<TYPE, VEC>(shared_w, p.weight, p.cols);
  } else {
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) dw[e] = make_float2(0.0f, 0.0f);
  }
  int turn = 0;
  for (long long r0 = static_cast<long long>(blockIdx.x) * per_block; r0 < p.rows; r0 += step, turn ^= 1) {
    const long long row = r0 + sub;
    const bool in = row < p.rows;
    r.at(row);
    P h[NV], dy[NV], dh[NV];
    if constexpr (AHEAD) {
      fetch(row + step, turn ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // this row's pieces have landed
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        r.load(h[i], p.h, row, p.ldh, i, in);
        r.load(dy[i], p.dy, row, p.lddy, i, in);
      }
      if (p.dh != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) r.load(dh[i], p.dh, row, p.lddh, i, in);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) dh[i].zero();
      }
    }
    // AHEAD: a piece from its place, once for each use: registers hold one piece at a time, not the row's
    auto take = [&](P(&v)[NV], int m, int i) {
      if constexpr (AHEAD) v[i].load(reinterpret_cast<const T*>(cell(turn, m, i)));
    };
    // xhat = h rstd is formed first, and dx = rstd g - (rstd mean(g xhat)) xhat + dh: every factor stays of the size of
    // dy or of dx. (rstd^3 mean(g h) would leave fp32 for rows of 1e13 and above, or of 1e-13 with a tiny eps.)
    // ALIGNED takes two elements to an instruction.
    const float rstd = AHEAD ? rstd_ahead : in ? p.rstd[row] : 0.0f;
    if constexpr (AHEAD) rstd_ahead = row + step < p.rows ? p.rstd[row + step] : 0.0f;
    float2 dots = make_float2(0.0f, 0.0f);  // ALIGNED
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[VEC];
      load_weights<MODE, TYPE, VEC>(w, r, p.weight, shared_w, i);
      take(h, 0, i);
      take(dy, 1, i);
      if constexpr (MODE == ALIGNED) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 xhat = __fmul2_rn(h[i].two(j), make_float2(rstd, rstd)), d = dy[i].two(j);
          dots = __ffma2_rn(__fmul2_rn(d, make_float2(w[j], w[j + 1])), xhat, dots);
          float2& sum = dw[(i * VEC + j) / 2];
          sum = __ffma2_rn(d, xhat, sum);
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xhat = h[i].get(j) * rstd, d = dy[i].get(j);
          dot = fmaf(d * w[j], xhat, dot);
          if constexpr (MODE == FLAT) {
            const int c = r.lo(i) + j;
            if (in && c >= 0 && c < p.cols) sums[sub * places + r.place(i, j)] += d * xhat;
          } else {
            float& sum = i & 1 ? dw[i / 2].y : dw[i / 2].x;
            sum = fmaf(d, xhat, sum);
          }
        }
      }
    }
    const float back = rstd * (row_warps.sum(MODE == ALIGNED ? dots.x + dots.y : dot, red[turn]) / static_cast<float>(p.cols));
    if (MODE == FLAT && p.tpr <= 32) __syncwarp();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[VEC];
      load_weights<MODE, TYPE, VEC>(w, r, p.weight, shared_w, i);
      take(h, 0, i);
      take(dy, 1, i);
      take(dh, 2, i);
      P o;
      if constexpr (MODE == ALIGNED) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 g = __fmul2_rn(dy[i].two(j), make_float2(w[j], w[j + 1]));
          const float2 xhat = __fmul2_rn(h[i].two(j), make_float2(rstd, rstd));
          const float2 v = __ffma2_rn(g, make_float2(rstd, rstd), __ffma2_rn(xhat, make_float2(-back, -back), dh[i].two(j)));
          w[j] = v.x;
          w[j + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = fmaf(dy[i].get(j) * w[j], rstd, fmaf(h[i].get(j) * rstd, -back, dh[i].get(j)));
      }
      o.set(w);
      r.store(o, p.dx, row, p.lddx, i, in);
    }
  }
  if constexpr (AHEAD) asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* out = p.partial + static_cast<long long>(blockIdx.x) * p.cols;
  if constexpr (MODE == FLAT) {
    __syncthreads();
    const int per = places / VEC;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      float s = 0.0f;
      for (int i = 0; i < per_block; ++i) s += sums[i * places + (c % VEC) * per + c / VEC];
      out[c] = s;
    }
  } else {
    // the block's sum over its rows, in row order; four columns a store
    constexpr int RUN = VEC < 4 ? 1 : 4;
    auto each = [&](auto use) {
#pragma unroll
      for (int e = 0; e < EPT; e += RUN)
        if (r.whole(e / VEC)) use(r.lo(e / VEC) + e % VEC, e);
    };
    auto value = [&](int e) -> float& { return e & 1 ? dw[e / 2].y : dw[e / 2].x; };
    auto store = [&](float* to, int e) {
      if constexpr (RUN == 1)
        *to = value(e);
      else
        *reinterpret_cast<float4*>(to) = make_float4(value(e), value(e + 1), value(e + 2), value(e + 3));
    };
    if (per_block > 1) {
      __syncthreads();
      if (sub > 0) each([&](int c, int e) { store(sums + (sub - 1) * p.cols + c, e); });
      __syncthreads();
      if (sub == 0)
        for (int s = 0; s + 1 < per_block; ++s)
          each([&](int c, int e) {
#pragma unroll
            for (int k = 0; k < RUN; ++k) value(e + k) += sums[s * p.cols + c + k];
          });
    }
    if (sub == 0) each([&](int c, int e) { store(out + c, e); });
  }
  grid_launch_dependents();
}

// dw[j] = sum of the blocks' partial rows: 32 columns a block, 32 threads a
// column, each a fixed share of the rows, added in order of the threads.
template <int TYPE>
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* partial, int rows, int cols, void* dw) {
  using E = Elem<TYPE>;
  __shared__ float part[32][33];
  grid_dependency_wait();
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int r = g; r < rows; r += 32) s += __ldcg(partial + static_cast<long long>(r) * cols + col);
  }
  part[g][c] = s;
  __syncthreads();
  // warp g adds up column g of the block
  s = warp_sum(part[c][g]);
  const int mine = blockIdx.x * 32 + g;
  if (c == 0 && mine < cols) static_cast<typename E::T*>(dw)[mine] = E::put(s);
  grid_launch_dependents();
}

// Blocks of the gradient, at most: each leaves one partial row of dw, which
// costs a write and a read, so wide rows have about three for each of a GB300's
// 152 SMs (what fits them at 64 registers) and narrow ones, whose blocks are
// small, more. (Numbers, since the size of the workspace goes by them, on a machine
// without a GPU too.) BF16 with dh, 304 / 456 / 608 / 912 blocks, us: 8192 x 1024 19.1 / 18.4 /
// 17.7 / 22.2, 30000 x 1024 55.3 / 47.8 / 45.0 / 53.3, 8192 x 2048 33.3 / 30.0 / 29.1 / 33.3,
// 8192 x 4096 60.8 / 52.0 / 48.8 / 56.0, 8192 x 8192 89.7 / 106 / 94 / 98: no one number is best for wide rows.
int grad_blocks(int64_t cols) { return cols <= 2048 ? 608 : 456; }

template <int TYPE, int MODE, int EPT>
cudaError_t launch_norm_mode(const NormParams& p, bool q8, int grid, int block, size_t smem, cudaStream_t s) {
  return q8 ? launch_dependent(rmsnorm_kernel<TYPE, MODE, EPT, true>, grid, block, smem, s, 1, p)
            : launch_dependent(rmsnorm_kernel<TYPE, MODE, EPT, false>, grid, block, smem, s, 1, p);
}

template <int TYPE>
cudaError_t launch_norm(const NormParams& p, int mode, bool few, bool q8, int grid, int block, cudaStream_t s) {
  const size_t smem = mode == FLAT ? size_t(p.cols + 8) * sizeof(typename Elem<TYPE>::T) : 0;
  if (mode == ALIGNED)
    return few ? launch_norm_mode<TYPE, ALIGNED, 8>(p, q8, grid, block, smem, s)
               : launch_norm_mode<TYPE, ALIGNED, kFullEpt<TYPE, ALIGNED>>(p, q8, grid, block, smem, s);
  if (mode == FLAT)
    return few ? launch_norm_mode<TYPE, FLAT, 8>(p, q8, grid, block, smem, s)
               : launch_norm_mode<TYPE, FLAT, kFullEpt<TYPE, FLAT>>(p, q8, grid, block, smem, s);
  return few ? launch_norm_mode<TYPE, SINGLE, 8>(p, q8, grid, block, smem, s)
             : launch_norm_mode<TYPE, SINGLE, kFullEpt<TYPE, SINGLE>>(p, q8, grid, block, smem, s);
}

// Dynamic shared memory of the gradient's kernel.
size_t grad_smem(const NormGradParams& p, int mode, bool ahead, int block, int es) {
  if (mode == FLAT) return size_t(p.cols + 8) * (size_t(block / p.tpr) * sizeof(float) + es);
  const size_t sums = size_t(block / p.tpr - 1) * size_t(p.cols) * sizeof(float);
  const size_t stages = ahead ? size_t(2 * 3) * kGradEpt * es * size_t(block) : 0;
  return sums > stages ? sums : stages;
}

// Most dynamic shared memory that a launch of the gradient takes: AHEAD goes up to here, and a FLAT row of
// kMaxFlatCols has 86 KB.
constexpr size_t kGradSmem = 200 * 1024;

// Launches one build of the gradient's kernel. Its limit is a property of the kernel, not of the launch, so it is set
// once, to the most that any launch takes: other host threads may be launching it with other sizes.
template <int TYPE, int MODE, bool AHEAD>
cudaError_t launch_norm_grad_mode(const NormGradParams& p, int dev, int grid, int block, size_t smem, cudaStream_t s) {
  static int configured[64] = {};
  auto kern = rmsnorm_grad_kernel<TYPE, MODE, AHEAD>;
  if (dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kGradSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, grid, block, smem, s, 1, p);
}

template <int TYPE>
cudaError_t launch_norm_grad(const NormGradParams& p, int mode, bool ahead, int dev, int grid, int block, void* dw,
                             cudaStream_t s) {
  const size_t smem = grad_smem(p, mode, ahead, block, sizeof(typename Elem<TYPE>::T));
  const cudaError_t e = mode == ALIGNED
                            ? (ahead ? launch_norm_grad_mode<TYPE, ALIGNED, true>(p, dev, grid, block, smem, s)
                                     : launch_norm_grad_mode<TYPE, ALIGNED, false>(p, dev, grid, block, smem, s))
                        : mode == FLAT ? launch_norm_grad_mode<TYPE, FLAT, false>(p, dev, grid, block, smem, s)
                                       : launch_norm_grad_mode<TYPE, SINGLE, false>(p, dev, grid, block, smem, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_weight_sum_kernel<TYPE>, (p.cols + 31) / 32, 1024, 0, s, 1, p.partial, grid, p.cols, dw);
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
  int mode = SINGLE;
  if (cols % v == 0 && aligned(x, ldx, es, 16) && aligned(weight, 0, es, 16) &&
      (residual == nullptr || aligned(residual, ldr, es, 16)) && (h == nullptr || aligned(h, ldh, es, 16)) &&
      aligned(y, ldy, eo, v * eo))
    mode = ALIGNED;
  else if (cols <= kMaxFlatCols && flat(x, ldx, cols, 16) && (residual == nullptr || flat(residual, ldr, cols, 16)) &&
           (h == nullptr || flat(h, ldh, cols, 16)) && flat(y, ldy, cols, v * eo))
    mode = FLAT;
  NormParams p = {x,   residual, weight, h,   y,         y_scale,   rstd, (long long)ldx, (long long)ldr,
                  (long long)ldh, (long long)ldy, int(rows), int(cols), 0, eps};
  // Eight elements a thread while the rows leave threads to spare (a row's latency is then one load of each
  // matrix and two reductions), 64 bytes once they fill the GPU (more loads in flight for each reduction) and past
  // what 1024 threads hold. BF16 with a residual, eight elements / 64 bytes, us: 608 x 1024 2.6 / 3.0, 1216 x 1024
  // (the limit) 3.4 / 3.3, 1 x 4096 2.3 / 2.9, 304 x 4096 (the limit) 2.9 / 3.4, 608 x 4096 5.4 / 4.8,
  // 152 x 7680 3.1 / 3.6, 304 x 7680 5.8 / 4.8.
  const bool few = cols <= 8000 && rows * cols <= int64_t(ctx.sm_count) * 8192;
  p.tpr = threads_per_row(cols, few ? 8 : mode == SINGLE ? 16 : 64 / es, mode, v);
  // FLAT blocks stage the weights, so they are few and take many rows: blocks of 512 / 128 threads, us: 2048 x 4095
  // 23.3 / 31.7, 8192 x 4095 84 / 103, 8192 x 1023 40.4 / 44.5, 30000 x 515 70 / 82. Others of 32 / 128 / 256 / 512:
  // 8192 x 1024 12.2 / 10.3 / 10.0 / 10.3, 30000 x 512 20.2 / 19.9 / 20.0 / 20.4, 100 x 512 2.1 / 2.1 / 2.1 / 2.4.
  const int least = mode == FLAT && !few ? 512 : 128;
  const int block = p.tpr < least ? least / p.tpr * p.tpr : p.tpr;
  const int64_t need = (rows + block / p.tpr - 1) / (block / p.tpr);
  const int64_t most = int64_t(ctx.sm_count) * (mode == FLAT ? 1024 / block + 1 : 2048 / block);
  const int grid = int(need < most ? need : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_norm<GEMM_TYPE_F16>(p, mode, few, q8, grid, block, s)
                        : type == GEMM_TYPE_BF16 ? launch_norm<GEMM_TYPE_BF16>(p, mode, few, q8, grid, block, s)
                                                 : launch_norm<GEMM_TYPE_F32>(p, mode, few, q8, grid, block, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int64_t gemm_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  return (rows < grad_blocks(cols) ? rows : grad_blocks(cols)) * cols * int64_t(sizeof(float));
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
  int mode = SINGLE;
  if (cols % v == 0 && aligned(dy, lddy, es, 16) && aligned(h, ldh, es, 16) && aligned(weight, 0, es, 16) &&
      aligned(dx, lddx, es, 16) && (dh == nullptr || aligned(dh, lddh, es, 16)))
    mode = ALIGNED;
  else if (cols <= kMaxFlatCols && flat(dy, lddy, cols, 16) && flat(h, ldh, cols, 16) && flat(dx, lddx, cols, 16) &&
           (dh == nullptr || flat(dh, lddh, cols, 16)))
    mode = FLAT;
  NormGradParams p = {dy, h, weight, rstd, dh, dx, static_cast<float*>(workspace), (long long)lddy, (long long)ldh,
                      (long long)lddh, (long long)lddx, int(rows), int(cols), 0};
  p.tpr = threads_per_row(cols, kGradEpt, mode, v);
  const int block = p.tpr >= 256 ? p.tpr : 256 / p.tpr * p.tpr;
  const bool ahead = mode == ALIGNED && grad_smem(p, mode, true, block, es) <= kGradSmem;
  const int64_t need = (rows + block / p.tpr - 1) / (block / p.tpr);
  const int grid = int(need < grad_blocks(cols) ? need : grad_blocks(cols));
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_norm_grad<GEMM_TYPE_F16>(p, mode, ahead, ctx.dev, grid, block, dw, s)
                        : type == GEMM_TYPE_BF16 ? launch_norm_grad<GEMM_TYPE_BF16>(p, mode, ahead, ctx.dev, grid, block, dw, s)
                                                 : launch_norm_grad<GEMM_TYPE_F32>(p, mode, ahead, ctx.dev, grid, block, dw, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
