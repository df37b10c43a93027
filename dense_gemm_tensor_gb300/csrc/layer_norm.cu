// Layer norm with the residual's addition and an optional 8-bit output, and its
// gradient (gemm_layernorm, gemm_layernorm_backward).
//
//   h = round(x + residual);  m = mean(h);  r = (mean((h - m)^2) + eps)^-1/2;  y = (h - m) r w + b
//   xhat = (h - m) r,  g = dy w:  dx = r (g - mean(g)) - r mean(g xhat) xhat + dh
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Both are bound by HBM: each matrix is read or written once. As in the
// root-mean-square norm a row stays in its threads' registers, here between three
// reductions: the mean, the squares of what is left of it (two passes over
// registers: mean(h^2) - m^2 would cancel where the mean is large), and the 8-bit
// scale. The ways to reach memory are row.cuh's; FLAT rows go by their shift.
// 8192 x 8192 BF16 with a residual: 86 us to BF16 (6.2 TB/s), 78 to E4M3 (6.0); the
// gradient 107 (5.0 TB/s), of 4097 x 5120 45 (3.8; 53% of the issue slots, 42% of the
// warps: neither is full, and the sums' second launch waits for the last block).
#include "row.cuh"

#include "dgt_feedforward.h"

namespace dgt {
namespace {

struct LayerParams {
  const void* x;
  const void* residual;
  const void* weight;
  const void* bias;
  void* h;
  void* y;
  float* scale;
  float* mean;
  float* rstd;
  long long ldx, ldr, ldh, ldy;
  int rows, cols, tpr;
  float eps;
};

// A row as the thread's pieces, as in row.cuh, but for FLAT rows: a block has rows of one shift only (rows `VEC` apart
// start at the same offset in their first piece), so that a thread's columns, its weights and its sums stay the same
// from row to row, and all that sets these rows apart is a mask on the first and the last piece. (8192 x 1023 BF16: 34
// us, its gradient 33; with any row in any block, and weights and sums looked up by column, 53 and 51; 8192 x 1024 11
// and 22.)
template <int MODE, int VEC>
struct Pieces {
  int tid, tpr, cols, shift;

  __device__ __forceinline__ int lo(int i) const { return (i * tpr + tid) * VEC - shift; }
  __device__ __forceinline__ int place(int i) const { return (i * tpr + tid) * VEC; }  // in an array of the row's pieces
  __device__ __forceinline__ bool whole(int i) const {
    return MODE == FLAT ? lo(i) >= 0 && lo(i) + VEC <= cols : lo(i) < cols;
  }
  __device__ __forceinline__ bool any(int i) const { return (MODE != FLAT || lo(i) + VEC > 0) && lo(i) < cols; }
  __device__ __forceinline__ bool has(int i, int j) const { return lo(i) + j >= 0 && lo(i) + j < cols; }
  // what is not the row's is `fill`
  template <int TYPE>
  __device__ __forceinline__ void mask(Pack<TYPE, VEC>& v, int i, float fill = 0.0f) const {
    if constexpr (MODE == FLAT)
      if (!whole(i)) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (!has(i, j)) v.v[j] = Elem<TYPE>::put(fill);
      }
  }
  // Elements from a row's start to the matrix's end, where a FLAT piece of it may reach past that end.
  __device__ __forceinline__ int left(long long row, int rows) const {
    return static_cast<int>(min(static_cast<long long>(rows) - row, static_cast<long long>(VEC))) * cols;
  }
  // (The neighbours' elements that a piece brings along may be on their way out of another block, where an output takes
  // the place of its input: they are masked, whatever they are.)
  template <int TYPE>
  __device__ __forceinline__ void load(Pack<TYPE, VEC>& v, const void* base, long long row, long long ld, int i, bool in,
                                       int left) const {
    using T = typename Pack<TYPE, VEC>::T;
    v.zero();
    if (!in || !any(i)) return;
    const T* p = static_cast<const T*>(base) + row * ld;
    if (MODE == FLAT && lo(i) + VEC > left) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (has(i, j)) v.v[j] = p[lo(i) + j];
    } else {
      v.stream(p + lo(i));
      mask(v, i);
    }
  }
  template <int TYPE>
  __device__ __forceinline__ void store(const Pack<TYPE, VEC>& v, void* base, long long row, long long ld, int i,
                                        bool in) const {
    using T = typename Pack<TYPE, VEC>::T;
    if (!in) return;
    T* p = static_cast<T*>(base) + row * ld;
    if (whole(i)) {
      v.store(p + lo(i));
    } else if constexpr (MODE == FLAT) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (has(i, j)) p[lo(i) + j] = v.v[j];
    }
  }
  __device__ __forceinline__ void store_q8(const float (&x)[VEC], void* base, long long row, long long ld, int i,
                                           bool in) const {
    if (!in) return;
    uint8_t* p = static_cast<uint8_t*>(base) + row * ld;
    if (whole(i)) {
      store_e4m3<VEC>(p + lo(i), x);
    } else if constexpr (MODE == FLAT) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (has(i, j)) p[lo(i) + j] = __nv_cvt_float_to_fp8(x[j], __NV_SATFINITE, __NV_E4M3);
    }
  }
  // Columns' weights as fp32, zeros past the row: from memory (L1 holds them), or from the block's copy in the order
  // of its pieces (FLAT).
  template <int TYPE>
  __device__ __forceinline__ void weights(float (&w)[VEC], const void* weight, const typename Elem<TYPE>::T* shared,
                                          int i) const {
    Pack<TYPE, VEC> v;
    v.zero();
    if constexpr (MODE == FLAT) {
      if (any(i)) v.load(shared + place(i));
    } else {
      if (whole(i)) v.load(static_cast<const typename Elem<TYPE>::T*>(weight) + lo(i));
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = v.get(j);
  }
};

// The rows of a block: all of them in turn, or those of one shift (FLAT).
template <int MODE, int VEC>
struct BlockRows {
  int cls, first, blocks;
  long long count;
  __device__ __forceinline__ BlockRows(int rows) {
    constexpr int CLASSES = MODE == FLAT ? VEC : 1;
    cls = blockIdx.x % CLASSES;
    first = blockIdx.x / CLASSES;
    blocks = max(static_cast<int>(gridDim.x) / CLASSES, 1);  // (fewer rows than classes have a block each)
    count = rows <= cls ? 0 : (static_cast<long long>(rows) - cls + CLASSES - 1) / CLASSES;
  }
  __device__ __forceinline__ long long row(long long q) const { return MODE == FLAT ? cls + VEC * q : q; }
};

// Pieces of a FLAT row of any shift.
__host__ __device__ constexpr int flat_places(int cols, int vec) { return (cols + vec - 1 + vec - 1) / vec * vec; }

// FLAT: weights in the order of the pieces, zeros around them.
template <int TYPE, int VEC>
__device__ __forceinline__ void stage_pieces(typename Elem<TYPE>::T* shared, const void* weight, int cols, int shift) {
  using E = Elem<TYPE>;
  const int n = flat_places(cols, VEC);
  // (eight loads in flight: one at a time took 2.5 us)
  for (int e0 = threadIdx.x; e0 < n; e0 += 8 * blockDim.x) {
    typename E::T v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = e0 + k * static_cast<int>(blockDim.x) - shift;
      v[k] = c >= 0 && c < cols ? static_cast<const typename E::T*>(weight)[c] : E::put(0.0f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = e0 + k * static_cast<int>(blockDim.x);
      if (e < n) shared[e] = v[k];
    }
  }
}

template <int TYPE, int MODE, int EPT, bool Q8>
__global__ void __launch_bounds__(kNormThreads<TYPE, EPT>, kNormThreads<TYPE, EPT> == 512 ? 2 : 1)
    layernorm_kernel(const LayerParams p) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = MODE == SINGLE ? 1 : 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][3][32];
  extern __shared__ uint4 dynamic[];
  T* shared_w = reinterpret_cast<T*>(dynamic);
  T* shared_b = shared_w + (MODE == FLAT ? flat_places(p.cols, VEC) : 0);
  const int per_block = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
  const BlockRows<MODE, VEC> rows(p.rows);
  const Pieces<MODE, VEC> r = {static_cast<int>(threadIdx.x) - sub * p.tpr, p.tpr, p.cols,
                               MODE == FLAT ? static_cast<int>(static_cast<long long>(rows.cls) * p.cols % VEC) : 0};
  const RowWarps row_warps(p.tpr, sub);
  grid_dependency_wait();
  if constexpr (MODE == FLAT) {
    stage_pieces<TYPE, VEC>(shared_w, p.weight, p.cols, r.shift);
    if (p.bias != nullptr) stage_pieces<TYPE, VEC>(shared_b, p.bias, p.cols, r.shift);
    __syncthreads();
  }
  int turn = 0;
  for (long long q0 = static_cast<long long>(rows.first) * per_block; q0 < rows.count;
       q0 += static_cast<long long>(rows.blocks) * per_block, turn ^= 1) {
    const long long row = rows.row(q0 + sub);
    const bool in = q0 + sub < rows.count;
    const int left = r.left(row, p.rows);
    P h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) r.load(h[i], p.x, row, p.ldx, i, in, left);
    if (p.residual != nullptr) {
      P a[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) r.load(a[i], p.residual, row, p.ldr, i, in, left);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = h[i].get(j) + a[i].get(j);
        h[i].set(x);
        if (p.h != nullptr) r.store(h[i], p.h, row, p.ldh, i, in);
      }
    }
    // (two elements to an instruction where a piece has two)
    float s = 0.0f;
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) s2 = __fadd2_rn(s2, h[i].two(j));
      } else {
        s += h[i].get(0);
      }
    }
    const float mean = row_warps.sum(s + (s2.x + s2.y), red[turn][0]) / static_cast<float>(p.cols);
    const float2 less = make_float2(-mean, -mean);
    s = 0.0f;
    s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (MODE == SINGLE) {
        const float d = r.whole(i) ? h[i].get(0) - mean : 0.0f;
        s = fmaf(d, d, s);
      } else if (r.whole(i)) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 d = __fadd2_rn(h[i].two(j), less);
          s2 = __ffma2_rn(d, d, s2);
        }
      } else if constexpr (MODE == FLAT) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = r.has(i, j) ? h[i].get(j) - mean : 0.0f;
          s = fmaf(d, d, s);
        }
      }
    }
    const float rstd = 1.0f / sqrtf(row_warps.sum(s + (s2.x + s2.y), red[turn][1]) / static_cast<float>(p.cols) + p.eps);
    const float2 by = make_float2(rstd, rstd);
    if (in && r.tid == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    // the output of piece i, before its rounding
    auto norm = [&](float* y, int i) {
      float w[VEC], b[VEC];
      r.template weights<TYPE>(w, p.weight, shared_w, i);
      if (p.bias != nullptr) {
        r.template weights<TYPE>(b, p.bias, shared_b, i);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = 0.0f;
      }
      if constexpr (VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 xhat = __fmul2_rn(__fadd2_rn(h[i].two(j), less), by);
          const float2 v = __ffma2_rn(xhat, make_float2(w[j], w[j + 1]), make_float2(b[j], b[j + 1]));
          y[j] = v.x;
          y[j + 1] = v.y;
        }
      } else {
        y[0] = fmaf((h[i].get(0) - mean) * rstd, w[0], b[0]);
      }
    };
    if constexpr (!Q8) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[VEC];
        norm(y, i);
        P o;
        o.set(y);
        r.store(o, p.y, row, p.ldy, i, in);
      }
    } else {
      // the row's outputs take the registers of h. |y| is compared by bit pattern: a NaN is above every number and
      // reaches the scale
      float y[EPT];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        norm(y + i * VEC, i);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (MODE == FLAT ? r.has(i, j) : r.whole(i)) top = max(top, __float_as_uint(y[i * VEC + j]) & 0x7FFFFFFFu);
      }
      const float amax = __uint_as_float(row_warps.max_bits(top, red[turn][2]));
      const float scale = (amax < 1e-12f ? 1e-12f : amax) / kE4M3Max;
      const float inv = 1.0f / scale;
      if (in && r.tid == 0) p.scale[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float q[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[j] = y[i * VEC + j] * inv;
        r.store_q8(q, p.y, row, p.ldy, i, in);
      }
    }
  }
  grid_launch_dependents();
}

constexpr int kGradEpt = 16;  // elements of a row per thread of the gradient

// cp.async of 16 bytes, of which `bytes` come from memory and the rest are zero.
__device__ __forceinline__ void copy16_part(uint4* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

struct LayerGradParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* mean;
  const float* rstd;
  const void* dh;
  void* dx;
  float* partial;  // a row of `cols` sums of dw and one of db per block
  long long lddy, ldh, lddh, lddx;
  int rows, cols, tpr;
};

// Two sums over a row's warps at once, with one barrier. After the first exchange the lower half of a warp adds up
// the first sum and the upper half the second, so that both take the steps of one.
__device__ __forceinline__ float2 sum_two(const RowWarps& w, float2 v, float2* red) {
  const int lane = threadIdx.x & 31;
  const bool up = lane & 16;
  auto fold = [&](float2 t) {
    float s = (up ? t.y : t.x) + __shfl_xor_sync(0xFFFFFFFFu, up ? t.x : t.y, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    return s;
  };
  float s = fold(v);
  if (w.warps > 1) {
    float* r = reinterpret_cast<float*>(red);
    if ((lane & 15) == 0) r[2 * (threadIdx.x >> 5) + (lane >> 4)] = s;
    __syncthreads();
    s = fold(lane < w.warps ? red[w.w0 + lane] : make_float2(0.0f, 0.0f));
  }
  return make_float2(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 16));
}

// A thread owns the same columns of each of its rows and adds dw and db up in registers. AHEAD: each thread copies its
// pieces of the next row to its own places in shared memory (cp.async) before it works on this one, so that loads are
// in flight during the reduction and the stores, and reads a piece from its place once for the sums and once for the
// output, so that registers hold one piece at a time beside the 32 sums.
template <int TYPE, int MODE, bool AHEAD>
__global__ void __launch_bounds__(int(kMaxCols) / kGradEpt, 1) layernorm_grad_kernel(const LayerGradParams p) {
  constexpr int EPT = kGradEpt;
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = MODE == SINGLE ? 1 : 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  constexpr int NV = EPT / VEC;
  __shared__ float2 red[2][32];
  extern __shared__ uint4 dynamic[];
  // FLAT: the weights; then the copies ahead, whose place (rows of the block - 1) x 2 rows of sums take at the end
  T* shared_w = reinterpret_cast<T*>(dynamic);
  uint4* stages = dynamic + (MODE == FLAT ? flat_places(p.cols, VEC) / VEC : 0);
  float* sums = reinterpret_cast<float*>(stages);
  const int places = MODE == FLAT ? flat_places(p.cols, VEC) : p.cols;
  const int per_block = blockDim.x / p.tpr, sub = threadIdx.x / p.tpr;
  const BlockRows<MODE, VEC> rows(p.rows);
  const Pieces<MODE, VEC> r = {static_cast<int>(threadIdx.x) - sub * p.tpr, p.tpr, p.cols,
                               MODE == FLAT ? static_cast<int>(static_cast<long long>(rows.cls) * p.cols % VEC) : 0};
  const RowWarps row_warps(p.tpr, sub);
  const long long step = static_cast<long long>(rows.blocks) * per_block;
  // AHEAD: piece i of h, dy or dh (m = 0, 1, 2) of stage s
  auto cell = [&](int s, int m, int i) { return stages + ((s * 3 + m) * NV + i) * blockDim.x + threadIdx.x; };
  auto fetch = [&](long long q, int s) {
    const long long row = rows.row(q);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (r.any(i)) {
        if (q < rows.count) {
          // (a piece that reaches past the matrix: the copy reads what there is)
          const int most = r.left(row, p.rows) - r.lo(i);
          const int bytes = MODE == FLAT && most < VEC ? most * int(sizeof(T)) : 16;
          copy16_part(cell(s, 0, i), static_cast<const T*>(p.h) + row * p.ldh + r.lo(i), bytes);
          copy16_part(cell(s, 1, i), static_cast<const T*>(p.dy) + row * p.lddy + r.lo(i), bytes);
          if (p.dh != nullptr) copy16_part(cell(s, 2, i), static_cast<const T*>(p.dh) + row * p.lddh + r.lo(i), bytes);
        } else if (per_block > 1) {  // a row past the last one counts as zeros
          *cell(s, 0, i) = *cell(s, 1, i) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const long long start = static_cast<long long>(rows.first) * per_block + sub;
  grid_dependency_wait();
  if constexpr (AHEAD) {
    // zeros where no copy lands: past the last column, and dh where there is none
#pragma unroll
    for (int i = 0; i < NV; ++i)
      for (int c = 0; c < 6; ++c)
        if (!r.any(i) || (c % 3 == 2 && p.dh == nullptr)) *cell(c / 3, c % 3, i) = make_uint4(0u, 0u, 0u, 0u);
    fetch(start, 0);
  }
  if constexpr (MODE == FLAT) {
    stage_pieces<TYPE, VEC>(shared_w, p.weight, p.cols, r.shift);
    __syncthreads();
  }
  // a row past the last one has dy = 0, mean = rstd = 0: it adds nothing
  auto statistics = [&](long long q) {
    if (q >= rows.count) return make_float2(0.0f, 0.0f);
    const long long row = rows.row(q);
    return make_float2(p.mean[row], p.rstd[row]);
  };
  float2 next = AHEAD ? statistics(start) : make_float2(0.0f, 0.0f);
  alignas(8) float dw[EPT], db[EPT];
#pragma unroll
  for (int e = 0; e < EPT; ++e) dw[e] = db[e] = 0.0f;
  int turn = 0;
  for (long long q0 = static_cast<long long>(rows.first) * per_block; q0 < rows.count; q0 += step, turn ^= 1) {
    const long long row = rows.row(q0 + sub);
    const bool in = q0 + sub < rows.count;
    P h[NV], dy[NV], dh[NV];
    float2 stat;
    if constexpr (AHEAD) {
      fetch(q0 + sub + step, turn ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // this row's pieces have landed
      stat = next;
      next = statistics(q0 + sub + step);
    } else {
      stat = statistics(q0 + sub);
      const int left = r.left(row, p.rows);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        r.load(h[i], p.h, row, p.ldh, i, in, left);
        r.load(dy[i], p.dy, row, p.lddy, i, in, left);
      }
      if (p.dh != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) r.load(dh[i], p.dh, row, p.lddh, i, in, left);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) dh[i].zero();
      }
    }
    const float mean = stat.x, rstd = stat.y;
    // AHEAD: a piece from its place, once for each use: registers hold one piece at a time, not the row's
    auto take = [&](P(&v)[NV], int m, int i) {
      if constexpr (AHEAD) v[i].load(reinterpret_cast<const T*>(cell(turn, m, i)));
    };
    // sums of g and of g xhat (outside the row dy is 0, and so is what is added); two elements to an instruction where
    // a piece has two
    float2 dots = make_float2(0.0f, 0.0f), gs = dots, gx = dots;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!r.any(i)) continue;
      float w[VEC];
      r.template weights<TYPE>(w, p.weight, shared_w, i);
      take(h, 0, i);
      take(dy, 1, i);
      r.mask(h[i], i, mean);  // (0 times a neighbour's infinity, or what -mean rstd may pass, is not 0)
      if constexpr (AHEAD) r.mask(dy[i], i);
      if constexpr (VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 xhat = __fmul2_rn(__fadd2_rn(h[i].two(j), make_float2(-mean, -mean)), make_float2(rstd, rstd));
          const float2 d = dy[i].two(j), g = __fmul2_rn(d, make_float2(w[j], w[j + 1]));
          gs = __fadd2_rn(gs, g);
          gx = __ffma2_rn(g, xhat, gx);
          float2& sw = *reinterpret_cast<float2*>(dw + i * VEC + j);
          float2& sb = *reinterpret_cast<float2*>(db + i * VEC + j);
          sw = __ffma2_rn(d, xhat, sw);
          sb = __fadd2_rn(sb, d);
        }
      } else {
        const float xhat = (h[i].get(0) - mean) * rstd, d = dy[i].get(0), g = d * w[0];
        dots.x += g;
        dots.y = fmaf(g, xhat, dots.y);
        dw[i] = fmaf(d, xhat, dw[i]);
        db[i] += d;
      }
    }
    if constexpr (VEC > 1) dots = make_float2(gs.x + gs.y, gx.x + gx.y);
    dots = sum_two(row_warps, dots, red[turn]);
    const float mean_g = dots.x / static_cast<float>(p.cols), back = rstd * (dots.y / static_cast<float>(p.cols));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[VEC];
      r.template weights<TYPE>(w, p.weight, shared_w, i);
      take(h, 0, i);
      take(dy, 1, i);
      take(dh, 2, i);
      P o;
      if constexpr (VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 xhat = __fmul2_rn(__fadd2_rn(h[i].two(j), make_float2(-mean, -mean)), make_float2(rstd, rstd));
          const float2 g = __ffma2_rn(dy[i].two(j), make_float2(w[j], w[j + 1]), make_float2(-mean_g, -mean_g));
          const float2 v = __ffma2_rn(g, make_float2(rstd, rstd), __ffma2_rn(xhat, make_float2(-back, -back), dh[i].two(j)));
          w[j] = v.x;
          w[j + 1] = v.y;
        }
      } else {
        w[0] = fmaf(fmaf(dy[i].get(0), w[0], -mean_g), rstd, fmaf((h[i].get(0) - mean) * rstd, -back, dh[i].get(0)));
      }
      o.set(w);
      r.store(o, p.dx, row, p.lddx, i, in);
    }
  }
  if constexpr (AHEAD) asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
  // the block's sums over its rows, in row order; four columns at a time
  constexpr int RUN = VEC < 4 ? 1 : 4;
  auto each = [&](auto use) {
#pragma unroll
    for (int e = 0; e < EPT; e += RUN)
      if (r.any(e / VEC)) use(r.place(e / VEC) + e % VEC, e);
  };
  auto store = [&](float* to, const float* from) {
    if constexpr (RUN == 1)
      *to = *from;
    else
      *reinterpret_cast<float4*>(to) = make_float4(from[0], from[1], from[2], from[3]);
  };
  if (per_block > 1) {
    __syncthreads();
    if (sub > 0)
      each([&](int at, int e) {
        store(sums + 2 * (sub - 1) * places + at, dw + e);
        store(sums + (2 * (sub - 1) + 1) * places + at, db + e);
      });
    __syncthreads();
    if (sub == 0)
      for (int s = 0; s + 1 < per_block; ++s)
        each([&](int at, int e) {
#pragma unroll
          for (int k = 0; k < RUN; ++k) {
            dw[e + k] += sums[2 * s * places + at + k];
            db[e + k] += sums[(2 * s + 1) * places + at + k];
          }
        });
  }
  if (sub == 0)
    each([&](int at, int e) {
      if constexpr (MODE == FLAT) {
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
          const int c = at + k - r.shift;
          if (c >= 0 && c < p.cols) {
            out[c] = dw[e + k];
            out[p.cols + c] = db[e + k];
          }
        }
      } else {
        store(out + at, dw + e);
        store(out + p.cols + at, db + e);
      }
    });
  grid_launch_dependents();
}

// dw and db from the blocks' partial rows (2 x cols each): 32 columns a block, 32
// threads a column, each a fixed share of the rows, added in order of the threads.
template <int TYPE>
__global__ void __launch_bounds__(1024) layer_weight_sum_kernel(const float* partial, int rows, int cols, void* dw,
                                                                void* db) {
  using E = Elem<TYPE>;
  __shared__ float part[32][33];
  grid_dependency_wait();
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < 2 * cols) {
#pragma unroll 8
    for (int r = g; r < rows; r += 32) s += __ldcg(partial + static_cast<long long>(r) * 2 * cols + col);
  }
  part[g][c] = s;
  __syncthreads();
  // warp g adds up column g of the block
  s = warp_sum(part[c][g]);
  const int mine = blockIdx.x * 32 + g;
  if (c == 0 && mine < 2 * cols) {
    void* to = mine < cols ? dw : db;
    if (to != nullptr) static_cast<typename E::T*>(to)[mine < cols ? mine : mine - cols] = E::put(s);
  }
  grid_launch_dependents();
}

// Blocks of the gradient, at most: what an SM holds of 16-bit rows at 64 registers a thread, for each of a GB300's 152
// (a number, since the size of the workspace goes by it, on a machine without a GPU too). BF16 with dh, 304 / 456 /
// 608 blocks, us: 4097 x 5120 (320 threads) 46.4 / 45.1 / 51.8, 8192 x 4096 (256) 77.7 / 64.0 / 59.4, 8192 x 8192
// (512) 108 / 127 / 118, 30000 x 1024 68.5 / 56.7 / 52.9. FP32 rows take the same number, of which a half or a third
// fit at a time (their stages are twice as large): 4097 x 5120 90 us, 8192 x 4096 123, 8192 x 8192 260, 30000 x 1024
// 109. (One block an SM with as many rows side by side, each with a barrier of its own, and so a third of the partial
// rows: 45.5, 60.6, 114, 57.7.)
constexpr int kGradThreads = 256;  // of a block, at least
int64_t grad_blocks(int64_t cols) {
  const int tpr = threads_per_row(cols, kGradEpt, ALIGNED, 8), fit = 1024 / (tpr < kGradThreads ? kGradThreads : tpr);
  return int64_t(152) * (fit < 1 ? 1 : fit);
}

// Blocks of `per` rows for `rows` of them, `most` at most. FLAT: as many for each of the v shifts that rows have.
int grid_of(int mode, int v, int64_t rows, int per, int64_t most) {
  const int64_t classes = mode != FLAT ? 1 : rows < v ? rows : v;
  const int64_t need = ((rows + classes - 1) / classes + per - 1) / per, fit = most / classes < 1 ? 1 : most / classes;
  return int(classes * (need < fit ? need : fit));
}

template <int TYPE, int MODE, int EPT, bool Q8>
cudaError_t launch_layer_build(const LayerParams& p, int dev, int grid, int block, size_t smem, cudaStream_t s) {
  auto kern = layernorm_kernel<TYPE, MODE, EPT, Q8>;
  if constexpr (MODE == FLAT) {  // weights and bias of the widest rows are more than a launch may take without asking
    static int configured[64] = {};
    if (dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
      constexpr int es = sizeof(typename Elem<TYPE>::T);
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 2 * flat_places(kMaxFlatCols, 16 / es) * es);
      if (e != cudaSuccess) return e;
      if (dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
  }
  return launch_dependent(kern, grid, block, smem, s, 1, p);
}
template <int TYPE, int MODE, int EPT>
cudaError_t launch_layer_mode(const LayerParams& p, bool q8, int dev, int grid, int block, size_t smem, cudaStream_t s) {
  return q8 ? launch_layer_build<TYPE, MODE, EPT, true>(p, dev, grid, block, smem, s)
            : launch_layer_build<TYPE, MODE, EPT, false>(p, dev, grid, block, smem, s);
}

// Elements a thread holds of a FLAT row: 32 bytes' worth, or 64 of rows of 12000 bytes and more. us with 32 / 64: BF16
// 30000 x 77 34 / 64, 8192 x 1023 34 / 42, 2048 x 4095 30 / 36, 8192 x 8191 234 / 188; FP32 30000 x 77 20 / 34, 2048 x
// 4095 54 / 42.
template <int TYPE>
constexpr int kFlatEpt = 32 / int(sizeof(typename Elem<TYPE>::T));
bool wide_flat(int64_t cols, int es) { return cols * es > 12000; }

template <int TYPE>
cudaError_t launch_layer(const LayerParams& p, int mode, bool few, bool q8, int dev, int grid, int block, cudaStream_t s) {
  constexpr int es = sizeof(typename Elem<TYPE>::T);
  const size_t smem = mode == FLAT ? 2 * size_t(flat_places(p.cols, 16 / es)) * es : 0;
  if (mode == ALIGNED)
    return few ? launch_layer_mode<TYPE, ALIGNED, 8>(p, q8, dev, grid, block, smem, s)
               : launch_layer_mode<TYPE, ALIGNED, kFullEpt<TYPE, ALIGNED>>(p, q8, dev, grid, block, smem, s);
  if (mode == FLAT)
    return few                        ? launch_layer_mode<TYPE, FLAT, 8>(p, q8, dev, grid, block, smem, s)
           : wide_flat(p.cols, es)    ? launch_layer_mode<TYPE, FLAT, kFullEpt<TYPE, FLAT>>(p, q8, dev, grid, block, smem, s)
                                      : launch_layer_mode<TYPE, FLAT, kFlatEpt<TYPE>>(p, q8, dev, grid, block, smem, s);
  return few ? launch_layer_mode<TYPE, SINGLE, 8>(p, q8, dev, grid, block, smem, s)
             : launch_layer_mode<TYPE, SINGLE, kFullEpt<TYPE, SINGLE>>(p, q8, dev, grid, block, smem, s);
}

// Dynamic shared memory of the gradient's kernel.
size_t grad_smem(const LayerGradParams& p, int mode, bool ahead, int block, int es) {
  const size_t places = mode == FLAT ? flat_places(p.cols, 16 / es) : p.cols;
  const size_t sums = 2 * size_t(block / p.tpr - 1) * places * sizeof(float);
  const size_t stages = ahead ? size_t(2 * 3) * kGradEpt * es * size_t(block) : 0;
  return (mode == FLAT ? places * es : 0) + (sums > stages ? sums : stages);
}

// Most dynamic shared memory that a launch of the gradient takes: AHEAD goes up to here.
constexpr size_t kGradSmem = 200 * 1024;

// Launches one build of the gradient's kernel. Its limit is a property of the kernel, not of the launch, so it is set
// once, to the most that any launch takes: other host threads may be launching it with other sizes.
template <int TYPE, int MODE, bool AHEAD>
cudaError_t launch_layer_grad_mode(const LayerGradParams& p, int dev, int grid, int block, size_t smem,
                                   cudaStream_t s) {
  static int configured[64] = {};
  auto kern = layernorm_grad_kernel<TYPE, MODE, AHEAD>;
  if (dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kGradSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_dependent(kern, grid, block, smem, s, 1, p);
}

template <int TYPE>
cudaError_t launch_layer_grad(const LayerGradParams& p, int mode, bool ahead, int dev, int grid, int block, void* dw,
                              void* db, cudaStream_t s) {
  const size_t smem = grad_smem(p, mode, ahead, block, sizeof(typename Elem<TYPE>::T));
  const cudaError_t e =
      mode == ALIGNED ? (ahead ? launch_layer_grad_mode<TYPE, ALIGNED, true>(p, dev, grid, block, smem, s)
                               : launch_layer_grad_mode<TYPE, ALIGNED, false>(p, dev, grid, block, smem, s))
      : mode == FLAT  ? (ahead ? launch_layer_grad_mode<TYPE, FLAT, true>(p, dev, grid, block, smem, s)
                               : launch_layer_grad_mode<TYPE, FLAT, false>(p, dev, grid, block, smem, s))
                      : launch_layer_grad_mode<TYPE, SINGLE, false>(p, dev, grid, block, smem, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(layer_weight_sum_kernel<TYPE>, (2 * p.cols + 31) / 32, 1024, 0, s, 1, p.partial, grid, p.cols,
                          dw, db);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_layernorm(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                   const void* weight, const void* bias, float eps, void* h, int64_t ldh, int y_type, void* y,
                   int64_t ldy, float* y_scale, float* mean, float* rstd, void* stream) {
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
  if (misaligned(x, es) || misaligned(residual, es) || misaligned(weight, es) || misaligned(bias, es) ||
      misaligned(h, es) || misaligned(y, eo) || misaligned(y_scale, 4) || misaligned(mean, 4) || misaligned(rstd, 4))
    return GEMM_ERR_MISALIGNED;
  // an output may be an input's very buffer (each element is read, then written, by one thread), or apart from it
  auto clash = [&](const void* o, int64_t ldo, int e_o, const void* i, int64_t ldi) {
    if (o == nullptr || i == nullptr || (o == i && ldo == ldi && e_o == es)) return false;
    return meet(o, rows, cols, ldo, e_o, i, rows, cols, ldi, es);
  };
  auto on_row = [&](const void* o, int64_t ldo, int e_o, const void* v) {  // o meets the weights or the bias
    return o != nullptr && v != nullptr && meet(o, rows, cols, ldo, e_o, v, 1, cols, cols, es);
  };
  auto on_vector = [&](const void* o, int64_t ldo, int e_o, const void* v) {  // o meets a number for each row
    return o != nullptr && v != nullptr && meet(o, rows, cols, ldo, e_o, v, 1, rows, rows, 4);
  };
  if (clash(h, ldh, es, x, ldx) || clash(h, ldh, es, residual, ldr) || clash(y, ldy, eo, x, ldx) ||
      (residual != nullptr && meet(y, rows, cols, ldy, eo, residual, rows, cols, ldr, es)) ||
      (h != nullptr && meet(y, rows, cols, ldy, eo, h, rows, cols, ldh, es)) || on_row(y, ldy, eo, weight) ||
      on_row(y, ldy, eo, bias) || on_row(h, ldh, es, weight) || on_row(h, ldh, es, bias))
    return GEMM_ERR_INVALID_VALUE;
  for (const float* v : {y_scale, mean, rstd})
    if (on_vector(x, ldx, es, v) || on_vector(residual, ldr, es, v) || on_vector(h, ldh, es, v) ||
        on_vector(y, ldy, eo, v))
      return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[9] = {x, weight, y, residual, bias, h, y_scale, mean, rstd};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  const int v = 16 / es;
  int mode = SINGLE;
  if (cols % v == 0 && aligned(x, ldx, es, 16) && aligned(weight, 0, es, 16) && aligned(bias, 0, es, 16) &&
      (residual == nullptr || aligned(residual, ldr, es, 16)) && (h == nullptr || aligned(h, ldh, es, 16)) &&
      aligned(y, ldy, eo, v * eo))
    mode = ALIGNED;
  else if (cols <= kMaxFlatCols && flat(x, ldx, cols, 16) &&
           (residual == nullptr || flat(residual, ldr, cols, 16)) && (h == nullptr || flat(h, ldh, cols, 16)) &&
           flat(y, ldy, cols, v * eo))
    mode = FLAT;
  LayerParams p = {x,       residual, weight,  bias,    h,         y,         y_scale, mean, rstd, (long long)ldx,
                   (long long)ldr, (long long)ldh, (long long)ldy, int(rows), int(cols), 0, eps};
  // Eight elements a thread while the rows leave threads to spare, 64 bytes' worth once they fill the GPU and past
  // what 1024 threads hold (the root-mean-square norm's rule: its loads and reductions are these).
  const bool few = cols <= 8000 && rows * cols <= int64_t(ctx.sm_count) * 8192;
  p.tpr = threads_per_row(cols, few ? 8 : mode == SINGLE ? 16 : mode == FLAT && !wide_flat(cols, es) ? 32 / es : 64 / es, mode, v);
  const int block = p.tpr < 128 ? 128 / p.tpr * p.tpr : p.tpr;
  const int grid = grid_of(mode, v, rows, block / p.tpr, int64_t(ctx.sm_count) * (2048 / block));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_layer<GEMM_TYPE_F16>(p, mode, few, q8, ctx.dev, grid, block, s)
                        : type == GEMM_TYPE_BF16 ? launch_layer<GEMM_TYPE_BF16>(p, mode, few, q8, ctx.dev, grid, block, s)
                                                 : launch_layer<GEMM_TYPE_F32>(p, mode, few, q8, ctx.dev, grid, block, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int64_t gemm_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  return (rows < grad_blocks(cols) ? rows : grad_blocks(cols)) * 2 * cols * int64_t(sizeof(float));
}

int gemm_layernorm_backward(int type, int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* h,
                            int64_t ldh, const void* weight, const float* mean, const float* rstd, const void* dh,
                            int64_t lddh, void* dx, int64_t lddx, void* dw, void* db, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (bad_type(type) || rows < 0 || cols < 0 || cols > kMaxCols || rows >= (int64_t(1) << 31))
    return GEMM_ERR_INVALID_VALUE;
  if (cols == 0) return GEMM_OK;
  const int es = type_bytes(type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CallContext ctx;
  if (dw == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (misaligned(dw, es) || misaligned(db, es)) return GEMM_ERR_MISALIGNED;
  if (db != nullptr && meet(dw, 1, cols, cols, es, db, 1, cols, cols, es)) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0) {  // no rows: dw = db = 0
    const int st = begin_call(&ctx);
    if (st != GEMM_OK) return st;
    if (!on_device(dw, ctx.dev) || (db != nullptr && !on_device(db, ctx.dev))) return GEMM_ERR_NOT_DEVICE_MEMORY;
    if (cudaMemsetAsync(dw, 0, size_t(cols) * es, s) != cudaSuccess) return GEMM_ERR_LAUNCH;
    return db == nullptr || cudaMemsetAsync(db, 0, size_t(cols) * es, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
  }
  if (dy == nullptr || h == nullptr || weight == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr ||
      workspace == nullptr || bad_ld(lddy, cols) || bad_ld(ldh, cols) || bad_ld(lddx, cols) ||
      (dh != nullptr && bad_ld(lddh, cols)) || workspace_bytes < gemm_layernorm_backward_workspace(rows, cols))
    return GEMM_ERR_INVALID_VALUE;
  if (misaligned(dy, es) || misaligned(h, es) || misaligned(weight, es) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(dh, es) || misaligned(dx, es) || misaligned(workspace, 16))
    return GEMM_ERR_MISALIGNED;
  auto clash = [&](const void* i, int64_t ldi) {
    if (i == nullptr || (i == dx && ldi == lddx)) return false;
    return meet(dx, rows, cols, lddx, es, i, rows, cols, ldi, es);
  };
  auto on_dx = [&](const void* v, int64_t n, int e_v) {
    return v != nullptr && meet(dx, rows, cols, lddx, es, v, 1, n, n, e_v);
  };
  if (clash(dy, lddy) || clash(dh, lddh) || clash(h, ldh) || on_dx(weight, cols, es) || on_dx(dw, cols, es) ||
      on_dx(db, cols, es) || on_dx(mean, rows, 4) || on_dx(rstd, rows, 4))
    return GEMM_ERR_INVALID_VALUE;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[10] = {dy, h, weight, mean, rstd, dx, dw, db, workspace, dh};
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
  LayerGradParams p = {dy,   h,      weight, mean, rstd, dh, dx, static_cast<float*>(workspace), (long long)lddy,
                       (long long)ldh, (long long)lddh, (long long)lddx, int(rows), int(cols), 0};
  p.tpr = threads_per_row(cols, kGradEpt, mode, v);
  const int block = p.tpr >= kGradThreads ? p.tpr : kGradThreads / p.tpr * p.tpr;
  const bool ahead = mode != SINGLE && grad_smem(p, mode, true, block, es) <= kGradSmem;
  const int grid = grid_of(mode, v, rows, block / p.tpr, rows < grad_blocks(cols) ? rows : grad_blocks(cols));
  const cudaError_t e =
      type == GEMM_TYPE_F16    ? launch_layer_grad<GEMM_TYPE_F16>(p, mode, ahead, ctx.dev, grid, block, dw, db, s)
      : type == GEMM_TYPE_BF16 ? launch_layer_grad<GEMM_TYPE_BF16>(p, mode, ahead, ctx.dev, grid, block, dw, db, s)
                               : launch_layer_grad<GEMM_TYPE_F32>(p, mode, ahead, ctx.dev, grid, block, dw, db, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
