// The dense gated product and its gradient (gemm_gated, gemm_gated_backward).
//
//   up = A W + bias;  C = act(up[:, :F]) * up[:, F:]
//   dup = [dC value act'(gate), dC act(gate)];  dA = dup W^T;  dW = A^T dup;  dbias = sum over rows of dup
//
// The products are the grouped kernel's (group_kernel.cuh) with one group: its
// tiles hold the same columns of both halves, so the forward pass writes C only
// (and the halves where a backward pass will need them). The gradient's dup is a
// pass of its own: both of its products read it, one along F and one along the
// rows, and it is a tenth of their time (8192 x 4096 -> 2 x 4096 BF16: 55 of 612-640
// us, the products 281 each: 1.95 PFLOP/s). The forward pass 8192 x 4096 -> 2 x 8192
// takes 535-555 us (2.0 PFLOP/s) in a burst, 600 to 635 at the power limit.
#include <cstring>

#include "elem.cuh"
#include "gated_few.h"
#include "group_launch.h"

namespace dgt {
namespace {

constexpr int kGateThreads = 256;
// Row blocks, at most, that leave partial sums of dbias (a number: the size of the workspace goes by it, on a machine
// without a GPU too).
constexpr int kBiasBlocks = 152;

struct GateGradParams {
  const void* dc;
  const void* up;
  void* dup;
  float* partial;  // a row of 2F sums for each row block, or null
  long long lddc, ldup, lddup;
  int rows, F, gate;
  int tx;             // threads across a block's columns
  int rows_per_block;
};

// act(x) and act'(x). Beyond +-30 (SiLU: +-88) the slope's second term is below fp32's least part of 1, and the
// clamp keeps infinities out of it; a NaN passes.
__device__ __forceinline__ void gate_slope(float x, int gate, float& act, float& slope) {
  if (gate == GEMM_GATE_SILU) {
    const float sig = __fdividef(1.0f, 1.0f + __expf(-x));
    const float xc = x > 88.0f ? 88.0f : x < -88.0f ? -88.0f : x;
    act = x * sig;
    slope = sig * (1.0f + xc * (1.0f - sig));
  } else if (gate == GEMM_GATE_RELU) {
    act = x < 0.0f ? 0.0f : x;
    slope = x > 0.0f ? 1.0f : x <= 0.0f ? 0.0f : x;
  } else {
    const float xc = x > 30.0f ? 30.0f : x < -30.0f ? -30.0f : x;
    if (gate == GEMM_GATE_GELU) {
      const float p = 0.5f * (1.0f + erff(x * 0.70710678118654752f));
      act = x * p;
      slope = p + xc * 0.3989422804014327f * __expf(-0.5f * xc * xc);
    } else {
      // x / (1 + exp(-2 u)), u = sqrt(2 / pi) (x + 0.044715 x^3)
      const float u2 = 1.5957691216057308f * (xc + 0.044715f * xc * xc * xc);
      const float p = __fdividef(1.0f, 1.0f + __expf(-u2));
      act = x * p;
      slope = p + xc * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * xc * xc);
    }
  }
}

// VEC 16-bit elements at a time.
template <int TYPE, int VEC>
struct Piece {
  using T = typename Elem<TYPE>::T;
  alignas(VEC * 2) T v[VEC];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const T* p = static_cast<const T*>(base) + at;
    if constexpr (VEC == 8)
      *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(v) = __ldcs(reinterpret_cast<const uint2*>(p));
    else if constexpr (VEC == 2)
      *reinterpret_cast<uint32_t*>(v) = __ldcs(reinterpret_cast<const uint32_t*>(p));
    else
      v[0] = *p;
  }
  __device__ __forceinline__ void store(void* base, long long at) const {
    T* p = static_cast<T*>(base) + at;
    if constexpr (VEC == 8)
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    else if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
    else if constexpr (VEC == 2)
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(v);
    else
      *p = v[0];
  }
};

// A thread owns VEC columns of each half and walks down its block's rows, several in flight; bound by HBM (3 F read
// and 2 F written a row). BIAS: its columns' sums, then the block's in the order of its threads.
template <int TYPE, int VEC, bool BIAS>
__global__ void __launch_bounds__(kGateThreads) gate_grad_kernel(const GateGradParams p) {
  using E = Elem<TYPE>;
  __shared__ float sums[BIAS ? kGateThreads * 2 * VEC : 1];
  const int x = threadIdx.x % p.tx, y = threadIdx.x / p.tx, ty = kGateThreads / p.tx;
  const long long col = (static_cast<long long>(blockIdx.x) * p.tx + x) * VEC;
  const bool in = col < p.F;
  float sg[VEC], sv[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sg[j] = sv[j] = 0.0f;
  grid_dependency_wait();
  const long long begin = static_cast<long long>(blockIdx.y) * p.rows_per_block;
  const long long end = min(begin + p.rows_per_block, static_cast<long long>(p.rows));
  if (in) {
    constexpr int AHEAD = 2;
    for (long long r0 = begin + y; r0 < end; r0 += AHEAD * ty) {
      Piece<TYPE, VEC> d[AHEAD], g[AHEAD], v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const long long r = r0 + i * ty;
        if (r < end) {
          d[i].load(p.dc, r * p.lddc + col);
          g[i].load(p.up, r * p.ldup + col);
          v[i].load(p.up, r * p.ldup + p.F + col);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const long long r = r0 + i * ty;
        if (r < end) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float act, slope;
            gate_slope(E::get(g[i].v[j]), p.gate, act, slope);
            const float dc = E::get(d[i].v[j]);
            const float dg = dc * E::get(v[i].v[j]) * slope, dv = dc * act;
            if constexpr (BIAS) {
              sg[j] += dg;
              sv[j] += dv;
            }
            // (rounded to 16 bits, as the tensor cores take both products' operands; FP16 past 65504 is infinite)
            g[i].v[j] = E::put(dg);
            v[i].v[j] = E::put(dv);
          }
          g[i].store(p.dup, r * p.lddup + col);
          v[i].store(p.dup, r * p.lddup + p.F + col);
        }
      }
    }
  }
  if constexpr (BIAS) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sums[(2 * j) * kGateThreads + threadIdx.x] = sg[j];
      sums[(2 * j + 1) * kGateThreads + threadIdx.x] = sv[j];
    }
    __syncthreads();
    if (y == 0 && in) {
      float* out = p.partial + static_cast<long long>(blockIdx.y) * 2 * p.F;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float a = 0.0f, b = 0.0f;
        for (int t = 0; t < ty; ++t) {
          a += sums[(2 * j) * kGateThreads + t * p.tx + x];
          b += sums[(2 * j + 1) * kGateThreads + t * p.tx + x];
        }
        out[col + j] = a;
        out[p.F + col + j] = b;
      }
    }
  }
  grid_launch_dependents();
}

// dbias from the row blocks' partial sums, in their order; 32 columns a block, a warp's share of the rows each.
template <int TYPE>
__global__ void __launch_bounds__(256) bias_sum_kernel(const float* partial, int rows, int cols, void* out) {
  using E = Elem<TYPE>;
  __shared__ float part[8][32];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  grid_dependency_wait();
  float s = 0.0f;
  if (col < cols)
    for (int r = g; r < rows; r += 8) s += __ldcg(partial + static_cast<long long>(r) * cols + col);
  part[g][c] = s;
  __syncthreads();
  if (g == 0 && col < cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][c];
    static_cast<typename E::T*>(out)[col] = E::put(s);
  }
  grid_launch_dependents();
}

// The value half of row-major weights that starts off a 16-byte boundary (m bytes past one), in rows that start on
// them: a tiled TMA copy has to start on such a boundary, its innermost coordinate as well as its address (an
// illegal instruction otherwise), so the half cannot be read at column F of W's own map. 16 bytes a thread, shifted together from the two aligned pieces that hold them; a row's last ones element by
// element. Bound by memory, and a second launch: 1000 x 3000 FP16 adds about 5 us. (Copied with the gate half, a warp a
// row, it took 14.)
struct HalfParams {
  const uint8_t* w;
  uint8_t* to;
  long long ld, pitch;  // bytes
  int rows, F, pieces;  // pieces of a row
};
__global__ void __launch_bounds__(256) copy_half_kernel(const HalfParams p) {
  grid_dependency_wait();
  const long long at = blockIdx.x * 256LL + threadIdx.x;
  const int row = static_cast<int>(at / p.pieces), i = static_cast<int>(at - static_cast<long long>(row) * p.pieces);
  if (row < p.rows) {
    const uint8_t* src = p.w + row * p.ld;
    const long long begin = 2LL * p.F + 16LL * i, end = 4LL * p.F;  // of this piece, and of the row
    const int m = static_cast<int>(begin & 15);
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (begin - m + 32 <= end) {
      const uint4 lo = *reinterpret_cast<const uint4*>(src + begin - m), hi = *reinterpret_cast<const uint4*>(src + begin - m + 16);
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      uint32_t a[6], b[5];
#pragma unroll
      for (int k = 0; k < 6; ++k) a[k] = m & 8 ? w[k + 2] : w[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) b[k] = m & 4 ? a[k + 1] : a[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(b[k], b[k + 1], (m & 3) * 8);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (begin + 2 * k < end)
          o[k >> 1] |= uint32_t(*reinterpret_cast<const uint16_t*>(src + begin + 2 * k)) << (16 * (k & 1));
    }
    *reinterpret_cast<uint4*>(p.to + row * p.pitch + 16LL * i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  grid_launch_dependents();
}

constexpr int64_t kIntLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kLdLimit = int64_t(1) << 39;

bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }
int64_t dup_pitch(int64_t F) { return (2 * F + 63) / 64 * 64; }
int64_t padded(int64_t bytes) { return (bytes + 127) / 128 * 128; }

int kind_of(int type) { return type == GEMM_TYPE_F16 ? KIND_F16 : KIND_BF16; }

bool meet(const void* a, int64_t rows_a, int64_t cols_a, int64_t ld_a, const void* b, int64_t rows_b, int64_t cols_b,
          int64_t ld_b) {
  if (a == nullptr || b == nullptr || rows_a == 0 || rows_b == 0 || cols_a == 0 || cols_b == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), a1 = a0 + uintptr_t(((rows_a - 1) * ld_a + cols_a) * 2);
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(b), b1 = b0 + uintptr_t(((rows_b - 1) * ld_b + cols_b) * 2);
  return a0 < b1 && b0 < a1;
}

// Row blocks of the gradient's first kernel: what fills the GPU, but for dbias at most kBiasBlocks.
struct GateGrid {
  int tx, blocks_x, blocks_y, rows_per_block;
};
GateGrid gate_grid(int64_t M, int64_t F, int vec, bool bias, int sms) {
  GateGrid g;
  const int64_t pieces = (F + vec - 1) / vec;
  g.tx = 32;
  while (g.tx < kGateThreads && g.tx < pieces) g.tx *= 2;
  g.blocks_x = int((pieces + g.tx - 1) / g.tx);
  const int64_t want = (sms * 8 + g.blocks_x - 1) / g.blocks_x, most = bias && want > kBiasBlocks ? kBiasBlocks : want;
  const int64_t rows = (M + most - 1) / most, step = kGateThreads / g.tx;
  g.rows_per_block = int((rows + step - 1) / step * step);
  g.blocks_y = int((M + g.rows_per_block - 1) / g.rows_per_block);
  return g;
}

template <int TYPE, int VEC>
cudaError_t launch_gate_grad(const GateGradParams& p, const GateGrid& g, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(g.blocks_x, g.blocks_y, 1);
  cfg.blockDim = dim3(kGateThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t launched = p.partial != nullptr ? cudaLaunchKernelEx(&cfg, gate_grad_kernel<TYPE, VEC, true>, p)
                                                    : cudaLaunchKernelEx(&cfg, gate_grad_kernel<TYPE, VEC, false>, p);
  const cudaError_t last = cudaGetLastError();
  const cudaError_t e = launched != cudaSuccess ? launched : last;
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int TYPE>
cudaError_t launch_gate_grad_type(const GateGradParams& p, int vec, const GateGrid& g, cudaStream_t s) {
  return vec == 8   ? launch_gate_grad<TYPE, 8>(p, g, s)
         : vec == 4 ? launch_gate_grad<TYPE, 4>(p, g, s)
         : vec == 2 ? launch_gate_grad<TYPE, 2>(p, g, s)
                    : launch_gate_grad<TYPE, 1>(p, g, s);
}

// Bytes of the copy of row-major weights' value half, where that is all of W that TMA cannot read in place.
int64_t half_bytes(int64_t F, int64_t K, int64_t ldw, int layout) {
  const bool off = layout == GEMM_B_ROW_MAJOR && F % 8 != 0 && K > 0 && (K == 1 || ldw % 8 == 0);
  return off ? K * padded(2 * F) : 0;
}

int copy_half(const void* W, int64_t ldw, int64_t K, int64_t F, void* to, int64_t ld, cudaStream_t stream) {
  const HalfParams h = {static_cast<const uint8_t*>(W), static_cast<uint8_t*>(to), (long long)ldw * 2, (long long)ld * 2,
                        int(K), int(F), int((2 * F + 15) / 16)};
  const int64_t blocks = (K * h.pieces + 255) / 256;
  if (blocks > kIntLimit) return GEMM_ERR_INVALID_VALUE;
  return launch_dependent(copy_half_kernel, int(blocks), 256, 0, stream, 1, h) == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// The product of few rows, where TMA reads both operands in place; F columns of C (gate -1: W has them alone). All
// arguments have been checked.
int run_few(int type, int64_t M, int64_t F, int64_t K, const void* A, int64_t lda, const void* W, int64_t ldw,
            bool row_major, const void* value, int64_t ldv, int gate, const void* bias, void* C, int64_t ldc, void* up,
            int64_t ldup, const CallContext& ctx, cudaStream_t s) {
  GatedFewLaunch L;
  memset(&L, 0, sizeof(L));
  GatedFewParams& p = L.p;
  p.g.status = ctx.status;
  p.g.epoch = ctx.epoch;
  p.g.debug = ctx.debug;
  p.g.wait_limit_ns = ctx.wait_limit_ns;
  p.g.C = C;
  p.g.ldc = ldc;
  p.g.bias = bias;
  p.g.num_kb = int((K + 63) / 64);
  p.M = int(M);
  p.F = int(F);
  const bool plain = gate < 0;
  p.value_at = plain ? 64 : value != nullptr ? 0 : int(F);
  p.gate = gate;
  p.up = up;
  p.ldup = ldup;
  L.row_major = row_major;
  L.bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  L.dev = ctx.dev;
  L.stream = s;
  p.tiles_t = int((M + L.bn - 1) / L.bn);
  const int64_t tiles = (plain ? (F + 127) / 128 : (F + 63) / 64) * p.tiles_t;
  L.deep = tiles <= ctx.sm_count;
  p.splits = choose_splits(tiles, p.g.num_kb, L.deep ? ctx.sm_count : 2 * ctx.sm_count);
  L.grid = int(tiles * p.splits);
  const CUtensorMapDataType dt = type == GEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const bool ok =
      (row_major ? encode_map_3d(&L.tmW, dt, W, plain ? F : 2 * F, K, ldw * 2, 1, 0, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)
                 : encode_map_3d(&L.tmW, dt, W, K, plain ? F : 2 * F, ldw * 2, 1, 0, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)) &&
      encode_map_3d(&L.tmA, dt, A, K, M, lda * 2, 1, 0, 64, L.bn, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return GEMM_ERR_DRIVER;
  L.tmV = L.tmW;
  if (value != nullptr && !encode_map_3d(&L.tmV, dt, value, F, K, ldv * 2, 1, 0, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  const cudaError_t e = type == GEMM_TYPE_F16 ? launch_gated_few_f16(L) : launch_gated_few_bf16(L);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// Sizes, types and flags that the forward call and the gradient share.
bool bad_sizes(int type, int64_t M, int64_t F, int64_t K, int layout, int activation) {
  return (type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16) || M < 0 || F < 0 || K < 0 || M > kIntLimit ||
         F > kIntLimit / 2 || K > kIntLimit || (layout != GEMM_B_ROW_MAJOR && layout != GEMM_B_K_MAJOR) ||
         activation < GEMM_GATE_SILU || activation > GEMM_GATE_RELU;
}

// Parts of the gradient's workspace: dup, the partial sums of dbias, then what the products stage (one after the
// other, so the larger of the two).
struct GradSpace {
  int64_t dup, partial, stage;
  int64_t total() const { return dup + partial + stage; }
};
GradSpace grad_space(int type, int64_t M, int64_t F, int64_t K, int64_t lda, int64_t ldw, int layout, bool da, bool dw,
                     bool db) {
  GradSpace s = {};
  if (M <= 0 || F <= 0 || (!da && !dw && !db)) return s;
  s.dup = padded(M * dup_pitch(F) * 2);
  s.partial = db ? padded(int64_t(kBiasBlocks < M ? kBiasBlocks : M) * 2 * F * 4) : 0;
  int64_t a = 0, w = 0;
  if (da && K > 0) {
    a = gemm_grouped_weights_workspace(type, 1, K, 2 * F, ldw, 0,
                                       layout == GEMM_B_K_MAJOR ? GEMM_B_ROW_MAJOR : GEMM_B_K_MAJOR, GEMM_ACT_NONE);
  }
  if (dw && K > 0) w = dense_wgrad_workspace(M, 2 * F, K, lda, dup_pitch(F));
  s.stage = padded(a > w ? a : w);
  return s;
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int64_t gemm_gated_workspace(int type, int64_t M, int64_t F, int64_t K, int64_t lda, int64_t ldw, int layout) {
  if (M <= 0 || F <= 0 || K <= 0) return 0;
  const int64_t half = half_bytes(F, K, ldw, layout);
  return gemm_grouped_rows_workspace(type, 1, M, K, M, lda, 0) +
         (half > 0 ? half : gemm_grouped_weights_workspace(type, 1, 2 * F, K, ldw, 0, layout, GEMM_ACT_SILU_GATED));
}

int gemm_gated(int type, int64_t M, int64_t F, int64_t K, const void* A, int64_t lda, const void* W, int64_t ldw,
               int layout, int activation, const void* bias, void* C, int64_t ldc, void* up, int64_t ldup,
               void* workspace, int64_t workspace_bytes, void* stream) {
  if (bad_sizes(type, M, F, K, layout, activation)) return GEMM_ERR_INVALID_VALUE;
  if (M > 0 && F > 0 && bias != nullptr && C != nullptr && meet(C, M, F, ldc, bias, 1, 2 * F, 2 * F))
    return GEMM_ERR_INVALID_VALUE;
  const gemm_grouped_epilogue_t epi = {1.0f, nullptr, nullptr, bias, GEMM_ACT_NONE};
  DenseProduct dense = {activation, up, ldup, nullptr, 0, nullptr, run_few, 64};
  const int64_t half = M > 0 && F > 0 ? half_bytes(F, K, ldw, layout) : 0;
  if (half > 0 && W != nullptr && C != nullptr && ldw >= 2 * F && ldw <= kLdLimit && !misaligned(W, 16)) {
    const int64_t rest = workspace_bytes - half;
    if (workspace == nullptr || rest < 0 || misaligned(workspace, 128)) return GEMM_ERR_MISALIGNED;
    if (meet(C, M, F, ldc, workspace, 1, half / 2, half / 2) || meet(up, M, 2 * F, ldup, workspace, 1, half / 2, half / 2) ||
        meet(W, K, 2 * F, ldw, workspace, 1, half / 2, half / 2) || meet(A, M, K, lda, workspace, 1, half / 2, half / 2))
      return GEMM_ERR_INVALID_VALUE;
    dense.copy = copy_half;
    dense.value = workspace;
    dense.ldv = padded(2 * F) / 2;
    workspace = rest > 0 ? static_cast<uint8_t*>(workspace) + half : nullptr;
    workspace_bytes = rest;
  }
  return run_grouped(kind_of(type), 1, nullptr, M, 2 * F, K, A, M, lda, nullptr, W, ldw, 0, C, ldc, layout, &epi,
                     workspace, workspace_bytes, stream, &dense);
}

int64_t gemm_gated_backward_workspace(int type, int64_t M, int64_t F, int64_t K, int64_t lda, int64_t ldw, int layout,
                                      int want_da, int want_dw, int want_dbias) {
  return grad_space(type, M, F, K, lda, ldw, layout, want_da != 0, want_dw != 0, want_dbias != 0).total();
}

int gemm_gated_backward(int type, int64_t M, int64_t F, int64_t K, const void* dC, int64_t lddc, const void* up,
                        int64_t ldup, const void* A, int64_t lda, const void* W, int64_t ldw, int layout,
                        int activation, void* dA, int64_t ldda, void* dW, int64_t lddw, void* dbias, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  if (bad_sizes(type, M, F, K, layout, activation)) return GEMM_ERR_INVALID_VALUE;
  const bool km = layout == GEMM_B_K_MAJOR;
  const int64_t w_rows = km ? 2 * F : K, w_cols = km ? K : 2 * F;
  if (M == 0 || K == 0) dA = nullptr;  // (F = 0: dA of no terms is zeros)
  if (F == 0 || K == 0) dW = nullptr;
  if (F == 0) dbias = nullptr;
  if (dA == nullptr && dW == nullptr && dbias == nullptr) return GEMM_OK;
  const bool terms = M > 0 && F > 0;
  // what the two products would refuse is refused before anything is launched
  if (dA != nullptr && (ldda < K || ldda > kLdLimit || (F > 0 && (W == nullptr || ldw < w_cols || ldw > kLdLimit))))
    return GEMM_ERR_INVALID_VALUE;
  if (dW != nullptr && (lddw < w_cols || lddw > kLdLimit || (M > 0 && (A == nullptr || lda < K || lda > kLdLimit))))
    return GEMM_ERR_INVALID_VALUE;
  if (terms && (dC == nullptr || up == nullptr || lddc < F || ldup < 2 * F || lddc > kLdLimit || ldup > kLdLimit))
    return GEMM_ERR_INVALID_VALUE;
  const GradSpace space = grad_space(type, M, F, K, lda, ldw, layout, dA != nullptr, dW != nullptr, dbias != nullptr);
  if (terms && (workspace == nullptr || workspace_bytes < space.total())) return GEMM_ERR_INVALID_VALUE;
  if (misaligned(dC, 2) || misaligned(up, 2) || misaligned(dA, 2) || misaligned(dW, 2) || misaligned(dbias, 2) ||
      misaligned(workspace, 128) || (terms && dA != nullptr && misaligned(W, 16)) ||
      (terms && dW != nullptr && misaligned(A, 16)))
    return GEMM_ERR_MISALIGNED;
  struct Matrix {
    const void* p;
    int64_t rows, cols, ld;
  };
  const Matrix outs[4] = {{dA, M, K, ldda},
                          {dW, w_rows, w_cols, lddw},
                          {dbias, 1, 2 * F, 2 * F},
                          {terms ? workspace : nullptr, 1, workspace_bytes / 2, workspace_bytes / 2}};
  const Matrix ins[4] = {{dC, M, F, lddc},
                         {up, M, 2 * F, ldup},
                         {dW != nullptr ? A : nullptr, M, K, lda},
                         {dA != nullptr ? W : nullptr, w_rows, w_cols, ldw}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (meet(outs[i].p, outs[i].rows, outs[i].cols, outs[i].ld, ins[j].p, ins[j].rows, ins[j].cols, ins[j].ld))
        return GEMM_ERR_INVALID_VALUE;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i].p, outs[i].rows, outs[i].cols, outs[i].ld, outs[j].p, outs[j].rows, outs[j].cols, outs[j].ld))
        return GEMM_ERR_INVALID_VALUE;
  }
  CallContext ctx;
  int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[8] = {dA, dW, dbias, terms ? workspace : nullptr, terms ? dC : nullptr, terms ? up : nullptr,
                         terms && dW != nullptr ? A : nullptr, terms && dA != nullptr ? W : nullptr};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* dup = ws;
  const int64_t lddup = dup_pitch(F);
  if (terms) {
    // the widest pieces that the rows of all matrices are made of
    int vec = 8;
    const uintptr_t all = reinterpret_cast<uintptr_t>(dC) | reinterpret_cast<uintptr_t>(up) | uintptr_t(F * 2) |
                          uintptr_t(M > 1 ? lddc * 2 : 0) | uintptr_t(M > 1 ? ldup * 2 : 0);
    while (vec > 1 && all % (vec * 2) != 0) vec /= 2;
    const GateGrid g = gate_grid(M, F, vec, dbias != nullptr, ctx.sm_count);
    GateGradParams p = {dC,
                        up,
                        ws,
                        dbias != nullptr ? reinterpret_cast<float*>(ws + space.dup) : nullptr,
                        (long long)lddc,
                        (long long)ldup,
                        (long long)lddup,
                        int(M),
                        int(F),
                        activation,
                        g.tx,
                        g.rows_per_block};
    cudaError_t e = type == GEMM_TYPE_F16 ? launch_gate_grad_type<GEMM_TYPE_F16>(p, vec, g, s)
                                          : launch_gate_grad_type<GEMM_TYPE_BF16>(p, vec, g, s);
    if (e == cudaSuccess && dbias != nullptr) {
      const int cols = int(2 * F), grid = (cols + 31) / 32;
      e = type == GEMM_TYPE_F16 ? launch_dependent(bias_sum_kernel<GEMM_TYPE_F16>, grid, 256, 0, s, 1, p.partial, g.blocks_y, cols, dbias)
                                : launch_dependent(bias_sum_kernel<GEMM_TYPE_BF16>, grid, 256, 0, s, 1, p.partial, g.blocks_y, cols, dbias);
    }
    if (e != cudaSuccess) return GEMM_ERR_LAUNCH;
  } else if (dbias != nullptr) {  // no rows
    if (cudaMemsetAsync(dbias, 0, size_t(2 * F) * 2, s) != cudaSuccess) return GEMM_ERR_LAUNCH;
  }
  uint8_t* stage = terms && space.stage > 0 ? ws + space.dup + space.partial : nullptr;
  if (dA != nullptr) {
    const DenseProduct dense = {-1, nullptr, 0, nullptr, 0, nullptr, run_few, 128};
    st = run_grouped(kind_of(type), 1, nullptr, M, K, 2 * F, dup, M, lddup, nullptr, W, ldw, 0, dA, ldda,
                     km ? GEMM_B_ROW_MAJOR : GEMM_B_K_MAJOR, nullptr, stage, space.stage, stream, &dense);
    if (st != GEMM_OK) return st;
  }
  if (dW != nullptr)
    st = run_wgrad(kind_of(type), 1, nullptr, M, 2 * F, K, A, M, lda, nullptr, dup, lddup, dW, lddw, 0, layout, stage,
                   space.stage, stream, true);
  return st;
}

}  // extern "C"
