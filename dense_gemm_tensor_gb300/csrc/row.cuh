// What the norms' kernels share (norm.cu, layer_norm.cu): a row as pieces of the
// threads that own it, reductions over its warps, and the host's choice among the
// ways to reach memory:
//   ALIGNED  rows start on 16-byte boundaries and hold whole 16-byte pieces
//   FLAT     every matrix is contiguous, from a 16-byte boundary, with rows of
//            any width: a row is the 16-byte pieces of the flat array that meet
//            it, and its first and last ones are partly other rows' (those two
//            go element by element). Weights, and the gradient's dw, are then at
//            another offset in every row: they sit in shared memory, element c
//            at (c mod VEC, c / VEC), where the lanes' accesses do not collide.
//   SINGLE   anything else: one element at a time
#pragma once

#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dgt {
namespace {

enum { ALIGNED = 0, FLAT = 1, SINGLE = 2 };

constexpr int64_t kMaxCols = 16384;
constexpr int64_t kMaxFlatCols = 11000;  // a FLAT row meets one piece more, and its weights (and dw) fit shared memory
constexpr float kE4M3Max = 448.0f;

// Elements a thread holds of a row: 8 (few rows, for their latency), or 64 bytes' worth; single elements take a
// register each, so 16 of them.
template <int TYPE, int MODE>
constexpr int kFullEpt = MODE == SINGLE ? 16 : 64 / int(sizeof(typename Elem<TYPE>::T));
// Threads of a block: 16384 columns' worth.
template <int TYPE, int EPT>
constexpr int kNormThreads = EPT == 8 ? 1024 : int(kMaxCols) / EPT;

// A row as the thread's pieces: piece i holds columns lo(i) .. lo(i) + VEC - 1.
template <int MODE, int VEC>
struct Row {
  int tid, tpr, cols, shift;

  __device__ __forceinline__ Row(int tid_, int tpr_, int cols_) : tid(tid_), tpr(tpr_), cols(cols_), shift(0) {}
  // FLAT: the row's first piece starts `shift` elements before it
  __device__ __forceinline__ void at(long long row) {
    if constexpr (MODE == FLAT) shift = static_cast<int>((row * cols) % VEC);
  }
  __device__ __forceinline__ int lo(int i) const { return (i * tpr + tid) * VEC - shift; }
  __device__ __forceinline__ bool whole(int i) const {
    return MODE == FLAT ? lo(i) >= 0 && lo(i) + VEC <= cols : lo(i) < cols;
  }
  // index of column lo(i) + j in shared memory
  __device__ __forceinline__ int place(int i, int j) const {
    const int c = lo(i) + j;
    return (c % VEC) * ((cols + VEC - 1) / VEC) + c / VEC;
  }
  template <int TYPE>
  __device__ __forceinline__ void load(Pack<TYPE, VEC>& v, const void* base, long long row, long long ld, int i,
                                       bool in) const {
    using T = typename Pack<TYPE, VEC>::T;
    v.zero();
    if (!in) return;
    const T* p = static_cast<const T*>(base) + row * ld;
    if (whole(i)) {
      v.stream(p + lo(i));
    } else if constexpr (MODE == FLAT) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (lo(i) + j >= 0 && lo(i) + j < cols) v.v[j] = p[lo(i) + j];
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
        if (lo(i) + j >= 0 && lo(i) + j < cols) p[lo(i) + j] = v.v[j];
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
        if (lo(i) + j >= 0 && lo(i) + j < cols) p[lo(i) + j] = __nv_cvt_float_to_fp8(x[j], __NV_SATFINITE, __NV_E4M3);
    }
  }
};

// Column weights of piece i as fp32: from memory (L1 holds them), or from shared memory (FLAT).
template <int MODE, int TYPE, int VEC>
__device__ __forceinline__ void load_weights(float (&w)[VEC], const Row<MODE, VEC>& r, const void* weight,
                                             const typename Elem<TYPE>::T* shared, int i) {
  using E = Elem<TYPE>;
  if constexpr (MODE == FLAT) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = r.lo(i) + j;
      w[j] = c >= 0 && c < r.cols ? E::get(shared[r.place(i, j)]) : 0.0f;
    }
  } else {
    Pack<TYPE, VEC> v;
    v.zero();
    if (r.whole(i)) v.load(static_cast<const typename E::T*>(weight) + r.lo(i));
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = v.get(j);
  }
}

// FLAT: the weights in shared memory, in place()'s order.
template <int TYPE, int VEC>
__device__ __forceinline__ void stage_weights(typename Elem<TYPE>::T* shared, const void* weight, int cols) {
  const int per = (cols + VEC - 1) / VEC;
  for (int c = threadIdx.x; c < cols; c += blockDim.x)
    shared[(c % VEC) * per + c / VEC] = static_cast<const typename Elem<TYPE>::T*>(weight)[c];
  __syncthreads();
}

// Reductions over the `warps` warps of a row, of which the first is the block's
// warp w0. All threads of the block call them together; `red` holds a value per
// warp and is not written again by the caller's next reduction (it alternates).
struct RowWarps {
  int warps, w0;
  __device__ __forceinline__ RowWarps(int tpr, int sub) : warps(tpr >> 5), w0(sub * (tpr >> 5)) {}
  __device__ __forceinline__ float sum(float v, float* red) const {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[w0 + lane] : 0.0f);
  }
  // the largest of non-negative bit patterns
  __device__ __forceinline__ uint32_t max_bits(uint32_t v, float* red_) const {
    uint32_t* red = reinterpret_cast<uint32_t*>(red_);
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xFFFFFFFFu, lane < warps ? red[w0 + lane] : 0u);
  }
};

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

bool aligned(const void* p, int64_t ld, int es, int to) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * es)) % to) == 0;
}

// Threads that own a row of `cols` elements, `ept` each: whole warps. A FLAT row may meet one piece more.
int threads_per_row(int64_t cols, int ept, int mode, int vec) {
  const int64_t most = cols + (mode == FLAT ? vec : 0);
  return int((most + 32 * ept - 1) / (32 * ept) * 32);
}

// A contiguous matrix from a `to`-byte boundary.
bool flat(const void* p, int64_t ld, int64_t cols, int to) {
  return ld == cols && reinterpret_cast<uintptr_t>(p) % to == 0;
}

bool bad_type(int type) { return type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F32; }
bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 39); }

bool meet(const void* a, int64_t rows_a, int64_t cols_a, int64_t ld_a, int es_a, const void* b, int64_t rows_b,
          int64_t cols_b, int64_t ld_b, int es_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), a1 = a0 + uintptr_t(((rows_a - 1) * ld_a + cols_a) * es_a);
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(b), b1 = b0 + uintptr_t(((rows_b - 1) * ld_b + cols_b) * es_b);
  return a0 < b1 && b0 < a1;
}

}  // namespace
}  // namespace dgt
