// Element access of the bandwidth-bound kernels (norm, combine): VEC elements
// of a type at a time, held as fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "dgt_experts.h"

namespace dgt {

template <int TYPE>
struct Elem;
template <>
struct Elem<GEMM_TYPE_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<GEMM_TYPE_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<GEMM_TYPE_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

inline int type_bytes(int type) { return type == GEMM_TYPE_F32 ? 4 : type == GEMM_TYPE_E4M3 ? 1 : 2; }

// VEC consecutive elements as loaded: 16 bytes, or one element (VEC = 1).
template <int TYPE, int VEC>
struct Pack {
  using E = Elem<TYPE>;
  using T = typename E::T;
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "16 bytes or one element");
  alignas(VEC * sizeof(T)) T v[VEC];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1)
      v[0] = *p;
    else
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
  }
  // a load of data that is read once: it leaves L1 to what is read again
  __device__ __forceinline__ void stream(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = *p;
    } else {
      uint4 q;
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                   : "l"(p)
                   : "memory");
      *reinterpret_cast<uint4*>(v) = q;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1)
      *p = v[0];
    else
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
  }
  __device__ __forceinline__ void zero() {
    if constexpr (VEC == 1)
      v[0] = E::put(0.0f);
    else
      *reinterpret_cast<uint4*>(v) = make_uint4(0u, 0u, 0u, 0u);
  }
  // Element i as fp32 (bfloat16 is the upper half of an fp32: a shift or a mask of its word).
  __device__ __forceinline__ float get(int i) const {
    if constexpr (TYPE == GEMM_TYPE_BF16 && VEC > 1) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(v)[i >> 1];
      return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
    } else {
      return E::get(v[i]);
    }
  }
  // Elements i and i + 1.
  __device__ __forceinline__ float2 two(int i) const { return make_float2(get(i), get(i + 1)); }
  // All elements from fp32, rounded to nearest even, two at a time.
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
    if constexpr (VEC == 1 || TYPE == GEMM_TYPE_F32) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = E::put(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        if constexpr (TYPE == GEMM_TYPE_BF16)
          *reinterpret_cast<__nv_bfloat162*>(v + i) = __floats2bfloat162_rn(x[i], x[i + 1]);
        else
          *reinterpret_cast<__half2*>(v + i) = __floats2half2_rn(x[i], x[i + 1]);
      }
    }
  }
};

// VEC values to E4M3 (round to nearest even, saturating; NaN stays NaN).
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    *p = __nv_cvt_float_to_fp8(x[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

}  // namespace dgt
