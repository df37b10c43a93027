// The dense gated product of few rows (gemm_gated), for sm_103a: bound by reading
// the weights once.
//
//   C[t][j] = act(g) v,  g = A[t] . W[:, j] + bias[j],  v = A[t] . W[:, F + j] + bias[F + j]
//
// The weights are the MMA's 128-row operand -- 64 gate columns of W and the 64 value
// columns that belong to them -- and the rows of A its narrow one (BN = 16, 32 or
// 64), so that a tile wastes nothing on rows that are not there. A tile's k-loop
// is shared by a cluster of `splits` CTAs: each has a run of slabs of 64, and they
// add their sums through distributed shared memory, in order, where gate and value
// meet. DEEP: one CTA to an SM, with all of its shared memory for loads in flight;
// else two, for more tiles than SMs. Warps: 0-3 take the sums out of tensor memory,
// 4 loads by TMA, 5 issues tcgen05.mma.
// The plain product (gate < 0; the gradient of A) is the same with 128 neighbouring
// columns to a tile. 16 x 4096 -> 2 x 8192 BF16 24.8 us (5.4 TB/s; the bytes 19.8,
// the rest is the launch, the first loads and the join), -> 2 x 2048 9.7.
#pragma once

#include "dgt_feedforward.h"
#include "gemm_kernel.cuh"
#include "split_join.cuh"

namespace dgt {

struct GatedFewParams {
  GemmParams g;  // C, ldc, bias, num_kb and the launch-wide status fields
  int M, F;      // rows of A; columns of C
  int value_at;  // where the value half starts in its map (a column of row-major W, else a row); plain: 64
  int gate;      // GEMM_GATE_*, or -1: no gate
  void* up;
  long long ldup;
  int splits;
  int tiles_t;  // tiles along the rows of A
};

constexpr int kFewThreads = 256;

// MN: W is row-major (K x 2F), the MMA's operand MN-major; else 2F x K, K-major.
template <int KIND, bool MN, int BN_, bool DEEP>
struct GatedFewCfg {
  static constexpr int BN = BN_;
  static constexpr int BK = 64;
  static constexpr int P_BYTES = 128 * 128;  // two boxes of 64 x 128 bytes, or of 64 rows of K x 128 bytes
  static constexpr int Q_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int SMEM_LIMIT = DEEP ? 227 * 1024 : 113 * 1024;  // one or two CTAs to an SM
  static constexpr int STAGES = (SMEM_LIMIT - 1024 - 256) / STAGE_BYTES;
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  static constexpr int SUM_LD = 129;
  static constexpr int BAR_BYTES = 256;
  static_assert((2 * STAGES + 1) * 8 + 16 <= BAR_BYTES, "barrier area");
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + BAR_BYTES;
  static_assert(BN * SUM_LD * 4 <= STAGES * STAGE_BYTES, "the sums reuse the stages");
  static constexpr uint32_t IDESC = (1u << 4) | (KindTraits<KIND>::fmt << 7) | (KindTraits<KIND>::fmt << 10) |
                                    ((MN ? 1u : 0u) << 15) | (uint32_t(BN >> 3) << 17) | (uint32_t(128 >> 4) << 24);
};

__device__ __forceinline__ float gate_of(float x, int gate) {
  if (gate == GEMM_GATE_SILU) return __fdividef(x, 1.0f + __expf(-x));
  if (gate == GEMM_GATE_RELU) return x < 0.0f ? 0.0f : x;
  if (gate == GEMM_GATE_GELU) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
  const float u = 0.79788456080286536f * (x + 0.044715f * x * x * x);
  return __fdividef(x, 1.0f + __expf(-2.0f * u));
}

template <int KIND>
__device__ __forceinline__ float from16(const void* base, long long at) {
  if constexpr (KIND == KIND_F16)
    return __half2float(static_cast<const __half*>(base)[at]);
  else
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
}
template <int KIND>
__device__ __forceinline__ void to16(void* base, long long at, float v) {
  if constexpr (KIND == KIND_F16)
    static_cast<__half*>(base)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v);
}

template <int KIND, bool MN, int BN, bool DEEP>
__global__ void __launch_bounds__(kFewThreads)
    gated_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmA, const __grid_constant__ GatedFewParams p) {
  using Cf = GatedFewCfg<KIND, MN, BN, DEEP>;
  constexpr int S = Cf::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - raw);
  const uint32_t sP = sbase, sQ = sbase + S * Cf::P_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sptr + S * Cf::STAGE_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * S;
  const uint32_t done_bar = empty0 + 8 * S;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(bars + 2 * S + 1);
  volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot) + 1;
  volatile int* consumed_slot = issued_slot + 1;
  float* sums = reinterpret_cast<float*>(sptr);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(blockIdx.x % p.splits);
  // (tiles of the same weights are neighbours)
  const int tile = static_cast<int>(blockIdx.x / p.splits);
  const bool plain = p.gate < 0;
  const int n0 = tile / p.tiles_t * (plain ? 128 : 64), row0 = tile % p.tiles_t * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.g.num_kb) * split / p.splits);
  const int kb1 = static_cast<int>(static_cast<long long>(p.g.num_kb) * (split + 1) / p.splits);

  if (warp == 4 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done_bar, 1);
    *issued_slot = 0;
    *consumed_slot = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), Cf::TMEM_COLS);
    tmem_relinquish();
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA producer
    if (!(p.g.debug & DEBUG_STALL_PRODUCER)) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % S;
        if (!warp_wait_short(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) break;
        if (elect_one()) {
          const uint32_t fb = full0 + 8 * s, w = sP + s * Cf::P_BYTES;
          const int k = kb * Cf::BK;
          mbar_arrive_expect_tx(fb, Cf::STAGE_BYTES);
          if constexpr (MN) {
            tma_load_3d(w, &tmW, fb, n0, k, 0);
            tma_load_3d(w + Cf::P_BYTES / 2, &tmV, fb, p.value_at + n0, k, 0);
          } else {
            tma_load_3d(w, &tmW, fb, k, n0, 0);
            tma_load_3d(w + Cf::P_BYTES / 2, &tmV, fb, k, p.value_at + n0, 0);
          }
          tma_load_3d(sQ + s * Cf::Q_BYTES, &tmA, fb, k, row0, 0);
        }
        __syncwarp();
      }
      if (lane == 0) *issued_slot = it;
    }
    grid_launch_dependents();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t P_STEP = (MN ? 16 * 128 : 32) / 16;
    const uint64_t p_desc = sdesc(sP, MN ? Cf::P_BYTES / 2 : 16, 1024, SWZ_128B), q_desc = sdesc(sQ, 16, 1024, SWZ_128B);
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S;
      if (!warp_wait_short(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8))) break;
      tc_fence_after();
      const uint64_t ps = p_desc + static_cast<uint32_t>(s) * (Cf::P_BYTES / 16);
      const uint64_t qs = q_desc + static_cast<uint32_t>(s) * (Cf::Q_BYTES / 16);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_issue<KIND>(tmem, ps + kk * P_STEP, qs + kk * 2, Cf::IDESC, it > 0 || kk > 0 ? 1u : 0u);
        mma_commit(empty0 + 8 * s);
      }
      __syncwarp();
    }
    if (lane == 0) *consumed_slot = it;
    if (elect_one()) mma_commit(done_bar);
    __syncwarp();
  }
  // every warp waits for the MMAs, also where the launch was aborted: nothing may read shared memory after this
  if (lane == 0 && !wait_short(done_bar, 0)) wait_phase_drain(p.g, done_bar, 0);
  __syncwarp();
  tc_fence_after();
  if (warp < 4) {
    // the stages have been read: the sums take their place
    constexpr int CH = BN < 32 ? BN : 32;
#pragma unroll
    for (int c = 0; c < BN; c += CH) {
      uint32_t r[CH];
      __syncwarp();
      tmem_ld_cols<CH>(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, r);
#pragma unroll
      for (int j = 0; j < CH; ++j) sums[(c + j) * Cf::SUM_LD + warp * 32 + lane] = __uint_as_float(r[j]);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  {
    // this CTA's share of the rows of A
    const int left = min(BN, p.M - row0), c0 = min(BN * split / p.splits, left), c1 = min(BN * (split + 1) / p.splits, left);
    if (plain) {
      for (int e = threadIdx.x; e < (c1 - c0) * 128; e += kFewThreads) {
        const int c = c0 + e / 128, r = e % 128, j = n0 + r;
        if (j < p.F)
          to16<KIND>(p.g.C, static_cast<long long>(row0 + c) * p.g.ldc + j, joined_sum(sums, c * Cf::SUM_LD + r, p.splits));
      }
    }
    for (int e = threadIdx.x; !plain && e < (c1 - c0) * 64; e += kFewThreads) {
      const int c = c0 + e / 64, r = e % 64, j = n0 + r;
      if (j >= p.F) continue;
      const int at = c * Cf::SUM_LD + r;
      const long long t = row0 + c;
      float gate = joined_sum(sums, at, p.splits), value = joined_sum(sums, at + 64, p.splits);
      if (p.g.bias != nullptr) {
        gate += from16<KIND>(p.g.bias, j);
        value += from16<KIND>(p.g.bias, p.F + static_cast<long long>(j));
      }
      to16<KIND>(p.g.C, t * p.g.ldc + j, gate_of(gate, p.gate) * value);
      if (p.up != nullptr) {
        to16<KIND>(p.up, t * p.ldup + j, gate);
        to16<KIND>(p.up, t * p.ldup + p.F + j, value);
      }
    }
  }

  // ------------------------------------------------------------------ teardown
  // loads issued but not consumed exist only when the launch was aborted: let them land
  if (threadIdx.x == 0 && *consumed_slot < *issued_slot) {
    const int issued = *issued_slot;
    for (int j = *consumed_slot; j < issued; ++j)
      if (!wait_phase_drain(p.g, full0 + 8 * (j % S), (j / S) & 1)) break;
  }
  if (p.splits > 1)
    cluster_sync();  // no CTA leaves while another may still read its sums
  else
    __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, Cf::TMEM_COLS);
  }
}

}  // namespace dgt
