// Products of E4M3 matrices with a scale for each block of 128 along K
// (gemm_e4m3_blocks), for sm_103a: what its kernels share, and the one for few rows.
//
//   C[i][j] = sum over blocks b of sa[i][b] sb[j][b] (sum over k of block b of A[i][k] B[j][k])
//
// A stage of the pipeline is one block (128 bytes of K), so the tensor cores sum a
// block into an accumulator of its own in tensor memory, and the epilogue warps
// take it from there, scale it and add it to the tile's sums, which they hold in
// registers.
//
// Few rows of A are bound by reading B. So B is the MMA's 128-row operand P, and A
// the narrow one Q (BN = 16, 32 or 64 of its rows): 128 lanes are 128 columns of C,
// and a narrow tile wastes nothing on rows that are not there. A tile's blocks are
// shared by a cluster of `splits` CTAs, and those add their sums through
// distributed shared memory, in order. Warps: 0-3 epilogue, 4 TMA producer, 5
// tcgen05.mma, 6 the scales of A's rows, 7 those of B's; these run up to
// kScaleRing blocks ahead (loaded as they were needed, four blocks at a time, each
// four cost a trip to memory). 16 x 8192 x 8192 15.4 us (4.4 TB/s; the bytes 9.9,
// the rest is the launch, the first loads and the join).
#pragma once

#include <type_traits>

#include "dgt_feedforward.h"
#include "gemm_kernel.cuh"
#include "split_join.cuh"

namespace dgt {

constexpr int kBlockK = 128;

// Scales of an operand: row r, block b at s[(r >> shift) * row + b * block].
struct BlockScales {
  const float* s;
  long long row, block;
  int shift;
  // (plain loads: the previous kernel on the stream, which this one's start overlaps, may be what writes the scales)
  __device__ __forceinline__ const float* from(int r, int b) const { return s + ((r >> shift) * row + b * block); }
  __device__ __forceinline__ float at(int r, int b) const { return *from(r, b); }
};

struct BlockParams {
  GemmParams g;  // C, ldc, num_kb, raster, tiles_m (of P), tiles_n (of Q) and the launch-wide status fields
  BlockScales ps, qs;
  int p_rows, q_rows;
  int splits;
};

constexpr int kBlockThreads = 256;
constexpr int kScaleRing = 16;

template <int BN_>
struct BlockCfg {
  static constexpr int BN = BN_;
  static constexpr int BM = 128;
  static constexpr int P_BYTES = BM * 128;
  static constexpr int Q_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int SCALE_BYTES = kScaleRing * (BN + BM) * 4;
  static constexpr int BAR_BYTES = 512;
  static constexpr int SMEM_LIMIT = 113 * 1024;  // two CTAs to an SM
  static constexpr int STAGES = (SMEM_LIMIT - 1024 - SCALE_BYTES - BAR_BYTES) / STAGE_BYTES;
  static constexpr int ACCS = 4;                 // accumulators in tensor memory
  static constexpr int TMEM_COLS = ACCS * BN;
  static constexpr int SUM_LD = BM + 1;          // a column of the shared sums (free of bank conflicts either way)
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + SCALE_BYTES + BAR_BYTES;
  static_assert(BN == 16 || BN == 32 || BN == 64, "tile width");
  static_assert(BN * SUM_LD * 4 <= STAGES * STAGE_BYTES, "the sums reuse the stages");
  static_assert((2 * STAGES + 2 * ACCS + 1 + 2 * kScaleRing) * 8 + 16 <= BAR_BYTES, "barrier area");
  // D fp32, E4M3 operands, both K-major
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
};

template <int BN>
__global__ void __launch_bounds__(kBlockThreads)
    block_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                 const __grid_constant__ BlockParams p) {
  using Cf = BlockCfg<BN>;
  constexpr int S = Cf::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - raw);
  const uint32_t sP = sbase, sQ = sbase + S * Cf::P_BYTES;
  float* scales = reinterpret_cast<float*>(sptr + S * Cf::STAGE_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sptr + S * Cf::STAGE_BYTES + Cf::SCALE_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * S;
  const uint32_t accf0 = empty0 + 8 * S;
  const uint32_t acce0 = accf0 + 8 * Cf::ACCS;
  const uint32_t scf0 = acce0 + 8 * Cf::ACCS;
  const uint32_t sce0 = scf0 + 8 * kScaleRing;
  const uint32_t drain_bar = sce0 + 8 * kScaleRing;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sptr + (drain_bar + 8 - sbase));
  volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot) + 1;
  volatile int* consumed_slot = issued_slot + 1;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(blockIdx.x % p.splits), tile = static_cast<int>(blockIdx.x / p.splits);
  int mb, nb;
  {
    const int band = p.g.raster * p.g.tiles_n, b = tile / band, first = b * p.g.raster;
    const int rows = min(p.g.raster, p.g.tiles_m - first), q = tile - b * band;
    nb = q / rows;
    mb = first + (q - nb * rows);
  }
  const int p0 = mb * Cf::BM, q0 = nb * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.g.num_kb) * split / p.splits);
  const int kb1 = static_cast<int>(static_cast<long long>(p.g.num_kb) * (split + 1) / p.splits);

  if (warp == 4 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < Cf::ACCS; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 4);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(scf0 + 8 * i, 2);
      mbar_init(sce0 + 8 * i, 4);
    }
    mbar_init(drain_bar, 1);
    *issued_slot = 0;
    *consumed_slot = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
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
  float* sums = reinterpret_cast<float*>(sptr);

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA producer
    if (!(p.g.debug & DEBUG_STALL_PRODUCER)) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % S;
        if (!warp_wait_short(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) break;
        if (elect_one()) {
          const uint32_t fb = full0 + 8 * s;
          mbar_arrive_expect_tx(fb, Cf::STAGE_BYTES);
          tma_load_3d(sP + s * Cf::P_BYTES, &tmP, fb, kb * kBlockK, p0, 0);
          tma_load_3d(sQ + s * Cf::Q_BYTES, &tmQ, fb, kb * kBlockK, q0, 0);
        }
        __syncwarp();
      }
      if (lane == 0) *issued_slot = it;
    }
    grid_launch_dependents();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    const uint64_t p_desc = sdesc(sP, 16, 1024, SWZ_128B), q_desc = sdesc(sQ, 16, 1024, SWZ_128B);
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S, b = it % Cf::ACCS;
      if (!warp_wait_short(p.g, acce0 + 8 * b, ((it / Cf::ACCS) & 1) ^ 1, ROLE_MMA | (0x80u << 8))) break;
      if (!warp_wait_short(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8))) break;
      tc_fence_after();
      const uint64_t ps = p_desc + static_cast<uint32_t>(s) * (Cf::P_BYTES / 16);
      const uint64_t qs = q_desc + static_cast<uint32_t>(s) * (Cf::Q_BYTES / 16);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8f6f4(tmem + b * BN, ps + kk * 2, qs + kk * 2, Cf::IDESC, kk > 0 ? 1u : 0u);
        mma_commit(empty0 + 8 * s);
        mma_commit(accf0 + 8 * b);
      }
      __syncwarp();
    }
    if (lane == 0) *consumed_slot = it;
    if (elect_one()) mma_commit(drain_bar);
    __syncwarp();
    if (lane == 0) wait_phase_drain(p.g, drain_bar, 0);
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------------------------------------------------------- scales: of A's rows (warp 6), of B's (warp 7)
    int it = 0;
    // hands the scales of the next block over: entries lane, lane + 32, ... of n
    auto put = [&](int at, int n, auto value) {
      const int slot = it % kScaleRing;
      if (!warp_wait_short(p.g, sce0 + 8 * slot, ((it / kScaleRing) & 1) ^ 1, ROLE_COPY | (slot << 8))) return false;
      float* to = scales + slot * (BN + Cf::BM) + at;
#pragma unroll
      for (int j = 0; j < Cf::BM / 32; ++j)
        if (lane + 32 * j < n) to[lane + 32 * j] = value(j);
      __syncwarp();
      if (lane == 0) mbar_arrive(scf0 + 8 * slot);
      ++it;
      return true;
    };
    // `per` entries a lane, AHEAD blocks ahead in registers
    auto stream = [&](const BlockScales& from, int first, int rows, int at, auto per_, auto ahead_) {
      constexpr int PER = decltype(per_)::value, AHEAD = decltype(ahead_)::value;
      const float* src[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) src[j] = from.s + min(first + lane + 32 * j, rows - 1) * from.row + kb0 * from.block;
      float next[AHEAD][PER];
      int loaded = kb0;
      auto load = [&]() {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (loaded + i < kb1) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
              next[i][j] = *src[j];
              src[j] += from.block;
            }
          }
        loaded += AHEAD;
      };
      load();
      for (int kb = kb0; kb < kb1; kb += AHEAD) {
        float now[AHEAD][PER];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
          for (int j = 0; j < PER; ++j) now[i][j] = next[i][j];
        load();
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (kb + i < kb1 && !put(at, at == 0 ? BN : Cf::BM, [&](int j) { return now[i][j < PER ? j : 0]; })) return;
      }
    };
    using std::integral_constant;
    if (warp == 6) {
      stream(p.qs, q0, p.q_rows, 0, integral_constant<int, BN == 64 ? 2 : 1>(), integral_constant<int, 8>());
    } else if (p.ps.shift == 0) {
      stream(p.ps, p0, p.p_rows, BN, integral_constant<int, 4>(), integral_constant<int, 4>());
    } else {
      // one scale for the tile's 128 rows: a lane has a block's
      auto load = [&](int kb) { return kb + lane < kb1 ? p.ps.at(p0, kb + lane) : 0.0f; };
      float next = load(kb0);
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; kb += 32) {
        const float now = next;
        next = load(kb + 32);
        for (int i = 0; ok && i < 32 && kb + i < kb1; ++i) {
          const float f = __shfl_sync(0xFFFFFFFFu, now, i);
          ok = put(BN, Cf::BM, [&](int) { return f; });
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue: lane = row of P
    constexpr int CH = BN < 32 ? BN : 32;
    float acc[BN];
#pragma unroll
    for (int c = 0; c < BN; ++c) acc[c] = 0.0f;
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int b = it % Cf::ACCS, slot = it % kScaleRing;
      if (!warp_wait_short(p.g, scf0 + 8 * slot, (it / kScaleRing) & 1, ROLE_EPILOGUE | (0x90u << 8))) break;
      if (!warp_wait_short(p.g, accf0 + 8 * b, (it / Cf::ACCS) & 1, ROLE_EPILOGUE | (b << 8))) break;
      tc_fence_after();
      const float* scale = scales + slot * (BN + Cf::BM);
      const float f = scale[BN + warp * 32 + lane];
#pragma unroll
      for (int c = 0; c < BN; c += CH) {
        uint32_t r[CH];
        __syncwarp();
        tmem_ld_cols<CH>(tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * BN + c, r);
        if (c + CH == BN) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acce0 + 8 * b);
        }
        // (the scales' product first: a block's sum times one of them may pass fp32's range where that does not)
        const float4* cs = reinterpret_cast<const float4*>(scale + c);
#pragma unroll
        for (int j = 0; j < CH; j += 4) {
          const float4 s4 = cs[j / 4];
          acc[c + j] = fmaf(__uint_as_float(r[j]), s4.x * f, acc[c + j]);
          acc[c + j + 1] = fmaf(__uint_as_float(r[j + 1]), s4.y * f, acc[c + j + 1]);
          acc[c + j + 2] = fmaf(__uint_as_float(r[j + 2]), s4.z * f, acc[c + j + 2]);
          acc[c + j + 3] = fmaf(__uint_as_float(r[j + 3]), s4.w * f, acc[c + j + 3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sce0 + 8 * slot);
    }
    // every MMA has read its stages (the last accumulator was waited for): the sums take their place
#pragma unroll
    for (int c = 0; c < BN; ++c) sums[c * Cf::SUM_LD + warp * 32 + lane] = acc[c];
  }

  // ------------------------------------------------------------------ the tile's sums to C
  __syncwarp();
  tc_fence_before();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  {
    // this CTA's share of the tile's rows of C
    const int o0 = BN * split / p.splits, o1 = BN * (split + 1) / p.splits;
    for (int e = threadIdx.x; e < (o1 - o0) * Cf::BM; e += kBlockThreads) {
      const int c = o0 + e / Cf::BM, r = e % Cf::BM;
      if (p0 + r >= p.p_rows || q0 + c >= p.q_rows) continue;
      const float v = joined_sum(sums, c * Cf::SUM_LD + r, p.splits);
      static_cast<__nv_bfloat16*>(p.g.C)[static_cast<long long>(q0 + c) * p.g.ldc + p0 + r] = __float2bfloat16_rn(v);
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
