// Products of E4M3 matrices with a scale for each block of 128 along K
// (gemm_e4m3_blocks), for sm_103a.
//
//   C[i][j] = sum over blocks b of sa[i][b] sb[j][b] (sum over k of block b of A[i][k] B[j][k])
//
// A stage of the pipeline is one block (128 bytes of K), so the tensor cores sum a
// block into an accumulator of its own in tensor memory, and the epilogue warps
// take it from there, scale it and add it to the tile's sums, which they hold in
// registers. Warps: 0-3 epilogue, 4 TMA producer, 5 tcgen05.mma, 6 the column
// scales (through a ring in shared memory).
//
// One CTA computes 128 rows of a "row operand" P against BN rows of a "column
// operand" Q. With many rows P is A and Q is B; with few (SWAP) P is B, so that
// 128 lanes are 128 columns of C and a narrow tile wastes nothing. Where the tiles
// do not fill the GPU a cluster of `splits` CTAs shares a tile: each takes a run of
// blocks, and they add their sums through distributed shared memory, in order.
#pragma once

#include "dgt_feedforward.h"
#include "gemm_kernel.cuh"

namespace dgt {

constexpr int kBlockK = 128;

// Scales of an operand: row r, block b at s[(r >> shift) * row + b * block].
struct BlockScales {
  const float* s;
  long long row, block;
  int shift;
  __device__ __forceinline__ float at(int r, int b) const { return __ldg(s + (r >> shift) * row + b * block); }
};

struct BlockParams {
  GemmParams g;  // C, ldc, num_kb, raster, tiles_m (of P), tiles_n (of Q) and the launch-wide status fields
  BlockScales ps, qs;
  int p_rows, q_rows;
  int splits;
};

constexpr int kBlockThreads = 256;
constexpr int kScaleRing = 4;

template <int BN_>
struct BlockCfg {
  static constexpr int BN = BN_;
  static constexpr int BM = 128;
  static constexpr int P_BYTES = BM * 128;
  static constexpr int Q_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int STAGES = BN >= 128 ? 3 : 5;  // two CTAs to an SM
  static constexpr int ACCS = BN >= 128 ? 2 : 4;    // accumulators in tensor memory
  static constexpr int TMEM_COLS = ACCS * BN < 64 ? 64 : ACCS * BN;
  static constexpr int SUM_LD = BM + 1;             // a column of the shared sums (free of bank conflicts either way)
  static constexpr int SCALE_BYTES = kScaleRing * BN * 4;
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + SCALE_BYTES + BAR_BYTES;
  static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128, "tile width");
  static_assert(BN * SUM_LD * 4 <= STAGES * STAGE_BYTES, "the sums reuse the stages");
  static_assert((2 * STAGES + 2 * ACCS + 1 + 2 * kScaleRing) * 8 + 16 <= BAR_BYTES, "barrier area");
  // D fp32, E4M3 operands, both K-major
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
};

// Loads BN_ (16 or 32) columns of the warp's 32 accumulator rows.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, r);
    tmem_wait_ld_into(r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// COLS: the column operand has a scale for each row of it, else one for the tile (its 128 rows' block).
template <int BN, bool COLS, bool SWAP>
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
      mbar_init(scf0 + 8 * i, 1);
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
        if (!warp_wait_phase(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) break;
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
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    const uint64_t p_desc = sdesc(sP, 16, 1024, SWZ_128B), q_desc = sdesc(sQ, 16, 1024, SWZ_128B);
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S, b = it % Cf::ACCS;
      if (!warp_wait_phase(p.g, acce0 + 8 * b, ((it / Cf::ACCS) & 1) ^ 1, ROLE_MMA | (0x80u << 8))) break;
      if (!warp_wait_phase(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8))) break;
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
  } else if (warp == 6) {
    // ---------------------------------------------------------------- column scales
    if constexpr (COLS) {
      // four blocks' scales ahead in registers, a lane has columns lane, lane + 32, ...
      constexpr int PER = (BN + 31) / 32;
      float next[kScaleRing][PER];
      auto load = [&](int kb) {
#pragma unroll
        for (int i = 0; i < kScaleRing; ++i)
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const int c = lane + 32 * j;
            next[i][j] = kb + i < kb1 && c < BN && q0 + c < p.q_rows ? p.qs.at(q0 + c, kb + i) : 0.0f;
          }
      };
      load(kb0);
      bool ok = true;
      for (int kb = kb0, round = 0; ok && kb < kb1; kb += kScaleRing, ++round) {
        float now[kScaleRing][PER];
#pragma unroll
        for (int i = 0; i < kScaleRing; ++i)
#pragma unroll
          for (int j = 0; j < PER; ++j) now[i][j] = next[i][j];
        load(kb + kScaleRing);
#pragma unroll
        for (int i = 0; i < kScaleRing; ++i) {
          if (!ok || kb + i >= kb1) break;
          ok = warp_wait_phase(p.g, sce0 + 8 * i, (round & 1) ^ 1, ROLE_COPY | (i << 8));
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (lane + 32 * j < BN) scales[i * BN + lane + 32 * j] = now[i][j];
          __syncwarp();
          if (lane == 0) mbar_arrive(scf0 + 8 * i);
        }
      }
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- epilogue: lane = row of P
    const int row = p0 + warp * 32 + lane;
    const int srow = min(row, p.p_rows - 1);
    constexpr int CH = BN < 32 ? BN : 32;
    float acc[BN];
#pragma unroll
    for (int c = 0; c < BN; ++c) acc[c] = 0.0f;
    float next[4];
    auto load = [&](int kb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        next[i] = kb + i < kb1 ? p.ps.at(srow, kb + i) : 0.0f;
        if (!COLS && kb + i < kb1) next[i] *= p.qs.at(q0, kb + i);
      }
    };
    load(kb0);
    bool ok = true;
    for (int kb = kb0; ok && kb < kb1; kb += 4) {
      float now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = next[i];
      load(kb + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kb + i >= kb1) break;
        const int it = kb + i - kb0, b = it % Cf::ACCS;
        if (COLS) {
          ok = warp_wait_phase(p.g, scf0 + 8 * i, (it / kScaleRing) & 1, ROLE_EPILOGUE | (0x90u << 8));
          if (!ok) break;
        }
        ok = warp_wait_phase(p.g, accf0 + 8 * b, (it / Cf::ACCS) & 1, ROLE_EPILOGUE | (b << 8));
        if (!ok) break;
        tc_fence_after();
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
          if constexpr (COLS) {
            const float4* cs = reinterpret_cast<const float4*>(scales + i * BN + c);
#pragma unroll
            for (int j = 0; j < CH; j += 4) {
              const float4 f = cs[j / 4];
              acc[c + j] = fmaf(__uint_as_float(r[j]) * f.x, now[i], acc[c + j]);
              acc[c + j + 1] = fmaf(__uint_as_float(r[j + 1]) * f.y, now[i], acc[c + j + 1]);
              acc[c + j + 2] = fmaf(__uint_as_float(r[j + 2]) * f.z, now[i], acc[c + j + 2]);
              acc[c + j + 3] = fmaf(__uint_as_float(r[j + 3]) * f.w, now[i], acc[c + j + 3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < CH; ++j) acc[c + j] = fmaf(__uint_as_float(r[j]), now[i], acc[c + j]);
          }
        }
        if (COLS) {
          __syncwarp();
          if (lane == 0) mbar_arrive(sce0 + 8 * i);
        }
      }
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
    // this CTA's share: columns of the tile (SWAP: C's rows), or rows of it
    const uint32_t local = smem_u32(sums);
    const int outer = SWAP ? BN : Cf::BM, inner = SWAP ? Cf::BM : BN;
    const int o0 = outer * split / p.splits, o1 = outer * (split + 1) / p.splits;
    for (int e = threadIdx.x; e < (o1 - o0) * inner; e += kBlockThreads) {
      const int o = o0 + e / inner, i = e % inner;
      const int r = SWAP ? i : o, c = SWAP ? o : i;
      if (p0 + r >= p.p_rows || q0 + c >= p.q_rows) continue;
      const uint32_t at = static_cast<uint32_t>((c * Cf::SUM_LD + r) * 4);
      float v;
      if (p.splits == 1) {
        v = sums[c * Cf::SUM_LD + r];
      } else {
        v = 0.0f;
        for (int z = 0; z < p.splits; ++z) v += ld_cluster_f32(mapa_shared(local + at, z));
      }
      const long long crow = SWAP ? q0 + c : p0 + r, ccol = SWAP ? p0 + r : q0 + c;
      static_cast<__nv_bfloat16*>(p.g.C)[crow * p.g.ldc + ccol] = __float2bfloat16_rn(v);
    }
  }
  grid_launch_dependents();

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
