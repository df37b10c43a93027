// The products with a scale for each block of 128 (block_few.cuh) on CTA pairs,
// for matrices that fill the GPU with 256-row tiles.
//
// A pair (cta_group::2) computes 256 x BN, each CTA 128 rows of it; persistent, a
// static share of the tiles in bands. The tensor cores need 2 BN cycles for a block
// of 128 x BN x 128; in that time the eight epilogue warps have to take the
// accumulators out of tensor memory (128 BN fp32 values, 512 bytes a cycle: BN
// cycles) and add them up (BN / 2 instructions of two values for each warp, two
// warps to a scheduler). So the sums are held two to a register pair, a load is in
// flight while the one before it is added, the accumulator is handed back as soon
// as its last load has landed, and the epilogue warps have most of the register
// file (setmaxnreg): 128 sums a thread stay in registers. The scales come through
// shared memory, copied by warps of their own some blocks ahead. COLS (a scale for
// each row of the column operand) has two instructions for one, the product of a
// value's scales and the addition. 8192^3: 357-364 us (3.0 PFLOP/s; 422 at the power
// limit), COLS 530 (500 with the sum times one scale first, which passes fp32's range
// where the two scales are far apart); 128 x 8192 x 8192, half of each tile empty, 23.7.
// Cycles a block of a 256-wide tile (128-wide), at 2070 MHz: 690-730 (490-500), COLS
// 1180 (650), and with an epilogue that waits and hands back but reads nothing 546
// (455), which is what loads of 24 and 32 KB a block and CTA allow. The rest is the
// epilogue, and of it no one unit is full: COLS of 256 columns has 46% of the issue
// slots, 23% of the FMA pipe, 42% of the shared-memory data pipe (every lane reads
// every column's scale: two wavefronts an LDS.128) and 42% of the tensor pipe.
#pragma once

#include "block_few.cuh"
#include "group_kernel.cuh"

namespace dgt {

constexpr int kPairThreads = 384;  // warps 0-3 and 8-11 epilogue, 4 producer, 5 MMA, 6 column scales, 7 row scales

template <int BN_>
struct BlockPairCfg {
  static constexpr int BN = BN_;
  static constexpr int BM = 128;        // rows of a CTA
  static constexpr int BNH = BN / 2;    // rows of the column operand a CTA loads
  static constexpr int P_BYTES = BM * 128;
  static constexpr int Q_BYTES = BNH * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int ACCS = 512 / BN;
  static constexpr int TMEM_COLS = 512;
  static constexpr int EPI_TILE = 32 * 128;
  static constexpr int EPI_STAGING = 8 * EPI_TILE;
  // a block's scales: of the 128 rows, then of the columns (COLS) or of each 128 of them
  static constexpr int SCALE_RING = 8;
  static constexpr int SCALES = BM + BN;
  static constexpr int SCALE_BYTES = SCALE_RING * SCALES * 4;
  static constexpr int BAR_BYTES = 512;
  static constexpr int SMEM_LIMIT = 232448;
  static constexpr int STAGES_FIT = (SMEM_LIMIT - 1024 - EPI_STAGING - SCALE_BYTES - BAR_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_STAGING + SCALE_BYTES + BAR_BYTES;
  static constexpr int COLS_PER_SET = BN / 2;  // columns of an epilogue warp
  static constexpr int BLOCKS = BN / 128;      // scales of the column operand without COLS
  static_assert(BN == 256 || BN == 128, "tile width");
  static_assert((2 * STAGES + 2 * ACCS + 2 * SCALE_RING + 1) * 8 + 16 <= BAR_BYTES, "barrier area");
  static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(2 * BM >> 4) << 24);
};

// Registers: 384 threads are launched with 168 each (64512); the epilogue's 256 take 216, the others keep 72.
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Arrives on an mbarrier of the cluster without publishing anything: what it hands
// over is tensor memory that this thread has finished reading (tcgen05.wait::ld).
// (The releasing form waits for the thread's memory operations, about 1000 cycles
// for every block: 8192^3 took 1144 us with it.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier (one of its expected count) once this thread's copies so far have landed.
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A wait of each lane by itself: the warp agrees on the outcome now and then (a vote at each wait held back what it
// releases: 8192^3 364 us, COLS 522, and 360 and 500 without, when the sum met one scale first).
__device__ __forceinline__ bool lane_wait(const GemmParams& g, uint32_t bar, uint32_t parity, uint32_t code) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_phase(g, bar, parity, code);
}

template <int BN, bool COLS>
__global__ void __launch_bounds__(kPairThreads, 1)
    block_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmC, const __grid_constant__ BlockParams p) {
  using Cf = BlockPairCfg<BN>;
  constexpr int S = Cf::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - raw);
  const uint32_t sP = sbase, sQ = sbase + S * Cf::P_BYTES, sE = sbase + S * Cf::STAGE_BYTES;
  float* scales = reinterpret_cast<float*>(sptr + S * Cf::STAGE_BYTES + Cf::EPI_STAGING);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sptr + S * Cf::STAGE_BYTES + Cf::EPI_STAGING + Cf::SCALE_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * S;
  const uint32_t accf0 = empty0 + 8 * S;
  const uint32_t acce0 = accf0 + 8 * Cf::ACCS;
  const uint32_t scf0 = acce0 + 8 * Cf::ACCS;  // a block's scales have landed
  const uint32_t sce0 = scf0 + 8 * Cf::SCALE_RING;  // this CTA's epilogue has read them
  const uint32_t drain_bar = sce0 + 8 * Cf::SCALE_RING;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sptr + (drain_bar + 8 - sbase));
  volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot) + 1;
  volatile int* consumed_slot = issued_slot + 1;

  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const bool leader = half == 0;
  const int unit = blockIdx.x / 2, nunits = gridDim.x / 2;
  const int tiles = p.g.tiles_m * p.g.tiles_n, kbs = p.g.num_kb;
  auto place = [&](int t, int& p0, int& q0) {
    int mb, nb;
    const int band = p.g.raster * p.g.tiles_n, b = t / band, first = b * p.g.raster;
    const int rows = min(p.g.raster, p.g.tiles_m - first), q = t - b * band;
    nb = q / rows;
    mb = first + (q - nb * rows);
    p0 = mb * 2 * Cf::BM + int(half) * Cf::BM;
    q0 = nb * BN;
  };

  if (warp == 4 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < Cf::ACCS; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 16);
    }
    for (int b = 0; b < Cf::SCALE_RING; ++b) {
      mbar_init(scf0 + 8 * b, COLS ? 64 : 32);
      mbar_init(sce0 + 8 * b, 8);
    }
    mbar_init(drain_bar, 1);
    *issued_slot = 0;
    *consumed_slot = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 5) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), Cf::TMEM_COLS);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));

  if (warp >= 4 && warp < 8) {
    registers_down<72>();
    if (warp == 4) {
      // -------------------------------------------------------------- TMA producer (each CTA)
      if (!(p.g.debug & DEBUG_STALL_PRODUCER)) {
        const uint32_t lead_full0 = mapa_shared(full0, 0);
        int it = 0;
        bool ok = true;
        for (int t = unit; ok && t < tiles; t += nunits) {
          int p0, q0;
          place(t, p0, q0);
          for (int kb = 0; kb < kbs; ++kb, ++it) {
            const int s = it % S;
            if (!group_wait(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) {
              ok = false;
              break;
            }
            if (elect_one()) {
              if (leader) mbar_arrive_expect_tx(full0 + 8 * s, 2 * Cf::STAGE_BYTES);
              tma_load_3d_pair(sP + s * Cf::P_BYTES, &tmP, lead_full0 + 8 * s, kb * kBlockK, p0, 0);
              tma_load_3d_pair(sQ + s * Cf::Q_BYTES, &tmQ, lead_full0 + 8 * s, kb * kBlockK, q0 + int(half) * Cf::BNH, 0);
            }
            __syncwarp();
          }
        }
        if (lane == 0) *issued_slot = it;
      }
      grid_launch_dependents();
    } else if (warp == 5 && leader) {
      // -------------------------------------------------------------- MMA issuer (the pair's leader)
      const uint64_t p_desc = sdesc(sP, 16, 1024, SWZ_128B), q_desc = sdesc(sQ, 16, 1024, SWZ_128B);
      int it = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += nunits) {
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int s = it % S, b = it % Cf::ACCS;
          if (!group_wait(p.g, acce0 + 8 * b, ((it / Cf::ACCS) & 1) ^ 1, ROLE_MMA | (0x80u << 8)) ||
              !group_wait(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ps = p_desc + static_cast<uint32_t>(s) * (Cf::P_BYTES / 16);
          const uint64_t qs = q_desc + static_cast<uint32_t>(s) * (Cf::Q_BYTES / 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8f6f4_pair(tmem + b * BN, ps + kk * 2, qs + kk * 2, Cf::IDESC, kk > 0 ? 1u : 0u);
            mma_commit_pair(accf0 + 8 * b, uint16_t(0x3u));
            mma_commit_pair(empty0 + 8 * s, uint16_t(0x3u));
          }
          __syncwarp();
        }
      }
      if (lane == 0) *consumed_slot = it;
      if (elect_one()) mma_commit_pair(drain_bar, uint16_t(1u));
      __syncwarp();
      if (lane == 0) wait_phase_drain(p.g, drain_bar, 0);
      __syncwarp();
    } else if (warp == 7 || (warp == 6 && COLS)) {
      // -------------------------------------------------------------- scales (each CTA)
      // Copied by each lane (entries lane, lane + 32, ...), up to SCALE_RING blocks ahead. (With two blocks ahead
      // in registers their latency held COLS back: 8192^3 579 us, 522 with the copies.)
      const bool rows = warp == 7;
      const uint32_t to0 = smem_u32(scales) + 4 * lane;
      int it = 0;
      bool ok = true;
      for (int t = unit; ok && t < tiles; t += nunits) {
        int p0, q0;
        place(t, p0, q0);
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          const int b = it % Cf::SCALE_RING;
          if (!group_wait(p.g, sce0 + 8 * b, ((it / Cf::SCALE_RING) & 1) ^ 1, ROLE_COPY | (b << 8))) {
            ok = false;
            break;
          }
          const uint32_t to = to0 + b * Cf::SCALES * 4;
          if (rows) {
#pragma unroll
            for (int j = 0; j < 4; ++j) copy4(to + 128 * j, p.ps.from(min(p0 + lane + 32 * j, p.p_rows - 1), kb));
            if (!COLS && lane < Cf::BLOCKS) copy4(to + 512, p.qs.from(min(q0 + 128 * lane, p.q_rows - 1), kb));
          } else {
#pragma unroll
            for (int j = 0; j < BN / 32; ++j) copy4(to + 512 + 128 * j, p.qs.from(min(q0 + lane + 32 * j, p.q_rows - 1), kb));
          }
          mbar_arrive_copies(scf0 + 8 * b);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---------------------------------------------------------------- epilogue: lane = row of P
    registers_up<216>();
    constexpr int NC = Cf::COLS_PER_SET;
    const int q = warp & 3, set = warp >> 3;
    const uint32_t stage = sE + static_cast<uint32_t>((set * 4 + q) * Cf::EPI_TILE);
    const uint32_t lead_acce0 = mapa_shared(acce0, 0);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + set * NC;
    const GroupOut out = {static_cast<uint16_t*>(p.g.C), p.g.ldc, 0, p.g.c_tma, p.g.c_gran, p.q_rows, 0};
    int it = 0;
    bool ok = true;
    for (int t = unit; ok && t < tiles; t += nunits) {
      int p0, q0;
      place(t, p0, q0);
      const int row0 = p0 + q * 32, col0 = q0 + set * NC;
      float2 acc[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
      for (int kb = 0; kb < kbs; ++kb, ++it) {
        const int b = it % Cf::ACCS, sb = it % Cf::SCALE_RING;
        if (!lane_wait(p.g, scf0 + 8 * sb, (it / Cf::SCALE_RING) & 1, ROLE_EPILOGUE | (sb << 8))) ok = false;
        if (!lane_wait(p.g, accf0 + 8 * b, (it / Cf::ACCS) & 1, ROLE_EPILOGUE | (b << 8))) ok = false;
        tc_fence_after();
        const uint32_t from = taddr + b * BN;
        __syncwarp();
        // the next CH columns are on their way while these are added
        constexpr int CH = 32;
        uint32_t r[2][CH];
        tmem_ld_32x32b_x32(from, r[0]);
        const float* scale = scales + sb * Cf::SCALES;
        const float f1 = COLS ? scale[q * 32 + lane] : scale[q * 32 + lane] * scale[Cf::BM + (set * NC) / 128];
        const float2 f = make_float2(f1, f1);
#pragma unroll
        for (int c = 0; c < NC / CH; ++c) {
          tmem_wait_ld_into(r[c & 1]);
          if (c + 1 < NC / CH) {
            tmem_ld_32x32b_x32(from + CH * (c + 1), r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(lead_acce0 + 8 * b);
          }
          const float4* cs = reinterpret_cast<const float4*>(scale + Cf::BM + set * NC + CH * c);
#pragma unroll
          for (int j = 0; j < CH / 2; j += 2) {
            const float2 x = make_float2(__uint_as_float(r[c & 1][2 * j]), __uint_as_float(r[c & 1][2 * j + 1]));
            const float2 y = make_float2(__uint_as_float(r[c & 1][2 * j + 2]), __uint_as_float(r[c & 1][2 * j + 3]));
            // COLS: the scales' product first (a block's sum times one of them may pass fp32's range where that does not)
            float2 fx = f, fy = f;
            if constexpr (COLS) {
              const float4 s4 = cs[j / 2];
              fx = __fmul2_rn(f, make_float2(s4.x, s4.y));
              fy = __fmul2_rn(f, make_float2(s4.z, s4.w));
            }
            acc[CH / 2 * c + j] = __ffma2_rn(x, fx, acc[CH / 2 * c + j]);
            acc[CH / 2 * c + j + 1] = __ffma2_rn(y, fy, acc[CH / 2 * c + j + 1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sce0 + 8 * sb);
        if (kb % 64 == 63 && !__all_sync(0xFFFFFFFFu, ok)) break;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (row0 < p.p_rows) {
#pragma unroll
        for (int c = 0; c < NC; c += 64) {
          if (col0 + c < p.q_rows) {
            // the tile's last TMA store has read it
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 v = acc[c / 2 + 4 * j + k];
                w[k] = pack2<KIND_BF16>(__float_as_uint(v.x), __float_as_uint(v.y));
              }
              st_shared_v4(stage_chunk(stage, lane, j), w[0], w[1], w[2], w[3]);
            }
            group_flush<true>(out, &tmC, stage, lane, row0, p.p_rows, col0 + c, 0);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }

  // ------------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // loads issued but not consumed exist only when the launch was aborted: let them land
  if (leader && threadIdx.x == 0 && *consumed_slot < *issued_slot) {
    const int issued = *issued_slot;
    for (int j = *consumed_slot; j < issued; ++j)
      if (!wait_phase_drain(p.g, full0 + 8 * (j % S), (j / S) & 1)) break;
  }
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, Cf::TMEM_COLS);
  }
}

}  // namespace dgt
