// Persistent grouped GEMM for sm_103a: every expert's rows times that
// expert's weights in one launch, and the weights' gradient.
//
// The mathematics (contraction in fp32, one rounding at the end):
//   product   C[s] = epilogue(A[row(s)] . W_e)          for s in group e
//   gradient  dW_e = sum over s in group e of P[s]^T Q[s] (P, Q: dC and A, or A and dC)
//
// It is the dense kernel's pipeline -- a TMA producer warp, one thread that
// issues tcgen05.mma, four epilogue warps per CTA, fp32 accumulators double
// buffered in tensor memory -- with the three things a ragged group needs:
//
//   * Tiles come from the offsets on the device. Each CTA scans the groups'
//     row-tile counts into shared memory once (one thread per few groups) and
//     finds a work item's group by binary search, so the host never reads the
//     group sizes and empty groups cost nothing but their table entry.
//   * Rows in slot order come by TMA boxes. Rows that the caller names are
//     gathered by TMA (tile::gather4: four rows of 128 bytes an instruction,
//     each lane of the producer warp issues one) where a group has few: an
//     instruction costs about 75 cycles, so 128 rows of a slab take 2400, four
//     times the MMA's 512, but a handful hides behind the weights' stream. For
//     large groups the host first permutes the rows into the stream's scratch
//     (one bandwidth-bound pass) and they are rows in slot order again. A group's
//     last tile fetches only the rows it has.
//   * The gradient contracts over a ragged number of rows. A group's last slab
//     of 64 rows may run into the next group's rows; its loads complete on a
//     barrier of their own, a sixth warp clears the rows past the end in shared
//     memory (both operands: an infinity or NaN of another group times zero
//     would be a NaN), and only then may the MMA read the stage.
//
// PAIR: a CTA pair (cta_group::2) computes a 256 x BN tile, each CTA loading
// 128 rows of A and half of the B columns; else one CTA computes 128 x BN.
// GATED: W's columns are gate and value halves; a tile holds the same BN / 2
// columns of both (in the pair each CTA loads one of them), and the epilogue
// stores silu(gate) * value, so the 2 x wider intermediate is never written.
#pragma once

#include "gemm_kernel.cuh"

namespace dgt {

// Four rows y0..y3 of a 2-D tensor, 128 bytes of each from column x, to 512
// consecutive bytes of (swizzled) shared memory.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y0,
                                            int32_t y1, int32_t y2, int32_t y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3)
      : "memory");
}
// The same, its completion signalled on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const void* tmap, uint32_t bar_cluster, int32_t x,
                                                 int32_t y0, int32_t y1, int32_t y2, int32_t y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3)
      : "memory");
}

constexpr int kMaxGroups = 1024;

// Operand arrangements.
enum : int {
  GROUP_W_MN = 0,   // product, W row-major (K x N): the MMA's B operand is MN-major
  GROUP_W_K = 1,    // product, W given as N x K: K-major
  GROUP_WGRAD = 2,  // weight gradient: both operands MN-major (rows of the contraction are slots)
};

struct GroupParams {
  // N, K, C, ldc, stride_c, c_tma, c_gran, num_kb, raster, tiles_m, tiles_n, alpha, act, bias and the launch-wide
  // status fields are used; N is the width of the accumulators' matrix (both halves of a gated product).
  GemmParams g;
  const int* offsets;
  int groups;
  int slots;
  const int* rows;  // row of the gathered operand for each slot, or null: the slot itself
  int a_rows;
  const float* row_scale;
  const float* col_scale;
  int gather_a;  // product: rows of A by gather (else boxes by slot)
  int plain;     // the epilogue is the identity
  int out_cols;  // columns of C (or of dW)
  int out_rows;  // gradient: rows of dW
  int gather_p, gather_q;  // gradient: the operand whose rows are gathered by TMA (else boxes by slot)
};

template <int KIND, int OPS, int BN_, bool PAIR, bool GATED>
struct GroupCfg {
  using T = typename KindTraits<KIND>::T;
  static constexpr int ES = sizeof(T);
  static constexpr bool WGRAD = OPS == GROUP_WGRAD;
  static constexpr bool B_KMAJOR = OPS == GROUP_W_K;
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int BM = 128;           // accumulator rows per CTA
  static constexpr int BMT = BM * CTAS;    // per tile
  static constexpr int BN = BN_;           // accumulator columns of a tile
  static constexpr int BNH = BN / CTAS;    // B columns per CTA
  static constexpr int OUT_BN = GATED ? BN / 2 : BN;  // columns of C per tile
  static constexpr int BK = 128 / ES;      // contraction elements of a stage (K-major: 128 bytes; MN-major: rows)
  static constexpr int UK = 32 / ES;
  static constexpr int KSTEPS = BK / UK;
  static constexpr int BOXN = 128 / ES;
  static constexpr int BOX_BYTES = BK * 128;
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BNH * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SMEM_LIMIT = 232448;
  static constexpr int BAR_BYTES = 512;
  static constexpr int TABLE_BYTES = WGRAD ? 0 : ((kMaxGroups + 2) * 4 + 127) / 128 * 128;
  static constexpr int FIXED = 1024 /*align slack*/ + BAR_BYTES + TABLE_BYTES;
  static constexpr int STAGES_FIT = (SMEM_LIMIT - FIXED - EPI_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int EPI_BUFS = epi_bufs_for(SMEM_LIMIT, FIXED + STAGES * STAGE_BYTES);
  static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE_BYTES + EPI_BUFS * EPI_BYTES;
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
  static constexpr int NUM_BARS = 4 * STAGES + 5;
  static constexpr int THREADS = WGRAD ? 224 : 192;
  static constexpr int A_BOX_ROWS = PAIR ? 128 : 32;  // rows of A per box: one CTA's tile may hold few
  static_assert(BN % 64 == 0 && BN >= 64 && BN <= 256, "tile width");
  static_assert(B_KMAJOR || ES == 2, "8-bit operands are read K-major");
  static_assert(B_KMAJOR || BNH % BOXN == 0, "MN-major B comes in whole boxes");
  static_assert(!GATED || B_KMAJOR || PAIR || (BN / 2) % BOXN == 0, "each half is whole boxes");
  static_assert(NUM_BARS * 8 + 64 <= BAR_BYTES, "barrier area");
  static_assert(STAGES >= 4 && SMEM_BYTES <= SMEM_LIMIT, "shared memory");
  static constexpr uint32_t IDESC = (1u << 4) | (KindTraits<KIND>::fmt << 7) | (KindTraits<KIND>::fmt << 10) |
                                    ((WGRAD ? 1u : 0u) << 15) | ((B_KMAJOR ? 0u : 1u) << 16) |
                                    (uint32_t(BN >> 3) << 17) | (uint32_t(BMT >> 4) << 24);
};

// A work item: group, first accumulator row and the rows' end (slots of the
// product, rows of dW for the gradient), tile column, slots of the group
// [begin, end) and k-slabs.
struct GroupTile {
  int e, m0, row_end, nb, begin, end, kbs;
};

// Start of group e (its end is the start of the next one); the numbers come
// from device memory, so they are kept inside [0, slots].
__device__ __forceinline__ int group_start(const GroupParams& p, int e) {
  if (e <= 0) return 0;
  return min(max(p.offsets[e], 0), p.slots);
}

// Place `r` of a group's tiles_m x tiles_n tiles, taken in bands of `raster`
// tile rows: down the band's rows, then across.
__device__ __forceinline__ void band_place(int r, int raster, int tiles_m, int tiles_n, int& mb, int& nb) {
  const int band = raster * tiles_n;
  const int b = r / band;
  const int first = b * raster;
  const int rows = min(raster, tiles_m - first);
  const int q = r - b * band;
  nb = q / rows;
  mb = first + (q - nb * rows);
}

template <class Cf>
__device__ __forceinline__ GroupTile group_tile(const GroupParams& p, const int* cum, int w) {
  GroupTile t;
  int mb;
  if constexpr (Cf::WGRAD) {
    const int per = p.g.tiles_m * p.g.tiles_n;
    t.e = w / per;
    band_place(w - t.e * per, p.g.raster, p.g.tiles_m, p.g.tiles_n, mb, t.nb);
    t.begin = group_start(p, t.e);
    t.end = max(t.begin, group_start(p, t.e + 1));
    t.m0 = mb * Cf::BMT;
    t.row_end = p.out_rows;
    t.kbs = (t.end - t.begin + Cf::BK - 1) / Cf::BK;
  } else {
    const int q = w / p.g.tiles_n;
    int lo = 0, hi = p.groups;  // the last group with cum <= q (group `groups`: the slots past the last group)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= q) lo = mid;
      else hi = mid - 1;
    }
    t.e = lo;
    band_place(w - cum[lo] * p.g.tiles_n, p.g.raster, cum[lo + 1] - cum[lo], p.g.tiles_n, mb, t.nb);
    t.begin = group_start(p, lo);
    t.end = lo < p.groups ? max(t.begin, group_start(p, lo + 1)) : p.slots;
    t.m0 = t.begin + mb * Cf::BMT;
    t.row_end = t.end;
    t.kbs = lo < p.groups ? p.g.num_kb : 0;
  }
  return t;
}

// Row of the gathered operand for slot s of a group [begin, end): slots past
// the end repeat the last one, so every address is a row of this group.
__device__ __forceinline__ int gathered_row(const GroupParams& p, int s, int end) {
  s = min(s, end - 1);
  const int r = p.rows != nullptr ? p.rows[s] : s;
  return min(max(r, 0), p.a_rows - 1);
}

// Writes the staged 32 x 64-byte tile to C[row0 .., col0 ..] of matrix z:
// rows before row_end and columns before p.out_cols only. TMA stores whole
// 32-row pieces (it clips at the tensor's end, not at a group's, so a piece
// that crosses the group's end is stored row by row).
template <bool CLIP>
__device__ __forceinline__ void group_flush(const GroupParams& p, const CUtensorMap* tmC, uint32_t stage, int lane,
                                            int row0, int row_end, int col0, int z) {
  const bool full_cols = col0 + 32 <= p.out_cols;
  if (p.g.c_tma && full_cols && (CLIP ? row0 < row_end : row0 + 32 <= row_end)) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(tmC, stage, col0, row0, z);
      bulk_commit_group();
    }
    return;
  }
  __syncwarp();
  uint16_t* base = static_cast<uint16_t*>(p.g.C) + z * p.g.stride_c + col0;
  if (p.g.c_gran >= 8 && full_cols) {
    const int l = lane & 7;
#pragma unroll
    for (int rr = 0; rr < 32; rr += 4) {
      const int r = rr + (lane >> 3);
      uint32_t lo, hi;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(lo), "=r"(hi)
                   : "r"(epi_chunk_addr(stage, r, l >> 1) + ((l & 1) << 3))
                   : "memory");
      if (row0 + r < row_end)
        *reinterpret_cast<uint2*>(base + static_cast<long long>(row0 + r) * p.g.ldc + l * 4) = make_uint2(lo, hi);
    }
  } else {
    const int l = lane & 15, col = col0 + 2 * l;
#pragma unroll 4
    for (int rr = 0; rr < 32; rr += 2) {
      const int r = rr + (lane >> 4);
      const uint32_t v = ld_shared_u32(epi_chunk_addr(stage, r, l >> 2) + ((l & 3) << 2));
      if (row0 + r < row_end && col < p.out_cols) {
        uint16_t* dst = base + static_cast<long long>(row0 + r) * p.g.ldc + 2 * l;
        if (p.g.c_gran >= 4 && col + 1 < p.out_cols) {
          *reinterpret_cast<uint32_t*>(dst) = v;
        } else {
          dst[0] = static_cast<uint16_t>(v & 0xFFFFu);
          if (col + 1 < p.out_cols) dst[1] = static_cast<uint16_t>(v >> 16);
        }
      }
    }
  }
  __syncwarp();
}

// The scaled and biased pre-activation of 32 accumulator columns from
// column `col` of group e: v = scale * col_scale[col] * acc + bias[col]. Each
// lane loads one column's scale and bias; shuffles hand them to every lane.
template <int KIND>
__device__ __forceinline__ void group_scale(const GroupParams& p, int e, int col, int lane, float scale,
                                            const uint32_t (&r)[32], float (&v)[32]) {
  const long long at = static_cast<long long>(e) * p.g.N + col + lane;
  const bool in = col + lane < p.g.N;
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = scale * __uint_as_float(r[k]);
  if (p.col_scale != nullptr) {
    const float c = in ? p.col_scale[at] : 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] *= __shfl_sync(0xFFFFFFFFu, c, k);
  }
  if (p.g.bias != nullptr) {
    float b = 0.0f;
    if (in) {
      if constexpr (KindTraits<KIND>::out == KIND_F16)
        b = __half2float(static_cast<const __half*>(p.g.bias)[at]);
      else
        b = __bfloat162float(static_cast<const __nv_bfloat16*>(p.g.bias)[at]);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] += __shfl_sync(0xFFFFFFFFu, b, k);
  }
}

template <int KIND, int OPS, int BN, bool PAIR, bool GATED>
__global__ void __launch_bounds__(224, 1)
    group_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAg,
                 const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmBg,
                 const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GroupParams p) {
  using Cf = GroupCfg<KIND, OPS, BN, PAIR, GATED>;
  constexpr int S = Cf::STAGES;
  constexpr bool WGRAD = Cf::WGRAD;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sptr = smem_raw + (sbase - raw);
  const uint32_t sA = sbase;
  const uint32_t sB = sbase + S * Cf::A_BYTES;
  const uint32_t sE = sbase + S * Cf::STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sptr + S * Cf::STAGE_BYTES + Cf::EPI_BUFS * EPI_BYTES);
  int* cum = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + Cf::BAR_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * S;
  const uint32_t accf0 = empty0 + 8 * S;
  const uint32_t acce0 = accf0 + 16;
  const uint32_t drain_bar = acce0 + 16;
  const uint32_t tailf0 = drain_bar + 8;   // gradient: a stage's ragged slab has landed in this CTA
  const uint32_t tailok0 = tailf0 + 8 * S; // gradient (leader): both CTAs have cleared its rows past the end
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(bars + Cf::NUM_BARS);
  volatile int* issued_slot = reinterpret_cast<volatile int*>(bars + Cf::NUM_BARS) + 1;
  volatile int* consumed_slot = issued_slot + 1;
  volatile int* ok_slot = issued_slot + 2;    // [2]
  volatile int* tail_slot = issued_slot + 4;  // ragged slabs issued, and seen landed
  int* warp_sums = reinterpret_cast<int*>(bars + Cf::NUM_BARS) + 8;  // [8]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t half = PAIR ? cluster_ctarank() : 0u;
  const bool leader = half == 0;
  const int unit = blockIdx.x / Cf::CTAS;
  const int nunits = gridDim.x / Cf::CTAS;

  if (warp == 4 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(tailf0 + 8 * s, 1);
      mbar_init(tailok0 + 8 * s, Cf::CTAS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 4 * Cf::CTAS);
    }
    mbar_init(drain_bar, 1);
    *issued_slot = 0;
    *consumed_slot = 0;
    tail_slot[0] = 0;
    tail_slot[1] = 0;
    fence_mbar_init();
    if (!WGRAD && p.g.num_kb > 0) {
      tma_prefetch_desc(p.gather_a ? &tmAg : &tmA);
      tma_prefetch_desc(&tmB);
    }
  }
  if (warp == 5) {
    const uint32_t slot = smem_u32(const_cast<uint32_t*>(tmem_slot));
    if constexpr (PAIR) {
      tmem_alloc_pair(slot, Cf::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(slot, Cf::TMEM_COLS);
      tmem_relinquish();
    }
  }
  // set-up done; from here on memory that earlier kernels wrote is read
  grid_dependency_wait();
  if constexpr (!WGRAD) {
    // row tiles of each group, and of the slots past the last one, summed in group order
    const int n = p.groups + 1;
    const int per = (n + Cf::THREADS - 1) / Cf::THREADS;  // at most 6
    const int e0 = threadIdx.x * per;
    int cnt[6];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int e = e0 + i;
      cnt[i] = 0;
      if (i < per && e < n) {
        const int b = group_start(p, e);
        const int z = e < p.groups ? group_start(p, e + 1) : p.slots;
        cnt[i] = z > b ? (z - b + Cf::BMT - 1) / Cf::BMT : 0;
      }
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      if (i < per && e0 + i < n) cum[e0 + i] = at;
      at += cnt[i];
    }
    if (threadIdx.x == Cf::THREADS - 1) cum[n] = at;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // barriers of both CTAs initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int work = WGRAD ? p.groups * p.g.tiles_m * p.g.tiles_n : cum[p.groups + 1] * p.g.tiles_n;

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA producer (every CTA)
    if (!(p.g.debug & DEBUG_STALL_PRODUCER)) {
      int it = 0, tails = 0;
      bool ok = true;
      const uint32_t lead_full0 = PAIR ? mapa_shared(full0, 0) : full0;
      for (int w = unit; ok && w < work; w += nunits) {
        const GroupTile t = group_tile<Cf>(p, cum, w);
        int r0 = 0, r1 = 0, r2 = 0, r3 = 0;  // product: this lane's four rows of A
        int pieces = 0, tx = 0;
        if constexpr (!WGRAD) {
          if (t.kbs == 0) continue;
          const int first = t.m0 + int(half) * Cf::BM;
          const int left = t.end - first;
          // pieces of A this CTA loads: quads of gathered rows, or boxes
          const int rows_per = p.gather_a ? 4 : Cf::A_BOX_ROWS;
          auto count = [&](int rows) { return (min(max(rows, 0), Cf::BM) + rows_per - 1) / rows_per; };
          pieces = count(left);
          tx = pieces * rows_per * 128 + Cf::B_BYTES;
          if (PAIR && leader) tx += count(left - Cf::BM) * rows_per * 128 + Cf::B_BYTES;
          if (p.gather_a && lane < pieces) {
            const int s = first + 4 * lane;
            r0 = gathered_row(p, s, t.end);
            r1 = gathered_row(p, s + 1, t.end);
            r2 = gathered_row(p, s + 2, t.end);
            r3 = gathered_row(p, s + 3, t.end);
          }
        }
        for (int kb = 0; kb < t.kbs; ++kb, ++it) {
          const int s = it % S;
          if (!warp_wait_phase(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) {
            ok = false;
            break;
          }
          const uint32_t a_dst = sA + s * Cf::A_BYTES;
          const uint32_t b_dst = sB + s * Cf::B_BYTES;
          uint32_t fb = lead_full0 + 8 * s;
          if constexpr (!WGRAD) {
            // (operands of the elected lane's loads are the same in every lane: the issue path wants them so)
            const int row0 = t.m0 + int(half) * Cf::BM;
            if (elect_one()) {
              if (leader) mbar_arrive_expect_tx(full0 + 8 * s, tx);
              const int x = kb * Cf::BK;
              if (!p.gather_a) {
#pragma unroll
                for (int j = 0; j < Cf::BM / Cf::A_BOX_ROWS; ++j)
                  if (j < pieces) {
                    if constexpr (PAIR)
                      tma_load_3d_pair(a_dst + j * Cf::A_BOX_ROWS * 128, &tmA, fb, x, row0 + j * Cf::A_BOX_ROWS, 0);
                    else
                      tma_load_3d(a_dst + j * Cf::A_BOX_ROWS * 128, &tmA, fb, x, row0 + j * Cf::A_BOX_ROWS, 0);
                  }
              }
              if constexpr (Cf::B_KMAJOR) {
                if constexpr (PAIR) {
                  const int n0 = GATED ? int(half) * (p.g.N / 2) + t.nb * Cf::OUT_BN : t.nb * BN + int(half) * Cf::BNH;
                  tma_load_3d_pair(b_dst, &tmB, fb, x, n0, t.e);
                } else if constexpr (GATED) {
                  tma_load_3d(b_dst, &tmB, fb, x, t.nb * Cf::OUT_BN, t.e);
                  tma_load_3d(b_dst + Cf::B_BYTES / 2, &tmB, fb, x, p.g.N / 2 + t.nb * Cf::OUT_BN, t.e);
                } else {
                  tma_load_3d(b_dst, &tmB, fb, x, t.nb * BN, t.e);
                }
              } else {
#pragma unroll
                for (int j = 0; j < Cf::BNH / Cf::BOXN; ++j) {
                  int n0;
                  if constexpr (PAIR) {
                    n0 = (GATED ? int(half) * (p.g.N / 2) + t.nb * Cf::OUT_BN : t.nb * BN + int(half) * Cf::BNH) +
                         j * Cf::BOXN;
                    tma_load_3d_pair(b_dst + j * Cf::BOX_BYTES, &tmB, fb, n0, x, t.e);
                  } else {
                    constexpr int HB = Cf::BNH / Cf::BOXN / 2;  // boxes of one half
                    n0 = GATED ? (j >= HB ? p.g.N / 2 : 0) + t.nb * Cf::OUT_BN + (j >= HB ? j - HB : j) * Cf::BOXN
                               : t.nb * BN + j * Cf::BOXN;
                    tma_load_3d(b_dst + j * Cf::BOX_BYTES, &tmB, fb, n0, x, t.e);
                  }
                }
              }
            }
            __syncwarp();
            if (p.gather_a && lane < pieces) {
              if constexpr (PAIR)
                tma_gather4_pair(a_dst + lane * 512, &tmAg, fb, kb * Cf::BK, r0, r1, r2, r3);
              else
                tma_gather4(a_dst + lane * 512, &tmAg, fb, kb * Cf::BK, r0, r1, r2, r3);
            }
          } else {
            const int s0 = t.begin + kb * Cf::BK;
            const bool tail = s0 + Cf::BK > t.end;
            // boxes of each operand that start inside it (the columns of the others are not stored)
            const int p0 = t.m0 + int(half) * Cf::BM;
            const int q0 = t.nb * BN + int(half) * Cf::BNH;
            constexpr int PB = Cf::BM / Cf::BOXN, QB = Cf::BNH / Cf::BOXN;
            auto boxes_in = [](int x0, int cols, int most) {
              return min(max((cols - x0 + Cf::BOXN - 1) / Cf::BOXN, 0), most);
            };
            const int np = boxes_in(p0, p.out_rows, PB), nq = boxes_in(q0, p.out_cols, QB);
            // A ragged slab: both operands of this CTA complete on its own barrier, and
            // the leader's full barrier has nothing to count.
            if (tail) fb = tailf0 + 8 * s;
            const int peer = PAIR ? boxes_in(p0 + Cf::BM, p.out_rows, PB) + boxes_in(q0 + Cf::BNH, p.out_cols, QB) : 0;
            if (elect_one()) {
              if (tail) {
                mbar_arrive_expect_tx(fb, (np + nq) * Cf::BOX_BYTES);
                if (leader) mbar_arrive(full0 + 8 * s);
              } else if (leader) {
                mbar_arrive_expect_tx(full0 + 8 * s, (np + nq + peer) * Cf::BOX_BYTES);
              }
              if (PAIR && !tail) {
#pragma unroll
                for (int j = 0; j < PB; ++j)
                  if (!p.gather_p && j < np)
                    tma_load_3d_pair(a_dst + j * Cf::BOX_BYTES, &tmA, fb, p0 + j * Cf::BOXN, s0, 0);
#pragma unroll
                for (int j = 0; j < QB; ++j)
                  if (!p.gather_q && j < nq)
                    tma_load_3d_pair(b_dst + j * Cf::BOX_BYTES, &tmB, fb, q0 + j * Cf::BOXN, s0, 0);
              } else {
#pragma unroll
                for (int j = 0; j < PB; ++j)
                  if (!p.gather_p && j < np) tma_load_3d(a_dst + j * Cf::BOX_BYTES, &tmA, fb, p0 + j * Cf::BOXN, s0, 0);
#pragma unroll
                for (int j = 0; j < QB; ++j)
                  if (!p.gather_q && j < nq) tma_load_3d(b_dst + j * Cf::BOX_BYTES, &tmB, fb, q0 + j * Cf::BOXN, s0, 0);
              }
            }
            tails += tail ? 1 : 0;
            __syncwarp();
            if (p.gather_p || p.gather_q) {
              // 16 quads of slots x the operand's boxes
              const int quad = lane & 15;
              r0 = gathered_row(p, s0 + 4 * quad, t.end);
              r1 = gathered_row(p, s0 + 4 * quad + 1, t.end);
              r2 = gathered_row(p, s0 + 4 * quad + 2, t.end);
              r3 = gathered_row(p, s0 + 4 * quad + 3, t.end);
              const uint32_t dst = (p.gather_p ? a_dst : b_dst) + quad * 512;
              const CUtensorMap* map = p.gather_p ? &tmAg : &tmBg;
              const int x0 = p.gather_p ? p0 : q0;
              for (int j = lane >> 4; j < (p.gather_p ? np : nq); j += 2) {
                if (PAIR && !tail)
                  tma_gather4_pair(dst + j * Cf::BOX_BYTES, map, fb, x0 + j * Cf::BOXN, r0, r1, r2, r3);
                else
                  tma_gather4(dst + j * Cf::BOX_BYTES, map, fb, x0 + j * Cf::BOXN, r0, r1, r2, r3);
              }
            }
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        *issued_slot = it;
        tail_slot[0] = tails;
      }
    }
    grid_launch_dependents();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer (the pair's leader)
    if (leader) {
      int it = 0, tc = 0;
      uint32_t tail_ph = 0;  // parity of each stage's next ragged slab
      bool ok = true;
      for (int w = unit; ok && w < work; w += nunits) {
        const GroupTile t = group_tile<Cf>(p, cum, w);
        if (t.kbs == 0) continue;
        const int b = tc & 1;
        if (!warp_wait_phase(p.g, acce0 + 8 * b, ((tc >> 1) & 1) ^ 1, ROLE_MMA | (0x80u << 8))) break;
        ++tc;
        tc_fence_after();
        const uint32_t d = tmem + b * Cf::ACC_COLS;
        for (int kb = 0; kb < t.kbs; ++kb, ++it) {
          const int s = it % S;
          ok = warp_wait_phase(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8));
          if (WGRAD && ok && t.begin + (kb + 1) * Cf::BK > t.end) {
            ok = warp_wait_phase(p.g, tailok0 + 8 * s, (tail_ph >> s) & 1u, ROLE_MMA | ((0x40u + s) << 8));
            tail_ph ^= 1u << s;
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_addr = sA + s * Cf::A_BYTES;
          const uint32_t b_addr = sB + s * Cf::B_BYTES;
          uint64_t ad[Cf::KSTEPS], bd[Cf::KSTEPS];
#pragma unroll
          for (int kk = 0; kk < Cf::KSTEPS; ++kk) {
            ad[kk] = WGRAD ? sdesc(a_addr + kk * Cf::UK * 128, Cf::BOX_BYTES, 1024, SWZ_128B)
                           : sdesc(a_addr + kk * 32, 16, 1024, SWZ_128B);
            bd[kk] = Cf::B_KMAJOR ? sdesc(b_addr + kk * 32, 16, 1024, SWZ_128B)
                                  : sdesc(b_addr + kk * Cf::UK * 128, Cf::BOX_BYTES, 1024, SWZ_128B);
          }
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < Cf::KSTEPS; ++kk) {
              const uint32_t acc = (kb > 0 || kk > 0) ? 1u : 0u;
              if constexpr (PAIR)
                mma_issue_pair<KIND>(d, ad[kk], bd[kk], Cf::IDESC, acc);
              else
                mma_issue<KIND>(d, ad[kk], bd[kk], Cf::IDESC, acc);
            }
            if constexpr (PAIR)
              mma_commit_pair(empty0 + 8 * s, uint16_t(0x3u));
            else
              mma_commit(empty0 + 8 * s);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          if constexpr (PAIR)
            mma_commit_pair(accf0 + 8 * b, uint16_t(0x3u));
          else
            mma_commit(accf0 + 8 * b);
        }
        __syncwarp();
      }
      if (lane == 0) *consumed_slot = it;
      if (elect_one()) {
        if constexpr (PAIR)
          mma_commit_pair(drain_bar, uint16_t(1u));
        else
          mma_commit(drain_bar);
      }
      __syncwarp();
      if (lane == 0) wait_phase_drain(p.g, drain_bar, 0);
      __syncwarp();
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- epilogue (every CTA)
    int tc = 0;
    EpiRing ring{sE + static_cast<uint32_t>(warp * Cf::EPI_BUFS * EPI_WARP_BYTES), Cf::EPI_BUFS, 0,
                 sE + static_cast<uint32_t>(Cf::EPI_BUFS * EPI_BYTES)};
    for (int w = unit; w < work; w += nunits) {
      const GroupTile t = group_tile<Cf>(p, cum, w);
      const int b = tc & 1;
      if (t.kbs > 0) {
        // the four warps take every decision together: thread 0 waits, the barrier publishes the outcome
        if (threadIdx.x == 0)
          ok_slot[b] = wait_phase(p.g, accf0 + 8 * b, (tc >> 1) & 1, ROLE_EPILOGUE | (b << 8)) ? 1 : 0;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!ok_slot[b]) break;
        ++tc;
        tc_fence_after();
      }
      const int row0 = t.m0 + int(half) * Cf::BM + warp * 32;
      const int col0 = t.nb * Cf::OUT_BN;
      const int z = WGRAD ? t.e : 0;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * Cf::ACC_COLS;
      const int ncols = min(Cf::OUT_BN, p.out_cols - col0);
      const int nchunks = row0 < t.row_end && ncols > 0 ? (ncols + 31) / 32 : 0;
      const bool null_group = !WGRAD && t.e >= p.groups;
      float scale = p.g.alpha;
      if (!WGRAD && p.row_scale != nullptr && !null_group && row0 + lane < t.end)
        scale *= p.row_scale[gathered_row(p, row0 + lane, t.end)];
      auto store = [&](int c, const uint32_t(&words)[16]) {
        const uint32_t stage = epi_acquire(p.g, lane, ring);
        epi_put_row(stage, lane, words);
        group_flush<WGRAD>(p, &tmC, stage, lane, row0, t.row_end, col0 + c * 32, z);
      };
      auto emit = [&](int c, const uint32_t(&r)[32], const uint32_t(&r2)[32]) {
        uint32_t words[16];
        if (WGRAD || p.plain || null_group) {
#pragma unroll
          for (int j = 0; j < 16; ++j) words[j] = pack2<KindTraits<KIND>::out>(r[2 * j], r[2 * j + 1]);
        } else {
          float v[32];
          group_scale<KIND>(p, t.e, col0 + c * 32, lane, scale, r, v);
          if constexpr (GATED) {
            float u[32];
            group_scale<KIND>(p, t.e, p.g.N / 2 + col0 + c * 32, lane, scale, r2, u);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = v[k] / (1.0f + expf(-v[k])) * u[k];
          } else {
            epi_activate(v, p.g.act);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            words[j] = pack2<KindTraits<KIND>::out>(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
        }
        store(c, words);
      };
      if (t.kbs == 0) {
        // nothing was accumulated (K = 0, an empty group's gradient, the slots past the last group)
        uint32_t zero[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) zero[k] = 0u;
        for (int c = 0; c < nchunks; ++c) emit(c, zero, zero);
        continue;
      }
      if constexpr (GATED) {
        for (int c = 0; c < nchunks; ++c) {
          uint32_t ra[32], rb[32];
          __syncwarp();
          tmem_ld_32x32b_x32(taddr + c * 32, ra);
          tmem_ld_32x32b_x32(taddr + BN / 2 + c * 32, rb);
          tmem_wait_ld_into(ra);
          tmem_wait_ld_into(rb);
          emit(c, ra, rb);
        }
      } else if (nchunks > 0) {
        for_each_acc_chunk(taddr, nchunks, [&](int c, const uint32_t(&r)[32]) { emit(c, r, r); });
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(mapa_shared(acce0 + 8 * b, 0));
        else
          mbar_arrive(acce0 + 8 * b);
      }
    }
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  } else if (WGRAD && warp == 6) {
    // ---------------------------------------------------------------- ragged slabs (every CTA)
    int it = 0, seen = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int w = unit; ok && w < work; w += nunits) {
      const GroupTile t = group_tile<Cf>(p, cum, w);
      if (t.kbs == 0) continue;
      const int valid = t.end - t.begin - (t.kbs - 1) * Cf::BK;
      it += t.kbs;
      if (valid == Cf::BK) continue;
      const int s = (it - 1) % S;
      if (!warp_wait_phase(p.g, tailf0 + 8 * s, (ph >> s) & 1u, ROLE_COPY | (s << 8))) {
        ok = false;
        break;
      }
      ph ^= 1u << s;
      ++seen;
      // clear rows [valid, BK) of every 128-byte-wide box (a whole row: the swizzle permutes within it)
      constexpr int NBOX = Cf::BM / Cf::BOXN + Cf::BNH / Cf::BOXN;
#pragma unroll
      for (int j = 0; j < NBOX; ++j) {
        const uint32_t box = j < Cf::BM / Cf::BOXN ? sA + s * Cf::A_BYTES + j * Cf::BOX_BYTES
                                                   : sB + s * Cf::B_BYTES + (j - Cf::BM / Cf::BOXN) * Cf::BOX_BYTES;
        for (int r = valid + (lane >> 3); r < Cf::BK; r += 4) st_shared_v4(box + r * 128 + (lane & 7) * 16, 0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(mapa_shared(tailok0 + 8 * s, 0));
        else
          mbar_arrive(tailok0 + 8 * s);
      }
    }
    if (lane == 0) tail_slot[1] = seen;
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
  if (WGRAD && threadIdx.x == 32 && tail_slot[1] < tail_slot[0]) {
    // the unseen ragged slabs are the last ones, at most one a stage: walk the work again and wait for them
    int it = 0, n = 0;
    uint32_t ph = 0;
    for (int w = unit; n < tail_slot[0] && w < work; w += nunits) {
      const GroupTile t = group_tile<Cf>(p, cum, w);
      it += t.kbs;
      if (t.kbs == 0 || (t.end - t.begin) % Cf::BK == 0) continue;
      const int s = (it - 1) % S;
      if (n++ >= tail_slot[1] && !wait_phase_drain(p.g, tailf0 + 8 * s, (ph >> s) & 1u)) break;
      ph ^= 1u << s;
    }
  }
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 5) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, Cf::TMEM_COLS);
    else
      tmem_dealloc(tmem, Cf::TMEM_COLS);
  }
}

}  // namespace dgt
