// Persistent grouped GEMM for sm_103a: every expert's rows times that
// expert's weights in one launch, and the weights' gradient.
//
// The mathematics (contraction in fp32, one rounding at the end):
//   product   C[s] = epilogue(A[row(s)] . W_e)          for s in group e
//   gradient  dW_e = sum over s in group e of P[s]^T Q[s] (P, Q: dC and A, or A and dC)
//
// It is the dense kernel's pipeline -- a TMA producer warp, one thread that
// issues tcgen05.mma, epilogue warps, fp32 accumulators double buffered in
// tensor memory -- with what ragged groups need:
//
//   * Tiles come from the offsets on the device, so the host never reads the
//     group sizes. A scheduler warp holds the tile counts of 32 groups at a time
//     (a lane each), finds a work item's group by ballot and hands the tiles to
//     the other warps through a ring in shared memory; empty groups cost nothing.
//   * Rows in slot order come by TMA boxes. Rows that the caller names are
//     gathered by TMA (tile::gather4: four rows of 128 bytes an instruction,
//     each lane of the producer warp issues one) where a group has few: an
//     instruction costs about 75 cycles, so 128 rows of a slab take 2400, four
//     times the MMA's 512, but a handful hides behind the weights' stream. For
//     larger groups the host first permutes the rows into the caller's workspace
//     (one bandwidth-bound pass) and they are rows in slot order again. A group's
//     last tile fetches only the rows it has.
//   * The gradient contracts over a ragged number of rows. A group's last slab
//     of 64 slots may run into the next group's rows, and an infinity or NaN of
//     another group times zero would be a NaN; so a small kernel first writes
//     every group's last slab, zero padded, to the workspace, and the producer
//     loads that one from there.
//   * The tiles are many and their k-loops short (1024 rows an expert are 16
//     slabs of the gradient), so the epilogue has to keep up: eight warps, each
//     storing 64 columns of its 32 rows with one TMA store.
//
// Large groups are bound by the tensor cores (the pipe is 88-94% busy) and by the
// rows that fill a group's last tile only in part: 16384 rows x 4096 x 4096 BF16
// take 334 us in 16 groups (1644 TFLOP/s) and 293 us in one. Small groups are bound
// by reading the weights: 16 tokens x 4 of 64 experts, 2048 -> 4096, 102 us, 6.8 TB/s.
//
// PAIR: a CTA pair (cta_group::2) computes a 256 x BN tile, each CTA loading
// 128 rows of A and half of the B columns; else one CTA computes 128 x BN.
// GATED: W's columns are gate and value halves; a tile holds the same BN / 2
// columns of both (in the pair each CTA loads one of them), and the epilogue
// stores silu(gate) * value, so the 2 x wider intermediate is never written.
#pragma once

#include "dgt_experts.h"
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
constexpr int kGroupThreads = 384;  // warps 0-3 and 8-11 epilogue, 4 producer, 5 MMA, 6 idle, 7 scheduler
constexpr int kGroupEpiWarps = 8;
constexpr int kTileRing = 4;        // tiles the scheduler is ahead

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
  int value_at;  // gated: where the value half starts in W (a column of row-major W, else a row)
  int plain;     // the epilogue is the identity
  int out_cols;  // columns of C (or of dW)
  int out_rows;  // gradient: rows of dW
  int wide_p, wide_q;  // gradient: an operand's map has 64-column blocks as its outer coordinate (two blocks a box)
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
  static constexpr int EPI_TILE = 32 * 128;                // one warp's 32 rows x 64 columns of a 16-bit C
  static constexpr int EPI_STAGING = kGroupEpiWarps * EPI_TILE;
  static constexpr int FIXED = 1024 /*align slack*/ + BAR_BYTES + EPI_STAGING;
  static constexpr int STAGES_FIT = (SMEM_LIMIT - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int SMEM_BYTES = FIXED + STAGES * STAGE_BYTES;
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
  static constexpr int NUM_BARS = 2 * STAGES + 5 + 2 * kTileRing;
  static constexpr int A_BOX_ROWS = PAIR ? 128 : 32;  // rows of A per box: one CTA's tile may hold few
  static_assert(BN % 64 == 0 && BN >= 64 && BN <= 256, "tile width");
  static_assert(B_KMAJOR || ES == 2, "8-bit operands are read K-major");
  static_assert(B_KMAJOR || BNH % BOXN == 0, "MN-major B comes in whole boxes");
  static_assert(!GATED || B_KMAJOR || PAIR || (BN / 2) % BOXN == 0, "each half is whole boxes");
  static_assert(OUT_BN % 64 == 0, "an epilogue warp stores 64 columns at a time");
  static_assert(NUM_BARS * 8 + 32 + kTileRing * 32 <= BAR_BYTES, "barrier area");
  static_assert(!WGRAD || (ES == 2 && BM == 2 * BOXN && BNH == 2 * BOXN), "two 64-column blocks of each operand per CTA");
  static_assert(STAGES >= 4 && SMEM_BYTES <= SMEM_LIMIT, "shared memory");
  static constexpr uint32_t IDESC = (1u << 4) | (KindTraits<KIND>::fmt << 7) | (KindTraits<KIND>::fmt << 10) |
                                    ((WGRAD ? 1u : 0u) << 15) | ((B_KMAJOR ? 0u : 1u) << 16) |
                                    (uint32_t(BN >> 3) << 17) | (uint32_t(BMT >> 4) << 24);
};

// A work item: group, first accumulator row and the rows' end (slots of the
// product, rows of dW for the gradient), tile column, slots of the group
// [begin, end) and k-slabs (-1: no more work).
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

// A value that every lane holds, as one the compiler knows to be the same in all
// of them. The producer's and the MMA warp's instructions take their operands
// from uniform registers, for which what decides their loops' ends has to be
// known as uniform too; else every slab pays for the moves: one token's four
// experts, 7168 -> 2048 BF16 (64 CTAs of 112 slabs), 38.8 us instead of 30.2, and
// 32768 E4M3 rows x 4096 x 4096, gated, 404 instead of 377.
__device__ __forceinline__ int uniform(int v) {
  return static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(v)));
}

// warp_wait_phase where the wait is mostly over before it begins: every lane
// tries once, and only a miss takes the timed path.
__device__ __forceinline__ bool group_wait(const GemmParams& g, uint32_t bar, uint32_t parity, uint32_t code) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return __any_sync(0xFFFFFFFFu, warp_wait_phase(g, bar, parity, code));
}

// The next tile of the ring, handed out by the scheduler: `n` counts this
// warp's tiles. All lanes return the same; kbs is -1 after the last one and
// when the launch was aborted. Warp-collective.
__device__ __forceinline__ GroupTile next_tile(const GemmParams& g, uint32_t schf0, uint32_t sche0, uint32_t ring, int n,
                                               uint32_t role) {
  const int s = n % kTileRing;
  GroupTile t;
  t.kbs = -1;
  if (!group_wait(g, schf0 + 8 * s, (n / kTileRing) & 1, role)) return t;
  __syncwarp();
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(t.e), "=r"(t.m0), "=r"(t.row_end), "=r"(t.nb)
               : "r"(ring + 32 * s)
               : "memory");
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(t.begin), "=r"(t.end)
               : "r"(ring + 32 * s + 16)
               : "memory");
  t.kbs = uniform(static_cast<int>(ld_shared_u32(ring + 32 * s + 24)));
  t.e = uniform(t.e);
  t.m0 = uniform(t.m0);
  t.row_end = uniform(t.row_end);
  t.nb = uniform(t.nb);
  t.begin = uniform(t.begin);
  t.end = uniform(t.end);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(sche0 + 8 * s);
  return t;
}

// Row of the gathered operand for slot s of a group [begin, end): slots past
// the end repeat the last one, so every address is a row of this group.
__device__ __forceinline__ int gathered_row(const GroupParams& p, int s, int end) {
  s = min(s, end - 1);
  const int r = p.rows != nullptr ? p.rows[s] : s;
  return min(max(r, 0), p.a_rows - 1);
}

// An epilogue warp's staging tile: 32 rows of 128 bytes in the layout of
// TMA's 128-byte swizzle; 16-byte chunk j of row r sits at r * 128 + ((j ^ (r mod 8)) * 16).
__device__ __forceinline__ uint32_t stage_chunk(uint32_t stage, int r, int j) {
  return stage + static_cast<uint32_t>(r * 128) + (static_cast<uint32_t>(j ^ (r & 7)) << 4);
}

// Writes the staged 32 x 64 tile to C[row0 .., col0 ..] of matrix z: rows
// before row_end and columns before p.out_cols only. TMA stores whole 32-row
// pieces (CLIP: it clips at the tensor's end; a group's end it does not know, so
// a piece that crosses it is stored row by row).
template <bool CLIP>
__device__ __forceinline__ void group_flush(const GroupParams& p, const CUtensorMap* tmC, uint32_t stage, int lane,
                                            int row0, int row_end, int col0, int z) {
  const bool full_cols = col0 + 64 <= p.out_cols;
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
  if (p.g.c_gran == 16) {
    // 8 lanes a row, 16 bytes a lane; the last lane of a ragged row element by element
    const int l = lane & 7, cols = p.out_cols - col0 - 8 * l;
#pragma unroll
    for (int rr = 0; rr < 32; rr += 4) {
      const int r = rr + (lane >> 3);
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(stage_chunk(stage, r, l))
                   : "memory");
      if (row0 + r < row_end) {
        uint16_t* dst = base + static_cast<long long>(row0 + r) * p.g.ldc + 8 * l;
        if (cols >= 8) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 7; ++k)
            if (k < cols) dst[k] = static_cast<uint16_t>(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu);
        }
      }
    }
  } else if (full_cols) {
    // Rows of any 2-byte alignment: 8 lanes a row store the 16-byte pieces that lie whole in the row's 128 bytes,
    // each shifted together from two staged chunks, and a lane each the eight columns around them.
    const int l = lane & 7;
#pragma unroll
    for (int rr = 0; rr < 32; rr += 4) {
      const int r = rr + (lane >> 3);
      uint16_t* dst = base + static_cast<long long>(row0 + r) * p.g.ldc;
      const int m = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1) & 7;  // columns past a 16-byte boundary
      uint32_t w[8];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(stage_chunk(stage, r, l))
                   : "memory");
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "r"(stage_chunk(stage, r, (l + 1) & 7))
                   : "memory");
      const int edge = l < 8 - m ? l : 56 + l;
      const uint32_t one = ld_shared_u16(stage_chunk(stage, r, edge >> 3) + ((edge & 7) << 1));
      if (row0 + r >= row_end) continue;
      if (m == 0) {
        *reinterpret_cast<uint4*>(dst + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
        continue;
      }
      // columns 8 l + 8 - m .. 8 l + 15 - m: element 8 - m of the two chunks
      const int s = 8 - m, q = s >> 1, bits = (s & 1) * 16;
      uint32_t a[6], b[5];
#pragma unroll
      for (int k = 0; k < 6; ++k) a[k] = q & 2 ? w[k + 2] : w[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) b[k] = q & 1 ? a[k + 1] : a[k];
      if (l < 7)
        *reinterpret_cast<uint4*>(dst + 8 * l + s) =
            make_uint4(__funnelshift_r(b[0], b[1], bits), __funnelshift_r(b[1], b[2], bits),
                       __funnelshift_r(b[2], b[3], bits), __funnelshift_r(b[3], b[4], bits));
      dst[edge] = static_cast<uint16_t>(one);
    }
  } else {
    // the matrix's last columns: a row at a time, two columns a lane
    const int col = col0 + 2 * lane;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      const uint32_t v = ld_shared_u32(stage_chunk(stage, r, lane >> 2) + ((lane & 3) << 2));
      if (row0 + r < row_end && col < p.out_cols) {
        uint16_t* dst = base + static_cast<long long>(row0 + r) * p.g.ldc + 2 * lane;
        dst[0] = static_cast<uint16_t>(v & 0xFFFFu);
        if (col + 1 < p.out_cols) dst[1] = static_cast<uint16_t>(v >> 16);
      }
    }
  }
  __syncwarp();
}

// The activation of every element. GELU's tanh form is v / (1 + exp(-2 u)) with
// u = sqrt(2 / pi) (v + 0.044715 v^3); like the gated SiLU it takes the hardware's
// exponential and reciprocal. The exponential of x is within 2 + 1.17 |x| units in
// the last place: 2^-22 near zero, 2^-18 at 20, 1.3e-5 at 88, so the result is within
// 4e-5 of its value before it is rounded to 16 bits (up to 2^-8, 2^-11 for float16). Where
// 1 + exp passes 2^126 (gates below -87.3) the quotient is 0 and not the 1e-36 that bfloat16 could
// hold. (With tanhf, which the dense products' epilogue takes, a 256-wide tile's took
// about 15000 cycles.)
__device__ __forceinline__ void group_activate(float (&v)[32], int act) {
  if (act == GEMM_ACT_GELU_TANH) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float u = 0.79788456080286536f * (v[k] + 0.044715f * v[k] * v[k] * v[k]);
      v[k] = __fdividef(v[k], 1.0f + __expf(-2.0f * u));
    }
  } else {
    epi_activate(v, act);
  }
}

template <bool PAIR>
__device__ __forceinline__ void wgrad_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (PAIR)
    tma_load_3d_pair(dst, map, bar, x, y, z);
  else
    tma_load_3d(dst, map, bar, x, y, z);
}

// The scaled and biased pre-activation of 32 accumulator columns from
// column `col` of group e: v = scale * col_scale[col] * acc + bias[col]. Each
// lane loads one column's scale and bias, and shuffles hand them to every lane.
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
__global__ void __launch_bounds__(kGroupThreads, 1)
    group_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                 const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(sptr + S * Cf::STAGE_BYTES + Cf::EPI_STAGING);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * S;
  const uint32_t accf0 = empty0 + 8 * S;
  const uint32_t acce0 = accf0 + 16;
  const uint32_t drain_bar = acce0 + 16;
  const uint32_t schf0 = drain_bar + 8;  // tile ring: entry written, entry read by every warp that takes tiles
  const uint32_t sche0 = schf0 + 8 * kTileRing;
  const uint32_t ring = (sche0 + 8 * kTileRing + 15u) & ~15u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sptr + (ring - sbase) + 32 * kTileRing);
  volatile int* issued_slot = reinterpret_cast<volatile int*>(tmem_slot) + 1;
  volatile int* consumed_slot = issued_slot + 1;

  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t half = PAIR ? cluster_ctarank() : 0u;
  const bool leader = half == 0;
  const int unit = blockIdx.x / Cf::CTAS;
  const int nunits = gridDim.x / Cf::CTAS;

  if (warp == 4 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, kGroupEpiWarps * Cf::CTAS);
    }
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(schf0 + 8 * i, 1);
      // every warp that takes tiles: epilogue, producer, the leader's MMA warp
      mbar_init(sche0 + 8 * i, kGroupEpiWarps + 1 + (leader ? 1 : 0));
    }
    mbar_init(drain_bar, 1);
    *issued_slot = 0;
    *consumed_slot = 0;
    fence_mbar_init();
    if (!WGRAD && p.g.num_kb > 0) {
      tma_prefetch_desc(p.gather_a ? &tmA2 : &tmA);
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
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // barriers of both CTAs initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA producer (every CTA)
    if (!(p.g.debug & DEBUG_STALL_PRODUCER)) {
      int it = 0;
      bool ok = true;
      const uint32_t lead_full0 = PAIR ? mapa_shared(full0, 0) : full0;
      for (int n = 0; ok; ++n) {
        const GroupTile t = next_tile(p.g, schf0, sche0, ring, n, ROLE_PRODUCER | (0x80u << 8));
        if (t.kbs < 0) break;
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
          if (!group_wait(p.g, empty0 + 8 * s, ((it / S) & 1) ^ 1, ROLE_PRODUCER | (s << 8))) {
            ok = false;
            break;
          }
          const uint32_t a_dst = sA + s * Cf::A_BYTES;
          const uint32_t b_dst = sB + s * Cf::B_BYTES;
          const uint32_t fb = lead_full0 + 8 * s;
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
                  const int n0 = GATED ? int(half) * p.value_at + t.nb * Cf::OUT_BN : t.nb * BN + int(half) * Cf::BNH;
                  tma_load_3d_pair(b_dst, &tmB, fb, x, n0, t.e);
                } else if constexpr (GATED) {
                  tma_load_3d(b_dst, &tmB, fb, x, t.nb * Cf::OUT_BN, t.e);
                  tma_load_3d(b_dst + Cf::B_BYTES / 2, &tmB, fb, x, p.value_at + t.nb * Cf::OUT_BN, t.e);
                } else {
                  tma_load_3d(b_dst, &tmB, fb, x, t.nb * BN, t.e);
                }
              } else {
#pragma unroll
                for (int j = 0; j < Cf::BNH / Cf::BOXN; ++j) {
                  int n0;
                  if constexpr (PAIR) {
                    n0 = (GATED ? int(half) * p.value_at + t.nb * Cf::OUT_BN : t.nb * BN + int(half) * Cf::BNH) +
                         j * Cf::BOXN;
                    tma_load_3d_pair(b_dst + j * Cf::BOX_BYTES, &tmB, fb, n0, x, t.e);
                  } else {
                    constexpr int HB = Cf::BNH / Cf::BOXN / 2;  // boxes of one half
                    n0 = GATED ? (j >= HB ? p.value_at : 0) + t.nb * Cf::OUT_BN + (j >= HB ? j - HB : j) * Cf::BOXN
                               : t.nb * BN + j * Cf::BOXN;
                    tma_load_3d(b_dst + j * Cf::BOX_BYTES, &tmB, fb, n0, x, t.e);
                  }
                }
              }
            }
            __syncwarp();
            if (p.gather_a && lane < pieces) {
              if constexpr (PAIR)
                tma_gather4_pair(a_dst + lane * 512, &tmA2, fb, kb * Cf::BK, r0, r1, r2, r3);
              else
                tma_gather4(a_dst + lane * 512, &tmA2, fb, kb * Cf::BK, r0, r1, r2, r3);
            }
          } else {
            // the group's last slab, where ragged, comes from its zero-padded copy: 64 rows for each group
            const int s0 = t.begin + kb * Cf::BK;
            const bool ragged = s0 + Cf::BK > t.end;
            const int y = ragged ? t.e * Cf::BK : s0;
            const CUtensorMap* map_p = ragged ? &tmA2 : &tmA;
            const CUtensorMap* map_q = ragged ? &tmB2 : &tmB;
            const bool wide_p = ragged || p.wide_p, wide_q = ragged || p.wide_q;
            const int p0 = t.m0 + int(half) * Cf::BM, q0 = t.nb * BN + int(half) * Cf::BNH;
            if (elect_one()) {
              if (leader) mbar_arrive_expect_tx(full0 + 8 * s, Cf::CTAS * Cf::STAGE_BYTES);
              if (wide_p) {
                wgrad_load<PAIR>(a_dst, map_p, fb, 0, y, p0 / Cf::BOXN);
              } else {
                wgrad_load<PAIR>(a_dst, map_p, fb, p0, y, 0);
                wgrad_load<PAIR>(a_dst + Cf::BOX_BYTES, map_p, fb, p0 + Cf::BOXN, y, 0);
              }
              if (wide_q) {
                wgrad_load<PAIR>(b_dst, map_q, fb, 0, y, q0 / Cf::BOXN);
              } else {
                wgrad_load<PAIR>(b_dst, map_q, fb, q0, y, 0);
                wgrad_load<PAIR>(b_dst + Cf::BOX_BYTES, map_q, fb, q0 + Cf::BOXN, y, 0);
              }
            }
          }
          __syncwarp();
        }
      }
      if (lane == 0) *issued_slot = it;
    }
    grid_launch_dependents();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer (the pair's leader)
    if (leader) {
      constexpr uint32_t A_STEP = (WGRAD ? Cf::UK * 128 : 32) / 16, B_STEP = (Cf::B_KMAJOR ? 32 : Cf::UK * 128) / 16;
      const uint64_t a_desc = sdesc(sA, WGRAD ? Cf::BOX_BYTES : 16, 1024, SWZ_128B);
      const uint64_t b_desc = sdesc(sB, Cf::B_KMAJOR ? 16 : Cf::BOX_BYTES, 1024, SWZ_128B);
      int it = 0, tc = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const GroupTile t = next_tile(p.g, schf0, sche0, ring, n, ROLE_MMA | (0x81u << 8));
        if (t.kbs < 0) break;
        if (t.kbs == 0) continue;
        const int b = tc & 1;
        if (!group_wait(p.g, acce0 + 8 * b, ((tc >> 1) & 1) ^ 1, ROLE_MMA | (0x80u << 8))) break;
        ++tc;
        tc_fence_after();
        const uint32_t d = tmem + b * Cf::ACC_COLS;
        for (int kb = 0; kb < t.kbs; ++kb, ++it) {
          const int s = it % S;
          if (!group_wait(p.g, full0 + 8 * s, (it / S) & 1, ROLE_MMA | (s << 8))) {
            ok = false;
            break;
          }
          tc_fence_after();
          // a descriptor's address field counts 16 bytes
          const uint64_t a_stage = a_desc + static_cast<uint32_t>(s) * (Cf::A_BYTES / 16);
          const uint64_t b_stage = b_desc + static_cast<uint32_t>(s) * (Cf::B_BYTES / 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < Cf::KSTEPS; ++kk) {
              const uint32_t acc = (kb > 0 || kk > 0) ? 1u : 0u;
              if constexpr (PAIR)
                mma_issue_pair<KIND>(d, a_stage + kk * A_STEP, b_stage + kk * B_STEP, Cf::IDESC, acc);
              else
                mma_issue<KIND>(d, a_stage + kk * A_STEP, b_stage + kk * B_STEP, Cf::IDESC, acc);
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
  } else if (warp < 4 || warp >= 8) {
    // ---------------------------------------------------------------- epilogue (every CTA)
    // warps q and q + 8 read tensor-memory lanes 32 q ..; the first takes 64-column pieces 0, 2, ..., the second 1, 3, ...
    const int q = warp & 3, set = warp >> 3;
    const uint32_t stage = sE + static_cast<uint32_t>((set * 4 + q) * Cf::EPI_TILE);
    int tc = 0;
    for (int n = 0;; ++n) {
      const GroupTile t = next_tile(p.g, schf0, sche0, ring, n, ROLE_EPILOGUE | (0x80u << 8));
      if (t.kbs < 0) break;
      const int b = tc & 1;
      if (t.kbs > 0) {
        if (!warp_wait_phase(p.g, accf0 + 8 * b, (tc >> 1) & 1, ROLE_EPILOGUE | (b << 8))) break;
        ++tc;
        tc_fence_after();
      }
      const int row0 = t.m0 + int(half) * Cf::BM + q * 32;
      const int col0 = t.nb * Cf::OUT_BN;
      const int z = WGRAD ? t.e : 0;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * Cf::ACC_COLS;
      const bool null_group = !WGRAD && t.e >= p.groups;
      const bool convert_only = WGRAD || p.plain || null_group;
      float scale = p.g.alpha;
      if (!WGRAD && p.row_scale != nullptr && !null_group && row0 + lane < t.end)
        scale *= p.row_scale[gathered_row(p, row0 + lane, t.end)];
      if (row0 < t.row_end) {
        for (int c = set * 64; c < Cf::OUT_BN && col0 + c < p.out_cols; c += 128) {
          uint32_t acc[2][32];
          if (t.kbs == 0) {
            // nothing was accumulated (K = 0, an empty group's gradient, the slots past the last group)
#pragma unroll
            for (int k = 0; k < 32; ++k) acc[0][k] = acc[1][k] = 0u;
          }
          uint32_t words[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int cc = c + 32 * h;
            if (t.kbs > 0) {
              __syncwarp();
              if constexpr (GATED) {
                tmem_ld_32x32b_x32(taddr + cc, acc[0]);
                tmem_ld_32x32b_x32(taddr + BN / 2 + cc, acc[1]);
                tmem_wait_ld_into(acc[0]);
                tmem_wait_ld_into(acc[1]);
              } else if (h == 0) {
                tmem_ld_32x32b_x32(taddr + cc, acc[0]);
                tmem_ld_32x32b_x32(taddr + cc + 32, acc[1]);
                tmem_wait_ld_into(acc[0]);
                tmem_wait_ld_into(acc[1]);
              }
            }
            const uint32_t(&r)[32] = GATED ? acc[0] : acc[h];
            if (convert_only) {
#pragma unroll
              for (int j = 0; j < 16; ++j) words[j] = pack2<KindTraits<KIND>::out>(r[2 * j], r[2 * j + 1]);
            } else {
              float v[32];
              group_scale<KIND>(p, t.e, col0 + cc, lane, scale, r, v);
              if constexpr (GATED) {
                float u[32];
                group_scale<KIND>(p, t.e, p.g.N / 2 + col0 + cc, lane, scale, acc[1], u);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __fdividef(v[k], 1.0f + __expf(-v[k])) * u[k];
              } else {
                group_activate(v, p.g.act);
              }
#pragma unroll
              for (int j = 0; j < 16; ++j)
                words[j] = pack2<KindTraits<KIND>::out>(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
            }
            if (h == 0) {
              // the tile's last TMA store has read it
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_v4(stage_chunk(stage, lane, 4 * h + j), words[4 * j], words[4 * j + 1], words[4 * j + 2],
                           words[4 * j + 3]);
          }
          group_flush<WGRAD>(p, &tmC, stage, lane, row0, t.row_end, col0 + c, z);
        }
      }
      if (t.kbs == 0) continue;
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
  } else if (warp == 7) {
    // ---------------------------------------------------------------- scheduler (every CTA)
    int n = 0;
    auto push = [&](const GroupTile& t) {
      const int s = n % kTileRing;
      const bool ok = warp_wait_phase(p.g, sche0 + 8 * s, ((n / kTileRing) & 1) ^ 1, ROLE_PRODUCER | (0x90u << 8));
      if (ok && lane == 0) {
        st_shared_v4(ring + 32 * s, t.e, t.m0, t.row_end, t.nb);
        st_shared_v4(ring + 32 * s + 16, t.begin, t.end, t.kbs, 0);
        mbar_arrive(schf0 + 8 * s);
      }
      ++n;
      return ok;
    };
    GroupTile t;
    bool ok = true;
    if constexpr (WGRAD) {
      const int per = p.g.tiles_m * p.g.tiles_n, work = p.groups * per;
      for (int w = unit; ok && w < work; w += nunits) {
        int mb;
        t.e = w / per;
        band_place(w - t.e * per, p.g.raster, p.g.tiles_m, p.g.tiles_n, mb, t.nb);
        t.begin = group_start(p, t.e);
        t.end = max(t.begin, group_start(p, t.e + 1));
        t.m0 = mb * Cf::BMT;
        t.row_end = p.out_rows;
        t.kbs = (t.end - t.begin + Cf::BK - 1) / Cf::BK;
        ok = push(t);
      }
    } else {
      // lane l: group base + l's slots and row tiles (group `groups`: the slots past the last one), and the tiles up
      // to and with it, counted from `before`
      int base = 0, before = 0, first = 0, last = 0, count = 0, incl = 0;
      auto load = [&]() {
        const int e = base + lane;
        first = e <= p.groups ? group_start(p, e) : p.slots;
        last = e < p.groups ? max(first, group_start(p, e + 1)) : p.slots;
        count = incl = (last - first + Cf::BMT - 1) / Cf::BMT;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += o;
        }
      };
      load();
      for (int w = unit; ok; w += nunits) {
        const int tile = w / p.g.tiles_n;  // row tile, were each column of tiles to be walked alone
        int sum = __shfl_sync(0xFFFFFFFFu, incl, 31);
        while (tile >= before + sum && base + 32 <= p.groups) {
          before += sum;
          base += 32;
          load();
          sum = __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (tile >= before + sum) break;
        const int l = __ffs(__ballot_sync(0xFFFFFFFFu, incl > tile - before)) - 1;
        const int tiles_m = __shfl_sync(0xFFFFFFFFu, count, l);
        const int tiles_before = before + __shfl_sync(0xFFFFFFFFu, incl, l) - tiles_m;
        int mb;
        band_place(w - tiles_before * p.g.tiles_n, p.g.raster, tiles_m, p.g.tiles_n, mb, t.nb);
        t.e = base + l;
        t.begin = __shfl_sync(0xFFFFFFFFu, first, l);
        t.end = __shfl_sync(0xFFFFFFFFu, last, l);
        t.m0 = t.begin + mb * Cf::BMT;
        t.row_end = t.end;
        t.kbs = t.e < p.groups ? p.g.num_kb : 0;
        ok = push(t);
      }
    }
    t.kbs = -1;
    if (ok) push(t);
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
