// C entry points of the grouped products (gemm_*_grouped) and of their weight
// gradient (gemm_*_grouped_wgrad): argument checks, tensor maps, the choice of
// kernel and the launch. The group sizes stay on the device.
#include <cstring>

#include "dgt_experts.h"
#include "group_launch.h"

namespace dgt {
namespace {

constexpr int64_t kIntLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kLdLimit = int64_t(1) << 39;

bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }

// TMA reads rows whose base and pitch are 16-byte multiples: rows of another pitch are copied first.
bool odd_pitch(int64_t ld, int es) { return (ld * es) % 16 != 0; }

// The pitch of a matrix of one row says nothing: any is as good as the next 16-byte multiple.
int64_t row_pitch(int64_t rows, int64_t cols, int64_t ld, int es) {
  return rows == 1 && ld >= cols ? (cols * es + 15) / 16 * 16 / es : ld;
}

// Widest store (16, 8, 4 or 2 bytes) that base, row pitch and matrix stride of a 16-bit matrix allow.
int store_granularity(const void* p, int64_t ld, int64_t stride) {
  const uint64_t v = uint64_t(reinterpret_cast<uintptr_t>(p)) | uint64_t(ld * 2) | uint64_t(stride * 2);
  int g = 16;
  while (g > 2 && v % g != 0) g >>= 1;
  return g;
}

struct Range {
  uintptr_t lo, hi;
};
// Bytes from the first to the last element of a rows x cols matrix (of `count` of them, `stride` apart).
Range range_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int es, int64_t count = 1, int64_t stride = 0) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + uintptr_t(((count - 1) * stride + (rows - 1) * ld + cols) * es)};
}
bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

CUtensorMapDataType map_type(int kind) {
  return kind == KIND_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : kind == KIND_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                            : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

void fill_common(const CallContext& ctx, GroupParams& p) {
  p.g.status = ctx.status;
  p.g.epoch = ctx.epoch;
  p.g.debug = ctx.debug;
  p.g.wait_limit_ns = ctx.wait_limit_ns;
}

// Copies of rows into the workspace ahead of a grouped kernel, a warp a row,
// 16 bytes a lane (the matrices start on 16-byte boundaries, their rows anywhere;
// bytes of the destination's pitch past the row are zero):
//   * `order`: the gathered operand's rows in slot order, order[s] = a[row(s)]
//   * `order_c`: the other operand's rows c[s], where their pitch is not TMA's
//   * `mats`: the weights of the groups that have slots, where TMA cannot read them in
//     place; a row of w_parts parts (the two halves of gated row-major weights) gets each
//     part on a boundary of its own
//   * `slab_a`, `slab_c` (the weights' gradient): the last slab of 64 slots of
//     every group whose count is not a multiple of 64, zeros past its end
// Bound by memory: one read of the rows (repeats of a token hit L2) and one
// write; 16384 slots of 4096 BF16 columns (134 MB written) take about 45 us.
struct StageRows {
  const uint8_t* a;
  const uint8_t* c;
  const uint8_t* w;
  const int* rows;
  const int* offsets;
  uint8_t* order;
  uint8_t* order_c;
  uint8_t* slab_a;
  uint8_t* slab_c;
  uint8_t* mats;
  long long ld_a, ld_c, ld_w, stride_w, pitch_a, pitch_c, pitch_w, bytes_a, bytes_c, bytes_w;  // (_w: of one part)
  int a_rows, groups, slots, w_rows, w_parts;
};

constexpr int kSlab = 64;

// A row that starts anywhere: each piece is shifted together from the two
// aligned ones that hold it, as long as the second lies whole in the row; the last
// pieces go byte by byte.
__device__ __forceinline__ void stage_shifted_row(const uint8_t* from, long long bytes, uint8_t* to, long long pitch,
                                                  int lane) {
  const int m = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
  if (from == nullptr) bytes = 0;
  const int pieces = static_cast<int>(pitch / 16), whole = static_cast<int>((m + bytes) / 16) - 1;
  const uint8_t* base = from - m;  // in the matrix, which starts on a boundary
#pragma unroll 2
  for (int c = lane; c < pieces; c += 32) {
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (c < whole) {
      const uint4 lo = *reinterpret_cast<const uint4*>(base + c * 16LL);
      const uint4 hi = *reinterpret_cast<const uint4*>(base + c * 16LL + 16);
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
      for (int i = 0; i < 16; ++i)
        if (c * 16LL + i < bytes) o[i >> 2] |= uint32_t(from[c * 16LL + i]) << (8 * (i & 3));
    }
    *reinterpret_cast<uint4*>(to + c * 16LL) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <bool SHIFTED>
__device__ __forceinline__ void stage_row(const uint8_t* from, long long bytes, uint8_t* to, long long pitch,
                                          int lane) {
  if constexpr (SHIFTED) {
    stage_shifted_row(from, bytes, to, pitch, lane);
    return;
  }
  const int pieces = static_cast<int>(pitch / 16);
  const int whole = from != nullptr ? static_cast<int>(bytes / 16) : 0;
  int c = lane;
  for (; c + 96 < whole; c += 128) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(from + (c + 32 * i) * 16LL);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(to + (c + 32 * i) * 16LL) = v[i];
  }
  for (; c < pieces; c += 32) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (c < whole) {
      const uint4 v = *reinterpret_cast<const uint4*>(from + c * 16LL);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if (from != nullptr && c == whole) {
      for (int i = 0; i < int(bytes - whole * 16LL); ++i) w[i >> 2] |= uint32_t(from[c * 16LL + i]) << (8 * (i & 3));
    }
    *reinterpret_cast<uint4*>(to + c * 16LL) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// SHIFTED: some rows start off 16-byte boundaries, which every copy of dC's rows
// and of the weights means. (A build of its own: with its registers and branches the
// rows of a training step's gradient, 16384 x 4096 BF16, took 3 us more.)
template <bool SHIFTED>
__global__ void __launch_bounds__(256) stage_rows_kernel(const StageRows p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  auto start = [&](int e) { return e <= 0 ? 0 : p.offsets == nullptr ? p.slots : min(max(p.offsets[e], 0), p.slots); };
  auto row = [&](int s) { return min(max(p.rows != nullptr ? p.rows[s] : s, 0), p.a_rows - 1); };
  const long long rows_a = p.order != nullptr ? start(p.groups) : 0;
  long long used = rows_a;
  if constexpr (SHIFTED) used += p.order_c != nullptr ? start(p.groups) : 0;
  const long long slabs = used + (p.slab_a != nullptr ? 2LL * p.groups * kSlab : 0);
  long long tasks = slabs;
  if constexpr (SHIFTED) tasks += p.mats != nullptr ? static_cast<long long>(p.groups) * p.w_rows * p.w_parts : 0;
  for (long long t = blockIdx.x * 8LL + (threadIdx.x >> 5); t < tasks; t += gridDim.x * 8LL) {
    if (t < rows_a) {
      stage_row<SHIFTED>(p.a + row(int(t)) * p.ld_a, p.bytes_a, p.order + t * p.pitch_a, p.pitch_a, lane);
      continue;
    }
    if constexpr (SHIFTED) {
      if (t < used) {
        const long long s = t - rows_a;
        stage_row<SHIFTED>(p.c + s * p.ld_c, p.bytes_c, p.order_c + s * p.pitch_c, p.pitch_c, lane);
        continue;
      }
      if (t >= slabs) {
        const long long part = t - slabs, r = part / p.w_parts;
        const int e = int(r / p.w_rows);
        if (start(e + 1) <= start(e)) continue;
        stage_row<SHIFTED>(p.w + e * p.stride_w + (r - static_cast<long long>(e) * p.w_rows) * p.ld_w +
                               (part - r * p.w_parts) * p.bytes_w,
                           p.bytes_w, p.mats + part * p.pitch_w, p.pitch_w, lane);
        continue;
      }
    }
    const int q = int(t - used), e = q / (2 * kSlab), r = (q >> 1) % kSlab;
    const int begin = start(e), end = max(begin, start(e + 1));
    if ((end - begin) % kSlab == 0) continue;
    const int s = begin + (end - begin) / kSlab * kSlab + r;
    const long long at = static_cast<long long>(e) * kSlab + r;
    if (q & 1)
      stage_row<SHIFTED>(s < end ? p.a + row(s) * p.ld_a : nullptr, p.bytes_a, p.slab_a + at * p.pitch_a, p.pitch_a, lane);
    else
      stage_row<SHIFTED>(s < end ? p.c + s * p.ld_c : nullptr, p.bytes_c, p.slab_c + at * p.pitch_c, p.pitch_c, lane);
  }
  grid_launch_dependents();
}

// Row pitch in bytes of staged rows: whole 128-byte lines.
int64_t staged_pitch(int64_t cols, int es) { return (cols * es + 127) / 128 * 128; }

int stage_rows(const CallContext& ctx, const StageRows& p, cudaStream_t stream) {
  const int64_t rows = (p.order != nullptr ? p.slots : 0) + (p.order_c != nullptr ? p.slots : 0) +
                       (p.slab_a != nullptr ? 2 * int64_t(p.groups) * kSlab : 0) +
                       (p.mats != nullptr ? int64_t(p.groups) * p.w_rows * p.w_parts : 0);
  const int64_t blocks = (rows + 7) / 8, most = int64_t(ctx.sm_count) * 8;
  const int grid = int(blocks < most ? blocks : most);
  const bool shifted = (p.a != nullptr && p.ld_a % 16 != 0) || (p.c != nullptr && p.ld_c % 16 != 0) ||
                       (p.w != nullptr && (p.ld_w | p.stride_w | (p.w_parts - 1) * p.bytes_w) % 16 != 0);
  const cudaError_t e = shifted ? launch_dependent(stage_rows_kernel<true>, grid, 256, 0, stream, 1, p)
                                : launch_dependent(stage_rows_kernel<false>, grid, 256, 0, stream, 1, p);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// The host knows the slots and the groups, not the group sizes, so its rules go by
// an average group. A group far above the average pays for that: 64 groups,
// 2048 x 4096 BF16, 960 rows (gathered) 171 us evenly spread and 213 with 700 in one
// group; 1100 rows (put in slot order first), 700 in one group, 178.
int64_t average_group(int64_t slots, int64_t groups) { return slots / (groups < slots ? groups : slots); }

// Named rows are put in slot order first from 16 rows a group on. 16 groups,
// 4096 x 4096 BF16, gathered on the way / staged: groups of 8 rows 92.6 / 93.9 us,
// 16 rows 104.7 / 98.4, 32 rows 138 / 99, 96 rows 351 / 115.
bool use_staging(int64_t slots, int64_t groups) { return average_group(slots, groups) >= 16; }

// A pair's 256-row tiles pay once an average group fills one CTA's 128 rows.
// 16 groups, 4096 x 4096 BF16, one CTA / a pair: groups of 64 rows 93 / 106 us,
// 96 rows 108 / 110, 128 rows 123 / 107, 256 rows 188 / 150; 64 groups, 2048 x 4096
// row-major: 96 rows 191 / 198, 128 rows 231 / 216.
bool use_pair(int64_t slots, int64_t groups) { return average_group(slots, groups) >= 128; }

// Tile rows per band: 8 row tiles of a group share each column tile's weights
// while those are in L2.
constexpr int kGroupRaster = 8;

// Bytes of the workspace for A's rows in slot order: those with names from 16 a group on, and all of a pitch that is
// not TMA's.
int64_t rows_workspace(int es, int64_t groups, int64_t slots, int64_t K, int64_t a_rows, int64_t lda, bool gathered) {
  const bool copied = odd_pitch(row_pitch(a_rows, K, lda, es), es) || (gathered && use_staging(slots, groups));
  return copied ? slots * staged_pitch(K, es) : 0;
}

// Weights that TMA cannot read where they are: rows or matrices off 16-byte multiples, or a value half that starts off
// one. They are copied, the groups with slots, in every call (a caller that keeps them aligned saves that: 16 tokens x
// 4 of 64 experts, gated row-major 2048 x 4090 BF16, 420 us against 113 for 2048 x 4096; 8192 tokens x 2 of 16, 4096 x
// 4090, 600 against 378. The copy runs at 6.3-6.9 TB/s.)
struct WeightCopy {
  int64_t rows, cols, ld;  // of W_e; ld as TMA may take it
  int parts;               // of a copied row
  int64_t pitch;           // of a copied part, bytes
  int64_t bytes;           // of the workspace: 0 where nothing is copied
};
// (The dense gated product copies the value half alone where that is all that is off: gated.cu.)
WeightCopy weight_copy(int es, int64_t groups, int64_t N, int64_t K, int64_t ldw, int64_t stride_w, bool row_major,
                       bool gated) {
  WeightCopy c;
  c.rows = row_major ? K : N;
  c.cols = row_major ? N : K;
  c.ld = row_pitch(c.rows, c.cols, ldw, es);
  c.parts = gated && row_major ? 2 : 1;
  c.pitch = staged_pitch(c.cols / c.parts, es);
  const bool odd = odd_pitch(c.ld, es) || (groups > 1 && odd_pitch(stride_w, es)) ||
                   (c.parts == 2 && odd_pitch(c.cols / 2, es));
  c.bytes = odd && K > 0 ? groups * c.rows * c.parts * c.pitch : 0;
  return c;
}

}  // namespace

int run_grouped(int kind, int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const void* A,
                int64_t a_rows, int64_t lda, const int32_t* rows, const void* W, int64_t ldw, int64_t stride_w, void* C,
                int64_t ldc, int layout, const gemm_grouped_epilogue_t* epi, void* workspace, int64_t workspace_bytes,
                void* stream, const DenseProduct* dense) {
  const int es = kind == KIND_E4M3 ? 1 : 2;
  if (groups < 1 || groups > kMaxGroups || slots < 0 || N < 0 || K < 0 || a_rows < 0 || slots > kIntLimit ||
      N > kIntLimit || K > kIntLimit || a_rows > kIntLimit)
    return GEMM_ERR_INVALID_VALUE;
  if (layout != GEMM_B_ROW_MAJOR && layout != GEMM_B_K_MAJOR) return GEMM_ERR_INVALID_VALUE;
  if (kind == KIND_E4M3 && layout != GEMM_B_K_MAJOR) return GEMM_ERR_INVALID_VALUE;
  const int act = epi != nullptr ? epi->activation : GEMM_ACT_NONE;
  if (act < GEMM_ACT_NONE || act > GEMM_ACT_SILU_GATED) return GEMM_ERR_INVALID_VALUE;
  const bool gated = act == GEMM_ACT_SILU_GATED || (dense != nullptr && dense->gate >= 0);
  if (gated && N % 2 != 0) return GEMM_ERR_INVALID_VALUE;
  if (slots == 0 || N == 0) return GEMM_OK;
  const int64_t out_cols = gated ? N / 2 : N;
  if ((offsets == nullptr && dense == nullptr) || C == nullptr || ldc < out_cols || ldc > kLdLimit)
    return GEMM_ERR_INVALID_VALUE;
  void* up = dense != nullptr ? dense->up : nullptr;
  const int64_t ldup = dense != nullptr ? dense->ldup : 0;
  if (up != nullptr && (ldup < N || ldup > kLdLimit)) return GEMM_ERR_INVALID_VALUE;
  if (rows == nullptr && a_rows < slots) return GEMM_ERR_INVALID_VALUE;
  // (with K = 0 rows of A may be named that it does not have: nothing of them is read but their scales)
  if (a_rows == 0 && epi != nullptr && epi->row_scale != nullptr) return GEMM_ERR_INVALID_VALUE;
  const int64_t w_rows = layout == GEMM_B_ROW_MAJOR ? K : N, w_cols = layout == GEMM_B_ROW_MAJOR ? N : K;
  if (K > 0) {
    if (A == nullptr || W == nullptr || a_rows == 0 || lda < K || ldw < w_cols || lda > kLdLimit || ldw > kLdLimit ||
        (groups > 1 && stride_w < (w_rows - 1) * ldw + w_cols) || stride_w < 0 || stride_w > kLdLimit)
      return GEMM_ERR_INVALID_VALUE;
  }
  if ((slots / 128 + groups + 1) * ((out_cols + 63) / 64) > kIntLimit) return GEMM_ERR_INVALID_VALUE;
  lda = row_pitch(a_rows, K, lda, es);
  const void* value = dense != nullptr ? dense->value : nullptr;  // (checked by the caller)
  const WeightCopy wc =
      weight_copy(es, groups, N, K, ldw, stride_w, layout == GEMM_B_ROW_MAJOR, gated && value == nullptr);
  ldw = wc.ld;
  const void* bias = epi != nullptr ? epi->bias : nullptr;
  const bool odd_a = K > 0 && odd_pitch(lda, es);
  if (K == 0 || (rows == nullptr && !odd_a && wc.bytes == 0)) workspace = nullptr;
  // A's rows come first in the workspace, then the weights. Named rows are gathered on the way where there is room for
  // the weights only.
  const int64_t a_bytes = slots * staged_pitch(K, es);
  bool copy_a = workspace != nullptr && (rows != nullptr || odd_a);
  if (wc.bytes > 0 && copy_a && !odd_a && workspace_bytes < a_bytes + wc.bytes) copy_a = false;
  if (workspace != nullptr && workspace_bytes < (copy_a ? a_bytes : 0) + wc.bytes)
    return odd_a || wc.bytes > 0 ? GEMM_ERR_MISALIGNED : GEMM_ERR_INVALID_VALUE;
  if (misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(C, 2) || misaligned(up, 2) || misaligned(bias, 2) ||
      misaligned(workspace, 128) ||
      (epi != nullptr && (misaligned(epi->row_scale, 4) || misaligned(epi->col_scale, 4))))
    return GEMM_ERR_MISALIGNED;
  if (K > 0 && (misaligned(A, 16) || misaligned(W, 16) || (workspace == nullptr && (odd_a || wc.bytes > 0))))
    return GEMM_ERR_MISALIGNED;
  const Range rc = range_of(C, slots, out_cols, ldc, 2);
  if (workspace != nullptr && meet(rc, range_of(workspace, 1, workspace_bytes, 0, 1))) return GEMM_ERR_INVALID_VALUE;
  if (K > 0 && (meet(rc, range_of(A, a_rows, K, lda, es)) ||
                meet(rc, range_of(W, w_rows, w_cols, ldw, es, groups, groups > 1 ? stride_w : 0))))
    return GEMM_ERR_INVALID_VALUE;
  if (up != nullptr) {
    const Range ru = range_of(up, slots, N, ldup, 2);
    if (meet(ru, rc) || (workspace != nullptr && meet(ru, range_of(workspace, 1, workspace_bytes, 0, 1))) ||
        (bias != nullptr && meet(ru, range_of(bias, 1, N, N, 2))) ||
        (K > 0 && (meet(ru, range_of(A, a_rows, K, lda, es)) || meet(ru, range_of(W, w_rows, w_cols, ldw, es)))))
      return GEMM_ERR_INVALID_VALUE;
  }

  CallContext ctx;
  int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  if (!on_device(C, ctx.dev) || (offsets != nullptr && !on_device(offsets, ctx.dev)) ||
      (rows != nullptr && !on_device(rows, ctx.dev)) || (up != nullptr && !on_device(up, ctx.dev)) || (bias != nullptr && !on_device(bias, ctx.dev)) || (workspace != nullptr && !on_device(workspace, ctx.dev)) || (K > 0 && (!on_device(A, ctx.dev) || !on_device(W, ctx.dev))))
    return GEMM_ERR_NOT_DEVICE_MEMORY;
  if (epi != nullptr && ((epi->row_scale != nullptr && !on_device(epi->row_scale, ctx.dev)) ||
                         (epi->col_scale != nullptr && !on_device(epi->col_scale, ctx.dev))))
    return GEMM_ERR_NOT_DEVICE_MEMORY;
  if (value != nullptr) {
    if (!on_device(value, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
    st = dense->copy(W, ldw, K, out_cols, dense->value, dense->ldv, static_cast<cudaStream_t>(stream));
    if (st != GEMM_OK) return st;
  }
  if (dense != nullptr && K > 0 && workspace == nullptr && few_rows(slots, out_cols, dense->few_columns, ctx.sm_count))
    return dense->few(kind == KIND_F16 ? GEMM_TYPE_F16 : GEMM_TYPE_BF16, slots, out_cols, K, A, lda, W, ldw,
                      layout == GEMM_B_ROW_MAJOR, value, dense->ldv, dense->gate, bias, C, ldc, up, ldup, ctx,
                      static_cast<cudaStream_t>(stream));
  GroupLaunch L;
  memset(&L, 0, sizeof(L));
  GroupParams& p = L.p;
  fill_common(ctx, p);
  p.offsets = offsets;
  p.groups = groups;
  p.slots = int(slots);
  p.rows = rows;
  p.a_rows = int(a_rows);
  p.row_scale = epi != nullptr ? epi->row_scale : nullptr;
  p.col_scale = epi != nullptr ? epi->col_scale : nullptr;
  p.g.alpha = epi != nullptr ? epi->alpha : 1.0f;
  p.g.bias = bias;
  p.g.act = act;
  p.plain = !gated && act == GEMM_ACT_NONE && bias == nullptr && p.row_scale == nullptr && p.col_scale == nullptr &&
            p.g.alpha == 1.0f;
  p.out_cols = int(out_cols);
  p.g.N = int(N);
  p.g.K = int(K);
  p.g.C = C;
  p.g.ldc = ldc;
  p.g.c_gran = store_granularity(C, ldc, 0);
  p.g.c_tma = p.g.c_gran == 16;
  p.g.num_kb = int((K * es + 127) / 128);
  p.g.raster = kGroupRaster;
  L.gated = gated;
  L.dev = ctx.dev;
  L.stream = static_cast<cudaStream_t>(stream);
  const int64_t active = groups < slots ? groups : slots;
  L.pair = use_pair(slots, groups);
  const int out_bn = (L.pair ? kGroupPairN : kGroupSingleN) / (gated ? 2 : 1);
  p.g.tiles_n = int((out_cols + out_bn - 1) / out_bn);
  const int64_t tiles = (slots / (L.pair ? 256 : 128) + active + 1) * p.g.tiles_n;  // at most
  const int64_t units = L.pair ? ctx.sm_count / 2 : ctx.sm_count;
  L.grid = int((tiles < units ? tiles : units) * (L.pair ? 2 : 1));

  const CUtensorMapDataType dt = map_type(kind);
  const uint32_t bk = 128 / es;
  p.value_at = int(N / 2);
  if (K > 0) {
    p.gather_a = rows != nullptr && !copy_a;
    StageRows q = {};
    q.offsets = offsets;
    q.groups = groups;
    q.slots = int(slots);
    if (copy_a) {
      q.a = static_cast<const uint8_t*>(A);
      q.ld_a = lda * es;
      q.bytes_a = K * es;
      q.pitch_a = staged_pitch(K, es);
      q.a_rows = int(a_rows);
      q.rows = rows;
      q.order = static_cast<uint8_t*>(workspace);
      A = workspace;
      lda = staged_pitch(K, es) / es;
    }
    int64_t w_cols_read = N;  // of row-major weights
    if (wc.bytes > 0) {
      q.w = static_cast<const uint8_t*>(W);
      q.ld_w = ldw * es;
      q.stride_w = groups > 1 ? stride_w * es : 0;
      q.bytes_w = wc.cols / wc.parts * es;
      q.pitch_w = wc.pitch;
      q.w_rows = int(wc.rows);
      q.w_parts = wc.parts;
      q.mats = static_cast<uint8_t*>(workspace) + (copy_a ? a_bytes : 0);
      W = q.mats;
      ldw = wc.parts * wc.pitch / es;
      stride_w = wc.rows * ldw;
      if (layout == GEMM_B_ROW_MAJOR) w_cols_read = ldw;
      if (wc.parts == 2) p.value_at = int(wc.pitch / es);
    }
    if (copy_a || wc.bytes > 0) {
      st = stage_rows(ctx, q, L.stream);
      if (st != GEMM_OK) return st;
    }
    const bool mapped =
        p.gather_a ? encode_map_2d(&L.tmA2, dt, A, K, a_rows, lda * es, bk, 1, CU_TENSOR_MAP_SWIZZLE_128B)
                   : encode_map_3d(&L.tmA, dt, A, K, slots, lda * es, 1, 0, bk, L.pair ? 128 : 32,
                                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (!mapped) return GEMM_ERR_DRIVER;
    const uint64_t mat = groups > 1 ? uint64_t(stride_w) * es : 0;
    bool ok;
    if (layout == GEMM_B_K_MAJOR) {
      const uint32_t box = L.pair ? kGroupPairN / 2 : gated ? kGroupSingleN / 2 : kGroupSingleN;
      ok = encode_map_3d(&L.tmB, dt, W, K, N, ldw * es, groups, mat, bk, box, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
      ok = encode_map_3d(&L.tmB, dt, W, w_cols_read, K, ldw * es, groups, mat, 128 / es, bk, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!ok) return GEMM_ERR_DRIVER;
    if (dense != nullptr && gated) {
      L.tmA2 = L.tmB;
      if (value != nullptr) {
        p.value_at = 0;
        if (!encode_map_3d(&L.tmA2, dt, value, out_cols, K, dense->ldv * es, 1, 0, 128 / es, bk, CU_TENSOR_MAP_SWIZZLE_128B))
          return GEMM_ERR_DRIVER;
      }
    }
  }
  if (p.g.c_tma && !encode_map_3d(&L.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT16, C, out_cols, slots, ldc * 2, 1, 0, 64, 32,
                                  CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  cudaError_t e;
  const bool km = layout == GEMM_B_K_MAJOR;
  if (dense != nullptr && gated) {
    p.gate = dense->gate;
    if (up != nullptr) {
      p.up = up;
      p.ldup = ldup;
      p.up_gran = store_granularity(up, ldup, 0);
      p.up_value_gran = store_granularity(static_cast<uint16_t*>(up) + out_cols, ldup, 0);
      if (p.up_gran == 16 && !encode_map_3d(&L.tmB2, CU_TENSOR_MAP_DATA_TYPE_UINT16, up, N, slots, ldup * 2, 1, 0, 64, 32,
                                            CU_TENSOR_MAP_SWIZZLE_128B))
        return GEMM_ERR_DRIVER;
      if (p.up_gran != 16) p.up_value_gran = p.up_value_gran == 16 ? 8 : p.up_value_gran;  // there is no map
    }
    e = kind == KIND_BF16 ? (km ? launch_gated_bf16_km(L) : launch_gated_bf16_rm(L))
                          : (km ? launch_gated_f16_km(L) : launch_gated_f16_rm(L));
  } else if (kind == KIND_E4M3)
    e = launch_group_e4m3_km(L);
  else if (kind == KIND_BF16)
    e = km ? launch_group_bf16_km(L) : launch_group_bf16_rm(L);
  else
    e = km ? launch_group_f16_km(L) : launch_group_f16_rm(L);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

namespace {

// The slabs, and the rows of A and of dC that are copied whole.
int64_t wgrad_workspace(int64_t groups, int64_t slots, int64_t N, int64_t K, bool copy_a, bool copy_c = false) {
  return groups * kSlab * (staged_pitch(N, 2) + staged_pitch(K, 2)) + (copy_a ? slots * staged_pitch(K, 2) : 0) +
         (copy_c ? slots * staged_pitch(N, 2) : 0);
}

}  // namespace

int64_t dense_wgrad_workspace(int64_t slots, int64_t N, int64_t K, int64_t lda, int64_t lddc) {
  return (odd_pitch(row_pitch(slots, K, lda, 2), 2) ? slots * staged_pitch(K, 2) : 0) +
         (odd_pitch(row_pitch(slots, N, lddc, 2), 2) ? slots * staged_pitch(N, 2) : 0);
}

int run_wgrad(int kind, int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const void* A,
              int64_t a_rows, int64_t lda, const int32_t* rows, const void* dC, int64_t lddc, void* dW, int64_t lddw,
              int64_t stride_dw, int layout, void* workspace, int64_t workspace_bytes, void* stream, bool dense) {
  if (groups < 1 || groups > kMaxGroups || slots < 0 || N < 0 || K < 0 || a_rows < 0 || slots > kIntLimit ||
      N > kIntLimit || K > kIntLimit || a_rows > kIntLimit)
    return GEMM_ERR_INVALID_VALUE;
  if (layout != GEMM_B_ROW_MAJOR && layout != GEMM_B_K_MAJOR) return GEMM_ERR_INVALID_VALUE;
  if (N == 0 || K == 0) return GEMM_OK;
  const bool km = layout == GEMM_B_K_MAJOR;
  const int64_t out_rows = km ? N : K, out_cols = km ? K : N;
  if ((offsets == nullptr && !dense) || dW == nullptr || lddw < out_cols || lddw > kLdLimit || stride_dw < 0 ||
      stride_dw > kLdLimit || (groups > 1 && stride_dw < (out_rows - 1) * lddw + out_cols))
    return GEMM_ERR_INVALID_VALUE;
  if (slots > 0 && (A == nullptr || dC == nullptr || a_rows == 0 || lda < K || lddc < N || lda > kLdLimit ||
                    lddc > kLdLimit || (rows == nullptr && a_rows < slots)))
    return GEMM_ERR_INVALID_VALUE;
  if (((out_rows + 255) / 256) * ((out_cols + 255) / 256) > kIntLimit / groups) return GEMM_ERR_INVALID_VALUE;
  lda = row_pitch(a_rows, K, lda, 2);
  lddc = row_pitch(slots, N, lddc, 2);
  const bool copy_a = rows != nullptr || odd_pitch(lda, 2), copy_c = odd_pitch(lddc, 2);
  if (slots == 0 || (dense && !copy_a && !copy_c)) workspace = nullptr;
  if (slots > 0 && !dense &&
      (workspace == nullptr || workspace_bytes < wgrad_workspace(groups, slots, N, K, rows != nullptr)))
    return GEMM_ERR_INVALID_VALUE;
  if (misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(dW, 2) || misaligned(workspace, 128))
    return GEMM_ERR_MISALIGNED;
  const int64_t need = dense ? dense_wgrad_workspace(slots, N, K, lda, lddc) : wgrad_workspace(groups, slots, N, K, copy_a, copy_c);
  if (slots > 0 && (misaligned(A, 16) || misaligned(dC, 16) || (need > 0 && (workspace == nullptr || workspace_bytes < need))))
    return GEMM_ERR_MISALIGNED;
  const Range rw = range_of(dW, out_rows, out_cols, lddw, 2, groups, groups > 1 ? stride_dw : 0);
  if (workspace != nullptr && meet(rw, range_of(workspace, 1, workspace_bytes, 0, 1))) return GEMM_ERR_INVALID_VALUE;
  if (slots > 0 && (meet(rw, range_of(A, a_rows, K, lda, 2)) || meet(rw, range_of(dC, slots, N, lddc, 2))))
    return GEMM_ERR_INVALID_VALUE;

  CallContext ctx;
  int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  if (!on_device(dW, ctx.dev) || (offsets != nullptr && !on_device(offsets, ctx.dev)) || (rows != nullptr && !on_device(rows, ctx.dev)) ||
      (workspace != nullptr && !on_device(workspace, ctx.dev)) ||
      (slots > 0 && (!on_device(A, ctx.dev) || !on_device(dC, ctx.dev))))
    return GEMM_ERR_NOT_DEVICE_MEMORY;
  GroupLaunch L;
  memset(&L, 0, sizeof(L));
  GroupParams& p = L.p;
  fill_common(ctx, p);
  p.offsets = offsets;
  p.groups = groups;
  p.slots = int(slots);
  p.rows = rows;
  p.a_rows = int(a_rows);
  p.plain = 1;
  p.out_rows = int(out_rows);
  p.out_cols = int(out_cols);
  p.g.C = dW;
  p.g.ldc = lddw;
  p.g.stride_c = groups > 1 ? stride_dw : 0;
  p.g.c_gran = store_granularity(dW, lddw, p.g.stride_c);
  p.g.c_tma = p.g.c_gran == 16;
  p.g.raster = kGroupRaster;
  p.g.tiles_m = int((out_rows + 255) / 256);
  p.g.tiles_n = int((out_cols + 255) / 256);
  L.pair = true;
  L.dev = ctx.dev;
  L.stream = static_cast<cudaStream_t>(stream);
  const int64_t tiles = int64_t(groups) * p.g.tiles_m * p.g.tiles_n;
  const int64_t units = ctx.sm_count / 2;
  L.grid = int(2 * (tiles < units ? tiles : units));
  const CUtensorMapDataType dt = map_type(kind);
  if (slots > 0) {
    // workspace: the groups' ragged slabs of dC and of A, then A's rows in slot order where the caller names them or
    // their pitch is not TMA's, then dC's rows where theirs is not
    StageRows q = {};
    q.a = static_cast<const uint8_t*>(A);
    q.c = static_cast<const uint8_t*>(dC);
    q.ld_a = lda * 2;
    q.ld_c = lddc * 2;
    q.bytes_a = K * 2;
    q.bytes_c = N * 2;
    q.pitch_a = staged_pitch(K, 2);
    q.pitch_c = staged_pitch(N, 2);
    q.a_rows = int(a_rows);
    q.rows = rows;
    q.offsets = offsets;
    q.groups = groups;
    q.slots = int(slots);
    uint8_t* next = static_cast<uint8_t*>(workspace);
    if (!dense) {  // (rows past a single group's end are past the tensors', where TMA reads zeros)
      q.slab_c = next;
      q.slab_a = q.slab_c + int64_t(groups) * kSlab * q.pitch_c;
      next = q.slab_a + int64_t(groups) * kSlab * q.pitch_a;
    }
    if (copy_a) {
      q.order = next;
      next += slots * q.pitch_a;
      A = q.order;
      lda = q.pitch_a / 2;
    }
    if (copy_c) {
      q.order_c = next;
      dC = q.order_c;
      lddc = q.pitch_c / 2;
    }
    if (!dense || copy_a || copy_c) st = stage_rows(ctx, q, L.stream);
    if (st != GEMM_OK) return st;
    // rows x cols with rows `ld` apart: 64-column blocks as the outer coordinate, two to a box, where the columns are
    // whole blocks (a block past the row's end would be memory past the matrix); else boxes of one block
    auto operand = [&](CUtensorMap* m, const void* base, int64_t cols, int64_t nrows, int64_t ld_bytes, int* wide) {
      *wide = cols % 64 == 0;
      return *wide ? encode_map_3d(m, dt, base, 64, nrows, ld_bytes, cols / 64, 128, 64, kSlab, CU_TENSOR_MAP_SWIZZLE_128B, 2)
                   : encode_map_3d(m, dt, base, cols, nrows, ld_bytes, 1, 0, 64, kSlab, CU_TENSOR_MAP_SWIZZLE_128B, 1);
    };
    auto slabs = [&](CUtensorMap* m, const void* base, int64_t pitch) {
      return encode_map_3d(m, dt, base, 64, int64_t(groups) * kSlab, pitch, pitch / 128, 128, 64, kSlab,
                           CU_TENSOR_MAP_SWIZZLE_128B, 2);
    };
    const bool ok = operand(km ? &L.tmA : &L.tmB, dC, N, slots, lddc * 2, km ? &p.wide_p : &p.wide_q) &&
                    operand(km ? &L.tmB : &L.tmA, A, K, slots, lda * 2, km ? &p.wide_q : &p.wide_p) &&
                    (dense || (slabs(km ? &L.tmA2 : &L.tmB2, q.slab_c, q.pitch_c) &&
                               slabs(km ? &L.tmB2 : &L.tmA2, q.slab_a, q.pitch_a)));
    if (!ok) return GEMM_ERR_DRIVER;
  }
  if (p.g.c_tma && !encode_map_3d(&L.tmC, CU_TENSOR_MAP_DATA_TYPE_UINT16, dW, out_cols, out_rows, lddw * 2, groups,
                                  uint64_t(p.g.stride_c) * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_ERR_DRIVER;
  const cudaError_t e = kind == KIND_BF16 ? launch_group_bf16_wgrad(L) : launch_group_f16_wgrad(L);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace dgt

extern "C" {

int64_t gemm_grouped_workspace(int type, int groups, int64_t slots, int64_t K) {
  if (groups < 1 || slots <= 0 || K <= 0 || !dgt::use_staging(slots, groups)) return 0;
  return slots * dgt::staged_pitch(K, type == GEMM_TYPE_E4M3 ? 1 : 2);
}

int64_t gemm_grouped_wgrad_workspace(int groups, int64_t slots, int64_t N, int64_t K, int gathered) {
  return groups < 1 || slots <= 0 || N <= 0 || K <= 0 ? 0 : dgt::wgrad_workspace(groups, slots, N, K, gathered != 0);
}

int64_t gemm_grouped_rows_workspace(int type, int groups, int64_t slots, int64_t K, int64_t a_rows, int64_t lda,
                                    int gathered) {
  if (groups < 1 || slots <= 0 || K <= 0) return 0;
  return dgt::rows_workspace(type == GEMM_TYPE_E4M3 ? 1 : 2, groups, slots, K, a_rows, lda, gathered != 0);
}

int64_t gemm_grouped_weights_workspace(int type, int groups, int64_t N, int64_t K, int64_t ldw, int64_t stride_w,
                                       int layout, int activation) {
  if (groups < 1 || N <= 0 || K <= 0) return 0;
  return dgt::weight_copy(type == GEMM_TYPE_E4M3 ? 1 : 2, groups, N, K, ldw, stride_w, layout == GEMM_B_ROW_MAJOR,
                          activation == GEMM_ACT_SILU_GATED)
      .bytes;
}

int64_t gemm_grouped_wgrad_rows_workspace(int groups, int64_t slots, int64_t N, int64_t K, int64_t a_rows, int64_t lda,
                                          int gathered, int64_t lddc) {
  if (groups < 1 || slots <= 0 || N <= 0 || K <= 0) return 0;
  return dgt::wgrad_workspace(groups, slots, N, K,
                              gathered != 0 || dgt::odd_pitch(dgt::row_pitch(a_rows, K, lda, 2), 2),
                              dgt::odd_pitch(dgt::row_pitch(slots, N, lddc, 2), 2));
}

int gemm_f16_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                     int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* W, int64_t ldw,
                     int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                     void* workspace, int64_t workspace_bytes, void* stream) {
  return dgt::run_grouped(dgt::KIND_F16, groups, offsets, slots, N, K, A, a_rows, lda, rows, W, ldw, stride_w, C, ldc,
                          layout, epilogue, workspace, workspace_bytes, stream, nullptr);
}

int gemm_bf16_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                      int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* W, int64_t ldw,
                      int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  return dgt::run_grouped(dgt::KIND_BF16, groups, offsets, slots, N, K, A, a_rows, lda, rows, W, ldw, stride_w, C, ldc,
                          layout, epilogue, workspace, workspace_bytes, stream, nullptr);
}

int gemm_e4m3_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint8_t* A,
                      int64_t a_rows, int64_t lda, const int32_t* rows, const uint8_t* W, int64_t ldw,
                      int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  return dgt::run_grouped(dgt::KIND_E4M3, groups, offsets, slots, N, K, A, a_rows, lda, rows, W, ldw, stride_w, C, ldc,
                          layout, epilogue, workspace, workspace_bytes, stream, nullptr);
}

int gemm_f16_grouped_wgrad(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                           int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* dC, int64_t lddc,
                           uint16_t* dW, int64_t lddw, int64_t stride_dw, int layout, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  return dgt::run_wgrad(dgt::KIND_F16, groups, offsets, slots, N, K, A, a_rows, lda, rows, dC, lddc, dW, lddw,
                        stride_dw, layout, workspace, workspace_bytes, stream, false);
}

int gemm_bf16_grouped_wgrad(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K,
                            const uint16_t* A, int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* dC,
                            int64_t lddc, uint16_t* dW, int64_t lddw, int64_t stride_dw, int layout, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  return dgt::run_wgrad(dgt::KIND_BF16, groups, offsets, slots, N, K, A, a_rows, lda, rows, dC, lddc, dW, lddw,
                        stride_dw, layout, workspace, workspace_bytes, stream, false);
}

}  // extern "C"
