// Weighted sum of a token's rows and its gradient (gemm_combine,
// gemm_combine_backward).
//
//   y[t] = residual[t] + sum_j w[t][j] z[slot[t][j]]
//   dz[slot[t][j]] = w[t][j] dy[t];  dw[t][j] = dy[t] . z[slot[t][j]]
//
// Bound by HBM: each row of z is read (and of dz written) once, by slot, as
// whole rows, so the gather costs no extra bytes. `tpt` threads take a token,
// one or more 16-byte pieces of its columns each; up to eight loads of rows are in flight per
// thread before the first is added, and they are added in the order of j. Rows
// that are not whole 16-byte pieces: contiguous matrices go by the pieces of
// the flat arrays (the *_flat kernels), anything else by single elements. The blocks stay on
// their SMs and walk the tokens: a token's slots are loaded while the rows of
// the one before are on their way, so that one memory latency, not two, stands
// between a block and its rows.
#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kMaxK = 32;
constexpr int kFlight = 8;  // rows of z a thread has in flight
constexpr int kThreads = 256;

struct CombineParams {
  const void* z;
  const int32_t* slots;
  const float* weights;
  const void* residual;
  void* y;
  long long ldz, ldr, ldy;
  int tokens, cols, k, nslots;
  int tpt, chunks;      // threads per token, column chunks per group of tokens
  long long work;       // groups of tokens x chunks
};

// Slots j0 .. j0 + N - 1 of a token (-1: none) and their weights.
template <int N>
struct Picks {
  int s[N];
  float w[N];

  __device__ __forceinline__ void load(const int32_t* slots, const float* weights, long long token, int k, int j0,
                                       int nslots, bool in) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = -1;
      w[j] = 0.0f;
      if (in && j0 + j < k) {
        const long long at = token * k + j0 + j;
        s[j] = slots[at];
        if (static_cast<uint32_t>(s[j]) >= static_cast<uint32_t>(nslots)) s[j] = -1;
        w[j] = weights != nullptr ? weights[at] : 1.0f;
      }
    }
  }
};

// PIECES of a row a thread, with a token's FLIGHT rows of each in flight: eight
// loads a thread whatever k is (k <= FLIGHT where a thread has several pieces).
// 8192 tokens x k x 4096 BF16 with a residual, one piece a thread against several:
// k 1 79.6 us and 29.2, k 2 83.3 and 40.3 (6.7 TB/s), k 4 90.5 and 61.0. 912 tokens, the limit for k 1: k 1 10.7 and
// 5.0, k 4 12.0 and 7.9; several were ahead below it too (228 tokens: 3.7 and 2.7, 4.4 and 3.8).
template <int TYPE, int VEC, int FLIGHT, int PIECES>
__global__ void __launch_bounds__(kThreads, 3) combine_kernel(const CombineParams p) {
  using P = Pack<TYPE, VEC>;
  using T = typename P::T;
  grid_dependency_wait();
  const int per_block = blockDim.x / p.tpt, sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt;
  const T* z = static_cast<const T*>(p.z);
  auto group = [&](long long u) { return p.chunks == 1 ? u : u / p.chunks; };
  long long u = blockIdx.x;
  long long token = group(u) * per_block + sub;
  Picks<FLIGHT> now;
  now.load(p.slots, p.weights, token, p.k, 0, p.nslots, u < p.work && token < p.tokens);
  for (; u < p.work; u += gridDim.x) {
    const long long next = group(u + gridDim.x) * per_block + sub;
    const int chunk = p.chunks == 1 ? 0 : int(u % p.chunks);
    const int col0 = (chunk * PIECES * p.tpt + tid) * VEC, step = p.tpt * VEC;
    const bool here = token < p.tokens;
    P res[PIECES];
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      res[q].zero();
      if (p.residual != nullptr && here && col0 + q * step < p.cols)
        res[q].stream(static_cast<const T*>(p.residual) + token * p.ldr + col0 + q * step);
    }
    auto finish = [&](int q) {
      if (!here || col0 + q * step >= p.cols) return;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += res[q].get(i);
      P out;
      out.set(acc);
      out.store(static_cast<T*>(p.y) + token * p.ldy + col0 + q * step);
    };
    if constexpr (PIECES == 1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    }
    Picks<FLIGHT> ahead;
    for (int j0 = 0; j0 < (PIECES == 1 ? p.k : 1); j0 += FLIGHT) {
      P row[PIECES][FLIGHT];
#pragma unroll
      for (int q = 0; q < PIECES; ++q)
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
          row[q][j].zero();
          if (here && col0 + q * step < p.cols && now.s[j] >= 0) row[q][j].stream(z + now.s[j] * p.ldz + col0 + q * step);
        }
      // the next slots: this token's, or the next one's
      const bool last = j0 + FLIGHT >= p.k;
      ahead.load(p.slots, p.weights, last ? next : token, p.k, last ? 0 : j0 + FLIGHT, p.nslots,
                 last ? u + gridDim.x < p.work && next < p.tokens : here);
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        if constexpr (PIECES > 1) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j)
          if (j0 + j < p.k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(now.w[j], row[q][j].get(i), acc[i]);
          }
        if constexpr (PIECES > 1) finish(q);
      }
      now = ahead;
    }
    if constexpr (PIECES == 1) finish(0);
    token = next;
  }
  grid_launch_dependents();
}

struct CombineGradParams {
  const void* dy;
  const void* z;
  const int32_t* slots;
  const float* weights;
  const int32_t* used;
  void* dz;
  float* dweights;
  long long lddy, ldz, lddz;
  int tokens, cols, k, nslots;
  int tpt;  // threads per token: 8, 16 or whole warps
};

// A block for each few tokens; tpt threads walk a token's columns, kFlight rows
// at a time (dy stays in L1 between the passes of a token with more rows). With
// many tokens a thread takes several pieces of each row, so that the slots and
// the dots' reductions cost it less (one piece each: 24 instructions an element,
// 55 us for 4099 tokens x 6 x 2048 BF16, 41.7 now), and where k is small PIECES of
// them at once, so that eight loads are in flight as well: 8192 tokens x k x 4096
// BF16, one and several at once: k 1 68.8 us and 40.3, k 2 80.9 and 54.4 (6.2 TB/s), k 4 107 and 92.7; 912 tokens
// 7.7 and 5.3, 8.6 and 7.3, 10.7 and 10.5.
template <int TYPE, int VEC, int FLIGHT, int PIECES>
__global__ void __launch_bounds__(kThreads, 3) combine_grad_kernel(const CombineGradParams p) {
  using P = Pack<TYPE, VEC>;
  using T = typename P::T;
  __shared__ float part[2][kThreads / 32][FLIGHT];
  grid_dependency_wait();
  const int sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt, lane = threadIdx.x & 31;
  const int per_block = blockDim.x / p.tpt;
  const T* z = static_cast<const T*>(p.z);
  T* dz = static_cast<T*>(p.dz);
  const long long token = static_cast<long long>(blockIdx.x) * per_block + sub;
  const bool in = token < p.tokens;
  int turn = 0;
  for (int j0 = 0; j0 < p.k; j0 += FLIGHT, turn ^= 1) {
    Picks<FLIGHT> pick;
    pick.load(p.slots, p.weights, token, p.k, j0, p.nslots, in);
    float dot[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) dot[j] = 0.0f;
    if (in) {
      const int step = p.tpt * VEC;
      for (int col0 = tid * VEC; col0 < p.cols; col0 += PIECES * step) {
        P d[PIECES], row[PIECES][FLIGHT];
#pragma unroll
        for (int q = 0; q < PIECES; ++q)
          if (col0 + q * step < p.cols) d[q].load(static_cast<const T*>(p.dy) + token * p.lddy + col0 + q * step);
        if (p.dweights != nullptr) {
#pragma unroll
          for (int q = 0; q < PIECES; ++q)
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j)
              if (pick.s[j] >= 0 && col0 + q * step < p.cols) row[q][j].stream(z + pick.s[j] * p.ldz + col0 + q * step);
        }
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
          const int col = col0 + q * step;
          if (col >= p.cols) continue;
          float g[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] = d[q].get(i);
#pragma unroll
          for (int j = 0; j < FLIGHT; ++j)
            if (pick.s[j] >= 0) {
              float o[VEC];
#pragma unroll
              for (int i = 0; i < VEC; ++i) o[i] = pick.w[j] * g[i];
              P out;
              out.set(o);
              out.store(dz + pick.s[j] * p.lddz + col);
            }
          if (p.dweights != nullptr) {
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j)
              if (pick.s[j] >= 0) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) dot[j] = fmaf(g[i], row[q][j].get(i), dot[j]);
              }
          }
        }
      }
    }
    if (p.dweights != nullptr) {
#pragma unroll
      for (int j = 0; j < FLIGHT; ++j)
        for (int d = (p.tpt < 32 ? p.tpt : 32) >> 1; d > 0; d >>= 1)
          dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
      if (p.tpt > 32) {
        // (the two halves of `part` alternate: one barrier a pass is enough)
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < FLIGHT; ++j) part[turn][threadIdx.x >> 5][j] = dot[j];
        }
        __syncthreads();
        if (tid < FLIGHT) {
          float sum = 0.0f;
          for (int i = 0; i < p.tpt >> 5; ++i) sum += part[turn][(threadIdx.x >> 5) + i][tid];
          if (in && j0 + tid < p.k) p.dweights[token * p.k + j0 + tid] = sum;
        }
      } else if (in && tid == 0) {
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j)
          if (j0 + j < p.k) p.dweights[token * p.k + j0 + j] = dot[j];
      }
    }
  }
  // rows of dz that no pair owns
  if (p.used != nullptr) {
    const int used = max(*p.used, 0);
    for (long long row = static_cast<long long>(used) + blockIdx.x; row < p.nslots; row += gridDim.x) {
      P o;
      o.zero();
      for (int col = threadIdx.x * VEC; col < p.cols; col += blockDim.x * VEC) o.store(dz + row * p.lddz + col);
    }
  }
  grid_launch_dependents();
}

// 16 bytes from element s (0 .. VEC) of the 32 that w holds; VEC elements are 16
// bytes. s is the same in every lane that calls this together.
template <int VEC>
__device__ __forceinline__ void shift_pieces(const uint32_t (&w)[8], int s, uint32_t* o) {
  constexpr int PER_WORD = VEC / 4;  // elements of a word
  const int r = (s % PER_WORD) * (32 / PER_WORD);
  switch (s / PER_WORD) {
    case 0:
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k], w[k + 1], r);
      break;
    case 1:
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k + 1], w[k + 2], r);
      break;
    case 2:
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k + 2], w[k + 3], r);
      break;
    case 3:
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k + 3], w[k < 3 ? k + 4 : 7], r);
      break;
    default:
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = w[k + 4];
      break;
  }
}

// VEC consecutive elements from element f >= 0 of a flat array that starts on a
// 16-byte boundary: the two 16-byte pieces that hold them, shifted together
// (element by element where the second piece would run past the array's
// `total` elements). f mod VEC is the same in every lane that calls this together.
template <int TYPE, int VEC>
__device__ __forceinline__ void load_across(Pack<TYPE, VEC>& out, const typename Elem<TYPE>::T* base, long long f,
                                            long long total) {
  const int m = static_cast<int>(f % VEC);
  const long long a = f - m;
  if (m == 0) {
    out.load(base + a);
    return;
  }
  if (a + 2 * VEC > total) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) out.v[i] = base[f + i];
    return;
  }
  const uint4 lo = *reinterpret_cast<const uint4*>(base + a);
  const uint4 hi = *reinterpret_cast<const uint4*>(base + a + VEC);
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  shift_pieces<VEC>(w, m, reinterpret_cast<uint32_t*>(out.v));
}

constexpr int kFlatFlight = 4;  // rows in flight of the flat kernels: each is two pieces

// combine over contiguous matrices whose rows are not whole pieces: a thread
// takes a 16-byte piece of the flat y; the row's first and last pieces, partly
// other rows', go element by element.
template <int TYPE>
__global__ void __launch_bounds__(kThreads, 3) combine_flat_kernel(const CombineParams p) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  grid_dependency_wait();
  const int per_block = blockDim.x / p.tpt, sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt;
  const T* z = static_cast<const T*>(p.z);
  const T* res = static_cast<const T*>(p.residual);
  T* y = static_cast<T*>(p.y);
  const long long total = static_cast<long long>(p.nslots) * p.cols;
  for (long long u = blockIdx.x; u < p.work; u += gridDim.x) {
    const long long token = u / p.chunks * per_block + sub;
    if (token >= p.tokens) continue;
    const long long row = token * p.cols;
    const int lo = (int(u % p.chunks) * p.tpt + tid) * VEC - static_cast<int>(row % VEC);
    if (lo >= p.cols) continue;
    const bool inside = lo >= 0 && lo + VEC <= p.cols;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += kFlight) {
      Picks<kFlight> pick;
      pick.load(p.slots, p.weights, token, p.k, j0, p.nslots, true);
#pragma unroll
      for (int h = 0; h < kFlight; h += kFlatFlight) {
        if (j0 + h >= p.k) break;
        P v[kFlatFlight];
#pragma unroll
        for (int j = 0; j < kFlatFlight; ++j) {
          v[j].zero();
          if (pick.s[h + j] < 0) continue;
          const long long f = static_cast<long long>(pick.s[h + j]) * p.cols + lo;
          if (inside) {
            load_across<TYPE, VEC>(v[j], z, f, total);
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (lo + i >= 0 && lo + i < p.cols) v[j].v[i] = z[f + i];
          }
        }
#pragma unroll
        for (int j = 0; j < kFlatFlight; ++j)
          if (j0 + h + j < p.k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(pick.w[h + j], v[j].get(i), acc[i]);
          }
      }
    }
    if (inside) {
      if (res != nullptr) {
        P r;
        r.load(res + row + lo);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] += r.get(i);
      }
      P out;
      out.set(acc);
      out.store(y + row + lo);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (lo + i >= 0 && lo + i < p.cols) {
          if (res != nullptr) acc[i] += Elem<TYPE>::get(res[row + lo + i]);
          y[row + lo + i] = Elem<TYPE>::put(acc[i]);
        }
    }
  }
  grid_launch_dependents();
}

// Its gradient: a thread takes 16-byte pieces of the flat z and dz (a row of
// both starts at the same place), and dy, which lies otherwise, from L1.
template <int TYPE>
__global__ void __launch_bounds__(kThreads, 3) combine_grad_flat_kernel(const CombineGradParams p) {
  using T = typename Elem<TYPE>::T;
  constexpr int VEC = 16 / sizeof(T);
  using P = Pack<TYPE, VEC>;
  __shared__ float part[2][kThreads / 32][kFlatFlight];
  grid_dependency_wait();
  const int sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt, lane = threadIdx.x & 31;
  const int per_block = blockDim.x / p.tpt;
  const T* z = static_cast<const T*>(p.z);
  const T* dy = static_cast<const T*>(p.dy);
  T* dz = static_cast<T*>(p.dz);
  const long long total = static_cast<long long>(p.tokens) * p.cols;
  const int pieces = (p.cols + VEC - 1) / VEC + 1;  // that a row meets at most
  int turn = 0;
  for (long long t0 = static_cast<long long>(blockIdx.x) * per_block; t0 < p.tokens;
       t0 += static_cast<long long>(gridDim.x) * per_block) {
    const long long token = t0 + sub;
    const bool in = token < p.tokens;
    for (int j0 = 0; j0 < p.k; j0 += kFlatFlight, turn ^= 1) {
      Picks<kFlatFlight> pick;
      pick.load(p.slots, p.weights, token, p.k, j0, p.nslots, in);
      float dot[kFlatFlight];
#pragma unroll
      for (int j = 0; j < kFlatFlight; ++j) dot[j] = 0.0f;
      for (int c = tid; c < pieces; c += p.tpt) {
        P v[kFlatFlight], d[kFlatFlight];
#pragma unroll
        for (int j = 0; j < kFlatFlight; ++j) {
          if (pick.s[j] < 0) continue;
          const long long row = static_cast<long long>(pick.s[j]) * p.cols;
          const int lo = c * VEC - static_cast<int>(row % VEC);
          if (lo < 0 || lo + VEC > p.cols) continue;
          v[j].zero();
          if (p.dweights != nullptr) v[j].stream(z + row + lo);
          load_across<TYPE, VEC>(d[j], dy, token * p.cols + lo, total);
        }
#pragma unroll
        for (int j = 0; j < kFlatFlight; ++j) {
          if (pick.s[j] < 0) continue;
          const long long row = static_cast<long long>(pick.s[j]) * p.cols;
          const int lo = c * VEC - static_cast<int>(row % VEC);
          if (lo >= 0 && lo + VEC <= p.cols) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              o[i] = pick.w[j] * d[j].get(i);
              dot[j] = fmaf(d[j].get(i), v[j].get(i), dot[j]);
            }
            P out;
            out.set(o);
            out.store(dz + row + lo);
          } else if (lo < p.cols) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (lo + i >= 0 && lo + i < p.cols) {
                const float g = Elem<TYPE>::get(dy[token * p.cols + lo + i]);
                if (p.dweights != nullptr) dot[j] = fmaf(g, Elem<TYPE>::get(z[row + lo + i]), dot[j]);
                dz[row + lo + i] = Elem<TYPE>::put(pick.w[j] * g);
              }
          }
        }
      }
      if (p.dweights != nullptr) {
#pragma unroll
        for (int j = 0; j < kFlatFlight; ++j)
          for (int d = (p.tpt < 32 ? p.tpt : 32) >> 1; d > 0; d >>= 1)
            dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
        if (p.tpt > 32) {
          if (lane == 0) {
#pragma unroll
            for (int j = 0; j < kFlatFlight; ++j) part[turn][threadIdx.x >> 5][j] = dot[j];
          }
          __syncthreads();
          if (tid < kFlatFlight) {
            float sum = 0.0f;
            for (int i = 0; i < p.tpt >> 5; ++i) sum += part[turn][(threadIdx.x >> 5) + i][tid];
            if (in && j0 + tid < p.k) p.dweights[token * p.k + j0 + tid] = sum;
          }
        } else if (in && tid == 0) {
#pragma unroll
          for (int j = 0; j < kFlatFlight; ++j)
            if (j0 + j < p.k) p.dweights[token * p.k + j0 + j] = dot[j];
        }
      }
    }
  }
  if (p.used != nullptr) {
    const long long first = static_cast<long long>(max(*p.used, 0)) * p.cols, end = static_cast<long long>(p.nslots) * p.cols;
    for (long long i = first + blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < end;
         i += static_cast<long long>(gridDim.x) * blockDim.x)
      dz[i] = Elem<TYPE>::put(0.0f);
  }
  grid_launch_dependents();
}

bool bad_type(int type) { return type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F32; }
bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 39); }
bool wide(const void* p, int64_t ld, int es) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * es)) % 16) == 0;
}
bool meet(const void* a, int64_t rows_a, int64_t ld_a, const void* b, int64_t rows_b, int64_t ld_b, int64_t cols, int es) {
  if (a == nullptr || b == nullptr || rows_a == 0 || rows_b == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), a1 = a0 + uintptr_t(((rows_a - 1) * ld_a + cols) * es);
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(b), b1 = b0 + uintptr_t(((rows_b - 1) * ld_b + cols) * es);
  return a0 < b1 && b0 < a1;
}

// Threads per token: 8, 16 or whole warps that cover its pieces in as few equal
// passes as 256 threads allow, or in `passes` where that is more.
int threads_per_token(int64_t nvec, int64_t passes = 1) {
  if (nvec <= 8) return 8;
  if (nvec <= 16) return 16;
  if (passes < (nvec + kThreads - 1) / kThreads) passes = (nvec + kThreads - 1) / kThreads;
  return int(((nvec + passes - 1) / passes + 31) / 32 * 32);
}

constexpr int64_t kInt = (int64_t(1) << 31) - 1;

// Pieces of a row a thread takes at once: one, or what makes eight loads with the token's k rows, where the tokens
// are enough to fill the GPU's threads that way.
int pieces_at_once(const CallContext& ctx, bool vec, int k, int64_t tokens, int64_t nvec) {
  const int pieces = k <= 2 ? 4 : k <= 4 ? 2 : 1;
  return vec && tokens * nvec >= int64_t(ctx.sm_count) * kThreads * 3 * pieces ? pieces : 1;
}

template <int TYPE>
cudaError_t launch_combine(const CombineParams& p, bool vec, bool flat, int pieces, int grid, int block, cudaStream_t s) {
  constexpr int VEC = 16 / int(sizeof(typename Elem<TYPE>::T));
  if (flat) return launch_dependent(combine_flat_kernel<TYPE>, grid, block, 0, s, 1, p);
  if (!vec) return launch_dependent(combine_kernel<TYPE, 1, kFlight, 1>, grid, block, 0, s, 1, p);
  return pieces == 4   ? launch_dependent(combine_kernel<TYPE, VEC, kFlight / 4, 4>, grid, block, 0, s, 1, p)
         : pieces == 2 ? launch_dependent(combine_kernel<TYPE, VEC, kFlight / 2, 2>, grid, block, 0, s, 1, p)
                       : launch_dependent(combine_kernel<TYPE, VEC, kFlight, 1>, grid, block, 0, s, 1, p);
}

template <int TYPE>
cudaError_t launch_combine_grad(const CombineGradParams& p, bool vec, bool flat, int pieces, int grid, int block,
                                cudaStream_t s) {
  constexpr int VEC = 16 / int(sizeof(typename Elem<TYPE>::T));
  if (flat) return launch_dependent(combine_grad_flat_kernel<TYPE>, grid, block, 0, s, 1, p);
  if (!vec) return launch_dependent(combine_grad_kernel<TYPE, 1, kFlight, 1>, grid, block, 0, s, 1, p);
  return pieces == 4   ? launch_dependent(combine_grad_kernel<TYPE, VEC, kFlight / 4, 4>, grid, block, 0, s, 1, p)
         : pieces == 2 ? launch_dependent(combine_grad_kernel<TYPE, VEC, kFlight / 2, 2>, grid, block, 0, s, 1, p)
                       : launch_dependent(combine_grad_kernel<TYPE, VEC, kFlight, 1>, grid, block, 0, s, 1, p);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_combine(int type, int64_t tokens, int64_t cols, int k, const void* z, int64_t ldz, int64_t nslots,
                 const int32_t* slots, const float* weights, const void* residual, int64_t ldr, void* y, int64_t ldy,
                 void* stream) {
  if (bad_type(type) || tokens < 0 || cols < 0 || nslots < 0 || k < 1 || k > kMaxK || tokens > kInt / k ||
      cols > (kInt >> 8) || nslots > kInt)
    return GEMM_ERR_INVALID_VALUE;
  if (tokens == 0 || cols == 0) return GEMM_OK;
  if ((nslots > 0 && (z == nullptr || bad_ld(ldz, cols))) || slots == nullptr || y == nullptr || bad_ld(ldy, cols) ||
      (residual != nullptr && bad_ld(ldr, cols)))
    return GEMM_ERR_INVALID_VALUE;
  const int es = type_bytes(type);
  if (misaligned(z, es) || misaligned(y, es) || misaligned(residual, es) || misaligned(slots, 4) ||
      misaligned(weights, 4))
    return GEMM_ERR_MISALIGNED;
  if (meet(y, tokens, ldy, z, nslots, ldz, cols, es) ||
      (!(y == residual && ldy == ldr) && meet(y, tokens, ldy, residual, tokens, ldr, cols, es)))
    return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[5] = {nslots > 0 ? z : nullptr, slots, y, weights, residual};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  const int v = 16 / es;
  const bool vec = cols % v == 0 && (nslots == 0 || wide(z, ldz, es)) && wide(y, ldy, es) &&
                   (residual == nullptr || wide(residual, ldr, es));
  auto flat_matrix = [&](const void* m, int64_t ld) {
    return m == nullptr || (ld == cols && reinterpret_cast<uintptr_t>(m) % 16 == 0);
  };
  const bool flat = !vec && cols >= v && flat_matrix(z, ldz) && flat_matrix(y, ldy) && flat_matrix(residual, ldr);
  const int64_t nvec = vec ? cols / v : flat ? (cols + v - 1) / v + 1 : cols;
  const int pieces = pieces_at_once(ctx, vec, k, tokens, nvec);
  CombineParams p = {z, slots, weights, residual, y, (long long)ldz, (long long)ldr, (long long)ldy, int(tokens),
                     int(cols), k, int(nslots), threads_per_token(nvec, pieces), 1, 0};
  p.chunks = int((nvec + int64_t(p.tpt) * pieces - 1) / (int64_t(p.tpt) * pieces));
  const int block = kThreads / p.tpt * p.tpt;
  p.work = (tokens + block / p.tpt - 1) / (block / p.tpt) * p.chunks;
  // as many blocks as are resident at once; the flat kernel has nothing to load ahead and takes a block for each group
  const int64_t most = flat ? kInt : int64_t(ctx.sm_count) * (3 * kThreads / block);
  const int grid = int(p.work < most ? p.work : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_combine<GEMM_TYPE_F16>(p, vec, flat, pieces, grid, block, s)
                        : type == GEMM_TYPE_BF16 ? launch_combine<GEMM_TYPE_BF16>(p, vec, flat, pieces, grid, block, s)
                                                 : launch_combine<GEMM_TYPE_F32>(p, vec, flat, pieces, grid, block, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_combine_backward(int type, int64_t tokens, int64_t cols, int k, const void* dy, int64_t lddy, const void* z,
                          int64_t ldz, int64_t nslots, const int32_t* slots, const float* weights,
                          const int32_t* used, void* dz, int64_t lddz, float* dweights, void* stream) {
  if (bad_type(type) || tokens < 0 || cols < 0 || nslots < 0 || k < 1 || k > kMaxK || tokens > kInt / k ||
      cols > (kInt >> 8) || nslots > kInt)
    return GEMM_ERR_INVALID_VALUE;
  if (cols == 0 && dweights == nullptr) return GEMM_OK;
  if (tokens == 0 && (nslots == 0 || used == nullptr)) return GEMM_OK;
  if (tokens > 0 && (slots == nullptr || (cols > 0 && (dy == nullptr || bad_ld(lddy, cols)))))
    return GEMM_ERR_INVALID_VALUE;
  if (nslots > 0 && cols > 0 && (dz == nullptr || bad_ld(lddz, cols) || (dweights != nullptr && (z == nullptr || bad_ld(ldz, cols)))))
    return GEMM_ERR_INVALID_VALUE;
  const int es = type_bytes(type);
  if (misaligned(z, es) || misaligned(dy, es) || misaligned(dz, es) || misaligned(slots, 4) ||
      misaligned(weights, 4) || misaligned(used, 4) || misaligned(dweights, 4))
    return GEMM_ERR_MISALIGNED;
  if (cols > 0 && (meet(dz, nslots, lddz, dy, tokens, lddy, cols, es) || meet(dz, nslots, lddz, z, nslots, ldz, cols, es)))
    return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  const int st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[7] = {dy, slots, nslots > 0 ? dz : nullptr, weights, used, dweights,
                         dweights != nullptr && nslots > 0 ? z : nullptr};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  const int v = 16 / es;
  const bool vec = cols % v == 0 && wide(dy, lddy, es) && wide(dz, lddz, es) && (dweights == nullptr || wide(z, ldz, es));
  auto flat_matrix = [&](const void* m, int64_t ld) { return ld == cols && reinterpret_cast<uintptr_t>(m) % 16 == 0; };
  const bool flat = !vec && cols >= v && flat_matrix(dy, lddy) && flat_matrix(dz, lddz) &&
                    (dweights == nullptr || flat_matrix(z, ldz));
  const int64_t nvec = vec ? cols / v : flat ? (cols + v - 1) / v + 1 : cols;
  // four pieces a thread once the tokens fill the GPU's threads that way: one / four, k 8 x 4096 BF16, us: 228 tokens
  // 7.9 / 9.7, 456 11.0 / 11.8, 912 (the limit) 20.3 / 17.8, 8192 179 / 178
  const int64_t passes = tokens * nvec >= int64_t(ctx.sm_count) * kThreads * 3 * 4 ? 4 : 1;
  const int pieces = pieces_at_once(ctx, vec, k, tokens, nvec);
  CombineGradParams p = {dy, z, slots, weights, used, dz, dweights, (long long)lddy, (long long)ldz, (long long)lddz,
                         int(tokens), int(cols), k, int(nslots), threads_per_token(nvec, passes)};
  const int block = kThreads / p.tpt * p.tpt;
  const int64_t need = (tokens + block / p.tpt - 1) / (block / p.tpt);
  // a block for each few tokens
  const int grid = int(need > 0 ? need : ctx.sm_count);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GEMM_TYPE_F16    ? launch_combine_grad<GEMM_TYPE_F16>(p, vec, flat, pieces, grid, block, s)
                        : type == GEMM_TYPE_BF16 ? launch_combine_grad<GEMM_TYPE_BF16>(p, vec, flat, pieces, grid, block, s)
                                                 : launch_combine_grad<GEMM_TYPE_F32>(p, vec, flat, pieces, grid, block, s);
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
