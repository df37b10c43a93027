// Routing to experts: scores, choice, weights and the expert order
// (gemm_route), and the gradient of the weights (gemm_route_backward).
//
// A warp takes a token: lane l holds the scores of experts l, l + 32, ..., sorts
// its keys (up to eight of them) and the warp takes the k largest one after
// another: a warp maximum of the lanes' heads, whose owner moves its list up. The
// softmax denominator is summed by halves -- within a lane, then across lanes
// 16, 8, 4, 2, 1 apart -- which with zeros past the last expert is the order of
// any power-of-two length, so the same logits give the same keys in every build
// of the kernel.
//
// The expert order is a stable counting sort of the token-major pairs: the pairs
// of every expert are counted, the counts summed over the experts, and a pair's
// place is its expert's start plus its rank among the block's pairs of that
// expert. The rank comes from bit masks in shared memory: each pair sets its bit
// in its expert's row, and counts the bits before it. Up to 32 tokens: one block
// does everything in one launch. More: the first launch leaves each block's
// count per expert, and in the second a block adds the counts of the blocks
// before it. (Ranking by match_any over 32 pairs at a time: 16 tokens x 8 of
// 256 experts 12.1 us; comparing each pair with every other 11.1 us.)
//
// The bytes are few (one read of the logits); the time is the selection's
// instructions and, for a serving step, latency. One launch (CUDA graph, FP32 sigmoid with a bias): 1 token of 32
// experts, k 1 3.6 us; of 256 6.2; 16 tokens 7.2; k 8 8.2; 4 of 8 groups 10.1. Two launches (BF16
// softmax): 33 tokens of 16, k 2 6.8 us; 16384 of 32, k 1 11.9; of 128 18.1; k 8 21.6.
#include <math.h>

#include "elem.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxK = 32;
// Blocks of the two-launch form, at most: one for each SM of a GB300 (a number, since the size of the workspace goes by
// it, on a machine without a GPU too). 76 / 152 / 304 blocks, us: 8192 x 16, k 2 12.6 / 9.3 / 14.1; 16384 x 128, k 8
// 34.6 / 21.8 / 30.2; 65536 x 128, k 8 120 / 65 / 72.
constexpr int kMaxBlocks = 152;
constexpr int kOneBlockTokens = 32;  // a warp each; more go to several blocks (128 tokens of 64 experts: 13.8 us in one)
constexpr int kMaskWords = 8192;     // of the ranking's bit masks: 32 KB

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* slots;
  int32_t* rows;
  int32_t* offsets;
  int32_t* counts;  // two-launch form: blocks x experts
  long long ld;
  int type, tokens, experts, k, score, groups, kept, renormalize, per_block, blocks;
  float scale;
};

__device__ __forceinline__ float load_logit(const void* p, int type, long long at) {
  if (type == GEMM_TYPE_F32) return static_cast<const float*>(p)[at];
  if (type == GEMM_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  return __half2float(static_cast<const __half*>(p)[at]);
}

// Order-preserving map of a float to an unsigned number (+-0 alike); 0 is below every number's image.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

// Sum of x[j] over all lanes and j by halves (see above).
template <int NPL>
__device__ __forceinline__ float halves_sum(const float (&e)[NPL]) {
  float x[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) x[j] = e[j];
#pragma unroll
  for (int w = NPL / 2; w > 0; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) x[j] = x[j] + x[j + w];
  return warp_sum(x[0]);
}

// The score of one logit above -inf, from the token's largest logit and its softmax denominator.
__device__ __forceinline__ float one_score(float l, int score, float top, float div) {
  return score == GEMM_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / div;
}

// The scores of one token: lane l's s[j] is expert l + 32 j (0 past the last
// one and for a logit of -inf); `there`: bit j set where the logit is above -inf.
template <int NPL>
__device__ __forceinline__ void token_scores(const void* logits, int type, long long base, int experts, int score,
                                             int lane, float (&s)[NPL], uint32_t& there, float& top, float& div) {
  top = -INFINITY;
  div = 1.0f;
  there = 0;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = lane + 32 * j;
    s[j] = e < experts ? load_logit(logits, type, base + e) : -INFINITY;
    if (!(s[j] == -INFINITY)) there |= 1u << j;
    top = fmaxf(top, s[j]);
  }
  if (score == GEMM_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) s[j] = (there >> j) & 1u ? one_score(s[j], score, top, div) : 0.0f;
    return;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll
  for (int j = 0; j < NPL; ++j) s[j] = (there >> j) & 1u ? expf(s[j] - top) : 0.0f;
  const float z = halves_sum(s);
  div = z == 0.0f ? 1.0f : z;
#pragma unroll
  for (int j = 0; j < NPL; ++j) s[j] = s[j] / div;
}

// The warp's largest of the lanes' candidates (key `best` of expert `e`; 0: none) goes to the lowest expert; returns its
// lane, or -1 if there is none, and the expert.
__device__ __forceinline__ int take_largest(uint32_t best, int e, int& won) {
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
  if (m == 0) return -1;
  const uint32_t who = __ballot_sync(0xFFFFFFFFu, best == m);
  int owner = __ffs(who) - 1;
  if (who & (who - 1)) owner = int(__reduce_min_sync(0xFFFFFFFFu, best == m ? uint32_t(e) : 0xFFFFFFFFu)) & 31;
  won = __shfl_sync(0xFFFFFFFFu, e, owner);
  return owner;
}

// Chooses one token's experts; lane i < k returns the i-th id (-1: none) and its weight.
template <int NPL>
__device__ __forceinline__ void route_token(const RouteParams& p, int token, int lane, int& id, float& weight) {
  const long long base = token * p.ld;
  float top, div;
  uint32_t u[NPL];  // the keys' order; 0: out
  bool nan = false;
  uint32_t kept = 0xFFFFFFFFu;
  const int per = p.experts / p.groups;
  {
    float key[NPL];
    uint32_t there;
    token_scores<NPL>(p.logits, p.type, base, p.experts, p.score, lane, key, there, top, div);
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      float v = -INFINITY;
      if ((there >> j) & 1u) {
        v = p.bias != nullptr ? key[j] + p.bias[lane + 32 * j] : key[j];
        nan = nan || key[j] != key[j];
        if (v != v) v = -INFINITY;
      }
      key[j] = v;
    }
    if (p.groups > 1) {
      // lane g gets group g's key: the sum of its two largest
      float mine = -INFINITY;
      if (per % 32 == 0) {
        // groups of whole rows of 32: the two largest of each row over the lanes, then of the group's rows
        float first = -INFINITY, second = -INFINITY;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          const uint32_t o = order_bits(key[j]);
          const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, o);
          const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, o == m1)) - 1;
          const uint32_t m2 = __reduce_max_sync(0xFFFFFFFFu, lane == owner ? 0u : o);
          const float a = order_value(m1), b = order_value(m2);
          if (32 * j / per == lane) {
            second = fmaxf(fmaxf(second, b), fminf(first, a));
            first = fmaxf(first, a);
          }
        }
        mine = first + second;
      } else {
        for (int g = 0; g < p.groups; ++g) {
          float a = -INFINITY, b = -INFINITY;  // this lane's two largest keys of the group
#pragma unroll
          for (int j = 0; j < NPL; ++j)
            if (lane + 32 * j >= g * per && lane + 32 * j < (g + 1) * per) {
              b = fmaxf(b, fminf(a, key[j]));
              a = fmaxf(a, key[j]);
            }
          // the largest of all lanes; its (first) owner puts its second one forward
          const uint32_t ua = order_bits(a);
          const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, ua);
          const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, ua == m1)) - 1;
          const uint32_t m2 = __reduce_max_sync(0xFFFFFFFFu, lane == owner ? order_bits(b) : ua);
          if (lane == g) mine = per > 1 ? order_value(m1) + order_value(m2) : order_value(m1);
        }
      }
      uint32_t best = lane < p.groups ? order_bits(mine) : 0u;
      kept = 0;
      for (int i = 0; i < p.kept; ++i) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
        const int g = __ffs(__ballot_sync(0xFFFFFFFFu, best == m)) - 1;
        kept |= 1u << g;
        if (lane == g) best = 0;
      }
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      u[j] = key[j] > -INFINITY ? order_bits(key[j]) : 0u;
      if (p.groups > 1 && !((kept >> ((lane + 32 * j) / per)) & 1u)) u[j] = 0;
    }
  }
  nan = __any_sync(0xFFFFFFFFu, nan);
  id = -1;
  if constexpr (NPL <= 8) {
    // in descending order, equal keys as they are (the lower expert first)
    int e[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) e[j] = lane + 32 * j;
#pragma unroll
    for (int a = NPL - 1; a > 0; --a)
#pragma unroll
      for (int j = 0; j < a; ++j) {
        const bool swap = u[j + 1] > u[j];
        const uint32_t hi = max(u[j], u[j + 1]), lo = min(u[j], u[j + 1]);
        const int eh = swap ? e[j + 1] : e[j], el = swap ? e[j] : e[j + 1];
        u[j] = hi;
        u[j + 1] = lo;
        e[j] = eh;
        e[j + 1] = el;
      }
    for (int i = 0; i < p.k; ++i) {
      int won;
      const int owner = take_largest(u[0], e[0], won);
      if (owner < 0) break;
      if (lane == i) id = won;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j + 1 < NPL; ++j) {
          u[j] = u[j + 1];
          e[j] = e[j + 1];
        }
        u[NPL - 1] = 0;
      }
    }
  } else {
    for (int i = 0; i < p.k; ++i) {
      uint32_t best = 0;
      int at = 0, won;
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (u[j] > best) {
          best = u[j];
          at = j;
        }
      const int owner = take_largest(best, lane + 32 * at, won);
      if (owner < 0) break;
      if (lane == i) id = won;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
          if (j == at) u[j] = 0;
      }
    }
  }
  // the chosen scores, from their logits once more (the same operations, so the same bits)
  weight = id >= 0 ? one_score(load_logit(p.logits, p.type, base + id), p.score, top, div) : 0.0f;
  if (p.renormalize) weight = weight / (warp_sum(weight) + 1e-20f);
  weight *= p.scale;
  if (nan) weight = __int_as_float(0x7FC00000);
}

// Places the block's n pairs (experts `ids`, -1: none; the first one is pair
// `first` of all): slots[i] and the slots' tokens. start[e]: the place of the block's first pair of
// expert e (used up). Block-collective; masks: kMaskWords words.
__device__ __forceinline__ void place_pairs(const RouteParams& p, const int32_t* ids, int n, long long first,
                                            int32_t* start, uint32_t* masks) {
  const int words = min((n + 31) / 32, kMaskWords / p.experts);  // per expert and pass
  for (int i0 = 0; i0 < n; i0 += 32 * words) {
    const int m = min(n - i0, 32 * words);
    for (int i = threadIdx.x; i < words * p.experts; i += blockDim.x) masks[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
      const int e = ids[i0 + i];
      if (e >= 0) atomicOr(&masks[(i >> 5) * p.experts + e], 1u << (i & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
      const int e = ids[i0 + i];
      int slot = -1;
      if (e >= 0) {
        slot = start[e] + __popc(masks[(i >> 5) * p.experts + e] & ((1u << (i & 31)) - 1u));
        for (int w = 0; w < i >> 5; ++w) slot += __popc(masks[w * p.experts + e]);
        p.rows[slot] = int((first + i0 + i) / p.k);
      }
      p.slots[first + i0 + i] = slot;
    }
    __syncthreads();
    if (i0 + m < n) {
      for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
        for (int w = 0; w < words; ++w) start[e] += __popc(masks[w * p.experts + e]);
      __syncthreads();
    }
  }
}

// Exclusive sum over the threads of the block; `sums` holds a value per warp.
__device__ __forceinline__ int block_exclusive(int v, int32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = lane < int(blockDim.x >> 5) ? sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
    if (lane >= d) before += o;
  }
  return incl - v + (warp > 0 ? __shfl_sync(0xFFFFFFFFu, before, warp - 1) : 0);
}

// The experts' starts from their counts: start[e] = sum of the counts before e
// (+ add[e]); offsets as well where they are wanted. Returns the sum of all counts. Block-collective.
__device__ __forceinline__ int expert_starts(const RouteParams& p, const int32_t* count, const int32_t* add,
                                             int32_t* start, bool offsets, int32_t* sums, int32_t* total) {
  const int per = (p.experts + blockDim.x - 1) / blockDim.x;
  int sum = 0;
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e < p.experts) sum += count[e];
  }
  int at = block_exclusive(sum, sums);
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e >= p.experts) break;
    const int c = count[e];
    if (offsets) p.offsets[e] = at;
    start[e] = at + (add != nullptr ? add[e] : 0);
    at += c;
    if (e == p.experts - 1) {
      *total = at;
      if (offsets) p.offsets[p.experts] = at;
    }
  }
  __syncthreads();
  return *total;
}

constexpr int kLeastThreads = 256;
template <int NPL>
constexpr int kRouteThreads = NPL <= 8 ? 1024 : NPL == 16 ? 512 : 256;  // by the registers of a lane's scores

// Tokens of the block: [first, first + the result). (first + per_block may pass 2^31 in the last block.)
__device__ __forceinline__ int block_tokens(const RouteParams& p, int& first) {
  const long long at = static_cast<long long>(blockIdx.x) * p.per_block, left = p.tokens - at;
  first = static_cast<int>(at);
  return static_cast<int>(left < p.per_block ? (left < 0 ? 0 : left) : p.per_block);
}

// One-block form: chooses, then orders the pairs.
// Two-launch form (p.blocks > 1): chooses and leaves the block's counts.
template <int NPL>
__global__ void __launch_bounds__(kRouteThreads<NPL>, 1) route_kernel(const RouteParams p) {
  __shared__ uint32_t masks[kMaskWords];
  __shared__ int32_t count[32 * NPL], start[32 * NPL];
  __shared__ int32_t chosen[kOneBlockTokens * kMaxK];
  __shared__ int32_t sums[32], total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool alone = p.blocks == 1;
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) count[e] = 0;
  grid_dependency_wait();
  __syncthreads();
  int t0;
  const int tokens = block_tokens(p, t0);
  for (int i = warp; i < tokens; i += warps) {
    const int t = t0 + i;
    int id;
    float w;
    route_token<NPL>(p, t, lane, id, w);
    if (lane < p.k) {
      p.ids[static_cast<long long>(t) * p.k + lane] = id;
      p.weights[static_cast<long long>(t) * p.k + lane] = w;
      if (id >= 0) atomicAdd(&count[id], 1);  // whole numbers: any order gives the same count
      if (alone) chosen[t * p.k + lane] = id;
    }
  }
  __syncthreads();
  if (!alone) {
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
      p.counts[static_cast<long long>(blockIdx.x) * p.experts + e] = count[e];
    grid_launch_dependents();
    return;
  }
  const int n = p.tokens * p.k;
  const int used = expert_starts(p, count, nullptr, start, true, sums, &total);
  place_pairs(p, chosen, n, 0, start, masks);
  for (int i = used + threadIdx.x; i < n; i += blockDim.x) p.rows[i] = -1;
  grid_launch_dependents();
}

// Second launch of the two-launch form: block b places its pairs.
__global__ void __launch_bounds__(1024, 1) route_place_kernel(const RouteParams p) {
  __shared__ uint32_t masks[kMaskWords];
  __shared__ int32_t all[kMaxExperts], before[kMaxExperts];
  __shared__ int32_t sums[32], total;
  int t0;
  const int n = block_tokens(p, t0) * p.k;
  const long long first = static_cast<long long>(t0) * p.k;
  for (int e = threadIdx.x; e < p.experts; e += blockDim.x) all[e] = before[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  // counts of all blocks and of those before this one: the threads split (block, expert) in whole rows
  const int parts = max(1, int(blockDim.x) / p.experts);
  for (int q = threadIdx.x; q < parts * p.experts; q += blockDim.x) {
    const int e = q % p.experts, part = q / p.experts;
    int sum = 0, ahead = 0;
#pragma unroll 8
    for (int b = part; b < p.blocks; b += parts) {
      const int c = __ldcg(p.counts + static_cast<long long>(b) * p.experts + e);
      sum += c;
      ahead += b < int(blockIdx.x) ? c : 0;
    }
    atomicAdd(&all[e], sum);
    atomicAdd(&before[e], ahead);
  }
  __syncthreads();
  const int used = expert_starts(p, all, before, before, blockIdx.x == 0, sums, &total);
  place_pairs(p, p.ids + first, n, first, before, masks);
  const long long pairs = static_cast<long long>(p.tokens) * p.k;
  for (long long i = used + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < pairs;
       i += static_cast<long long>(gridDim.x) * blockDim.x)
    p.rows[i] = -1;
  grid_launch_dependents();
}

// dlogits of one token: the weights' gradient through the renormalisation,
// then through the scores. With c = sum of the chosen scores + 1e-20 and
// w_j = scale s_j / c: ds_j = (scale dw_j - sum_i dw_i w_i) / c; without
// renormalisation ds_j = scale dw_j. Softmax: dl_e = s_e (ds_e - sum_i ds_i s_i)
// (ds = 0 off the choice); sigmoid: dl_e = ds_e s_e (1 - s_e).
template <int NPL>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteParams p, const float* dweights, void* dlogits,
                                                         long long ldd) {
  __shared__ float rows[8][32 * NPL];
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  for (long long t = (blockIdx.x * 256LL + threadIdx.x) >> 5; t < p.tokens; t += gridDim.x * 8LL) {
    float s[NPL], ds[NPL];
    uint32_t there;
    float top, div;
    token_scores<NPL>(p.logits, p.type, t * p.ld, p.experts, p.score, lane, s, there, top, div);
    int id = -1;
    float dw = 0.0f;
    if (lane < p.k) {
      id = p.ids[t * p.k + lane];
      if (id < 0 || id >= p.experts) id = -1;
      if (id >= 0) dw = dweights[t * p.k + lane] * p.scale;
    }
    // the chosen scores, and their gradients, change lanes through the warp's row of shared memory
    float* row = rows[threadIdx.x >> 5];
#pragma unroll
    for (int j = 0; j < NPL; ++j) row[lane + 32 * j] = s[j];
    __syncwarp();
    const float chosen = id >= 0 ? row[id] : 0.0f;  // lane i: the score of the i-th choice
    float d = dw;
    if (p.renormalize) {
      const float c = warp_sum(chosen) + 1e-20f;
      const float mean = warp_sum(dw * (chosen / c));
      d = id >= 0 ? (dw - mean) / c : 0.0f;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NPL; ++j) row[lane + 32 * j] = 0.0f;
    __syncwarp();
    if (id >= 0) row[id] = d;  // a token's ids are distinct
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NPL; ++j) ds[j] = row[lane + 32 * j];
    __syncwarp();
    float dot = 0.0f;
    if (p.score == GEMM_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < NPL; ++j) dot += ds[j] * s[j];
      dot = warp_sum(dot);
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = lane + 32 * j;
      if (e >= p.experts) continue;
      const float g = p.score == GEMM_SCORE_SOFTMAX ? s[j] * (ds[j] - dot) : ds[j] * s[j] * (1.0f - s[j]);
      const long long at = t * ldd + e;
      if (p.type == GEMM_TYPE_F32)
        static_cast<float*>(dlogits)[at] = g;
      else if (p.type == GEMM_TYPE_BF16)
        static_cast<__nv_bfloat16*>(dlogits)[at] = __float2bfloat16_rn(g);
      else
        static_cast<__half*>(dlogits)[at] = __float2half_rn(g);
    }
  }
  grid_launch_dependents();
}

bool bad_type(int type) { return type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F32; }
bool misaligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) % size) != 0; }

// Registers of scores per lane: the smallest build that covers the experts.
int scores_per_lane(int experts) {
  int n = 1;
  while (32 * n < experts) n *= 2;
  return n;
}

// Blocks and tokens per block of gemm_route.
void route_shape(int64_t tokens, int* blocks, int* per_block) {
  if (tokens <= kOneBlockTokens) {
    *blocks = 1;
    *per_block = int(tokens);
    return;
  }
  int64_t per = (tokens + kMaxBlocks - 1) / kMaxBlocks;
  if (per < 32) per = 32;
  *per_block = int(per);
  *blocks = int((tokens + per - 1) / per);
}

int check_config(int64_t tokens, int experts, const gemm_route_config_t* c) {
  if (c == nullptr || tokens < 0 || experts < 1 || experts > kMaxExperts || c->k < 1 || c->k > kMaxK ||
      c->k > experts || (c->score != GEMM_SCORE_SOFTMAX && c->score != GEMM_SCORE_SIGMOID) ||
      tokens > ((int64_t(1) << 31) - 1) / c->k)
    return GEMM_ERR_INVALID_VALUE;
  return GEMM_OK;
}

template <int NPL>
cudaError_t launch_route(const RouteParams& p, cudaStream_t s) {
  // one block: a warp for each token
  const int most = kRouteThreads<NPL>, few = p.blocks > 1 ? most : p.tokens * 32;
  const int block = few > most ? most : few < kLeastThreads ? kLeastThreads : few;
  cudaError_t e = launch_dependent(route_kernel<NPL>, p.blocks, block, 0, s, 1, p);
  if (e != cudaSuccess || p.blocks == 1) return e;
  return launch_dependent(route_place_kernel, p.blocks, 1024, 0, s, 1, p);
}

template <int NPL>
cudaError_t launch_route_grad(const RouteParams& p, const float* dw, void* dl, long long ldd, int sms, cudaStream_t s) {
  int64_t blocks = (int64_t(p.tokens) + 7) / 8;
  if (blocks > int64_t(sms) * 8) blocks = int64_t(sms) * 8;
  return launch_dependent(route_grad_kernel<NPL>, int(blocks), 256, 0, s, 1, p, dw, dl, ldd);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int64_t gemm_route_workspace(int64_t tokens, int experts, int k) {
  if (tokens <= 0 || experts < 1 || experts > kMaxExperts || k < 1) return 0;
  int blocks, per;
  route_shape(tokens, &blocks, &per);
  return blocks > 1 ? int64_t(blocks) * experts * int64_t(sizeof(int32_t)) : 0;
}

int gemm_route(int type, int64_t tokens, int experts, const void* logits, int64_t ld, const float* bias,
               const gemm_route_config_t* config, int32_t* ids, float* weights, int32_t* slots, int32_t* rows,
               int32_t* offsets, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_config(tokens, experts, config);
  if (st != GEMM_OK) return st;
  if (bad_type(type) || config->groups < 1 || config->groups > 32 || experts % config->groups != 0 ||
      config->kept_groups < 1 || config->kept_groups > config->groups ||
      config->k > config->kept_groups * (experts / config->groups))
    return GEMM_ERR_INVALID_VALUE;
  if (offsets == nullptr || (tokens > 0 && (logits == nullptr || ids == nullptr || weights == nullptr ||
                                            slots == nullptr || rows == nullptr || ld < experts ||
                                            ld > (int64_t(1) << 39))))
    return GEMM_ERR_INVALID_VALUE;
  const int64_t need = gemm_route_workspace(tokens, experts, config->k);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GEMM_ERR_INVALID_VALUE;
  if (misaligned(logits, type_bytes(type)) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4) ||
      misaligned(slots, 4) || misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(workspace, 16))
    return GEMM_ERR_MISALIGNED;
  CallContext ctx;
  st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[8] = {offsets, tokens > 0 ? logits : nullptr, tokens > 0 ? ids : nullptr,
                         tokens > 0 ? weights : nullptr, tokens > 0 ? slots : nullptr, tokens > 0 ? rows : nullptr,
                         bias, need > 0 ? workspace : nullptr};
  for (const void* q : ptrs)
    if (q != nullptr && !on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  RouteParams p = {};
  p.logits = logits;
  p.bias = bias;
  p.ids = ids;
  p.weights = weights;
  p.slots = slots;
  p.rows = rows;
  p.offsets = offsets;
  p.counts = static_cast<int32_t*>(workspace);
  p.ld = ld;
  p.type = type;
  p.tokens = int(tokens);
  p.experts = experts;
  p.k = config->k;
  p.score = config->score;
  p.groups = config->groups;
  p.kept = config->kept_groups;
  p.renormalize = config->renormalize != 0;
  p.scale = config->scale;
  route_shape(tokens, &p.blocks, &p.per_block);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (scores_per_lane(experts)) {
    case 1: e = launch_route<1>(p, s); break;
    case 2: e = launch_route<2>(p, s); break;
    case 4: e = launch_route<4>(p, s); break;
    case 8: e = launch_route<8>(p, s); break;
    case 16: e = launch_route<16>(p, s); break;
    default: e = launch_route<32>(p, s); break;
  }
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_route_backward(int type, int64_t tokens, int experts, const void* logits, int64_t ld, const int32_t* ids,
                        const float* dweights, const gemm_route_config_t* config, void* dlogits, int64_t ldd,
                        void* stream) {
  int st = check_config(tokens, experts, config);
  if (st != GEMM_OK) return st;
  if (bad_type(type)) return GEMM_ERR_INVALID_VALUE;
  if (tokens == 0) return GEMM_OK;
  if (logits == nullptr || ids == nullptr || dweights == nullptr || dlogits == nullptr || ld < experts ||
      ldd < experts || ld > (int64_t(1) << 39) || ldd > (int64_t(1) << 39))
    return GEMM_ERR_INVALID_VALUE;
  const int es = type_bytes(type);
  if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(ids, 4) || misaligned(dweights, 4))
    return GEMM_ERR_MISALIGNED;
  // dlogits may be the logits' own buffer and pitch (a warp reads its token before it writes it), or apart from it
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(logits), a1 = a0 + uintptr_t(((tokens - 1) * ld + experts) * es);
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(dlogits), b1 = b0 + uintptr_t(((tokens - 1) * ldd + experts) * es);
  if (!(a0 == b0 && ld == ldd) && a0 < b1 && b0 < a1) return GEMM_ERR_INVALID_VALUE;
  CallContext ctx;
  st = begin_call(&ctx);
  if (st != GEMM_OK) return st;
  const void* ptrs[4] = {logits, ids, dweights, dlogits};
  for (const void* q : ptrs)
    if (!on_device(q, ctx.dev)) return GEMM_ERR_NOT_DEVICE_MEMORY;
  RouteParams p = {};
  p.logits = logits;
  p.ids = const_cast<int32_t*>(ids);
  p.ld = ld;
  p.type = type;
  p.tokens = int(tokens);
  p.experts = experts;
  p.k = config->k;
  p.score = config->score;
  p.renormalize = config->renormalize != 0;
  p.scale = config->scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (scores_per_lane(experts)) {
    case 1: e = launch_route_grad<1>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
    case 2: e = launch_route_grad<2>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
    case 4: e = launch_route_grad<4>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
    case 8: e = launch_route_grad<8>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
    case 16: e = launch_route_grad<16>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
    default: e = launch_route_grad<32>(p, dweights, dlogits, ldd, ctx.sm_count, s); break;
  }
  return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
