// Routing by scores: from router logits to expert ids and weights, and the
// gradient back to the logits together with the balance and z losses.
//
// Page "Qwen3.5-MoE与Qwen3-MoE架构差异深度解析", section 3.3 (a per-expert
// balance term added before the selection; the load-balancing loss), sections 2.2
// and 4.1 (load balancing, router z-loss); page "Qwen3.5 Block在llama.cpp中的映射与优化原理",
// section 1.1 (experts in groups).
//
// One warp per token.  Lane i holds the V = P / 32 consecutive experts
// [i V, i V + V), P = E rounded up to a power of two (at least 32), so that
//  - a lane's logits are one contiguous piece of the row (16 bytes for 256
//    bf16 logits),
//  - the pairwise sum over neighbours (the order the header fixes for the
//    softmax denominator) is V - 1 adds in the lane and five xor shuffles,
//  - equal values resolve to the lower expert id by taking the lowest lane.
#include <math.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kScoredThreads = 256;
constexpr int kScoredWarps = kScoredThreads / 32;
constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxGroups = 32;

struct ScoredParams {
  const void* logits;  // fp32 or bf16 [T, E], rows `ld` elements apart
  int64_t ld;
  const float* bias;  // [E] or null: added for the selection only
  int T, E, k, kmax;
  int n_groups, topk_groups, group_top;
  int renorm;
  float scale;
  int32_t* ids;
  float* w;
  int32_t* k_dev;
  unsigned int* err;
};

// Order-preserving map of fp32 values onto uint32; 0 stands for "unavailable"
// and is below the key of every value above -inf.
__device__ __forceinline__ uint32_t choice_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if constexpr (BF16) return bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(row) + e));
  return __ldg(static_cast<const float*>(row) + e);
}

// The lane's V logits of one row as they lie in memory, so that a row can be
// on its way while another is worked on: 16-byte (or narrower whole-lane)
// loads when `vec` says that every lane's piece is aligned and inside the row
// (2) or inside or wholly past it (1), else one load per expert.  Experts past
// E read as -inf.
template <int V, bool BF16>
struct RawLogits {
  static constexpr int W = BF16 ? (V + 1) / 2 : V;
  static constexpr uint32_t kNone = BF16 ? 0xFF80FF80u : 0xFF800000u;
  uint32_t w[W];

  __device__ __forceinline__ void load(const void* row, int e0, int E, int vec) {
    if (vec == 1 && e0 >= E) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = kNone;
    } else if (vec && V >= (BF16 ? 2 : 4)) {
      const uint32_t* p = static_cast<const uint32_t*>(row) + (BF16 ? e0 / 2 : e0);
      if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
          w[4 * i] = q.x;
          w[4 * i + 1] = q.y;
          w[4 * i + 2] = q.z;
          w[4 * i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = __ldg(p + i);
      }
    } else if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int e = e0 + 2 * i;
        const uint32_t lo = e < E ? __ldg(p + e) : 0xFF80u;
        const uint32_t hi = V > 1 && e + 1 < E ? __ldg(p + e + 1) : 0xFF80u;
        w[i] = lo | (hi << 16);
      }
    } else {
      const uint32_t* p = static_cast<const uint32_t*>(row);
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = e0 + i < E ? __ldg(p + e0 + i) : kNone;
    }
  }
  __device__ __forceinline__ void get(float (&l)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (BF16)
        l[v] = __uint_as_float((v & 1) ? w[v / 2] & 0xFFFF0000u : w[v / 2] << 16);
      else
        l[v] = __uint_as_float(w[v]);
    }
  }
};

template <int V, bool BF16>
__device__ __forceinline__ void load_logits(float (&l)[V], const void* row, int e0, int E,
                                            int vec) {
  RawLogits<V, BF16> raw;
  raw.load(row, e0, E, vec);
  raw.get(l);
}

__device__ __forceinline__ float sigmoid_f32(float l) {
  return __frcp_rn(__fadd_rn(1.0f, expf(-l)));
}

// Pairwise sum over neighbouring experts, the same bits in every lane.
template <int V>
__device__ __forceinline__ float neighbour_sum(const float (&x)[V]) {
  float t[V];
#pragma unroll
  for (int v = 0; v < V; ++v) t[v] = x[v];
#pragma unroll
  for (int n = V; n > 1; n >>= 1)
#pragma unroll
    for (int v = 0; v < n / 2; ++v) t[v] = __fadd_rn(t[2 * v], t[2 * v + 1]);
  float s = t[0];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(kFull, s, o));
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The two largest of two pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  const float lo = fminf(a1, b1);
  a1 = fmaxf(a1, b1);
  a2 = fmaxf(lo, fmaxf(a2, b2));
}

// Strikes the choices outside the best `topk_groups` groups (c = -inf).  A
// group's value is its best choice, or the sum of its two best (of the only
// one, if it has one); a group without any available expert is never ahead of
// one that has; equal values go to the lower group.  xs: 32 V floats of shared
// memory; the lanes share the groups' experts there, a power of two of them
// to a group, because a group need not be a run of whole lanes.
template <int V>
__device__ __forceinline__ void limit_groups(const ScoredParams& p, float (&c)[V], int e0,
                                             float* xs) {
  const int lane = threadIdx.x & 31;
  const int G = p.n_groups, gsz = p.E / G;
  int width = 1;
  while (2 * width * G <= 32) width *= 2;
  const int g = lane / width, from = g * gsz + (lane & (width - 1)), to = g < G ? (g + 1) * gsz : 0;
  __syncwarp();
#pragma unroll
  for (int v = 0; v < V; ++v) xs[e0 + v] = c[v];
  __syncwarp();
  float a1 = -INFINITY, a2 = -INFINITY;
  for (int e = from; e < to; e += width) merge_top2(a1, a2, xs[e], -INFINITY);
  for (int o = 1; o < width; o <<= 1) {
    const float b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
    merge_top2(a1, a2, b1, b2);
  }
  const float val = p.group_top == 2 && a2 > -INFINITY ? __fadd_rn(a1, a2) : a1;
  const uint32_t kv = a1 > -INFINITY ? choice_key(val) : 0u;
  const uint32_t mine = __shfl_sync(kFull, kv, lane < G ? lane * width : 0);  // lane h: group h
  int rank = 0;
  for (int h = 0; h < G; ++h) {
    const uint32_t o = __shfl_sync(kFull, mine, h);
    rank += o > mine || (o == mine && h < lane);
  }
  const unsigned chosen = __ballot_sync(kFull, lane < G && rank < p.topk_groups);
  if (g < G && !((chosen >> g) & 1u))
    for (int e = from; e < to; e += width) xs[e] = -INFINITY;
  __syncwarp();
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = xs[e0 + v];
}

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float redux_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Weights and ids of the token whose slot `lane` chose (id, s).
__device__ __forceinline__ void store_chosen(const ScoredParams& p, int64_t t, int id, float s) {
  const int lane = threadIdx.x & 31;
  float w = s;
  if (p.renorm) {
    const float tot = warp_sum(s);
    w = tot > 0.0f ? __fdiv_rn(s, tot) : 0.0f;
  }
  if (lane < p.kmax) {
    p.ids[t * p.kmax + lane] = id;
    p.w[t * p.kmax + lane] = __fmul_rn(w, p.scale);
  }
}

// The definition as it stands: exact scores of every expert, then k rounds of
// a warp argmax.  For the tokens whose fast selection is not certain.
template <int V, bool BF16, bool SIGMOID>
__device__ __noinline__ void route_token_exact(const ScoredParams& p, int64_t t, int vec,
                                              float* xs) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  float s[V], c[V];
  uint32_t key[V];
  {
    float l[V];
    const char* row = static_cast<const char*>(p.logits) + t * p.ld * (BF16 ? 2 : 4);
    load_logits<V, BF16>(l, row, e0, p.E, vec);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = fabsf(l[v]) < INFINITY ? 1u : 0u;
    if constexpr (SIGMOID) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = key[v] ? sigmoid_f32(l[v]) : 0.0f;
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) m = key[v] ? fmaxf(m, l[v]) : m;
      m = redux_max(m);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = key[v] ? expf(__fsub_rn(l[v], m)) : 0.0f;
      const float den = neighbour_sum(s);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = key[v] ? __fdiv_rn(s[v], den) : 0.0f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = p.bias && e0 + v < p.E ? __fadd_rn(s[v], __ldg(p.bias + e0 + v)) : s[v];
    if (!key[v] || !(c[v] > -INFINITY)) c[v] = -INFINITY;
  }
  if (p.n_groups > 1) limit_groups<V>(p, c, e0, xs);
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = c[v] > -INFINITY ? choice_key(c[v]) : 0u;
  int my_id = -1;
  float my_s = 0.0f;
  for (int r = 0; r < p.k; ++r) {
    uint32_t bk = 0u;
    int bv = 0;
    float bs = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > bk) {
        bk = key[v];
        bv = v;
        bs = s[v];
      }
    const uint32_t top = __reduce_max_sync(kFull, bk);
    if (top == 0u) break;  // no expert left: the remaining slots stay empty
    const int win = __ffs(__ballot_sync(kFull, bk == top)) - 1;
    const int id = __shfl_sync(kFull, e0 + bv, win);
    const float sv = __shfl_sync(kFull, bs, win);
    if (lane == r) {
      my_id = id;
      my_s = sv;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v == id) key[v] = 0u;
  }
  store_chosen(p, t, my_id, my_s);
}

// 1 / (1 + exp(-l)) to 1e-6 absolute: the hardware's 2^x and reciprocal, two
// instructions where expf and an exact division take some twenty.
__device__ __forceinline__ float sigmoid_approx(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * l));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// Largest two of the lane's V values.
template <int V>
__device__ __forceinline__ void lane_top2(const float (&c)[V], float& a1, float& a2) {
  if constexpr (V == 1) {
    a1 = c[0];
    a2 = -INFINITY;
  } else {
    float hi[V / 2], lo[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      hi[v] = fmaxf(c[2 * v], c[2 * v + 1]);
      lo[v] = fminf(c[2 * v], c[2 * v + 1]);
    }
#pragma unroll
    for (int n = V / 2; n > 1; n >>= 1)
#pragma unroll
      for (int v = 0; v < n / 2; ++v) {
        float x1 = hi[2 * v], x2 = lo[2 * v];
        merge_top2(x1, x2, hi[2 * v + 1], lo[2 * v + 1]);
        hi[v] = x1;
        lo[v] = x2;
      }
    a1 = hi[0];
    a2 = lo[0];
  }
}

// Ids and weights of one token per warp and step.
//
// Only the handful of experts around the cut needs exact scores.  Choices
// c~ from the hardware exponential and reciprocal are within eps of the exact
// fp32 ones (scores are at most 1: the sigmoid's error is below 1e-6, the
// softmax's below 1e-6 of the score; a choice adds one rounding of itself).
// The k-th largest of the lanes' two best c~ is a lower bound of the k-th
// largest choice, so every chosen expert has c~ >= bound - 2 eps.  Those candidates
// (about k + 2 of 256) get one lane each, their exact scores and their ranks
// by counting, and the lanes with rank < k are the answer.  Groups are cut on
// c~ too when the cut is wider than the approximation.  More than 16
// candidates (many equal choices) and groups too close to call go to
// route_token_exact.  The ids do not depend on which way was taken; the sum that
// renormalizes the weights runs over the candidates here and in rank order
// there, so their last bit may.
//
// Bound by the issue rate: some 560 instructions per token of 256 experts
// (issue slots 70 % used, ALU 61 %).  Measured, k 8 of 256 bf16 experts in 8
// groups, 65536 tokens: 45 us (37.7 MB: 6 us at the copy rate); with exact
// scores for every expert and k rounds of argmax 93 us; 64 experts 21 us.  For
// the CTAs per SM, V = 32 (more than 512 experts) spills 130-160 bytes a
// thread, V = 8 without LANES 40, the other V 4 or none.  A
// lane per token (rows in shared memory) was no faster: 47 us, 83 us for fp32
// rows, whose 32 rows per warp leave few warps.
//
// Two tokens share the last part of the work: the candidates of one on lanes
// 0-15, those of the other on lanes 16-31.
// LANES: groups, if any, are whole aligned runs of lanes (a power of two of
// them), so that their values are joined by shuffles alone; decided at run
// time the size above takes 46 us.
template <int V, bool BF16, bool SIGMOID, bool LANES>
__global__ void __launch_bounds__(kScoredThreads, V <= 8 ? 4 : 2)
    route_scored_kernel(ScoredParams p, int vec, int per) {
  constexpr int C = 16;  // candidates of a token
  __shared__ __align__(16) int cand_id[kScoredWarps][2 * C];
  __shared__ __align__(16) float cand_x[kScoredWarps][2 * C];
  __shared__ __align__(16) float group_x[kScoredWarps][32 * V];  // groups that straddle lanes
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * V;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.k_dev = p.k;
  float b[V];
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    b[v] = p.bias && e0 + v < p.E ? __ldg(p.bias + e0 + v) : 0.0f;
    if (b[v] != b[v]) {
      bad = true;
      b[v] = -INFINITY;
    }
  }
  constexpr float eps = 1e-6f;
  const int G = p.n_groups, gsz = p.E / G, span = gsz / V;  // span: lanes of a group
  // lanes that work on a group: its own when groups are whole aligned runs of
  // lanes, else as many as fit (a power of two), over shared memory
  int width = 1;
  if (LANES) width = span;
  else
    while (2 * width * G <= 32) width *= 2;
  const int my_group = LANES ? e0 / gsz : lane / width;  // >= G: none

  // The candidates of the token whose logits lie at `row` into ids[]; their
  // number, or -1 when they are not certain or too many.  m, den: the
  // softmax's largest logit and denominator.
  auto candidates = [&](const char* row, int* ids, float& m, float& den) -> int {
    float l[V], c[V];
    load_logits<V, BF16>(l, row, e0, p.E, vec);
#pragma unroll
    for (int v = 0; v < V; ++v) bad |= !(l[v] < INFINITY);
    if constexpr (SIGMOID) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = sigmoid_approx(l[v]);
    } else {
      m = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) m = l[v] < INFINITY ? fmaxf(m, l[v]) : m;
      m = redux_max(m);
      float ex[V];
#pragma unroll
      for (int v = 0; v < V; ++v) ex[v] = fabsf(l[v]) < INFINITY ? expf(__fsub_rn(l[v], m)) : 0.0f;
      den = neighbour_sum(ex);
      const float inv = __fdividef(1.0f, den);
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = ex[v] * inv;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = fabsf(l[v]) < INFINITY ? c[v] + b[v] : -INFINITY;
    float best, second;
    lane_top2<V>(c, best, second);
    bool live = true;  // the lane's group is among the chosen
    if (G > 1) {
      float a1 = best, a2 = second;
      float* xs = group_x[warp];
      const int from = my_group * gsz + (lane & (width - 1));
      const int to = my_group < G ? (my_group + 1) * gsz : 0;
      if constexpr (!LANES) {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) xs[e0 + v] = c[v];
        __syncwarp();
        a1 = a2 = -INFINITY;
        for (int e = from; e < to; e += width) merge_top2(a1, a2, xs[e], -INFINITY);
      }
      for (int o = 1; o < width; o <<= 1) {
        const float b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
        merge_top2(a1, a2, b1, b2);
      }
      // every lane of a group holds the group's value
      const bool pair = p.group_top == 2 && a2 > -INFINITY;
      const float val = pair ? a1 + a2 : a1;
      // how far val may be from the exact value: the choices' errors, each
      // relative to its choice, which do not cancel as the choices may
      const float mag = pair ? fabsf(a1) + fabsf(a2) : fabsf(a1);
      const float err = mag < INFINITY ? fmaf(mag, 0x1p-21f, 2.0f * eps) : 0.0f;
      const float mine = my_group < G ? val : -INFINITY;
      const bool first = (lane & (width - 1)) == 0;  // one lane of each group
      float rest = mine, cut = -INFINITY;
#pragma unroll 4
      for (int r = 0; r < p.topk_groups; ++r) {
        cut = redux_max(rest);
        if (rest == cut) rest = -INFINITY;
      }
      int groups = __popc(__ballot_sync(kFull, first && mine >= cut && mine > -INFINITY));
      if (groups > p.topk_groups) {  // equal values left together: count them
        rest = mine;
        groups = 0;
        while (groups < p.topk_groups) {
          cut = redux_max(rest);
          groups += __popc(__ballot_sync(kFull, first && rest == cut));
          if (rest == cut) rest = -INFINITY;
        }
      }
      live = mine >= cut && mine > -INFINITY;
      const float least = redux_min(live ? mine - err : INFINITY);  // a chosen group's value
      const float next = redux_max(live ? -INFINITY : mine + err);  // another's
      // as many groups as asked (or all that have an expert), and the others
      // clearly below
      const bool sure = next == -INFINITY ? groups <= p.topk_groups
                                          : groups == p.topk_groups && least > next;
      if (!sure) return -1;
      if constexpr (!LANES) {  // strike the other groups' choices
        if (!live)
          for (int e = from; e < to; e += width) xs[e] = -INFINITY;
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = xs[e0 + v];
        lane_top2<V>(c, best, second);
        live = true;
      }
    }
    float bound = -INFINITY;
    float rest = live ? best : -INFINITY, after = live ? second : -INFINITY;
#pragma unroll 8
    for (int r = 0; r < p.k; ++r) {
      bound = redux_max(rest);
      if (rest == bound) {
        rest = after;
        after = -INFINITY;
      }
    }
    // -FLT_MAX when fewer than k lanes have an expert: all of them are candidates
    float cut = fmaxf(bound - (2.0f * eps + fabsf(bound) * 0x1p-20f), -3.4028234e38f);
    if (bound == -INFINITY) cut = -3.4028234e38f;
    unsigned mine = 0u;  // the lane's candidates, one bit each
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c[v] >= cut) mine |= 1u << v;
    if (!live) mine = 0u;
    int n = 0;
    for (unsigned who = __ballot_sync(kFull, mine != 0u); who; who = __ballot_sync(kFull, mine != 0u)) {
      const int at = n + __popc(who & lanemask_lt());
      if (mine != 0u && at < C) ids[at] = e0 + __ffs(mine) - 1;
      mine &= mine - 1u;
      n += __popc(who);
    }
    return n <= C ? n : -1;
  };

  // a warp takes two neighbouring tokens per step, or (few tokens) one
  const int64_t step = (int64_t)gridDim.x * kScoredWarps * per;
  const int half = lane >> 4, i = lane & 15;
  for (int64_t t = ((int64_t)blockIdx.x * kScoredWarps + warp) * per; t < p.T; t += step) {
    const char* row = static_cast<const char*>(p.logits) + t * p.ld * (BF16 ? 2 : 4);
    const char* row1 = row + p.ld * (BF16 ? 2 : 4);
    const bool two = per == 2 && t + 1 < p.T;
    float m0 = 0.0f, den0 = 1.0f, m1 = 0.0f, den1 = 1.0f;
    const int n0 = candidates(row, cand_id[warp], m0, den0);
    const int n1 = two ? candidates(row1, cand_id[warp] + C, m1, den1) : 0;
    __syncwarp();
    const int n = half ? n1 : n0;
    const float m = half ? m1 : m0, den = half ? den1 : den0;
    int id = 0x7FFFFFFF;
    float s = 0.0f, x = -INFINITY;
    if (i < n) {
      id = cand_id[warp][lane];
      const float q = load_logit<BF16>(half ? row1 : row, id);
      s = SIGMOID ? sigmoid_f32(q) : __fdiv_rn(expf(__fsub_rn(q, m)), den);
      x = p.bias ? __fadd_rn(s, __ldg(p.bias + id)) : s;
    }
    cand_x[warp][lane] = x;
    __syncwarp();
    int rank = 0;
    const float* xs = &cand_x[warp][half * C];
    for (int j = 0; j < max(n0, n1); j += 4) {  // past the candidates: -inf, never ahead
      const float4 q = *reinterpret_cast<const float4*>(xs + j);
      rank += q.x > x;
      rank += q.y > x;
      rank += q.z > x;
      rank += q.w > x;
    }
    if (i >= n) rank = 32;
    // distinct choices have the ranks 0 .. n - 1; equal ones go by id
    const unsigned seen = __reduce_or_sync(kFull, i < n ? 1u << (rank + 16 * half) : 0u);
    if (__popc(seen) != max(n0, 0) + max(n1, 0)) {
      for (int j = 0; j < n; ++j)
        rank += xs[j] == x && cand_id[warp][half * C + j] < id;
    }
    const bool chosen = rank < p.k;
    float w = chosen ? s : 0.0f;
    if (p.renorm) {
      float tot = w;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
      w = tot > 0.0f ? __fdiv_rn(w, tot) : 0.0f;
    }
    const int64_t out = (t + half) * p.kmax;
    if (chosen) {
      p.ids[out + rank] = id;
      p.w[out + rank] = __fmul_rn(w, p.scale);
    }
    if (n >= 0 && i >= min(n, p.k) && i < p.kmax && (half == 0 || two)) {
      p.ids[out + i] = -1;
      p.w[out + i] = 0.0f;
    }
    if (n0 < 0) route_token_exact<V, BF16, SIGMOID>(p, t, vec, group_x[warp]);
    if (n1 < 0) route_token_exact<V, BF16, SIGMOID>(p, t + 1, vec, group_x[warp]);
    __syncwarp();
  }
  if (bad) raise_device_error(p.err, MOE_DEVERR_BAD_SCORE);
}

// ---- gradient and losses ---------------------------------------------------

struct ScoredGradParams {
  const void* logits;
  int64_t ld;
  const int32_t* ids;     // [T, kmax]
  const float* d_w;       // [T, kmax] or null (the losses' gradient only)
  const int32_t* counts;  // [E] or null (no balance loss)
  int T, E, k, kmax;
  int renorm;
  float scale, balance, z;
  void* d_logits;  // like logits, rows ld_out elements apart
  int64_t ld_out;
  float* part;  // [grid][2]: the block's parts of sum_te c_e q_te (the balance loss) and of sum_t lse^2
  unsigned int* err;
};

// Four sums over the warp at once, every lane with all four: at the first two
// steps a lane keeps half of the values that it holds and sends the rest, so
// nine shuffles instead of twenty.
__device__ __forceinline__ void warp_sum4(float& a, float& b, float& c, float& d) {
  const int lane = threadIdx.x & 31;
  const bool h16 = (lane & 16) != 0, h8 = (lane & 8) != 0;
  float x = h16 ? c : a, y = h16 ? d : b;
  x += __shfl_xor_sync(kFull, h16 ? a : c, 16);
  y += __shfl_xor_sync(kFull, h16 ? b : d, 16);
  float z = h8 ? y : x;
  z += __shfl_xor_sync(kFull, h8 ? x : y, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  a = __shfl_sync(kFull, z, 0);
  b = __shfl_sync(kFull, z, 8);
  c = __shfl_sync(kFull, z, 16);
  d = __shfl_sync(kFull, z, 24);
}

__device__ __forceinline__ float exp_approx(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(1.4426950408889634f * x));
  return e;
}

// The sigmoid s = 1 / (1 + e) and its derivative s (1 - s) = e s^2, e = e^-l: of
// full relative accuracy where s saturates, which s - s^2 loses (7 % of it at
// l = 14, all past 17).  e is held at 2^127, where s is 0 and e s must be too.
__device__ __forceinline__ float sigmoid_slope(float l, float& slope) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(-1.4426950408889634f * l, 127.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  slope = e * s * s;
  return s;
}

// One token per warp and step, its V experts per lane in registers.  With
// u_e = exp(l_e - max) or the sigmoid, U its sum, c_e = d balance / d q_e:
//   slots    r = sum dw u / sum u over the chosen, d u_j = (dw_j - r) U / sum u
//            (renormalized; scale-free, so the softmax needs no division), or dw_j
//   softmax  d l = s (d u + c - sum c s - [sum dw s when not renormalized])
//   sigmoid  d l = s (1 - s) (d u + (c - sum c s / U) / U)
//   z        d l += 2 z / T lse softmax(l)
// so one joint reduction of four sums (and the z loss's fifth) serves all of
// it.  The hardware exponential and reciprocal are good to a few 1e-7 here,
// far inside the rounding of the differences they enter.  The chosen slots'
// d u meets its expert's lane through a row of shared memory per warp.
//
// Bound by the issue rate and the shuffles' latency: some 370 instructions per
// token of 256 experts, issue slots 61 % used.  Measured, 32768 x 256 bf16,
// sigmoid: 18.4 us (35.7 MB: 5.3 at the copy rate; with s - s^2 for the
// sigmoid's slope 17.8), softmax 16.1; 4096 x 128 fp32, softmax 4.0 with the
// losses' kernel.
constexpr int grad_ctas_per_sm(int V) { return V <= 4 ? 4 : V <= 16 ? 2 : 1; }

template <int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kScoredThreads, grad_ctas_per_sm(V)) route_scored_backward_kernel(ScoredGradParams p,
                                                                               int vec) {
  constexpr int P = 32 * V;
  __shared__ __align__(16) float scatter[kScoredWarps][P];
  __shared__ float loss_part[kScoredWarps][2];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * V;
  float* buf = scatter[warp];
  float coef[V];  // c_e = d balance / d q_te; the loss itself is sum_te c_e q_te
  // coef = balance * E / (k T) * counts / T
  const float unit = p.counts ? p.balance * ((float)p.E / ((float)p.k * (float)p.T)) / (float)p.T : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    coef[v] = p.counts && e0 + v < p.E ? unit * (float)__ldg(p.counts + e0 + v) : 0.0f;
    buf[e0 + v] = 0.0f;
  }
  const bool need_z = p.z != 0.0f;
  const float zt = 2.0f * p.z / (float)p.T;
  float lse2 = 0.0f, bal = 0.0f;
  bool bad = false;
  __syncwarp();
  const int64_t step = (int64_t)gridDim.x * kScoredWarps;
  const bool slot = p.d_w && lane < p.k;
  int64_t t = (int64_t)blockIdx.x * kScoredWarps + warp;
  RawLogits<V, BF16> raw;
  int next_id = -1;
  float next_dw = 0.0f;
  auto fetch = [&](int64_t to) {
    raw.load(static_cast<const char*>(p.logits) + to * p.ld * (BF16 ? 2 : 4), e0, p.E, vec);
    if (slot) {
      next_id = __ldg(p.ids + to * p.kmax + lane);
      next_dw = __ldg(p.d_w + to * p.kmax + lane);
    }
  };
  if (t < p.T) fetch(t);
  for (; t < p.T; t += step) {
    const char* row = static_cast<const char*>(p.logits) + t * p.ld * (BF16 ? 2 : 4);
    float l[V];
    raw.get(l);
    int id = next_id;
    float dw = next_dw * p.scale;
    if (t + step < p.T) fetch(t + step);  // the next token's, while this one is worked on
    if (id >= p.E) {
      bad = true;
      id = -1;
    }
    float lj = id >= 0 ? load_logit<BF16>(row, id) : -INFINITY;
    if (!(lj < INFINITY)) lj = -INFINITY;
    if (id < 0) dw = 0.0f;
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = l[v] < INFINITY ? l[v] : -INFINITY;  // NaN and +inf: unavailable
      m = fmaxf(m, l[v]);
    }
    m = redux_max(m);
    const bool some = m > -INFINITY;
    if (!some) m = 0.0f;  // every exponential is 0
    float u[V], ex[SIGMOID ? V : 1];  // u: the sigmoid's slope, the softmax's u
    float su = 0.0f, sc = 0.0f, ez = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float s = SIGMOID ? sigmoid_slope(l[v], u[v]) : u[v] = exp_approx(l[v] - m);
      su += s;
      sc = fmaf(coef[v], s, sc);
    }
    if constexpr (SIGMOID) {
      if (need_z) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          ex[v] = exp_approx(l[v] - m);
          ez += ex[v];
        }
        ez = warp_sum(ez);
      }
    }
    const float uj = SIGMOID ? sigmoid_approx(lj) : exp_approx(lj - m);  // 0 without a slot
    float st = uj, sd = dw * uj;
    warp_sum4(su, sc, st, sd);
    if constexpr (!SIGMOID) ez = su;
    const float uinv = su > 0.0f ? __fdividef(1.0f, su) : 0.0f;
    // q = u uinv for both scores (the softmax's U makes u its unnormalised s)
    float dp;
    if (p.renorm) {
      const float r = __fdividef(sd, st);
      // one chosen expert has the constant weight `scale`: no gradient, not
      // the rounding of dw - dw
      const unsigned with = __ballot_sync(kFull, uj > 0.0f);
      const bool several = (with & (with - 1u)) != 0u;
      dp = several && id >= 0 ? __fdividef((dw - r) * (SIGMOID ? 1.0f : su), st) : 0.0f;
    } else {
      dp = dw;
    }
    if (id >= 0) buf[id] = dp;
    const float zc = need_z && some ? zt * (m + __logf(ez)) * __fdividef(1.0f, ez) : 0.0f;
    if (need_z && some) {
      const float lse = m + __logf(ez);
      lse2 = fmaf(lse, lse, lse2);
    }
    // what is the same for all of the token's experts: sum c q, and the
    // softmax's sum of d u s when the weights are not renormalized
    const float dotq = sc * uinv;
    bal += dotq;
    const float off = SIGMOID || p.renorm ? dotq : fmaf(sd, uinv, dotq);
    __syncwarp();
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float own = buf[e0 + v];
      if constexpr (SIGMOID) {
        const float ds = fmaf(coef[v] - off, uinv, own);
        d[v] = ds * u[v];
        if (need_z) d[v] = fmaf(zc, ex[v], d[v]);
      } else {
        d[v] = fmaf(zc, u[v], u[v] * uinv * (own + (coef[v] - off)));
      }
    }
    __syncwarp();
    if (id >= 0) buf[id] = 0.0f;
    char* out = static_cast<char*>(p.d_logits) + t * p.ld_out * (BF16 ? 2 : 4);
    if (e0 < p.E) {  // some lanes may lie past the experts
      if constexpr (BF16) {
        if (vec && V >= 2) {
          uint32_t w2[V / 2 > 0 ? V / 2 : 1];
#pragma unroll
          for (int v = 0; v < V / 2; ++v)
            w2[v] = (uint32_t)f32_to_bf16_rne(d[2 * v]) | ((uint32_t)f32_to_bf16_rne(d[2 * v + 1]) << 16);
          uint32_t* o = reinterpret_cast<uint32_t*>(out) + e0 / 2;
          if constexpr (V >= 8) {
#pragma unroll
            for (int i = 0; i < V / 8; ++i)
              reinterpret_cast<uint4*>(o)[i] =
                  make_uint4(w2[4 * i], w2[4 * i + 1], w2[4 * i + 2], w2[4 * i + 3]);
          } else {
#pragma unroll
            for (int v = 0; v < V / 2; ++v) o[v] = w2[v];
          }
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (e0 + v < p.E) reinterpret_cast<uint16_t*>(out)[e0 + v] = f32_to_bf16_rne(d[v]);
        }
      } else {
        if (vec && V >= 4) {
#pragma unroll
          for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(out)[e0 / 4 + i] =
                make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (e0 + v < p.E) reinterpret_cast<float*>(out)[e0 + v] = d[v];
        }
      }
    }
    __syncwarp();
  }
  if (bad) raise_device_error(p.err, MOE_DEVERR_BAD_EXPERT);
  // the block's sums, warps in order
  if (lane == 0) {
    loss_part[warp][0] = bal;
    loss_part[warp][1] = lse2;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float a = 0.0f;
    for (int w = 0; w < kScoredWarps; ++w) a += loss_part[w][threadIdx.x];
    p.part[2 * blockIdx.x + threadIdx.x] = a;
  }
}

// losses[0] = sum_te c_e q_te, losses[1] = z mean lse^2: the blocks' parts in
// one order (per lane, then a butterfly), a warp for each loss.
__global__ void __launch_bounds__(64) route_losses_kernel(ScoredGradParams p, int blocks,
                                                          float* losses) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, which = threadIdx.x >> 5;
  float a = 0.0f;
#pragma unroll 8
  for (int b = lane; b < blocks; b += 32) a += p.part[2 * b + which];
  a = warp_sum(a);
  if (lane == 0) losses[which] = which ? p.z * (a / (float)p.T) : a;
}

constexpr int kGradMaxBlocks = 1024;  // blocks whose sums the workspace holds

int lane_values(int E) {
  int v = 1;
  while (32 * v < E) v <<= 1;
  return v;
}

template <template <int, bool, bool> class F, typename... A>
moe_status_t dispatch_scored(int V, bool bf16, bool sig, A&&... a) {
#define MOE_SCORED_CASE(v)                                                             \
  case v:                                                                              \
    if (bf16) return sig ? F<v, true, true>::go(a...) : F<v, true, false>::go(a...);   \
    return sig ? F<v, false, true>::go(a...) : F<v, false, false>::go(a...);
  switch (V) {
    MOE_SCORED_CASE(1)
    MOE_SCORED_CASE(2)
    MOE_SCORED_CASE(4)
    MOE_SCORED_CASE(8)
    MOE_SCORED_CASE(16)
    MOE_SCORED_CASE(32)
  }
#undef MOE_SCORED_CASE
  return MOE_ERR_UNSUPPORTED;
}

int scored_grid(int T) {
  int64_t g = ((int64_t)T + kScoredWarps - 1) / kScoredWarps;
  const int64_t cap = (int64_t)moe_host::sm_count() * 8;
  if (g > cap) g = cap;
  return (int)(g < 1 ? 1 : g);
}

template <int V, bool BF16, bool SIG>
struct ForwardLaunch {
  static moe_status_t go(const ScoredParams& p, int vec, cudaStream_t st) {
    // two tokens per warp once every SM has some warps (measured: 64 tokens
    // 2.7 us with one, 3.3 with two; 4096 tokens 5.4 and 4.7)
    const int per = p.T > moe_host::sm_count() * kScoredWarps ? 2 : 1;
    const int span = p.E / p.n_groups / V;
    const bool lanes = p.n_groups == 1 || (p.E / p.n_groups % V == 0 && (span & (span - 1)) == 0);
    return moe_host::launch(lanes ? route_scored_kernel<V, BF16, SIG, true>
                                  : route_scored_kernel<V, BF16, SIG, false>,
                            scored_grid((p.T + per - 1) / per), kScoredThreads, 0, st, p, vec, per);
  }
};
template <int V, bool BF16, bool SIG>
struct BackwardLaunch {
  static moe_status_t go(const ScoredGradParams& p, int grid, int vec, cudaStream_t st) {
    return moe_host::launch(route_scored_backward_kernel<V, BF16, SIG>, grid, kScoredThreads, 0, st,
                            p, vec);
  }
};

// Whole-lane vector accesses: every lane's V values lie inside the row, or all
// past it (2: no lane lies past it), and on a 16-byte (or whole-piece)
// boundary.
int can_vector(const void* base, int64_t ld, int E, int V, int size) {
  const int piece = V * size < 16 ? V * size : 16;
  return E % V == 0 && ld * size % piece == 0 &&
                 (reinterpret_cast<uintptr_t>(base) % piece) == 0
             ? (E == 32 * V ? 2 : 1)
             : 0;
}

bool scored_shape_ok(int T, int E, int k, int kmax, int dtype, int score, int64_t ld) {
  return T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= kmax && kmax <= 16 && k <= E && ld >= E &&
         (int64_t)T * kmax <= (1 << 24) &&
         (dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16) &&
         (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_route_scored(const void* logits, int logits_dtype, int64_t ld,
                                         const float* select_bias, int T, int E, int score,
                                         int n_groups, int topk_groups, int group_top, int k,
                                         int kmax, int renormalize, float scale,
                                         int32_t* topk_ids, float* topk_w, int32_t* k_dev,
                                         moe_stream_t stream) {
  using namespace moe_host;
  if (!scored_shape_ok(T, E, k, kmax, logits_dtype, score, ld)) return MOE_ERR_INVALID_ARG;
  if (n_groups < 1 || n_groups > kMaxGroups || E % n_groups || topk_groups < 1 ||
      topk_groups > n_groups || (group_top != 1 && group_top != 2))
    return MOE_ERR_INVALID_ARG;
  if (k > topk_groups * (E / n_groups)) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || isinf(scale)) return MOE_ERR_INVALID_ARG;
  if (!k_dev) return MOE_ERR_INVALID_ARG;
  const int size = logits_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (T > 0 && (!logits || !topk_ids || !topk_w)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {select_bias, topk_ids, topk_w, k_dev};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % size) return MOE_ERR_INVALID_ARG;
  ScoredParams p;
  p.logits = logits;
  p.ld = ld;
  p.bias = select_bias;
  p.T = T;
  p.E = E;
  p.k = k;
  p.kmax = kmax;
  p.n_groups = n_groups;
  p.topk_groups = topk_groups;
  p.group_top = group_top;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.ids = topk_ids;
  p.w = topk_w;
  p.k_dev = k_dev;
  p.err = device_error_word();
  const int V = lane_values(E);
  return dispatch_scored<ForwardLaunch>(V, logits_dtype == MOE_DTYPE_BF16,
                                        score == MOE_SCORE_SIGMOID, p,
                                        can_vector(logits, ld, E, V, size),
                                        reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_route_backward_workspace_size(int E) {
  if (E < 1 || E > 1024) return 0;
  return (size_t)kGradMaxBlocks * 2 * sizeof(float);
}

extern "C" moe_status_t moe_route_scored_backward(
    const void* logits, int logits_dtype, int64_t ld, const int32_t* topk_ids,
    const float* d_topk_w, const int32_t* expert_counts, int T, int E, int score, int k, int kmax,
    int renormalize, float scale, float balance_coef, float z_coef, void* d_logits, int64_t ld_out,
    float* losses, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe_host;
  if (!scored_shape_ok(T, E, k, kmax, logits_dtype, score, ld) || ld_out < E)
    return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || isinf(scale) || !isfinite(balance_coef) || !isfinite(z_coef))
    return MOE_ERR_INVALID_ARG;
  if (balance_coef != 0.0f && !expert_counts) return MOE_ERR_INVALID_ARG;
  if (!losses || !workspace || workspace_bytes < moe_route_backward_workspace_size(E))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !d_logits || d_logits == logits || (d_topk_w && !topk_ids)))
    return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {topk_ids, d_topk_w, expert_counts, losses, workspace};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MOE_ERR_INVALID_ARG;
  const int size = logits_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % size || reinterpret_cast<uintptr_t>(d_logits) % size)
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(losses, 0, 2 * sizeof(float), st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  ScoredGradParams p;
  p.logits = logits;
  p.ld = ld;
  p.ids = topk_ids;
  p.d_w = d_topk_w;
  p.counts = balance_coef != 0.0f ? expert_counts : nullptr;
  p.T = T;
  p.E = E;
  p.k = k;
  p.kmax = kmax;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.balance = balance_coef;
  p.z = z_coef;
  p.d_logits = d_logits;
  p.ld_out = ld_out;
  p.part = static_cast<float*>(workspace);
  p.err = device_error_word();
  const int V = lane_values(E);
  // as many blocks as run at once: none queues
  // (and at least two tokens per warp, once there are some)
  int grid = scored_grid(T > 512 ? (T + 1) / 2 : T);
  const int most = grad_ctas_per_sm(V) * sm_count();
  if (grid > most) grid = most;
  if (grid > kGradMaxBlocks) grid = kGradMaxBlocks;
  const int vec = can_vector(d_logits, ld_out, E, V, size) ? can_vector(logits, ld, E, V, size) : 0;
  const moe_status_t s =
      dispatch_scored<BackwardLaunch>(V, logits_dtype == MOE_DTYPE_BF16,
                                      score == MOE_SCORE_SIGMOID, p, grid, vec, st);
  if (s != MOE_OK) return s;
  return launch(route_losses_kernel, 1, 64, 0, st, p, grid, losses);
}
