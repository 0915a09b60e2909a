// One AdamW step over many tensors in one launch, states in 32 or 8 bits.
//
//   g = grad (* grad_scale)
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
// Eight-bit states hold 256 consecutive elements of a tensor with one scale:
//   m = s sign(c) (c / 127)^2,        s = max |m|
//   sqrt v = s (c / 255)^2,           s = max sqrt v,  c >= 1 where v > 0
// so that small values keep a relative step (1 / c) and a second moment never
// becomes zero, which would let its update grow without bound.  The step itself
// uses m and v before they are coded again.  The operations that lead to m, v and
// the codes are rounded to fp32 one by one (no contraction), so the codes are
// those of the formulas as written, whatever surrounds them: they come from the
// hardware's approximate roots, and where one is so near a border between two
// codes that its error could matter, from the rounded ones.  The step itself has
// an approximate root and quotient (2 ulp each).
//
// The table of tensors travels as a kernel parameter, so a captured graph
// holds its own and nothing is kept between calls.  CTAs walk over runs of
// units of 2048 elements; a thread takes eight consecutive ones, a warp one
// block of 256.
#include <math.h>

#include <algorithm>
#include <vector>

#include "dense.cuh"

namespace moe {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = kAdamThreads * 8;
constexpr int kAdamBlock = 256;  // elements that share a scale
static_assert(kAdamBlock == 32 * 8, "a warp codes a block");

struct AdamTensor {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float decay;  // weight decay
  float keep;   // 1 - lr * decay for an lr of the host
};

// Kernel parameters hold at most 32764 bytes; few tensors take a small table,
// whose launch is cheaper for the host.
constexpr int kFewTensors = 16, kMostTensors = 424;

template <int CAP>
struct AdamTable {
  AdamTensor t[CAP];
  int first[CAP + 1];  // first unit of each tensor, and their number
  int count;
};

struct AdamParams {
  double beta1, beta2;
  float b1, b2, a1, a2;  // beta and 1 - beta
  float eps, lr;
  const float* lr_dev;
  const float* grad_scale;
  int32_t* step;  // steps done, CTAs that have read it
  int count_step;
  int tiny_eps;   // below 1e-15
};

enum { kParamF32, kParamMaster, kParamBf16 };

// beta^t by squaring: t <= 2^31 costs some 60 products, a relative error of
// t 2^-53 where the power is not yet zero.
__device__ __forceinline__ double power(double b, int t) {
  double r = 1.0;
  for (unsigned n = (unsigned)t; n; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

// The tensor that unit u belongs to.
template <int CAP>
__device__ __forceinline__ int tensor_of(const AdamTable<CAP>& tab, int u) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Byte e (0 .. 3) of w as a float, without a conversion: the byte becomes the end
// of 2^23's mantissa.
__device__ __forceinline__ float byte_float(uint32_t w, int e) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (uint32_t)e)) - 8388608.0f;
}
__device__ __forceinline__ float signed_byte_float(uint32_t w, int e) {
  return __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7440u | (uint32_t)e)) - 8388736.0f;
}
__device__ __forceinline__ float decode_m(float c, float s) {
  const float a = __fmul_rn(c, (float)(1.0 / 127.0));
  return __fmul_rn(__fmul_rn(a, fabsf(a)), s);
}
__device__ __forceinline__ float decode_r(float c, float s) {
  const float a = __fmul_rn(c, (float)(1.0 / 255.0));
  return __fmul_rn(__fmul_rn(a, a), s);
}
// One instruction each; inputs below 2^-126 count as zero.
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Rounding to an integer by the addition of 1.5 2^23: the sum's lowest byte is the
// integer's.  `off` becomes the largest distance from one.
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ uint32_t round_code(float t, float& off) {
  const float q = __fadd_rn(t, kRound);
  off = fmaxf(off, fabsf(__fsub_rn(t, __fsub_rn(q, kRound))));
  return __float_as_uint(q);
}
// The lowest bytes of four words.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
}

// The block's largest value; values are not negative, and a NaN counts as largest.
__device__ __forceinline__ float block_max(const float (&x)[8]) {
  unsigned top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]));
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top));
}
// A block's scale and its reciprocal, from the largest value.  A block whose
// reciprocal is not finite holds zeros, one with a value that is not finite NaN.
__device__ __forceinline__ float block_scale(float s, float& inv) {
  inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  if (inv == INFINITY) s = inv = 0.0f;
  if (s == INFINITY) s = NAN;
  return s;
}

// Eight bytes at any alignment; zeros past n.
__device__ __forceinline__ uint2 load_codes(const void* p, int64_t at, int n, bool vec) {
  const uint8_t* s = static_cast<const uint8_t*>(p) + at;
  if (vec && n == 8) return *reinterpret_cast<const uint2*>(s);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) w[e >> 2] |= (uint32_t)s[e] << ((e & 3) * 8);
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* p, int64_t at, int n, bool vec, uint2 q) {
  uint8_t* d = static_cast<uint8_t*>(p) + at;
  if (vec && n == 8) {
    *reinterpret_cast<uint2*>(d) = q;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) d[e] = (uint8_t)((e < 4 ? q.x : q.y) >> ((e & 3) * 8));
}

template <bool BF16>
__device__ __forceinline__ void load8(float (&f)[8], const void* p, int64_t at, int n, bool vec) {
  Vec8<BF16> v;
  if (vec && n == 8) v.load(p, at);
  else v.load_some(p, at, n);
  v.get(f);
}
template <bool BF16>
__device__ __forceinline__ void store8(const float (&f)[8], void* p, int64_t at, int n, bool vec) {
  Vec8<BF16> v;
  v.set(f);
  if (vec && n == 8) v.store(p, at);
  else v.store_some(p, at, n);
}

__device__ __forceinline__ bool at16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <int CAP, int PARAM, bool G_BF16, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, AdamParams p) {
  __shared__ float correction[2];  // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  pdl_wait();
  // No early trigger: a kernel behind this one may read weights before its own
  // wait, and these are weights.
  const int tid = threadIdx.x, lane = tid & 31;
  const float scale = p.grad_scale ? *p.grad_scale : 1.0f;
  if (!(fabsf(scale) < INFINITY)) return;  // for every thread alike
  int done = 0;
  if (tid < 2) {
    done = *reinterpret_cast<volatile int32_t*>(p.step);
    const double left = 1.0 - power(tid ? p.beta2 : p.beta1, done + 1);
    correction[tid] = (float)(1.0 / (tid ? sqrt(left) : left));
  }
  __syncthreads();
  const float c1 = correction[0], c2 = correction[1];
  const float lr = p.lr_dev ? *p.lr_dev : p.lr;
  const int units = tab.first[tab.count];
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x);
  const int u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  int ti = u0 < u1 ? tensor_of(tab, u0) : 0;
  for (int u = u0; u < u1; ++u) {
    while (u >= tab.first[ti + 1]) ++ti;
    const AdamTensor& t = tab.t[ti];
    const int64_t at = (int64_t)(u - tab.first[ti]) * kAdamUnit + tid * 8;
    const int64_t left = t.n - at;
    const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    const bool vec = at16(t.param) && at16(t.grad) && at16(t.master) && at16(t.m) && at16(t.v);
    float w[8], g[8], m[8], v[8];
    load8<G_BF16>(g, t.grad, at, n, vec);
    if constexpr (PARAM == kParamBf16) load8<true>(w, t.param, at, n, vec);
    else load8<false>(w, PARAM == kParamMaster ? t.master : t.param, at, n, vec);
    if constexpr (EIGHT) {
      const int64_t b = at / kAdamBlock;
      const bool on = b * kAdamBlock < t.n;
      const float sm = on ? t.m_scale[b] : 0.0f, sr = on ? t.v_scale[b] : 0.0f;
      const uint2 cm = load_codes(t.m, at, n, vec), cv = load_codes(t.v, at, n, vec);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] = decode_m(signed_byte_float(e < 4 ? cm.x : cm.y, e & 3), sm);
        const float r = decode_r(byte_float(e < 4 ? cv.x : cv.y, e & 3), sr);
        v[e] = __fmul_rn(r, r);
      }
    } else {
      load8<false>(m, t.m, at, n, vec);
      load8<false>(v, t.v, at, n, vec);
    }
    const float keep = p.lr_dev ? fmaf(-lr, t.decay, 1.0f) : t.keep;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.grad_scale) g[e] = __fmul_rn(g[e], scale);
      m[e] = __fadd_rn(__fmul_rn(m[e], p.b1), __fmul_rn(g[e], p.a1));
      v[e] = __fadd_rn(__fmul_rn(v[e], p.b2), __fmul_rn(__fmul_rn(g[e], g[e]), p.a2));
      // with an eps that small, second moments below 2^-126 matter
      const float step = p.tiny_eps ? __fdiv_rn(m[e] * c1, fmaf(__fsqrt_rn(v[e]), c2, p.eps))
                                    : m[e] * c1 * rcp_approx(fmaf(sqrt_approx(v[e]), c2, p.eps));
      w[e] = fmaf(step, -lr, w[e] * keep);
    }
    if constexpr (PARAM != kParamF32) store8<true>(w, t.param, at, n, vec);
    if constexpr (PARAM != kParamBf16)
      store8<false>(w, PARAM == kParamMaster ? (void*)t.master : t.param, at, n, vec);
    if constexpr (EIGHT) {
      float x[8], im, ir;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < n ? fabsf(m[e]) : 0.0f;
      const float sm = block_scale(block_max(x), im);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] : 0.0f;
      const float top = block_max(v), sr = block_scale(__fsqrt_rn(top), ir);  // the root keeps the order
      uint32_t cm[8], cv[8];
      // an approximate root is 2^-22 of itself off, two of them 255 2^-21 = 1.2e-4 of a code
      float off = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = 127.0f * sqrt_approx(__fmul_rn(x[e], im));
        const float b = 255.0f * sqrt_approx(sqrt_approx(v[e]) * ir);
        cm[e] = round_code(copysignf(a, m[e]), off);
        cv[e] = round_code(v[e] > 0.0f ? fmaxf(b, 1.0f) : b, off);
      }
      if (off > 0.4995f || top < 0x1p-100f) {  // or so small that the hardware's roots lose it
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = __fmul_rn(__fsqrt_rn(__fmul_rn(x[e], im)), 127.0f);
          const float b = __fmul_rn(__fsqrt_rn(__fmul_rn(__fsqrt_rn(v[e]), ir)), 255.0f);
          cm[e] = round_code(copysignf(a, m[e]), off);
          cv[e] = round_code(v[e] > 0.0f ? fmaxf(b, 1.0f) : b, off);
        }
      }
      store_codes(t.m, at, n, vec, make_uint2(pack_bytes(cm[0], cm[1], cm[2], cm[3]),
                                               pack_bytes(cm[4], cm[5], cm[6], cm[7])));
      store_codes(t.v, at, n, vec, make_uint2(pack_bytes(cv[0], cv[1], cv[2], cv[3]),
                                               pack_bytes(cv[4], cv[5], cv[6], cv[7])));
      if (lane == 0 && n > 0) {
        t.m_scale[at / kAdamBlock] = sm;
        t.v_scale[at / kAdamBlock] = sr;
      }
    } else {
      store8<false>(m, t.m, at, n, vec);
      store8<false>(v, t.v, at, n, vec);
    }
  }
  if (p.count_step && tid == 0) {
    __threadfence();  // this CTA's read of the count comes first
    if (atomicAdd(p.step + 1, 1) == (int)gridDim.x - 1) {  // every CTA has read it
      p.step[1] = 0;
      p.step[0] = done + 1;
    }
  }
  __threadfence();
}

// The values that eight-bit states stand for, the tensors one after the other.  A
// tensor's place in the output has any alignment: a warp writes its block in
// 16-byte pieces from the first boundary on, the codes shifted to fit.
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_values_kernel(const __grid_constant__ AdamTable<CAP> tab) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = tab.first[tab.count];
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x);
  const int u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  int ti = u0 < u1 ? tensor_of(tab, u0) : 0;
  for (int u = u0; u < u1; ++u) {
    while (u >= tab.first[ti + 1]) ++ti;
    const AdamTensor& t = tab.t[ti];
    const int64_t b = (int64_t)(u - tab.first[ti]) * (kAdamUnit / kAdamBlock) + warp;
    if (b * kAdamBlock >= t.n) continue;
    const float scale[2] = {t.m_scale[b], t.v_scale[b]};
    const int n = (int)min((int64_t)kAdamBlock, t.n - b * kAdamBlock);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* c = static_cast<const uint8_t*>(h ? t.v : t.m) + b * kAdamBlock;
      float* out = (h ? t.master : static_cast<float*>(t.param)) + b * kAdamBlock;
      auto value = [&](uint32_t w, int e) {
        if (h == 0) return decode_m(signed_byte_float(w, e), scale[0]);
        const float r = decode_r(byte_float(w, e), scale[1]);
        return __fmul_rn(r, r);
      };
      const bool words = (reinterpret_cast<uintptr_t>(c) & 3u) == 0;
      const int head = (int)((16u - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / 4;
      const int quads = words && n > head ? (n - head) / 4 : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int q = i * 32 + lane;
        if (q >= quads) continue;
        const int e = head + 4 * q;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(c + (e & ~3));
        // the last word is read only where its bytes are needed
        const uint32_t lo = w[0], hi = head ? w[1] : 0u;
        const uint32_t four = __funnelshift_r(lo, hi, head * 8);
        *reinterpret_cast<float4*>(out + e) =
            make_float4(value(four, 0), value(four, 1), value(four, 2), value(four, 3));
      }
      if (words) {  // what lies before the first boundary and behind the last piece
        if (lane < head && lane < n) out[lane] = value(c[lane], 0);
        const int e = head + 4 * quads + lane;
        if (lane < 4 && e < n) out[e] = value(c[e], 0);
      } else {
        for (int e = lane; e < n; e += 32) out[e] = value(c[e], 0);
      }
    }
  }
}

// ---- host ------------------------------------------------------------------

using moe_host::aligned4;

int64_t units_of(int64_t n) { return (n + kAdamUnit - 1) / kAdamUnit; }

template <int CAP>
moe_status_t launch_step(const AdamTable<CAP>& tab, const AdamParams& p, int param, bool g_bf16,
                         bool eight, cudaStream_t st) {
  const int64_t most = (int64_t)moe_host::sm_count() * 8;
  const int units = tab.first[tab.count];
  const int grid = units < 1 ? 1 : (int)(units < most ? units : most);
  auto go = [&](auto kern) { return moe_host::launch(kern, dim3(grid), dim3(kAdamThreads), 0, st, tab, p); };
#define MOE_ADAM(P)                                                                      \
  (g_bf16 ? (eight ? go(adamw_kernel<CAP, P, true, true>) : go(adamw_kernel<CAP, P, true, false>)) \
          : (eight ? go(adamw_kernel<CAP, P, false, true>) : go(adamw_kernel<CAP, P, false, false>)))
  switch (param) {
    case kParamF32: return MOE_ADAM(kParamF32);
    case kParamMaster: return MOE_ADAM(kParamMaster);
    default: return MOE_ADAM(kParamBf16);
  }
#undef MOE_ADAM
}

// Runs `each(table, last)` over the tensors that are not empty, as many at a
// time as a table holds; once with an empty table if there are none.
template <typename F>
moe_status_t over_tables(const std::vector<AdamTensor>& all, F&& each) {
  size_t i = 0;
  // tables of about the same number of tensors
  const size_t tables = (all.size() + kMostTensors - 1) / kMostTensors;
  const int most = tables ? (int)((all.size() + tables - 1) / tables) : 0;
  do {
    auto fill = [&](auto& tab) {
      tab.count = 0;
      tab.first[0] = 0;
      for (; i < all.size() && tab.count < most; ++i) {
        const int64_t next = tab.first[tab.count] + units_of(all[i].n);
        if (next > INT32_MAX) break;  // never with the first: n has a limit
        tab.t[tab.count] = all[i];
        tab.first[++tab.count] = (int)next;
      }
    };
    moe_status_t r;
    if (all.size() - i <= kFewTensors) {
      AdamTable<kFewTensors> tab;
      fill(tab);
      r = each(tab, i == all.size());
    } else {
      AdamTable<kMostTensors> tab;
      fill(tab);
      r = each(tab, i == all.size());
    }
    if (r) return r;
  } while (i < all.size());
  return MOE_OK;
}

constexpr int64_t kMostElements = (int64_t)1 << 40;

bool at_least_aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int count,
                                       int param_dtype, int grad_dtype, int state_bits, double lr,
                                       const float* lr_dev, double beta1, double beta2, double eps,
                                       const float* grad_scale, int32_t* step,
                                       moe_stream_t stream) try {
  using namespace moe;
  if (count < 0 || (count > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
  if ((param_dtype != MOE_DTYPE_F32 && param_dtype != MOE_DTYPE_BF16) ||
      (grad_dtype != MOE_DTYPE_F32 && grad_dtype != MOE_DTYPE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (state_bits != 32 && state_bits != 8) return MOE_ERR_UNSUPPORTED;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
      !(eps < INFINITY) || (!lr_dev && !(fabs(lr) < INFINITY)))
    return MOE_ERR_INVALID_ARG;
  if (!step || !aligned4(step) || !aligned4(lr_dev) || !aligned4(grad_scale))
    return MOE_ERR_INVALID_ARG;
  const int psize = param_dtype == MOE_DTYPE_BF16 ? 2 : 4, gsize = grad_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  const bool eight = state_bits == 8;
  std::vector<AdamTensor> all;
  all.reserve(count);
  std::vector<const void*> seen;
  seen.reserve(count);
  int masters = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > kMostElements || !(fabs((double)t.weight_decay) < INFINITY))
      return MOE_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || !at_least_aligned(t.param, psize) ||
        !at_least_aligned(t.grad, gsize) || !aligned4(t.master))
      return MOE_ERR_INVALID_ARG;
    if (eight ? (!t.exp_avg_scale || !t.exp_avg_sq_scale || !aligned4(t.exp_avg_scale) ||
                 !aligned4(t.exp_avg_sq_scale))
              : (!aligned4(t.exp_avg) || !aligned4(t.exp_avg_sq)))
      return MOE_ERR_INVALID_ARG;
    if (t.master && param_dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
    masters += t.master != nullptr;
    const double keep = 1.0 - lr * (double)t.weight_decay;
    all.push_back(AdamTensor{t.param, t.grad, t.master, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale,
                             t.exp_avg_sq_scale, t.n, t.weight_decay, (float)keep});
    seen.push_back(t.param);
  }
  if (masters != 0 && masters != (int)all.size()) return MOE_ERR_UNSUPPORTED;
  // a tensor given twice would be stepped by two CTAs at once
  std::sort(seen.begin(), seen.end());
  if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return MOE_ERR_INVALID_ARG;
  AdamParams p{beta1, beta2, (float)beta1, (float)beta2, (float)(1.0 - beta1), (float)(1.0 - beta2),
               (float)eps, (float)lr, lr_dev, grad_scale, step, 0,
               eps < 1e-15};
  const int param = param_dtype == MOE_DTYPE_F32 ? kParamF32 : masters ? kParamMaster : kParamBf16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return over_tables(all, [&](const auto& tab, bool last) {
    p.count_step = last;
    return launch_step(tab, p, param, grad_dtype == MOE_DTYPE_BF16, eight, st);
  });
} catch (...) {
  return MOE_ERR_CUDA;  // host memory ran out
}

extern "C" moe_status_t moe_adamw_values(const moe_adamw_tensor_t* tensors, int count,
                                         float* exp_avg, float* exp_avg_sq,
                                         moe_stream_t stream) try {
  using namespace moe;
  if (count < 0 || (count > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
  std::vector<AdamTensor> all;
  all.reserve(count);
  int64_t at = 0;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > kMostElements) return MOE_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.exp_avg || !t.exp_avg_sq || !t.exp_avg_scale || !t.exp_avg_sq_scale ||
        !aligned4(t.exp_avg_scale) || !aligned4(t.exp_avg_sq_scale) || !exp_avg || !exp_avg_sq ||
        !aligned4(exp_avg) || !aligned4(exp_avg_sq))
      return MOE_ERR_INVALID_ARG;
    all.push_back(AdamTensor{exp_avg + at, nullptr, exp_avg_sq + at, t.exp_avg, t.exp_avg_sq,
                             t.exp_avg_scale, t.exp_avg_sq_scale, t.n, 0.0f, 0.0f});
    at += t.n;
  }
  if (all.empty()) return MOE_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return over_tables(all, [&](const auto& tab, bool) {
    constexpr int kCap = (int)(sizeof(tab.t) / sizeof(tab.t[0]));
    const int64_t most = (int64_t)moe_host::sm_count() * 8;
    const int units = tab.first[tab.count];
    return moe_host::launch(adamw_values_kernel<kCap>, dim3((unsigned)(units < most ? units : most)),
                            dim3(kAdamThreads), 0, st, tab);
  });
} catch (...) {
  return MOE_ERR_CUDA;
}
