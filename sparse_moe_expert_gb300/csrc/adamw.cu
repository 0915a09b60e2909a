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
// holds its own and nothing is kept between calls.  CTAs walk over units of 2048
// elements, all of them close together; a thread takes eight consecutive ones, a warp
// one block of 256, and the next unit is on its way during the present one.
//
// Measured, 64M fp32 elements with bf16 gradients: 32 bits 257 us, 6.5 TB/s, .95 of the
// copy rate (CTAs that stay 290, runs of units per CTA 263); 8 bits 195 us, 4.6 TB/s,
// bound by its 75 instructions per element (runs of units 206, eight CTAs per SM's
// worth of them 223).
#include <math.h>

#include <algorithm>
#include <vector>

#include "dense.cuh"

namespace moe {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = kAdamThreads * 8;
constexpr int kAdamCtas = 3;  // resident per SM
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
  int tiny_eps;   // so small that a root below 2^-63 counts beside it
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

// Pairs of values: one instruction for both.  Each result is rounded on its own, but
// a product and a sum that follow each other may be joined.
__device__ __forceinline__ float2 mul2_rn(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ float2 decode_m2(float2 c, float s) {
  const float2 a = mul2_rn(c, both((float)(1.0 / 127.0)));
  return mul2_rn(mul2_rn(a, make_float2(fabsf(a.x), fabsf(a.y))), both(s));
}
__device__ __forceinline__ float2 decode_r2(float2 c, float s) {
  const float2 a = mul2_rn(c, both((float)(1.0 / 255.0)));
  return mul2_rn(mul2_rn(a, a), both(s));
}
// Bytes e and e + 1 of w, which become floats without a conversion, as the end of
// 2^23's mantissa.
__device__ __forceinline__ float2 byte_floats(uint32_t w, int e) {
  return add2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (uint32_t)e)),
                             __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441u + (uint32_t)e))),
                 both(-8388608.0f));
}
__device__ __forceinline__ float2 signed_byte_floats(uint32_t w, int e) {
  const uint32_t u = w ^ 0x80808080u;
  return add2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u | (uint32_t)e)),
                             __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441u + (uint32_t)e))),
                 both(-8388736.0f));
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
__device__ __forceinline__ void round_codes(float2 t, uint32_t& a, uint32_t& b, float& off) {
  const float2 q = add2_rn(t, both(kRound));
  const float2 d = ffma2(add2_rn(q, both(-kRound)), both(-1.0f), t);
  off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
  a = __float_as_uint(q.x);
  b = __float_as_uint(q.y);
}
// The lowest bytes of four words.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
}

// The block's largest magnitude; a NaN counts as largest.
__device__ __forceinline__ float block_max(const float2 (&x)[4]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    top = max(top, max(__float_as_uint(x[i].x) & 0x7FFFFFFFu, __float_as_uint(x[i].y) & 0x7FFFFFFFu));
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
__device__ __forceinline__ void load8(Vec8<BF16>& v, const void* p, int64_t at, int n, bool vec) {
  if (vec && n == 8) v.load(p, at);
  else v.load_some(p, at, n);
}
template <bool BF16>
__device__ __forceinline__ void store8(const float2 (&p)[4], void* d, int64_t at, int n, bool vec) {
  const float f[8] = {p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
  Vec8<BF16> v;
  v.set(f);
  if (vec && n == 8) v.store(d, at);
  else v.store_some(d, at, n);
}
template <bool BF16>
__device__ __forceinline__ void pairs(float2 (&p)[4], const Vec8<BF16>& v) {
  float f[8];
  v.get(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

__device__ __forceinline__ bool at16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// What a thread reads of eight elements, as loaded; zeros past the tensor's end,
// which the step leaves zero, so that they do not count in a block's scale.
template <int PARAM, bool G_BF16, bool EIGHT>
struct AdamRaw {
  Vec8<G_BF16> g;
  Vec8<PARAM == kParamBf16> w;
  Vec8<false> m, v;  // 32-bit states
  uint2 cm, cv;      // 8-bit states, their scales
  float sm, sr;
};

// A unit of a tensor: where this thread's elements are.
struct AdamPlace {
  int ti;
  int64_t at;
  int n;  // 0 .. 8
  bool vec;
};

template <int CAP, int PARAM, bool G_BF16, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas)
    adamw_kernel(const __grid_constant__ AdamTable<CAP> tab, AdamParams p) {
  __shared__ float correction[2];  // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  pdl_wait();
  // No early trigger: a kernel behind this one may read weights before its own
  // wait, and these are weights.
  const int tid = threadIdx.x, lane = tid & 31;
  const float scale = p.grad_scale ? *p.grad_scale : 1.0f;
  if (!(fabsf(scale) < INFINITY)) return;  // for every thread alike
  const int units = tab.first[tab.count];
  using Raw = AdamRaw<PARAM, G_BF16, EIGHT>;
  auto place = [&](int u, int ti) {
    while (u >= tab.first[ti + 1]) ++ti;
    const AdamTensor& t = tab.t[ti];
    AdamPlace a;
    a.ti = ti;
    a.at = (int64_t)(u - tab.first[ti]) * kAdamUnit + tid * 8;
    const int64_t left = t.n - a.at;
    a.n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    a.vec = at16(t.param) && at16(t.grad) && at16(t.master) && at16(t.m) && at16(t.v);
    return a;
  };
  auto load = [&](Raw& r, const AdamPlace& a) {
    const AdamTensor& t = tab.t[a.ti];
    load8(r.g, t.grad, a.at, a.n, a.vec);
    load8(r.w, PARAM == kParamMaster ? (const void*)t.master : t.param, a.at, a.n, a.vec);
    if constexpr (EIGHT) {
      const int64_t b = a.at / kAdamBlock;
      const bool on = b * kAdamBlock < t.n;
      r.sm = on ? t.m_scale[b] : 0.0f;
      r.sr = on ? t.v_scale[b] : 0.0f;
      r.cm = load_codes(t.m, a.at, a.n, a.vec);
      r.cv = load_codes(t.v, a.at, a.n, a.vec);
    } else {
      load8(r.m, t.m, a.at, a.n, a.vec);
      load8(r.v, t.v, a.at, a.n, a.vec);
    }
  };
  AdamPlace here = {}, next = {};
  Raw raw, ahead;
  if (blockIdx.x < units) {
    here = place(blockIdx.x, tensor_of(tab, blockIdx.x));
    load(raw, here);
  }
  int done = 0;
  if (tid < 2) {
    done = *reinterpret_cast<volatile int32_t*>(p.step);
    const double left = 1.0 - power(tid ? p.beta2 : p.beta1, done + 1);
    correction[tid] = (float)(1.0 / (tid ? sqrt(left) : left));
  }
  __syncthreads();
  const float c1 = correction[0], c2 = correction[1];
  const float lr = p.lr_dev ? *p.lr_dev : p.lr;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    if (u < units - (int)gridDim.x) {  // the next unit is on its way during this one
      next = place(u + gridDim.x, here.ti);
      load(ahead, next);
    }
    const AdamTensor& t = tab.t[here.ti];
    const int64_t at = here.at;
    const int n = here.n;
    const bool vec = here.vec;
    float2 w[4], g[4], m[4], v[4];
    pairs(g, raw.g);
    pairs(w, raw.w);
    if constexpr (EIGHT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = decode_m2(signed_byte_floats(i < 2 ? raw.cm.x : raw.cm.y, 2 * i & 3), raw.sm);
        const float2 r = decode_r2(byte_floats(i < 2 ? raw.cv.x : raw.cv.y, 2 * i & 3), raw.sr);
        v[i] = mul2_rn(r, r);
      }
    } else {
      pairs(m, raw.m);
      pairs(v, raw.v);
    }
    const float keep = p.lr_dev ? fmaf(-lr, t.decay, 1.0f) : t.keep;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = mul2_rn(g[i], both(scale));
      // products and sums one by one: the compiler may join those of pairs
      m[i].x = __fadd_rn(__fmul_rn(m[i].x, p.b1), __fmul_rn(g[i].x, p.a1));
      m[i].y = __fadd_rn(__fmul_rn(m[i].y, p.b1), __fmul_rn(g[i].y, p.a1));
      const float2 q = mul2_rn(g[i], g[i]);
      v[i].x = __fadd_rn(__fmul_rn(v[i].x, p.b2), __fmul_rn(q.x, p.a2));
      v[i].y = __fadd_rn(__fmul_rn(v[i].y, p.b2), __fmul_rn(q.y, p.a2));
      g[i] = mul2_rn(m[i], both(c1));
    }
    if (p.tiny_eps) {  // second moments below 2^-126 matter then
#pragma unroll
      for (int i = 0; i < 4; ++i)
        g[i] = make_float2(__fdiv_rn(g[i].x, fmaf(__fsqrt_rn(v[i].x), c2, p.eps)),
                           __fdiv_rn(g[i].y, fmaf(__fsqrt_rn(v[i].y), c2, p.eps)));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = ffma2(make_float2(sqrt_approx(v[i].x), sqrt_approx(v[i].y)), both(c2), both(p.eps));
        g[i] = mul2_rn(g[i], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ffma2(g[i], both(-lr), mul2_rn(w[i], both(keep)));
    if constexpr (PARAM != kParamF32) store8<true>(w, t.param, at, n, vec);
    if constexpr (PARAM != kParamBf16)
      store8<false>(w, PARAM == kParamMaster ? (void*)t.master : t.param, at, n, vec);
    if constexpr (EIGHT) {
      float im, ir;
      const float sm = block_scale(block_max(m), im);
      const float top = block_max(v), sr = block_scale(__fsqrt_rn(top), ir);  // the root keeps the order
      uint32_t cm[8], cv[8];
      // A hardware root is 2^-23 of itself off.  With the roundings after it m's code is
      // 127 (1 + 1/2) 2^-23 = 2.3e-5 off, v's, whose first error the second root halves,
      // 255 (1/2 + 1 + 3/4) 2^-23 = 6.9e-5.
      float off_m = 0.0f, off_v = 0.0f;
      auto code = [&](int i, float2 a, float2 b) {
        a = make_float2(__fmul_rn(a.x, 127.0f), __fmul_rn(a.y, 127.0f));
        b = make_float2(__fmul_rn(b.x, 255.0f), __fmul_rn(b.y, 255.0f));
        round_codes(make_float2(copysignf(a.x, m[i].x), copysignf(a.y, m[i].y)), cm[2 * i], cm[2 * i + 1], off_m);
        round_codes(make_float2(v[i].x > 0.0f ? fmaxf(b.x, 1.0f) : b.x, v[i].y > 0.0f ? fmaxf(b.y, 1.0f) : b.y),
                    cv[2 * i], cv[2 * i + 1], off_v);
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = mul2_rn(make_float2(fabsf(m[i].x), fabsf(m[i].y)), both(im));
        const float2 y = mul2_rn(make_float2(sqrt_approx(v[i].x), sqrt_approx(v[i].y)), both(ir));
        code(i, make_float2(sqrt_approx(x.x), sqrt_approx(x.y)), make_float2(sqrt_approx(y.x), sqrt_approx(y.y)));
      }
      // Near a border, or so small that the hardware's root loses some: it takes a v below
      // 2^-126 for zero, whose code becomes 1.  That is the formula's, 255 (v / top)^(1/4) <
      // 1.5, where top > 2^-126 (255 / 1.5)^4 = 2^-96.4.
      if (off_m > 0.49996f || off_v > 0.4999f || top < 0x1p-96f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = mul2_rn(make_float2(fabsf(m[i].x), fabsf(m[i].y)), both(im));
          const float2 y = mul2_rn(make_float2(__fsqrt_rn(v[i].x), __fsqrt_rn(v[i].y)), both(ir));
          code(i, make_float2(__fsqrt_rn(x.x), __fsqrt_rn(x.y)), make_float2(__fsqrt_rn(y.x), __fsqrt_rn(y.y)));
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
    here = next;
    raw = ahead;
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
// 16-byte pieces from the first boundary on, the codes shifted to fit.  A CTA per unit:
// 400 tensors, 52M elements, 108 us, .71 of the copy rate (the codes of one state after
// the other's 115; so with eight CTAs per SM that walk 115, with four 148).
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_values_kernel(const __grid_constant__ AdamTable<CAP> tab) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ti = tensor_of(tab, blockIdx.x);
  const AdamTensor& t = tab.t[ti];
  const int64_t b = (int64_t)(blockIdx.x - tab.first[ti]) * (kAdamUnit / kAdamBlock) + warp;
  if (b * kAdamBlock >= t.n) return;
  const float scale[2] = {t.m_scale[b], t.v_scale[b]};
  const int n = (int)min((int64_t)kAdamBlock, t.n - b * kAdamBlock);
  const uint8_t* codes[2] = {static_cast<const uint8_t*>(t.m) + b * kAdamBlock,
                             static_cast<const uint8_t*>(t.v) + b * kAdamBlock};
  float* outs[2] = {static_cast<float*>(t.param) + b * kAdamBlock, t.master + b * kAdamBlock};
  bool words[2];
  int head[2], quads[2];  // values in front of the first boundary, pieces
  uint32_t four[2][2];    // a lane's codes: all are on their way before the first store
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    words[h] = (reinterpret_cast<uintptr_t>(codes[h]) & 3u) == 0;
    head[h] = (int)((16u - (reinterpret_cast<uintptr_t>(outs[h]) & 15u)) & 15u) / 4;
    // pieces whose words of codes are all there
    quads[h] = words[h] ? max(head[h] ? n / 4 - 1 : n / 4, 0) : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = i * 32 + lane;
      if (q >= quads[h]) continue;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(codes[h]) + q;
      const uint32_t lo = w[0], hi = head[h] ? w[1] : 0u;
      four[h][i] = __funnelshift_r(lo, hi, head[h] * 8);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* out = outs[h];
    auto values = [&](uint32_t w, int e) {  // of bytes e and e + 1
      if (h == 0) return decode_m2(signed_byte_floats(w, e), scale[0]);
      const float2 r = decode_r2(byte_floats(w, e), scale[1]);
      return mul2_rn(r, r);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = i * 32 + lane;
      if (q >= quads[h]) continue;
      const float2 a = values(four[h][i], 0), b = values(four[h][i], 2);
      *reinterpret_cast<float4*>(out + head[h] + 4 * q) = make_float4(a.x, a.y, b.x, b.y);
    }
    if (words[h]) {  // what lies before the first boundary and behind the last piece
      if (lane < head[h] && lane < n) out[lane] = values(codes[h][lane], 0).x;
      const int e = head[h] + 4 * quads[h] + lane;
      if (lane < 8 && e < n) out[e] = values(codes[h][e], 0).x;
    } else {
      for (int e = lane; e < n; e += 32) out[e] = values(codes[h][e], 0).x;
    }
  }
}

// ---- host ------------------------------------------------------------------

using moe_host::aligned4;

int64_t units_of(int64_t n) { return (n + kAdamUnit - 1) / kAdamUnit; }

template <int CAP>
moe_status_t launch_step(const AdamTable<CAP>& tab, const AdamParams& p, int param, bool g_bf16,
                         bool eight, cudaStream_t st) {
  // 8 bits: CTAs that stay; 32 bits: more than fit, each done sooner (both sides above)
  const int64_t most = (int64_t)moe_host::sm_count() * (eight ? kAdamCtas : 8);
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
        if (next > (1 << 30)) break;  // never with the first: n has a limit
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

struct Span {
  uintptr_t lo, hi;
};
// The buffers of one kind, by address.  Tensors made one after the other are mostly in order.
struct Spans {
  std::vector<Span> v;
  uintptr_t top = 0;     // behind the last byte of any
  bool sorted = true;
  void add(const void* p, int64_t bytes) {
    if (!p || bytes == 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + (uintptr_t)bytes;
    sorted = sorted && (v.empty() || v.back().lo <= lo);
    top = hi > top ? hi : top;
    v.push_back({lo, hi});
  }
  void order() {
    if (!sorted) std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  }
};
// Ordered buffers of one kind that share nothing.
bool apart(const Spans& s) {
  for (size_t i = 1; i < s.v.size(); ++i)
    if (s.v[i].lo < s.v[i - 1].hi) return false;
  return true;
}
// None of b's shares memory with one of a's, which share nothing; both ordered.
bool apart(const Spans& a, const Spans& b) {
  if (a.v.empty() || b.v.empty() || a.top <= b.v.front().lo || b.top <= a.v.front().lo) return true;
  size_t i = 0;
  for (const Span& s : b.v) {
    while (i < a.v.size() && a.v[i].hi <= s.lo) ++i;
    if (i == a.v.size()) return true;
    if (a.v[i].lo < s.hi) return false;
  }
  return true;
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
  // what is written (param, master, states and their scales), and the gradients
  constexpr int kWritten = 6;
  Spans kinds[kWritten + 1];
  for (auto& k : kinds) k.v.reserve(count);
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
    const int64_t state = t.n * (eight ? 1 : 4), scales = eight ? (t.n + kAdamBlock - 1) / kAdamBlock * 4 : 0;
    kinds[0].add(t.param, t.n * psize);
    kinds[1].add(t.master, t.n * 4);
    kinds[2].add(t.exp_avg, state);
    kinds[3].add(t.exp_avg_sq, state);
    kinds[4].add(t.exp_avg_scale, scales);
    kinds[5].add(t.exp_avg_sq_scale, scales);
    kinds[kWritten].add(t.grad, t.n * gsize);
  }
  if (masters != 0 && masters != (int)all.size()) return MOE_ERR_UNSUPPORTED;
  // what one CTA writes no other may read or write
  for (auto& k : kinds) k.order();
  for (int i = 0; i < kWritten; ++i) {
    if (!apart(kinds[i])) return MOE_ERR_INVALID_ARG;
    for (int j = i + 1; j <= kWritten; ++j)
      if (!apart(kinds[i], kinds[j])) return MOE_ERR_INVALID_ARG;
  }
  // The hardware's root takes v below 2^-126 for zero: the divisor loses up to 2^-63 / sqrt(1
  // - beta2^t), which is 2^-23 of eps or less from here on (2.9e-11 for beta2 = 0.999).
  const bool tiny_eps = eps < 0x1p-40 / sqrt(1.0 - beta2);
  AdamParams p{beta1, beta2, (float)beta1, (float)beta2, (float)(1.0 - beta1), (float)(1.0 - beta2),
               (float)eps, (float)lr, lr_dev, grad_scale, step, 0,
               tiny_eps};
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
    return moe_host::launch(adamw_values_kernel<kCap>, dim3((unsigned)tab.first[tab.count]),
                            dim3(kAdamThreads), 0, st, tab);
  });
} catch (...) {
  return MOE_ERR_CUDA;
}
