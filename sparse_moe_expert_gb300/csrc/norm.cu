// Layer and RMS norm of rows, and their gradient.
//
// With s = x (+ residual, rounded to x's type and stored), over a row of H:
//   mu   = mean s (RMS: 0),  rstd = (mean (s - mu)^2 + eps)^-1/2
//   out  = (s - mu) rstd w + b
// and backwards, with xh = (s - mu) rstd and c = d w:
//   d_s  = rstd (c - mean c - xh mean(c xh)) (+ d_sum)      (RMS: no mean c)
//   d_w  = sum_t d xh,   d_b = sum_t d
// The row stays in registers between its sums, so each value is read once; the
// variance is summed from the centred values.  All sums are fp32 in an order
// that the sizes fix.  A thread owns columns, and in the gradient it keeps
// their d_w and d_b over all rows of its CTA; the CTAs' sums are joined by a
// second kernel in the CTAs' order, those of a few rows by their cluster.
//
// Bound by the bytes where there are many rows, by launch and latency where there are
// few.  Measured (device time, share of the copy rate): norm of 1 x 4096 bf16 with
// residual 2.4 us; of 8192 x 4096 bf16 with weight and bias 26.6, .74; gradient of 64 x
// 2048 fp32 6.5; of 16384 x 4096 bf16 with d_sum 101, .78.
#include "async.cuh"
#include "dense.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kNormMaxWidth = 8192;  // 512 threads with two vectors of eight each
constexpr int kNormWarpWidth = 512;  // up to this width a warp takes a row
// Rows from which warps take a row each of wider ones as well (us, a CTA per row and a
// warp: bf16 4096 wide, 608 rows 4.3, 5.1; 1024 7.4, 5.9; 16384 69, 45; 8192 wide, 608
// 7.3, 9.3; 1024 13.8, 10.9; fp32 4096 wide, 608 5.3, 5.1; 1024 9.8, 7.6; but fp32 8192
// wide, whose rows fill the registers, 16384 216, 361).
constexpr int kNormWarpRows = 1024;

struct NormParams {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  const void* bias;
  int w_bf16;
  int T, H;
  float eps;
  int rms;
  void* out;
  void* summed;
  float* mean;
  float* rstd;
};

// Column of value e of a thread's vector j.  VEC: eight consecutive ones;
// else neighbours lie in neighbouring threads.
template <bool VEC>
__device__ __forceinline__ int column(int j, int e) {
  return VEC ? (j * (int)blockDim.x + (int)threadIdx.x) * 8 + e
             : (j * 8 + e) * (int)blockDim.x + (int)threadIdx.x;
}

template <bool BF16, bool VEC>
struct RowVec {
  Vec8<BF16> v;
  // columns of vector j of the row at p; zeros past H
  __device__ __forceinline__ void load(const void* p, int64_t row, int j, int H) {
    if constexpr (VEC) {
      const int c = column<true>(j, 0);
      if (c < H) v.load(p, row + c);
      else v.zero();
    } else {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(j, e);
        if constexpr (BF16) w[e] = c < H ? static_cast<const uint16_t*>(p)[row + c] : 0u;
        else w[e] = c < H ? static_cast<const uint32_t*>(p)[row + c] : 0u;
      }
      if constexpr (BF16) {
        v.q[0] = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                            w[6] | (w[7] << 16));
      } else {
        v.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        v.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t row, int j, int H) const {
    if constexpr (VEC) {
      const int c = column<true>(j, 0);
      if (c < H) v.store(p, row + c);
    } else if constexpr (BF16) {
      const uint32_t w[4] = {v.q[0].x, v.q[0].y, v.q[0].z, v.q[0].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(j, e);
        if (c < H) static_cast<uint16_t*>(p)[row + c] = (uint16_t)(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
      }
    } else {
      float f[8];
      v.get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(j, e);
        if (c < H) static_cast<float*>(p)[row + c] = f[e];
      }
    }
  }
};

// Weight or bias at a thread's vector j.
template <bool VEC>
__device__ __forceinline__ void load_param(float (&f)[8], const void* p, int bf16, int j, int H) {
  if (bf16) {
    RowVec<true, VEC> v;
    v.load(p, 0, j, H);
    v.v.get(f);
  } else {
    RowVec<false, VEC> v;
    v.load(p, 0, j, H);
    v.v.get(f);
  }
}

// blockDim.x threads take a row; blockDim.y rows per CTA when those are a warp.
template <bool X_BF16, bool OUT_BF16, int NV, bool VEC>
__global__ void __launch_bounds__(512) layer_norm_kernel(NormParams p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_trigger();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.T) return;  // whole warps, which are on their own where there is more than one row
  float f[NV][8];
  RowVec<X_BF16, VEC> x[NV], r[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j].load(p.x, t * p.ldx, j, p.H);
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j].load(p.residual, t * p.ldr, j, p.H);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j].v.get(f[j]);
    if (p.residual) {
      float g[8];
      r[j].v.get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[j][e] += g[e];
      x[j].v.set(f[j]);
      x[j].store(p.summed, t * p.H, j, p.H);
      x[j].v.get(f[j]);  // the sum as stored
    }
  }
  const float inv_h = 1.0f / (float)p.H;
  float mu = 0.0f;
  if (!p.rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += f[j][e];
    block_sum(s, part[0]);
    mu = s[0] * inv_h;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (column<VEC>(j, e) < p.H) f[j][e] -= mu;
      q[0] = fmaf(f[j][e], f[j][e], q[0]);
    }
  block_sum(q, part[1]);
  const float rstd = 1.0f / sqrtf(q[0] * inv_h + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[t] = mu;
    if (p.rstd) p.rstd[t] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f[j][e] * rstd;
    if (p.weight) {
      float w[8];
      load_param<VEC>(w, p.weight, p.w_bf16, j, p.H);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= w[e];
    }
    if (p.bias) {
      float b[8];
      load_param<VEC>(b, p.bias, p.w_bf16, j, p.H);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += b[e];
    }
    RowVec<OUT_BF16, VEC> o;
    o.v.set(y);
    o.store(p.out, t * p.H, j, p.H);
  }
}

// ---- gradient ----------------------------------------------------------------

struct NormGradParams {
  const void* d_out;
  int64_t ldd;
  const void* x;
  int64_t ldx;
  const void* d_sum;
  int64_t lds;
  const float* mean;  // null: RMS
  const float* rstd;
  const void* weight;
  int w_bf16;
  int T, H;
  void* d_x;
  float* part;  // [CTAs][2][H], or null: no weight or bias gradient
};

// CTAs walk over rows; the next row's values are on their way while the
// present one is summed.
template <bool D_BF16, bool X_BF16, int NV, bool VEC>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(NormGradParams p) {
  extern __shared__ __align__(16) float join[];  // [rows][2][H], where a CTA takes several rows
  __shared__ float part[2][2][32];
  pdl_wait();
  pdl_trigger();
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.0f;
  const float inv_h = 1.0f / (float)p.H;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowVec<D_BF16, VEC> d[NV];
  RowVec<X_BF16, VEC> x[NV], s[NV];
  float mu = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      d[j].load(p.d_out, row * p.ldd, j, p.H);
      x[j].load(p.x, row * p.ldx, j, p.H);
      if (p.d_sum) s[j].load(p.d_sum, row * p.lds, j, p.H);
    }
    mu = p.mean ? p.mean[row] : 0.0f;
    rstd = p.rstd[row];
  };
  if (t < p.T) fetch(t);
  int buf = 0;
  for (; t < p.T; t += step, buf ^= 1) {
    const float r = rstd;
    float c[NV][8], xh[NV][8], ds[NV][8];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8];
      d[j].v.get(c[j]);
      x[j].v.get(xh[j]);
      if (p.d_sum) s[j].v.get(ds[j]);
      if (p.weight) load_param<VEC>(w, p.weight, p.w_bf16, j, p.H);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[j][e] = column<VEC>(j, e) < p.H ? (xh[j][e] - mu) * r : 0.0f;
        db[j][e] += c[j][e];
        dw[j][e] = fmaf(c[j][e], xh[j][e], dw[j][e]);
        if (p.weight) c[j][e] *= w[e];
        sum[0] += c[j][e];
        sum[1] = fmaf(c[j][e], xh[j][e], sum[1]);
      }
    }
    if (t + step < p.T) fetch(t + step);
    block_sum(sum, part[buf][0]);
    const float m0 = p.mean ? sum[0] * inv_h : 0.0f, m1 = sum[1] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = r * (c[j][e] - m0 - xh[j][e] * m1);
        if (p.d_sum) y[e] += ds[j][e];
      }
      RowVec<X_BF16, VEC> o;
      o.v.set(y);
      o.store(p.d_x, t * p.H, j, p.H);
    }
  }
  if (!p.part) return;
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.H;
  const bool several = blockDim.y > 1;
  float* mine = several ? join + (int64_t)threadIdx.y * 2 * p.H : out;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    RowVec<false, VEC> o;
    o.v.set(dw[j]);
    o.store(mine, 0, j, p.H);
    o.v.set(db[j]);
    o.store(mine, p.H, j, p.H);
  }
  if (!several) return;
  __syncthreads();
  for (int i = threadIdx.y * 32 + threadIdx.x; i < 2 * p.H; i += 32 * blockDim.y) {
    float s = join[i];
    for (int w = 1; w < (int)blockDim.y; ++w) s += join[w * 2 * p.H + i];
    out[i] = s;
  }
}

// ---- many rows of whole vectors ---------------------------------------------------

// Pairs of fp32 values (one instruction for both).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return ffma2(a, make_float2(1.0f, 1.0f), b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return ffma2(a, b, make_float2(0.0f, 0.0f)); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
// (x - mu) rstd.  The mean goes first: x rstd - mu rstd in one operation less keeps the
// rounding of mu rstd, the same one for a whole row (xh of rows whose mean is 1e3 of their
// deviations 2e-5 of itself off, against 3e-8).
__device__ __forceinline__ float2 centred(float2 x, float mu, float rstd) {
  return mul2(add2(x, both(-mu)), both(rstd));
}

template <bool BF16>
__device__ __forceinline__ void get2(float2 (&f)[4], const Vec8<BF16>& v) {
  if constexpr (BF16) {
    const uint32_t w[4] = {v.q[0].x, v.q[0].y, v.q[0].z, v.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = bf16x2_to_f32x2(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = make_float2(__uint_as_float(v.q[i].x), __uint_as_float(v.q[i].y));
      f[2 * i + 1] = make_float2(__uint_as_float(v.q[i].z), __uint_as_float(v.q[i].w));
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void set2(Vec8<BF16>& v, const float2 (&f)[4]) {
  const float g[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  v.set(g);
}
__device__ __forceinline__ void load2(float2 (&f)[4], const void* p, int bf16, int col) {
  if (bf16) {
    Vec8<true> v;
    v.load(p, col);
    get2(f, v);
  } else {
    Vec8<false> v;
    v.load(p, col);
    get2(f, v);
  }
}

// A warp takes a row, which it holds as loaded (packed) between its sums, so no
// warp waits for another; a bulk copy brings its next row into shared memory
// meanwhile.  Weight and bias lie there as fp32, [H] each, in front of the rows: from
// global memory they would not stay in the L1 that is left.  One CTA per SM, its
// warps as many as registers and shared memory allow.  8192 x 4096 bf16, us: 26.6 (a CTA
// per row 37, rows in shared memory read three times 40, weights through L1 43 to 56).
// Dynamic shared memory of a CTA, at most, and of one of `n` per SM (which has 228 KB
// and keeps 1 KB for each).
constexpr size_t kNormRoom = 226 * 1024;
constexpr int norm_room(int n) {
  const int share = 228 * 1024 / n - 1536;
  return share < (int)kNormRoom ? share : (int)kNormRoom;
}
// Warps whose rows (4 or 8 registers per vector and lane) the registers hold.
constexpr int warp_rows_most(bool bf16, int nv) { return nv * (bf16 ? 4 : 8) <= 64 ? 16 : 12; }

template <bool X_BF16, bool OUT_BF16, int NV>
__global__ void __launch_bounds__(warp_rows_most(X_BF16, NV) * 32, 1)
    layer_norm_warp_kernel(NormParams p, int stage_bytes, unsigned int* err) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int params = (p.weight ? 1 : 0) + (p.bias ? 1 : 0);
  float* w_s = reinterpret_cast<float*>(smem);
  float* b_s = w_s + (p.weight ? p.H : 0);
  unsigned char* at = smem + (size_t)params * p.H * 4 + (size_t)warp * stage_bytes;
  uint64_t* bar = bars + warp;
  const uint32_t x_bytes = p.H * (X_BF16 ? 2 : 4);
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  auto fetch = [&](int64_t t) {  // by lane 0
    mbar_arrive_expect_tx(bar, p.residual ? 2 * x_bytes : x_bytes);
    bulk_g2s(at, static_cast<const unsigned char*>(p.x) + t * p.ldx * (X_BF16 ? 2 : 4), x_bytes, bar);
    if (p.residual)
      bulk_g2s(at + x_bytes, static_cast<const unsigned char*>(p.residual) + t * p.ldr * (X_BF16 ? 2 : 4),
               x_bytes, bar);
  };
  // neighbouring rows go to different SMs, so that the last turn is shared out
  const int64_t step = (int64_t)gridDim.x * warps;
  int64_t t = (int64_t)warp * gridDim.x + blockIdx.x;
  if (t < p.T && lane == 0) fetch(t);
  for (int c = threadIdx.x * 8; c < p.H; c += blockDim.x * 8) {
    float2 f[4];
    Vec8<false> v;
    if (p.weight) {
      load2(f, p.weight, p.w_bf16, c);
      set2(v, f);
      v.store(w_s, c);
    }
    if (p.bias) {
      load2(f, p.bias, p.w_bf16, c);
      set2(v, f);
      v.store(b_s, c);
    }
  }
  __syncthreads();
  const float inv_h = 1.0f / (float)p.H;
  uint32_t phase = 0;
  for (; t < p.T; t += step, phase ^= 1u) {
    const bool ok = mbar_wait(bar, phase, kWaitBudgetCycles);
    if (!__all_sync(0xFFFFFFFFu, ok)) {  // its copy has not ended in a second: nothing else to wait for
      if (lane == 0) raise_device_error(err, MOE_DEVERR_TIMEOUT);
      return;
    }
    Vec8<X_BF16> x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * 32 + lane) * 8;
      if (c < p.H) x[j].load(at, c);
      else x[j].zero();
    }
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * 32 + lane) * 8;
        if (c >= p.H) continue;
        Vec8<X_BF16> r;
        float2 f[4], g[4];
        r.load(at + x_bytes, c);
        get2(f, x[j]);
        get2(g, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = add2(f[i], g[i]);
        set2(x[j], f);
        x[j].store(p.summed, t * p.H + c);
      }
    }
    __syncwarp();
    if (lane == 0 && t + step < p.T) fetch(t + step);
    float mu = 0.0f;
    if (!p.rms) {
      float2 s2[2] = {};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2 f[4];
        get2(f, x[j]);
        s2[j & 1] = add2(s2[j & 1], add2(add2(f[0], f[1]), add2(f[2], f[3])));
      }
      float s[1] = {(s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)};
      warp_sum(s);
      mu = s[0] * inv_h;
    }
    float2 q2[2] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if ((j * 32 + lane) * 8 >= p.H) continue;
      float2 f[4];
      get2(f, x[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = add2(f[i], both(-mu));
        q2[i & 1] = ffma2(d, d, q2[i & 1]);
      }
    }
    float q[1] = {(q2[0].x + q2[0].y) + (q2[1].x + q2[1].y)};
    warp_sum(q);
    const float rstd = 1.0f / sqrtf(q[0] * inv_h + p.eps);
    if (lane == 0) {
      if (p.mean) p.mean[t] = mu;
      if (p.rstd) p.rstd[t] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * 32 + lane) * 8;
      if (c >= p.H) continue;
      float2 f[4], w[4];
      get2(f, x[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(add2(f[i], both(-mu)), both(rstd));
      if (p.weight) {
        load2(w, w_s, 0, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w[i]);
      }
      if (p.bias) {
        load2(w, b_s, 0, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = add2(f[i], w[i]);
      }
      Vec8<OUT_BF16> o;
      set2(o, f);
      o.store(p.out, t * p.H + c);
    }
  }
}

// The gradient: bulk copies bring the rows of a CTA's next turns into shared memory
// while it works on one.  A thread takes NV vectors of eight columns.  One vector
// leaves registers for its weights and for two CTAs of 512 threads per SM; two of them
// need twice the registers, and the weights lie in shared memory in front of the rows
// (bf16 with d_sum, us with one vector and two: 16384 x 4096 98, 123; 4096 x 8192,
// where one takes CTAs of 1024 threads, 64, 49).
constexpr int kRingMost = 8;
constexpr int kRingThreads = 512;
struct RingPlan {
  int nv, threads, per_sm, stages;
  int stage_bytes;
};

template <bool D_BF16, bool X_BF16, int NV>
__global__ void __launch_bounds__(kRingThreads, NV == 1 ? 2 : 1)
    layer_norm_backward_ring_kernel(NormGradParams p, int stages, int stage_bytes, unsigned int* err) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kRingMost];
  __shared__ float2 part[2][kRingThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const uint32_t d_bytes = p.H * (D_BF16 ? 2 : 4), x_bytes = p.H * (X_BF16 ? 2 : 4);
  float* w_s = reinterpret_cast<float*>(smem);
  unsigned char* rows = smem + (NV > 1 && p.weight ? (size_t)p.H * 4 : 0);
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int64_t step = gridDim.x;
  const uint32_t row_bytes = d_bytes + x_bytes + (p.d_sum ? x_bytes : 0);
  auto fetch = [&](int64_t t, int s) {  // by thread 0
    unsigned char* at = rows + (size_t)s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], row_bytes);
    bulk_g2s(at, static_cast<const unsigned char*>(p.d_out) + t * p.ldd * (D_BF16 ? 2 : 4), d_bytes, &full[s]);
    bulk_g2s(at + d_bytes, static_cast<const unsigned char*>(p.x) + t * p.ldx * (X_BF16 ? 2 : 4), x_bytes,
             &full[s]);
    if (p.d_sum)
      bulk_g2s(at + d_bytes + x_bytes, static_cast<const unsigned char*>(p.d_sum) + t * p.lds * (X_BF16 ? 2 : 4),
               x_bytes, &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s)
      if (blockIdx.x + s * step < p.T) fetch(blockIdx.x + s * step, s);
  const float2 zero = make_float2(0.0f, 0.0f);
  float2 dw[NV][4], db[NV][4], w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = both(1.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = zero;
    const int col = (j * (int)blockDim.x + tid) * 8;
    if (!p.weight || col >= p.H) continue;
    load2(w, p.weight, p.w_bf16, col);
    if constexpr (NV > 1) {  // read by this thread alone
      Vec8<false> v;
      set2(v, w);
      v.store(w_s, col);
    }
  }
  const float inv_h = 1.0f / (float)p.H;
  // the next row's statistics are on their way during this one
  float mu = 0.0f, rstd = 0.0f;
  if (blockIdx.x < p.T) {
    if (p.mean) mu = p.mean[blockIdx.x];
    rstd = p.rstd[blockIdx.x];
  }
  int s = 0, buf = 0, bad = 0;
  uint32_t phase = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += step, buf ^= 1) {
    const float r = rstd, m = mu;
    if (t + step < p.T) {
      if (p.mean) mu = p.mean[t + step];
      rstd = p.rstd[t + step];
    }
    if (!mbar_wait(&full[s], phase, kWaitBudgetCycles)) bad = 1;
    const unsigned char* at = rows + (size_t)s * stage_bytes;
    float2 c[NV][4], xh[NV][4], s0 = zero, s1 = zero;
    Vec8<X_BF16> ds[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * (int)blockDim.x + tid) * 8;
      if (col >= p.H) continue;
      Vec8<D_BF16> dv;
      Vec8<X_BF16> xv;
      dv.load(at, col);
      xv.load(at + d_bytes, col);
      if (p.d_sum) ds[j].load(at + d_bytes + x_bytes, col);
      get2(c[j], dv);
      get2(xh[j], xv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xh[j][i] = centred(xh[j][i], m, r);
        db[j][i] = add2(db[j][i], c[j][i]);
        dw[j][i] = ffma2(c[j][i], xh[j][i], dw[j][i]);
      }
      if (NV > 1 && p.weight) load2(w, w_s, 0, col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[j][i] = mul2(c[j][i], w[i]);
        s0 = add2(s0, c[j][i]);
        s1 = ffma2(c[j][i], xh[j][i], s1);
      }
    }
    float sum[2] = {s0.x + s0.y, s1.x + s1.y};
    warp_sum(sum);
    if (lane == 0) part[buf][warp] = make_float2(sum[0], sum[1]);
    bad = __syncthreads_or(bad);  // and the stage has been read
    if (bad) break;
    if (tid == 0 && t + stages * step < p.T) fetch(t + stages * step, s);
    const float2 mine = lane < warps ? part[buf][lane] : zero;
    sum[0] = mine.x;
    sum[1] = mine.y;
    warp_sum(sum);
    const float2 m0 = both(p.mean ? -r * (sum[0] * inv_h) : 0.0f), m1 = both(-r * (sum[1] * inv_h));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * (int)blockDim.x + tid) * 8;
      if (col >= p.H) continue;
      float2 g[4];
      if (p.d_sum) get2(g, ds[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[j][i] = ffma2(c[j][i], both(r), ffma2(xh[j][i], m1, m0));
        if (p.d_sum) c[j][i] = add2(c[j][i], g[i]);
      }
      Vec8<X_BF16> o;
      set2(o, c[j]);
      o.store(p.d_x, t * p.H + col);
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  if (bad) {  // copies in flight end before the CTA may
    if (tid == 0) {
      raise_device_error(err, MOE_DEVERR_TIMEOUT);
      for (int i = 0; i < stages; ++i) mbar_wait(&full[i], i < s ? phase ^ 1u : phase, kWaitBudgetCycles);
    }
    return;
  }
  if (!p.part) return;
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * (int)blockDim.x + tid) * 8;
    if (col >= p.H) continue;
    Vec8<false> o;
    set2(o, dw[j]);
    o.store(out, col);
    set2(o, db[j]);
    o.store(out, p.H + col);
  }
}

// ---- the gradient of a few rows ----------------------------------------------------
//
// One launch: groups of threads take a row each, a vector of eight per thread, and the
// CTAs of one cluster join their sums of d_w and d_b through shared memory, groups and
// then CTAs in their order.
constexpr int kFewThreads = 512;
constexpr int kFewCtas = 16;
// Rows a group takes, at most.  A call of one launch costs the host less than one of two,
// while a cluster's joint and 16 SMs cost the device more the wider the rows (us on the
// device and per call, this form and the others: 64 x 64 3.2, 6.3 and 3.2, 9.7; 64 x 2048
// fp32, two rows per group, 6.5, 6.9 and 5.8, 9.9; 128 x 2048, four, 9.2, 9.5 and 6.2, 9.8).
constexpr int kFewTurns = 2;

template <bool D_BF16, bool X_BF16>
__global__ void __launch_bounds__(kFewThreads, 1)
    layer_norm_backward_few_kernel(NormGradParams p, int per, float* d_weight, float* d_bias) {
  extern __shared__ __align__(16) float join[];  // [groups][2][H]
  __shared__ float2 part[2][kFewThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = tid / per, groups = blockDim.x / per, member = tid - group * per;
  const int col = member * 8, rank = blockIdx.x;
  const bool on = col < p.H;
  const float2 zero = make_float2(0.0f, 0.0f);
  float2 dw[4], db[4], w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dw[i] = db[i] = zero;
    w[i] = both(1.0f);
  }
  Vec8<D_BF16> d;
  Vec8<X_BF16> x, s;
  float mu = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t t) {
    if (on) {
      d.load(p.d_out, t * p.ldd + col);
      x.load(p.x, t * p.ldx + col);
      if (p.d_sum) s.load(p.d_sum, t * p.lds + col);
    } else {
      d.zero();
      x.zero();
      s.zero();
    }
    if (p.mean) mu = p.mean[t];
    rstd = p.rstd[t];
  };
  const int64_t step = (int64_t)kFewCtas * groups;
  int64_t t = (int64_t)rank * groups + group;
  if (t < p.T) fetch(t);
  if (p.weight && on) load2(w, p.weight, p.w_bf16, col);
  const float inv_h = 1.0f / (float)p.H;
  for (int buf = 0; t < p.T; t += step, buf ^= 1) {  // alike for a group
    const float r = rstd, m = mu;
    float2 c[4], xh[4], g[4], s0 = zero, s1 = zero;
    get2(c, d);
    get2(xh, x);
    if (p.d_sum) get2(g, s);
    if (t + step < p.T) fetch(t + step);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xh[i] = on ? centred(xh[i], m, r) : zero;
      db[i] = add2(db[i], c[i]);
      dw[i] = ffma2(c[i], xh[i], dw[i]);
      c[i] = mul2(c[i], w[i]);
      s0 = add2(s0, c[i]);
      s1 = ffma2(c[i], xh[i], s1);
    }
    float sum[2] = {s0.x + s0.y, s1.x + s1.y};
    warp_sum(sum);
    if (per > 32) {
      if (lane == 0) part[buf][warp] = make_float2(sum[0], sum[1]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(per) : "memory");
      const float2 mine = lane < per / 32 ? part[buf][group * (per / 32) + lane] : zero;
      sum[0] = mine.x;
      sum[1] = mine.y;
      warp_sum(sum);
    }
    const float2 m0 = both(p.mean ? -r * (sum[0] * inv_h) : 0.0f), m1 = both(-r * (sum[1] * inv_h));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = ffma2(c[i], both(r), ffma2(xh[i], m1, m0));
      if (p.d_sum) c[i] = add2(c[i], g[i]);
    }
    Vec8<X_BF16> o;
    set2(o, c);
    if (on) o.store(p.d_x, t * p.H + col);
  }
  if (on) {
    float* mine = join + group * 2 * p.H + col;
    Vec8<false> o;
    set2(o, dw);
    o.store(mine, 0);
    set2(o, db);
    o.store(mine, p.H);
  }
  __syncthreads();
  if (groups > 1) {  // into the first group's place
    for (int i = tid; i < 2 * p.H; i += blockDim.x) {
      float v = join[i];
      for (int k = 1; k < groups; ++k) v += join[k * 2 * p.H + i];
      join[i] = v;
    }
  }
  cluster_barrier();
  for (int i = rank * blockDim.x + tid; i < 2 * p.H; i += kFewCtas * blockDim.x) {
    float* out = i < p.H ? d_weight : d_bias;
    if (!out) continue;
    float f[kFewCtas];
#pragma unroll
    for (int q = 0; q < kFewCtas; ++q)
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f[q]) : "r"(cluster_addr(join + i, q)));
#pragma unroll
    for (int q = 1; q < kFewCtas; ++q) f[0] += f[q];
    out[i < p.H ? i : i - p.H] = f[0];
  }
  cluster_barrier();  // no CTA leaves while its sums are read
}

// ---- column sums ---------------------------------------------------------------

constexpr int kColThreads = 1024;
constexpr int kColLanes = kColThreads / 32;

// 32 columns per CTA; a warp sums a run of the rows, the runs are added in order.
__global__ void __launch_bounds__(kColThreads)
    column_sums_kernel(const float* part, int rows, int64_t ld, int cols, float* out, float* more) {
  __shared__ float sum[kColLanes][32];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  if (blockIdx.y) {
    part += cols;
    out = more;
  }
  if (!out) return;
  const int per = (rows + kColLanes - 1) / kColLanes;
  const int r0 = lane * per, r1 = min(r0 + per, rows);
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 16
    for (int r = r0; r < r1; ++r) s += part[r * ld + c];
  }
  sum[lane][threadIdx.x & 31] = s;
  __syncthreads();
  if (lane == 0 && c < cols) {
    s = sum[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kColLanes; ++i) s += sum[i][threadIdx.x];
    out[c] = s;
  }
}

// How a row is shared out: vectors per thread, threads, rows per CTA.
struct Shape {
  int nv, threads, rows;
};

bool type_ok(int t) { return t == MOE_DTYPE_F32 || t == MOE_DTYPE_BF16; }

// Whether rows of this tensor can be read eight values at a time.
bool vec_ok(const void* p, int dtype, int64_t ld) {
  return p == nullptr || (moe_host::aligned16(p) && (dtype == MOE_DTYPE_BF16 ? ld % 8 : ld % 4) == 0);
}

bool element_aligned(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_DTYPE_BF16 ? 1u : 3u)) == 0;
}

Shape norm_shape(int H, int want) {
  const int vecs = (H + 7) / 8;
  if (H <= kNormWarpWidth) return {vecs <= 32 ? 1 : 2, 32, 8};
  int nv = want;
  if (vecs > 512) nv = 2;
  return {nv, ((vecs + nv - 1) / nv + 31) / 32 * 32, 1};
}

// CTAs of one vector per thread make 1024 threads per SM, of narrow rows eight CTAs;
// then as many stages as the shared memory holds.
RingPlan ring_plan(int H, int row_bytes, int weight_bytes) {
  RingPlan r;
  r.nv = H <= kRingThreads * 8 ? 1 : 2;
  r.threads = ((H / 8 + r.nv - 1) / r.nv + 31) / 32 * 32;
  r.per_sm = r.nv == 2 ? 1 : 1024 / r.threads < 8 ? 1024 / r.threads : 8;
  r.stage_bytes = row_bytes;
  auto stages = [&] { return (norm_room(r.per_sm) - weight_bytes) / row_bytes; };
  while (r.per_sm > 1 && stages() < 2) --r.per_sm;
  r.stages = stages() < kRingMost ? stages() : kRingMost;
  return r;
}

template <bool X_BF16, bool OUT_BF16, bool VEC>
moe_status_t launch_norm(const NormParams& p, const Shape& s, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)p.T + s.rows - 1) / s.rows)), block(s.threads, s.rows);
  using moe_host::launch;
  if (s.nv == 1) return launch(layer_norm_kernel<X_BF16, OUT_BF16, 1, VEC>, grid, block, 0, st, p);
  return launch(layer_norm_kernel<X_BF16, OUT_BF16, 2, VEC>, grid, block, 0, st, p);
}

template <bool D_BF16, bool X_BF16, bool VEC>
moe_status_t launch_norm_grad(const NormGradParams& p, const Shape& s, int grid, cudaStream_t st) {
  const dim3 block(s.threads, s.rows);
  const size_t smem = s.rows > 1 ? (size_t)s.rows * p.H * 8 : 0;
  using moe_host::launch;
  if (s.nv == 1)
    return launch(layer_norm_backward_kernel<D_BF16, X_BF16, 1, VEC>, grid, block, smem, st, p);
  return launch(layer_norm_backward_kernel<D_BF16, X_BF16, 2, VEC>, grid, block, smem, st, p);
}

// CTAs of the gradient, at most: as many as the workspace has room for.
int norm_grad_ctas(int64_t T, int H) {
  const Shape s = norm_shape(H, 2);
  const int per_sm = s.rows > 1 ? 4 : ring_plan((H + 7) / 8 * 8, 1, 0).per_sm;
  const int64_t most = (int64_t)moe_host::sm_count() * per_sm;
  const int64_t need = (T + s.rows - 1) / s.rows;
  return (int)(need < most ? need : most);
}

template <auto Kernel>
moe_status_t launch_ring(const NormGradParams& p, const RingPlan& r, int weight_bytes, int grid,
                         cudaStream_t st) {
  if (const moe_status_t s = moe_host::allow_smem<Kernel>(kNormRoom)) return s;
  return moe_host::launch(Kernel, dim3(grid), dim3(r.threads),
                          (size_t)weight_bytes + (size_t)r.stages * r.stage_bytes, st, p, r.stages,
                          r.stage_bytes, moe_host::device_error_word());
}

template <bool D_BF16, bool X_BF16>
moe_status_t norm_grad_ring(const NormGradParams& p, int& grid, cudaStream_t st) {
  const int weight = p.weight && p.H > kRingThreads * 8 ? p.H * 4 : 0;
  const RingPlan r =
      ring_plan(p.H, p.H * ((D_BF16 ? 2 : 4) + (X_BF16 ? 2 : 4) * (p.d_sum ? 2 : 1)), weight);
  const int most = moe_host::sm_count() * r.per_sm;
  if (grid > most) grid = most;
  return r.nv == 1
             ? launch_ring<layer_norm_backward_ring_kernel<D_BF16, X_BF16, 1>>(p, r, weight, grid, st)
             : launch_ring<layer_norm_backward_ring_kernel<D_BF16, X_BF16, 2>>(p, r, weight, grid, st);
}

// Threads for a row of the form for few rows, and the rows that it takes, at most.
int few_per(int H) { return (H / 8 + 31) / 32 * 32; }
int few_most(int H) { return kFewTurns * kFewCtas * (kFewThreads / few_per(H)); }

// Whether the device holds clusters of this size for the form for few rows.
template <auto Kernel>
bool few_fit() {
  static std::atomic<int> known[moe_host::kMaxCachedDevices] = {};  // 1 yes, -1 no
  std::atomic<int>& mine = known[moe_host::device_index()];
  int n = mine.load(std::memory_order_relaxed);
  if (n == 0) {
    n = -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kFewCtas);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kFewThreads * 8 * 8;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kFewCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, Kernel, &cfg) == cudaSuccess && clusters > 0)
      n = 1;
    cudaGetLastError();
    mine.store(n, std::memory_order_relaxed);
  }
  return n > 0;
}

template <bool D_BF16, bool X_BF16>
bool few_fit_as() {
  return few_fit<layer_norm_backward_few_kernel<D_BF16, X_BF16>>();
}

template <bool D_BF16, bool X_BF16>
moe_status_t norm_grad_few(const NormGradParams& p, float* d_weight, float* d_bias, cudaStream_t st) {
  const int per = few_per(p.H), groups = kFewThreads / per;
  return moe_host::launch_clusters(layer_norm_backward_few_kernel<D_BF16, X_BF16>, dim3(kFewCtas),
                                   groups * per, (size_t)groups * p.H * 8, dim3(kFewCtas, 1, 1), st, p, per,
                                   d_weight, d_bias);
}

template <bool X_BF16, bool OUT_BF16, int NV>
moe_status_t launch_norm_warps(const NormParams& p, cudaStream_t st) {
  constexpr auto kern = layer_norm_warp_kernel<X_BF16, OUT_BF16, NV>;
  const int row_bytes = p.H * (X_BF16 ? 2 : 4) * (p.residual ? 2 : 1);
  const int params = ((p.weight ? 1 : 0) + (p.bias ? 1 : 0)) * p.H * 4;
  const int room = ((int)kNormRoom - params) / row_bytes, most = warp_rows_most(X_BF16, NV);
  int warps = room < most ? room : most;
  // Warps that all have rows in the last turn too (us, as many as there is room for and
  // these: 4096 x 4096 fp32 31.7, 26.0; 3001 x 4096 bf16 14.1, 12.7; 8192 27.2, 26.6; 4096
  // 15.9, 16.4).  A single turn's spare warps help to load weight and bias.
  const int64_t sms = moe_host::sm_count(), turns = (p.T + sms * warps - 1) / (sms * warps);
  if (turns > 1) warps = (int)((p.T + sms * turns - 1) / (sms * turns));
  if (const moe_status_t s = moe_host::allow_smem<kern>(kNormRoom)) return s;
  return moe_host::launch(kern, dim3(moe_host::sm_count()), dim3(warps * 32),
                          (size_t)params + (size_t)warps * row_bytes, st, p, row_bytes, moe_host::device_error_word());
}

template <bool X_BF16, bool OUT_BF16>
moe_status_t norm_warps(const NormParams& p, cudaStream_t st) {
  if (p.H <= 1024) return launch_norm_warps<X_BF16, OUT_BF16, 4>(p, st);
  if (p.H <= 2048) return launch_norm_warps<X_BF16, OUT_BF16, 8>(p, st);
  if constexpr (X_BF16)
    if (p.H > 4096) return launch_norm_warps<X_BF16, OUT_BF16, 32>(p, st);
  return launch_norm_warps<X_BF16, OUT_BF16, 16>(p, st);
}

}  // namespace
}  // namespace moe

namespace moe_host {

moe_status_t column_sums(const float* part, int rows, int64_t ld, int cols, float* out, float* more,
                         cudaStream_t st) {
  if (cols == 0) return MOE_OK;
  return launch(moe::column_sums_kernel, dim3((cols + 31) / 32, more ? 2 : 1), dim3(moe::kColThreads), 0,
                st, part, rows, ld, cols, out, more);
}

}  // namespace moe_host

extern "C" moe_status_t moe_layer_norm(const void* x, int x_dtype, int64_t ld_x,
                                       const void* residual, int64_t ld_residual,
                                       const void* weight, const void* bias, int weight_dtype,
                                       int T, int H, int kind, float eps, int out_dtype, void* out,
                                       void* summed, float* mean, float* rstd,
                                       moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 1 || H > kNormMaxWidth) return MOE_ERR_INVALID_ARG;
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
  if (!type_ok(x_dtype) || !type_ok(out_dtype) || !type_ok(weight_dtype)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !out || ld_x < H || (residual && (!summed || ld_residual < H))) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(x, x_dtype) || !element_aligned(residual, x_dtype) ||
      !element_aligned(summed, x_dtype) || !element_aligned(weight, weight_dtype) ||
      !element_aligned(bias, weight_dtype) || !element_aligned(out, out_dtype) ||
      !moe_host::aligned4(mean) || !moe_host::aligned4(rstd))
    return MOE_ERR_INVALID_ARG;
  NormParams p{x,   ld_x, residual, ld_residual, weight, bias, weight_dtype == MOE_DTYPE_BF16,
               T,   H,    eps,      kind == MOE_NORM_RMS, out, summed, mean, rstd};
  const bool vec = H % 8 == 0 && vec_ok(x, x_dtype, ld_x) && vec_ok(residual, x_dtype, ld_residual) &&
                   vec_ok(residual ? summed : nullptr, x_dtype, H) && vec_ok(weight, weight_dtype, H) &&
                   vec_ok(bias, weight_dtype, H) && vec_ok(out, out_dtype, H);
  const Shape s = norm_shape(H, vec && T > moe_host::sm_count() ? 2 : 1);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool xb = x_dtype == MOE_DTYPE_BF16, ob = out_dtype == MOE_DTYPE_BF16;
  if (vec && H > kNormWarpWidth && (xb || H <= 4096) && T >= kNormWarpRows)
    return xb ? (ob ? norm_warps<true, true>(p, st) : norm_warps<true, false>(p, st))
              : (ob ? norm_warps<false, true>(p, st) : norm_warps<false, false>(p, st));
  if (vec)
    return xb ? (ob ? launch_norm<true, true, true>(p, s, st) : launch_norm<true, false, true>(p, s, st))
              : (ob ? launch_norm<false, true, true>(p, s, st) : launch_norm<false, false, true>(p, s, st));
  return xb ? (ob ? launch_norm<true, true, false>(p, s, st) : launch_norm<true, false, false>(p, s, st))
            : (ob ? launch_norm<false, true, false>(p, s, st) : launch_norm<false, false, false>(p, s, st));
}

extern "C" size_t moe_layer_norm_workspace_size(int T, int H) {
  using namespace moe;
  if (T < 1 || H < 1 || H > kNormMaxWidth) return 16;
  return (size_t)norm_grad_ctas(T, H) * 2 * H * sizeof(float);
}

extern "C" moe_status_t moe_layer_norm_backward(
    const void* d_out, int d_dtype, int64_t ld_d, const void* x, int x_dtype, int64_t ld_x,
    const float* mean, const float* rstd, const void* weight, int weight_dtype, const void* d_sum,
    int64_t ld_sum, int T, int H, void* d_x, float* d_weight, float* d_bias, void* workspace,
    size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 1 || H > kNormMaxWidth) return MOE_ERR_INVALID_ARG;
  if (!type_ok(x_dtype) || !type_ok(d_dtype) || !type_ok(weight_dtype)) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned4(d_weight) || !moe_host::aligned4(d_bias)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool sums = d_weight || d_bias;
  int grid = norm_grad_ctas(T, H);
  if (T > 0) {
    if (!d_out || !x || !rstd || !d_x || ld_d < H || ld_x < H || (d_sum && ld_sum < H))
      return MOE_ERR_INVALID_ARG;
    if (!element_aligned(d_out, d_dtype) || !element_aligned(x, x_dtype) ||
        !element_aligned(d_sum, x_dtype) || !element_aligned(d_x, x_dtype) ||
        !element_aligned(weight, weight_dtype) || !moe_host::aligned4(mean) ||
        !moe_host::aligned4(rstd))
      return MOE_ERR_INVALID_ARG;
    if (sums && (!workspace || !moe_host::aligned16(workspace) ||
                 workspace_bytes < moe_layer_norm_workspace_size(T, H)))
      return MOE_ERR_INVALID_ARG;
    NormGradParams p{d_out, ld_d, x, ld_x, d_sum, ld_sum, mean, rstd, weight,
                     weight_dtype == MOE_DTYPE_BF16, T, H, d_x,
                     sums ? static_cast<float*>(workspace) : nullptr};
    const bool vec = H % 8 == 0 && vec_ok(d_out, d_dtype, ld_d) && vec_ok(x, x_dtype, ld_x) &&
                     vec_ok(d_sum, x_dtype, ld_sum) && vec_ok(d_x, x_dtype, H) &&
                     vec_ok(weight, weight_dtype, H);
    const bool db = d_dtype == MOE_DTYPE_BF16, xb = x_dtype == MOE_DTYPE_BF16;
    if (sums && vec && H <= kFewThreads * 8 && T <= few_most(H)) {
      const bool fits = db ? (xb ? few_fit_as<true, true>() : few_fit_as<true, false>())
                           : (xb ? few_fit_as<false, true>() : few_fit_as<false, false>());
      if (fits)
        return db ? (xb ? norm_grad_few<true, true>(p, d_weight, d_bias, st)
                        : norm_grad_few<true, false>(p, d_weight, d_bias, st))
                  : (xb ? norm_grad_few<false, true>(p, d_weight, d_bias, st)
                        : norm_grad_few<false, false>(p, d_weight, d_bias, st));
    }
    const Shape run = norm_shape(H, vec ? 2 : 1);
    moe_status_t r;
    if (vec && run.rows == 1)
      r = db ? (xb ? norm_grad_ring<true, true>(p, grid, st) : norm_grad_ring<true, false>(p, grid, st))
             : (xb ? norm_grad_ring<false, true>(p, grid, st) : norm_grad_ring<false, false>(p, grid, st));
    else if (vec)
      r = db ? (xb ? launch_norm_grad<true, true, true>(p, run, grid, st)
                   : launch_norm_grad<true, false, true>(p, run, grid, st))
             : (xb ? launch_norm_grad<false, true, true>(p, run, grid, st)
                   : launch_norm_grad<false, false, true>(p, run, grid, st));
    else
      r = db ? (xb ? launch_norm_grad<true, true, false>(p, run, grid, st)
                   : launch_norm_grad<true, false, false>(p, run, grid, st))
             : (xb ? launch_norm_grad<false, true, false>(p, run, grid, st)
                   : launch_norm_grad<false, false, false>(p, run, grid, st));
    if (r) return r;
  }
  if (!sums) return MOE_OK;
  return moe_host::column_sums(static_cast<const float*>(workspace), T ? grid : 0, 2 * (int64_t)H, H,
                               d_weight, d_bias, st);
}
