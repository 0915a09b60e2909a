// Gradient of the weighted combine: page "Qwen3.5 Block在llama.cpp中的映射与
// 优化原理", section 4.2, out[t] = sum_j w[t, j] y[row(t, j)], so
//   d_w[t, j]     = sum_m d_out[t, m] y[row, m]   (fp32 sums)
//   d_y[row, m]   = w[t, j] d_out[t, m]           (rounded to y's type once)
//
// CTAs walk over tokens.  A thread takes 16 bytes of each chosen row and the
// same columns of d_out, which it reads once for all k slots; all k row loads
// are in flight together, and the next token's row numbers and weights are
// fetched meanwhile, so that no load waits for another.  The k partial dot
// products are joined by a reduce-scatter over the warp and then over the
// warps in order.  Bound by HBM.  Measured, 4096 tokens x 8 bf16 rows of 2048
// (272 MB): 45.6 us, 6.0 TB/s, 0.88 of the copy rate; before the rows were
// fetched ahead and together, 95 us; with four CTAs per SM instead of three
// (64 registers, spills) 47 us.  The weights' gradient alone (144 MB): 25.5 us.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kCgThreads = 256;
constexpr int kCgWarps = kCgThreads / 32;
constexpr int kCgSlots = 8;  // slots in flight; kmax > 8 takes two passes over d_out
constexpr int kCgMaxSlots = 16;
constexpr int kCgCtas = 3;  // resident per SM

struct CombineGradParams {
  const uint16_t* d_out;
  const void* y;
  const int32_t* inv_pos;
  const float* w;
  const int32_t* k_dev;
  int T, kmax, H;
  float* d_w;
  void* d_y;  // or null
  unsigned int* err;
};

// Eight values per lane -> lane 4 i holds the warp's sum of value i (lanes
// 4 i .. 4 i + 3 alike).
__device__ __forceinline__ float reduce8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16, c = 8; c > 1; off >>= 1, c >>= 1) {
    const bool hi = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < c / 2; ++j) {
      const float keep = hi ? v[j + c / 2] : v[j];
      const float send = hi ? v[j] : v[j + c / 2];
      v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, off);
    }
  }
  v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 2);
  v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 1);
  return v[0];
}

template <bool BF16_Y>
__global__ void __launch_bounds__(kCgThreads, kCgCtas) combine_backward_kernel(CombineGradParams p) {
  constexpr int V = BF16_Y ? 8 : 4;
  __shared__ float part[2][kCgMaxSlots][kCgWarps];
  __shared__ int row_s[2][kCgMaxSlots];
  __shared__ float w_s[2][kCgMaxSlots];
  pdl_wait();
  pdl_trigger();
  const int k = min(max(*p.k_dev, 0), p.kmax);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = p.H / V;
  const int rows = p.T * p.kmax;
  // slot j of token t: its row (MOE_DROPPED: none) and weight, by thread j
  auto fetch = [&](int64_t t, int& r, float& w) {
    r = MOE_DROPPED;
    w = 0.0f;
    if (threadIdx.x < k && t < p.T) {
      r = __ldg(p.inv_pos + t * p.kmax + threadIdx.x);
      w = __ldg(p.w + t * p.kmax + threadIdx.x);
      if (r >= rows || (r < 0 && r != MOE_DROPPED)) {
        raise_device_error(p.err, MOE_DEVERR_BAD_INDEX);
        r = MOE_DROPPED;
      }
    }
  };
  int nr;
  float nw;
  fetch(blockIdx.x, nr, nw);
  int buf = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
    if (threadIdx.x < kCgMaxSlots) {
      row_s[buf][threadIdx.x] = nr;
      w_s[buf][threadIdx.x] = nw;
    }
    __syncthreads();
    fetch(t + gridDim.x, nr, nw);
    for (int j0 = 0; j0 < p.kmax; j0 += kCgSlots) {
      float acc[kCgSlots];
#pragma unroll
      for (int j = 0; j < kCgSlots; ++j) acc[j] = 0.0f;
      for (int c = threadIdx.x; c < nvec; c += kCgThreads) {
        uint4 q[kCgSlots];
#pragma unroll
        for (int j = 0; j < kCgSlots; ++j) {
          const int r = row_s[buf][j0 + j];
          if (r >= 0) q[j] = ldg_nc_v4(static_cast<const uint4*>(p.y) + (int64_t)r * nvec + c);
        }
        float d[V];
        if constexpr (BF16_Y) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.d_out + t * p.H) + c);
          const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = bf16x2_to_f32x2(w4[e]);
            d[2 * e] = f.x;
            d[2 * e + 1] = f.y;
          }
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p.d_out + t * p.H) + c);
          const float2 a = bf16x2_to_f32x2(x.x), b = bf16x2_to_f32x2(x.y);
          d[0] = a.x;
          d[1] = a.y;
          d[2] = b.x;
          d[3] = b.y;
        }
        if (p.d_y) {  // the rows' gradient does not wait for y
#pragma unroll
          for (int j = 0; j < kCgSlots; ++j) {
            const int r = row_s[buf][j0 + j];
            if (r < 0) continue;
            const float w = w_s[buf][j0 + j];
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (BF16_Y)
                o[e] = (uint32_t)f32_to_bf16_rne(w * d[2 * e]) |
                       ((uint32_t)f32_to_bf16_rne(w * d[2 * e + 1]) << 16);
              else
                o[e] = __float_as_uint(w * d[e]);
            }
            static_cast<uint4*>(p.d_y)[(int64_t)r * nvec + c] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < kCgSlots; ++j) {
          if (row_s[buf][j0 + j] < 0) continue;
          const uint32_t w4[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BF16_Y) {
              const float2 f = bf16x2_to_f32x2(w4[e]);
              acc[j] = fmaf(d[2 * e], f.x, acc[j]);
              acc[j] = fmaf(d[2 * e + 1], f.y, acc[j]);
            } else {
              acc[j] = fmaf(d[e], __uint_as_float(w4[e]), acc[j]);
            }
          }
        }
      }
      const float s = reduce8(acc);
      if ((lane & 3) == 0) part[buf][j0 + (lane >> 2)][warp] = s;
    }
    __syncthreads();
    // the other buffers serve the next token meanwhile
    if (threadIdx.x < p.kmax) {
      float s = 0.0f;
#pragma unroll
      for (int x = 0; x < kCgWarps; ++x) s += part[buf][threadIdx.x][x];
      p.d_w[t * p.kmax + threadIdx.x] = s;
    }
  }
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_combine_backward(const uint16_t* d_out, const void* y, int y_dtype,
                                             const int32_t* inv_pos, const float* topk_w,
                                             const int32_t* k_dev, int T, int kmax, int H,
                                             float* d_topk_w, void* d_y, moe_stream_t stream) {
  using namespace moe_host;
  if (T < 0 || H <= 0 || H % 64 != 0 || kmax < 1 || kmax > 16) return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * kmax > (1 << 24)) return MOE_ERR_INVALID_ARG;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!k_dev || !aligned4(k_dev)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {d_out, y, inv_pos, topk_w, d_topk_w};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (d_y && (!aligned16(d_y) || d_y == y)) return MOE_ERR_INVALID_ARG;
  moe::CombineGradParams p{d_out, y,        inv_pos, topk_w, k_dev, T,
                           kmax,  H,        d_topk_w, d_y,   device_error_word()};
  const int64_t cap = (int64_t)sm_count() * moe::kCgCtas;
  const int grid = (int)(T < cap ? T : cap);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (y_dtype == MOE_DTYPE_BF16)
    return launch(moe::combine_backward_kernel<true>, grid, moe::kCgThreads, 0, st, p);
  return launch(moe::combine_backward_kernel<false>, grid, moe::kCgThreads, 0, st, p);
}
