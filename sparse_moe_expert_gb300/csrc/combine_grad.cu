// Gradient of the weighted combine: page "Qwen3.5 Block在llama.cpp中的映射与
// 优化原理", section 4.2, out[t] = sum_j w[t, j] y[row(t, j)], so
//   d_w[t, j]     = sum_m d_out[t, m] y[row, m]   (fp32 sums)
//   d_y[row, m]   = w[t, j] d_out[t, m]           (rounded to y's type once)
//
// One CTA per token: a thread takes 16 bytes of each chosen row and the same
// columns of d_out, which it reads once for all k slots; the k partial dot
// products are joined by xor shuffles and then over the warps in order.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kCgThreads = 256;
constexpr int kCgWarps = kCgThreads / 32;
constexpr int kCgSlots = 8;  // slots in flight; k > 8 takes two passes over d_out

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

template <bool BF16_Y>
__global__ void __launch_bounds__(kCgThreads) combine_backward_kernel(CombineGradParams p) {
  constexpr int V = BF16_Y ? 8 : 4;
  __shared__ float part[kCgWarps][kCgSlots];
  pdl_wait();
  pdl_trigger();
  const int k = min(max(*p.k_dev, 0), p.kmax);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = p.H / V;
  const int64_t rows = (int64_t)p.T * p.kmax;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    for (int j0 = 0; j0 < p.kmax; j0 += kCgSlots) {
      int64_t r[kCgSlots];
      float w[kCgSlots], acc[kCgSlots];
#pragma unroll
      for (int j = 0; j < kCgSlots; ++j) {
        r[j] = j0 + j < k ? __ldg(p.inv_pos + t * p.kmax + j0 + j) : MOE_DROPPED;
        w[j] = j0 + j < k ? __ldg(p.w + t * p.kmax + j0 + j) : 0.0f;
        if (r[j] >= rows || (r[j] < 0 && r[j] != MOE_DROPPED)) {
          if (threadIdx.x == 0) raise_device_error(p.err, MOE_DEVERR_BAD_INDEX);
          r[j] = MOE_DROPPED;
        }
        acc[j] = 0.0f;
      }
      for (int c = threadIdx.x; c < nvec; c += kCgThreads) {
        float d[V];
        if constexpr (BF16_Y) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(p.d_out + t * p.H) + c);
          const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = bf16x2_to_f32x2(w4[e]);
            d[2 * e] = f.x;
            d[2 * e + 1] = f.y;
          }
        } else {
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(p.d_out + t * p.H) + c);
          const float2 a = bf16x2_to_f32x2(q.x), b = bf16x2_to_f32x2(q.y);
          d[0] = a.x;
          d[1] = a.y;
          d[2] = b.x;
          d[3] = b.y;
        }
        uint4 q[kCgSlots];
#pragma unroll
        for (int j = 0; j < kCgSlots; ++j)
          if (r[j] >= 0)
            q[j] = ldg_nc_v4(static_cast<const char*>(p.y) + ((r[j] * nvec + c) << 4));
#pragma unroll
        for (int j = 0; j < kCgSlots; ++j) {
          if (r[j] < 0) continue;
          const uint32_t w4[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BF16_Y) {
              const float2 f = bf16x2_to_f32x2(w4[e]);
              acc[j] = fmaf(d[2 * e], f.x, acc[j]);
              acc[j] = fmaf(d[2 * e + 1], f.y, acc[j]);
              o[e] = (uint32_t)f32_to_bf16_rne(w[j] * d[2 * e]) |
                     ((uint32_t)f32_to_bf16_rne(w[j] * d[2 * e + 1]) << 16);
            } else {
              acc[j] = fmaf(d[e], __uint_as_float(w4[e]), acc[j]);
              o[e] = __float_as_uint(w[j] * d[e]);
            }
          }
          if (p.d_y)
            *reinterpret_cast<uint4*>(static_cast<char*>(p.d_y) + ((r[j] * nvec + c) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < kCgSlots; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        if (lane == 0) part[warp][j] = acc[j];
      }
      __syncthreads();
      if (threadIdx.x < kCgSlots && j0 + threadIdx.x < p.kmax) {
        float s = 0.0f;
#pragma unroll
        for (int x = 0; x < kCgWarps; ++x) s += part[x][threadIdx.x];
        p.d_w[t * p.kmax + j0 + threadIdx.x] = s;
      }
      __syncthreads();
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
  if (!k_dev) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {d_out, y, inv_pos, topk_w, d_topk_w};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (d_y && (!aligned16(d_y) || d_y == y)) return MOE_ERR_INVALID_ARG;
  moe::CombineGradParams p{d_out, y,        inv_pos, topk_w, k_dev, T,
                           kmax,  H,        d_topk_w, d_y,   device_error_word()};
  const int64_t cap = (int64_t)sm_count() * 64;
  const int grid = (int)(T < cap ? T : cap);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (y_dtype == MOE_DTYPE_BF16)
    return launch(moe::combine_backward_kernel<true>, grid, moe::kCgThreads, 0, st, p);
  return launch(moe::combine_backward_kernel<false>, grid, moe::kCgThreads, 0, st, p);
}
