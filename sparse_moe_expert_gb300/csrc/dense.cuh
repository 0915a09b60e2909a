// Shared by the norms and the dense product: rows of eight values, sums over
// a block, and column sums joined in a fixed order.
#pragma once

#include "common.cuh"

namespace moe {

// Eight consecutive values as loaded: 16 bytes of bf16, 32 of fp32.
template <bool BF16>
struct Vec8 {
  uint4 q[BF16 ? 1 : 2];

  __device__ __forceinline__ void load(const void* p, int64_t at) {
    if constexpr (BF16) {
      q[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      q[0] = s[0];
      q[1] = s[1];
    }
  }
  // The first n values at any alignment, zeros behind them.
  __device__ __forceinline__ void load_some(const void* p, int64_t at, int n) {
    if constexpr (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(p) + at;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < n ? s[2 * i] : 0u, hi = 2 * i + 1 < n ? s[2 * i + 1] : 0u;
        w[i] = lo | (hi << 16);
      }
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const uint32_t* s = static_cast<const uint32_t*>(p) + at;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < n ? s[i] : 0u;
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void zero() {
    q[0] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!BF16) q[1] = q[0];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (BF16) {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = bf16x2_to_f32x2(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    } else {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
  // The values rounded to the type (nearest even).
  __device__ __forceinline__ void set(const float (&f)[8]) {
    if constexpr (BF16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_to_bf16_rne(f[2 * i]) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1]) << 16);
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      q[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3]));
      q[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                        __float_as_uint(f[7]));
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at) const {
    if constexpr (BF16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = q[0];
    } else {
      uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(p) + at);
      d[0] = q[0];
      d[1] = q[1];
    }
  }
  __device__ __forceinline__ void store_some(void* p, int64_t at, int n) const {
    if constexpr (BF16) {
      uint16_t* d = static_cast<uint16_t*>(p) + at;
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) d[i] = (uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
    } else {
      uint32_t* d = static_cast<uint32_t*>(p) + at;
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) d[i] = w[i];
    }
  }
};

// The warp's sums of N values, in every lane.
template <int N>
__device__ __forceinline__ void warp_sum(float (&v)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

// The sums over the block of N values, in every thread, in a fixed order.
// `part` holds N * 32 floats that no thread may still read; a caller that sums
// again right away gives another part.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  warp_sum(v);
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? part[i * 32 + lane] : 0.0f;
  warp_sum(v);
}

}  // namespace moe

namespace moe_host {

// out[c] = sum over r of part[r, c] for c < cols, then more[c] = the same of the
// next cols columns (either may be null); part fp32 [rows, ld].  The rows are added
// in runs, the runs in order.
moe_status_t column_sums(const float* part, int rows, int64_t ld, int cols, float* out, float* more,
                         cudaStream_t st);

}  // namespace moe_host
