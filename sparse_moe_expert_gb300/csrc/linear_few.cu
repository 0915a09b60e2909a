// d_w of a product of up to 8 rows of x, bound by writing it:
//   d_w[n, k] = sum_t d_z[t, n] x[t, k] (+ d_w)
// A thread keeps x of its eight columns in fp32 and writes row after row; a warp's rows are
// 512 bytes of bf16 or 1 KB of fp32.  The tensor cores' tiles hold 128 rows for the same
// bytes and are late with them.  Measured, us, tiles and this, one row of x: 4096 -> 22016
// bf16 78, 28; fp32 92, 95; 4096 -> 4096 bf16 17, 6.7; fp32 22, 18; 2048 -> 1536 bf16 6.9, 3.7;
// eight rows: 4096 -> 22016 78, 41; 4096 -> 4096 17, 14.5; 2048 -> 1536 6.5, 8.2.
#include "linear.cuh"

namespace moe {
namespace {

constexpr int kFewLinThreads = 256;
constexpr int kFewRows = 256;    // rows of d_z held at a time

// Rows n0 .. n0 + count of d_z^T as fp32, [row][T], zeros for tokens past the last.
template <int T>
__device__ __forceinline__ void hold_dz(float* s, const uint16_t* dz, int64_t ld, int tokens, int n0,
                                        int count) {
  for (int i = threadIdx.x; i < count * T; i += kFewLinThreads) {
    const int t = i / count, r = i - t * count;  // neighbours read neighbouring n
    s[r * T + t] = t < tokens ? bf16_bits_to_f32(dz[t * ld + n0 + r]) : 0.0f;
  }
}

template <int T, bool OUT_BF16>
__global__ void __launch_bounds__(kFewLinThreads)
    linear_few_dw_kernel(const uint16_t* dz, int64_t ld, const uint16_t* x, int64_t ldx, int tokens, int N,
                         int K, int run, int add, void* d_w) {
  __shared__ __align__(16) float few[kFewRows * T];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.y * 256 + lane * 8;
  const int n0 = blockIdx.x * run, count = min(run, N - n0);
  hold_dz<T>(few, dz, ld, tokens, n0, count);
  __syncthreads();
  if (col >= K) return;
  float2 f[T][4];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (t < tokens) q = *reinterpret_cast<const uint4*>(x + t * ldx + col);
    f[t][0] = bf16x2_to_f32x2(q.x);
    f[t][1] = bf16x2_to_f32x2(q.y);
    f[t][2] = bf16x2_to_f32x2(q.z);
    f[t][3] = bf16x2_to_f32x2(q.w);
  }
  for (int r = warp; r < count; r += kFewLinThreads / 32) {
    const int64_t at = (int64_t)(n0 + r) * K + col;
    Vec8<OUT_BF16> old;
    if (add) old.load(d_w, at);
    float2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float z = few[r * T + t];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = ffma2(make_float2(z, z), f[t][i], acc[i]);
    }
    float y[8] = {acc[0].x, acc[0].y, acc[1].x, acc[1].y, acc[2].x, acc[2].y, acc[3].x, acc[3].y};
    if (add) {
      float g[8];
      old.get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += g[i];
    }
    Vec8<OUT_BF16> o;
    o.set(y);
    o.store(d_w, at);
  }
}

template <int T>
moe_status_t few_dw(const uint16_t* dz, int64_t ld, const uint16_t* x, int64_t ldx, int tokens, int N, int K,
                    bool add, bool bf16, void* d_w, cudaStream_t st) {
  // runs of rows: eight CTAs per SM or more, a row per warp at least
  const int64_t across = ((int64_t)K + 255) / 256;
  int run = kFewRows;
  while (run > 8 && ((int64_t)N + run - 1) / run * across < 8 * (int64_t)moe_host::sm_count()) run /= 2;
  const dim3 grid((unsigned)(((int64_t)N + run - 1) / run), (unsigned)across);
  using moe_host::launch;
  return bf16 ? launch(linear_few_dw_kernel<T, true>, grid, dim3(kFewLinThreads), 0, st, dz, ld, x, ldx, tokens,
                       N, K, run, add ? 1 : 0, d_w)
              : launch(linear_few_dw_kernel<T, false>, grid, dim3(kFewLinThreads), 0, st, dz, ld, x, ldx, tokens,
                       N, K, run, add ? 1 : 0, d_w);
}

}  // namespace

// Up to four rows always, eight where there is much to write (both sides above).
bool linear_few_serves(int tokens, int N, int K) {
  return K <= 65535 * 256 &&  // the grid's height
         (tokens <= 4 || (tokens <= 8 && (int64_t)N * K >= (int64_t)1 << 23));
}

moe_status_t linear_few_dw(const uint16_t* dz, int64_t ld, const uint16_t* x, int64_t ldx, int tokens, int N,
                           int K, bool add, bool bf16, void* d_w, cudaStream_t st) {
  if (tokens <= 2) return few_dw<2>(dz, ld, x, ldx, tokens, N, K, add, bf16, d_w, st);
  if (tokens <= 4) return few_dw<4>(dz, ld, x, ldx, tokens, N, K, add, bf16, d_w, st);
  return few_dw<8>(dz, ld, x, ldx, tokens, N, K, add, bf16, d_w, st);
}

}  // namespace moe
