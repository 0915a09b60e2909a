// Gradient of the dense product: the gradient of the pre-activations, its
// column sums, and the two products over it (linear.cu).
//
//   d_z[t, n] = d_out[t, n] act'(z[t, n]); SwiGLU: d_gate = d_out u silu'(g),
//               d_up = d_out silu(g)                     (held in bf16, as z is)
//   d_bias    = sum_t d_z (before that rounding),  d_x = d_z W,  d_w = d_z^T x
// One pass over d_out and z makes d_z and the partial column sums: a thread
// takes eight columns of every eighth row of its CTA's run of rows, the CTAs'
// sums are joined in their order.  Without an activation d_out is d_z.  That pass
// over 4096 rows with bias, us and share of the copy rate: SwiGLU of 11008 40, .83; SiLU
// 61, .65; GELU 66, .60 (bound by the issue of the functions; with two CTAs per SM, expf
// and erff 51, 86 and 134).
#include "linear.cuh"

namespace moe {
namespace {

constexpr int kDzRows = 8;  // rows a CTA takes at a time, one per warp
constexpr int kDzCols = 32 * 8;

struct DzParams {
  const void* d_out;
  int64_t ld_d;
  const uint16_t* z;  // [T, N], null without an activation
  uint16_t* d_z;      // [T, ld_z], or null: the sums alone
  int64_t ld_z;
  float* part;        // [runs][N], or null
  int T, N, cols, act;
  int run;            // rows of a CTA
  int vec;
};

// silu(z) and its derivative s (1 + z (1 - s)), s = 1 / (1 + e^-z).
__device__ __forceinline__ float silu_slope(float z, float& value) {
  const float s = __fdividef(1.0f, 1.0f + __expf(-z));
  value = z * s;
  return s * fmaf(z, 1.0f - s, 1.0f);
}
// Phi(z) + z phi(z) of two values.
__device__ __forceinline__ float2 gelu_slope2(float2 z) {
  float2 bell;
  const float2 q = normal_tail2(z, bell);
  return make_float2(fmaf(z.x * 0.39894228f, bell.x, z.x > 0.0f ? 1.0f - q.x : q.x),
                     fmaf(z.y * 0.39894228f, bell.y, z.y > 0.0f ? 1.0f - q.y : q.y));
}

// KIND: no activation, SiLU or GELU, SwiGLU.
enum { kDzNone, kDzOne, kDzGated };

template <bool D_BF16, int KIND>
__global__ void __launch_bounds__(256, 4) linear_dz_kernel(DzParams p) {
  constexpr bool SWIGLU = KIND == kDzGated;
  constexpr int kUnroll = KIND == kDzNone ? 4 : 1;  // rows of a thread at a time
  __shared__ float join[SWIGLU ? 2 : 1][kDzRows][kDzCols];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * kDzCols + threadIdx.x * 8;
  const int n = min(8, p.cols - c);
  const bool vec = p.vec != 0;
  float sum[SWIGLU ? 2 : 1][8] = {};
  const int64_t t1 = min((int64_t)(blockIdx.y + 1) * p.run, (int64_t)p.T);
  if (n > 0) {
#pragma unroll kUnroll
    for (int64_t t = (int64_t)blockIdx.y * p.run + threadIdx.y; t < t1; t += kDzRows) {
      Vec8<D_BF16> dv;
      if (vec) dv.load(p.d_out, t * p.ld_d + c);
      else dv.load_some(p.d_out, t * p.ld_d + c, n);
      float d[SWIGLU ? 2 : 1][8];
      dv.get(d[0]);
      if constexpr (KIND != kDzNone) {
        Vec8<true> zv;
        float z[8];
        const int64_t at = t * p.N + c;
        if (vec) zv.load(p.z, at);
        else zv.load_some(p.z, at, n);
        zv.get(z);
        if constexpr (SWIGLU) {
          float u[8];
          if (vec) zv.load(p.z, at + p.cols);
          else zv.load_some(p.z, at + p.cols, n);
          zv.get(u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v;
            const float s = silu_slope(z[i], v);
            d[1][i] = d[0][i] * v;
            d[0][i] = d[0][i] * u[i] * s;
          }
        } else if (p.act == MOE_ACT_GELU) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 s = gelu_slope2(make_float2(z[i], z[i + 1]));
            d[0][i] *= s.x;
            d[0][i + 1] *= s.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v;
            d[0][i] *= silu_slope(z[i], v);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[h][i] += d[h][i];
        if (p.d_z) {
          Vec8<true> o;
          o.set(d[h]);
          const int64_t at = t * p.ld_z + h * p.cols + c;
          if (vec) o.store(p.d_z, at);
          else o.store_some(p.d_z, at, n);
        }
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) join[h][threadIdx.y][threadIdx.x * 8 + i] = sum[h][i];
  __syncthreads();
  const int i = threadIdx.y * 32 + threadIdx.x, col = blockIdx.x * kDzCols + i;
  if (col >= p.cols) return;
#pragma unroll
  for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
    float s = join[h][0][i];
#pragma unroll
    for (int y = 1; y < kDzRows; ++y) s += join[h][y][i];
    p.part[(int64_t)blockIdx.y * p.N + h * p.cols + col] = s;
  }
}

// Rows of a CTA: enough runs for four CTAs per SM, eight rows each at least.
int dz_run(int64_t T, int64_t cols) {
  const int64_t blocks = (cols + kDzCols - 1) / kDzCols;
  int64_t runs = ((int64_t)moe_host::sm_count() * 4 + blocks - 1) / blocks;
  const int64_t most = (T + kDzRows - 1) / kDzRows;
  if (runs > most) runs = most;
  if (runs > 65535) runs = 65535;
  return (int)((((T + runs - 1) / runs) + kDzRows - 1) / kDzRows * kDzRows);
}
int64_t dz_runs(int64_t T, int run) { return (T + run - 1) / run; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_linear_backward_workspace_size(int T, int N, int activation) {
  using namespace moe;
  if (T < 1 || N < 1) return 16;
  const int cols = activation == MOE_ACT_SWIGLU ? N / 2 : N;
  if (cols < 1) return 16;
  return (size_t)dz_runs(T, dz_run(T, cols)) * N * sizeof(float);
}

extern "C" moe_status_t moe_linear_backward(const void* d_out, int d_dtype, int64_t ld_d,
                                            const uint16_t* x, int64_t ld_x, const uint16_t* w,
                                            const uint16_t* preact, int T, int K, int N,
                                            int activation, uint16_t* d_preact, int64_t ld_dp,
                                            uint16_t* d_x, void* d_w, int d_w_dtype, int accumulate,
                                            float* d_bias, void* workspace, size_t workspace_bytes,
                                            moe_stream_t stream) {
  using namespace moe;
  using moe_host::aligned16;
  using moe_host::aligned4;
  if (T < 0 || K < 8 || K % 8 != 0 || N < 1) return MOE_ERR_INVALID_ARG;
  if (T > kLinearMost || K > kLinearMost || N > kLinearMost) return MOE_ERR_INVALID_ARG;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool swiglu = activation == MOE_ACT_SWIGLU;
  if (swiglu && N % 2 != 0) return MOE_ERR_INVALID_ARG;
  if ((d_dtype != MOE_DTYPE_F32 && d_dtype != MOE_DTYPE_BF16) ||
      (d_w_dtype != MOE_DTYPE_F32 && d_w_dtype != MOE_DTYPE_BF16))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(d_x) || !aligned16(d_w) || !aligned4(d_bias))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over nothing
    if (d_w && !accumulate &&
        cudaMemsetAsync(d_w, 0, (size_t)N * K * (d_w_dtype == MOE_DTYPE_BF16 ? 2 : 4), st) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    return d_bias ? moe_host::column_sums(nullptr, 0, N, N, d_bias, nullptr, st) : MOE_OK;
  }
  const int cols = swiglu ? N / 2 : N;
  if (!d_out || ld_d < cols || (reinterpret_cast<uintptr_t>(d_out) & (d_dtype == MOE_DTYPE_BF16 ? 1u : 3u)))
    return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_NONE && (!preact || (reinterpret_cast<uintptr_t>(preact) & 1u)))
    return MOE_ERR_INVALID_ARG;
  if ((d_x && !w) || (d_w && (!x || ld_x < K || ld_x % 8 != 0))) return MOE_ERR_INVALID_ARG;
  // d_out itself serves where it is d_z and a tensor map can describe it
  const bool direct = activation == MOE_ACT_NONE && d_dtype == MOE_DTYPE_BF16 && aligned16(d_out) &&
                      ld_d % 8 == 0;
  if (!direct && (d_x || d_w) && !d_preact) return MOE_ERR_INVALID_ARG;
  if (!direct && d_preact && (!aligned16(d_preact) || ld_dp < N || ld_dp % 8 != 0))
    return MOE_ERR_INVALID_ARG;
  if (d_bias && (!workspace || !aligned16(workspace) ||
                 workspace_bytes < moe_linear_backward_workspace_size(T, N, activation)))
    return MOE_ERR_INVALID_ARG;
  uint16_t* made = direct ? nullptr : d_preact;
  if (made || d_bias) {
    const int run = dz_run(T, cols);
    // one run of rows: its sums are the bias's gradient
    const bool whole = dz_runs(T, run) == 1;
    DzParams p{d_out, ld_d, preact, made, ld_dp,
               d_bias ? (whole ? d_bias : static_cast<float*>(workspace)) : nullptr, T, N, cols,
               activation, run, 0};
    p.vec = cols % 8 == 0 && aligned16(d_out) && ld_d % 8 == 0 && aligned16(preact) && N % 8 == 0;
    const dim3 grid((cols + kDzCols - 1) / kDzCols, (unsigned)dz_runs(T, run)), block(32, kDzRows);
    using moe_host::launch;
    const bool db = d_dtype == MOE_DTYPE_BF16;
    auto go = [&](auto kern) { return launch(kern, grid, block, 0, st, p); };
    const moe_status_t r =
        swiglu ? (db ? go(linear_dz_kernel<true, kDzGated>) : go(linear_dz_kernel<false, kDzGated>))
        : activation != MOE_ACT_NONE
            ? (db ? go(linear_dz_kernel<true, kDzOne>) : go(linear_dz_kernel<false, kDzOne>))
            : (db ? go(linear_dz_kernel<true, kDzNone>) : go(linear_dz_kernel<false, kDzNone>));
    if (r) return r;
    if (d_bias && !whole)
      if (const moe_status_t s = moe_host::column_sums(p.part, (int)dz_runs(T, run), N, N, d_bias, nullptr, st))
        return s;
  }
  const uint16_t* dz = direct ? static_cast<const uint16_t*>(d_out) : d_preact;
  const int64_t ld = direct ? ld_d : ld_dp;
  if (d_w && linear_few_serves(T, N, K)) {
    if (const moe_status_t s = linear_few_dw(dz, ld, x, ld_x, T, N, K, accumulate != 0,
                                             d_w_dtype == MOE_DTYPE_BF16, d_w, st))
      return s;
    d_w = nullptr;
  }
  const LinearEpi ex{nullptr, nullptr, d_x, nullptr, T, K, K, MOE_ACT_NONE, 1, 0};
  const LinearEpi ew{nullptr, accumulate ? d_w : nullptr, d_w, nullptr, N, K, K, MOE_ACT_NONE,
                     d_w_dtype == MOE_DTYPE_BF16, 0};
  const LinearOp z_rows{dz, ld, true}, z_cols{dz, ld, false}, w_cols{w, K, false}, x_cols{x, ld_x, false};
  if (d_x && d_w) {
    const LinearOp a[2] = {z_rows, z_cols}, b[2] = {w_cols, x_cols};
    const int sums[2] = {N, T};
    LinearEpi e[2] = {ex, ew};
    return linear_products(a, b, sums, e, st);
  }
  if (d_x) return linear_product(z_rows, w_cols, N, ex, st);
  if (d_w) return linear_product(z_cols, x_cols, T, ew, st);
  return MOE_OK;
}
