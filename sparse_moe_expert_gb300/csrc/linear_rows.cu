// The dense product for a few rows of x (a decode step): out = act(x W^T + bias)
// + residual, bound by reading W once.
//
// A CTA takes 16 rows of W at a time (SwiGLU: 8 of the gate, 8 of up) and its warps
// runs of four blocks of 32 k in turn.  A lane holds eight consecutive k of its row
// of W and of its token, which serve as two k-halves of mma.sync m16n8k16 in the same
// order on both sides; W goes from global memory straight into the operand, and
// x comes through L1, where the CTA's warps find it again.  The CTAs stay, two per
// SM, and ask for W one turn ahead, across the joint of a group of rows, whose
// sums meet in shared memory in warp order: nothing waits with no load on its way.
// Measured, one token, us and share of the copy rate: 4096 -> 22016 SwiGLU 29.1, .91;
// 11008 -> 4096 16.8, .79; 4096 -> 4096 7.8, .63 (with CTAs that end with their rows
// 32.4, 32.9, 12.9; those of 16 warps 54 at 4096 -> 22016).
#include "linear.cuh"

namespace moe {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;

__device__ __forceinline__ void rows_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: eights of tokens.
template <int NT, bool SWIGLU>
__global__ void __launch_bounds__(kRowsThreads, 2)
    linear_rows_kernel(const uint16_t* x, int64_t ldx, const uint16_t* w, int K, int units, LinearEpi e) {
  constexpr int kTokens = NT * 8;
  constexpr int kDeep = NT > 2 ? 2 : 4;  // blocks of 32 k in a turn
  constexpr int kSpan = SWIGLU ? 8 : 16;  // output columns of a unit
  __shared__ float sums[2][kRowsWarps][16][kTokens + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint16_t* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = x + (int64_t)min(i * 8 + g, e.M - 1) * ldx + 8 * t;
  const int turns = ((K + 31) / 32 + kRowsWarps * kDeep - 1) / (kRowsWarps * kDeep);
  auto first_k = [&](int turn) { return (turn * kRowsWarps + warp) * kDeep * 32 + 8 * t; };
  auto load = [&](uint4 (&a)[kDeep], uint4 (&b)[kDeep], int unit, int turn) {
    // this lane's two rows of W; a row past the end reads the last one and is not stored
    const int col = unit * kSpan;
    const int n0 = min(col + g, e.cols - 1);
    const int n1 = SWIGLU ? e.cols + n0 : min(col + 8 + g, e.cols - 1);
    const int k = first_k(turn);
    const uint16_t* w0 = w + (int64_t)n0 * K + k;
    const uint16_t* w1 = w + (int64_t)n1 * K + k;
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const bool on = unit < units && k + d * 32 < K;
      a[d] = on ? ldg_nc_v4(w0 + d * 32) : zero;
      b[d] = on ? ldg_nc_v4(w1 + d * 32) : zero;
    }
  };
  float acc[NT][4];
  uint4 a[kDeep], b[kDeep];
  int unit = blockIdx.x, turn = 0, buf = 0;
  load(a, b, unit, 0);
  while (unit < units) {
    if (turn == 0) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    }
    const bool last = turn + 1 == turns;
    uint4 na[kDeep], nb[kDeep];
    load(na, nb, last ? unit + gridDim.x : unit, last ? 0 : turn + 1);
    const int k = first_k(turn);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      uint4 q[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        q[i] = k + d * 32 < K ? __ldg(reinterpret_cast<const uint4*>(xr[i] + (k - 8 * t) + d * 32)) : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        rows_mma(acc[i], a[d].x, b[d].x, a[d].y, b[d].y, q[i].x, q[i].y);
        rows_mma(acc[i], a[d].z, b[d].z, a[d].w, b[d].w, q[i].z, q[i].w);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      a[d] = na[d];
      b[d] = nb[d];
    }
    if (!last) {
      ++turn;
      continue;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[buf][warp][g + (j >> 1) * 8][i * 8 + 2 * t + (j & 1)] = acc[i][j];
    __syncthreads();
    // a thread takes eight columns of a token; the other buffer serves the next unit meanwhile
    constexpr int kGroups = SWIGLU ? 1 : 2;
    for (int i = tid; i < e.M * kGroups; i += kRowsThreads) {
      const int r = i / kGroups, c = i % kGroups * 8;
      float z[2][8];
#pragma unroll
      for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          float s = 0.0f;
#pragma unroll
          for (int v = 0; v < kRowsWarps; ++v) s += sums[buf][v][h * 8 + c + y][r];
          z[h][y] = s;
        }
      finish8<SWIGLU>(e, r, unit * kSpan + c, z[0], z[1]);
    }
    buf ^= 1;
    turn = 0;
    unit += gridDim.x;
  }
}

template <bool SWIGLU>
moe_status_t launch_rows(const uint16_t* x, int64_t ldx, const uint16_t* w, int K, const LinearEpi& e,
                         cudaStream_t st) {
  const int span = SWIGLU ? 8 : 16, units = (e.cols + span - 1) / span;
  const int most = 2 * moe_host::sm_count();
  const dim3 grid(units < most ? units : most), block(kRowsThreads);
  using moe_host::launch;
  if (e.M <= 8) return launch(linear_rows_kernel<1, SWIGLU>, grid, block, 0, st, x, ldx, w, K, units, e);
  if (e.M <= 16) return launch(linear_rows_kernel<2, SWIGLU>, grid, block, 0, st, x, ldx, w, K, units, e);
  return launch(linear_rows_kernel<4, SWIGLU>, grid, block, 0, st, x, ldx, w, K, units, e);
}

}  // namespace

moe_status_t linear_rows(const uint16_t* x, int64_t ldx, const uint16_t* w, int K, const LinearEpi& e,
                         cudaStream_t st) {
  return e.act == MOE_ACT_SWIGLU ? launch_rows<true>(x, ldx, w, K, e, st)
                                 : launch_rows<false>(x, ldx, w, K, e, st);
}

}  // namespace moe
