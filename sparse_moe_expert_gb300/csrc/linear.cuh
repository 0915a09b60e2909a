// Shared by the kernels of the dense product: operands, the epilogue, and the
// tensor-core pieces that the small and the paired tiles have in common.
#pragma once

#include <cuda.h>

#include "async.cuh"
#include "dense.cuh"
#include "tc.cuh"

namespace moe {

// The largest T, K and N: sizes are rounded up to whole tiles and turns in 32 bits.
constexpr int kLinearMost = INT32_MAX - 4095;

// An operand of D[i, j] = sum_k A[i, k] B[j, k].  `rows` are i or j.
struct LinearOp {
  const uint16_t* p;
  int64_t ld;      // elements between rows, or between k where rows are contiguous
  bool row_major;  // false: element (row, k) at k * ld + row
};

// What happens to the sums.  Output column c of `cols`; SWIGLU has a second
// accumulator for it, of B's row cols + c.
struct LinearEpi {
  const float* bias;     // [N], or null
  const void* residual;  // [M, cols] of the output's type, or null
  void* out;             // [M, cols]
  uint16_t* preact;      // bf16 [M, N], or null
  int M, N, cols, act;
  int out_bf16;
  int vec;  // eight columns at a time are aligned everywhere
};

__device__ __forceinline__ float silu_f32(float z) {
  return __fdividef(z, __fadd_rn(1.0f, __expf(-z)));
}
// Phi(-|z|), the tail of the normal distribution, and `bell` = e^(-z^2 / 2), of two values.
// Phi(-z) e^(z^2 / 2) is t P(t) with t = 1 / (1 + 0.36 z), P of degree 6 fitted to 0 <= z <=
// 14 with the least largest relative error, 9e-7.  The tail is 2e-6 and its exponential's
// z^2 2^-24 off, relative, so that a product with it keeps its digits for negative z.  (erff and
// erfcf are more instructions: the gradient's pass over 4096 x 11008 GELU values 76 us, 66.)
__device__ __forceinline__ float2 normal_tail2(float2 z, float2& bell) {
  const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 d = ffma2(a, make_float2(0.36f, 0.36f), make_float2(1.0f, 1.0f));
  const float2 t = make_float2(__fdividef(1.0f, d.x), __fdividef(1.0f, d.y));
  bell = make_float2(__expf(-0.5f * z.x * z.x), __expf(-0.5f * z.y * z.y));
  auto step = [&](float2 h, float c) { return ffma2(h, t, make_float2(c, c)); };
  float2 h = make_float2(0.047057092f, 0.047057092f);
  h = step(h, -0.17976743f);
  h = step(h, 0.18095775f);
  h = step(h, 0.02654673f);
  h = step(h, 0.13972023f);
  h = step(h, 0.14177227f);
  h = step(h, 0.14371306f);
  return make_float2(h.x * t.x * bell.x, h.y * t.y * bell.y);
}
// z Phi(z).
__device__ __forceinline__ void gelu2(float& z0, float& z1) {
  float2 bell;
  const float2 q = normal_tail2(make_float2(z0, z1), bell);
  z0 *= z0 > 0.0f ? 1.0f - q.x : q.x;
  z1 *= z1 > 0.0f ? 1.0f - q.y : q.y;
}

__device__ __forceinline__ void load8_at(float (&f)[8], const float* p, int n, bool vec) {
  Vec8<false> v;
  if (vec) v.load(p, 0);
  else v.load_some(p, 0, n);
  v.get(f);
}

template <bool BF16>
__device__ __forceinline__ void finish8_as(const LinearEpi& e, int64_t row, int col, int n, bool vec,
                                           float (&y)[8]) {
  const int64_t at = row * e.cols + col;
  if (e.residual) {
    Vec8<BF16> v;
    float f[8];
    if (vec) v.load(e.residual, at);
    else v.load_some(e.residual, at, n);
    v.get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += f[i];
  }
  Vec8<BF16> o;
  o.set(y);
  if (vec) o.store(e.out, at);
  else o.store_some(e.out, at, n);
}

// Bias, pre-activation, activation, residual and the store of the sums z (and
// u, the second half of SWIGLU) of eight columns of a row < M.
template <bool SWIGLU>
__device__ __forceinline__ void finish8(const LinearEpi& e, int64_t row, int col, float (&z)[8],
                                        float (&u)[8]) {
  const int n = min(8, e.cols - col);
  if (n <= 0) return;
  const bool vec = e.vec != 0;  // whole groups of eight then
  if (e.bias) {
    float b[8];
    load8_at(b, e.bias + col, n, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
    if constexpr (SWIGLU) {
      load8_at(b, e.bias + e.cols + col, n, vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
  }
  if (e.preact) {
    Vec8<true> v;
    const int64_t at = row * e.N + col;
    v.set(z);
    if (vec) v.store(e.preact, at);
    else v.store_some(e.preact, at, n);
    if constexpr (SWIGLU) {
      v.set(u);
      if (vec) v.store(e.preact, at + e.cols);
      else v.store_some(e.preact, at + e.cols, n);
    }
  }
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (SWIGLU) y[i] = swiglu_f32(z[i], u[i]);
    else y[i] = z[i];
  }
  if constexpr (!SWIGLU) {
    if (e.act == MOE_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = silu_f32(z[i]);
    } else if (e.act == MOE_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) gelu2(y[i], y[i + 1]);
    }
  }
  if (e.out_bf16) finish8_as<true>(e, row, col, n, vec, y);
  else finish8_as<false>(e, row, col, n, vec, y);
}

// ---- tensor-core pieces --------------------------------------------------------

constexpr int kLinBK = 64;  // k per stage: 128 bytes of a row

// Descriptor of an operand tile in shared memory.  Rows contiguous in k: see
// smem_desc_sw128.  Else 64 rows x 64 k blocks of 8 KB, in which each k holds
// 128 bytes of rows: blocks 8192 bytes apart (leading offset), eights of k 1024
// bytes apart (stride offset).
template <bool ROW_MAJOR>
__device__ __forceinline__ uint64_t operand_desc(const void* p) {
  if constexpr (ROW_MAJOR) return smem_desc_sw128(p);
  uint64_t d = (smem_u32(p) >> 4) & 0x3FFFull;
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= 1ull << 46;
  d |= 2ull << 61;
  return d;
}
// 16 k further on, in units of 16 bytes.
template <bool ROW_MAJOR>
__device__ __forceinline__ constexpr uint64_t operand_step() {
  return ROW_MAJOR ? 2 : 128;
}
// Instruction descriptor with the operands' orders.
template <bool A_ROW, bool B_ROW>
__host__ __device__ constexpr uint32_t idesc_linear(int M, int N) {
  return idesc_bf16(M, N) | (A_ROW ? 0u : 1u << 15) | (B_ROW ? 0u : 1u << 16);
}

// True in the one lane that issues for its warp, the same one every time.
__device__ __forceinline__ bool elected() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(on));
  return on != 0;
}

__device__ __forceinline__ void linear_tma_2d(void* dst, const CUtensorMap* tm, int c0, int c1,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Map of an operand: boxes of 64 k x `box_rows` rows, or of 64 rows x 64 k.
bool linear_map(CUtensorMap* m, const LinearOp& op, int rows, int K, int box_rows);

// D = A B^T for M rows of A and e.N rows of B, by pairs of CTAs, and the time this
// takes, estimated in us.
moe_status_t linear_pairs(const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e,
                          cudaStream_t st);
float linear_pairs_us(const LinearEpi& e, int K, bool b_rows);
// Two products, B by columns, in one launch; the first one's tiles come first.
moe_status_t linear_pairs_both(const LinearOp (&a)[2], const LinearOp (&b)[2], const int (&K)[2],
                               const LinearEpi (&e)[2], cudaStream_t st);
float linear_pairs_both_us(const LinearEpi (&e)[2], const int (&K)[2]);
// The same for up to kLinearRowsMost rows of A, both operands in rows.
constexpr int kLinearRowsMost = 32;
moe_status_t linear_rows(const uint16_t* x, int64_t ldx, const uint16_t* w, int K,
                         const LinearEpi& e, cudaStream_t st);
// d_w = d_z^T x (+ d_w) of a few rows, where this serves the sizes.
bool linear_few_serves(int tokens, int N, int K);
moe_status_t linear_few_dw(const uint16_t* dz, int64_t ld, const uint16_t* x, int64_t ldx, int tokens, int N,
                           int K, bool add, bool bf16, void* d_w, cudaStream_t st);
// Which of the forms serves the call.
moe_status_t linear_product(const LinearOp& a, const LinearOp& b, int K, LinearEpi e, cudaStream_t st);
// The same for two products with B by columns.
moe_status_t linear_products(const LinearOp (&a)[2], const LinearOp (&b)[2], const int (&K)[2],
                             LinearEpi (&e)[2], cudaStream_t st);

}  // namespace moe
