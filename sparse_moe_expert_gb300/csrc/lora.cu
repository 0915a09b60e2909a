// Low-rank adapters of many requests beside a shared (or per-expert) product:
//   out[r] = base[r] + scale_a (x[r] A_a,e^T) B_a,e^T
// where row r belongs to a token whose request uses adapter a (or none) and,
// in an expert layer, to expert e.  Page "Qwen3.5-MoE与Qwen3-MoE架构差异深度
// 解析", section 4.4 (expert-level LoRA).
//
// Two kernels: the shrink v[r] = scale x[r] A^T (contraction over K, rank R
// wide) and the expand out[r] = base[r] + v[r] B^T (contraction over R).
// Both are bound by memory: a matrix of one adapter is read for a handful of
// rows, or x, base and out are streamed past a small matrix.  Operands go
// from global memory straight into mma.sync fragments: the order of the
// contraction index is free, so lane t of a quad takes contiguous elements
// of its row (16 bytes of x and A, 8 bytes of B) and no shared-memory
// staging is needed.
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// v[r, j] = scale * sum_k x[r, k] A[j, k].  One CTA per row; the warps take
// blocks of 32 k in turn and their sums are added in warp order.  NT: eights
// of the rank (rounded up).
template <int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(LoraParams p) {
  __shared__ float red[kLoraWarps][NT * 8];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if (r >= lora_rows(p)) return;
  const LoraRow row = lora_row(p, r);
  if (row.slot < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int nt = p.R >> 3;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + row.x_row * p.K) + t;
  const uint4* ar = reinterpret_cast<const uint4*>(p.a + ((int64_t)row.slot * p.R + g) * p.K) + t;
  const int64_t astep = (int64_t)p.K;  // 8 rows of A in uint4
  float acc[NT][4];
#pragma unroll
  for (int q = 0; q < NT; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
  const int blocks = p.K >> 5;
#pragma unroll 2
  for (int kb = warp; kb < blocks; kb += kLoraWarps) {
    uint4 xv = make_uint4(0u, 0u, 0u, 0u);
    if (g == 0) xv = __ldg(xr + kb * 4);
    uint4 av[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q)
      if (q < nt) av[q] = ldg_nc_v4(ar + q * astep + kb * 4);
    const uint32_t f0[4] = {xv.x, 0u, xv.y, 0u}, f1[4] = {xv.z, 0u, xv.w, 0u};
#pragma unroll
    for (int q = 0; q < NT; ++q)
      if (q < nt) {
        mma_bf16(acc[q], f0, av[q].x, av[q].y);
        mma_bf16(acc[q], f1, av[q].z, av[q].w);
      }
  }
  if (g == 0) {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      red[warp][q * 8 + 2 * t] = acc[q][0];
      red[warp][q * 8 + 2 * t + 1] = acc[q][1];
    }
  }
  __syncthreads();
  if (threadIdx.x < p.R) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) s += red[w][threadIdx.x];
    const float sc = p.scales ? __ldg(p.scales + row.slot / p.E) : 1.0f;
    p.v[(int64_t)r * p.R + threadIdx.x] = s * sc;
  }
}

// Eight consecutive values of a row of base (fp32 or bf16).
template <bool BF16>
__device__ __forceinline__ void load8(float (&f)[8], const void* base, int64_t at) {
  if constexpr (BF16) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf16x2_to_f32x2(w4[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* out, int64_t at, const float (&f)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)f32_to_bf16_rne(f[2 * i]) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// Three bf16 terms whose sum is the fp32 value to 2^-26 of it (two values packed per word).
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t ah = f32_to_bf16_rne(a), bh = f32_to_bf16_rne(b);
  const float ar = a - bf16_bits_to_f32(ah), br = b - bf16_bits_to_f32(bh);
  const uint32_t am = f32_to_bf16_rne(ar), bm = f32_to_bf16_rne(br);
  const uint32_t al = f32_to_bf16_rne(ar - bf16_bits_to_f32(am));
  const uint32_t bl = f32_to_bf16_rne(br - bf16_bits_to_f32(bm));
  hi = ah | (bh << 16);
  mid = am | (bm << 16);
  lo = al | (bl << 16);
}

// acc[q] += v (one row, lanes with g = 0) B^T for the lane's 32-column block at
// `col`: column 2t + i of eight q is column 8t + 2q + i of the block, so a
// lane ends with eight consecutive columns.
__device__ __forceinline__ void expand_block(float (&acc)[4][4], const LoraParams& p, int64_t slot,
                                             const float* v, bool live, int col) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint16_t* b0 = p.b + (slot * p.N + col + 8 * (g >> 1) + (g & 1)) * p.R + 4 * t;
  for (int s = 0; s < p.R; s += 16) {
    const bool in = s + 4 * t < p.R;
    uint2 bq[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      bq[q] = in ? __ldg(reinterpret_cast<const uint2*>(b0 + (int64_t)(2 * q) * p.R + s))
                 : make_uint2(0u, 0u);
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (in && live) f = *reinterpret_cast<const float4*>(v + s + 4 * t);
    uint32_t h0, m0, l0, h1, m1, l1;
    split3(f.x, f.y, h0, m0, l0);
    split3(f.z, f.w, h1, m1, l1);
    const uint32_t fh[4] = {h0, 0u, h1, 0u}, fm[4] = {m0, 0u, m1, 0u}, fl[4] = {l0, 0u, l1, 0u};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      mma_bf16(acc[q], fl, bq[q].x, bq[q].y);
      mma_bf16(acc[q], fm, bq[q].x, bq[q].y);
      mma_bf16(acc[q], fh, bq[q].x, bq[q].y);
    }
  }
}

// out[r, n] = base[r, n] + sum_j v[r, j] B[n, j], or SiLU(gate) * up of it.
template <bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(LoraParams p) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if (r >= lora_rows(p)) return;
  const LoraRow row = lora_row(p, r);
  if (row.slot < 0 && !SWIGLU && p.base == p.out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int cols = SWIGLU ? p.N / 2 : p.N;
  for (int col = (blockIdx.y * kLoraWarps + warp) * 32; col < cols;
       col += gridDim.y * kLoraWarps * 32) {
    float f[SWIGLU ? 2 : 1][8];
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
      float acc[4][4];
      float b8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b8[i] = 0.0f;
      if (g == 0 && p.base) load8<BASE_BF16>(b8, p.base, (int64_t)r * p.N + h * cols + col + 8 * t);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[q][0] = b8[2 * q];
        acc[q][1] = b8[2 * q + 1];
        acc[q][2] = acc[q][3] = 0.0f;
      }
      if (row.slot >= 0)
        expand_block(acc, p, row.slot, p.v + (int64_t)r * p.R, g == 0, h * cols + col);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[h][2 * q] = acc[q][0];
        f[h][2 * q + 1] = acc[q][1];
      }
    }
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[0][i] = swiglu_f32(f[0][i], f[1][i]);
    }
    if (g == 0) store8<OUT_BF16>(p.out, (int64_t)r * cols + col + 8 * t, f[0]);
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace {

// From this many rows on they are grouped by adapter, if each adapter (and
// expert) may expect two or more.
constexpr int kLoraGroupRows = 192;

bool lora_groups(int64_t rows, int E, int n_adapters) {
  return rows >= kLoraGroupRows && rows >= 2 * (int64_t)n_adapters * E &&
         n_adapters <= kLoraPlanAdapters;
}

// CTAs per tile in the grouped shrink: enough for two per SM when the tiles
// alone are too few, with at least four k-blocks of 64 each.
int lora_splits(int64_t rows, int K) {
  const int64_t tiles = (rows + kLoraTileRows - 1) / kLoraTileRows;
  int s = 1;
  while (s < kLoraMaxSplit && 2 * s * tiles <= 2 * moe_host::sm_count() && 2 * s * 256 <= K) s *= 2;
  return s;
}

struct LoraSpace {
  size_t rows, tiles, total;  // v comes first
};

LoraSpace lora_space(int64_t rows, int E, int n_adapters, int R) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  LoraSpace s{};
  const size_t one = (size_t)(rows ? rows : 1) * R * sizeof(float);
  if (!lora_groups(rows, E, n_adapters)) {
    s.total = one;
    return s;
  }
  s.rows = up((size_t)rows * kLoraMaxTerms * rank_pad(R) * sizeof(uint16_t));
  s.tiles = s.rows + up((size_t)rows * sizeof(int2));
  s.total = s.tiles + (size_t)(1 + lora_tile_capacity(rows, E, n_adapters)) * sizeof(int4);
  return s;
}

}  // namespace

extern "C" size_t moe_lora_workspace_size(int T, int kmax, int E, int n_adapters, int R) {
  if (T < 0 || kmax < 1 || kmax > 16 || E < 1 || n_adapters < 1 || R < 1 || R > kMaxRank) return 0;
  return lora_space((int64_t)T * kmax, E, n_adapters, R).total;
}

extern "C" moe_status_t moe_lora_apply(const uint16_t* x, int x_by_token,
                                       const int32_t* adapter_ids, const int32_t* topk_ids,
                                       const int32_t* sorted_assign,
                                       const int32_t* expert_offsets, int T, int kmax, int E,
                                       int n_adapters, int K, int N, int R,
                                       const uint16_t* lora_a, const uint16_t* lora_b,
                                       const float* scales, const void* base, int base_dtype,
                                       int epilogue, int out_dtype, void* out, void* workspace,
                                       size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe_host;
  if (T < 0 || kmax < 1 || kmax > 16 || E < 1 || E > 1024 || (int64_t)T * kmax > (1 << 24))
    return MOE_ERR_INVALID_ARG;
  if (n_adapters < 1 || (int64_t)n_adapters * E > (1 << 20)) return MOE_ERR_INVALID_ARG;
  if (K <= 0 || K % 64 || N <= 0 || N % 64 || R <= 0 || R % 8 || R > kMaxRank)
    return MOE_ERR_INVALID_ARG;
  if (epilogue != MOE_EPILOGUE_RAW && epilogue != MOE_EPILOGUE_SWIGLU) return MOE_ERR_INVALID_ARG;
  for (int dt : {base_dtype, out_dtype})
    if (dt != MOE_DTYPE_F32 && dt != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  const bool swiglu = epilogue == MOE_EPILOGUE_SWIGLU;
  if (swiglu && T > 0 && !base) return MOE_ERR_INVALID_ARG;
  if (swiglu && base_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (!swiglu && base_dtype != out_dtype) return MOE_ERR_UNSUPPORTED;
  if (!sorted_assign && (kmax != 1 || E != 1 || topk_ids || expert_offsets))
    return MOE_ERR_INVALID_ARG;
  if (sorted_assign && (!topk_ids || !expert_offsets)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const void* ptrs[] = {x, lora_a, lora_b, out, workspace};
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!adapter_ids || !aligned16(base)) return MOE_ERR_INVALID_ARG;
  if (swiglu && base == out) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_lora_workspace_size(T, kmax, E, n_adapters, R))
    return MOE_ERR_INVALID_ARG;
  LoraParams p;
  p.x = x;
  p.x_by_token = x_by_token != 0 || !sorted_assign;
  p.adapter_ids = adapter_ids;
  p.topk_ids = topk_ids;
  p.sorted = sorted_assign;
  p.offsets = expert_offsets;
  p.T = T;
  p.kmax = kmax;
  p.E = E;
  p.n_adapters = n_adapters;
  p.K = K;
  p.N = N;
  p.R = R;
  p.a = lora_a;
  p.b = lora_b;
  p.scales = scales;
  p.base = base;
  p.out = out;
  p.v = static_cast<float*>(workspace);
  p.err = device_error_word();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rows = T * kmax;
  if (lora_groups(rows, E, n_adapters)) {
    const LoraSpace sp = lora_space(rows, E, n_adapters, R);
    char* ws = static_cast<char*>(workspace);
    int4* tiles = reinterpret_cast<int4*>(ws + sp.tiles);
    const LoraPlan plan{reinterpret_cast<int2*>(ws + sp.rows),
                        tiles,
                        tiles + 1,
                        lora_tile_capacity(rows, E, n_adapters),
                        lora_splits(rows, K),
                        static_cast<uint16_t*>(workspace),
                        !swiglu && base == out};
    return lora_grouped(p, plan, rows, swiglu, out_dtype == MOE_DTYPE_BF16, st);
  }
  moe_status_t s;
  if (R <= 16) s = launch(lora_shrink_kernel<2>, rows, kLoraThreads, 0, st, p);
  else if (R <= 32) s = launch(lora_shrink_kernel<4>, rows, kLoraThreads, 0, st, p);
  else if (R <= 64) s = launch(lora_shrink_kernel<8>, rows, kLoraThreads, 0, st, p);
  else s = launch(lora_shrink_kernel<16>, rows, kLoraThreads, 0, st, p);
  if (s != MOE_OK) return s;
  const int cols = swiglu ? N / 2 : N;
  const dim3 grid(rows, (cols + kLoraWarps * 32 - 1) / (kLoraWarps * 32));
  const bool bf = out_dtype == MOE_DTYPE_BF16;
  if (swiglu)
    return bf ? launch(lora_expand_kernel<false, true, true>, grid, kLoraThreads, 0, st, p)
              : launch(lora_expand_kernel<false, false, true>, grid, kLoraThreads, 0, st, p);
  return bf ? launch(lora_expand_kernel<true, true, false>, grid, kLoraThreads, 0, st, p)
            : launch(lora_expand_kernel<false, false, false>, grid, kLoraThreads, 0, st, p);
}
