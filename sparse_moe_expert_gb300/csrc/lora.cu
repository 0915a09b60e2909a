// Low-rank adapters of many requests beside a shared (or per-expert) product:
//   out[r] = base[r] + scale_a (x[r] A_a,e^T) B_a,e^T
// where row r belongs to a token whose request uses adapter a (or none) and,
// in an expert layer, to expert e.  Page "Qwen3.5-MoE与Qwen3-MoE架构差异深度
// 解析", section 4.4 (expert-level LoRA).
//
// Bound by memory: one adapter's matrices are read for a handful of rows, or
// x, base and out are streamed past small matrices (lora_tc.cu).
//
// Few rows (this file): a cluster of CTAs per row, one launch.  The CTAs share
// K, join their parts of v = scale x A^T through distributed shared memory,
// and share the columns of v B^T; the first columns of B and base are
// requested before the join, so both matrices are on their way at once.
// One launch and one round trip to memory per matrix bound it.  Measured,
// K = N = 4096, bf16: one row of rank 16 4.0 us (two kernels, one CTA per row:
// 7.1); 64 rows of rank 32 over 64 adapters 8.9 us (23 MB, 2.6 TB/s); 64 tokens
// on 4 of 64 experts, gate and up of 768 with 2048 inputs, 8.9 us (25 MB).  With
// SwiGLU and ranks 24 and 32 the kernel spills 20 bytes a thread.
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

template <bool BF16>
__device__ __forceinline__ float load_value(const void* base, int64_t at) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(base)[at]);
  return static_cast<const float*>(base)[at];
}

// Sum of 16 products, four partial sums: two 16-byte pieces of a row of B with
// the same entries of v.
__device__ __forceinline__ float dot16(const uint4 (&b)[2], const float (&v)[16]) {
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t w[4] = {b[q].x, b[q].y, b[q].z, b[q].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_f32x2(w[i]);
      acc[i] = fmaf(v[8 * q + 2 * i], f.x, acc[i]);
      acc[i] = fmaf(v[8 * q + 2 * i + 1], f.y, acc[i]);
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// L values per lane, L lanes (neighbours) per column: lane s of the L gets the
// sum over them of value s.
template <int L>
__device__ __forceinline__ float reduce_lanes(float (&a)[L]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) {
    const bool hi = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < off; ++j) {
      const float keep = hi ? a[j + off] : a[j];
      const float send = hi ? a[j] : a[j + off];
      a[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, off);
    }
  }
  return a[0];
}

// One row per cluster.  x A^T: the warps take blocks of 32 k in turn; lane
// (g, t) holds 8 consecutive k (t) of row g of each eight of A as an
// mma.sync fragment (the order of the contraction index is free), so that
// the tensor core also adds over the lanes; the row of x is row 0 of the
// tile.  v B^T in fp32: a warp takes 32 columns, L = NT / 2 lanes to a row of
// B (neighbouring 16-byte pieces, so that a load covers whole sectors of few
// rows), and a reduce-scatter leaves every lane with one column.  NT: eights
// of the rank (rounded up).
// CTAs of the row kernel that an SM holds at once, by registers.
constexpr int row_ctas_per_sm(int NT) { return NT <= 4 ? 4 : NT <= 8 ? 2 : 1; }

template <int NT, bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
__global__ void __launch_bounds__(kLoraThreads, row_ctas_per_sm(NT)) lora_row_kernel(LoraParams p, int ctas) {
  __shared__ __align__(16) float red[kLoraWarps][NT * 8];
  __shared__ __align__(16) float part[NT * 8];
  __shared__ __align__(16) float v[NT * 8];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int entry = p.sorted ? __ldg(p.sorted + r) : r;  // beside the row count, not after it
  if (r >= lora_rows(p)) return;                         // the whole cluster alike
  const LoraRow row = lora_row(p, r, entry);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int nt = p.R >> 3;
  const int cols = SWIGLU ? p.N / 2 : p.N;
  constexpr int H = SWIGLU ? 2 : 1;
  // columns a lane takes at once (more cost registers, and with them CTAs)
  constexpr int U = NT * H <= 2 ? 2 : 1;
  constexpr int L = NT / 2;  // lanes of a row of B
  const int stride = ctas * kLoraThreads;
  const int first = (rank * kLoraWarps + warp) * 32;         // this warp's first columns
  const int own = (lane % L) * (32 / L) + lane / L;          // the lane's among 32
  const int64_t base_row = (int64_t)r * p.N;
  const uint16_t* bm = p.b + (int64_t)max(row.slot, 0) * p.N * p.R;
  uint4 b[U][H][L][2];
  float z[U][H];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * stride;
      if (c < cols) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          z[u][h] = p.base ? load_value<BASE_BF16>(p.base, base_row + h * cols + c + own) : 0.0f;
          if (row.slot >= 0) {
            const uint4* src = reinterpret_cast<const uint4*>(
                bm + ((int64_t)h * cols + c + lane / L) * p.R) + lane % L;
            const int64_t step = (int64_t)(32 / L) * p.R / 8;
#pragma unroll
            for (int i = 0; i < L; ++i)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (lane % L + L * q < nt) b[u][h][i][q] = __ldg(src + i * step + L * q);
                else b[u][h][i][q] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
    }
  };
  if (row.slot >= 0) {
    const uint4* xr = reinterpret_cast<const uint4*>(p.x + row.x_row * p.K) + t;
    const uint4* ar = reinterpret_cast<const uint4*>(p.a + ((int64_t)row.slot * p.R + g) * p.K) + t;
    float acc[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
    const int blocks = p.K >> 5;
#pragma unroll(NT <= 4 ? 4 : 2)
    for (int kb = rank * kLoraWarps + warp; kb < blocks; kb += ctas * kLoraWarps) {
      uint4 xv = make_uint4(0u, 0u, 0u, 0u);
      if (g == 0) xv = __ldg(xr + kb * 4);
      uint4 av[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (q < nt) av[q] = ldg_nc_v4(ar + (int64_t)q * p.K + kb * 4);
      const uint32_t f0[4] = {xv.x, 0u, xv.y, 0u}, f1[4] = {xv.z, 0u, xv.w, 0u};
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (q < nt) {
          mma_bf16(acc[q], f0, av[q].x, av[q].y);
          mma_bf16(acc[q], f1, av[q].z, av[q].w);
        }
    }
    if (first < cols) fetch(first);
    if (g == 0) {
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        red[warp][q * 8 + 2 * t] = acc[q][0];
        red[warp][q * 8 + 2 * t + 1] = acc[q][1];
      }
    }
    __syncthreads();
    if (tid < p.R) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kLoraWarps; ++w) s += red[w][tid];
      part[tid] = s;
    }
    cluster_barrier();
    if (tid < p.R) {
      float s = 0.0f;
      for (int c = 0; c < ctas; ++c) {  // rank order
        float q;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q) : "r"(cluster_addr(part + tid, c)));
        s += q;
      }
      v[tid] = s * (p.scales ? __ldg(p.scales + row.slot / p.E) : 1.0f);
    }
    __syncthreads();
    // no CTA may leave while another reads its part: arrive now, wait at the end
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if (row.slot >= 0 || SWIGLU || p.base != p.out) {
    float vr[16];
    if (row.slot >= 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = (lane % L + L * (i / 8)) * 8 + i % 8;
        vr[i] = j < p.R ? v[j] : 0.0f;
      }
    }
    for (int c0 = first; c0 < cols; c0 += U * stride) {
      if (row.slot < 0 || c0 != first) fetch(c0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * stride;
        if (c >= cols) break;
        if (row.slot >= 0) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            float a[L];
#pragma unroll
            for (int i = 0; i < L; ++i) a[i] = dot16(b[u][h][i], vr);
            z[u][h] += reduce_lanes<L>(a);
          }
        }
        float o = z[u][0];
        if constexpr (SWIGLU) o = swiglu_f32(z[u][0], z[u][H - 1]);
        const int64_t at = (int64_t)r * cols + c + own;
        if constexpr (OUT_BF16) static_cast<uint16_t*>(p.out)[at] = f32_to_bf16_rne(o);
        else static_cast<float*>(p.out)[at] = o;
      }
    }
  }
  if (row.slot >= 0) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <int NT, bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
moe_status_t launch_rows(const LoraParams& p, int rows, cudaStream_t st) {
  // CTAs per row: as many as run at once without queueing, 8 at most
  int ctas = row_ctas_per_sm(NT) * moe_host::sm_count() / rows;
  ctas = ctas < 1 ? 1 : ctas > 8 ? 8 : ctas;
  return moe_host::launch_clusters(lora_row_kernel<NT, BASE_BF16, OUT_BF16, SWIGLU>,
                                   dim3((unsigned)rows * ctas), kLoraThreads, 0, dim3(ctas), st, p,
                                   ctas);
}

template <bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
moe_status_t lora_few(const LoraParams& p, int rows, cudaStream_t st) {
  if (p.R <= 16) return launch_rows<2, BASE_BF16, OUT_BF16, SWIGLU>(p, rows, st);
  if (p.R <= 32) return launch_rows<4, BASE_BF16, OUT_BF16, SWIGLU>(p, rows, st);
  if (p.R <= 64) return launch_rows<8, BASE_BF16, OUT_BF16, SWIGLU>(p, rows, st);
  return launch_rows<16, BASE_BF16, OUT_BF16, SWIGLU>(p, rows, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace {

// Whether the rows are grouped by adapter (lora_tc.cu) or each gets its own
// cluster.  A cluster costs its row's A and B from L2, so rows x rank; the
// grouping costs two more launches and gains when rows share matrices.
// Measured, K = N = 4096 bf16, us (own cluster / grouped): rank 16, 256 rows
// 11.2 / 18.0 over 8 adapters, 13.4 / 18.8 over 64; 384 rows 18.3 / 17.5 and
// 21.8 / 19.1; rank 64, 64 rows 10.5 / 16.2 over 8, 15.0 / 24.1 over 64; 96 rows
// 22.5 / 16.3 and 32.9 / 26.9; 128 rows 16.7 / 16.6 and 25.8 / 27.5; 256 rows
// 28.0 / 20.3 and 46.0 / 31.1.  Far more rows
// are grouped even if every adapter could have few of them: which of the
// adapters a batch uses is known on the device only.  The grouping's counters
// hold kLoraPlanAdapters adapters; with more every row has its own cluster,
// however many rows there are.
bool lora_groups(int64_t rows, int E, int n_adapters, int R) {
  const int64_t cost = rows * R;
  return n_adapters <= kLoraPlanAdapters &&
         ((cost >= 6144 && rows >= 4 * (int64_t)n_adapters * E) || cost >= 32768);
}

// CTAs per tile in the grouped shrink, with the tiles that full ones and one
// rest per adapter make and at least four k-blocks of 64 each: as many as two
// per SM hold at once, or somewhat more where each keeps a long range of K,
// since a tile's time goes with its range and whole tiles share out badly.
// Measured, us for s = 1, 2, 4, 8 (rounds of CTAs at s = 1): 4096 rows, 64
// adapters, K 4096 (0.3) 68, 53, 48, 57; 16384 rows, 32 adapters, K 4096 (0.5)
// 103, 92, 97, 120; 8000 rows, 300 adapters, K 4096 (1.2) 117, 106, 130, 168;
// 2048 tokens on 4 of 32 experts, 4 adapters, K 2048 (0.6) 51, 45, 49, 67; on 8
// of 128 (2.1) 91, 103, 153, 223; 777 rows, 40 adapters, K 4096 (0.15) 54, 38,
// 31, 32.
int lora_splits(int64_t rows, int64_t slots, int K) {
  const int64_t tiles = (rows + kLoraTileRows - 1) / kLoraTileRows + (slots < rows ? slots : rows);
  const int64_t held = 2 * moe_host::sm_count();
  int s = 1;
  while (s < kLoraMaxSplit && 2 * s * 256 <= K) {
    const int64_t ctas = 2 * s * tiles;
    // at most a round, or 1.3 of them per 1024 of K
    if (ctas > held && ctas * 10240 > held * 13 * (K / (2 * s))) break;
    s *= 2;
  }
  return s;
}

struct LoraSpace {
  size_t rows, tiles, total;  // v comes first
};

LoraSpace lora_space(int64_t rows, int E, int n_adapters, int R) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  LoraSpace s{};
  if (!lora_groups(rows, E, n_adapters, R)) {
    s.total = 256;  // the rows' form needs none; a size of 0 means bad arguments
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
  for (const void* q : {(const void*)adapter_ids, (const void*)topk_ids, (const void*)sorted_assign,
                        (const void*)expert_offsets, (const void*)scales})
    if (!aligned4(q)) return MOE_ERR_INVALID_ARG;
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
  p.err = device_error_word();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rows = T * kmax;
  if (lora_groups(rows, E, n_adapters, R)) {
    const LoraSpace sp = lora_space(rows, E, n_adapters, R);
    char* ws = static_cast<char*>(workspace);
    int4* tiles = reinterpret_cast<int4*>(ws + sp.tiles);
    const LoraPlan plan{reinterpret_cast<int2*>(ws + sp.rows),
                        tiles,
                        tiles + 1,
                        lora_tile_capacity(rows, E, n_adapters),
                        lora_splits(rows, (int64_t)E * n_adapters, K),
                        static_cast<uint16_t*>(workspace),
                        !swiglu && base == out};
    return lora_grouped(p, plan, rows, swiglu, out_dtype == MOE_DTYPE_BF16, st);
  }
  const bool bf = out_dtype == MOE_DTYPE_BF16;
  if (swiglu)
    return bf ? lora_few<false, true, true>(p, rows, st) : lora_few<false, false, true>(p, rows, st);
  return bf ? lora_few<true, true, false>(p, rows, st) : lora_few<false, false, false>(p, rows, st);
}
