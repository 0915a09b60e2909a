// Parameters and row lookup shared by the adapter kernels.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxRank = 128;
__host__ __device__ constexpr int rank_pad(int R) { return (R + 15) / 16 * 16; }
constexpr int kLoraMaxTerms = 3;

struct LoraParams {
  const uint16_t* x;
  int x_by_token;
  const int32_t* adapter_ids;  // [T]
  const int32_t* topk_ids;     // [T, kmax], null: one projection (E = 1)
  const int32_t* sorted;       // [T kmax], null: rows are tokens
  const int32_t* offsets;      // [E + 1]
  int T, kmax, E, n_adapters;
  int K, N, R;
  const uint16_t* a;  // [n_adapters, E, R, K]
  const uint16_t* b;  // [n_adapters, E, N, R]
  const float* scales;
  const void* base;
  void* out;
  unsigned int* err;
};

// Which matrices a row uses.
struct LoraRow {
  int slot;       // adapter * E + expert, or -1: no adapter
  int64_t x_row;  // row of x
};

__device__ __forceinline__ int lora_rows(const LoraParams& p) {
  if (!p.sorted) return p.T;
  return min(max(__ldg(p.offsets + p.E), 0), p.T * p.kmax);
}

// `a`: the row's entry of sorted (r itself without one).
__device__ __forceinline__ LoraRow lora_row(const LoraParams& p, int r, int a) {
  int e = 0;
  if (p.sorted) {
    if (a < 0 || a >= p.T * p.kmax) {
      raise_device_error(p.err, MOE_DEVERR_BAD_INDEX);
      return {-1, 0};
    }
    e = __ldg(p.topk_ids + a);
  }
  const int token = a / p.kmax;
  const int ad = __ldg(p.adapter_ids + token);
  LoraRow row{-1, p.x_by_token ? token : r};
  if (e < 0 || e >= p.E) {
    raise_device_error(p.err, MOE_DEVERR_BAD_EXPERT);
  } else if (ad >= p.n_adapters) {
    raise_device_error(p.err, MOE_DEVERR_BAD_ADAPTER);
  } else if (ad >= 0) {
    row.slot = ad * p.E + e;
  }
  return row;
}

__device__ __forceinline__ LoraRow lora_row(const LoraParams& p, int r) {
  return lora_row(p, r, p.sorted ? __ldg(p.sorted + r) : r);
}

// Which row of x a row uses (the row's slot is known).
__device__ __forceinline__ int lora_x_row(const LoraParams& p, int r) {
  return p.sorted && p.x_by_token ? __ldg(p.sorted + r) / p.kmax : r;
}

// A shared-memory address of this CTA as CTA `rank` of the cluster has it, and
// the barrier of the cluster's CTAs.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}

// Rows grouped by the matrices they use, made on the device for one call.
// rows[pos] = (row, row of x).  A tile is a run of positions of one slot:
// (slot or -1, first position, rows, 0).  Large tiles (up to 128 rows) fill
// the list from the front, small ones (up to 16) from the back; counts[0] =
// (large, small, 0, 0).
constexpr int kLoraTileRows = 128;
constexpr int kLoraSmallRows = 16;
constexpr int kLoraSmallMost = 32;  // a rest of at most this many rows takes small tiles
constexpr int kLoraMaxSplit = 8;    // CTAs that share a tile's K in the grouped shrink
struct LoraPlan {
  int2* rows;
  int4* counts;
  int4* tiles;
  int64_t capacity;  // tiles the list holds
  int splits;        // CTAs (a cluster) that share a tile's K: 1, 2, 4 or 8
  uint16_t* terms;   // v as bf16 terms side by side: [rows][terms * padded rank]
  int skip_none;     // rows without an adapter need no work
};

// Most adapters the grouping's counters hold in shared memory.
constexpr int kLoraPlanAdapters = 2048;

inline int64_t lora_tile_capacity(int64_t rows, int E, int n_adapters) {
  const int64_t most =
      rows / kLoraTileRows + (int64_t)(kLoraSmallMost / kLoraSmallRows) * E * (n_adapters + 1);
  return rows < most ? rows : most;
}

moe_status_t lora_grouped(const LoraParams& p, const LoraPlan& plan, int64_t rows, bool swiglu,
                          bool out_bf16, cudaStream_t st);

}  // namespace moe
