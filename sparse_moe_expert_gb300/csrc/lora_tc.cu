// Adapters of many rows: the grouped form of moe_lora_apply (lora.cu has the
// formula and the form for few rows).
//
// Rows are grouped by the matrices they use (lora_plan_kernel), so that a
// tile of up to 128 rows meets one pair A, B on the tensor cores (tcgen05,
// accumulators in TMEM):
//   shrink: D[row, j]  = sum_k x[row, k] A[j, k]; M = 128 rows, N = the rank,
//           a unit is one tile and one range of K (partial sums, added in
//           range order by the expand, keep the result reproducible);
//   expand: D[row, n]  = sum_j v[row, j] B[n, j]; 128 rows x 128 columns, v as
//           two or three bf16 terms side by side along the contraction, so
//           that the fp32 value enters to 2^-17 (bf16 base) or 2^-26 (fp32 base,
//           whose bf16 and fp32 activations are then the same numbers).
// Both stream x, base and out once; the tensor cores take the operands from
// shared memory, so the load/store path carries little else (with mma.sync
// the fragments of v and B would cost it more than base and out together).
#include "async.cuh"
#include "lora.cuh"
#include "tc.cuh"

namespace moe {
namespace {

// ---- grouping --------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanUnroll = 4;

// CTA (e, c): counts the rows of expert e per adapter (the last bin: none),
// the ones before its range c separately, and places its range; range 0 also
// lists the expert's tiles.  The order of rows within an
// adapter is left open (shared-memory atomics): a row's result does not
// depend on its place in a tile.
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(LoraParams p, LoraPlan pl) {
  extern __shared__ int plan_s[];
  pdl_wait();
  pdl_trigger();
  const int bins = p.n_adapters + 1;
  int* cnt = plan_s;
  int* cursor = cnt + bins;
  int* start = cursor + bins;
  __shared__ int tile_base;
  const int tid = threadIdx.x, lane = tid & 31;
  const int e = blockIdx.x, rows = lora_rows(p);
  const int lo = p.sorted ? min(max(__ldg(p.offsets + e), 0), rows) : 0;
  const int n = (p.sorted ? min(max(__ldg(p.offsets + e + 1), lo), rows) : rows) - lo;
  // ranges of whole kPlanThreads rows
  const int64_t step = (int64_t)gridDim.y * kPlanThreads;
  const int64_t per = (n + step - 1) / step * kPlanThreads;
  if (per * blockIdx.y >= n) return;
  const int c0 = (int)(per * blockIdx.y), c1 = (int)(c0 + per < n ? c0 + per : n);
  for (int i = tid; i < bins; i += kPlanThreads) cnt[i] = cursor[i] = 0;
  __syncthreads();
  auto bin_of = [&](int i) {
    const int s = lora_row(p, lo + i).slot;
    return s < 0 ? p.n_adapters : s / p.E;
  };
  for (int i0 = 0; i0 < n; i0 += kPlanThreads * kPlanUnroll) {
    int b[kPlanUnroll];
#pragma unroll
    for (int u = 0; u < kPlanUnroll; ++u) {
      const int i = i0 + u * kPlanThreads + tid;
      b[u] = i < n ? bin_of(i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kPlanUnroll; ++u) {
      const int i = i0 + u * kPlanThreads + tid;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, b[u]);
      if (b[u] >= 0 && (same & lanemask_lt()) == 0u) {
        atomicAdd(&cnt[b[u]], __popc(same));
        if (i < c0) atomicAdd(&cursor[b[u]], __popc(same));  // c0 is a multiple of 32
      }
    }
  }
  __syncthreads();
  if (tid < 32) {
    int carry = 0, tiles = 0;
    for (int x0 = 0; x0 < bins; x0 += 32) {
      const int x = x0 + lane;
      const int v = x < bins ? cnt[x] : 0;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      if (x < bins) {
        start[x] = carry + incl - v;
        cursor[x] += carry + incl - v;
        if (x < p.n_adapters || !pl.skip_none) tiles += (v + kLoraTileRows - 1) / kLoraTileRows;
      }
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (c0 == 0) {
      tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
      if (lane == 0) tile_base = atomicAdd(&pl.tiles[0].x, tiles);
    }
  }
  __syncthreads();
  for (int i0 = c0; i0 < c1; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const int b = i < c1 ? bin_of(i) : -1;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
    int at = 0;
    if (b >= 0 && (same & lanemask_lt()) == 0u) at = atomicAdd(&cursor[b], __popc(same));
    at = __shfl_sync(0xFFFFFFFFu, at, __ffs(same) - 1);
    if (b >= 0) pl.perm[lo + at + __popc(same & lanemask_lt())] = lo + i;
  }
  if (c0 == 0 && tid < 32) {
    int carry = tile_base;
    for (int x0 = 0; x0 < bins; x0 += 32) {
      const int x = x0 + lane;
      const int v = x < bins && (x < p.n_adapters || !pl.skip_none) ? cnt[x] : 0;
      const int tiles = (v + kLoraTileRows - 1) / kLoraTileRows;
      int incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      const int slot = x < p.n_adapters ? x * p.E + e : -1;
      for (int j = 0; j < tiles; ++j) {
        const int64_t at = (int64_t)carry + incl - tiles + j;
        if (at < pl.capacity)  // always, when the offsets are a prefix sum
          pl.tiles[1 + at] = make_int4(slot, lo + start[x] + j * kLoraTileRows,
                                       min(kLoraTileRows, v - j * kLoraTileRows), 0);
        else
          raise_device_error(p.err, MOE_DEVERR_BAD_INDEX);
      }
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
  }
}

// ---- shared by the two products ---------------------------------------------

constexpr int kTcThreads = 256;
constexpr int kBlockBytes = 16384;  // 128 rows x 128 bytes, 128-byte swizzled

// 16 bytes global -> shared; `on` false writes zeros.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 32 columns x 16 lanes: lane (g, t) of the warp gets, for the eight-column
// groups q = 0..3, columns 8q + 2t, 8q + 2t + 1 of rows g (r[4q], r[4q + 1])
// and g + 8 (r[4q + 2], r[4q + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Waits; a wait that runs out sets the device error and `bad`, which the CTA
// joins at its next barrier (__syncthreads_or) so that all threads leave
// their loop together.
__device__ __forceinline__ void wait_or_flag(uint64_t* bar, uint32_t parity, int& bad,
                                             unsigned int* err) {
  if (!mbar_wait_sleep(bar, parity, kWaitBudgetCycles)) {
    bad = 1;
    raise_device_error(err, MOE_DEVERR_TIMEOUT);
  }
}

__device__ __forceinline__ int lora_tiles(const LoraPlan& pl) {
  return (int)min((int64_t)pl.tiles[0].x, pl.capacity);
}

__host__ __device__ constexpr int rank_pad(int R) { return (R + 15) / 16 * 16; }

// ---- shrink ----------------------------------------------------------------

constexpr int kShrinkStages = 4;

__global__ void __launch_bounds__(kTcThreads) lora_shrink_tc_kernel(LoraParams p, LoraPlan pl,
                                                                   int64_t rows_cap,
                                                                   uint32_t tmem_cols) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t done[kShrinkStages];
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int RP = rank_pad(p.R);
  const int stage_bytes = kBlockBytes + RP * 128;
  if (tid == 0) {
    for (int s = 0; s < kShrinkStages; ++s) mbar_init(&done[s], 1);
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 0) {
    tmem_alloc(&tmem_sh, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // only now: a later kernel may not take TMEM from a CTA still to come
  const uint32_t tmem = tmem_sh;
  const uint32_t idesc = idesc_bf16(128, RP);
  int bad = 0;
  const int ntiles = lora_tiles(pl), splits = pl.splits;
  const int nkb = p.K / 64;
  uint32_t phase[kShrinkStages] = {};  // parity of each stage's next completion
  const int c = tid & 7, r0 = tid >> 3;  // this thread's 16-byte column and first row
  for (int u = blockIdx.x; u < ntiles * splits; u += gridDim.x) {
    const int4 tile = pl.tiles[1 + u / splits];
    const int ks = u % splits;
    if (tile.x < 0) continue;
    const int kb0 = ks * nkb / splits, nb = (ks + 1) * nkb / splits - kb0;
    const uint16_t* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 32 * i;
      xr[i] = r < tile.z ? p.x + lora_row(p, pl.perm[tile.y + r]).x_row * p.K + kb0 * 64 + c * 8
                         : nullptr;
    }
    const uint16_t* ar = p.a + ((int64_t)tile.x * p.R + r0) * p.K + kb0 * 64 + c * 8;
    auto load = [&](int kb) {
      unsigned char* xs = smem + (kb % kShrinkStages) * stage_bytes;
      unsigned char* as = xs + kBlockBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (xr[i]) cp_async16(xs + sw128_offset(r0 + 32 * i, c), xr[i] + kb * 64, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        if (r < RP)
          cp_async16(as + sw128_offset(r, c), r < p.R ? ar + (int64_t)32 * i * p.K + kb * 64 : p.a,
                     r < p.R);
      }
    };
    for (int kb = 0; kb < kShrinkStages - 1; ++kb) {
      if (kb < nb) load(kb);
      cp_async_commit();
    }
    bool ok = true;
    for (int kb = 0; kb < nb; ++kb) {
      cp_async_wait<kShrinkStages - 2>();
      fence_proxy_async_smem();
      ok = !__syncthreads_or(bad);
      if (!ok) break;
      const int s = kb % kShrinkStages;
      if (warp == 0) {
        const uint64_t xd = smem_desc_sw128(smem + s * stage_bytes);
        const uint64_t ad = smem_desc_sw128(smem + s * stage_bytes + kBlockBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_bf16(tmem, xd + 2 * k, ad + 2 * k, idesc, kb > 0 || k > 0);
        umma_commit(&done[s]);
      }
      // the stage that k-block kb + 3 takes was read by the MMAs of kb - 1
      const int nx = kb + kShrinkStages - 1;
      if (kb > 0) {
        const int sp = (kb - 1) % kShrinkStages;
        wait_or_flag(&done[sp], phase[sp], bad, p.err);
        phase[sp] ^= 1u;
      }
      if (nx < nb) load(nx);
      cp_async_commit();
    }
    if (ok) {
      const int sp = (nb - 1) % kShrinkStages;
      wait_or_flag(&done[sp], phase[sp], bad, p.err);
      phase[sp] ^= 1u;
    }
    cp_async_wait<0>();
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    if (warp < 4) {
      const int row = warp * 32 + lane;
      const float sc = p.scales ? __ldg(p.scales + tile.x / p.E) : 1.0f;
      float* out = p.v + ((int64_t)ks * rows_cap + tile.y + row) * p.R;
      for (int j = 0; j < RP; j += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + j, r);
        tmem_ld_wait();
        if (row < tile.z) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (j + 4 * q < p.R)
              *reinterpret_cast<float4*>(out + j + 4 * q) =
                  make_float4(sc * __uint_as_float(r[4 * q]), sc * __uint_as_float(r[4 * q + 1]),
                              sc * __uint_as_float(r[4 * q + 2]), sc * __uint_as_float(r[4 * q + 3]));
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, tmem_cols);
}

// ---- expand ----------------------------------------------------------------

// Eight consecutive values of base held as loaded (16 bytes bf16, 32 fp32).
template <bool BF16>
struct Base8 {
  uint4 q[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (BF16) {
      q[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    } else {
      const uint4* b = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      q[0] = b[0];
      q[1] = b[1];
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
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[4 * h] = __uint_as_float(q[h].x);
        f[4 * h + 1] = __uint_as_float(q[h].y);
        f[4 * h + 2] = __uint_as_float(q[h].z);
        f[4 * h + 3] = __uint_as_float(q[h].w);
      }
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void put8(void* out, int64_t at, const float (&f)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

constexpr int kExpandCols = 128;  // accumulator columns of a unit

// Accumulator columns [32 b, 32 b + 32), b = 0..3, are 32 consecutive output
// columns each (SWIGLU: b 0, 1 the gate's, b 2, 3 the same columns of up), in
// an order that leaves lane t of a quad with eight consecutive ones: column
// 8 q + 2 t + i of a block is its column 8 t + 2 q + i.
template <int TERMS, bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
__global__ void __launch_bounds__(kTcThreads, 2) lora_expand_tc_kernel(LoraParams p, LoraPlan pl,
                                                                    int64_t rows_cap) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int RP = rank_pad(p.R);
  const int vblocks = (TERMS * RP + 63) / 64, bblocks = (RP + 63) / 64;
  unsigned char* vs = smem;
  unsigned char* bs = smem + vblocks * kBlockBytes;  // two slots of bblocks blocks
  if (tid == 0) {
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 0) {
    tmem_alloc(&tmem_sh, kExpandCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = tmem_sh;
  const uint32_t idesc = idesc_bf16(128, kExpandCols);
  int bad = 0;
  const int ntiles = lora_tiles(pl);
  const int cols = SWIGLU ? p.N / 2 : p.N;                      // output columns
  const int span = SWIGLU ? kExpandCols / 2 : kExpandCols;      // of them in a unit
  const int chunks = (cols + span - 1) / span;
  const int64_t units = (int64_t)ntiles * chunks;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;

  // B rows of a unit -> slot `s`
  auto load_b = [&](int64_t u, int s) {
    const int4 tile = pl.tiles[1 + u / chunks];
    if (tile.x < 0) return;
    const int col0 = (int)(u % chunks) * span;
    const int nc = RP / 8;
    unsigned char* dst = bs + s * bblocks * kBlockBytes;
    const uint16_t* src = p.b + (int64_t)tile.x * p.N * p.R;
    for (int i = tid; i < kExpandCols * nc; i += kTcThreads) {
      const int row = i / nc, ch = i % nc;
      const int b = row >> 5, w = row & 31;
      int n = col0 + row;
      if (SWIGLU) n = (b >> 1) * cols + col0 + (b & 1) * 32 + w;
      // beyond the matrix: only columns that are never stored
      const bool in = (SWIGLU ? col0 + (b & 1) * 32 : col0 + b * 32) < cols;
      const int drow = b * 32 + 8 * ((w & 7) >> 1) + 2 * (w >> 3) + (w & 1);
      const bool on = in && ch * 8 < p.R;
      cp_async16(dst + (ch >> 3) * kBlockBytes + sw128_offset(drow, ch & 7),
                 on ? src + (int64_t)n * p.R + ch * 8 : p.b, on);
    }
  };

  const int g = lane >> 2, t = lane & 3;
  const int lq = (warp & 3) * 32;  // this warp's accumulator rows
  const int half = warp >> 2;      // and its two 32-column blocks: half (+ 2 or + 1)
  int cur_tile = -1, slot = 0;
  int4 tile = make_int4(-1, 0, 0, 0);
  int64_t row_at[4] = {};  // this lane's four rows (-1: none)
  uint32_t parity = 0;
  if (u0 < u1) load_b(u0, 0);
  cp_async_commit();
  for (int64_t u = u0; u < u1; ++u) {
    const int ti = (int)(u / chunks);
    if (ti != cur_tile) {
      cur_tile = ti;
      tile = pl.tiles[1 + ti];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lq + g + 8 * i;
        row_at[i] = r < tile.z ? (int64_t)pl.perm[tile.y + r] : -1;
      }
      if (tile.x >= 0) {
        // v (the K ranges' sums) -> bf16 terms; rows past the tile's are never stored
        const int quads = RP / 4;
        for (int i = tid; i < tile.z * quads; i += kTcThreads) {
          const int r = i / quads, j = (i % quads) * 4;
          float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (j < p.R) {
            const float* src = p.v + (int64_t)(tile.y + r) * p.R + j;
            for (int s = 0; s < pl.splits; ++s) {
              const float4 q = __ldcg(reinterpret_cast<const float4*>(src + s * rows_cap * p.R));
              f.x += q.x;
              f.y += q.y;
              f.z += q.z;
              f.w += q.w;
            }
          }
#pragma unroll
          for (int x = 0; x < TERMS; ++x) {
            const uint32_t a = pack_bf16x2(f.x, f.y), b = pack_bf16x2(f.z, f.w);
            const int col = x * RP + j;
            *reinterpret_cast<uint2*>(vs + (col >> 6) * kBlockBytes +
                                      sw128_offset(r, (col & 63) >> 3) + (col & 4) * 2) =
                make_uint2(a, b);
            const float2 fa = bf16x2_to_f32x2(a), fb = bf16x2_to_f32x2(b);
            f.x -= fa.x;
            f.y -= fa.y;
            f.z -= fb.x;
            f.w -= fb.y;
          }
        }
      }
    }
    if (u + 1 < u1) load_b(u + 1, slot ^ 1);
    cp_async_commit();
    // base of the unit, in flight while B lands and the MMAs run
    const int col0 = (int)(u % chunks) * span;
    Base8<BASE_BF16> bq[2][4];
    int colb[2];  // first output column of the two blocks in base
    bool in[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = SWIGLU ? col0 + half * 32 : col0 + (half + 2 * h) * 32;
      in[h] = o < cols;
      colb[h] = (SWIGLU ? h * cols : 0) + o + 8 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.base && in[h] && row_at[i] >= 0) bq[h][i].load(p.base, row_at[i] * p.N + colb[h]);
        else bq[h][i].zero();
      }
    }
    cp_async_wait<1>();
    fence_proxy_async_smem();
    if (__syncthreads_or(bad)) break;
    if (tile.x >= 0) {
      if (warp == 0) {
        for (int x = 0; x < TERMS; ++x)
          for (int j = 0; j < RP; j += 16) {
            const int col = x * RP + j;
            const uint64_t ad = smem_desc_sw128(vs + (col >> 6) * kBlockBytes) + ((col & 63) >> 3);
            const uint64_t bd =
                smem_desc_sw128(bs + (slot * bblocks + (j >> 6)) * kBlockBytes) + ((j & 63) >> 3);
            umma_bf16(tmem, ad, bd, idesc, x > 0 || j > 0);
          }
        umma_commit(&done);
      }
      wait_or_flag(&done, parity, bad, p.err);
      parity ^= 1u;
      tc_fence_after();
    }
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {  // accumulator rows lq + 16 hr ..
      float z[2][2][8];               // [block][row g, g + 8]
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[16];
        if (tile.x >= 0) {
          tmem_ld_16x256b_x4(tmem + ((uint32_t)(lq + 16 * hr) << 16) + (half + 2 * h) * 32, r);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bq[h][2 * hr + i].get(z[h][i]);
          if (tile.x >= 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              z[h][i][2 * q] += __uint_as_float(r[4 * q + 2 * i]);
              z[h][i][2 * q + 1] += __uint_as_float(r[4 * q + 2 * i + 1]);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = row_at[2 * hr + i];
        if (row < 0) continue;
        if constexpr (SWIGLU) {
          if (!in[0]) continue;
#pragma unroll
          for (int x = 0; x < 8; ++x) z[0][i][x] = swiglu_f32(z[0][i][x], z[1][i][x]);
          put8<OUT_BF16>(p.out, row * cols + colb[0], z[0][i]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (in[h]) put8<OUT_BF16>(p.out, row * cols + colb[h], z[h][i]);
        }
      }
    }
    slot ^= 1;
    tc_fence_before();
    __syncthreads();  // the accumulator, v and the old slot of B are free again
    tc_fence_after();
  }
  cp_async_wait<0>();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kExpandCols);
}

template <int TERMS, bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
moe_status_t launch_expand(const LoraParams& p, const LoraPlan& plan, int64_t rows,
                           int64_t capacity, cudaStream_t st) {
  using namespace moe_host;
  const int RP = rank_pad(p.R);
  const size_t smem =
      ((TERMS * RP + 63) / 64 + 2 * ((RP + 63) / 64)) * (size_t)kBlockBytes + 1024;
  auto kern = lora_expand_tc_kernel<TERMS, BASE_BF16, OUT_BF16, SWIGLU>;
  static size_t set_max[kMaxCachedDevices] = {};
  const int dev = device_index();
  if (smem > set_max[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    set_max[dev] = smem;
  }
  const int per_sm = smem <= 110 * 1024 ? 2 : 1;
  const int span = SWIGLU ? kExpandCols / 2 : kExpandCols;
  const int cols = SWIGLU ? p.N / 2 : p.N;
  int64_t grid = capacity * ((cols + span - 1) / span);
  if (grid > (int64_t)sm_count() * per_sm) grid = (int64_t)sm_count() * per_sm;
  return launch(kern, (int)grid, kTcThreads, smem, st, p, plan, rows);
}

}  // namespace

moe_status_t lora_grouped(const LoraParams& p, const LoraPlan& plan, int64_t rows, bool swiglu,
                          bool out_bf16, cudaStream_t st) {
  using namespace moe_host;
  const int64_t capacity = plan.capacity;
  if (cudaMemsetAsync(plan.tiles, 0, sizeof(int4), st) != cudaSuccess) return MOE_ERR_CUDA;
  const size_t plan_smem = (size_t)3 * (p.n_adapters + 1) * sizeof(int);
  if (plan_smem > 48 * 1024 &&
      cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)plan_smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  // an expert has about T rows at most; longer ones only make the ranges longer
  int64_t chunks = ((int64_t)p.T + kPlanThreads - 1) / kPlanThreads;
  if (chunks > 64) chunks = 64;
  moe_status_t s = launch(lora_plan_kernel, dim3(p.E, (unsigned)chunks), kPlanThreads, plan_smem, st,
                          p, plan);
  if (s != MOE_OK) return s;
  const int RP = rank_pad(p.R);
  const size_t smem = (size_t)kShrinkStages * (kBlockBytes + RP * 128) + 1024;
  static size_t set_max[kMaxCachedDevices] = {};
  const int dev = device_index();
  if (smem > set_max[dev]) {
    if (cudaFuncSetAttribute(lora_shrink_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem) != cudaSuccess)
      return MOE_ERR_CUDA;
    set_max[dev] = smem;
  }
  uint32_t tmem_cols = 32;
  while ((int)tmem_cols < RP) tmem_cols <<= 1;
  const int per_sm = smem <= 110 * 1024 ? 2 : 1;
  int64_t grid = capacity * plan.splits;
  if (grid > (int64_t)sm_count() * per_sm) grid = (int64_t)sm_count() * per_sm;
  s = launch(lora_shrink_tc_kernel, (int)grid, kTcThreads, smem, st, p, plan, rows, tmem_cols);
  if (s != MOE_OK) return s;
  if (swiglu)
    return out_bf16 ? launch_expand<3, false, true, true>(p, plan, rows, capacity, st)
                    : launch_expand<3, false, false, true>(p, plan, rows, capacity, st);
  return out_bf16 ? launch_expand<2, true, true, false>(p, plan, rows, capacity, st)
                  : launch_expand<3, false, false, false>(p, plan, rows, capacity, st);
}

}  // namespace moe
