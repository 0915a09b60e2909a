// Adapters of many rows: the grouped form of moe_lora_apply (lora.cu has the
// formula and the form for few rows).
//
// Rows are grouped by the matrices they use (lora_plan_kernel).  A tile of up
// to 128 rows meets one pair A, B on the tensor cores (tcgen05, accumulators
// in TMEM):
//   shrink: D[row, j]  = sum_k x[row, k] A[j, k]; M = 128 rows, N = the rank;
//           when tiles are few, a cluster of 2 to 8 CTAs shares a tile's K and
//           joins the sums through distributed shared memory in rank order;
//   expand: D[row, n]  = sum_j v[row, j] B[n, j]; 128 rows x 64 columns, v as
//           two or three bf16 terms side by side along the contraction, so
//           that the fp32 value enters to 2^-17 (bf16 base) or 2^-26 (fp32 base,
//           whose bf16 and fp32 activations are then the same numbers).
// Both stream x, base and out once; the tensor cores take the operands from
// shared memory, so the load/store path carries little else (with mma.sync
// the fragments of v and B would cost it more than base and out together).
// What is left of an adapter's rows after whole tiles, 32 at most, goes in
// tiles of up to 16 rows through mma.sync with operands straight from global
// memory: there A and B are the bulk of the bytes, each read once per tile,
// and a 128-row accumulator would leave three of four warps without rows.
// (With rests of up to 16, 32, 48, 96 rows in small tiles, us: 2048 tokens x 8
// of 128 experts, 4 adapters, rank 16, SwiGLU 116, 97, 101, 97; 8192 tokens, 8
// adapters, rank 64 122, 120, 121, 127; 4000 tokens, 300 adapters 57, 63, 64, 64.)
//
// Measured, 8192 tokens, 8 adapters, 4096 -> 11008, rank 64, bf16: 112 us, of
// it plan 6, shrink 22 (67 MB of x: 10 at the copy rate; 1 us per k-block of 64,
// the latency of its loads), expand 80 (360 MB: 53 at the copy rate, 58 to 84
// for a bare copy with its access pattern).  777 tokens, 40 adapters, rank 32,
// fp32: 30.1 us, of it plan 5, shrink 12, expand 12, each bound by its chain of
// dependent loads.  The shrink spills 52 to 100 bytes a thread at its 128
// registers (two CTAs per SM), the SwiGLU expand 76.  Gathering the shrink's rows with TMA (four rows of 128 bytes
// per request) was slower, 128 and 43 us: the requests follow one another at
// some 40 ns.
#include "async.cuh"
#include "lora.cuh"
#include "tc.cuh"

namespace moe {
namespace {

// ---- grouping --------------------------------------------------------------

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanUnroll = 4;
constexpr int kPlanRanges = 8;  // CTAs that share an expert's rows, at most

// Tiles of an adapter's n rows.
__device__ __forceinline__ int2 tiles_of(int n) {
  const int rest = n % kLoraTileRows;
  const bool small = rest <= kLoraSmallMost;
  return make_int2(n / kLoraTileRows + (small ? 0 : 1),
                   small ? (rest + kLoraSmallRows - 1) / kLoraSmallRows : 0);
}

template <typename T>
__device__ __forceinline__ T warp_scan_incl(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// A cluster per expert e: CTA c of it counts its range of the expert's rows
// per adapter (the last bin: none), each warp its part of the range in
// counters of its own, learns the other CTAs' counts through distributed
// shared memory, and places its rows, the warps independently.  The first CTA
// also lists the expert's tiles.  Rows of an adapter stay in order, so that
// every row meets the same tile, and the same sums, each time; the order of
// the experts' tiles is left open.
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(LoraParams p, LoraPlan pl) {
  extern __shared__ int plan_s[];
  __shared__ unsigned tile_total;  // as first_tile
  __shared__ int2 tile_base;       // the expert's first tiles in the list
  pdl_wait();
  pdl_trigger();
  const int bins = p.n_adapters + 1;
  int* own = plan_s;                 // this CTA's counts
  int* cnt = own + bins;             // the expert's
  int* start = cnt + bins;           // first position of each adapter
  unsigned* first_tile = reinterpret_cast<unsigned*>(start + bins);  // and tile: large, small
  int* cursor = start + 2 * bins;    // [warp][bins]: counts, then next positions
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e = blockIdx.x, rows = lora_rows(p);
  const int ranges = gridDim.y, range = blockIdx.y;  // the cluster's size, the rank in it
  const int lo = p.sorted ? min(max(__ldg(p.offsets + e), 0), rows) : 0;
  const int n = (p.sorted ? min(max(__ldg(p.offsets + e + 1), lo), rows) : rows) - lo;
  if (n <= 0) {  // for the whole cluster alike
    if (p.E == 1 && range == 0 && tid == 0) *pl.counts = make_int4(0, 0, 0, 0);
    return;
  }
  // this warp's rows, whole groups of 32
  const int64_t per = (((int64_t)n + ranges * kPlanWarps - 1) / (ranges * kPlanWarps) + 31) / 32 * 32;
  const int64_t w0 = per * (range * kPlanWarps + warp);
  const int c0 = (int)(w0 < n ? w0 : n), c1 = (int)(w0 + per < n ? w0 + per : n);
  for (int i = tid; i < kPlanWarps * bins; i += kPlanThreads) cursor[i] = 0;
  __syncthreads();
  auto bin_of = [&](int i) {
    const int s = lora_row(p, lo + i).slot;
    return s < 0 ? p.n_adapters : p.E == 1 ? s : s / p.E;
  };
  int* mine = cursor + warp * bins;
  int kept[kPlanUnroll];  // the bins of the warp's first rows
#pragma unroll
  for (int u = 0; u < kPlanUnroll; ++u) {
    const int i = c0 + u * 32 + lane;
    kept[u] = i < c1 ? bin_of(i) : -1;
  }
#pragma unroll
  for (int u = 0; u < kPlanUnroll; ++u)
    if (kept[u] >= 0) atomicAdd(&mine[kept[u]], 1);
  for (int i = c0 + kPlanUnroll * 32 + lane; i < c1; i += 32) atomicAdd(&mine[bin_of(i)], 1);
  __syncthreads();
  // counts of the CTA, and where in it each warp's rows begin
  for (int x = tid; x < bins; x += kPlanThreads) {
    int sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int v = cursor[w * bins + x];
      cursor[w * bins + x] = sum;
      sum += v;
    }
    own[x] = sum;
    cnt[x] = sum;
  }
  __syncthreads();
  if (ranges > 1) {
    cluster_barrier();
    for (int x = tid; x < bins; x += kPlanThreads) {
      int v[kPlanRanges];
#pragma unroll
      for (int r = 0; r < kPlanRanges; ++r)
        if (r < ranges)
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(cluster_addr(own + x, r)));
      int total = 0, before = 0;
#pragma unroll
      for (int r = 0; r < kPlanRanges; ++r)
        if (r < ranges) {
          total += v[r];
          if (r < range) before += v[r];
        }
      cnt[x] = total;
      for (int w = 0; w < kPlanWarps; ++w) cursor[w * bins + x] += before;
    }
    __syncthreads();
    cluster_arrive();  // the other CTAs' counts have been read
  }
  // rows without an adapter are copied, which large tiles do as well
  auto tiles_in = [&](int x) {
    if (x >= bins || (x == p.n_adapters && pl.skip_none)) return make_int2(0, 0);
    if (x == p.n_adapters) return make_int2((cnt[x] + kLoraTileRows - 1) / kLoraTileRows, 0);
    return tiles_of(cnt[x]);
  };
  // large tiles above, small ones (two per adapter at most) below
  constexpr int kSmallBits = 13;
  constexpr unsigned kSmallMask = (1u << kSmallBits) - 1;
  static_assert(kLoraSmallMost / kLoraSmallRows * kLoraPlanAdapters <= kSmallMask, "small tiles fit");
  if (warp == 0) {
    int carry = 0;
    unsigned tcarry = 0;
    for (int x0 = 0; x0 < bins; x0 += 32) {
      const int x = x0 + lane;
      const int v = x < bins ? cnt[x] : 0;
      const int2 k = tiles_in(x);
      const unsigned kk = ((unsigned)k.x << kSmallBits) + k.y;
      const int incl = warp_scan_incl(v);
      const unsigned tincl = warp_scan_incl(kk);
      if (x < bins) {
        start[x] = carry + incl - v;
        first_tile[x] = tcarry + tincl - kk;
      }
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
      tcarry += __shfl_sync(0xFFFFFFFFu, tincl, 31);
    }
    if (lane == 0) tile_total = tcarry;
  }
  __syncthreads();
  if (range == 0 && tid == kPlanThreads - 1) {
    const int large = tile_total >> kSmallBits, small = tile_total & kSmallMask;
    if (p.E == 1) {
      *pl.counts = make_int4(large, small, 0, 0);
      tile_base = make_int2(0, 0);
    } else {
      tile_base = make_int2(atomicAdd(&pl.counts->x, large), atomicAdd(&pl.counts->y, small));
    }
  }
  auto place = [&](int i, int b) {  // the warp together
    const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
    const int before = __popc(same & lanemask_lt());
    int at = 0;
    if (b >= 0) at = mine[b];
    __syncwarp();
    if (b >= 0 && before == 0) mine[b] = at + __popc(same);
    __syncwarp();
    if (b >= 0) pl.rows[lo + start[b] + at + before] = make_int2(lo + i, lora_x_row(p, lo + i));
  };
#pragma unroll
  for (int u = 0; u < kPlanUnroll; ++u)
    if (c0 + u * 32 < c1) place(c0 + u * 32 + lane, kept[u]);
  for (int i0 = c0 + kPlanUnroll * 32; i0 < c1; i0 += 32)
    place(i0 + lane, i0 + lane < c1 ? bin_of(i0 + lane) : -1);
  if (ranges > 1) cluster_wait();
  if (range != 0) return;
  __syncthreads();
  // the tiles, eight threads per adapter
  auto put = [&](int64_t at, int slot, int first, int num) {
    if (at >= 0 && at < pl.capacity)  // always, when the offsets are a prefix sum
      pl.tiles[at] = make_int4(slot, first, num, 0);
    else
      raise_device_error(p.err, MOE_DEVERR_BAD_INDEX);
  };
  const int2 base = tile_base;
  for (int x = tid >> 3; x < bins; x += kPlanThreads / 8) {
    const int2 k = tiles_in(x);
    const int64_t x0 = (int64_t)base.x + (first_tile[x] >> kSmallBits);
    const int64_t y0 = pl.capacity - 1 - ((int64_t)base.y + (first_tile[x] & kSmallMask));
    const int slot = x < p.n_adapters ? x * p.E + e : -1;
    const int first = lo + start[x], v = cnt[x], done = k.x * kLoraTileRows;
    for (int j = tid & 7; j < k.x; j += 8)
      put(x0 + j, slot, first + j * kLoraTileRows, min(kLoraTileRows, v - j * kLoraTileRows));
    for (int j = tid & 7; j < k.y; j += 8)
      put(y0 - j, slot, first + done + j * kLoraSmallRows, min(kLoraSmallRows, v - done - j * kLoraSmallRows));
  }
}

// ---- shared by the two products ---------------------------------------------

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
  if (!bad && !mbar_wait_sleep(bar, parity, kWaitBudgetCycles)) {
    bad = 1;
    raise_device_error(err, MOE_DEVERR_TIMEOUT);
  }
}

// (large, small) tiles; never more than the list holds.  Past L1, which may
// hold an earlier call's numbers where a kernel reads them before its wait.
__device__ __forceinline__ int2 lora_tiles(const LoraPlan& pl) {
  const int4 c = __ldcg(pl.counts);
  const int large = (int)min((int64_t)max(c.x, 0), pl.capacity);
  return make_int2(large, (int)min((int64_t)max(c.y, 0), pl.capacity - large));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- shrink ----------------------------------------------------------------

constexpr int kShrinkThreads = 256;
constexpr int kShrinkWarps = kShrinkThreads / 32;
// k-blocks in shared memory.  Four for ranks up to 32; with more the expand's
// CTAs find less room to start beside the shrink's.  us with 3 / 4 / 5: 777
// rows, rank 32 30.5 / 29.7 / -; 4096 rows, rank 16 37.9 / 36.3 / 36.5; 8192
// rows, rank 64, N 11008 111.3 / 114.5 / -.
__host__ __device__ constexpr int shrink_stages(int NT) { return NT > 4 ? 3 : 4; }

// A tile of up to 16 rows, k in [k0, k1): the warps take blocks of 32 k in
// turn, fragments straight from global memory (lane t of a quad holds 8
// consecutive k of its row), their sums added in warp order.  NT: eights of
// the rank (rounded up).
template <int NT>
__device__ __forceinline__ void shrink_small(const LoraParams& p, const LoraPlan& pl, int4 tile,
                                             int k0, int k1, float* part, int pitch, float* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int nt = p.R >> 3;
  const bool on0 = g < tile.z, on1 = g + 8 < tile.z;
  const uint4* x0 = reinterpret_cast<const uint4*>(
      p.x + (int64_t)(on0 ? pl.rows[tile.y + g].y : 0) * p.K + k0) + t;
  const uint4* x1 = reinterpret_cast<const uint4*>(
      p.x + (int64_t)(on1 ? pl.rows[tile.y + g + 8].y : 0) * p.K + k0) + t;
  const uint4* ar = reinterpret_cast<const uint4*>(p.a + ((int64_t)tile.x * p.R + g) * p.K + k0) + t;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  constexpr int RW = NT * 8;
  constexpr int Q = NT < 8 ? NT : 8;  // eights of the rank at a time, for the registers
#pragma unroll 1
  for (int q0 = 0; q0 < NT; q0 += Q) {
    float acc[Q][4];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
#pragma unroll(NT <= 2 ? 4 : 2)
    for (int kb = warp; kb < (k1 - k0) >> 5; kb += kShrinkWarps) {
      const uint4 a = on0 ? __ldg(x0 + kb * 4) : zero, b = on1 ? __ldg(x1 + kb * 4) : zero;
      uint4 w[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q0 + q < nt) w[q] = ldg_nc_v4(ar + (int64_t)(q0 + q) * p.K + kb * 4);
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q0 + q < nt) {
          mma_bf16(acc[q], a.x, b.x, a.y, b.y, w[q].x, w[q].y);
          mma_bf16(acc[q], a.z, b.z, a.w, b.w, w[q].z, w[q].w);
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float* at = red + (warp * kLoraSmallRows + g) * RW + (q0 + q) * 8 + 2 * t;
      *reinterpret_cast<float2*>(at) = make_float2(acc[q][0], acc[q][1]);
      *reinterpret_cast<float2*>(at + 8 * RW) = make_float2(acc[q][2], acc[q][3]);
    }
  }
  __syncthreads();
  for (int i = tid; i < kLoraSmallRows * RW; i += kShrinkThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kShrinkWarps; ++w) s += red[w * kLoraSmallRows * RW + i];
    if (i % RW < p.R) part[(i / RW) * pitch + i % RW] = s;
  }
}

// The values' next bf16 terms, which are taken off them.  A finite value past
// bf16's largest number gives that one and leaves the rest; an infinity or a
// NaN is its first term alone (what is left of it would be a NaN, and so would
// the sum of its terms' products).
__device__ __forceinline__ uint32_t take_term(float& lo, float& hi) {
  constexpr float top = 0x1.FEp127f;
  const bool l = fabsf(lo) < INFINITY, h = fabsf(hi) < INFINITY;
  const uint32_t w = pack_bf16x2(l ? fminf(fmaxf(lo, -top), top) : lo,
                                 h ? fminf(fmaxf(hi, -top), top) : hi);
  const float2 f = bf16x2_to_f32x2(w);
  lo = l ? lo - f.x : 0.0f;
  hi = h ? hi - f.y : 0.0f;
  return w;
}

// A cluster walks over the tiles, its CTAs each over their range of K; the
// joined sums are scaled and stored as bf16 terms, ready for the expand.
template <int NT>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_tc_kernel(
    LoraParams p, LoraPlan pl, int terms, uint32_t tmem_cols) {
  constexpr int kStages = shrink_stages(NT);
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int RP = rank_pad(p.R);
  const int stage_bytes = kBlockBytes + RP * 128;
  // sums of a tile, over the stages once their products are done; the small
  // tiles' per-warp sums lie behind them
  float* part = reinterpret_cast<float*>(smem);
  const int pitch = RP + 4;
  float* red = part + kLoraSmallRows * pitch;
  if (tid == 0) {
    mbar_init(&done, 1);
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
  const int2 ntiles = lora_tiles(pl);
  const int splits = pl.splits, rank = blockIdx.x % splits;
  const int nkb = p.K / 64;
  const int kb0 = rank * nkb / splits, nb = (rank + 1) * nkb / splits - kb0;
  uint32_t parity = 0;  // of the next completion (warp 0)
  const int c = tid & 7, r0 = tid >> 3;  // this thread's 16-byte column and first row
  for (int ti = blockIdx.x / splits; ti < ntiles.x + ntiles.y; ti += gridDim.x / splits) {
    const bool is_small = ti >= ntiles.x;
    const int4 tile = pl.tiles[is_small ? pl.capacity - 1 - (ti - ntiles.x) : ti];
    if (tile.x < 0) continue;  // the whole cluster alike
    if (is_small) {
      shrink_small<NT>(p, pl, tile, kb0 * 64, (kb0 + nb) * 64, part, pitch, red);
    } else {
      const uint16_t* xr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        xr[i] = r < tile.z ? p.x + (int64_t)pl.rows[tile.y + r].y * p.K + kb0 * 64 + c * 8 : nullptr;
      }
      const uint16_t* ar = p.a + ((int64_t)tile.x * p.R + r0) * p.K + kb0 * 64 + c * 8;
      const int64_t a_step = (int64_t)32 * p.K;
      // the next k-block -> stage s
      auto load = [&](int s) {
        unsigned char* at = smem + s * stage_bytes + sw128_offset(r0, c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (xr[i]) {
            cp_async16(at + i * 4096, xr[i], true);
            xr[i] += 64;
          }
#pragma unroll
        for (int i = 0; i < (NT * 8 + 31) / 32; ++i) {
          const int r = r0 + 32 * i;
          if (r < RP)
            cp_async16(at + kBlockBytes + i * 4096, r < p.R ? ar + i * a_step : p.a, r < p.R);
        }
        ar += 64;
      };
      for (int kb = 0; kb < kStages - 1; ++kb) {
        if (kb < nb) load(kb);
        cp_async_commit();
      }
      int s = 0, before = kStages - 1;  // stages of this k-block and of the one before
      for (int kb = 0; kb < nb; ++kb) {
        cp_async_wait<kStages - 2>();
        fence_proxy_async_smem();
        // the products of the k-block before have had this one's wait to end
        if (warp == 0 && kb > 0) {
          wait_or_flag(&done, parity, bad, p.err);
          parity ^= 1u;
        }
        if (__syncthreads_or(bad)) {
          bad = 1;
          break;
        }
        if (warp == 0) {
          const uint64_t xd = smem_desc_sw128(smem + s * stage_bytes);
          const uint64_t ad = smem_desc_sw128(smem + s * stage_bytes + kBlockBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem, xd + 2 * k, ad + 2 * k, idesc, kb > 0 || k > 0);
          umma_commit(&done);
        }
        if (kb + kStages - 1 < nb) load(before);
        cp_async_commit();
        before = s;
        s = s == kStages - 1 ? 0 : s + 1;
      }
      if (warp == 0) {
        wait_or_flag(&done, parity, bad, p.err);
        parity ^= 1u;
      }
      cp_async_wait<0>();
      __syncthreads();
      tc_fence_after();
      // rows of the tile in warps 0-3, half of the columns in each warp of a pair
      const int row = (warp & 3) * 32 + lane;
      for (int j = (warp >> 2) * 16; j < RP; j += 32) {
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + j, r);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(part + row * pitch + j + 4 * q) =
              make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                          __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
      }
      tc_fence_before();
    }
    __syncthreads();
    if (splits > 1) cluster_barrier();
    tc_fence_after();
    // join in rank order, each CTA its share of the values
    const float sc = p.scales ? __ldg(p.scales + tile.x / p.E) : 1.0f;
    const int quads = RP / 4;
    for (int i = rank * kShrinkThreads + tid; i < tile.z * quads; i += splits * kShrinkThreads) {
      const int r = i / quads, j = (i - r * quads) * 4;
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j < p.R) {
        const float* at = part + r * pitch + j;
        float4 q[kLoraMaxSplit];
#pragma unroll
        for (int s = 0; s < kLoraMaxSplit; ++s)
          if (s < splits) {
            if (s == rank)
              q[s] = *reinterpret_cast<const float4*>(at);
            else
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(q[s].x), "=f"(q[s].y), "=f"(q[s].z), "=f"(q[s].w)
                           : "r"(cluster_addr(at, s)));
          }
#pragma unroll
        for (int s = 0; s < kLoraMaxSplit; ++s)
          if (s < splits) {
            f.x += q[s].x;
            f.y += q[s].y;
            f.z += q[s].z;
            f.w += q[s].w;
          }
        f.x *= sc;
        f.y *= sc;
        f.z *= sc;
        f.w *= sc;
      }
      uint16_t* out = pl.terms + (int64_t)(tile.y + r) * terms * RP + j;
      for (int x = 0; x < terms; ++x) {
        const uint32_t a = take_term(f.x, f.y), b = take_term(f.z, f.w);
        *reinterpret_cast<uint2*>(out + x * RP) = make_uint2(a, b);
      }
    }
    __syncthreads();
    if (splits > 1) cluster_barrier();
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, tmem_cols);
}

// ---- expand ----------------------------------------------------------------

// 16 bytes of a row of base.  A unit reads 128 (bf16) or 256 bytes of each of
// its rows; asking L2 for 256 at a time makes DRAM's pieces longer: 8192 x 11008
// bf16 over both directions 114.7 us for the call, 118.5 without.
__device__ __forceinline__ uint4 load_ahead(const void* p) {
  uint4 v;
  asm volatile("ld.global.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Eight consecutive values of base held as loaded (16 bytes bf16, 32 fp32).
template <bool BF16>
struct Base8 {
  uint4 q[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (BF16) {
      q[0] = load_ahead(static_cast<const uint16_t*>(base) + at);
    } else {
      const float* b = static_cast<const float*>(base) + at;
      q[0] = load_ahead(b);
      q[1] = load_ahead(b + 4);
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

constexpr int kExpandThreads = 128;  // of a group of warps
constexpr int kExpandCols = 64;      // accumulator columns of a group in a large unit

// v's terms of the `n` rows from position `first` -> shared memory, 128-byte
// swizzled; rows n .. up to `fill` become zeros.  Asynchronous copies.
template <int TERMS, int THREADS>
__device__ __forceinline__ void stage_v(const LoraPlan& pl, int RP, int first, int n, int fill,
                                        unsigned char* vs) {
  const int pieces = TERMS * RP / 8, c0 = threadIdx.x & 3;
  for (int r = threadIdx.x >> 2; r < fill; r += THREADS / 4) {
    const uint16_t* src = pl.terms + (int64_t)(first + (r < n ? r : 0)) * (TERMS * RP);
    for (int c = c0; c < pieces; c += 4)
      cp_async16(vs + (c >> 3) * kBlockBytes + sw128_offset(r, c & 7), src + c * 8, r < n);
  }
}

// Operands of a small tile's 32-column block that do not wait for v: the
// lane's pieces of B for the first 64 of the rank (columns col .. of B's rows,
// in the order of the large units), requested before v has landed.
struct SmallB {
  uint2 q[4][4];  // [16 of the rank][eight columns]
  __device__ __forceinline__ static uint2 piece(const uint16_t* b0, int R, int s, int i) {
    const int t = threadIdx.x & 3;
    return s + 4 * t < R ? __ldg(reinterpret_cast<const uint2*>(b0 + (int64_t)(2 * i) * R + s))
                         : make_uint2(0u, 0u);
  }
  __device__ __forceinline__ void load(const uint16_t* b0, int R) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[s][i] = 16 * s < R ? piece(b0, R, 16 * s, i) : make_uint2(0u, 0u);
  }
};

// acc[q] += v B^T for rows g and g + 8: the lane's columns 8 t + 2 q + {0, 1}.
template <int TERMS>
__device__ __forceinline__ void small_step(float (&acc)[4][4], const uint2 (&bq)[4], int RP, int s,
                                           const unsigned char* vs) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int x = TERMS - 1; x >= 0; --x) {  // the small terms first
    const int c = x * RP + s + 4 * t;
    const unsigned char* at = vs + (c >> 6) * kBlockBytes + (c & 4) * 2;
    const uint2 lo = *reinterpret_cast<const uint2*>(at + sw128_offset(g, (c & 63) >> 3));
    const uint2 hi = *reinterpret_cast<const uint2*>(at + sw128_offset(g + 8, (c & 63) >> 3));
#pragma unroll
    for (int q = 0; q < 4; ++q) mma_bf16(acc[q], lo.x, hi.x, lo.y, hi.y, bq[q].x, bq[q].y);
  }
}

template <int TERMS>
__device__ __forceinline__ void small_block(float (&acc)[4][4], const SmallB& b,
                                            const uint16_t* b0, int R, const unsigned char* vs) {
  const int RP = rank_pad(R);
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (16 * s < R) small_step<TERMS>(acc, b.q[s], RP, 16 * s, vs);
  for (int s = 64; s < R; s += 16) {
    uint2 bq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bq[i] = SmallB::piece(b0, R, s, i);
    small_step<TERMS>(acc, bq, RP, s, vs);
  }
}

// Large units: accumulator columns [32 h, 32 h + 32), h = 0, 1, are 32
// consecutive output columns each (SWIGLU: the gate's, then the same ones of
// up), in an order that leaves lane t of a quad with eight consecutive ones:
// column 8 q + 2 t + i of a block is its column 8 t + 2 q + i.  A lane's
// pieces of base are requested one unit ahead, as soon as the registers of
// the unit before are consumed, so loads are in flight through the waits.
// GROUPS of four warps have columns of their own and share v.
template <int TERMS, bool BASE_BF16, bool OUT_BF16, bool SWIGLU, int GROUPS>
__global__ void __launch_bounds__(kExpandThreads* GROUPS, GROUPS > 1 ? 1 : BASE_BF16 ? 4 : 3)
    lora_expand_tc_kernel(LoraParams p, LoraPlan pl) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t done;
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int RP = rank_pad(p.R);
  const int vblocks = (TERMS * RP + 63) / 64, bblocks = (RP + 63) / 64;
  constexpr int kThreads = kExpandThreads * GROUPS;
  constexpr int kBBytes = GROUPS * kExpandCols * 128;  // the unit's rows of B x 128 bytes
  unsigned char* vs = smem;
  unsigned char* bs = smem + vblocks * kBlockBytes;  // two slots of bblocks
  if (tid == 0) {
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  const uint32_t idesc = idesc_bf16(128, GROUPS * kExpandCols);
  const int cols = SWIGLU ? p.N / 2 : p.N;                       // output columns
  constexpr int gspan = SWIGLU ? kExpandCols / 2 : kExpandCols;  // of them a group's in a large unit
  constexpr int span = GROUPS * gspan;                           // and the unit's
  constexpr int sspan = kThreads;                                // a small unit's, 32 per warp
  const int group = warp / 4;
  const int chunks = (cols + span - 1) / span, schunks = (cols + sspan - 1) / sspan;

  // B rows of the unit at (tile slot, col0) -> slot `s` of shared memory: a
  // thread takes every second 16-byte piece of one row
  const int brow = (tid >> 1) & 63, bh = brow >> 5, bw = brow & 31;
  const int bdst = group * 64 + bh * 32 + 8 * ((bw & 7) >> 1) + 2 * (bw >> 3) + (bw & 1);
  auto load_b = [&](int slot_id, int col0, int s) {
    col0 += group * gspan;
    if (slot_id < 0 || (GROUPS > 1 && col0 >= cols)) return;
    const int n = SWIGLU ? bh * cols + col0 + bw : col0 + brow;
    unsigned char* dst = bs + s * bblocks * kBBytes;
    const uint16_t* src = p.b + ((int64_t)slot_id * p.N + n) * p.R;
    for (int ch = tid & 1; ch < RP / 8; ch += 2) {
      const bool on = ch * 8 < p.R;
      cp_async16(dst + (ch >> 3) * kBBytes + sw128_offset(bdst, ch & 7), on ? src + ch * 8 : p.b, on);
    }
  };

  // The plan was complete before the kernel just before this one (the shrink)
  // let it start: its first tile and that tile's rows of B need no wait.
  const int2 ntiles = lora_tiles(pl);
  // every CTA gets its share of the large units and of the small ones, which
  // take about as long for a fraction of the bytes
  const int64_t large = (int64_t)ntiles.x * chunks, small = (int64_t)ntiles.y * schunks;
  const int64_t u0 = large * blockIdx.x / gridDim.x, lend = large * (blockIdx.x + 1) / gridDim.x;
  int ti = (int)(u0 / chunks), col0 = (int)(u0 % chunks) * span;  // the unit, step by step
  int4 tile = make_int4(-1, 0, 0, 0);
  if (u0 < lend) {
    tile = __ldcg(pl.tiles + ti);
    load_b(tile.x, col0, 0);
  }
  cp_async_commit();
  pdl_wait();
  if (warp == 0) {
    tmem_alloc(&tmem_sh, GROUPS * kExpandCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = tmem_sh;

  int bad = 0, slot = 0;
  bool fresh = true;  // the unit is the first of its tile here
  int64_t row_at[4] = {};  // this lane's four rows (-1: none)
  Base8<BASE_BF16> bq[2][4];
  uint32_t parity = 0;
  auto load_base = [&](int i, int col0) {
    col0 += group * gspan;
    const bool on = p.base && row_at[i] >= 0 && (GROUPS == 1 || col0 < cols);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = (SWIGLU ? h * cols + col0 : col0 + h * 32) + 8 * t;
      if (on) bq[h][i].load(p.base, row_at[i] * p.N + col);
      else bq[h][i].zero();
    }
  };
  for (int64_t u = u0; u < lend; ++u) {
    const int gcol = col0 + group * gspan;
    if (fresh) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (warp & 3) * 32 + g + 8 * i;
        row_at[i] = r < tile.z ? (int64_t)pl.rows[tile.y + r].x : -1;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) load_base(i, col0);
      if (tile.x >= 0) stage_v<TERMS, kThreads>(pl, RP, tile.y, tile.z, tile.z, vs);
      cp_async_commit();
    }
    const bool last = u + 1 >= lend, more = !last && col0 + span < cols;  // more: of this tile
    int4 next = tile;
    if (!last) {
      if (!more) next = pl.tiles[ti + 1];
      load_b(next.x, more ? col0 + span : 0, slot ^ 1);
    }
    cp_async_commit();
    cp_async_wait<1>();
    fence_proxy_async_smem();
    if (__syncthreads_or(bad)) break;
    if (tile.x >= 0) {
      if (warp == 0) {
        for (int x = TERMS - 1; x >= 0; --x)  // the small terms first
          for (int j = 0; j < RP; j += 16) {
            const int col = x * RP + j;
            const uint64_t ad = smem_desc_sw128(vs + (col >> 6) * kBlockBytes) + ((col & 63) >> 3);
            const uint64_t bd =
                smem_desc_sw128(bs + (slot * bblocks + (j >> 6)) * kBBytes) + ((j & 63) >> 3);
            umma_bf16(tmem, ad, bd, idesc, x < TERMS - 1 || j > 0);
          }
        umma_commit(&done);
      }
      wait_or_flag(&done, parity, bad, p.err);
      parity ^= 1u;
      tc_fence_after();
    }
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {  // accumulator rows 32 (warp % 4) + 16 hr ..
      float z[2][2][8];               // [block][row g, g + 8]
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[16];
        if (tile.x >= 0) {
          tmem_ld_16x256b_x4(
              tmem + ((uint32_t)((warp & 3) * 32 + 16 * hr) << 16) + group * kExpandCols + h * 32, r);
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
      if (more) {
        load_base(2 * hr, col0 + span);
        load_base(2 * hr + 1, col0 + span);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = row_at[2 * hr + i];
        if (row < 0 || (GROUPS > 1 && gcol >= cols)) continue;
        if constexpr (SWIGLU) {
#pragma unroll
          for (int x = 0; x < 8; ++x) z[0][i][x] = swiglu_f32(z[0][i][x], z[1][i][x]);
          put8<OUT_BF16>(p.out, row * cols + gcol + 8 * t, z[0][i]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            put8<OUT_BF16>(p.out, row * cols + gcol + h * 32 + 8 * t, z[h][i]);
        }
      }
    }
    slot ^= 1;
    fresh = !more;
    col0 = more ? col0 + span : 0;
    ti += more ? 0 : 1;
    tile = next;
    tc_fence_before();
    __syncthreads();  // the accumulator, v and the old slot of B are free again
    tc_fence_after();
  }
  cp_async_wait<0>();
  const bool stop = __syncthreads_or(bad) != 0;

  constexpr int H = SWIGLU ? 2 : 1;
  const int64_t s0 = small * blockIdx.x / gridDim.x, s1 = small * (blockIdx.x + 1) / gridDim.x;
  ti = (int)(s0 / schunks);
  int chunk = (int)(s0 % schunks);
  fresh = true;
  for (int64_t u = s0; u < s1 && !stop; ++u, ++chunk) {
    if (chunk == schunks) {
      chunk = 0;
      ++ti;
      fresh = true;
    }
    const int col = chunk * sspan + warp * 32;
    const bool stage = fresh;
    fresh = false;
    if (stage) {
      tile = pl.tiles[pl.capacity - 1 - ti];
      __syncthreads();  // no warp still reads the tile before
      stage_v<TERMS, kThreads>(pl, RP, tile.y, tile.z, kLoraSmallRows, vs);
      cp_async_commit();
      row_at[0] = g < tile.z ? (int64_t)pl.rows[tile.y + g].x : -1;
      row_at[1] = g + 8 < tile.z ? (int64_t)pl.rows[tile.y + g + 8].x : -1;
    }
    const bool on = col < cols;  // the warp's 32 columns exist
    SmallB sb[H];
    Base8<BASE_BF16> b[H][2];
    const uint16_t* b0[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      b0[h] = p.b + ((int64_t)tile.x * p.N + h * cols + col + 8 * (g >> 1) + (g & 1)) * p.R + 4 * t;
      if (on) {
        sb[h].load(b0[h], p.R);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (p.base && row_at[i] >= 0)
            b[h][i].load(p.base, row_at[i] * p.N + h * cols + col + 8 * t);
          else
            b[h][i].zero();
        }
      }
    }
    if (stage) {
      cp_async_wait<0>();
      __syncthreads();
    }
    if (!on) continue;
    float z[H][2][8];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float acc[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
      small_block<TERMS>(acc, sb[h], b0[h], p.R, vs);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[h][i].get(z[h][i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          z[h][i][2 * q] += acc[q][2 * i];
          z[h][i][2 * q + 1] += acc[q][2 * i + 1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (row_at[i] < 0) continue;
      if constexpr (SWIGLU) {
#pragma unroll
        for (int x = 0; x < 8; ++x) z[0][i][x] = swiglu_f32(z[0][i][x], z[H - 1][i][x]);
      }
      put8<OUT_BF16>(p.out, row_at[i] * cols + col + 8 * t, z[0][i]);
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, GROUPS * kExpandCols);
}

// Shared memory of a CTA, and how many of them an SM holds.
size_t expand_smem(int terms, int RP, int groups) {
  return ((terms * RP + 63) / 64) * (size_t)kBlockBytes +
         2 * ((RP + 63) / 64) * (size_t)(groups * kExpandCols * 128) + 1024;
}
int expand_per_sm(size_t smem, int most) {
  const int n = (int)(224 * 1024 / (smem + 1024));
  return n < 1 ? 1 : n > most ? most : n;
}

template <int TERMS, bool BASE_BF16, bool OUT_BF16, bool SWIGLU, int GROUPS>
moe_status_t launch_expand_groups(const LoraParams& p, const LoraPlan& plan, cudaStream_t st) {
  using namespace moe_host;
  const size_t smem = expand_smem(TERMS, rank_pad(p.R), GROUPS);
  constexpr auto kern = lora_expand_tc_kernel<TERMS, BASE_BF16, OUT_BF16, SWIGLU, GROUPS>;
  const moe_status_t s = allow_smem<kern>(expand_smem(TERMS, kMaxRank, GROUPS));
  if (s != MOE_OK) return s;
  const int per_sm = expand_per_sm(smem, GROUPS > 1 ? 1 : BASE_BF16 ? 4 : 3);
  const int cols = SWIGLU ? p.N / 2 : p.N;
  const int span = GROUPS * (SWIGLU ? kExpandCols / 2 : kExpandCols);
  int64_t grid = plan.capacity * ((cols + span - 1) / span);
  if (grid > (int64_t)sm_count() * per_sm) grid = (int64_t)sm_count() * per_sm;
  return launch(kern, (int)grid, kExpandThreads * GROUPS, smem, st, p, plan);
}

// v of a wide rank leaves room for one CTA per SM; two groups of warps then
// share it.  4096 rows, rank 128, 4096 -> 4096, fp32: 78 us for the call, 86
// with one group.
template <int TERMS, bool BASE_BF16, bool OUT_BF16, bool SWIGLU>
moe_status_t launch_expand(const LoraParams& p, const LoraPlan& plan, cudaStream_t st) {
  if constexpr (TERMS > 2)
    if (expand_per_sm(expand_smem(TERMS, rank_pad(p.R), 1), 2) == 1)
      return launch_expand_groups<TERMS, BASE_BF16, OUT_BF16, SWIGLU, 2>(p, plan, st);
  return launch_expand_groups<TERMS, BASE_BF16, OUT_BF16, SWIGLU, 1>(p, plan, st);
}

template <int NT>
moe_status_t launch_shrink(const LoraParams& p, const LoraPlan& plan, int terms, cudaStream_t st) {
  using namespace moe_host;
  constexpr int kStages = shrink_stages(NT);
  const int RP = rank_pad(p.R);
  const size_t smem = (size_t)kStages * (kBlockBytes + RP * 128) + 1024;
  // the least padded rank of this instantiation, and what lies over its stages
  constexpr int least = NT == 2 ? 16 : rank_pad(NT * 4 + 8);
  static_assert(kLoraSmallRows * (NT * 8 + 4) * 4 + kShrinkWarps * kLoraSmallRows * NT * 8 * 4 <=
                    kStages * (kBlockBytes + least * 128), "the small tiles' sums fit");
  static_assert(kLoraTileRows * (NT * 8 + 4) * 4 <= kStages * (kBlockBytes + least * 128),
                "a tile's sums fit");
  const moe_status_t s = allow_smem<lora_shrink_tc_kernel<NT>>(
      (size_t)kStages * (kBlockBytes + NT * 8 * 128) + 1024);
  if (s != MOE_OK) return s;
  uint32_t tmem_cols = 32;
  while ((int)tmem_cols < RP) tmem_cols <<= 1;
  constexpr int per_sm = 2;
  int64_t clusters = (int64_t)sm_count() * per_sm / plan.splits;
  if (clusters > plan.capacity) clusters = plan.capacity;
  return moe_host::launch_clusters(lora_shrink_tc_kernel<NT>, dim3((unsigned)(clusters * plan.splits)),
                         kShrinkThreads, smem, dim3(plan.splits), st, p, plan, terms, tmem_cols);
}

}  // namespace

moe_status_t lora_grouped(const LoraParams& p, const LoraPlan& plan, int64_t rows, bool swiglu,
                          bool out_bf16, cudaStream_t st) {
  using namespace moe_host;
  // with several experts their CTAs add to the counts
  if (p.E > 1 && cudaMemsetAsync(plan.counts, 0, sizeof(int4), st) != cudaSuccess)
    return MOE_ERR_CUDA;
  auto plan_bytes = [](int adapters) {
    return (size_t)(4 + kPlanWarps) * (adapters + 1) * sizeof(int);
  };
  moe_status_t s = allow_smem<lora_plan_kernel>(plan_bytes(kLoraPlanAdapters));
  if (s != MOE_OK) return s;
  // CTAs per expert: one per 1024 of the rows that an expert has on average
  int ranges = 1;
  while (ranges < kPlanRanges && (int64_t)ranges * 1024 * p.E < rows) ranges *= 2;
  s = moe_host::launch_clusters(lora_plan_kernel, dim3(p.E, ranges), kPlanThreads,
                                plan_bytes(p.n_adapters), dim3(1, ranges), st, p, plan);
  if (s != MOE_OK) return s;
  const int terms = out_bf16 && !swiglu ? 2 : 3;
  if (p.R <= 16) s = launch_shrink<2>(p, plan, terms, st);
  else if (p.R <= 32) s = launch_shrink<4>(p, plan, terms, st);
  else if (p.R <= 64) s = launch_shrink<8>(p, plan, terms, st);
  else s = launch_shrink<16>(p, plan, terms, st);
  if (s != MOE_OK) return s;
  if (swiglu)
    return out_bf16 ? launch_expand<3, false, true, true>(p, plan, st)
                    : launch_expand<3, false, false, true>(p, plan, st);
  return out_bf16 ? launch_expand<2, true, true, false>(p, plan, st)
                  : launch_expand<3, false, false, false>(p, plan, st);
}

}  // namespace moe
