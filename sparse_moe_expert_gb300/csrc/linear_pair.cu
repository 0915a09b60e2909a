// The dense product for many rows: pairs of CTAs on 256 x BN tiles.
//
// Two SMs of a cluster share one tile (tcgen05 cta_group::2): each holds 128 rows
// of A, half of B's rows and the sums of its own rows, and the even CTA issues
// the products for both, so a byte of B read from L2 serves 256 rows.  With one
// CTA per 128 x 128 tile (linear.cu) each SM would have to take in 32 KB per 64 k
// and 256 cycles; the pair takes 32 KB per 512 cycles.  Persistent: one warp
// loads (TMA, a ring of k-blocks of 64), one issues the products (a single lane
// each), eight take the sums of the tile before out of the second half of TMEM
// meanwhile.  Tiles run through A's rows eight tiles at a time, so that a wave of
// pairs meets in L2.  Bound by the tensor cores: 8192^3 565 us, 1.95 PFLOP/s; the
// gradient's two products at 4096 x 4096 x 11008 394 us, 96 % of them busy; 3001 x
// 11008 x 4096 with GELU and residual 162 us, 84 % (143 at the peak rate; 2 % of the
// tiles' rows are empty).
//
// A launch takes one product or two, one after the other: of the gradient's two,
// neither fills its last wave (256 and 688 tiles on 76 pairs: 4 and 10 turns for 3.4
// and 9.1), and the pairs that the first leaves early begin with the second.
#include <cstring>

#include "linear.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kPairThreads = 320;
constexpr int kPairEpiWarps = 8;
constexpr int kPairM = 256;
constexpr int kPairGroup = 8;  // row tiles that are walked together
constexpr int kPairTmem = 512;

constexpr int kPairN = 256;    // widest tile
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = (128 + kPairN / 2) * 128;
constexpr int kPairStrip = 32 * 128;  // an epilogue warp's: 32 rows x 128 bytes
constexpr size_t kPairRing = (size_t)kPairStages * kPairStageBytes;
constexpr size_t kPairSmem = kPairRing + kPairEpiWarps * kPairStrip + 1024;

// As linear_tma_2d, on a barrier of either CTA of the pair (`bar` as the
// cluster has it).
__device__ __forceinline__ void pair_tma_2d(void* dst, const CUtensorMap* tm, int c0, int c1,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// By one thread of the even CTA, for the pair.
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on this barrier of both CTAs once the products this thread issued are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One product of a launch.
struct PairProduct {
  CUtensorMap a, b;
  LinearEpi e;
  int K, bn;
  int m_tiles, n_tiles;
  int tiles;   // 0: no such product
};
// The tiles are dealt to the pairs in turns.  Of the first product the `heavy` first
// pairs have one tile more; the others begin the second with `extra` turns of
// their own, then it is dealt to all.
struct PairWork {
  PairProduct product[2];
  int heavy, extra;
  int rows_first;  // which of two has its A in rows
};
struct PairTile {
  int which;  // -1: none left
  int m, n;
};

template <bool TWO>
__device__ __forceinline__ PairTile pair_tile(const PairWork& w, int pair, int pairs, int i) {
  int t = pair + i * pairs, which = 0;
  if (TWO && t >= w.product[0].tiles) {
    const int first = w.product[0].tiles;
    i -= pair < first ? (first - pair + pairs - 1) / pairs : 0;
    const int light = pairs - w.heavy;
    if (pair >= w.heavy && i < w.extra) {
      t = pair - w.heavy + i * light;
    } else {
      if (pair >= w.heavy) i -= w.extra;
      t = w.extra * light + pair + i * pairs;
    }
    which = 1;
  }
  const PairProduct& q = w.product[which];
  if (t >= q.tiles) return {-1, 0, 0};
  const int per = kPairGroup * q.n_tiles, g = t / per, r = t - g * per;
  const int rows = min(kPairGroup, q.m_tiles - g * kPairGroup);
  return {which, g * kPairGroup + r % rows, r / rows};
}

// ---- the epilogue of rows of whole 16-byte pieces --------------------------------

// The residual of a row's 32 columns, asked for ahead.
struct Residual32 {
  uint4 q[8];  // bf16: the first four
  __device__ __forceinline__ void ask(const LinearEpi& e, int64_t row, int col, int n) {
    if (row >= e.M) return;
    const int64_t at = row * e.cols + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e.out_bf16) {
        if (i < 4 && i * 8 < n)
          q[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.residual) + at + i * 8);
      } else if (i * 4 < n) {
        q[i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(e.residual) + at + i * 4);
      }
    }
  }
};

// A warp's strip of 32 rows x 128 bytes in shared memory: piece p (16 bytes) of row r lies
// at p ^ (r & 7), without bank conflicts.
__device__ __forceinline__ unsigned char* strip_at(unsigned char* strip, int row, int piece) {
  return strip + row * 128 + ((piece ^ (row & 7)) << 4);
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void strip_hold(unsigned char* strip, const uint32_t (&r)[2][16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<uint4*>(strip_at(strip, lane, q)) =
        make_uint4(r[q >> 2][(q & 3) * 4], r[q >> 2][(q & 3) * 4 + 1], r[q >> 2][(q & 3) * 4 + 2],
                   r[q >> 2][(q & 3) * 4 + 3]);
}

// SwiGLU's 32 columns of a row, of which `left` are there: a lane has both halves and
// stores its row itself (4096 x 2048 x 1536 19.7 us, through the strip 20.3).
__device__ __forceinline__ void gated_finish(const LinearEpi& e, int64_t row, int col, int left,
                                             const uint32_t (&r)[4][16], const Residual32& res) {
  float z[32], u[32];
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    z[x] = __uint_as_float(r[x >> 4][x & 15]);
    u[x] = __uint_as_float(r[2 + (x >> 4)][x & 15]);
  }
  if (e.bias) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (4 * q >= left) continue;
      const float4 b = *reinterpret_cast<const float4*>(e.bias + col + 4 * q);
      const float4 d = *reinterpret_cast<const float4*>(e.bias + e.cols + col + 4 * q);
      z[4 * q] += b.x;
      z[4 * q + 1] += b.y;
      z[4 * q + 2] += b.z;
      z[4 * q + 3] += b.w;
      u[4 * q] += d.x;
      u[4 * q + 1] += d.y;
      u[4 * q + 2] += d.z;
      u[4 * q + 3] += d.w;
    }
  }
  if (e.preact) {
    uint16_t* p = e.preact + row * e.N + col;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (8 * q >= left) continue;
      store_bf16x8(p + 8 * q, z + 8 * q);
      store_bf16x8(p + e.cols + 8 * q, u + 8 * q);
    }
  }
#pragma unroll
  for (int x = 0; x < 32; ++x) z[x] = swiglu_f32(z[x], u[x]);
  if (!e.out_bf16) {
    float* p = static_cast<float*>(e.out) + row * e.cols + col;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (4 * q >= left) continue;
      float4 f = make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
      if (e.residual) {
        f.x += __uint_as_float(res.q[q].x);
        f.y += __uint_as_float(res.q[q].y);
        f.z += __uint_as_float(res.q[q].z);
        f.w += __uint_as_float(res.q[q].w);
      }
      *reinterpret_cast<float4*>(p + 4 * q) = f;
    }
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(e.out) + row * e.cols + col;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (8 * q >= left) continue;
    if (e.residual) {
      const uint32_t w[4] = {res.q[q].x, res.q[q].y, res.q[q].z, res.q[q].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = bf16x2_to_f32x2(w[x]);
        z[8 * q + 2 * x] += f.x;
        z[8 * q + 2 * x + 1] += f.y;
      }
    }
    store_bf16x8(p + 8 * q, z + 8 * q);
  }
}

// What four columns of a row are added to, asked for ahead: eight lanes take a row, a lane
// the rows lane / 8 + 4 i, in two halves of four.
struct StripAdd {
  float4 bias;
  uint4 residual[4];  // of the half to come; bf16: two words of each
  // `n` columns and `rows` rows are there
  __device__ __forceinline__ void ask_bias(const LinearEpi& e, int64_t col, int n) {
    const int c = (threadIdx.x & 7) * 4;
    bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (e.bias && c < n) bias = *reinterpret_cast<const float4*>(e.bias + col + c);
  }
  __device__ __forceinline__ void ask(int h, const LinearEpi& e, int64_t row0, int rows, int64_t col, int n) {
    const int lane = threadIdx.x & 31, c = (lane & 7) * 4;
    if (!e.residual || c >= n) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (h * 4 + i) * 4 + (lane >> 3);
      const int64_t at = (row0 + r) * e.cols + col + c;
      if (r >= rows) continue;
      if (e.out_bf16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.residual) + at);
        residual[i].x = v.x;
        residual[i].y = v.y;
      } else {
        residual[i] = *reinterpret_cast<const uint4*>(static_cast<const float*>(e.residual) + at);
      }
    }
  }
};

// The sums of 32 rows x 32 columns in the warp's strip -> columns col .. col + n of the
// outputs.  Rows leave as whole 64 or 128 bytes; four of them are read before the first is
// stored, so that their chains run side by side.  Against lanes that finish and store their
// own rows, 16 bytes at a time (us, 3001 x 4096 sums over 256, then d_w and both gradients
// of 512 x 4096 x 4096 in fp32): bias 19.1, 17.6; GELU, bias and residual 46.6, 29.6; fp32
// 22.2, 17.6; fp32 with residual 35.3, 30.3; d_w 35.1, 25.7; both 50.5, 37.3; bf16 SiLU
// alone loses, 17.7, 21.8 (with all eight rows at once, or their residuals, registers spill: 65, 91).
template <int ACT, bool OUT_BF16>
__device__ __forceinline__ void strip_rows(const LinearEpi& e, unsigned char* strip, int64_t row0, int rows,
                                           int64_t col, int n, StripAdd& add) {
  const int lane = threadIdx.x & 31, c = (lane & 7) * 4;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const uint4 present[4] = {add.residual[0], add.residual[1], add.residual[2], add.residual[3]};
    if (h == 0) add.ask(1, e, row0, rows, col, n);
    if (c >= n) continue;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const float4*>(strip_at(strip, (h * 4 + i) * 4 + (lane >> 3), lane & 7));
    const int64_t first = row0 + h * 16 + (lane >> 3);
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = h * 16 + i * 4 + (lane >> 3) < rows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x += add.bias.x;
      v[i].y += add.bias.y;
      v[i].z += add.bias.z;
      v[i].w += add.bias.w;
    }
    if (e.preact) {
      uint16_t* p = e.preact + first * e.N + col + c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (on[i])
          *reinterpret_cast<uint2*>(p + i * 4 * (int64_t)e.N) =
              make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ACT == MOE_ACT_SILU) {
        v[i] = make_float4(silu_f32(v[i].x), silu_f32(v[i].y), silu_f32(v[i].z), silu_f32(v[i].w));
      } else if constexpr (ACT == MOE_ACT_GELU) {
        gelu2(v[i].x, v[i].y);
        gelu2(v[i].z, v[i].w);
      }
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q = present[i];
        const float2 lo = OUT_BF16 ? bf16x2_to_f32x2(q.x) : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        const float2 hi = OUT_BF16 ? bf16x2_to_f32x2(q.y) : make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
        v[i].x += lo.x;
        v[i].y += lo.y;
        v[i].z += hi.x;
        v[i].w += hi.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!on[i]) continue;
      const int64_t at = (first + i * 4) * e.cols + col + c;
      if constexpr (OUT_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.out) + at) =
            make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(e.out) + at) = v[i];
    }
  }
}

__device__ __forceinline__ void strip_wide(const LinearEpi& e, unsigned char* strip, int64_t row0, int rows,
                                           int64_t col, int n, StripAdd& add) {
  if (e.act == MOE_ACT_GELU) {
    if (e.out_bf16) strip_rows<MOE_ACT_GELU, true>(e, strip, row0, rows, col, n, add);
    else strip_rows<MOE_ACT_GELU, false>(e, strip, row0, rows, col, n, add);
  } else if (e.act == MOE_ACT_SILU) {
    if (e.out_bf16) strip_rows<MOE_ACT_SILU, true>(e, strip, row0, rows, col, n, add);
    else strip_rows<MOE_ACT_SILU, false>(e, strip, row0, rows, col, n, add);
  } else {
    if (e.out_bf16) strip_rows<MOE_ACT_NONE, true>(e, strip, row0, rows, col, n, add);
    else strip_rows<MOE_ACT_NONE, false>(e, strip, row0, rows, col, n, add);
  }
}

// ---- the epilogue of rows off their 16-byte boundary ----------------------------
//
// A lane's sums are a row of the tile.  Stored from there, single values would go to as
// many lines as there are lanes, so a strip of 32 rows x 128 bytes goes through shared
// memory and neighbouring lanes take neighbouring columns (335 x 408 x 3468, us: 20.0
// without, 12.3).  Rows of whole 16-byte pieces have a strip of their own above; bf16 sums
// as they are and SwiGLU's leave from the lanes.

// The strip -> `n` columns at `col` of the warp's rows (of which `rows` are there)
// of a matrix with rows of `ld` elements, plus what `residual` has there.  By the
// warp together.
template <bool BF16>
__device__ __forceinline__ void strip_store(unsigned char* strip, void* p, const void* residual,
                                            int64_t row0, int rows, int64_t ld, int64_t col, int n) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
    for (int c = lane; c < n; c += 32) {
      const int64_t at = (row0 + r) * ld + col + c;
      float f = *reinterpret_cast<float*>(strip_at(strip, r, c / 4) + (c % 4) * 4);
      if constexpr (BF16) {
        if (residual) f += bf16_bits_to_f32(static_cast<const uint16_t*>(residual)[at]);
        static_cast<uint16_t*>(p)[at] = f32_to_bf16_rne(f);
      } else {
        if (residual) f += static_cast<const float*>(residual)[at];
        static_cast<float*>(p)[at] = f;
      }
    }
  __syncwarp();
}

// Sixteen of a row's sums with their bias; columns past `left` get any.
__device__ __forceinline__ void strip_sums(float (&z)[16], uint32_t tmem, const float* bias, int left) {
  uint32_t r[16];
  tmem_ld16(tmem, r);
  tmem_ld_wait();
#pragma unroll
  for (int x = 0; x < 16; ++x) z[x] = __uint_as_float(r[x]) + (bias && x < left ? bias[x] : 0.0f);
}

// 32 columns of the tile, from accumulator column `tmem` on, to column `col` of the
// outputs; `done` is called when nothing reads the sums any more, if `last`.
template <bool SWIGLU, typename F>
__device__ __forceinline__ void strip_finish(const LinearEpi& e, unsigned char* strip, uint32_t tmem, int up,
                                             int64_t row0, int rows, int col, int n, bool last, F&& done) {
  const int lane = threadIdx.x & 31;
  auto hold = [&](int c, const float (&z)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(strip_at(strip, lane, c / 4 + q)) =
          make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
  };
  if (e.preact) {
#pragma unroll 1
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
#pragma unroll 1
      for (int c = 0; c < n; c += 16) {
        float z[16];
        strip_sums(z, tmem + h * up + c, e.bias ? e.bias + h * e.cols + col + c : nullptr, n - c);
        hold(c, z);
      }
      __syncwarp();
      strip_store<true>(strip, e.preact, nullptr, row0, rows, e.N, h * e.cols + col, n);
    }
  }
#pragma unroll 1
  for (int c = 0; c < n; c += 16) {
    float z[16];
    strip_sums(z, tmem + c, e.bias ? e.bias + col + c : nullptr, n - c);
    if constexpr (SWIGLU) {
      float u[16];
      strip_sums(u, tmem + up + c, e.bias ? e.bias + e.cols + col + c : nullptr, n - c);
#pragma unroll
      for (int x = 0; x < 16; ++x) z[x] = swiglu_f32(z[x], u[x]);
    } else if (e.act == MOE_ACT_SILU) {
#pragma unroll
      for (int x = 0; x < 16; ++x) z[x] = silu_f32(z[x]);
    } else if (e.act == MOE_ACT_GELU) {
#pragma unroll
      for (int x = 0; x < 16; x += 2) gelu2(z[x], z[x + 1]);
    }
    hold(c, z);
  }
  if (last) done();
  __syncwarp();
  if (e.out_bf16) strip_store<true>(strip, e.out, e.residual, row0, rows, e.cols, col, n);
  else strip_store<false>(strip, e.out, e.residual, row0, rows, e.cols, col, n);
}

// A's order.  Of two products one has it in rows of k, the other by columns.
enum { kACols, kARows, kABoth };

template <int A_ORDER, bool B_ROW, bool SWIGLU>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairWork work, unsigned int* err) {
  constexpr int kStages = kPairStages, kStageBytes = kPairStageBytes;
  constexpr bool kTwo = A_ORDER == kABoth;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], sums_full[2], sums_empty[2], drain;
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sums_full[b], 1);
      mbar_init(&sums_empty[b], 2 * kPairEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_sh)),
                 "r"(kPairTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // the other CTA's barriers are there as well
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tmem_sh;
  // One lane of a warp runs each of the first two roles: with all lanes at the
  // barriers the loops took some 600 cycles per block of k, more than its products.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity, kWaitBudgetCycles)) return true;
    raise_device_error(err, MOE_DEVERR_TIMEOUT);
    return false;
  };
  if (warp == 0) {
    if (elected()) {
      int s = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      const uint32_t bar0 = cluster_addr(full, 0);  // the even CTA's
      for (int i = 0; ok; ++i) {
        const PairTile at = pair_tile<kTwo>(work, pair, pairs, i);
        if (at.which < 0) break;
        const PairProduct& q = work.product[kTwo ? at.which : 0];
        const int bn = q.bn, nkb = (q.K + kLinBK - 1) / kLinBK;
        const bool a_rows = kTwo ? at.which == work.rows_first : A_ORDER == kARows;
        const CUtensorMap *tm_a = &q.a, *tm_b = &q.b;
        const uint32_t bytes = (uint32_t)(256 + bn) * 128;
        const int row0 = at.m * kPairM + cta * 128;
        const int col0 = SWIGLU ? cta * q.e.cols + at.n * (bn / 2) : at.n * bn + cta * (bn / 2);
        for (int kb = 0; kb < nkb; ++kb) {
          if (issued >= kStages && !(ok = wait(&empty[s], phase ^ 1u))) break;
          unsigned char* a = smem + s * kStageBytes;
          unsigned char* b = a + 128 * 128;
          const uint32_t bar = bar0 + s * 8;
          const int k = kb * kLinBK;
          if (cta == 0) mbar_arrive_expect_tx(&full[s], bytes);
          if (a_rows) {
            pair_tma_2d(a, tm_a, k, row0, bar);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) pair_tma_2d(a + j * 8192, tm_a, row0 + j * 64, k, bar);
          }
          if constexpr (B_ROW) {
            pair_tma_2d(b, tm_b, k, col0, bar);
          } else {
            for (int j = 0; j < bn / 128; ++j) pair_tma_2d(b + j * 8192, tm_b, col0 + j * 64, k, bar);
          }
          ++issued;
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && cta == 0) {  // copies in flight end before the pair may
        const int64_t first = issued > kStages ? issued - kStages : 0;
        for (int64_t i = first; i < issued; ++i)
          mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, kWaitBudgetCycles);
      }
    }
  } else if (warp == 1) {
    if (cta == 0 && elected()) {
      const uint64_t a_rows = operand_desc<true>(smem), a_cols = operand_desc<false>(smem);
      const uint64_t b_desc = operand_desc<B_ROW>(smem + 128 * 128);
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const PairTile at = pair_tile<kTwo>(work, pair, pairs, i);
        if (at.which < 0) break;
        const PairProduct& q = work.product[kTwo ? at.which : 0];
        const int nkb = (q.K + kLinBK - 1) / kLinBK, buf = i & 1;
        const bool rows = kTwo ? at.which == work.rows_first : A_ORDER == kARows;
        const uint32_t idesc = (rows ? idesc_linear<true, B_ROW>(kPairM, 0)
                                     : idesc_linear<false, B_ROW>(kPairM, 0)) |
                               ((uint32_t)(q.bn >> 3) << 17);
        const uint64_t a0 = rows ? a_rows : a_cols;
        const uint64_t a_step = rows ? operand_step<true>() : operand_step<false>();
        if (i >= 2 && !(ok = wait(&sums_empty[buf], (uint32_t)((i >> 1) - 1) & 1u))) break;
        const uint32_t d = tmem + buf * kPairN;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!(ok = wait(&full[s], phase))) break;
          tc_fence_after();
          const uint64_t ad = a0 + s * (kStageBytes >> 4), bd = b_desc + s * (kStageBytes >> 4);
          pair_mma(d, ad, bd, idesc, kb > 0);
#pragma unroll
          for (int k = 1; k < 4; ++k)
            pair_mma(d, ad + k * a_step, bd + k * operand_step<B_ROW>(), idesc, 1);
          pair_commit(&empty[s]);
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) pair_commit(&sums_full[buf]);
      }
      if (!ok) {  // products in flight end before the pair may
        pair_commit(&drain);
        mbar_wait(&drain, 0u, kWaitBudgetCycles);
      }
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    unsigned char* strip = smem + kPairRing + (warp - 2) * kPairStrip;
    for (int i = 0;; ++i) {
      const PairTile at = pair_tile<kTwo>(work, pair, pairs, i);
      if (at.which < 0) break;
      const LinearEpi e = work.product[kTwo ? at.which : 0].e;  // in registers
      const int bn = work.product[kTwo ? at.which : 0].bn, buf = i & 1;
      const int span = SWIGLU ? bn / 2 : bn;  // output columns of the tile
      const int64_t row = (int64_t)at.m * kPairM + cta * 128 + quad * 32 + lane;
      // the residual's part of the tile comes into L2 during the products
      if (e.residual && row < e.M) {
        const int size = e.out_bf16 ? 2 : 4;
        const int c1 = min(span, e.cols - at.n * span) * size;
        const char* p = static_cast<const char*>(e.residual) + (row * e.cols + (int64_t)at.n * span) * size;
        for (int c = half * 128; c < c1; c += 256) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
      }
      // a tile's products may take a while themselves: some 600 cycles per block of k
      const long long blocks = (work.product[kTwo ? at.which : 0].K + kLinBK - 1) / kLinBK;
      int ok = mbar_wait_sleep(&sums_full[buf], (uint32_t)(i >> 1) & 1u, kWaitBudgetCycles + blocks * 4096);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        raise_device_error(err, MOE_DEVERR_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t base = tmem + buf * kPairN + ((uint32_t)(quad * 32) << 16);
      auto done = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) remote_arrive(cluster_addr(&sums_empty[buf], 0));
      };
      const int64_t below = e.M - (row - lane);
      const int rows = below >= 32 ? 32 : below > 0 ? (int)below : 0;  // of this warp that are there
      const bool plain = !SWIGLU && e.out_bf16 && e.act == MOE_ACT_NONE && !e.bias && !e.residual && !e.preact;
      if (plain && e.vec) {
        uint16_t* out = static_cast<uint16_t*>(e.out) + row * e.cols + at.n * span;
        const int width = min(span, e.cols - at.n * span);
        bool left = false;
#pragma unroll 1
        for (int c = half * 32; c < span; c += 64) {
          uint32_t r[2][16];
          tmem_ld16(base + c, r[0]);
          tmem_ld16(base + c + 16, r[1]);
          tmem_ld_wait();
          if (c + 64 >= span) {
            done();
            left = true;
          }
          if (row >= e.M) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float f[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = __uint_as_float(r[q >> 1][(q & 1) * 8 + x]);
            if (c + q * 8 < width) store_bf16x8(out + c + q * 8, f);
          }
        }
        if (!left) done();
      } else if (e.vec) {
        const int width = min(span, e.cols - at.n * span);  // columns that are there
        bool left = false;
#pragma unroll 1
        for (int c = half * 32; c < span; c += 64) {
          Residual32 res;
          StripAdd add;
          if constexpr (SWIGLU) {
            if (e.residual) res.ask(e, row, at.n * span + c, width - c);
          } else {
            add.ask_bias(e, at.n * span + c, width - c);
            add.ask(0, e, row - lane, rows, at.n * span + c, width - c);
          }
          uint32_t r[SWIGLU ? 4 : 2][16];
          tmem_ld16(base + c, r[0]);
          tmem_ld16(base + c + 16, r[1]);
          if constexpr (SWIGLU) {
            tmem_ld16(base + span + c, r[2]);
            tmem_ld16(base + span + c + 16, r[3]);
          }
          tmem_ld_wait();
          if (c + 64 >= span) {  // the sums are in registers
            done();
            left = true;
          }
          if constexpr (SWIGLU) {
            if (lane < rows) gated_finish(e, row, at.n * span + c, width - c, r, res);
          } else {
            strip_hold(strip, r);
            __syncwarp();
            strip_wide(e, strip, row - lane, rows, at.n * span + c, width - c, add);
            __syncwarp();
          }
        }
        if (!left) done();  // no columns of this tile for this warp
      } else {
        const int64_t row0 = row - lane;
        const int width = min(span, e.cols - at.n * span);  // columns that are there
        bool left = false;
        for (int c = half * 32; c < width; c += 64) {
          const bool last = c + 64 >= width;
          left |= last;
          strip_finish<SWIGLU>(e, strip, base + c, span, row0, rows, at.n * span + c, min(32, width - c),
                               last, done);
        }
        if (!left) done();  // no columns of this tile for this warp
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPairTmem)
                 : "memory");
}

// Pairs that the current device holds at once.
template <auto Kernel>
int pairs_resident(size_t smem) {
  static std::atomic<int> known[moe_host::kMaxCachedDevices] = {};
  std::atomic<int>& mine = known[moe_host::device_index()];
  int n = mine.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (moe_host::sm_count() / 2));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = moe_host::sm_count() / 2;
    }
    mine.store(n, std::memory_order_relaxed);
  }
  return n;
}

// Columns of a tile: the width whose waves cost least.  A block of 64 k takes a
// time like bn + 217 (8192^3, ns per block at 256, 224, 192, 160, 128, 96: 322,
// 288, 266, 249, 228, 208), so a narrower tile pays where it fills the last wave:
// us at 256 and at the width taken, 3001 x 11008 x 4096 179, 163 (224), 4096 x 2048
// x 1536 SwiGLU 28.4, 23.6 (192), 4096^3 91, 83 (224).  A B by columns comes in
// blocks of 64 rows for each CTA.  SwiGLU's halves are multiples of 16, so their last
// chunk of 32 columns may read 16 of what lies behind them (the other half, or TMEM that
// no tile has); the epilogue's `width` keeps those from being stored.
struct PairChoice {
  int bn;
  int64_t waves;
};
PairChoice choose_pairs(const LinearEpi& e, int pairs, bool b_rows) {
  const int64_t m_tiles = (e.M + kPairM - 1) / kPairM;
  const int unit = e.act == MOE_ACT_SWIGLU ? 32 : b_rows ? 16 : 128;
  PairChoice best{0, 0};
  for (int bn = kPairN; bn >= 96; bn -= unit) {
    const int span = e.act == MOE_ACT_SWIGLU ? bn / 2 : bn;
    const int64_t waves = (m_tiles * ((e.cols + span - 1) / span) + pairs - 1) / pairs;
    if (!best.bn || waves * (bn + 217) < best.waves * (best.bn + 217)) best = {bn, waves};
  }
  return best;
}

// One product with tiles of this width; fails only if no map describes an operand.
bool set_product(PairProduct& q, const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e, int bn) {
  const int span = e.act == MOE_ACT_SWIGLU ? bn / 2 : bn;
  q.e = e;
  q.K = K;
  q.bn = bn;
  q.m_tiles = (e.M + kPairM - 1) / kPairM;
  q.n_tiles = (e.cols + span - 1) / span;
  q.tiles = q.m_tiles * q.n_tiles;
  return linear_map(&q.a, a, e.M, K, 128) && linear_map(&q.b, b, e.N, K, bn / 2);
}

bool too_many(const LinearEpi& e) {
  return (int64_t)((e.M + kPairM - 1) / kPairM) * ((e.cols + 47) / 48) > INT32_MAX / 4;
}

template <int A_ORDER, bool B_ROW, bool SWIGLU>
moe_status_t launch_pairs(const PairWork& w, int pairs, cudaStream_t st) {
  constexpr auto kern = linear_pair_kernel<A_ORDER, B_ROW, SWIGLU>;
  return moe_host::launch_clusters(kern, dim3(2 * pairs), kPairThreads, kPairSmem, dim3(2, 1, 1), st, w,
                                   moe_host::device_error_word());
}

template <int A_ORDER, bool B_ROW, bool SWIGLU>
moe_status_t one_product(const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e, cudaStream_t st) {
  constexpr auto kern = linear_pair_kernel<A_ORDER, B_ROW, SWIGLU>;
  if (too_many(e)) return MOE_ERR_INVALID_ARG;
  if (const moe_status_t s = moe_host::allow_smem<kern>(kPairSmem)) return s;
  const int most = pairs_resident<kern>(kPairSmem);
  PairWork w;
  memset(&w, 0, sizeof w);
  if (!set_product(w.product[0], a, b, K, e, choose_pairs(e, most, B_ROW).bn)) return MOE_ERR_CUDA;
  const int tiles = w.product[0].tiles;
  return launch_pairs<A_ORDER, B_ROW, SWIGLU>(w, tiles < most ? tiles : most, st);
}

float block_us(int K, int bn) { return (K + kLinBK - 1) / kLinBK * (bn + 217) * 0.5e-3f; }
int64_t tiles_at(const LinearEpi& e, int bn) {
  return (int64_t)((e.M + kPairM - 1) / kPairM) * ((e.cols + bn - 1) / bn);
}

// How two products are dealt: widths, the turns that the light pairs have for
// themselves, and the time, by the same estimate as for one.
struct BothChoice {
  int bn[2];
  int extra;
  float us;
};
BothChoice choose_both(const LinearEpi (&e)[2], const int (&K)[2], int pairs) {
  BothChoice best{{0, 0}, 0, 1e30f};
  for (int b0 = 128; b0 <= 256; b0 += 128)
    for (int b1 = 128; b1 <= 256; b1 += 128) {
      const int64_t t0 = tiles_at(e[0], b0), t1 = tiles_at(e[1], b1);
      const float c0 = block_us(K[0], b0) + 1.0f, c1 = block_us(K[1], b1) + 1.0f;
      const int64_t whole = t0 / pairs, heavy = t0 % pairs, light = pairs - heavy;
      for (int extra = 0; extra <= 64 && extra * light <= t1 && (extra == 0 || heavy); ++extra) {
        const int64_t rest = (t1 - extra * light + pairs - 1) / pairs;
        const float busy = (whole + 1) * c0 + rest * c1, idle = whole * c0 + (extra + rest) * c1;
        const float us = 3.9f + (heavy && busy > idle ? busy : idle);
        if (us < best.us) best = {{b0, b1}, extra, us};
      }
    }
  return best;
}

}  // namespace

// Fitted to the same measurements as the small tiles' estimate (linear.cu).
float linear_pairs_us(const LinearEpi& e, int K, bool b_rows) {
  const PairChoice c = choose_pairs(e, moe_host::sm_count() < 2 ? 1 : moe_host::sm_count() / 2, b_rows);
  const float waves = (float)c.waves;
  return 4.9f + waves * block_us(K, c.bn) + (waves - 1.0f);
}

moe_status_t linear_pairs(const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e,
                          cudaStream_t st) {
  if (e.act == MOE_ACT_SWIGLU) return one_product<kARows, true, true>(a, b, K, e, st);
  if (!a.row_major) return one_product<kACols, false, false>(a, b, K, e, st);
  return b.row_major ? one_product<kARows, true, false>(a, b, K, e, st)
                     : one_product<kARows, false, false>(a, b, K, e, st);
}

float linear_pairs_both_us(const LinearEpi (&e)[2], const int (&K)[2]) {
  return choose_both(e, K, moe_host::sm_count() < 2 ? 1 : moe_host::sm_count() / 2).us;
}

moe_status_t linear_pairs_both(const LinearOp (&a)[2], const LinearOp (&b)[2], const int (&K)[2],
                               const LinearEpi (&e)[2], cudaStream_t st) {
  constexpr auto kern = linear_pair_kernel<kABoth, false, false>;
  if (too_many(e[0]) || too_many(e[1])) return MOE_ERR_INVALID_ARG;
  if (const moe_status_t s = moe_host::allow_smem<kern>(kPairSmem)) return s;
  const int pairs = pairs_resident<kern>(kPairSmem);
  const BothChoice c = choose_both(e, K, pairs);
  PairWork w;
  memset(&w, 0, sizeof w);
  for (int i = 0; i < 2; ++i)
    if (!set_product(w.product[i], a[i], b[i], K[i], e[i], c.bn[i])) return MOE_ERR_CUDA;
  w.heavy = w.product[0].tiles % pairs;
  w.extra = c.extra;
  w.rows_first = a[0].row_major ? 0 : 1;
  return launch_pairs<kABoth, false, false>(w, pairs, st);
}

}  // namespace moe
