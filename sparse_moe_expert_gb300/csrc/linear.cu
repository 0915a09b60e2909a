// The dense product out = act(x W^T + bias) + residual on the tensor cores, and
// the products of its gradient, which are the same sums over other axes:
//   forward  D[t, n] = sum_k x[t, k] W[n, k]       both operands in rows of k
//   d_x      D[t, k] = sum_n d_z[t, n] W[n, k]     W by columns
//   d_w      D[n, k] = sum_t d_z[t, n] x[t, k]     both by columns
// tcgen05 takes either order from shared memory (the descriptors say which), so
// nothing is transposed.
#include "linear.cuh"

#include "lora.cuh"

namespace moe {

bool make_tensor_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                        uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                        CUtensorMapSwizzle sw);

bool linear_map(CUtensorMap* m, const LinearOp& op, int rows, int K, int box_rows) {
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  return op.row_major
             ? make_tensor_map_2d(m, bf16, op.p, K, rows, (uint64_t)op.ld * 2, kLinBK, box_rows, sw)
             : make_tensor_map_2d(m, bf16, op.p, rows, K, (uint64_t)op.ld * 2, 64, kLinBK, sw);
}

namespace {

// ---- one tile per CTA, K shared by a cluster -----------------------------------
//
// 128 x BN tiles.  A cluster of `splits` CTAs takes a tile, each CTA a run of K;
// the sums meet in shared memory and are added in rank order, each CTA a share
// of the rows.  64 x 1536 -> 4096 with residual takes 6.5 us (2.0 for its bytes): the
// launch, a TMA round trip, six blocks of k (0.14 us each), the joint and the store follow
// each other.

constexpr int kTileThreads = 256;
constexpr int kTileM = 128;
constexpr int kTileMaxSplit = 8;
constexpr int kTileMaxStages = 8;
__host__ __device__ constexpr int tile_stage_bytes(int BN) { return (kTileM + BN) * 128; }
// Stages that leave room for two CTAs per SM, and those that take all of it.
constexpr int tile_stages(int BN, bool alone) { return (alone ? 196608 : 98304) / tile_stage_bytes(BN); }
constexpr size_t tile_smem(int BN, bool alone) {
  const size_t ring = (size_t)tile_stages(BN, alone) * tile_stage_bytes(BN);
  const size_t sums = (size_t)kTileM * (BN + 4) * 4;
  return (ring > sums ? ring : sums) + 1024;
}

// By one thread.
__device__ __forceinline__ void tile_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` once the products this thread issued are done.
__device__ __forceinline__ void tile_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
}

template <int BN, bool A_ROW, bool B_ROW, bool SWIGLU>
__global__ void __launch_bounds__(kTileThreads, 2)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       LinearEpi e, int K, int splits, int stages, int m_tiles, unsigned int* err) {
  constexpr int kStageBytes = tile_stage_bytes(BN);
  constexpr int kOut = SWIGLU ? BN / 2 : BN;  // output columns of the tile
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kTileMaxStages], empty[kTileMaxStages], done;
  __shared__ uint32_t tmem_sh;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % splits, tile = blockIdx.x / splits;
  const int row0 = tile % m_tiles * kTileM, col0 = tile / m_tiles * kOut;
  const int nkb = (K + kLinBK - 1) / kLinBK;
  const int kb0 = (int)((int64_t)rank * nkb / splits);
  const int nb = (int)((int64_t)(rank + 1) * nkb / splits) - kb0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_sh, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // after the allocation: a later kernel may not take TMEM from a CTA still to come
  const uint32_t tmem = tmem_sh;
  int bad = 0;
  // one lane of a warp loads, one of another issues the products
  if (warp == 0) {
    if (elected()) {
      int issued = 0;
      uint32_t phase = 0;
      for (int kb = 0, s = 0; kb < nb; ++kb) {
        if (kb >= stages && !mbar_wait(&empty[s], phase ^ 1u, kWaitBudgetCycles)) {
          bad = 1;
          break;
        }
        unsigned char* a = smem + s * kStageBytes;
        unsigned char* b = a + kTileM * 128;
        const int k = (kb0 + kb) * kLinBK;
        mbar_arrive_expect_tx(&full[s], kStageBytes);
        if constexpr (A_ROW) {
          linear_tma_2d(a, &tm_a, k, row0, &full[s]);
        } else {
#pragma unroll
          for (int j = 0; j < kTileM / 64; ++j) linear_tma_2d(a + j * 8192, &tm_a, row0 + j * 64, k, &full[s]);
        }
        if constexpr (SWIGLU) {
          linear_tma_2d(b, &tm_b, k, col0, &full[s]);
          linear_tma_2d(b + kOut * 128, &tm_b, k, e.cols + col0, &full[s]);
        } else if constexpr (B_ROW) {
          linear_tma_2d(b, &tm_b, k, col0, &full[s]);
        } else {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j) linear_tma_2d(b + j * 8192, &tm_b, col0 + j * 64, k, &full[s]);
        }
        issued = kb + 1;
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (bad)  // copies in flight end before the CTA may
        for (int kb = issued > stages ? issued - stages : 0; kb < issued; ++kb)
          mbar_wait(&full[kb % stages], (uint32_t)(kb / stages) & 1u, kWaitBudgetCycles);
    }
  } else if (warp == 1) {
    if (elected()) {
      const uint32_t idesc = idesc_linear<A_ROW, B_ROW>(kTileM, BN);
      const uint64_t a_desc = operand_desc<A_ROW>(smem), b_desc = operand_desc<B_ROW>(smem + kTileM * 128);
      uint32_t phase = 0;
      for (int kb = 0, s = 0; kb < nb; ++kb) {
        if (!mbar_wait(&full[s], phase, kWaitBudgetCycles)) {
          bad = 1;
          break;
        }
        tc_fence_after();
        const uint64_t ad = a_desc + s * (kStageBytes >> 4), bd = b_desc + s * (kStageBytes >> 4);
        tile_mma(tmem, ad, bd, idesc, kb > 0);
#pragma unroll
        for (int k = 1; k < 4; ++k)
          tile_mma(tmem, ad + k * operand_step<A_ROW>(), bd + k * operand_step<B_ROW>(), idesc, 1);
        tile_commit(&empty[s]);
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      tile_commit(&done);
      if (!mbar_wait(&done, 0u, kWaitBudgetCycles)) bad = 1;
    }
  }
  __syncwarp();
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) raise_device_error(err, MOE_DEVERR_TIMEOUT);
  tc_fence_after();
  // the ring is free: the sums take its place, [row][BN + 4] fp32
  float* part = reinterpret_cast<float*>(smem);
  constexpr int kPitch = BN + 4;
  const int row = (warp & 3) * 32 + lane;
#pragma unroll 1
  for (int j = (warp >> 2) * 16; j < BN; j += 32) {
    uint32_t r[16];
    tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + j, r);
    tmem_ld_wait();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(part + row * kPitch + j + 4 * q) =
          make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                      __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
  }
  tc_fence_before();
  __syncthreads();
  if (splits > 1) cluster_barrier();
  if (warp == 1) tmem_dealloc(tmem, BN);
  if (!bad) {
    constexpr int kGroups = kOut / 8;
    const int rows = min(kTileM, e.M - row0);
    for (int i = rank * kTileThreads + tid; i < rows * kGroups; i += splits * kTileThreads) {
      const int r = i / kGroups, c = i % kGroups * 8;
      float z[2][8];
#pragma unroll
      for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
        const float* at = part + r * kPitch + h * kOut + c;
#pragma unroll
        for (int x = 0; x < 8; ++x) z[h][x] = 0.0f;
        for (int q = 0; q < splits; ++q) {
          float4 f[2];
          if (q == rank) {
            f[0] = *reinterpret_cast<const float4*>(at);
            f[1] = *reinterpret_cast<const float4*>(at + 4);
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f[y].x), "=f"(f[y].y), "=f"(f[y].z), "=f"(f[y].w)
                           : "r"(cluster_addr(at + 4 * y, q)));
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            z[h][4 * y] += f[y].x;
            z[h][4 * y + 1] += f[y].y;
            z[h][4 * y + 2] += f[y].z;
            z[h][4 * y + 3] += f[y].w;
          }
        }
      }
      finish8<SWIGLU>(e, row0 + r, col0 + c, z[0], z[1]);
    }
  }
  if (splits > 1) cluster_barrier();
}

template <int BN, bool A_ROW, bool B_ROW, bool SWIGLU>
moe_status_t launch_tiles(const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e, int splits,
                          cudaStream_t st) {
  constexpr int kOut = SWIGLU ? BN / 2 : BN;
  constexpr auto kern = linear_tile_kernel<BN, A_ROW, B_ROW, SWIGLU>;
  const int m_tiles = (e.M + kTileM - 1) / kTileM;
  const int64_t tiles = (int64_t)m_tiles * ((e.cols + kOut - 1) / kOut);
  if (tiles > (INT32_MAX / kTileMaxSplit)) return MOE_ERR_INVALID_ARG;
  CUtensorMap ta, tb;
  if (!linear_map(&ta, a, e.M, K, kTileM) || !linear_map(&tb, b, e.N, K, SWIGLU ? kOut : BN))
    return MOE_ERR_CUDA;
  if (const moe_status_t s = moe_host::allow_smem<kern>(tile_smem(BN, true))) return s;
  const bool alone = tiles * splits <= moe_host::sm_count();
  return moe_host::launch_clusters(kern, dim3((unsigned)(tiles * splits)), kTileThreads,
                                   tile_smem(BN, alone), dim3(splits, 1, 1), st, ta, tb, e, K, splits,
                                   tile_stages(BN, alone), m_tiles,
                                   moe_host::device_error_word());
}

template <int BN>
moe_status_t tiles_as(const LinearOp& a, const LinearOp& b, int K, const LinearEpi& e, int splits,
                      cudaStream_t st) {
  if (e.act == MOE_ACT_SWIGLU) return launch_tiles<BN, true, true, true>(a, b, K, e, splits, st);
  if (a.row_major)
    return b.row_major ? launch_tiles<BN, true, true, false>(a, b, K, e, splits, st)
                       : launch_tiles<BN, true, false, false>(a, b, K, e, splits, st);
  return launch_tiles<BN, false, false, false>(a, b, K, e, splits, st);
}

// Width and splits of the small tiles by an estimate in us, fitted to
// measurements over M 40 .. 512, N and K 256 .. 11008 (every width with every
// split): a block of 64 k takes .14 us (64 columns) or .215 (128) with a CTA per
// SM and twice as long with two; joining splits costs more the more CTAs there
// are.  What it takes is 2 % slower than the best of them in the mean, 22 % at
// worst (128 x 256 x 11008: 5.8 us for 4.8).
struct TileChoice {
  int bn, splits;
  float us;
};
TileChoice choose_tiles(const LinearEpi& e, int K) {
  const int sms = moe_host::sm_count(), nkb = (K + kLinBK - 1) / kLinBK;
  const int64_t m_tiles = (e.M + kTileM - 1) / kTileM;
  TileChoice best{64, 1, 1e30f};
  for (int bn = 64; bn <= 128; bn += 64)
    for (int splits = 1; splits <= kTileMaxSplit; splits *= 2) {
      const int span = e.act == MOE_ACT_SWIGLU ? bn / 2 : bn;
      const int64_t ctas = m_tiles * ((e.cols + span - 1) / span) * splits;
      if (splits > 1 && (nkb < splits * 4 || ctas > 2 * sms)) break;
      const int per = (nkb + splits - 1) / splits;
      const float join = splits == 1 ? 0.0f : splits == 2 ? 0.4f : splits == 4 ? 1.2f : 4.0f;
      const float crowd = ctas <= sms / 2 ? 1.0f : ctas <= sms ? 1.5f : 6.0f;
      const int64_t rounds = (ctas + 2 * sms - 1) / (2 * sms);
      const float us = (bn == 64 ? 3.4f : 4.6f) + join * crowd +
                       (ctas <= sms ? per * (bn == 64 ? 0.14f : 0.215f)
                                    : rounds * (per * (bn == 64 ? 0.29f : 0.40f) + 1.5f));
      if (us < best.us) best = {bn, splits, us};
    }
  return best;
}

}  // namespace

static void set_vec(LinearEpi& e) {
  using moe_host::aligned16;
  e.vec = e.cols % 8 == 0 && aligned16(e.out) && aligned16(e.residual) && aligned16(e.preact) &&
          aligned16(e.bias);
}

moe_status_t linear_product(const LinearOp& a, const LinearOp& b, int K, LinearEpi e, cudaStream_t st) {
  set_vec(e);
  // The form for few rows reads x for every 16 rows of W: past 16 rows of x that
  // shows where W is large (us for 32 rows, this form and tiles: 4096 x 22016 48,
  // 34; 4096 x 4096 11.4, 10.4; 1536 x 4096 6.4, 9.0; 2048 x 1536 6.1, 7.1).
  if (a.row_major && b.row_major && e.M <= kLinearRowsMost &&
      (e.M <= 16 || (int64_t)e.N * K < (1 << 24)))
    return linear_rows(a.p, a.ld, b.p, K, e, st);
  const TileChoice t = choose_tiles(e, K);
  // a pair's tile has 256 rows: with 128 or fewer half of it would be empty
  if (e.M > 128 && linear_pairs_us(e, K, b.row_major) < t.us) return linear_pairs(a, b, K, e, st);
  return t.bn == 64 ? tiles_as<64>(a, b, K, e, t.splits, st) : tiles_as<128>(a, b, K, e, t.splits, st);
}

// The product with the longer tiles first.
moe_status_t linear_products(const LinearOp (&a)[2], const LinearOp (&b)[2], const int (&K)[2],
                             LinearEpi (&e)[2], cudaStream_t st) {
  const int f = K[0] >= K[1] ? 0 : 1, g = 1 - f;
  float apart = 0.0f;
  for (int i = 0; i < 2; ++i) {
    set_vec(e[i]);
    const float tiles = choose_tiles(e[i], K[i]).us, pairs = linear_pairs_us(e[i], K[i], false);
    apart += e[i].M > 128 && pairs < tiles ? pairs : tiles;
  }
  if (e[0].M > 128 && e[1].M > 128) {
    const LinearEpi ee[2] = {e[f], e[g]};
    const int kk[2] = {K[f], K[g]};
    if (linear_pairs_both_us(ee, kk) < apart) {
      const LinearOp aa[2] = {a[f], a[g]}, bb[2] = {b[f], b[g]};
      return linear_pairs_both(aa, bb, kk, ee, st);
    }
  }
  if (const moe_status_t s = linear_product(a[0], b[0], K[0], e[0], st)) return s;
  return linear_product(a[1], b[1], K[1], e[1], st);
}

}  // namespace moe

extern "C" moe_status_t moe_linear(const uint16_t* x, int64_t ld_x, const uint16_t* w,
                                   const float* bias, const void* residual, int T, int K, int N,
                                   int activation, int out_dtype, void* out, uint16_t* preact,
                                   moe_stream_t stream) {
  using namespace moe;
  using moe_host::aligned16;
  using moe_host::aligned4;
  if (T < 0 || K < 8 || K % 8 != 0 || N < 1) return MOE_ERR_INVALID_ARG;
  if (T > kLinearMost || K > kLinearMost || N > kLinearMost) return MOE_ERR_INVALID_ARG;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (activation == MOE_ACT_SWIGLU && N % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out || !aligned16(x) || !aligned16(w) || ld_x < K || ld_x % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  const uintptr_t odd = out_dtype == MOE_DTYPE_BF16 ? 1u : 3u;
  if ((reinterpret_cast<uintptr_t>(out) & odd) || (reinterpret_cast<uintptr_t>(residual) & odd) ||
      (reinterpret_cast<uintptr_t>(preact) & 1u) || !aligned4(bias))
    return MOE_ERR_INVALID_ARG;
  const int cols = activation == MOE_ACT_SWIGLU ? N / 2 : N;
  const LinearEpi e{bias, residual, out, preact, T, N, cols, activation, out_dtype == MOE_DTYPE_BF16, 0};
  return linear_product({x, ld_x, true}, {w, K, true}, K, e, reinterpret_cast<cudaStream_t>(stream));
}
