// Tensor-core products by CTA pairs, with the epilogues of the vocabulary cross
// entropy and of the Newton-Schulz orthogonalisation.
//
// C[M, N] = epilogue(sum_k A(m, k) B(n, k)), 16-bit operands, fp32 accumulation
// in TMEM, for a batch of equal problems.  A cluster of two CTAs works on one
// tile of 256 x BN (tcgen05 cta_group::2): CTA r of the pair holds rows
// 128 r .. 128 r + 127 of A and of the accumulator and the BN / 2 rows
// (BN / 2) r .. of B, so each SM loads half of the shared operand.  Against the
// 128 x 256 tiles of one CTA that cuts the operand bytes an SM takes from L2 by a
// third, which is what bounds those.  The pair is persistent: it walks tiles
// cluster, cluster + clusters, ...
//   warp 0      TMA producer (both CTAs): the CTA's halves of the A and B k-slabs,
//               64 deep, into a ring of stages; all bytes are counted on the
//               leader's (CTA 0's) barrier
//   warp 1      allocates TMEM (both); the leader's lane 0 issues tcgen05.mma
//               (M 256, N BN, K 16) into one of two accumulators and commits to
//               both CTAs' barriers
//   warps 2-9   epilogue (both CTAs): 32 rows x BN / 2 columns each, while the
//               other accumulator fills; outputs leave through shared memory by
//               TMA, which also clips ragged edges
// Operands are K-major (row-major [rows, K]) or MN-major (row-major [K, rows]),
// with M, N and K of any size: the tensor maps end at the real extents, so tiles
// past an edge read zeros.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr int kBM = 256, kBK = 64;
constexpr int kThreads = 320, kEpiWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <int BN>
struct PairSmem {
  static constexpr int kA = 128 * kBK * 2;       // 16 KB: this CTA's half of the A slab
  static constexpr int kB = (BN / 2) * kBK * 2;  // this CTA's half of the B slab
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kOut = kStages * kStage;               // 4 KB staging per epilogue warp
  static constexpr int kBars = kOut + kEpiWarps * 4096;       // full, empty [stages]; acc_full, acc_empty [2]; drain
  static constexpr int kMisc = kBars + (2 * kStages + 5) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;            // slack for 1024-byte alignment
};
static_assert(PairSmem<256>::kAlloc <= 232448 && PairSmem<128>::kAlloc <= 232448, "shared memory of one SM");

// ------------------------------------------------------------ cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared location `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` (same offset) in both CTAs once every MMA issued so far is done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Load into this CTA's shared memory, bytes counted on `bar`, which may lie in the
// other CTA of the pair.
__device__ __forceinline__ void pair_tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                              int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(src),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, int bf16) {
  if (bf16) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&t);
  }
  return pack_half2(lo, hi);
}

// ---------------------------------------------------------------- tile order
// Tiles of one batch entry are taken in groups of group_m tile rows, row fastest
// within a group: the pairs at work at one time then cover a compact patch of C
// and share both operands' slabs in L2.  For a symmetric product only tiles that
// reach the diagonal or lie right of it are computed; the epilogue writes the
// mirror image.
struct Tile {
  int b, m, n;  // batch entry, tile row (256), tile column (BN)
};
template <int BN, bool SYM>
__device__ __forceinline__ Tile tile_at(const PairArgs& a, int t, int tm, int tn, int per_batch) {
  Tile r;
  r.b = t / per_batch;
  t -= r.b * per_batch;
  if (SYM) {
    int m = 0;
    for (int left = tn; t >= left; ++m) {
      t -= left;
      left -= kBM / BN;
    }
    r.m = m;
    r.n = m * (kBM / BN) + t;
    return r;
  }
  const int in_group = a.group_m * tn;
  const int g = t / in_group;
  t -= g * in_group;
  const int rows = min(a.group_m, tm - g * a.group_m);
  r.n = t / rows;
  r.m = g * a.group_m + (t - r.n * rows);
  return r;
}

// sum of n floats by one warp, in an order that depends on n alone
__device__ __forceinline__ float warp_total(const float* p, int n) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  int i = lane_id();
  for (; i + 96 < n; i += 128) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += __ldcg(p + i + 32 * j);
  }
  for (int j = 0; i < n; i += 32, ++j) s[j] += __ldcg(p + i);
  return warp_sum((s[0] + s[1]) + (s[2] + s[3]));
}

template <int EPI, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tc_pair_kernel(const __grid_constant__ PairArgs a) {
  using S = PairSmem<BN>;
  constexpr int kStages = S::kStages;
  constexpr bool kSym = EPI == PAIR_GRAM || EPI == PAIR_SQUARE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + S::kBars;
  auto bar_full = [&](int s) { return bar0 + 8 * s; };
  auto bar_empty = [&](int s) { return bar0 + 8 * kStages + 8 * s; };
  auto bar_acc_full = [&](int b) { return bar0 + 16 * kStages + 8 * b; };
  auto bar_acc_empty = [&](int b) { return bar0 + 16 * kStages + 16 + 8 * b; };
  const uint32_t BAR_DRAIN = bar0 + 16 * kStages + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const uint32_t rank = cluster_rank();
  const int clusters = gridDim.x / 2, cluster = blockIdx.x / 2;
  const int tm = (a.M + kBM - 1) / kBM, tn = (a.N + BN - 1) / BN;
  int per_batch = tm * tn;
  if (kSym) {
    per_batch = 0;
    for (int m = 0; m < tm; ++m) per_batch += max(tn - m * (kBM / BN), 0);
  }
  const int num_tiles = per_batch * a.batch;
  const int k_steps = (a.K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full(b), 1);
      mbar_init(bar_acc_empty(b), 2 * kEpiWarps);
    }
    mbar_init(BAR_DRAIN, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) pair_tmem_alloc(smem_u32(tmem_slot), 2 * BN);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.tm_a);
    tma_prefetch_desc(&a.tm_b);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t lim = a.wait_limit_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t cnt = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += clusters) {
        const Tile tile = tile_at<BN, kSym>(a, t, tm, tn, per_batch);
        const int m0 = tile.m * kBM + (int)rank * 128, n0 = tile.n * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < k_steps; ++kb, ++cnt) {
          const int s = cnt % kStages;
          const uint32_t ph = (cnt / kStages) & 1;
          if (!mbar_wait(bar_empty(s), ph ^ 1, abort_flag, a.status, lim)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(bar_full(s), 2 * S::kStage);
          const uint32_t full = map_rank(bar_full(s), 0);
          const uint32_t dA = sbase + s * S::kStage, dB = dA + S::kA;
          const int k0 = kb * kBK;
          if (a.a_mn) {
#pragma unroll
            for (int c = 0; c < 2; ++c) pair_tma_load(dA + c * 8192, &a.tm_a, full, m0 + 64 * c, k0, tile.b);
          } else {
            pair_tma_load(dA, &a.tm_a, full, k0, m0, tile.b);
          }
          if (a.b_mn) {
#pragma unroll
            for (int c = 0; c < BN / 128; ++c) pair_tma_load(dB + c * 8192, &a.tm_b, full, n0 + 64 * c, k0, tile.b);
          } else {
            pair_tma_load(dB, &a.tm_b, full, k0, n0, tile.b);
          }
        }
      }
      if (*abort_flag && rank == 0) {
        // let the pair's copies in flight land before the CTAs exit
        const uint32_t first = cnt > (uint32_t)kStages ? cnt - kStages : 0;
        for (uint32_t c = first; c < cnt; ++c)
          (void)mbar_wait(bar_full(c % kStages), (c / kStages) & 1, abort_flag, nullptr, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = idesc_f16(a.ab_bf16 ? 1u : 0u, a.a_mn ? 1u : 0u, a.b_mn ? 1u : 0u, kBM, BN);
      // K-major: LBO unused, SBO = 8 rows x 128 B, one K = 16 step moves 32 B;
      // MN-major: LBO = the 8 KB stride between 64-wide chunks, SBO = 8 k-rows x
      // 128 B, one step moves 16 k-rows = 2 KB
      const uint64_t dA0 = smem_desc_sw128(sbase, a.a_mn ? 8192 : 16, 1024);
      const uint64_t dB0 = smem_desc_sw128(sbase + S::kA, a.b_mn ? 8192 : 16, 1024);
      const uint32_t offA = a.a_mn ? 2048 : 32, offB = a.b_mn ? 2048 : 32;
      uint32_t cnt = 0, lt = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += clusters, ++lt) {
        const uint32_t b = lt & 1;
        if (!mbar_wait(bar_acc_empty(b), ((lt >> 1) & 1) ^ 1, abort_flag, a.status, lim)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem + b * BN;
        for (int kb = 0; kb < k_steps; ++kb, ++cnt) {
          const int s = cnt % kStages;
          if (!mbar_wait(bar_full(s), (cnt / kStages) & 1, abort_flag, a.status, lim)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = desc_off(dA0, s * S::kStage), db = desc_off(dB0, s * S::kStage);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            pair_mma(acc, desc_off(da, kk * offA), desc_off(db, kk * offB), idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          pair_commit(bar_empty(s));
        }
        if (!ok) break;
        pair_commit(bar_acc_full(b));
      }
      // every MMA issued has completed before TMEM is released
      pair_commit(BAR_DRAIN);
      (void)mbar_wait(BAR_DRAIN, 0, abort_flag, nullptr, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t quarter = warp & 3;     // TMEM lanes 32 * quarter .. + 31
    const int half = (int)(warp - 2) >> 2;  // columns [half * BN / 2, + BN / 2)
    const uint32_t stage = sbase + S::kOut + (warp - 2) * 4096;
    uint8_t* const stage_p = smem + S::kOut + (warp - 2) * 4096;
    const uint32_t acc_empty_leader[2] = {map_rank(bar_acc_empty(0), 0), map_rank(bar_acc_empty(1), 0)};
    uint32_t lt = 0;
    // one 16-byte piece of the warp's staging rows of 128 bytes, 128-byte swizzle
    auto stage16 = [&](int piece, uint4 v) {
      *reinterpret_cast<uint4*>(stage_p + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
    };
    // the staging buffer is free again once the last copy out of it has read it
    auto stage_free = [&]() {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    };
    auto stage_out = [&](auto issue) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        issue();
        bulk_commit();
      }
    };
    int alpha_batch = -1;
    float alpha = 0.f;  // Newton-Schulz: the shift of the Gram matrix's diagonal
    for (int t = cluster; t < num_tiles; t += clusters, ++lt) {
      const uint32_t b = lt & 1;
      const Tile tile = tile_at<BN, kSym>(a, t, tm, tn, per_batch);
      const int row0 = tile.m * kBM + (int)rank * 128 + (int)quarter * 32;
      const int row = row0 + (int)lane;
      const int col0 = tile.n * BN + half * (BN / 2);
      if (EPI == PAIR_GRAM || EPI == PAIR_SQUARE || EPI == PAIR_UPDATE) {
        if (tile.b != alpha_batch) {
          alpha_batch = tile.b;
          alpha = a.num_sums ? warp_total(a.sums + (long long)tile.b * a.num_sums, a.num_sums) * a.sums_mul : a.sums_mul;
        }
      }
      if (!mbar_wait(bar_acc_full(b), (lt >> 1) & 1, abort_flag, a.status, lim)) break;
      tc_fence_after();
      const uint32_t src = tmem + b * BN + half * (BN / 2) + ((quarter * 32) << 16);
      // the accumulator goes back to the leader's MMA thread
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_leader[b]);
      };
      auto load32 = [&](int c, float* v) {
        uint32_t r[32];
        RA_TMEM_LD32(src + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      };

      if (EPI == PAIR_STATS) {
        // Online softmax statistics of the tile's columns for this row, and the
        // target's logit where it lies among them.  Bound by the matrix product;
        // the exponentials (BN / 2 per thread and tile) hide behind it for K > 256.
        const long long y = row < a.M ? a.targets[row] : -1;
        const int ycol = (y >= col0 && y < col0 + BN / 2) ? (int)(y - col0) : -1;
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
          float v[32];
          load32(c, v);
          if (c == BN / 2 - 32) release();
          if (col0 + c + 32 > a.N) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col0 + c + j >= a.N) v[j] = -INFINITY;
          }
          float mk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mk[k] = fmax3(v[k], v[k + 4], v[k + 8]);
#pragma unroll
          for (int j = 12; j < 28; j += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mk[k] = fmax3(mk[k], v[j + k], v[j + 4 + k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) mk[k] = fmaxf(mk[k], v[28 + k]);
          const float mx = fmax3(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]), m);
          // a row without a finite logit so far keeps l = 0 (0 - (-inf) must not be formed)
          const float ref = mx == -INFINITY ? 0.f : mx * kLog2e;
          float s0 = l * ex2_approx(m * kLog2e - ref), s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            s0 += ex2_approx(fmaf(v[j], kLog2e, -ref));
            s1 += ex2_approx(fmaf(v[j + 1], kLog2e, -ref));
            s2 += ex2_approx(fmaf(v[j + 2], kLog2e, -ref));
            s3 += ex2_approx(fmaf(v[j + 3], kLog2e, -ref));
          }
          l = (s0 + s1) + (s2 + s3);
          m = mx;
          if (__any_sync(0xffffffffu, ycol >= c && ycol < c + 32)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (ycol == c + j) a.target_logit[row] = v[j];
          }
        }
        if (row < a.M && col0 < a.N) a.stats[(long long)(tile.n * 2 + half) * a.M + row] = make_float2(m, l);
      } else if (EPI == PAIR_DLOGITS) {
        // d = g (e^{z - lse} - [column = target]), rounded to the operand type of
        // the two products that follow (bf16: any range; fp16: g is brought near
        // 2^13 by a power of two that those products take out again)
        const long long y = row < a.M ? a.targets[row] : a.ignore;
        const bool live = row < a.M && y != a.ignore && y >= 0 && y < a.vocab;
        const float g = live ? a.grad[row] * (a.scale ? a.scale[0] : 1.f) : 0.f;
        const float lse2 = live ? a.lse[row] * kLog2e : 0.f;
        const long long yc = y - a.col_off - col0;
        const int ycol = (live && yc >= 0 && yc < BN / 2) ? (int)yc : -1;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 64) {
          stage_free();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            load32(c + 32 * h, v);
            if (c == BN / 2 - 64 && h == 1) release();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = ex2_approx(fmaf(v[j], kLog2e, -lse2));
            const int cc = c + 32 * h;
            if (__any_sync(0xffffffffu, ycol >= cc && ycol < cc + 32)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (ycol == cc + j) v[j] -= 1.f;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = live ? v[j] * g : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              stage16(4 * h + j, make_uint4(pack_pair(v[8 * j], v[8 * j + 1], a.ab_bf16),
                                            pack_pair(v[8 * j + 2], v[8 * j + 3], a.ab_bf16),
                                            pack_pair(v[8 * j + 4], v[8 * j + 5], a.ab_bf16),
                                            pack_pair(v[8 * j + 6], v[8 * j + 7], a.ab_bf16)));
          }
          stage_out([&]() {
            if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_c, stage, col0 + c, row0, tile.b);
          });
        }
      } else if (EPI == PAIR_STORE) {
        // c = mul * acc (+ what c_add holds): 16-bit or fp32 out; fp32 may be added
        // to what is there (each element once per launch, so the sum's order is fixed)
        const float mul = a.scale ? a.scale[1] : 1.f;
        if (a.c_dtype == RA_F32) {
#pragma unroll 1
          for (int c = 0; c < BN / 2; c += 32) {
            stage_free();
            float v[32];
            load32(c, v);
            if (c == BN / 2 - 32) release();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stage16(j, make_uint4(__float_as_uint(v[4 * j] * mul), __float_as_uint(v[4 * j + 1] * mul),
                                    __float_as_uint(v[4 * j + 2] * mul), __float_as_uint(v[4 * j + 3] * mul)));
            stage_out([&]() {
              if (row0 < a.M && col0 + c < a.N) {
                if (a.c_accumulate) tma_add_3d(&a.tm_c, stage, col0 + c, row0, tile.b);
                else tma_store_3d(&a.tm_c, stage, col0 + c, row0, tile.b);
              }
            });
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < BN / 2; c += 64) {
            stage_free();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[32];
              load32(c + 32 * h, v);
              if (c == BN / 2 - 64 && h == 1) release();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= mul;
              if (a.c_add && row < a.M) {  // N is a multiple of 8 where c_add is used
                const float4* p = reinterpret_cast<const float4*>(a.c_add + (long long)row * a.N + col0 + c + 32 * h);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  if (col0 + c + 32 * h + 4 * j < a.N) {
                    const float4 f = p[j];
                    v[4 * j] += f.x;
                    v[4 * j + 1] += f.y;
                    v[4 * j + 2] += f.z;
                    v[4 * j + 3] += f.w;
                  }
                }
              }
              const int bf = a.c_dtype == RA_BF16;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                stage16(4 * h + j,
                        make_uint4(pack_pair(v[8 * j], v[8 * j + 1], bf), pack_pair(v[8 * j + 2], v[8 * j + 3], bf),
                                   pack_pair(v[8 * j + 4], v[8 * j + 5], bf), pack_pair(v[8 * j + 6], v[8 * j + 7], bf)));
            }
            stage_out([&]() {
              if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_c, stage, col0 + c, row0, tile.b);
            });
          }
        }
      } else if (EPI == PAIR_GRAM || EPI == PAIR_SQUARE) {
        // GRAM:   A' = X X^T - alpha I
        // SQUARE: B' = (b + 2 c alpha) A' + c A'^2
        // both symmetric: a tile right of the diagonal block also writes its mirror
        // image.  Values leave as fp16 times a power of two.
        const bool mirror = tile.n * BN >= (tile.m + 1) * kBM;
        const float lin = EPI == PAIR_SQUARE ? (a.ns_b + 2.f * a.ns_c * alpha) * a.ns_lin : 0.f;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 64) {
          stage_free();
          uint32_t pk[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            load32(c + 32 * h, v);
            if (c == BN / 2 - 64 && h == 1) release();
            const int cc = col0 + c + 32 * h;
            if (EPI == PAIR_GRAM) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = v[j] * a.ns_acc - (row == cc + j ? alpha * a.ns_out : 0.f);
            } else {
              uint4 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = (row < a.M && cc + 8 * j < a.N)
                           ? *reinterpret_cast<const uint4*>(a.hi_in + ((long long)tile.b * a.M + row) * a.ld + cc + 8 * j)
                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 f = unpack_half2(ww[q]);
                  v[8 * j + 2 * q] = fmaf(v[8 * j + 2 * q], a.ns_acc, lin * f.x);
                  v[8 * j + 2 * q + 1] = fmaf(v[8 * j + 2 * q + 1], a.ns_acc, lin * f.y);
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[16 * h + j] = pack_half2(v[2 * j], v[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              stage16(4 * h + j, make_uint4(pk[16 * h + 4 * j], pk[16 * h + 4 * j + 1], pk[16 * h + 4 * j + 2],
                                            pk[16 * h + 4 * j + 3]));
          }
          stage_out([&]() {
            if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_c, stage, col0 + c, row0, tile.b);
          });
          if (mirror) {  // rows col0 + c .. + 63, columns row0 .. + 31
            stage_free();
            uint16_t* out = reinterpret_cast<uint16_t*>(stage_p);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              out[(2 * j) * 32 + lane] = (uint16_t)(pk[j] & 0xffffu);
              out[(2 * j + 1) * 32 + lane] = (uint16_t)(pk[j] >> 16);
            }
            stage_out([&]() {
              if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_ct, stage, row0, col0 + c, tile.b);
            });
          }
        }
      } else if (EPI == PAIR_UPDATE) {
        // X <- (a + b alpha + c alpha^2) X + B' X (or X B'), X as two fp16 terms;
        // the last step writes the result itself
        const float own = a.ns_a + alpha * (a.ns_b + a.ns_c * alpha);
        float sq = 0.f;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
          float v[32];
          const int cc = col0 + c;
          const long long off = ((long long)tile.b * a.M + row) * a.ld + cc;
          uint4 wh[4], wl[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = row < a.M && cc + 8 * j < a.N;
            wh[j] = in ? *reinterpret_cast<const uint4*>(a.hi_in + off + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
            wl[j] = in ? *reinterpret_cast<const uint4*>(a.lo + off + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
          }
          load32(c, v);
          if (c == BN / 2 - 32) release();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t hh[4] = {wh[j].x, wh[j].y, wh[j].z, wh[j].w}, ll[4] = {wl[j].x, wl[j].y, wl[j].z, wl[j].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = unpack_half2(hh[q]), e = unpack_half2(ll[q]);
              v[8 * j + 2 * q] = fmaf(v[8 * j + 2 * q], a.ns_acc, own * (f.x + e.x));
              v[8 * j + 2 * q + 1] = fmaf(v[8 * j + 2 * q + 1], a.ns_acc, own * (f.y + e.y));
            }
          }
          if (a.out) {
            if (row < a.M && cc < a.N) {
              const long long o = tile.b * a.out_bstride + (long long)row * a.out_ld + cc;
              if (a.out_vec && cc + 32 <= a.N) {
                if (a.c_dtype == RA_F32) {
                  float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    p[j] = make_float4(v[4 * j] * a.ns_out, v[4 * j + 1] * a.ns_out, v[4 * j + 2] * a.ns_out,
                                       v[4 * j + 3] * a.ns_out);
                } else {
                  uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o);
                  const int bf = a.c_dtype == RA_BF16;
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    p[j] = make_uint4(pack_pair(v[8 * j] * a.ns_out, v[8 * j + 1] * a.ns_out, bf),
                                      pack_pair(v[8 * j + 2] * a.ns_out, v[8 * j + 3] * a.ns_out, bf),
                                      pack_pair(v[8 * j + 4] * a.ns_out, v[8 * j + 5] * a.ns_out, bf),
                                      pack_pair(v[8 * j + 6] * a.ns_out, v[8 * j + 7] * a.ns_out, bf));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  if (cc + j < a.N) {
                    if (a.c_dtype == RA_F32) static_cast<float*>(a.out)[o + j] = v[j] * a.ns_out;
                    else if (a.c_dtype == RA_BF16)
                      static_cast<__nv_bfloat16*>(a.out)[o + j] = __float2bfloat16_rn(v[j] * a.ns_out);
                    else static_cast<__half*>(a.out)[o + j] = __float2half_rn(v[j] * a.ns_out);
                  }
                }
              }
            }
          } else {
            if (row < a.M) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float x = cc + j < a.N ? v[j] : 0.f;
                sq = fmaf(x, x, sq);
              }
            }
            // 32 rows x 32 columns: the high terms in the staging buffer's first
            // half, the low terms in its second, 64-byte rows, no swizzle
            stage_free();
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              hi[j] = pack_half2(v[2 * j], v[2 * j + 1]);
              const float2 f = unpack_half2(hi[j]);
              lo[j] = pack_half2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              *reinterpret_cast<uint4*>(stage_p + lane * 64 + 16 * j) =
                  make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
              *reinterpret_cast<uint4*>(stage_p + 2048 + lane * 64 + 16 * j) =
                  make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
            }
            stage_out([&]() {
              if (row0 < a.M && cc < a.N) {
                tma_store_3d(&a.tm_c, stage, cc, row0, tile.b);
                tma_store_3d(&a.tm_ct, stage + 2048, cc, row0, tile.b);
              }
            });
          }
        }
        if (!a.out) {
          sq = warp_sum(sq);
          const int per = per_batch * 2 * kEpiWarps;
          if (lane == 0)
            a.sums_out[(long long)tile.b * per + ((t - tile.b * per_batch) * 2 + (int)rank) * kEpiWarps + (int)(warp - 2)] = sq;
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tmem, 2 * BN);
}

}  // namespace

int pair_tiles(const PairArgs& a, int bn) {
  const int tm = (a.M + kBM - 1) / kBM, tn = (a.N + bn - 1) / bn;
  if (a.epi == PAIR_GRAM || a.epi == PAIR_SQUARE) {
    int n = 0;
    for (int m = 0; m < tm; ++m) n += tn - m * (kBM / bn) > 0 ? tn - m * (kBM / bn) : 0;
    return n;
  }
  return tm * tn;
}

cudaError_t launch_tc_pair(const PairArgs& a, int bn, int num_sms, cudaStream_t st) {
  if (a.M <= 0 || a.N <= 0 || a.K <= 0 || a.batch <= 0 || a.group_m <= 0 || num_sms < 2) return cudaErrorInvalidValue;
  const long long tiles = (long long)pair_tiles(a, bn) * a.batch;
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = num_sms / 2;
  const int grid = 2 * (int)(tiles < pairs ? tiles : pairs);
  auto run = [&](auto kernel, int smem) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    kernel<<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
  };
  cudaError_t e = cudaErrorInvalidValue;
  auto pick = [&](auto epi) {
    constexpr int E = decltype(epi)::value;
    if (bn == 256) e = run(tc_pair_kernel<E, 256>, PairSmem<256>::kAlloc);
    else if (bn == 128) e = run(tc_pair_kernel<E, 128>, PairSmem<128>::kAlloc);
  };
  switch (a.epi) {
    case PAIR_STATS: pick(std::integral_constant<int, PAIR_STATS>{}); break;
    case PAIR_DLOGITS: pick(std::integral_constant<int, PAIR_DLOGITS>{}); break;
    case PAIR_STORE: pick(std::integral_constant<int, PAIR_STORE>{}); break;
    case PAIR_GRAM: pick(std::integral_constant<int, PAIR_GRAM>{}); break;
    case PAIR_SQUARE: pick(std::integral_constant<int, PAIR_SQUARE>{}); break;
    case PAIR_UPDATE: pick(std::integral_constant<int, PAIR_UPDATE>{}); break;
    default: break;
  }
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaSuccess;
}

}  // namespace ra
