// Building blocks of the tensor-core products by CTA pairs: C = A B^T on tiles of
// 256 x 256 or 256 x 128 by a cluster of two CTAs (tcgen05 cta_group::2), 16-bit
// operands, fp32 accumulation in TMEM.
//
// CTA r of the pair holds rows 128 r .. 128 r + 127 of A and of the accumulator and
// rows (bn / 2) r .. of B, so each SM loads half of the shared operand: against the
// 128 x 256 tiles of a single CTA that cuts the operand bytes an SM takes from L2 by a
// third, which is what bounds those (the feed-forward products reach 1470-1505
// TFLOP/s that way; these 1760 on 4096 x 32768 x 2048 logits alone and 1640-1670 on 8192 x
// 131072 x 2048, 2.6-2.7 ms for calls back to back at the power limit, 2.5 in a cool run).
//   warp 0      TMA producer (both CTAs): the CTA's halves of the A and B k-slabs,
//               64 deep, into a ring of stages; all bytes are counted on the
//               leader's (CTA 0's) barrier
//   warp 1      allocates TMEM (both); the leader's lane 0 issues tcgen05.mma
//               (M 256, N bn, K 16) into one of two accumulators and commits to
//               both CTAs' barriers
//   8 warps     epilogue (both CTAs): 32 rows x bn / 2 columns each, while the
//               other accumulator fills
// A k-slab takes 0.33 us, of a narrow tile as of a wide one (0.98 against 1.86 PFLOP/s on
// 8192 x 131072 x 2048 products), so the narrow one pays only where more tiles find an
// idle pair, by its shorter epilogue.  Rings of 4, 5 and 6 stages run alike.
// Operands are K-major (row-major [rows, K]) or MN-major (row-major [K, rows]), of
// any size: the tensor maps end at the real extents, so what lies past an edge reads
// as zeros.
#pragma once

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

constexpr int kPairEpiWarps = 8;

// Shared memory: a ring of `Stages` k-slabs, `WarpBytes` of staging per epilogue warp,
// the barriers (full, empty [Stages]; acc_full, acc_empty [2]; drain; `Extra` more).
template <int Stages, int WarpBytes, int Extra>
struct PairSmem {
  static constexpr int kStages = Stages;
  static constexpr int kA = 128 * 64 * 2;       // this CTA's half of the A slab
  static constexpr int kStage = kA + 128 * 64 * 2;
  static constexpr int kOut = kStages * kStage;
  static constexpr int kBars = kOut + kPairEpiWarps * WarpBytes;
  static constexpr int kMisc = kBars + (2 * kStages + 5 + Extra) * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;  // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "shared memory of one SM");
};

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
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
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
__device__ __forceinline__ void bulk_wait_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, int bf16) {
  if (bf16) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&t);
  }
  return pack_half2(lo, hi);
}

// How an operand is read, slab by slab: K-major through by_k (boxes of 64 k x rows) or
// MN-major through by_mn (boxes of 64 rows x 64 k).  A symmetric matrix of which only
// the blocks of 256 right of and on the diagonal are held is read K-major there and, left
// of the diagonal, MN-major from the block's mirror image.
struct Operand {
  const CUtensorMap *by_k, *by_mn;
  int mode;  // 0: K-major, 1: MN-major, 2: symmetric, upper blocks
  __device__ __forceinline__ bool mn_at(int block, int slab) const { return mode == 1 || (mode == 2 && slab / 4 < block); }
  // the slab from which on the majorness differs from `slab`'s
  __device__ __forceinline__ int change(int block, int slab) const {
    return mode == 2 && slab / 4 < block ? 4 * block : 0x7fffffff;
  }
};

// ------------------------------------------------------------- the CTA's frame
// Barriers, TMEM and limits of one CTA of a pair; the roles below count their k-slabs
// (cnt) and accumulators (lt) through the whole launch.
template <class S>
struct Pair {
  uint8_t* smem;
  uint32_t sbase, bar0, rank, tmem;
  volatile int* abort;
  int* status;
  uint64_t lim;

  __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8 * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8 * (S::kStages + s); }
  __device__ __forceinline__ uint32_t acc_full(int b) const { return bar0 + 8 * (2 * S::kStages + b); }
  __device__ __forceinline__ uint32_t acc_empty(int b) const { return bar0 + 8 * (2 * S::kStages + 2 + b); }
  __device__ __forceinline__ uint32_t drain() const { return bar0 + 8 * (2 * S::kStages + 4); }
  __device__ __forceinline__ uint32_t extra(int i) const { return bar0 + 8 * (2 * S::kStages + 5 + i); }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    return mbar_wait(bar, parity, abort, status, lim);
  }

  // init_extra: initialises the kernel's own barriers (one thread)
  template <class F>
  __device__ __forceinline__ void begin(uint8_t* smem_raw, int* status_word, uint64_t limit, F init_extra) {
    smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    sbase = smem_u32(smem);
    bar0 = sbase + S::kBars;
    rank = cluster_rank();
    abort = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
    status = status_word;
    lim = limit;
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
    if (threadIdx.x == 0) {
      for (int s = 0; s < S::kStages; ++s) {
        mbar_init(full(s), 1);
        mbar_init(empty(s), 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(acc_full(b), 1);
        // the CTA's own epilogue warps, and in the leader the peer's, passed on as one
        mbar_init(acc_empty(b), kPairEpiWarps + (rank == 0 ? 1 : 0));
      }
      mbar_init(drain(), 1);
      init_extra();
      *abort = 0;
      fence_barrier_init();
    }
    if (warp_id() == 1) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    tmem = __shfl_sync(0xffffffffu, *slot, 0);
  }
  __device__ __forceinline__ void end() {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal it
    tc_fence_after();
    if (warp_id() == 1)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }

  // Producer (one lane of warp 0 in both CTAs): k-slabs [k_from, k_to) of the tile
  // whose first row and column are m0 and n0.  a_rows < 128: all of A's rows, K-major, lie
  // in the leader and are that few: the peer loads none, and what the rest of the A slab
  // holds makes only rows of C that nobody reads.  fold > 0: A's slabs are those of matrices
  // batch, batch + 1, ... of `fold` slabs each, B's those of the one matrix again and again.
  __device__ __forceinline__ bool produce(uint32_t& cnt, const Operand& A, const Operand& B, int bn, int m0, int n0,
                                          int batch, int k_from, int k_to, int a_rows = 128, int fold = 0) const {
    const int a_block = m0 / 256, b_block = n0 / 256;
    m0 += (int)rank * 128;
    n0 += (int)rank * (bn / 2);
    const uint32_t bytes = (a_rows < 128 ? a_rows * 128 : 2 * S::kA) + bn * 128;
    for (int kb = k_from; kb < k_to; ++kb, ++cnt) {
      const int s = cnt % S::kStages;
      if (!wait(empty(s), ((cnt / S::kStages) & 1) ^ 1)) return false;
      if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
      const uint32_t bar = map_rank(full(s), 0);
      const uint32_t dA = sbase + s * S::kStage, dB = dA + S::kA;
      const int z = fold ? kb / fold : 0, k0 = (kb - z * fold) * 64;
      if (A.mn_at(a_block, kb)) {
        pair_tma_load(dA, A.by_mn, bar, m0, k0, batch + z);
        pair_tma_load(dA + 8192, A.by_mn, bar, m0 + 64, k0, batch + z);
      } else if (a_rows == 128 || rank == 0) {
        pair_tma_load(dA, A.by_k, bar, k0, m0, batch + z);
      }
      if (B.mn_at(b_block, kb)) {
        pair_tma_load(dB, B.by_mn, bar, n0, k0, batch);
        if (bn == 256) pair_tma_load(dB + 8192, B.by_mn, bar, n0 + 64, k0, batch);
      } else {
        pair_tma_load(dB, B.by_k, bar, k0, n0, batch);
      }
    }
    return true;
  }
  // After a wait gave up: let the pair's copies in flight land before the CTAs exit.  Their bytes
  // are counted in the leader, which has not expected those of stages that only the peer had
  // reached: the peer stays for a millisecond, a copy takes microseconds.
  __device__ __forceinline__ void producer_drain(uint32_t cnt) const {
    if (rank != 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
      return;
    }
    const uint32_t first = cnt > (uint32_t)S::kStages ? cnt - S::kStages : 0;
    for (uint32_t c = first; c < cnt; ++c)
      mbar_drain(full(c % S::kStages), (c / S::kStages) & 1);
  }

  // MMA issuer (warp 1 of the leader, whole warp): k-slabs [k_from, k_to) of one tile.
  // All lanes run the loop and one elected lane issues, so that descriptors and counters
  // stay warp-uniform: computed in a single lane's branch they cost more to issue than
  // the tensor pipe takes for a narrow tile's product (64 cycles).
  // K-major operands: LBO unused, SBO = 8 rows x 128 B, one K = 16 step moves 32 B;
  // MN-major: LBO = the 8 KB stride between 64-wide chunks, SBO = 8 k-rows x 128 B,
  // one step moves 16 k-rows = 2 KB.
  __device__ __forceinline__ bool multiply(uint32_t& cnt, uint32_t& lt, int ab_bf16, const Operand& A,
                                           const Operand& B, int bn, int m0, int n0, int k_from, int k_to) const {
    const uint32_t b = lt & 1;
    const bool issuer = elect_lane();
    if (!__all_sync(0xffffffffu, wait(acc_empty(b), ((lt >> 1) & 1) ^ 1))) return false;
    tc_fence_after();
    const uint32_t acc = tmem + b * 256;
    const uint32_t idesc0 = idesc_f16(ab_bf16 ? 1u : 0u, 0, 0, 256, bn);
    uint32_t accumulate = 0;
    for (int kb = k_from; kb < k_to;) {
      // the slabs up to `end` are of one majorness
      const bool a_mn = A.mn_at(m0 / 256, kb), b_mn = B.mn_at(n0 / 256, kb);
      const int end = min(k_to, min(A.change(m0 / 256, kb), B.change(n0 / 256, kb)));
      const uint64_t da0 = smem_desc_sw128(sbase, a_mn ? 8192 : 16, 1024);
      const uint64_t db0 = smem_desc_sw128(sbase + S::kA, b_mn ? 8192 : 16, 1024);
      const uint32_t idesc = idesc0 | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16);
      const uint32_t offA = a_mn ? 2048 : 32, offB = b_mn ? 2048 : 32;
      for (; kb < end; ++kb, ++cnt) {
        const uint32_t s = cnt % S::kStages;
        if (!__all_sync(0xffffffffu, wait(full(s), (cnt / S::kStages) & 1))) return false;
        tc_fence_after();
        const uint64_t da = desc_off(da0, s * S::kStage), db = desc_off(db0, s * S::kStage);
        if (issuer) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            pair_mma(acc, desc_off(da, kk * offA), desc_off(db, kk * offB), idesc, kk ? 1u : accumulate);
          pair_commit(empty(s));
        }
        accumulate = 1;
        __syncwarp();
      }
    }
    if (issuer) pair_commit(acc_full(b));
    __syncwarp();
    ++lt;
    return true;
  }
  // Every MMA issued has completed before TMEM is released.
  __device__ __forceinline__ void multiply_drain() const {
    if (elect_lane()) pair_commit(drain());
    __syncwarp();
    mbar_drain(drain(), 0);
  }

  // Epilogue: the accumulator goes back to the leader's MMA thread (whole warp).  The
  // warps of the peer arrive in their own CTA, where `forward` passes it on: an arrival
  // in the other CTA waits for the warp's stores under way, 0.5 us in the epilogue.
  __device__ __forceinline__ void release(uint32_t b) const {
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(acc_empty(b));
  }
  // Warp 1 of the peer: one tile's release.
  __device__ __forceinline__ bool forward(uint32_t& lt) const {
    const uint32_t b = lt & 1;
    if (!__all_sync(0xffffffffu, wait(acc_empty(b), (lt >> 1) & 1))) return false;
    if (lane_id() == 0) mbar_arrive_cluster(map_rank(acc_empty(b), 0));
    __syncwarp();
    ++lt;
    return true;
  }
};

// 32 columns of the accumulator, this thread's row.
__device__ __forceinline__ void tmem_load32(uint32_t src, float* v) {
  uint32_t r[32];
  RA_TMEM_LD32(src, r);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

// 64 columns, with one wait.
__device__ __forceinline__ void tmem_load64(uint32_t src, float* v) {
  uint32_t r0[32], r1[32];
  RA_TMEM_LD32(src, r0);
  RA_TMEM_LD32(src + 32, r1);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = __uint_as_float(r0[j]);
    v[32 + j] = __uint_as_float(r1[j]);
  }
}

// ---------------------------------------------------------------- tile order
// Tiles of one problem are taken in groups of group_m tile rows, row fastest within a
// group: the pairs at work at one time then cover a compact patch of C and share both
// operands' slabs in L2.
struct Tile {
  int m, n;  // tile row (256), tile column (bn)
};
__device__ __forceinline__ Tile tile_grouped(int t, int tm, int tn, int group_m) {
  const int in_group = group_m * tn;
  const int g = t / in_group;
  t -= g * in_group;
  const int rows = min(group_m, tm - g * group_m);
  const int n = t / rows;
  return Tile{g * group_m + (t - n * rows), n};
}

}  // namespace ra
