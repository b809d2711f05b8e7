// Newton-Schulz orthogonalisation of a batch of matrices: one launch for the norm and
// one persistent launch for everything else, on CTA pairs (ra_pair.cuh).
//
// The iteration is a chain of products, 3 per step, each of which needs all of the one
// before:
//   GRAM     A' = X X^T - alpha I      (X^T X where rows > cols), alpha = |X|_F^2 / m
//   SQUARE   B' = (b + 2 c alpha) A' + c A'^2
//   UPDATE   X <- (a + b alpha + c alpha^2) X + B' X   (X B')
// which is a X + (b A + c A^2) X with A = A' + alpha I.  The products' operands are fp16
// (times powers of two); taking alpha I out keeps the rounding of the Gram matrix's
// large common diagonal out of the result, and X is carried as two fp16 terms (hi the
// operand, hi + lo the state).  Where |G| is far below eps, X is tiny at first and grows by
// the polynomial's slope at each step: it is held times a power of two that falls from step
// to step (without, norms of 1e-5 eps left errors of 3e-3, and of 1e-8 eps nothing).  A' and
// B' are symmetric: blocks left of the diagonal are
// neither computed nor held, the products read their mirror images (ra_pair.cuh).
//
// One launch because the chain of a small matrix is all latency: as launches of their
// own the products of a 128 x 512 matrix took 7 us each.  All tiles of the chain, step by
// step and phase by phase, form one sequence that the pairs take in turn.  A tile waits
// until all tiles of its matrix's phase before are written (a count per matrix), so that
// with several matrices one's phase ends while another's runs and no pair idles at the
// phases' ends.  Tiles wait only for earlier ones in the sequence, and the launch is
// cooperative, so all pairs are there.  Every wait is bounded: a CTA that gives up marks
// the launch's word, records RA_ERR_TIMEOUT, and the others leave when they see the mark.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <mutex>

#include "ra_ns.cuh"
#include "ra_pair.cuh"

namespace ra {
namespace {

constexpr int kThreads = 320;  // producer, MMA issuer, 8 epilogue warps
// 5 stages of 32 KB; 8 KB of staging per epilogue warp (two tiles of 32 rows x 64
// columns).  Extra barriers: staging filled [8].
using S = PairSmem<5, 8192, 8>;

// Bound by reading G once.  Also readies the chain's words.
__global__ void __launch_bounds__(512) ns_sumsq_kernel(const __grid_constant__ NsInput in, float* parts,
                                                       unsigned int* words, int num_words) {
  __shared__ float part[3][16];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < num_words; i += 512) words[i] = 0u;
  const unsigned chunks = (in.cols + 7) / 8;
  const unsigned total = in.rows * chunks;  // at most 2^29: sides are at most 2^16
  float s[3] = {0.f, 0.f, 0.f};
  for (unsigned i = blockIdx.x * 512 + threadIdx.x; i < total; i += gridDim.x * 512 * kNsBatch) {
    NsRaw g[kNsBatch];
#pragma unroll
    for (int k = 0; k < kNsBatch; ++k) {
      const unsigned j = i + k * gridDim.x * 512, r = j / chunks, c = (j - r * chunks) * 8;
      g[k] = load8(in, blockIdx.y * in.bstride + r * in.ld + c, j < total ? in.cols - (int)c : 0);
    }
#pragma unroll
    for (int k = 0; k < kNsBatch; ++k) {
      float v[8];
      unpack8(in, g[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) ns_add_square(v[j], s);
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = warp_sum(s[k]);
    if ((threadIdx.x & 31) == 0) part[k][threadIdx.x >> 5] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) x += part[threadIdx.x][j];
    parts[((long long)blockIdx.y * kNsParts + blockIdx.x) * 3 + threadIdx.x] = x;
  }
}

// sum of n floats by one warp, in an order that depends on n alone
__device__ __forceinline__ float warp_total(const float* p, int n) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i = lane_id(); i < n; i += 256) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += i + 32 * j < n ? __ldcg(p + i + 32 * j) : 0.f;
  }
  return warp_sum(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
}

// 2^e for e of at most 0; 0 below fp32's normal numbers.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __int_as_float((e + 127) << 23); }

// Tiles of a symmetric product: only those that reach the diagonal or lie right of it.
__device__ __forceinline__ Tile tile_sym(int t, int tn, int bn) {
  int m = 0;
  for (int left = tn; t >= left; ++m) {
    t -= left;
    left -= 256 / bn;
  }
  return Tile{m, m * (256 / bn) + t};
}

// One phase as every role sees it.  Unit u of a phase is split u / tiles of tile
// u % tiles, which takes an even share of the k-slabs; only with at least as many pairs
// as units is K split, so that the splits of a tile, which wait for each other's sums, are
// all under way.
struct Phase {
  int M, N, bn, tm, tn, per, tiles, sym, k_slabs, splits, units;
  Operand A, B;
  __device__ __forceinline__ int k_at(int split) const { return k_slabs * split / splits; }
};
__device__ __forceinline__ Phase phase_at(const NsArgs& a, int step, int kind) {
  Phase f;
  f.bn = a.bn[kind];
  f.splits = a.splits[kind];
  f.sym = kind != NS_UPDATE;
  const int x = step & 1;
  int K = a.m;
  if (kind == NS_UPDATE) {
    f.M = a.rows; f.N = a.cols;
    if (a.tall) {
      f.A = Operand{&a.x_k[x], nullptr, 0};
      f.B = Operand{&a.b_col, &a.b_mn, 2};
    } else {
      f.A = Operand{&a.b_row, &a.b_mn, 2};
      f.B = Operand{nullptr, &a.x_mn[x], 1};
    }
  } else {
    f.M = f.N = a.m;
    if (kind == NS_SQUARE) {
      f.A = Operand{&a.a_row, &a.a_mn, 2};
      f.B = Operand{&a.a_col, &a.a_mn, 2};
    } else if (a.tall) {
      K = a.rows;
      f.A = f.B = Operand{nullptr, &a.x_mn[x], 1};
    } else {
      K = a.cols;
      f.A = Operand{&a.x_k[x], nullptr, 0};
      f.B = Operand{&a.x_kb[x], nullptr, 0};
    }
  }
  f.k_slabs = (K + 63) / 64;
  f.tm = (f.M + 255) / 256;
  f.tn = (f.N + f.bn - 1) / f.bn;
  f.per = a.per[kind];
  f.tiles = f.per * a.batch;
  f.units = f.tiles * f.splits;
  return f;
}
// The first of a phase's units that a pair takes, `base` units of the sequence before it.
__device__ __forceinline__ int first_unit(int base, int cluster, int clusters) {
  const int u = cluster - base;
  return u < 0 ? u + clusters : u;
}
// Units of one matrix that are done before a phase begins.
__device__ __forceinline__ unsigned ready_units(const NsArgs& a, int step, int kind) {
  const unsigned g = a.per[NS_GRAM] * a.splits[NS_GRAM], q = a.per[NS_SQUARE] * a.splits[NS_SQUARE],
                 u = a.per[NS_UPDATE] * a.splits[NS_UPDATE];
  return step * (g + q + u) + (kind > NS_GRAM ? g : 0) + (kind > NS_SQUARE ? q : 0);
}
__device__ __forceinline__ Tile phase_tile(const NsArgs& a, const Phase& f, int t) {
  return f.sym ? tile_sym(t, f.tn, f.bn) : tile_grouped(t, f.tm, f.tn, a.group_m);
}

// CTAs that scale batch entry b: the entries are shared out in teams, entry b to the CTAs
// c = b mod teams.
__device__ __forceinline__ unsigned ns_teams(const NsArgs& a) { return min((unsigned)a.batch, gridDim.x); }
__device__ __forceinline__ unsigned ns_team_size(const NsArgs& a, unsigned b) {
  const unsigned teams = ns_teams(a), team = b % teams;
  return (gridDim.x - team + teams - 1) / teams;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_chain_kernel(const __grid_constant__ NsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ unsigned int s_passed;    // this CTA's units whose matrix is ready for them
  // epilogue warps that have finished a unit, for four units in flight: a warp is never
  // three units ahead of another, since a unit's accumulator is the one two units before
  __shared__ unsigned int s_finished[4];
  if (threadIdx.x == 0) s_passed = s_finished[0] = s_finished[1] = s_finished[2] = s_finished[3] = 0u;
  Pair<S> p{};
  p.begin(smem_raw, a.status, a.wait_limit_ns, [&] {
    for (int w = 0; w < kPairEpiWarps; ++w) mbar_init(p.extra(w), 1);
  });
  const uint32_t warp = warp_id(), lane = lane_id();
  const int clusters = gridDim.x / 2, cluster = blockIdx.x / 2;
  // a wait on another CTA's word goes on: false once the limit is past or some CTA has
  // given up
  auto still = [&](uint64_t t0, uint32_t it) {
    const bool gone = *reinterpret_cast<volatile unsigned*>(a.words) != 0u;
    if (!gone && !*p.abort && globaltimer_ns() - t0 <= p.lim && it <= 0x7fffffffu) return true;
    *p.abort = 1;
    report(p.status, RA_ERR_TIMEOUT);
    return false;
  };

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        tma_prefetch_desc(&a.x_k[i]);
        tma_prefetch_desc(&a.x_kb[i]);
        tma_prefetch_desc(&a.x_mn[i]);
        tma_prefetch_desc(&a.hi_io[i]);
      }
      for (const CUtensorMap* m : {&a.a_row, &a.a_col, &a.a_mn, &a.b_row, &a.b_col, &a.b_mn, &a.lo_io, &a.a_io, &a.b_io})
        tma_prefetch_desc(m);
    }
    // ------------------------------------------------------------ producer
    // also waits for the units' matrices and tells the epilogue warps
    if (lane == 0) {
      uint32_t cnt = 0, passed = 0;
      unsigned seen = 0;
      int seen_b = -1, base = 0;
      bool ok = true;
      for (int step = 0; step < a.steps && ok; ++step) {
        for (int kind = NS_GRAM; kind <= NS_UPDATE && ok; ++kind) {
          const Phase f = phase_at(a, step, kind);
          for (int u = first_unit(base, cluster, clusters); u < f.units && ok; u += clusters) {
            const int s = u / f.tiles, t = u - s * f.tiles, b = t / f.per;
            const unsigned need = kPairEpiWarps * ns_team_size(a, b) + 2u * ready_units(a, step, kind);
            if (b != seen_b || seen < need) {  // counts only grow: often the last look still holds
              const unsigned* count = a.counts + b;
              const uint64_t t0 = globaltimer_ns();
              for (uint32_t it = 1;; ++it) {
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(count) : "memory");
                if (seen >= need) break;
                if ((it & 63u) == 0 && !still(t0, it)) { ok = false; break; }
              }
              if (!ok) break;
              seen_b = b;
              asm volatile("fence.proxy.async;" ::: "memory");
            }
            ++passed;
            asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(&s_passed)), "r"(passed) : "memory");
            const Tile tile = phase_tile(a, f, t - b * f.per);
            ok = p.produce(cnt, f.A, f.B, f.bn, tile.m * 256, tile.n * f.bn, b, f.k_at(s), f.k_at(s + 1));
          }
          base = (base + f.units) % clusters;
        }
      }
      if (!ok) atomicExch(a.words, 1u);
      if (*p.abort) p.producer_drain(cnt);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t cnt = 0, lt = 0;
    int base = 0;
    bool ok = true;
    for (int step = 0; step < a.steps && ok; ++step) {
      for (int kind = NS_GRAM; kind <= NS_UPDATE && ok; ++kind) {
        const Phase f = phase_at(a, step, kind);
        for (int u = first_unit(base, cluster, clusters); u < f.units && ok; u += clusters) {
          const int s = u / f.tiles, t = u - s * f.tiles;
          const Tile tile = phase_tile(a, f, t % f.per);
          ok = p.rank == 0 ? p.multiply(cnt, lt, 0, f.A, f.B, f.bn, tile.m * 256, tile.n * f.bn, f.k_at(s), f.k_at(s + 1))
                           : p.forward(lt);
        }
        base = (base + f.units) % clusters;
      }
    }
    if (p.rank == 0) p.multiply_drain();
  } else {
    // ------------------------------------------------------------ epilogue
    const int w = (int)warp - 2;
    const uint32_t quarter = warp & 3;  // TMEM lanes 32 * quarter .. + 31
    const int half = w >> 2;            // columns [half * bn / 2, + bn / 2)
    const uint32_t stage = p.sbase + S::kOut + w * 8192;
    uint8_t* const stage_p = p.smem + S::kOut + w * 8192;
    const uint32_t FILLED = p.extra(w);
    uint32_t loads = 0, fills = 0, lt = 0;  // staging loads issued and received
    // a 16-byte piece of the staging rows of 128 bytes, 128-byte swizzle; buf 0 or 1
    auto piece = [&](int buf, int j) {
      return reinterpret_cast<uint4*>(stage_p + buf * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4));
    };
    auto count = [&](int b) {
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counts + b) : "memory");
    };
    // What lane 0 wrote for the CTA's unit-th unit, one of matrix b, is done (copies and
    // partial sums); the last of the CTA's epilogue warps counts the unit.
    auto finish = [&](uint32_t unit, int b) {
      if (lane == 0) {
        bulk_wait_all();
        asm volatile("fence.proxy.async;" ::: "memory");
        const uint32_t slot = smem_u32(&s_finished[unit & 3]);
        unsigned before;
        asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(slot) : "memory");
        if (before == kPairEpiWarps - 1) {
          asm volatile("st.relaxed.cta.shared.u32 [%0], 0;" ::"r"(slot) : "memory");
          count(b);
        }
      }
      __syncwarp();
    };
    // ---- phase 0: X = sx G / (|G|_F + eps) as two fp16 terms
    {
      const unsigned chunks = (a.in.cols + 7) / 8, per = a.in.rows * chunks;
      const unsigned teams = ns_teams(a), team = blockIdx.x % teams;
      const unsigned id = (blockIdx.x / teams) * 256 + (threadIdx.x - 64), all = ns_team_size(a, team) * 256;
      for (int b = team; b < a.batch; b += teams) {
        float f[3];
        int shift;
        ns_factor(a.parts + (long long)b * kNsParts * 3, a.num_parts, a.sx, a.eps, f, &shift);
        if (id == 0) a.shifts[b] = shift;
        for (unsigned i = id; i < per; i += all * kNsBatch) {
          NsRaw g[kNsBatch];
#pragma unroll
          for (int k = 0; k < kNsBatch; ++k) {
            const unsigned q = i + k * all, r = q / chunks, c = (q - r * chunks) * 8;
            g[k] = load8(a.in, b * a.in.bstride + r * a.in.ld + c, q < per ? a.in.cols - (int)c : 0);
          }
#pragma unroll
          for (int k = 0; k < kNsBatch; ++k) {
            const unsigned q = i + k * all, r = q / chunks, c = (q - r * chunks) * 8;
            if (q >= per) break;
            float v[8];
            unpack8(a.in, g[k], v);
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = ((v[2 * j] * f[0]) * f[1]) * f[2], y = ((v[2 * j + 1] * f[0]) * f[1]) * f[2];
              h[j] = pack_half2(x, y);
              const float2 high = unpack_half2(h[j]);
              l[j] = pack_half2(x - high.x, y - high.y);
            }
            // rows are padded to a multiple of 64 elements: whole 16-byte pieces
            const long long o = ((long long)b * a.rows + r) * a.ld + c;
            *reinterpret_cast<uint4*>(a.hi0 + o) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(a.lo + o) = make_uint4(l[0], l[1], l[2], l[3]);
          }
        }
        asm volatile("fence.proxy.async;" ::: "memory");
        __threadfence();
        __syncwarp();
        if (lane == 0) count(b);
      }
    }
    bool ok = true;
    uint32_t units = 0;  // units this CTA has begun
    int base = 0;
    for (int step = 0; step < a.steps && ok; ++step) {
      const float* sums = a.sums[step & 1];
      float* sums_out = a.sums[(step + 1) & 1];
      const bool last = step == a.steps - 1;
      for (int kind = NS_GRAM; kind <= NS_UPDATE && ok; ++kind) {
        const Phase f = phase_at(a, step, kind);
        const int cols = f.bn / 2;
        for (int u = first_unit(base, cluster, clusters); u < f.units; u += clusters, ++lt) {
          const uint32_t acc = lt & 1;
          const int split = u / f.tiles, t = u - split * f.tiles, b = t / f.per;
          // the matrix is ready once the producer says so
          ++units;
          if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t it = 1;; ++it) {
              unsigned x;
              asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(x) : "r"(smem_u32(&s_passed)) : "memory");
              if (x >= units) break;
              if ((it & 255u) == 0 && !still(t0, it)) { ok = false; break; }
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
          __syncwarp();  // what lane 0 has acquired holds for every lane (the shuffle orders no memory)
          if (!ok) break;
          const uint32_t src = p.tmem + acc * 256 + half * cols + ((quarter * 32) << 16);
          // Splits share the finishing of their tile: of the 16 pieces of 32 rows x 64
          // columns that a CTA's warps hold (two each), split s finishes pieces s, s +
          // splits, ...; it leaves its sums of the others in memory, for the CTAs that
          // finish them, and takes theirs.  A column of 32 rows is one line.
          const long long mine =
              ((a.split_base[kind] + (long long)t * f.splits + split) * 2 + p.rank) * kPairEpiWarps + w;
          auto other = [&](int s) { return mine + (s - split) * 2 * kPairEpiWarps; };
          auto finishes = [&](int c) { return f.splits == 1 || (2 * w + (c >> 6)) % f.splits == split; };
          const unsigned now = step * 3 + kind + 1;
          const Tile tile = phase_tile(a, f, t - b * f.per);
          const int row0 = tile.m * 256 + (int)p.rank * 128 + (int)quarter * 32;
          const int row = row0 + (int)lane;
          const int col0 = tile.n * f.bn + half * cols;
          // GRAM writes through staging buffer 0; SQUARE reads A' and UPDATE the two
          // terms of X into the staging buffers, change them in place and write back
          auto prefetch = [&](int c) {
            if (lane == 0) {
              bulk_wait_read();
              if (kind != NS_GRAM) {
                mbar_arrive_expect_tx(FILLED, kind == NS_UPDATE ? 8192 : 4096);
                if (kind == NS_UPDATE) {
                  tma_load_3d(stage, &a.hi_io[step & 1], FILLED, col0 + c, row0, b);
                  tma_load_3d(stage + 4096, &a.lo_io, FILLED, col0 + c, row0, b);
                } else {
                  tma_load_3d(stage, &a.a_io, FILLED, col0 + c, row0, b);
                }
              }
            }
            __syncwarp();
            if (kind != NS_GRAM) ++loads;
          };
          int next = 0;  // the next piece to finish
          while (next < cols && !finishes(next)) next += 64;
          if (next < cols) prefetch(next);
          // X is held times 2^held in this step, its Gram matrix without; the new X times 2^then,
          // the result without
          const float shift = (float)__ldcg(a.shifts + b);
          const int held = max((int)floorf(shift - step * a.growth), 0);
          const int then = last ? 0 : max((int)floorf(shift - (step + 1) * a.growth), 0);
          const float gram_mul = pow2(-2 * held), new_mul = pow2(then - held);
          // alpha: the mean of the Gram matrix's diagonal, at first about 1 / m
          const float alpha =
              gram_mul *
              (step ? warp_total(sums + (long long)b * a.sums_ld, 16 * a.per[NS_UPDATE] * a.splits[NS_UPDATE]) * a.alpha_mul
                    : 1.f / (float)a.m);
          float sq = 0.f;  // UPDATE: squares of this warp's part of the new X
          const float lin = (a.cb + 2.f * a.cc * alpha) * a.square_lin;
          const float own = (a.ca + alpha * (a.cb + a.cc * alpha)) * new_mul, update_acc = a.update_acc * new_mul;
          const float gram_acc = a.gram_acc * gram_mul;
          const float diagonal = alpha * a.sa;
          if (!p.wait(p.acc_full(acc), (lt >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          if (f.splits > 1) {
            float* q = a.partials + mine * (128 * 32) + lane;
#pragma unroll 1
            for (int c = 0; c < cols; c += 64) {
              if (finishes(c)) continue;
              float v[64];
              tmem_load64(src + c, v);
#pragma unroll
              for (int j = 0; j < 64; ++j) __stcg(q + (c + j) * 32, v[j]);
            }
            __syncwarp();
            if (lane == 0)
              asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(a.flags + mine), "r"(now) : "memory");
            if (next >= cols) {
              p.release(acc);  // nothing to finish here
            } else {
              for (int s0 = 0; s0 < f.splits && ok; s0 += 32) {  // a flag per lane
                const int s = s0 + (int)lane;
                if (s < f.splits && s != split) {
                  const uint64_t t0 = globaltimer_ns();
                  for (uint32_t it = 1;; ++it) {
                    unsigned x;
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(a.flags + other(s)) : "memory");
                    if (x >= now) break;
                    if ((it & 63u) == 0 && !still(t0, it)) { ok = false; break; }
                  }
                }
                ok = __all_sync(0xffffffffu, ok);
              }
              __syncwarp();  // a lane reads the sums of all splits, whose flags other lanes acquired
            }
          }
          if (!ok) break;
          bool first = true;
#pragma unroll 1
          for (int c = next; c < cols; c = next, first = false) {
            for (next = c + 64; next < cols && !finishes(next);) next += 64;
            if (!first) prefetch(c);
            float v[64];
            tmem_load64(src + c, v);
            if (next >= cols) p.release(acc);
            for (int s = 0; s < f.splits; ++s) {
              if (s == split) continue;
              const float* q = a.partials + other(s) * (128 * 32) + lane + c * 32;
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] += __ldcg(q + j * 32);
            }
            if (kind != NS_GRAM) {
              if (!p.wait(FILLED, fills & 1)) { ok = false; break; }
              ++fills;
            }
            const bool inside = row0 < f.M && col0 + c < f.N;
            if (kind == NS_GRAM) {
              const int diag = row - col0 - c;  // this row's column of the diagonal
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = fmaf(v[j], gram_acc, j == diag ? -diagonal : 0.f);
            } else if (kind == NS_SQUARE) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 q = *piece(0, j);
                const uint32_t qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 g = unpack_half2(qq[i]);
                  v[8 * j + 2 * i] = fmaf(v[8 * j + 2 * i], a.square_acc, lin * g.x);
                  v[8 * j + 2 * i + 1] = fmaf(v[8 * j + 2 * i + 1], a.square_acc, lin * g.y);
                }
              }
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 q = *piece(0, j), r = *piece(1, j);
                const uint32_t qq[4] = {q.x, q.y, q.z, q.w}, rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 g = unpack_half2(qq[i]), e = unpack_half2(rr[i]);
                  v[8 * j + 2 * i] = fmaf(v[8 * j + 2 * i], update_acc, own * (g.x + e.x));
                  v[8 * j + 2 * i + 1] = fmaf(v[8 * j + 2 * i + 1], update_acc, own * (g.y + e.y));
                }
              }
            }
            if (kind == NS_UPDATE && last) {
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] *= a.out_mul;
              ns_write_rows<64>(a.out, a.out_dtype, a.out_vec, b * a.out_bstride + (long long)row0 * a.out_ld + col0 + c,
                                a.out_ld, f.M - row0, f.N - col0 - c, v, reinterpret_cast<float*>(stage_p));
              fence_proxy_async_smem();
              __syncwarp();
              continue;
            }
            // what lies past the edges came in as zeros on both sides
            if (kind == NS_UPDATE) {
              float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 64; ++j) s4[j & 3] = fmaf(v[j], v[j], s4[j & 3]);
              sq += (s4[0] + s4[1]) + (s4[2] + s4[3]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t hi[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) hi[i] = pack_half2(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
              *piece(0, j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              if (kind == NS_UPDATE) {
                uint32_t lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 g = unpack_half2(hi[i]);
                  lo[i] = pack_half2(v[8 * j + 2 * i] - g.x, v[8 * j + 2 * i + 1] - g.y);
                }
                *piece(1, j) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && inside) {
              if (kind == NS_UPDATE) {
                tma_store_3d(&a.hi_io[(step + 1) & 1], stage, col0 + c, row0, b);
                tma_store_3d(&a.lo_io, stage + 4096, col0 + c, row0, b);
              } else {
                tma_store_3d(kind == NS_GRAM ? &a.a_io : &a.b_io, stage, col0 + c, row0, b);
              }
              bulk_commit();
            }
          }
          if (!ok) break;
          if (kind == NS_UPDATE && !last) {
            sq = warp_sum(sq);
            if (lane == 0)
              sums_out[(long long)b * a.sums_ld +
                       (((t - b * f.per) * f.splits + split) * 2 + (int)p.rank) * kPairEpiWarps + w] = sq;
          }
          finish(units, b);
        }
        base = (base + f.units) % clusters;
      }
    }
    if (lane == 0) bulk_wait_all();
    // after a wait gave up: a staging load in flight lands before the CTA exits
    if (loads != fills) mbar_drain(FILLED, fills & 1);
  }
  p.end();
}

int ns_sumsq_blocks(const NsInput& in) {
  const long long chunks = (long long)in.rows * ((in.cols + 7) / 8);
  const long long n = (chunks + 1023) / 1024;
  return (int)(n < 1 ? 1 : n < kNsParts ? n : kNsParts);
}

// Pairs of CTAs that run at the same time on the current device (0: unknown yet).
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_pairs[kMaxDevices] = {};

}  // namespace

cudaError_t ns_max_pairs(int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_pairs[dev]) {
    e = cudaFuncSetAttribute(ns_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kAlloc;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, ns_chain_kernel, &cfg)) != cudaSuccess) return e;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    g_pairs[dev] = n < sms / 2 ? n : sms / 2;
  }
  *pairs = g_pairs[dev];
  return cudaSuccess;
}

int ns_phase_tiles(const NsArgs& a, int kind, int bn) {
  const int M = kind == NS_UPDATE ? a.rows : a.m, N = kind == NS_UPDATE ? a.cols : a.m;
  const int tm = (M + 255) / 256, tn = (N + bn - 1) / bn;
  if (kind == NS_UPDATE) return tm * tn;
  int n = 0;
  for (int m = 0; m < tm; ++m) n += tn - m * (256 / bn) > 0 ? tn - m * (256 / bn) : 0;
  return n;
}

cudaError_t launch_ns(NsArgs& a, int pairs, cudaStream_t st) {
  a.num_parts = ns_sumsq_blocks(a.in);
  ns_sumsq_kernel<<<dim3(a.num_parts, a.batch), 512, 0, st>>>(a.in, a.parts, a.words, kNsWords + a.batch);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, ns_chain_kernel, (const NsArgs&)a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaSuccess;
}

}  // namespace ra
