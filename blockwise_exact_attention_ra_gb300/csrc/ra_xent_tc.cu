// The tensor-core products of the vocabulary cross entropy, on CTA pairs
// (ra_pair.cuh):
//   PAIR_STATS    logits' softmax statistics and the target's logit (forward)
//   PAIR_DLOGITS  gradient of one block's logits, recomputed from x and w in the same pieces
//   PAIR_STORE    dx = d W and dw = d^T x, whole or split along K, in one launch
// The logits themselves stay in TMEM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "ra_pair.cuh"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// 5 stages of 32 KB (4, 5 and 6 run alike); two staging buffers of 4 KB per epilogue warp.
using S = PairSmem<5, 8192, 0>;
// Three warpgroups: producer, MMA issuer and two idle warps; then the 8 epilogue warps.
// The logits' kernels give the first one's registers to the others: 40 + 2 x 232 = 3 x 168.
constexpr int kThreads = 384;
// The logits' kernels add the tensor core's sums of at most 12 k-slabs (768 products) up in
// registers: the accumulator rounds towards zero, which over 2048 products left logits of
// 16 off by 1e-5 and the loss of a sure token by as much.  Errors of loss and lse on 8192 x
// 131072 x 2048 (2-norm, relative), and the time of the kernel by itself: whole 1.5e-6, 2.37
// ms; 16 slabs 7e-7, 2.46 ms; 12 slabs 5e-7, 2.49 ms; 4 slabs 2e-7, 2.80 ms; a sum in fp32 has
// 4e-7.  The backward needs the forward's very logits: with sums of its own over the whole of D
// the gradients of tokens with losses of 1e-4 to 1e-3 were off by 0.13 to 0.75 of their norm (now
// 4e-3), for 1382 us a step instead of 1415 (4096 x 32768 x 2048).
constexpr int kChunk = 12;
__device__ __forceinline__ int chunk_slabs(int slabs) {
  const int chunks = (slabs + kChunk - 1) / kChunk;
  return (slabs + chunks - 1) / chunks;
}

// The units of one or two problems shared out over the pairs.  A unit is a tile, or one
// split of its K.  The first problem's units go round the pairs; where the last round
// leaves pairs idle, those take as many of the second's as fit into one unit of the first
// (by k-slabs; a unit takes 6 slabs' time at least, its epilogue); the rest goes round
// again, beginning with them.  With dx (128 tiles of 128
// slabs) and dw (256 of 64) on 76 pairs the longest share is 448 slabs; in launches of
// their own they take 2 x 128 + 4 x 64 = 512.
struct Share {
  int units0, units1, pairs, pair, over, fill, mine0;
  __device__ __forceinline__ Share(const PairArgs& a, int pair_, int pairs_) : pairs(pairs_), pair(pair_) {
    const int cost0 = max(slabs(a.q[0]), 6), cost1 = a.problems > 1 ? max(slabs(a.q[1]), 6) : 1;
    units0 = tiles(a.q[0]) * a.q[0].splits;
    units1 = a.problems > 1 ? tiles(a.q[1]) * a.q[1].splits : 0;
    over = units0 % pairs;                                        // pairs of the last round
    mine0 = units0 / pairs + (pair < over ? 1 : 0);
    fill = over ? (cost0 + cost1 / 2) / cost1 : 0;                // units of the second that fill it up
  }
  static __device__ __forceinline__ int tiles(const PairProblem& q) {
    return ((q.M + 255) / 256) * ((q.N + q.bn - 1) / q.bn);
  }
  static __device__ __forceinline__ int slabs(const PairProblem& q) { return ((q.K + 63) / 64 + q.splits - 1) / q.splits; }
  // The n-th unit of this pair: index within its problem, the problem in *which; -1: none.
  __device__ __forceinline__ int unit(int n, int* which) const {
    *which = 0;
    if (n < mine0) return pair + n * pairs;
    *which = 1;
    n -= mine0;
    const int idle = pairs - over;
    int place = pair - over;  // the idle pairs come first
    if (place >= 0) {
      if (n < fill) {
        const int j = place + n * idle;
        return j < units1 ? j : -1;
      }
      n -= fill;
    } else {
      place += pairs;
    }
    const int j = (over ? fill * idle : 0) + place + n * pairs;
    return j < units1 ? j : -1;
  }
};

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    xent_pair_kernel(const __grid_constant__ PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  Pair<S> p{};
  p.begin(smem_raw, a.status, a.wait_limit_ns, [] {});
  pdl_trigger();
  pdl_wait();
  const uint32_t warp = warp_id(), lane = lane_id();
  const Share share(a, blockIdx.x / 2, gridDim.x / 2);
  // split s of a problem takes an even share of the k-slabs
  // (k-slabs times splits stay below 2^24 * 76)
  auto k_at = [&](const PairProblem& q, int s) {
    const unsigned slabs = (q.K + 63) / 64;
    return (int)(q.splits == 1 ? (s ? slabs : 0u) : slabs * s / q.splits);
  };
  int which = 0, u = 0;

  if (warp >= 4) {
    if (EPI != PAIR_STORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const uint32_t quarter = warp & 3;      // TMEM lanes 32 * quarter .. + 31
    const int half = (int)(warp - 4) >> 2;  // columns [half * bn / 2, + bn / 2)
    const uint32_t stage = p.sbase + S::kOut + (warp - 4) * 8192;
    uint8_t* const stage_p = p.smem + S::kOut + (warp - 4) * 8192;
    // one 16-byte piece of staging rows of 128 bytes, 128-byte swizzle; buffer 0 or 1
    auto stage16 = [&](int buf, int piece, uint4 v) {
      *reinterpret_cast<uint4*>(stage_p + buf * 4096 + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
    };
    // A bulk group per buffer filled, also where there is nothing to copy.  With the buffers
    // taken in turn, waiting for all groups but the latest frees the one that is next.
    auto stage_out = [&](auto issue) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        issue();
        bulk_commit();
      }
    };
    // 64 columns as 16-bit values into buffer buf
    auto stage64 = [&](int buf, const float* v, int bf) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        stage16(buf, j, make_uint4(pack_pair(v[8 * j], v[8 * j + 1], bf), pack_pair(v[8 * j + 2], v[8 * j + 3], bf),
                                   pack_pair(v[8 * j + 4], v[8 * j + 5], bf), pack_pair(v[8 * j + 6], v[8 * j + 7], bf)));
    };
    int buf = 0;  // the next buffer
    uint32_t lt = 0;
    for (int n = 0; (u = share.unit(n, &which)) >= 0; ++n, ++lt) {
      const PairProblem& q = a.q[which];
      const uint32_t b = lt & 1;
      const int bn = q.bn, cols = bn / 2;
      const int tm = (q.M + 255) / 256, tn = (q.N + bn - 1) / bn, split = u / (tm * tn);
      const Tile t = tile_grouped(u - split * tm * tn, tm, tn, q.group_m);
      const int row0 = t.m * 256 + (int)p.rank * 128 + (int)quarter * 32;
      const int row = row0 + (int)lane;
      const int col0 = t.n * bn + half * cols;
      const uint32_t from = p.tmem + half * cols + ((quarter * 32) << 16);

      float z[EPI == PAIR_STORE ? 1 : 128];
      if (EPI != PAIR_STORE) {
        // The logits of the tile's columns for this row, the same bits in both passes: the
        // gradient of a sure token is what is left of z - lse.
        const int slabs = (q.K + 63) / 64, chunk = chunk_slabs(slabs);
        bool ok = true;
        for (int k0 = 0; k0 < slabs; k0 += chunk, ++lt) {
          const uint32_t acc = lt & 1;
          ok = p.wait(p.acc_full(acc), (lt >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (row0 < q.M && col0 < q.N) {
            const uint32_t src = from + acc * 256;
            if (k0 == 0) {
              tmem_load64(src, z);
              if (cols > 64) tmem_load64(src + 64, z + 64);
            } else {
#pragma unroll
              for (int c = 0; c < 128; c += 32) {
                if (c < cols) {
                  float v[32];
                  tmem_load32(src + c, v);
#pragma unroll
                  for (int j = 0; j < 32; ++j) z[c + j] += v[j];
                }
              }
            }
          }
          p.release(acc);
        }
        if (!ok) break;
        --lt;  // counted once more at the end of the loop
        if (row0 >= q.M || col0 >= q.N) continue;
      }
      if (EPI == PAIR_STATS) {
        // Softmax statistics of these columns, and the target's logit where it lies among
        // them.  Bound by the matrix product.
        const long long y = row < q.M ? a.targets[row] : -1;
        const int ycol = (y >= col0 && y < col0 + cols) ? (int)(y - col0) : -1;
        float m = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (c < cols) {
            if (col0 + c + 32 > q.N) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (col0 + c + j >= q.N) z[c + j] = -INFINITY;
            }
            float mk[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mk[k] = fmax3(z[c + k], z[c + k + 4], z[c + k + 8]);
#pragma unroll
            for (int j = 12; j < 28; j += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mk[k] = fmax3(mk[k], z[c + j + k], z[c + j + 4 + k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) mk[k] = fmaxf(mk[k], z[c + 28 + k]);
            m = fmax3(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]), m);
          }
        }
        // with no finite logit the sum is 0 (-inf - (-inf) is not formed)
        const float ref = m == -INFINITY ? 0.f : m * kLog2e;
        const float2 log2e = make_float2(kLog2e, kLog2e), off = make_float2(-ref, -ref);
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (c < cols) {
            if (__any_sync(0xffffffffu, ycol >= c && ycol < c + 32)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (ycol == c + j) a.target_logit[row] = z[c + j];
            }
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 e = __ffma2_rn(make_float2(z[c + j], z[c + j + 1]), log2e, off);
              s2[(j / 2) & 1] = __fadd2_rn(s2[(j / 2) & 1], make_float2(ex2_approx(e.x), ex2_approx(e.y)));
            }
          }
        }
        if (row < q.M)
          a.stats[(long long)(t.n * 2 + half) * q.M + row] =
              make_float2(m, (s2[0].x + s2[1].x) + (s2[0].y + s2[1].y));
        continue;
      }
      if (EPI == PAIR_DLOGITS) {
        // d = g (e^{z - lse} - [column = target]), rounded to the operand type of
        // the two products that follow (bf16: any range; fp16: g is brought near
        // 2^13 by a power of two that those products take out again).  With few rows a
        // gradient is little more than one element of d times a row of w or x, whose
        // rounding nothing averages out: there what it takes away is kept as a second term.
        const long long y = row < q.M ? a.targets[row] : a.ignore;
        const bool live = row < q.M && y != a.ignore && y >= 0 && y < a.vocab;
        const float g = live ? a.grad[row] * (a.scale ? a.scale[0] : 1.f) : 0.f;
        const float lse = live ? a.lse[row] : 0.f;
        const long long yc = y - a.col_off - col0;
        const int ycol = (live && yc >= 0 && yc < cols) ? (int)yc : -1;
        const float2 log2e = make_float2(kLog2e, kLog2e), off = make_float2(-lse, -lse), gg = make_float2(g, g);
#pragma unroll
        for (int c = 0; c < 128; c += 64) {
          if (c >= cols) break;
          if (lane == 0) {
            if (a.two_terms) bulk_wait_read();
            else bulk_wait_read_but_one();
          }
          float* const v = z + c;
          const bool target = __any_sync(0xffffffffu, ycol >= c && ycol < c + 64);
          float own = 0.f;
          if (target) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (ycol == c + j) own = v[j];
            own = logit_gradient(own - lse, true);
          }
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const float2 e = __fmul2_rn(__fadd2_rn(make_float2(v[j], v[j + 1]), off), log2e);
            v[j] = ex2_approx(e.x);
            v[j + 1] = ex2_approx(e.y);
          }
          if (target) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (ycol == c + j) v[j] = own;
          }
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const float2 e = __fmul2_rn(make_float2(v[j], v[j + 1]), gg);
            v[j] = live ? e.x : 0.f;  // a row without loss may hold anything
            v[j + 1] = live ? e.y : 0.f;
          }
          __syncwarp();
          stage64(buf, v, a.ab_bf16);
          stage_out([&]() {
            if (col0 + c < q.N) tma_store_3d(&q.tm_c, stage + buf * 4096, col0 + c, row0, 0);
          });
          if (a.two_terms) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              v[j] -= a.ab_bf16 ? to_f32(__float2bfloat16_rn(v[j])) : to_f32(__float2half_rn(v[j]));
            stage64(buf ^ 1, v, a.ab_bf16);
            stage_out([&]() {
              if (col0 + c < q.N) tma_store_3d(&q.tm_c, stage + (buf ^ 1) * 4096, col0 + c, row0, 1);
            });
          }
          buf ^= 1;
        }
      } else {
        if (!p.wait(p.acc_full(b), (lt >> 1) & 1)) break;
        tc_fence_after();
        const uint32_t src = from + b * 256;
        if (row0 >= q.M || col0 >= q.N) {  // nothing of this warp's part is inside
          p.release(b);
          continue;
        }
        // c = mul * acc (+ c_add): 16-bit or fp32 out; fp32 may be added to what is
        // there (each element once per launch, so the sum's order is fixed).  Split
        // along K, each split has a plane of its own.
        const float mul = a.scale ? a.scale[1] : 1.f;
        const bool f32 = q.c_dtype == RA_F32;
#pragma unroll 1
        for (int c = 0; c < cols; c += 64) {
          // fp32 takes both buffers at once, 16-bit values one at a time
          if (lane == 0) {
            if (f32) bulk_wait_read();
            else bulk_wait_read_but_one();
          }
          float v[64];
          tmem_load64(src + c, v);
          if (c == cols - 64) p.release(b);
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] *= mul;
          __syncwarp();
          if (f32) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              stage16(j >> 3, j & 7, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
            // a group for each buffer; buffer 1's is the latest, so a 16-bit piece that follows
            // takes buffer 0
            stage_out([&]() {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int cc = col0 + c + 32 * h;
                if (cc < q.N) {
                  if (q.c_accumulate) tma_add_3d(&q.tm_c, stage + h * 4096, cc, row0, split);
                  else tma_store_3d(&q.tm_c, stage + h * 4096, cc, row0, split);
                }
                if (h == 0) bulk_commit();
              }
            });
            buf = 0;
          } else {
            if (q.c_add && row < q.M) {  // N is a multiple of 8 where c_add is used
              const float4* add = reinterpret_cast<const float4*>(q.c_add + (long long)row * q.N + col0 + c);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (col0 + c + 4 * j < q.N) {
                  const float4 f = add[j];
                  v[4 * j] += f.x;
                  v[4 * j + 1] += f.y;
                  v[4 * j + 2] += f.z;
                  v[4 * j + 3] += f.w;
                }
              }
            }
            stage64(buf, v, q.c_dtype == RA_BF16);
            stage_out([&]() {
              if (col0 + c < q.N) tma_store_3d(&q.tm_c, stage + buf * 4096, col0 + c, row0, 0);
            });
            buf ^= 1;
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else {
    if (EPI != PAIR_STORE) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      if (lane == 0) {
        uint32_t cnt = 0;
        bool ok = true;
        for (int n = 0; ok && (u = share.unit(n, &which)) >= 0; ++n) {
          const PairProblem& q = a.q[which];
          const int tm = (q.M + 255) / 256, tn = (q.N + q.bn - 1) / q.bn, s = u / (tm * tn);
          const Tile t = tile_grouped(u - s * tm * tn, tm, tn, q.group_m);
          const Operand A{&q.tm_a, &q.tm_a, q.a_mn}, B{&q.tm_b, &q.tm_b, q.b_mn};
          ok = p.produce(cnt, A, B, q.bn, t.m * 256, t.n * q.bn, 0, k_at(q, s), k_at(q, s + 1), q.a_rows, q.fold);
        }
        if (*p.abort) p.producer_drain(cnt);
      }
    } else if (warp == 1) {
      uint32_t cnt = 0, lt = 0;
      bool ok = true;
      for (int n = 0; ok && (u = share.unit(n, &which)) >= 0; ++n) {
        const PairProblem& q = a.q[which];
        const int s = u / Share::tiles(q);
        const Operand A{nullptr, nullptr, q.a_mn}, B{nullptr, nullptr, q.b_mn};
        const int k1 = k_at(q, s + 1);
        for (int k0 = k_at(q, s); ok && k0 < k1;) {
          const int k = EPI != PAIR_STORE ? min(k0 + chunk_slabs(k1), k1) : k1;  // one split: k1 slabs
          ok = p.rank == 0 ? p.multiply(cnt, lt, a.ab_bf16, A, B, q.bn, 0, 0, k0, k) : p.forward(lt);
          k0 = k;
        }
      }
      if (p.rank == 0) p.multiply_drain();
    }
  }
  p.end();
}

}  // namespace

cudaError_t launch_xent_pair(const PairArgs& a, int num_sms, cudaStream_t st) {
  if (a.problems < 1 || a.problems > 2 || (a.problems > 1 && a.epi != PAIR_STORE) || num_sms < 2)
    return cudaErrorInvalidValue;
  long long units = 0;
  for (int i = 0; i < a.problems; ++i) {
    const PairProblem& q = a.q[i];
    if (q.M <= 0 || q.N <= 0 || q.K <= 0 || q.group_m <= 0 || (q.bn != 128 && q.bn != 256) || q.splits < 1 ||
        q.splits > (q.K + 63) / 64)
      return cudaErrorInvalidValue;
    units += (long long)((q.M + 255) / 256) * ((q.N + q.bn - 1) / q.bn) * q.splits;
  }
  if (units > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = num_sms / 2;
  const int grid = 2 * (int)(units < pairs ? units : pairs);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto run = [&](auto epi) {
    auto kernel = xent_pair_kernel<decltype(epi)::value>;
    // the attribute is set once per device (setting it twice does no harm)
    static std::atomic<unsigned long long> ready{0};
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(ready.load(std::memory_order_acquire) & bit)) {
      const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
      if (err != cudaSuccess) return err;
      if (dev <= 63) ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_pdl(kernel, grid, kThreads, S::kAlloc, st, a);
  };
  switch (a.epi) {
    case PAIR_STATS: e = run(std::integral_constant<int, PAIR_STATS>{}); break;
    case PAIR_DLOGITS: e = run(std::integral_constant<int, PAIR_DLOGITS>{}); break;
    case PAIR_STORE: e = run(std::integral_constant<int, PAIR_STORE>{}); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaSuccess;
}

}  // namespace ra
