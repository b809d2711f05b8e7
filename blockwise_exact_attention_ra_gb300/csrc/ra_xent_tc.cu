// The tensor-core products of the vocabulary cross entropy, on CTA pairs
// (ra_pair.cuh):
//   PAIR_STATS    logits' softmax statistics and the target's logit (forward)
//   PAIR_DLOGITS  gradient of one block's logits, recomputed from x and w
//   PAIR_STORE    dx = d W and dw = d^T x, whole or split along K
// The logits themselves stay in TMEM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "ra_pair.cuh"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
using S = PairSmem<6, 4096, 0>;  // 6 stages of 32 KB, 4 KB of staging per epilogue warp

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    xent_pair_kernel(const __grid_constant__ PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  Pair<S> p;
  p.begin(smem_raw, a.status, a.wait_limit_ns, [] {});
  const uint32_t warp = warp_id(), lane = lane_id();
  const int clusters = gridDim.x / 2, cluster = blockIdx.x / 2;
  const int bn = a.bn;
  const int tm = (a.M + 255) / 256, tn = (a.N + bn - 1) / bn;
  const int tiles = tm * tn, units = tiles * a.splits;
  const int k_steps = (a.K + 63) / 64;
  // unit u: tile u % tiles of split u / tiles, which takes an even share of the k-slabs
  auto k_at = [&](int s) { return (int)((long long)k_steps * s / a.splits); };
  const Operand A{&a.tm_a, &a.tm_a, a.a_mn}, B{&a.tm_b, &a.tm_b, a.b_mn};

  if (warp == 0) {
    if (lane == 0) {
      uint32_t cnt = 0;
      bool ok = true;
      for (int u = cluster; u < units && ok; u += clusters) {
        const int s = u / tiles;
        const Tile t = tile_grouped(u - s * tiles, tm, tn, a.group_m);
        ok = p.produce(cnt, A, B, bn, t.m * 256, t.n * bn, 0, k_at(s), k_at(s + 1));
      }
      if (*p.abort) p.producer_drain(cnt);
    }
  } else if (warp == 1) {
    uint32_t cnt = 0, lt = 0;
    bool ok = true;
    for (int u = cluster; u < units && ok; u += clusters) {
      const int s = u / tiles;
      ok = p.rank == 0 ? p.multiply(cnt, lt, a.ab_bf16, A, B, bn, 0, 0, k_at(s), k_at(s + 1)) : p.forward(lt);
    }
    if (p.rank == 0) p.multiply_drain();
  } else {
    const uint32_t quarter = warp & 3;      // TMEM lanes 32 * quarter .. + 31
    const int half = (int)(warp - 2) >> 2;  // columns [half * bn / 2, + bn / 2)
    const int cols = bn / 2;
    const uint32_t stage = p.sbase + S::kOut + (warp - 2) * 4096;
    uint8_t* const stage_p = p.smem + S::kOut + (warp - 2) * 4096;
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
    uint32_t lt = 0;
    for (int u = cluster; u < units; u += clusters, ++lt) {
      const uint32_t b = lt & 1;
      const int split = u / tiles;
      const Tile t = tile_grouped(u - split * tiles, tm, tn, a.group_m);
      const int row0 = t.m * 256 + (int)p.rank * 128 + (int)quarter * 32;
      const int row = row0 + (int)lane;
      const int col0 = t.n * bn + half * cols;
      if (!p.wait(p.acc_full(b), (lt >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t src = p.tmem + b * 256 + half * cols + ((quarter * 32) << 16);

      if (EPI == PAIR_STATS) {
        // Online softmax statistics of the tile's columns for this row, and the
        // target's logit where it lies among them.  Bound by the matrix product;
        // the exponentials (bn / 2 per thread and tile) hide behind it for K > 256.
        const long long y = row < a.M ? a.targets[row] : -1;
        const int ycol = (y >= col0 && y < col0 + cols) ? (int)(y - col0) : -1;
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          float v[32];
          tmem_load32(src + c, v);
          if (c == cols - 32) p.release(b);
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
          // a row without a finite logit so far keeps l = 0 (-inf - (-inf) is not formed)
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
        if (row < a.M && col0 < a.N) a.stats[(long long)(t.n * 2 + half) * a.M + row] = make_float2(m, l);
      } else if (EPI == PAIR_DLOGITS) {
        // d = g (e^{z - lse} - [column = target]), rounded to the operand type of
        // the two products that follow (bf16: any range; fp16: g is brought near
        // 2^13 by a power of two that those products take out again)
        const long long y = row < a.M ? a.targets[row] : a.ignore;
        const bool live = row < a.M && y != a.ignore && y >= 0 && y < a.vocab;
        const float g = live ? a.grad[row] * (a.scale ? a.scale[0] : 1.f) : 0.f;
        const float lse2 = live ? a.lse[row] * kLog2e : 0.f;
        const long long yc = y - a.col_off - col0;
        const int ycol = (live && yc >= 0 && yc < cols) ? (int)yc : -1;
#pragma unroll 1
        for (int c = 0; c < cols; c += 64) {
          stage_free();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int cc = c + 32 * h;
            float v[32];
            tmem_load32(src + cc, v);
            if (cc == cols - 32) p.release(b);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = ex2_approx(fmaf(v[j], kLog2e, -lse2));
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
            if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_c, stage, col0 + c, row0, 0);
          });
        }
      } else {
        // c = mul * acc (+ c_add): 16-bit or fp32 out; fp32 may be added to what is
        // there (each element once per launch, so the sum's order is fixed).  Split
        // along K, each split has a plane of its own.
        const float mul = a.scale ? a.scale[1] : 1.f;
        if (a.c_dtype == RA_F32) {
#pragma unroll 1
          for (int c = 0; c < cols; c += 32) {
            stage_free();
            float v[32];
            tmem_load32(src + c, v);
            if (c == cols - 32) p.release(b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stage16(j, make_uint4(__float_as_uint(v[4 * j] * mul), __float_as_uint(v[4 * j + 1] * mul),
                                    __float_as_uint(v[4 * j + 2] * mul), __float_as_uint(v[4 * j + 3] * mul)));
            stage_out([&]() {
              if (row0 < a.M && col0 + c < a.N) {
                if (a.c_accumulate) tma_add_3d(&a.tm_c, stage, col0 + c, row0, split);
                else tma_store_3d(&a.tm_c, stage, col0 + c, row0, split);
              }
            });
          }
        } else {
          const int bf = a.c_dtype == RA_BF16;
#pragma unroll 1
          for (int c = 0; c < cols; c += 64) {
            stage_free();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int cc = c + 32 * h;
              float v[32];
              tmem_load32(src + cc, v);
              if (cc == cols - 32) p.release(b);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= mul;
              if (a.c_add && row < a.M) {  // N is a multiple of 8 where c_add is used
                const float4* q = reinterpret_cast<const float4*>(a.c_add + (long long)row * a.N + col0 + cc);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  if (col0 + cc + 4 * j < a.N) {
                    const float4 f = q[j];
                    v[4 * j] += f.x;
                    v[4 * j + 1] += f.y;
                    v[4 * j + 2] += f.z;
                    v[4 * j + 3] += f.w;
                  }
                }
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                stage16(4 * h + j,
                        make_uint4(pack_pair(v[8 * j], v[8 * j + 1], bf), pack_pair(v[8 * j + 2], v[8 * j + 3], bf),
                                   pack_pair(v[8 * j + 4], v[8 * j + 5], bf), pack_pair(v[8 * j + 6], v[8 * j + 7], bf)));
            }
            stage_out([&]() {
              if (row0 < a.M && col0 + c < a.N) tma_store_3d(&a.tm_c, stage, col0 + c, row0, 0);
            });
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  p.end();
}

}  // namespace

cudaError_t launch_xent_pair(const PairArgs& a, int num_sms, cudaStream_t st) {
  if (a.M <= 0 || a.N <= 0 || a.K <= 0 || a.group_m <= 0 || num_sms < 2 || (a.bn != 128 && a.bn != 256) ||
      a.splits < 1 || a.splits > (a.K + 63) / 64)
    return cudaErrorInvalidValue;
  const long long units = (long long)((a.M + 255) / 256) * ((a.N + a.bn - 1) / a.bn) * a.splits;
  if (units > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = num_sms / 2;
  const int grid = 2 * (int)(units < pairs ? units : pairs);
  auto run = [&](auto epi) {
    auto kernel = xent_pair_kernel<decltype(epi)::value>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
    if (err != cudaSuccess) return err;
    kernel<<<grid, kPairThreads, S::kAlloc, st>>>(a);
    return cudaGetLastError();
  };
  cudaError_t e;
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
