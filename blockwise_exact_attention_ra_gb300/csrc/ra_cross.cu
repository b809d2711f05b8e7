// The kernels around cross attention's products: the join of states over parts of the keys,
// the sizes of dO and v, fp16 operand copies, the backward pass's row terms and its last
// conversions.  All are bound by what they read and write.
#include <math.h>

#include "ra_device.cuh"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 256;

__device__ __forceinline__ int len_at(const int* kv_len, int b, int Nkv) {
  if (!kv_len) return Nkv;
  const int v = __ldg(kv_len + b);
  return v < 0 ? 0 : v > Nkv ? Nkv : v;
}

// Eight values as `dtype` at element i of p.
__device__ __forceinline__ void put8(void* p, int dtype, long long i, const float (&f)[8]) {
  if (dtype == RA_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else if (dtype == RA_BF16) {
    __align__(16) __nv_bfloat16 e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = __float2bfloat16_rn(f[j]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = *reinterpret_cast<const uint4*>(e);
  } else {
    __align__(16) __half e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = __float2half_rn(f[j]);
    *reinterpret_cast<uint4*>(static_cast<__half*>(p) + i) = *reinterpret_cast<const uint4*>(e);
  }
}
__device__ __forceinline__ void get8(const void* p, int dtype, long long i, float (&f)[8]) {
  if (dtype == RA_F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = s[0], b = s[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    return;
  }
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == RA_BF16) {
    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __bfloat162float(e[j]);
  } else {
    const __half* e = reinterpret_cast<const __half*>(&v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __half2float(e[j]);
  }
}
__device__ __forceinline__ bool past_fp16(const float (&f)[8]) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) bad |= fabsf(f[j]) > 65504.f && fabsf(f[j]) < INFINITY;
  return bad;
}

// Joins the states (m_s, l_s, o_s) of a row: m = max m_s, w_s = e^{m_s - m},
// o = sum w_s o_s / sum w_s l_s, lse = m + ln sum w_s l_s.  Parts that saw no key left no
// o_s.  W warps share a row's parts (a single one would wait for each four of up to 256 in
// turn: 45 us) and add up their sums in order; a lane holds d / 32 columns.
template <int W>
__global__ void __launch_bounds__(kThreads) cross_join_kernel(CrossState p, int splits, int B, int Nq, int Hq, int d, void* o,
                                                              int o_dtype, Lay ol, float* lse) {
  __shared__ float4 sums[kThreads / 32][32];
  __shared__ float totals[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % W;
  const long long rows = (long long)B * Nq * Hq, row = (long long)blockIdx.x * (kThreads / 32 / W) + warp / W;
  const bool there = row < rows;
  const int h = (int)(row % Hq);
  const long long bn = row / Hq;
  const int n = (int)(bn % Nq), b = (int)(bn / Nq);
  const long long at = ((long long)b * Hq + h) * Nq + n;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (there) {
    for (int s = lane; s < splits; s += 32) m = fmaxf(m, p.m[s * rows + at]);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    for (int s0 = share; s0 < splits; s0 += 32 * W) {  // lane j looks at part s0 + j W
      float w = 0.f;
      const int mine = s0 + lane * W;
      if (mine < splits) {
        w = ex2_approx((p.m[mine * rows + at] - ref) * kLog2e);
        const float ls = p.l[mine * rows + at];
        // a NaN stays one, whatever its part's maximum
        if (w > 0.f || ls != ls) l += w * ls;
      }
      const int last = min(32, (splits - s0 + W - 1) / W);
#pragma unroll 8
      for (int j = 0; j < last; ++j) {
        const float ws = __shfl_sync(0xffffffffu, w, j);
        if (!(ws > 0.f)) continue;
        const float* src = p.o + ((s0 + j * W) * rows + row) * d;
        if (d == 128) {
          const float4 v = reinterpret_cast<const float4*>(src)[lane];
          acc.x = fmaf(ws, v.x, acc.x);
          acc.y = fmaf(ws, v.y, acc.y);
          acc.z = fmaf(ws, v.z, acc.z);
          acc.w = fmaf(ws, v.w, acc.w);
        } else {
          const float2 v = reinterpret_cast<const float2*>(src)[lane];
          acc.x = fmaf(ws, v.x, acc.x);
          acc.y = fmaf(ws, v.y, acc.y);
        }
      }
    }
    l = warp_sum(l);
  }
  if (W > 1) {
    sums[warp][lane] = acc;
    if (lane == 0) totals[warp] = l;
    __syncthreads();
    if (share) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float4 v = sums[warp + w][lane];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      l += totals[warp + w];
    }
  }
  if (!there) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  const long long out = lay_at(ol, b, n, h);
  if (d == 128) {
    if (o_dtype == RA_F32) {
      reinterpret_cast<float4*>(static_cast<float*>(o) + out)[lane] = acc;
    } else {
      uint2 v;
      if (o_dtype == RA_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x, acc.y), y = __floats2bfloat162_rn(acc.z, acc.w);
        v = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      } else {
        v = make_uint2(pack_half2(acc.x, acc.y), pack_half2(acc.z, acc.w));
      }
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(o) + out)[lane] = v;
    }
  } else if (o_dtype == RA_F32) {
    reinterpret_cast<float2*>(static_cast<float*>(o) + out)[lane] = make_float2(acc.x, acc.y);
  } else if (o_dtype == RA_BF16) {
    reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(o) + out)[lane] = __floats2bfloat162_rn(acc.x, acc.y);
  } else {
    reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(o) + out)[lane] = pack_half2(acc.x, acc.y);
  }
  if (lane == 0) lse[at] = l == 0.f ? -INFINITY : m + logf(l);
}

// Keys and values as fp16, by blocks block, block + blocks, ...
__device__ __forceinline__ void copy_keys(const CrossKeysArgs& a, long long block, long long blocks) {
  const int per_row = a.Hkv * a.d / 8, dtype = a.bf16 ? RA_BF16 : RA_F16;
  const long long total = (long long)a.B * a.Nkv * per_row;
  bool bad = false;
  for (long long t = block * kThreads + threadIdx.x; t < total; t += blocks * kThreads) {
    const long long bn = t / per_row;
    const int e = (int)(t - bn * per_row) * 8, g = e / a.d, b = (int)(bn / a.Nkv), n = (int)(bn - (long long)b * a.Nkv);
    const bool there = n < len_at(a.kv_len, b, a.Nkv);
    const long long src = lay_at(a.kvl, b, n, g) + (e - g * a.d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const void* x = i ? a.v : a.k;
      void* y = i ? a.v16 : a.k16;
      if (!y) continue;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (there) {
        get8(x, dtype, src, f);
        bad |= past_fp16(f);
      }
      put8(y, RA_F16, t * 8, f);
    }
  }
  if (bad) report(a.status, RA_ERR_RANGE);
}

__global__ void __launch_bounds__(kThreads) cross_keys_kernel(const __grid_constant__ CrossKeysArgs a) {
  copy_keys(a, blockIdx.x, gridDim.x);
}

// Bounds of the norms of the rows of dO and of v for each key head (for cross_scale).  A lane
// keeps the largest sum of squares of its eight columns over the rows that it reads of a head; the root of
// the sum of these over a row's d / 8 lanes is at least every row's norm, and for values without a
// pattern less than twice the largest.  No lane needs another until the end: the sums row
// by row took 29 us instead of 23 for 67 MB, bound by instructions; what is left (16 us for 34 MB, 2 TB/s) are two
// or three rounds of loads behind the latency of a launch.  Sums that leave fp32's range are
// left out, so that infinities and NaN, which lose their own gradients whatever the scale, leave the
// others theirs; a lane that met some, or nothing larger than 2^-50, reads its rows again at another scale.
// It adds 6 us to 15 (77 queries, 590 keys, 8 heads of 128) and 28 to 648 (2 x 4096 x 4096, 16 heads of 128).
__global__ void __launch_bounds__(kThreads) cross_range_kernel(const __grid_constant__ CrossRangeArgs a) {
  pdl_trigger();
  const bool values = (int)blockIdx.x >= a.blocks;
  const CrossRangeArgs::Side& t = a.side[values];
  const int G = a.d / 8, slots = kThreads / G, slot = threadIdx.x / G;
  const int unit = (values ? blockIdx.x - a.blocks : blockIdx.x) / t.chunks, chunk = (values ? blockIdx.x - a.blocks : blockIdx.x) - unit * t.chunks;
  const int tiles = (t.H + t.heads - 1) / t.heads, b = unit / tiles, h = (unit - b * tiles) * t.heads + slot % t.heads;
  const int N = values ? len_at(a.kv_len, b, a.Nkv) : a.Nq, tokens = slots / t.heads, step = tokens * t.chunks;
  const bool mine = slot / t.heads < tokens && h < t.H;
  const int first = mine ? chunk * tokens + slot / t.heads : N;
  const uint16_t* x = static_cast<const uint16_t*>(t.x) + lay_at(t.l, b, 0, mine ? h : 0) + threadIdx.x % G * 8;
  bool left_out = false;
  auto largest = [&](float by) {
    float top = 0.f;
    for (long long n = first; n < N; n += 4ll * step) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = n + (long long)k * step < N ? *reinterpret_cast<const uint4*>(x + (n + (long long)k * step) * t.l.rs) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float sum = 0.f;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 f = a.bf16 ? make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)) : unpack_half2(w[j]);
          f.x *= by;
          f.y *= by;
          sum = fmaf(f.y, f.y, fmaf(f.x, f.x, sum));
        }
        left_out |= !(sum < 1e37f);
        if (sum < 1e37f) top = fmaxf(top, sum);
      }
    }
    return top;
  };
  // log2 of the largest sum; of those past fp32's range too, or of small ones where there is no other
  float own = log2f(largest(1.f));
  if (left_out) own = fmaxf(own, log2f(largest(8.470329472543003e-22f)) + 140.f);
  if (own < -99.f) own = fmaxf(own, log2f(largest(1.2676506002282294e30f)) - 200.f);
  // the lanes' sums, joined
  float most = own;
  for (int o = G >> 1; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  float sum = most == -INFINITY ? 0.f : exp2f(own - most);
  for (int o = G >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % G || most == -INFINITY) return;
  const int norm = (int)ceilf(8.f * (most + log2f(sum)) + 0.01f);
  int2* const range = a.range + (long long)b * a.Hkv + h / (t.H / a.Hkv);
  int* const to = values ? &range->y : &range->x;
  if (norm > *static_cast<volatile int*>(to)) atomicMax(to, norm);
}

// What the backward kernel needs, the query side by the first row_blocks blocks (d / 8 lanes
// a row (b, n, h), n up to Np), the key side by the others.
__global__ void __launch_bounds__(kThreads) cross_prepare_kernel(const __grid_constant__ CrossRowsArgs a,
                                                                 const __grid_constant__ CrossKeysArgs keys, int row_blocks) {
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= row_blocks) {
    copy_keys(keys, blockIdx.x - row_blocks, gridDim.x - row_blocks);
    return;
  }
  const int G = a.d / 8, lane = threadIdx.x % G, in_dtype = a.bf16 ? RA_BF16 : RA_F16;
  const unsigned rows = (unsigned)a.B * a.Np * a.Hq, step = row_blocks * (kThreads / G);  // up to 2^31 rows
  if (blockIdx.x == 0 && threadIdx.x < 64) a.sched[threadIdx.x] = 0u;
  bool bad = false;
  // the warp's rows end together: its lanes meet in the sums
  const unsigned first = blockIdx.x * (kThreads / G) + threadIdx.x / G, group = a.Hq / a.Hkv;
  for (unsigned base = first - (threadIdx.x % 32) / G; base < rows; base += step) {
    const unsigned i = base + (threadIdx.x % 32) / G, bn = i / a.Hq, h = i - bn * a.Hq, b = bn / a.Np, n = bn - b * a.Np;
    const bool there = i < rows && (int)n < a.Nq;
    float dot = 0.f, mul = 0.f;
    if (there) {
      const CrossScale sc = cross_scale(a.range, b * a.Hkv + h / group, a.bf16);
      mul = sc.mul;
      const long long src = lay_at(a.ql, b, n, h) + 8 * lane;
      const long long row = (((long long)b * a.Nq + n) * a.Hq + h) * a.d + 8 * lane;
      float f[8], g[8];
      get8(a.dO, in_dtype, src, f);
      get8(a.o, a.o_dtype, src, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] *= sc.copy;
        dot = fmaf(f[j], g[j], dot);
      }
      if (a.do16) {
        put8(a.do16, RA_F16, row, f);
        get8(a.q, in_dtype, src, g);
        bad |= past_fp16(g);
        put8(a.q16, RA_F16, row, g);
      }
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      put8(a.dq_acc, RA_F32, row, zero);
    }
    for (int o = G >> 1; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0 && i < rows) {
      const long long at = ((long long)b * a.Hq + h) * a.Np + n;
      const float lse = there ? a.lse[((long long)b * a.Hq + h) * a.Nq + n] : -INFINITY;
      const bool seen = lse != -INFINITY;
      a.D[at] = seen ? -dot * mul : 0.f;
      a.lse2[at] = seen ? (float)kCrossP - lse * kLog2e : -INFINITY;  // P = 0
    }
  }
  if (bad) report(a.status, RA_ERR_RANGE);
}

__global__ void __launch_bounds__(kThreads) cross_sum_kernel(const float* parts, int splits, int B, int Nkv, int Hkv, int d,
                                                             void* dk, void* dv, int dtype, Lay kvl) {
  pdl_trigger();
  pdl_wait();
  const int per_row = Hkv * d / 8;
  const long long plane = (long long)B * Nkv * Hkv * d, total = plane / 8;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < 2 * total; i += (long long)gridDim.x * kThreads) {
    const int which = i >= total;
    const long long t = i - which * total, bn = t / per_row;
    const int e = (int)(t - bn * per_row) * 8, g = e / d, b = (int)(bn / Nkv), n = (int)(bn - (long long)b * Nkv);
    float f[8], x[8];
    const float* src = parts + (long long)which * splits * plane + t * 8;
    get8(src, RA_F32, 0, f);
    for (int s = 1; s < splits; ++s) {
      get8(src, RA_F32, s * plane, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += x[j];
    }
    put8(which ? dv : dk, dtype, lay_at(kvl, b, n, g) + (e - g * d), f);
  }
}

__global__ void __launch_bounds__(kThreads) cross_dq_kernel(const float* acc, float scale, const int2* range, int bf16, int B,
                                                            int Nq, int Hq, int Hkv, int d, void* dq, int dtype, Lay ql) {
  pdl_wait();
  const unsigned G = d / 8, lane = threadIdx.x % G * 8, per = kThreads / G, rows = (unsigned)B * Nq * Hq, group = Hq / Hkv;
  for (unsigned i = blockIdx.x * per + threadIdx.x / G; i < rows; i += gridDim.x * per) {
    const unsigned bn = i / Hq, h = i - bn * Hq, b = bn / Nq, n = bn - b * Nq;
    float f[8];
    get8(acc, RA_F32, (long long)i * d + lane, f);
    const float mul = scale * cross_scale(range, b * Hkv + h / group, bf16).ds;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= mul;
    put8(dq, dtype, lay_at(ql, b, n, h) + lane, f);
  }
}

unsigned blocks_for(long long threads) {
  const long long b = (threads + kThreads - 1) / kThreads;
  return (unsigned)(b < 1 ? 1 : b > 152 * 16 ? 152 * 16 : b);
}

}  // namespace

cudaError_t launch_cross_join(const CrossState& part, int splits, int B, int Nq, int Hq, int d, void* o, int o_dtype,
                              Lay ol, float* lse, cudaStream_t st) {
  const long long rows = (long long)B * Nq * Hq;
  auto run = [&](auto kernel, int warps) {
    const int per = kThreads / 32 / warps;
    return launch_pdl(kernel, (int)((rows + per - 1) / per), kThreads, 0, st, part, splits, B, Nq, Hq, d, o, o_dtype, ol, lse);
  };
  const cudaError_t e = splits > 8 ? run(cross_join_kernel<8>, 8) : splits > 2 ? run(cross_join_kernel<2>, 2) : run(cross_join_kernel<1>, 1);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_cross_keys(const CrossKeysArgs& a, cudaStream_t st) {
  cross_keys_kernel<<<blocks_for((long long)a.B * a.Nkv * a.Hkv * a.d / 8), kThreads, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_cross_range(CrossRangeArgs& a, cudaStream_t st) {
  // a block's rows lie together: of heads where those do, else of tokens; four blocks an SM in all
  // (16 x 4000 keys of 2 heads of 128, 64 queries: the backward pass takes 111 us, with eight 117, with two 113)
  const int slots = kThreads / (a.d / 8);
  long long units[2], most[2], all = 0;
  for (int i = 0; i < 2; ++i) {
    CrossRangeArgs::Side& t = a.side[i];
    const int N = i ? a.Nkv : a.Nq;
    t.heads = t.l.hs > t.l.rs ? 1 : t.H < slots ? t.H : slots;
    units[i] = (long long)a.B * ((t.H + t.heads - 1) / t.heads);
    const long long tokens = 4 * (slots / t.heads);
    most[i] = (N + tokens - 1) / tokens;
    all += units[i] * most[i];
  }
  for (int i = 0; i < 2; ++i) {
    const long long want = most[i] * 152 * 4 / all + 1;
    a.side[i].chunks = (int)(want < most[i] ? want : most[i]);
  }
  a.blocks = (int)(units[0] * a.side[0].chunks);
  cross_range_kernel<<<(unsigned)(a.blocks + units[1] * a.side[1].chunks), kThreads, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_cross_prepare(const CrossRowsArgs& a, const CrossKeysArgs& keys, cudaStream_t st) {
  const unsigned rows = blocks_for((long long)a.B * a.Np * a.Hq * a.d / 8);
  const unsigned more = keys.k16 ? blocks_for((long long)keys.B * keys.Nkv * keys.Hkv * keys.d / 8) : 0;
  const cudaError_t e = launch_pdl(cross_prepare_kernel, (int)(rows + more), kThreads, 0, st, a, keys, (int)rows);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_cross_sum(const float* parts, int splits, int B, int Nkv, int Hkv, int d, void* dk, void* dv, int dtype,
                             Lay kvl, cudaStream_t st) {
  const cudaError_t e = launch_pdl(cross_sum_kernel, (int)blocks_for((long long)B * Nkv * Hkv * d / 4), kThreads, 0, st, parts,
                                   splits, B, Nkv, Hkv, d, dk, dv, dtype, kvl);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_cross_dq(const float* dq_acc, float scale, const int2* range, int bf16, int B, int Nq, int Hq, int Hkv, int d,
                            void* dq, int dtype, Lay ql, cudaStream_t st) {
  const cudaError_t e = launch_pdl(cross_dq_kernel, (int)blocks_for((long long)B * Nq * Hq * d / 8), kThreads, 0, st, dq_acc,
                                   scale, range, bf16, B, Nq, Hq, Hkv, d, dq, dtype, ql);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace ra
