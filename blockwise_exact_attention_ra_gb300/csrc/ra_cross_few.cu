// Cross attention of a few queries (single tokens, drafted ones) against many keys: bound
// by reading K and V once.
//
// A block takes one key/value head of one batch entry and one part of its keys; the query
// rows of the heads that share it (Nq Hq / Hkv <= 32) are the rows of m16n8k16 products, so
// that K and V are read once for all of them.  Its four warps take blocks of 16 keys in
// turn, each through a ring of its own in shared memory that cp.async fills (rows past the
// length with zeros: 0 x NaN would not be 0), and keep their own online-softmax state;
// nothing is waited for but a warp's own copies until the four states are joined at the end.
// Then up to eight blocks with parts of the same keys, a cluster, join theirs through
// distributed shared memory, each some of the rows; more parts are joined by a kernel.
//
// Measured (bf16, d 128, a token each): 16 entries of 4096 keys, 8 key heads of four query
// heads, two parts: 44 us, 6.1 TB/s (46 us with a kernel for the join); 131072 keys, 8 heads:
// 85 us, 6.3 TB/s.  20 rows (two tiles of products, all registers, eight warps an SM) against
// 131072 keys of 4 heads, fp16: 55 us, 4.9 TB/s.
//
// Products are fp32 sums of the inputs as they are; P enters the second as two terms of
// their type, hi and P - hi (rounding 2^-17 relative for bf16, 2^-23 for fp16: the tensor
// cores have time for it).  The running maximum is raised lazily, as in ra_fwd_tc.cu.
#include <math.h>

#include <type_traits>

#include "ra_device.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kKeys = 16, kStages = 3;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct FewSmem {
  static constexpr int kTile = kKeys * D * 2;          // K or V of 16 keys
  static constexpr int kWarp = kStages * 2 * kTile;
  static constexpr int kBytes = kWarps * kWarp;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x, y as a pair of T, and what that rounding takes from them as another
template <typename T>
__device__ __forceinline__ void two_terms(float x, float y, uint32_t* hi, uint32_t* lo) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    *hi = pack_half2(x, y);
    const float2 h = unpack_half2(*hi);
    *lo = pack_half2(x - h.x, y - h.y);
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The shared address of this block's `addr` in block `rank` of the cluster, and reads there.
__device__ __forceinline__ uint32_t shared_of(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 read2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 read4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kThreads) cross_few_kernel(const __grid_constant__ CrossFewArgs a) {
  using L = FewSmem<D>;
  constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // 16-byte pieces of a row; rows a warp copies at a time
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 states[kWarps][16 * MT], joined[16 * MT];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.Hq / a.Hkv, rows = a.Nq * group;
  const int unit = blockIdx.x / a.splits, split = blockIdx.x - unit * a.splits;
  const int b = unit / a.Hkv, g = unit - b * a.Hkv;
  int len = a.Nkv;
  if (a.kv_len) {
    const int v = __ldg(a.kv_len + b);
    len = v < 0 ? 0 : v > a.Nkv ? a.Nkv : v;
  }
  const int blocks = (len + kKeys - 1) / kKeys, per = (blocks + a.splits - 1) / a.splits;
  const int first = split * per, last = min(blocks, first + per);
  const int count = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;  // of this warp
  const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
  const T* kbase = static_cast<const T*>(a.k) + lay_at(a.kvl, b, 0, g);
  const T* vbase = static_cast<const T*>(a.v) + lay_at(a.kvl, b, 0, g);
  const int cc = lane % kChunks, cr = lane / kChunks;
  auto load = [&](int i) {  // the warp's block i
    if (i < count) {
      const int key0 = (first + warp + i * kWarps) * kKeys;
      const uint32_t dst = ring + (i % kStages) * 2 * L::kTile;
#pragma unroll
      for (int j = 0; j < kKeys / kRows; ++j) {
        const int r = j * kRows + cr, key = key0 + r;
        const bool there = key < len;
        const long long at = (long long)(there ? key : 0) * a.kvl.rs + cc * 8;
        const uint32_t to = dst + r * (D * 2) + ((cc ^ (r & 7)) << 4);
        copy16(to, kbase + at, there);
        copy16(to + L::kTile, vbase + at, there);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);

  // query rows: row r is query r / group of head g group + r % group
  uint32_t qf[MT][D / 16][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = t * 16 + half * 8 + (lane >> 2);
      const int n = r / group, h = g * group + r - n * group;
      const T* src = static_cast<const T*>(a.q) + (r < rows ? lay_at(a.ql, b, n, h) : 0) + 2 * (lane & 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[t][k][half] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
        qf[t][k][2 + half] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
      }
    }
  float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
  }
  const float sl2 = a.scale_log2;
  const int mat = lane >> 3, mr = lane & 7;
  for (int i = 0; i < count; ++i) {
    copy_wait<kStages - 2>();
    __syncwarp();
    load(i + kStages - 1);  // into the place that the last turn read
    const uint32_t kt = ring + (i % kStages) * 2 * L::kTile, vt = kt + L::kTile;
    float s[MT][2][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[t][j][0] = s[t][j][1] = s[t][j][2] = s[t][j][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[4];
      const int key = (mat >> 1) * 8 + mr, chunk = 2 * k + (mat & 1);
      ldsm4(f, kt + key * (D * 2) + ((chunk ^ (key & 7)) << 4));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        mma16816<T>(s[t][0], qf[t][k], f[0], f[1]);
        mma16816<T>(s[t][1], qf[t][k], f[2], f[3]);
      }
    }
    const int left = len - (first + warp + i * kWarps) * kKeys;
    if (left < kKeys) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (j * 8 + 2 * (lane & 3) + (c & 1) >= left) s[t][j][c] = -INFINITY;
    }
    uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float alpha[2];
      bool raise = false;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float mx = fmaxf(fmaxf(s[t][0][2 * half], s[t][0][2 * half + 1]), fmaxf(s[t][1][2 * half], s[t][1][2 * half + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;
        const bool up = mx > m[t][half] + kRescaleThreshold;  // also from -inf
        alpha[half] = up ? ex2_approx(m[t][half] - mx) : 1.f;
        if (up) m[t][half] = mx;
        raise |= up;
      }
      if (__any_sync(0xffffffffu, raise)) {
        l[t][0] *= alpha[0];
        l[t][1] *= alpha[1];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[t][j][0] *= alpha[0];
          o[t][j][1] *= alpha[0];
          o[t][j][2] *= alpha[1];
          o[t][j][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float neg = m[t][half] == -INFINITY ? 0.f : -m[t][half];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float x = ex2_approx(fmaf(s[t][j][2 * half], sl2, neg));
          const float y = ex2_approx(fmaf(s[t][j][2 * half + 1], sl2, neg));
          l[t][half] += x + y;
          two_terms<T>(x, y, &hi[t][2 * j + half], &lo[t][2 * j + half]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t f[4];
      const int key = (mat & 1) * 8 + mr, chunk = 2 * j + (mat >> 1);
      ldsm4t(f, vt + key * (D * 2) + ((chunk ^ (key & 7)) << 4));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        mma16816<T>(o[t][2 * j], hi[t], f[0], f[1]);
        mma16816<T>(o[t][2 * j + 1], hi[t], f[2], f[3]);
        mma16816<T>(o[t][2 * j], lo[t], f[0], f[1]);
        mma16816<T>(o[t][2 * j + 1], lo[t], f[2], f[3]);
      }
    }
    __syncwarp();
  }
  copy_wait<0>();
  // the warps' states, joined: each leaves (m, l) and O in its own ring
  float* mine = reinterpret_cast<float*>(smem + warp * L::kWarp);
  static_assert(16 * MT * D * 4 <= L::kWarp, "a warp's O fits its ring");
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float sum = l[t][half];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = t * 16 + half * 8 + (lane >> 2);
      if ((lane & 3) == 0) states[warp][r] = make_float2(m[t][half], sum);
    }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = t * 16 + half * 8 + (lane >> 2);
        *reinterpret_cast<float2*>(mine + r * D + 8 * j + 2 * (lane & 3)) =
            make_float2(o[t][j][2 * half], o[t][j][2 * half + 1]);
      }
  __syncthreads();
  // a row's eight columns from c on, final or a part's
  auto finish = [&](int r, int c, float top, float sum, float (&acc)[8]) {
    const int n = r / group, h = g * group + r - n * group, part = split / a.cluster;
    const long long at = ((long long)(part * a.B + b) * a.Hq + h) * a.Nq + n;
    if (a.splits > a.cluster) {
      float* out = a.part.o + (((long long)(part * a.B + b) * a.Nq + n) * a.Hq + h) * D + c;
      reinterpret_cast<float4*>(out)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (c == 0) {
        a.part.m[at] = top == -INFINITY ? top : top * kLn2;
        a.part.l[at] = sum;
      }
      return;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long out = lay_at(a.ol, b, n, h) + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= inv;
    if (a.o_dtype == RA_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.o) + out);
      p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.o_dtype == RA_BF16) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
          p[j] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
          p[j] = pack_half2(acc[2 * j], acc[2 * j + 1]);
        }
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out) = make_uint4(p[0], p[1], p[2], p[3]);
    }
    if (c == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  };
  for (int i = threadIdx.x; i < rows * kChunks; i += kThreads) {
    const int r = i / kChunks, c = (i - r * kChunks) * 8;
    float top = -INFINITY, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, states[w][r].x);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = states[w][r];
      const float weight = ex2_approx(st.x - ref);
      sum += weight * st.y;
      const float* src = reinterpret_cast<const float*>(smem + w * L::kWarp) + r * D + c;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(weight, src[j], acc[j]);
    }
    if (a.cluster == 1) {
      finish(r, c, top, sum, acc);
    } else {  // in the place of the first warp's, which this thread alone has read
      float* to = reinterpret_cast<float*>(smem) + r * D + c;
      reinterpret_cast<float4*>(to)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(to)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (c == 0) joined[r] = make_float2(top, sum);
    }
  }
  if (a.cluster == 1) return;
  cluster_sync();
  const int rank = split % a.cluster;
  for (int i = rank * kThreads + threadIdx.x; i < rows * kChunks; i += a.cluster * kThreads) {
    const int r = i / kChunks, c = (i - r * kChunks) * 8;
    const uint32_t state = smem_u32(&joined[r]), values = smem_u32(smem) + (r * D + c) * 4;
    float top = -INFINITY, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.cluster; ++k) top = fmaxf(top, read2(shared_of(state, k)).x);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int k = 0; k < a.cluster; ++k) {
      const float2 st = read2(shared_of(state, k));
      const float weight = ex2_approx(st.x - ref);
      sum += weight * st.y;
      const float4 x = read4(shared_of(values, k)), y = read4(shared_of(values + 16, k));
      acc[0] = fmaf(weight, x.x, acc[0]);
      acc[1] = fmaf(weight, x.y, acc[1]);
      acc[2] = fmaf(weight, x.z, acc[2]);
      acc[3] = fmaf(weight, x.w, acc[3]);
      acc[4] = fmaf(weight, y.x, acc[4]);
      acc[5] = fmaf(weight, y.y, acc[5]);
      acc[6] = fmaf(weight, y.z, acc[6]);
      acc[7] = fmaf(weight, y.w, acc[7]);
    }
    finish(r, c, top, sum, acc);
  }
  cluster_sync();  // what others read stays until they have
}

// Backward pass: D_i = sum_j P_ij (dO_i . v_j) of rows that few keys share, which is dO . o
// without o's rounding.  A block takes 128 query rows of a head, a warp 16 of them with all
// keys, 64 at a time in shared memory for all warps; P from the saved lse, everything else as
// above.  It runs beside the operand copies and waits for them only before it writes.
// Measured, beside the rest of the backward pass (bf16, d 128): 2 x 4096 queries of 16 heads, 400
// keys: 80 us of 257, 330 TFLOP/s, bound by what shared memory gives to products of 16 rows (operands
// a product ahead: the same); 8192 queries, 128 keys: 36 of 163; 3 x 1924 queries of 32 heads, 3 keys:
// 29 of 197, reading q and dO (64 with O from a forward pass on tcgen05).
constexpr int kDotWarps = 8, kDotKeys = 64;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kDotWarps, 2) cross_dot_kernel(const __grid_constant__ CrossDotArgs a) {
  constexpr int kChunks = D / 8, kTile = kDotKeys * D * 2;  // K or V of a stage; two stages
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = (a.Nq + 127) / 128, unit = blockIdx.x / tiles, b = unit / a.Hq, h = unit - b * a.Hq;
  const int row0 = (blockIdx.x - unit * tiles) * 128 + warp * 16, g = h / (a.Hq / a.Hkv);
  int len = a.Nkv;
  if (a.kv_len) {
    const int v = __ldg(a.kv_len + b);
    len = v < 0 ? 0 : v > a.Nkv ? a.Nkv : v;
  }
  if (len == 0 || len > a.max_keys) {
    pdl_wait();  // what comes after waits for this kernel alone
    return;
  }
  const T* kbase = static_cast<const T*>(a.k) + lay_at(a.kvl, b, 0, g);
  const T* vbase = static_cast<const T*>(a.v) + lay_at(a.kvl, b, 0, g);
  auto load = [&](int key0) {
    const uint32_t stage = smem_u32(smem) + (key0 / kDotKeys & 1) * 2 * kTile;
    const int keys = min(kDotKeys, (len - key0 + 15) & ~15);  // of whole products
    for (int i = threadIdx.x; i < keys * kChunks; i += 32 * kDotWarps) {
      const int r = i / kChunks, c = i - r * kChunks;
      const bool there = key0 + r < len;
      const long long at = (long long)(there ? key0 + r : 0) * a.kvl.rs + c * 8;
      const uint32_t to = stage + r * (D * 2) + ((c ^ (r & 7)) << 4);
      copy16(to, kbase + at, there);
      copy16(to + kTile, vbase + at, there);
    }
    copy_commit();
  };
  load(0);
  uint32_t qf[D / 16][4], df[D / 16][4];
  float lse2[2], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int n = row0 + half * 8 + (lane >> 2);
    const bool there = n < a.Nq;
    const long long at = (there ? lay_at(a.ql, b, n, h) : 0) + 2 * (lane & 3);
    const float lse = there ? a.lse[((long long)b * a.Hq + h) * a.Nq + n] : -INFINITY;
    lse2[half] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const T* q = static_cast<const T*>(a.q) + at + 16 * k;
      const T* dO = static_cast<const T*>(a.dO) + at + 16 * k;
      qf[k][half] = there ? *reinterpret_cast<const uint32_t*>(q) : 0u;
      qf[k][2 + half] = there ? *reinterpret_cast<const uint32_t*>(q + 8) : 0u;
      df[k][half] = there ? *reinterpret_cast<const uint32_t*>(dO) : 0u;
      df[k][2 + half] = there ? *reinterpret_cast<const uint32_t*>(dO + 8) : 0u;
    }
  }
  const int mat = lane >> 3, mr = lane & 7;
  for (int key0 = 0; key0 < len; key0 += kDotKeys) {
    copy_wait<0>();
    __syncthreads();
    if (key0 + kDotKeys < len) load(key0 + kDotKeys);  // into the place that the last turn read
    const uint32_t kt = smem_u32(smem) + (key0 / kDotKeys & 1) * 2 * kTile, vt = kt + kTile;
    const int keys = min(kDotKeys, (len - key0 + 15) & ~15);
    for (int j0 = 0; j0 < keys; j0 += 16) {
      float s[2][4], dp[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][c] = dp[j][c] = 0.f;
      const uint32_t key = j0 + (mat >> 1) * 8 + mr;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = key * (D * 2) + (((2 * k + (mat & 1)) ^ (key & 7)) << 4);
        uint32_t f[4];
        ldsm4(f, kt + at);
        mma16816<T>(s[0], qf[k], f[0], f[1]);
        mma16816<T>(s[1], qf[k], f[2], f[3]);
        ldsm4(f, vt + at);
        mma16816<T>(dp[0], df[k], f[0], f[1]);
        mma16816<T>(dp[1], df[k], f[2], f[3]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = ex2_approx(fmaf(s[j][c], a.scale_log2, lse2[c >> 1]));
          if (key0 + j0 + j * 8 + 2 * (lane & 3) + (c & 1) < len) sum[c >> 1] = fmaf(p, dp[j][c], sum[c >> 1]);
        }
    }
  }
  pdl_wait();
  const CrossScale sc = cross_scale(a.range, b * a.Hkv + g, std::is_same<T, __nv_bfloat16>::value);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float v = sum[half];
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    const int n = row0 + half * 8 + (lane >> 2);
    if ((lane & 3) == 0 && n < a.Nq && lse2[half] != -INFINITY) a.D[((long long)b * a.Hq + h) * a.Np + n] = -v * sc.copy * sc.mul;
  }
}

}  // namespace

cudaError_t launch_cross_dot(const CrossDotArgs& a, cudaStream_t st) {
  auto run = [&](auto kernel) {
    const int smem = 4 * kDotKeys * a.d * 2, blocks = a.B * a.Hq * ((a.Nq + 127) / 128);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kernel, blocks, 32 * kDotWarps, smem, st, a);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (a.d == 128) return a.bf16 ? run(cross_dot_kernel<__nv_bfloat16, 128>) : run(cross_dot_kernel<__half, 128>);
  if (a.d == 64) return a.bf16 ? run(cross_dot_kernel<__nv_bfloat16, 64>) : run(cross_dot_kernel<__half, 64>);
  return cudaErrorInvalidValue;
}

cudaError_t launch_cross_few(const CrossFewArgs& a, cudaStream_t st) {
  const int rows = a.Nq * (a.Hq / a.Hkv);
  if (rows > kCrossFewRows || a.cluster < 1 || a.cluster > 8 || a.splits % a.cluster) return cudaErrorInvalidValue;
  auto run = [&](auto kernel, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * a.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  auto typed = [&](auto t) {
    using T = decltype(t);
    if (a.d == 128)
      return rows <= 16 ? run(cross_few_kernel<T, 128, 1>, FewSmem<128>::kBytes)
                        : run(cross_few_kernel<T, 128, 2>, FewSmem<128>::kBytes);
    if (a.d == 64)
      return rows <= 16 ? run(cross_few_kernel<T, 64, 1>, FewSmem<64>::kBytes)
                        : run(cross_few_kernel<T, 64, 2>, FewSmem<64>::kBytes);
    return cudaErrorInvalidValue;
  };
  return a.bf16 ? typed(__nv_bfloat16{}) : typed(__half{});
}

}  // namespace ra
