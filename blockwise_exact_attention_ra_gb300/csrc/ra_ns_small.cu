// Newton-Schulz orthogonalisation of matrices whose smaller side m is at most 128: one
// launch, a cluster of up to 16 CTAs per matrix, nothing but the gradient and the result in
// global memory.
//
// X (m x n, turned if the gradient is tall) is cut into slices of C columns, one per CTA of
// the cluster, and stays there for the whole iteration: in TMEM as fp32 (the state) and in
// shared memory as fp16 (the operand).  Each step
//   1. each CTA multiplies its slice with itself (M 128, N 128, K C): a partial Gram matrix,
//      left in shared memory as fp32;
//   2. the CTAs add the partial matrices up through distributed shared memory, each its
//      share of the rows, subtract alpha I and write A' (fp16) into every CTA's memory;
//   3. each CTA forms B' = (b + 2 c alpha) A' + c A'^2 for itself (M 128, N 128, K 128),
//      while the slice in TMEM is multiplied by a + b alpha + c alpha^2;
//   4. the update's product adds B' X to it (M 128, N C, K 128), and the slice is rounded to
//      fp16 again.
// (alpha and why it is taken out: see ra_ns_tc.cu.)  Bound by latency: two cluster barriers,
// three short products and their epilogues per step.  The general chain needs 20 us a step
// here, in memory and with tiles that fill a quarter of the tensor cores' rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "ra_ns.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;

template <int C>
struct SmallSmem {
  static constexpr int kHi = 0;                       // X's slice, fp16: C / 64 tiles of 128 rows x 64 columns
  static constexpr int kA = kHi + C * 256;            // A', then B': 2 such tiles
  static constexpr int kP = kA + 2 * 16384;           // partial Gram matrix, fp32 128 x 128
  static constexpr int kTrace = kP + 65536;           // [cluster rank][warp]
  static constexpr int kNorm = kTrace + kMaxCluster * 8 * 4;  // [cluster rank][warp][3]
  static constexpr int kMisc = kNorm + kMaxCluster * 8 * 12;  // barrier, TMEM address, abort
  static constexpr int kAlloc = kMisc + 32 + 1024;    // slack for 1024-byte alignment
};

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t clustersize() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_load(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// 32 columns of TMEM, this thread's row.
__device__ __forceinline__ void tmem_get(uint32_t src, float* v) {
  uint32_t r[32];
  RA_TMEM_LD32(src, r);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_put(uint32_t dst, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(v[j]);
  RA_TMEM_ST32(dst, r);
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1) ns_small_kernel(const __grid_constant__ NsSmallArgs a) {
  using S = SmallSmem<C>;
  constexpr int kCols = C / 2;            // columns of the slice per thread
  constexpr uint32_t kTmemCols = C == 64 || C == 128 ? 256 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t BAR = sbase + S::kMisc;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::kMisc + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 12);
  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = ctarank(), size = clustersize();
  const int entry = blockIdx.x / size;
  if (threadIdx.x == 0) {
    mbar_init(BAR, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  const uint32_t quarter = warp & 3, half = warp >> 2;
  const int row = (int)(quarter * 32 + lane);               // row of X, A', B'
  const uint32_t lanes = (quarter * 32) << 16;
  const uint32_t tD = tmem + half * 64 + lanes;             // a product of 128 columns, this thread's 64
  const uint32_t tX = tmem + 128 + half * kCols + lanes;    // the slice, this thread's columns
  uint32_t phase = 0;
  // a 16-byte piece of a row of 64 fp16 values, 128-byte swizzle; tile of 128 rows
  auto piece = [&](int base, int tile, int j) {
    return reinterpret_cast<uint4*>(smem + base + tile * 16384 + row * 128 + ((j ^ (row & 7)) << 4));
  };
  // a product issued by one thread of warp 0; everyone waits for it (a wait that gives up
  // goes on with what is there: the cluster's barriers need every thread)
  auto start = [&](auto issue) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      if (elect_lane()) {
        issue();
        mma_commit(BAR);
      }
      __syncwarp();
    }
  };
  auto finish = [&]() {
    (void)mbar_wait(BAR, phase, abort_flag, a.status, a.wait_limit_ns);
    phase ^= 1;
    tc_fence_after();
  };

  // ---- X = G / (|G|_F + eps); TMEM holds sb sx X, shared memory fp16(sx X)
  float x[kCols];
  {
    const int first = (int)rank * C + (int)half * kCols;    // column of X
    const long long at = entry * a.in.bstride;
    if (a.tall) {  // X's columns are G's rows: the lanes read consecutive elements
      uint32_t u[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        u[j] = (row < a.m && first + j < a.n) ? load_bits(a.in, at + (first + j) * a.in.ld + row) : 0u;
#pragma unroll
      for (int j = 0; j < kCols; ++j) x[j] = bits_value(a.in, u[j]);
    } else {
      NsRaw g[kCols / 8];
#pragma unroll
      for (int j = 0; j < kCols; j += 8)
        g[j / 8] = load8(a.in, at + row * a.in.ld + first + j, row < a.m ? a.n - first - j : 0);
#pragma unroll
      for (int j = 0; j < kCols; j += 8) unpack8(a.in, g[j / 8], x + j);
    }
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kCols; ++j) ns_add_square(x[j], s);
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = warp_sum(s[k]);
    cluster_arrive();  // every CTA of the cluster runs
    cluster_wait();
    if (lane < size) {
#pragma unroll
      for (int k = 0; k < 3; ++k) peer_store(mapa(sbase + S::kNorm + (rank * 8 + warp) * 12 + 4 * k, lane), s[k]);
    }
    cluster_arrive();
    cluster_wait();
    float f[3];
    ns_factor(reinterpret_cast<const float*>(smem + S::kNorm), (int)size * 8, a.sx, a.eps, f);
#pragma unroll
    for (int j = 0; j < kCols; ++j) x[j] = ((x[j] * f[0]) * f[1]) * f[2];
  }
  // this thread's columns as fp16 into the operand's tiles (x holds sx X)
  auto put_hi = [&]() {
#pragma unroll
    for (int j = 0; j < kCols; j += 8) {
      const int c = (int)half * kCols + j;
      *piece(S::kHi, c / 64, (c % 64) / 8) =
          make_uint4(pack_half2(x[j], x[j + 1]), pack_half2(x[j + 2], x[j + 3]), pack_half2(x[j + 4], x[j + 5]),
                     pack_half2(x[j + 6], x[j + 7]));
    }
  };
  put_hi();
#pragma unroll
  for (int j = 0; j < kCols; j += 32) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = x[j + i] * a.sb;
    tmem_put(tX + j, v);
  }
  tmem_st_wait();

  const uint32_t idesc_sq = idesc_f16(0, 0, 0, 128, 128), idesc_up = idesc_f16(0, 0, 1, 128, C);
  for (int step = 0; step < a.steps; ++step) {
    // 1. partial Gram matrix
    start([&] {
      const uint64_t d = smem_desc_sw128(sbase + S::kHi, 16, 1024);
#pragma unroll
      for (int k = 0; k < C / 16; ++k) {
        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
        mma_ss(tmem, desc_off(d, off), desc_off(d, off), idesc_sq, k > 0);
      }
    });
    finish();
    float trace = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      tmem_get(tD + 32 * h, v);
      const int c0 = (int)half * 64 + 32 * h;
#pragma unroll
      for (int j = 0; j < 32; ++j) trace += c0 + j == row ? v[j] : 0.f;
      // fp32 rows of 512 bytes; pieces of 16 bytes swizzled within groups of eight
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = c0 / 4 + j;
        *reinterpret_cast<float4*>(smem + S::kP + row * 512 + ((q ^ (row & 7)) << 4)) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    trace = warp_sum(trace);
    if (lane < size) peer_store(mapa(sbase + S::kTrace + (rank * 8 + warp) * 4, lane), trace);
    cluster_arrive();
    cluster_wait();
    // 2. this CTA's share of the rows, summed over the cluster in rank order
    float alpha = 0.f;
    for (uint32_t i = lane; i < size * 8; i += 32) alpha += reinterpret_cast<const float*>(smem + S::kTrace)[i];
    alpha = warp_sum(alpha) * a.alpha_mul;
    const float shift = alpha * a.sa;
    const int share = 128 / (int)size;  // the cluster's size is a power of two
    for (int i = threadIdx.x; i < share * 32; i += kThreads) {
      const int r = (int)rank * share + i / 32, q = i % 32;
      const uint32_t at = sbase + S::kP + r * 512 + ((q ^ (r & 7)) << 4);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (uint32_t p = 0; p < size; ++p) {
        const float4 v = peer_load(mapa(at, p));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const int d = r < a.m ? r - 4 * q : -1;  // the diagonal's place among the four
      s.x = fmaf(s.x, a.gram_acc, d == 0 ? -shift : 0.f);
      s.y = fmaf(s.y, a.gram_acc, d == 1 ? -shift : 0.f);
      s.z = fmaf(s.z, a.gram_acc, d == 2 ? -shift : 0.f);
      s.w = fmaf(s.w, a.gram_acc, d == 3 ? -shift : 0.f);
      const uint32_t lo = pack_half2(s.x, s.y), hi = pack_half2(s.z, s.w);
      // columns 4 q .. + 3: tile q / 16, piece (q % 16) / 2, its half q % 2
      const uint32_t to =
          sbase + S::kA + (q >> 4) * 16384 + r * 128 + ((((q & 15) >> 1) ^ (r & 7)) << 4) + (q & 1) * 8;
      for (uint32_t p = 0; p < size; ++p) peer_store(mapa(to, p), lo, hi);
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    cluster_arrive();
    cluster_wait();
    // 3. B'
    start([&] {
      const uint64_t d = smem_desc_sw128(sbase + S::kA, 16, 1024);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
        mma_ss(tmem, desc_off(d, off), desc_off(d, off), idesc_sq, k > 0);
      }
    });
    const float own = a.ca + alpha * (a.cb + a.cc * alpha);
#pragma unroll 1
    for (int j = 0; j < kCols; j += 32) {
      float v[32];
      tmem_get(tX + j, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= own;
      tmem_put(tX + j, v);
    }
    tmem_st_wait();
    finish();
    const float lin = (a.cb + 2.f * a.cc * alpha) * a.square_lin;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      tmem_get(tD + 32 * h, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4* at = piece(S::kA, (int)half, 4 * h + j);
        const uint4 q = *at;
        const uint32_t qq[4] = {q.x, q.y, q.z, q.w};
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 g = unpack_half2(qq[i]);
          w[i] = pack_half2(fmaf(v[8 * j + 2 * i], a.square_acc, lin * g.x),
                            fmaf(v[8 * j + 2 * i + 1], a.square_acc, lin * g.y));
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    // 4. X += B' X on what is in TMEM
    start([&] {
      const uint64_t da = smem_desc_sw128(sbase + S::kA, 16, 1024);
      const uint64_t db = smem_desc_sw128(sbase + S::kHi, 16384, 1024);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ss(tmem + 128, desc_off(da, (k >> 2) * 16384 + (k & 3) * 32), desc_off(db, k * 2048), idesc_up, 1u);
    });
    finish();
#pragma unroll
    for (int j = 0; j < kCols; j += 32) {
      tmem_get(tX + j, x + j);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[j + i] *= a.inv_sb;
    }
    if (step + 1 < a.steps) put_hi();
  }

  // ---- the result
  {
    const int first = (int)rank * C + (int)half * kCols;
    const long long at = entry * a.out_bstride;
#pragma unroll
    for (int j = 0; j < kCols; ++j) x[j] *= a.out_mul;
    if (a.tall) {  // X's columns are the result's rows: the lanes write consecutive elements
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        if (row < a.m && first + j < a.n) {
          const long long o = at + (first + j) * a.out_ld + row;
          if (a.out_dtype == RA_F32) static_cast<float*>(a.out)[o] = x[j];
          else if (a.out_dtype == RA_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x[j]);
          else static_cast<__half*>(a.out)[o] = __float2half_rn(x[j]);
        }
      }
    } else {
      constexpr int kPart = kCols < 64 ? kCols : 64;
      const int row0 = row - (int)lane;
      // the partial Gram matrices' place: their last readers have passed a cluster barrier
      float* const stage = reinterpret_cast<float*>(smem + S::kP + warp * 8192);
#pragma unroll
      for (int j = 0; j < kCols; j += kPart)
        ns_write_rows<kPart>(a.out, a.out_dtype, a.out_vec, at + row0 * a.out_ld + first + j, a.out_ld, a.m - row0,
                             a.n - first - j, x + j, stage);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int C>
cudaError_t run(const NsSmallArgs& a, int cluster, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<unsigned long long> ready{0};
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(ns_small_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallSmem<C>::kAlloc);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(ns_small_kernel<C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.in.batch * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SmallSmem<C>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ns_small_kernel<C>, a);
}

}  // namespace

cudaError_t launch_ns_small(const NsSmallArgs& a, int slice, int cluster, cudaStream_t st) {
  if (a.m < 1 || a.m > 128 || a.n < 1 || cluster < 1 || cluster > kMaxCluster || (cluster & (cluster - 1)) ||
      (long long)slice * cluster < a.n)
    return cudaErrorInvalidValue;
  cudaError_t e = cudaErrorInvalidValue;
  if (slice == 64) e = run<64>(a, cluster, st);
  else if (slice == 128) e = run<128>(a, cluster, st);
  else if (slice == 256) e = run<256>(a, cluster, st);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace ra
