// The vocabulary cross entropy's logits for few tokens (at most 16), where reading w is all
// there is to do: their softmax statistics, or one block's gradient of them.
//
// The pair kernels multiply tiles of 256 rows whatever their number, 0.33 us per 64 x 256
// slab of w and pair, in rounds of 76 tiles; here w goes from memory straight into
// registers as the left operand of warp-level products (m16n8k16, 16 entries of the
// vocabulary by 8 tokens), each element once, and x waits in shared memory.  The forward in
// us, against the pair kernel's: 8 tokens, 4096 x 2000 (D x V) 18.4 (32.8), 512 x 32768 16.4
// (20.5), 2048 x 65536 63.5 (73.7); 16 tokens, 512 x 32768 18.4 (22.5).  With 32 tokens it
// would read x from shared memory twice as often as w from memory and lose: 2048 x 65536 82
// (76).
//   - A unit is 16 entries.  Four warps share its columns, 32 at a time; a lane loads 16
//     bytes of two entries and takes them as the operands of two products: which columns of
//     a product are which is the same for w and x, so any order does.
//   - The warps' sums meet in shared memory and are added up there in fp32.  So are a
//     warp's own after every four groups (128 products), since the tensor core's sums are
//     not rounded to nearest.
//   - Each lane then holds one logit of each eighth token: statistics go on in registers
//     over the units, gradients are written.
// Units go round the CTAs first, so that the last round is spread over all SMs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 16, kShare = 4, kGroups = kWarps / kShare;
constexpr int kUnroll = 4;       // groups of 32 columns in flight per warp
constexpr long long kNoLoss = -(1ll << 62);

template <int NT>
struct Few {
  static constexpr int kTokens = 8 * NT;
  static constexpr int kLine = NT == 1 ? 8 : 8 * NT + 8;  // floats of one entry's sums (no bank twice)
  static constexpr int kSums = 16 * kLine;                // one warp's sums
  static constexpr int kSumsBytes = kGroups * 2 * kShare * kSums * 4;
  static constexpr int kStatBytes = kWarps * kTokens * 8;
};
// Columns of x's rows in shared memory: padded to whole groups and to 64 bytes past a
// multiple of 128, so that two rows lie in different banks.
__host__ __device__ constexpr int x_line(int D) { return (D + 31) / 32 * 32 + ((D + 31) / 32 % 2 ? 0 : 32); }

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void fold(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  const float ref = mx == -INFINITY ? 0.f : mx;
  l = l * ex2_approx((m - ref) * kLog2e) + l2 * ex2_approx((m2 - ref) * kLog2e);
  m = mx;
}

template <typename T, int NT, bool GRAD>
__global__ void __launch_bounds__(kWarps * 32, 1) xent_few_kernel(const __grid_constant__ XentFewArgs a) {
  using F = Few<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const sums = reinterpret_cast<float*>(smem);
  float2* const stat = reinterpret_cast<float2*>(smem + F::kSumsBytes);
  T* const xs = reinterpret_cast<T*>(smem + F::kSumsBytes + F::kStatBytes);
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / kShare, part = warp % kShare;
  const int g = lane >> 2, t = lane & 3;
  const int chunks = a.D / 8, groups = (chunks + 3) / 4, line = x_line(a.D);
  for (int i = threadIdx.x; i < F::kTokens * (line / 8); i += kWarps * 32) {
    const int n = i / (line / 8), c = i - n * (line / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < a.T && c < chunks) v = *(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + n * a.xs) + c);
    *reinterpret_cast<uint4*>(xs + n * line + 8 * c) = v;
  }
  // this lane's tokens: lane % 8 + 8 j; its entry of a unit: 4 part + lane / 8
  const int token = lane & 7, entry = 4 * part + (lane >> 3);
  long long y[NT];
  float m[NT], l[NT], mul[NT], lse[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = token + 8 * j;
    y[j] = n < a.T ? a.targets[n] : -1;
    m[j] = -INFINITY;
    l[j] = mul[j] = lse[j] = 0.f;
    if (GRAD) {
      const bool live = n < a.T && y[j] != a.ignore && y[j] >= 0 && y[j] < a.vocab;
      if (live) {
        mul[j] = a.grad[n] * (a.scale ? a.scale[0] : 1.f);
        lse[j] = a.lse[n];
      }
      y[j] = live ? y[j] - a.col_off : kNoLoss;
    }
  }
  __syncthreads();

  const int units = (a.V + 15) / 16;
  int flip = 0;
  for (int u = blockIdx.x + gridDim.x * group; u < units; u += gridDim.x * kGroups, flip ^= 1) {
    const uint4* const w0 = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + min(16 * u + g, a.V - 1) * a.ws);
    const uint4* const w1 =
        reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + min(16 * u + g + 8, a.V - 1) * a.ws);
    float acc[NT][4], tot[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][k] = tot[j][k] = 0.f;
    for (int c = part; c < groups; c += kShare * kUnroll) {
      uint4 p[kUnroll], q[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = 4 * (c + kShare * k) + t;
        p[k] = q[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < chunks) {
          p[k] = __ldg(w0 + i);
          q[k] = __ldg(w1 + i);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (c + kShare * k >= groups) break;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 b = *reinterpret_cast<const uint4*>(xs + (8 * j + g) * line + 32 * (c + kShare * k) + 8 * t);
          mma(acc[j], p[k].x, q[k].x, p[k].y, q[k].y, b.x, b.y, T());
          mma(acc[j], p[k].z, q[k].z, p[k].w, q[k].w, b.z, b.w, T());
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          tot[j][k] += acc[j][k];
          acc[j][k] = 0.f;
        }
    }
    // the last unit's sums are read by then: each warp has passed the barrier since
    float* const mine = sums + ((group * 2 + flip) * kShare + part) * F::kSums;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(mine + g * F::kLine + 8 * j + 2 * t) =
          make_float2(tot[j][0], tot[j][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * F::kLine + 8 * j + 2 * t) =
          make_float2(tot[j][2], tot[j][3]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kShare * 32) : "memory");
    const float* const all = sums + (group * 2 + flip) * kShare * F::kSums + entry * F::kLine + token;
    const int v = 16 * u + entry;
#pragma unroll
    for (int j = 0; j < NT && v < a.V; ++j) {
      const int n = token + 8 * j;
      const float* s = all + 8 * j;
      const float z = (s[0] + s[F::kSums]) + (s[2 * F::kSums] + s[3 * F::kSums]);
      if (GRAD) {
        if (n < a.T) {
          // two terms: see PAIR_DLOGITS; a row without loss may hold anything
          const float d = y[j] == kNoLoss ? 0.f : mul[j] * logit_gradient(z - lse[j], y[j] == v);
          const T high = from_f32<T>(d);
          static_cast<T*>(a.d)[n * a.ld + v] = high;
          static_cast<T*>(a.d)[(a.T + n) * a.ld + v] = from_f32<T>(d - to_f32(high));
        }
      } else {
        if (y[j] == v) a.target_logit[n] = z;
        fold(m[j], l[j], z, 1.f);
      }
    }
    __syncwarp();
  }
  if constexpr (!GRAD) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1)
        fold(m[j], l[j], __shfl_xor_sync(0xffffffffu, m[j], o), __shfl_xor_sync(0xffffffffu, l[j], o));
      if (lane < 8) stat[warp * F::kTokens + 8 * j + lane] = make_float2(m[j], l[j]);
    }
    __syncthreads();
    const int n = threadIdx.x;
    if (n >= a.T) return;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 s = stat[k * F::kTokens + n];
      fold(top, sum, s.x, s.y);
    }
    a.stats[(long long)blockIdx.x * a.T + n] = make_float2(top, sum);
  }
}

template <int NT>
constexpr long long few_smem(int D) {
  return Few<NT>::kSumsBytes + Few<NT>::kStatBytes + Few<NT>::kTokens * 2ll * x_line(D);
}
constexpr int kMostSmem = 227 * 1024;

template <typename T, int NT, bool GRAD>
cudaError_t launch_t(const XentFewArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(xent_few_kernel<T, NT, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(bit, std::memory_order_release);
  }
  e = launch_pdl(xent_few_kernel<T, NT, GRAD>, a.blocks, kWarps * 32, few_smem<NT>(a.D), st, a);
  if (e == cudaSuccess) count_launch();
  return e;
}
template <typename T, int NT>
cudaError_t launch_g(const XentFewArgs& a, cudaStream_t st) {
  return a.d ? launch_t<T, NT, true>(a, st) : launch_t<T, NT, false>(a, st);
}
template <typename T>
cudaError_t launch_n(const XentFewArgs& a, cudaStream_t st) {
  return a.T <= 8 ? launch_g<T, 1>(a, st) : launch_g<T, 2>(a, st);
}

}  // namespace

bool xent_few(long long T, int D) {
  return T <= 8 ? few_smem<1>(D) <= kMostSmem : T <= 16 && few_smem<2>(D) <= kMostSmem;
}

cudaError_t launch_xent_few(const XentFewArgs& a, cudaStream_t st) {
  if (!xent_few(a.T, a.D) || a.blocks < 1) return cudaErrorInvalidValue;
  return a.bf16 ? launch_n<__nv_bfloat16>(a, st) : launch_n<__half>(a, st);
}

}  // namespace ra
