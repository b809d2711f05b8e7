// The small kernels around the vocabulary cross entropy's products: the final
// reduction of the loss, the gradient's scale, and the sum of a split product's planes.
// All are bound by their reads or by launch latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- cross entropy
// lse_t = m + ln sum_p l_p e^{m_p - m} over the column parts p, m = max_p m_p;
// loss_t = lse_t - z_{t, y_t}.  A block takes Rows rows: with 32, lane = row while reading,
// so that every read is a full line, and the warps share the parts; with 1 all threads
// share the parts of that row.  Then a warp folds one row's shares.
__device__ __forceinline__ void fold_stats(float& m, float& l, float2 s) {
  const float mx = fmaxf(m, s.x);
  const float ref = mx == -INFINITY ? 0.f : mx;
  l = l * ex2_approx((m - ref) * kLog2e) + s.y * ex2_approx((s.x - ref) * kLog2e);
  m = mx;
}
template <int Rows>
__global__ void __launch_bounds__(Rows == 1 ? 256 : 1024)
    xent_finish_kernel(const float2* stats, int parts, const float* target_logit, const long long* targets,
                       long long ignore, long long V, long long T, float* loss, float* lse, int* status) {
  constexpr int kThreads = Rows == 1 ? 256 : 1024;
  constexpr int kShares = kThreads / Rows;  // threads per row
  __shared__ float2 part[Rows][kShares + 1];
  pdl_trigger();
  pdl_wait();
  const int r = threadIdx.x % Rows, first = threadIdx.x / Rows;
  const long long t = (long long)blockIdx.x * Rows + r;
  float m = -INFINITY, l = 0.f;
  if (t < T) {
    int p = first;
    for (; p + 3 * kShares < parts; p += 4 * kShares) {
      float2 s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = stats[(long long)(p + j * kShares) * T + t];
#pragma unroll
      for (int j = 0; j < 4; ++j) fold_stats(m, l, s[j]);
    }
    for (; p < parts; p += kShares) fold_stats(m, l, stats[(long long)p * T + t]);
  }
  part[r][first] = make_float2(m, l);
  __syncthreads();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * Rows + w;
  if (w >= Rows || row >= T) return;
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < kShares; j += 32) fold_stats(m, l, part[w][j + lane]);
  const float top = warp_max(m);
  l = warp_sum(l * ex2_approx((m - (top == -INFINITY ? 0.f : top)) * kLog2e));
  if (lane) return;
  const float z = top + logf(l);
  lse[row] = z;
  const long long y = targets[row];
  float out = 0.f;
  if (y != ignore) {
    if (y >= 0 && y < V) {
      out = z - target_logit[row];
    } else {
      out = NAN;
      report(status, RA_ERR_INVALID_ARG);
    }
  }
  loss[row] = out;
}

// The logits of a single token on the CUDA cores, bound by reading w once: their statistics,
// or one block's gradient of them (two terms, as in ra_xent_few.cu).  A warp takes kEntries
// vocabulary entries at a time: each lane holds eight columns of every one and multiplies
// them with x from shared memory (fp32), then the lanes' sums are added up.  The
// tensor-core kernel would multiply tiles of 256 rows of which one is filled, in rounds of
// 76 tiles: 37 us against 32768 x 2048 weights.  (For two tokens and more: ra_xent_few.cu.)
// Sums are plain fp32, which keeps the loss of a single sure token exact, and both
// directions form the same ones, so that z - lse in the gradient is.
constexpr int kEntries = 2;
template <typename T, bool GRAD>
__global__ void __launch_bounds__(256) xent_token_kernel(const __grid_constant__ XentFewArgs a) {
  extern __shared__ float xf[];  // [D]
  __shared__ float2 part[8];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = a.V;
  const T* const x = static_cast<const T*>(a.x);
  const T* const w = static_cast<const T*>(a.w);
  for (int i = threadIdx.x; i < a.D; i += 256) xf[i] = to_f32(x[i]);
  __syncthreads();
  long long y = a.targets[0];
  float m = -INFINITY, l = 0.f, mul = 0.f, lse = 0.f;
  const bool live = y != a.ignore && y >= 0 && y < a.vocab;
  if (GRAD) {
    y -= a.col_off;
    if (live) {
      mul = a.grad[0] * (a.scale ? a.scale[0] : 1.f);
      lse = a.lse[0];
    }
  }
  const int chunks = a.D / 8;
  for (int v0 = (blockIdx.x * 8 + warp) * kEntries; v0 < V; v0 += gridDim.x * 8 * kEntries) {
    float acc[kEntries][2];
#pragma unroll
    for (int r = 0; r < kEntries; ++r) acc[r][0] = acc[r][1] = 0.f;
#pragma unroll 8
    for (int c = lane; c < chunks; c += 32) {
      uint4 q[kEntries];
#pragma unroll
      for (int r = 0; r < kEntries; ++r)
        q[r] = __ldg(reinterpret_cast<const uint4*>(w + (long long)min(v0 + r, V - 1) * a.ws) + c);
      const float4* xp = reinterpret_cast<const float4*>(xf + 8 * c);
      const float4 x0 = xp[0], x1 = xp[1];
#pragma unroll
      for (int r = 0; r < kEntries; ++r) {
        const T* e = reinterpret_cast<const T*>(&q[r]);
        acc[r][0] = fmaf(x0.x, to_f32(e[0]), acc[r][0]);
        acc[r][1] = fmaf(x0.y, to_f32(e[1]), acc[r][1]);
        acc[r][0] = fmaf(x0.z, to_f32(e[2]), acc[r][0]);
        acc[r][1] = fmaf(x0.w, to_f32(e[3]), acc[r][1]);
        acc[r][0] = fmaf(x1.x, to_f32(e[4]), acc[r][0]);
        acc[r][1] = fmaf(x1.y, to_f32(e[5]), acc[r][1]);
        acc[r][0] = fmaf(x1.z, to_f32(e[6]), acc[r][0]);
        acc[r][1] = fmaf(x1.w, to_f32(e[7]), acc[r][1]);
      }
    }
    if (GRAD) {
      float z = 0.f;
#pragma unroll
      for (int r = 0; r < kEntries; ++r) {
        const float t = warp_sum(acc[r][0] + acc[r][1]);
        if (lane == r) z = t;
      }
      const int v = v0 + lane;
      if (lane < kEntries && v < V) {
        const float d = live ? mul * logit_gradient(z - lse, y == v) : 0.f;
        const T high = from_f32<T>(d);
        static_cast<T*>(a.d)[v] = high;
        static_cast<T*>(a.d)[a.ld + v] = from_f32<T>(d - to_f32(high));
      }
      continue;
    }
    float z[kEntries], mx = m;
#pragma unroll
    for (int r = 0; r < kEntries; ++r) {
      z[r] = warp_sum(acc[r][0] + acc[r][1]);
      if (lane == 0 && y == v0 + r && v0 + r < V) a.target_logit[0] = z[r];
      if (v0 + r >= V) z[r] = -INFINITY;
      mx = fmaxf(mx, z[r]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    l *= ex2_approx((m - ref) * kLog2e);
#pragma unroll
    for (int r = 0; r < kEntries; ++r) l += ex2_approx((z[r] - ref) * kLog2e);
    m = mx;
  }
  if (GRAD) return;
  if (lane == 0) part[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x == 0) {
    float top = -INFINITY, sum = 0.f;
    for (int j = 0; j < 8; ++j) top = fmaxf(top, part[j].x);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int j = 0; j < 8; ++j) sum += part[j].y * ex2_approx((part[j].x - ref) * kLog2e);
    a.stats[blockIdx.x] = make_float2(top, sum);
  }
}

__global__ void __launch_bounds__(1024) xent_scale_kernel(const float* grad, const long long* targets,
                                                          long long ignore, long long V, long long T, float* scale) {
  __shared__ float part[32];
  pdl_trigger();
  pdl_wait();
  float m = 0.f;
  for (long long t = threadIdx.x; t < T; t += 1024) {
    const long long y = targets[t];
    const float g = fabsf(grad[t]);
    // an infinity or NaN concerns its own token alone
    if (y != ignore && y >= 0 && y < V && g < INFINITY) m = fmaxf(m, g);
  }
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  m = warp_max(part[threadIdx.x]);
  if (threadIdx.x == 0) {
    int k = 0;
    if (m > 0.f) {
      k = 13 - ilogbf(m);  // -114 at least
      k = k > 126 ? 126 : k;  // 2^-126 is the smallest normal number
    }
    scale[0] = ldexpf(1.f, k);
    scale[1] = ldexpf(1.f, -k);
  }
}

// Sum of fp32 planes in order, converted.  Bound by reading the planes.
template <typename T>
__global__ void __launch_bounds__(256) sum_planes_kernel(const float* planes, int count, long long n, T* out) {
  pdl_trigger();
  pdl_wait();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n / 4; i += (long long)gridDim.x * 256) {
    float4 s = reinterpret_cast<const float4*>(planes)[i];
#pragma unroll 4
    for (int k = 1; k < count; ++k) {
      const float4 v = reinterpret_cast<const float4*>(planes + k * n)[i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    out[4 * i] = from_f32<T>(s.x);
    out[4 * i + 1] = from_f32<T>(s.y);
    out[4 * i + 2] = from_f32<T>(s.z);
    out[4 * i + 3] = from_f32<T>(s.w);
  }
}

}  // namespace

cudaError_t launch_xent_token(const XentFewArgs& a, cudaStream_t st) {
  if (a.T != 1 || a.D * 4 > kXentTokenSmem || a.blocks < 1) return cudaErrorInvalidValue;
  auto run = [&](auto kernel) { return launch_pdl(kernel, a.blocks, 256, a.D * 4, st, a); };
  const cudaError_t e = a.bf16 ? (a.d ? run(xent_token_kernel<__nv_bfloat16, true>) : run(xent_token_kernel<__nv_bfloat16, false>))
                               : (a.d ? run(xent_token_kernel<__half, true>) : run(xent_token_kernel<__half, false>));
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_xent_finish(const float2* stats, int parts, const float* target_logit, const long long* targets,
                               long long ignore, long long V, long long T, float* loss, float* lse, int* status,
                               cudaStream_t st) {
  // up to 304 rows a block each keeps the reads of all of them in flight at once
  const cudaError_t e = T <= 304 ? launch_pdl(xent_finish_kernel<1>, (int)T, 256, 0, st, stats, parts, target_logit,
                                              targets, ignore, V, T, loss, lse, status)
                                 : launch_pdl(xent_finish_kernel<32>, (int)((T + 31) / 32), 1024, 0, st, stats, parts,
                                              target_logit, targets, ignore, V, T, loss, lse, status);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_xent_scale(const float* grad, const long long* targets, long long ignore, long long V, long long T,
                              float* scale, cudaStream_t st) {
  const cudaError_t e = launch_pdl(xent_scale_kernel, 1, 1024, 0, st, grad, targets, ignore, V, T, scale);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_sum_planes(const float* planes, int count, long long n, void* out, int dtype, cudaStream_t st) {
  const long long blocks = (n / 4 + 255) / 256;
  const int grid = (int)(blocks < 1216 ? blocks : 1216);
  const cudaError_t e =
      dtype == RA_F32 ? launch_pdl(sum_planes_kernel<float>, grid, 256, 0, st, planes, count, n, static_cast<float*>(out))
      : dtype == RA_BF16
          ? launch_pdl(sum_planes_kernel<__nv_bfloat16>, grid, 256, 0, st, planes, count, n, static_cast<__nv_bfloat16*>(out))
          : launch_pdl(sum_planes_kernel<__half>, grid, 256, 0, st, planes, count, n, static_cast<__half*>(out));
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace ra
