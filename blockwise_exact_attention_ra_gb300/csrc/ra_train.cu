// The small kernels around the vocabulary cross entropy's products: the final
// reduction of the loss, the gradient's scale, and the sum of a split product's planes.
// All are bound by their reads or by launch latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- cross entropy
// lse_t = m + ln sum_p l_p e^{m_p - m} over the column parts p, m = max_p m_p;
// loss_t = lse_t - z_{t, y_t}.  A block takes 32 rows; its 32 warps share the parts
// (lane = row, so every read is a full line) and meet in shared memory.
__global__ void __launch_bounds__(1024) xent_finish_kernel(const float2* stats, int parts, const float* target_logit,
                                                          const long long* targets, long long ignore, long long V,
                                                          long long T, float* loss, float* lse, int* status) {
  __shared__ float2 part[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * 32 + lane;
  float m = -INFINITY, l = 0.f;
  auto fold = [&](float2 s) {
    const float mx = fmaxf(m, s.x);
    const float ref = mx == -INFINITY ? 0.f : mx;
    l = l * ex2_approx((m - ref) * kLog2e) + s.y * ex2_approx((s.x - ref) * kLog2e);
    m = mx;
  };
  if (t < T) {
    int p = w;
    for (; p + 96 < parts; p += 128) {
      float2 s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = stats[(long long)(p + 32 * j) * T + t];
#pragma unroll
      for (int j = 0; j < 4; ++j) fold(s[j]);
    }
    for (; p < parts; p += 32) fold(stats[(long long)p * T + t]);
  }
  part[w][lane] = make_float2(m, l);
  __syncthreads();
  // warp w folds row w's 32 values, one per lane
  const long long row = (long long)blockIdx.x * 32 + w;
  if (row >= T) return;
  const float2 q = part[lane][w];
  m = warp_max(q.x);
  l = warp_sum(q.y * ex2_approx((q.x - (m == -INFINITY ? 0.f : m)) * kLog2e));
  if (lane) return;
  const float z = m + logf(l);
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

__global__ void __launch_bounds__(1024) xent_scale_kernel(const float* grad, const long long* targets,
                                                          long long ignore, long long V, long long T, float* scale) {
  __shared__ float part[32];
  float m = 0.f;
  for (long long t = threadIdx.x; t < T; t += 1024) {
    const long long y = targets[t];
    if (y != ignore && y >= 0 && y < V) m = fmaxf(m, fabsf(grad[t]));
  }
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  m = warp_max(part[threadIdx.x]);
  if (threadIdx.x == 0) {
    int k = 0;
    if (m > 0.f && m < INFINITY) {
      k = 13 - ilogbf(m);
      k = k > 100 ? 100 : (k < -100 ? -100 : k);
    }
    scale[0] = ldexpf(1.f, k);
    scale[1] = ldexpf(1.f, -k);
  }
}

// Sum of fp32 planes in order, converted.  Bound by reading the planes.
template <typename T>
__global__ void __launch_bounds__(256) sum_planes_kernel(const float* planes, int count, long long n, T* out) {
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

cudaError_t launch_xent_finish(const float2* stats, int parts, const float* target_logit, const long long* targets,
                               long long ignore, long long V, long long T, float* loss, float* lse, int* status,
                               cudaStream_t st) {
  xent_finish_kernel<<<(unsigned)((T + 31) / 32), 1024, 0, st>>>(stats, parts, target_logit, targets, ignore, V, T, loss,
                                                                lse, status);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_xent_scale(const float* grad, const long long* targets, long long ignore, long long V, long long T,
                              float* scale, cudaStream_t st) {
  xent_scale_kernel<<<1, 1024, 0, st>>>(grad, targets, ignore, V, T, scale);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_sum_planes(const float* planes, int count, long long n, void* out, int dtype, cudaStream_t st) {
  const long long blocks = (n / 4 + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 1216 ? blocks : 1216);
  if (dtype == RA_F32) sum_planes_kernel<<<grid, 256, 0, st>>>(planes, count, n, static_cast<float*>(out));
  else if (dtype == RA_BF16) sum_planes_kernel<<<grid, 256, 0, st>>>(planes, count, n, static_cast<__nv_bfloat16*>(out));
  else sum_planes_kernel<<<grid, 256, 0, st>>>(planes, count, n, static_cast<__half*>(out));
  count_launch();
  return cudaGetLastError();
}

}  // namespace ra
