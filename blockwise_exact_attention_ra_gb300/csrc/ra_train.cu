// The small kernels around the CTA-pair products: the vocabulary cross entropy's
// final reduction and gradient scale, and the Newton-Schulz iteration's norm and
// first operand.  All are bound by their reads or by launch latency.
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
// loss_t = lse_t - z_{t, y_t}.  A block takes 32 rows; its 8 warps share the parts
// (lane = row, so every read is a full line) and meet in shared memory.
__global__ void __launch_bounds__(256) xent_finish_kernel(const float2* stats, int parts, const float* target_logit,
                                                          const long long* targets, long long ignore, long long V,
                                                          long long T, float* loss, float* lse, int* status) {
  __shared__ float2 part[8][32];
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
    for (; p + 24 < parts; p += 32) {
      float2 s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = stats[(long long)(p + 8 * j) * T + t];
#pragma unroll
      for (int j = 0; j < 4; ++j) fold(s[j]);
    }
    for (; p < parts; p += 8) fold(stats[(long long)p * T + t]);
  }
  part[w][lane] = make_float2(m, l);
  __syncthreads();
  if (w != 0 || t >= T) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) fold(part[j][lane]);
  const float z = m + logf(l);
  lse[t] = z;
  const long long y = targets[t];
  float out = 0.f;
  if (y != ignore) {
    if (y >= 0 && y < V) {
      out = z - target_logit[t];
    } else {
      out = NAN;
      report(status, RA_ERR_INVALID_ARG);
    }
  }
  loss[t] = out;
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

// ------------------------------------------------------------- Newton-Schulz
__device__ __forceinline__ float load_as_f32(const void* p, int dtype, long long i) {
  if (dtype == RA_F32) return static_cast<const float*>(p)[i];
  if (dtype == RA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// Eight consecutive elements of a row (fewer at its end; the rest read as zero).
template <bool VEC>
__device__ __forceinline__ void load8(const NsInput& in, long long off, int left, float* v) {
  if (VEC && left >= 8) {
    if (in.dtype == RA_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(in.g) + off);
      const float4 x = p[0], y = p[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in.g) + off);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if (in.dtype == RA_BF16) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]));
        else f = unpack_half2(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? load_as_f32(in.g, in.dtype, off + j) : 0.f;
}

// Squares are summed in three accumulators by magnitude, the large values scaled
// down and the small ones up, so that none of them overflows or vanishes (J. L.
// Blue, "A Portable Fortran Program to Find the Euclidean Norm of a Vector", 1978).
constexpr float kBig = 1099511627776.f, kSmall = 1.f / 1099511627776.f;         // 2^40, 2^-40
constexpr float kDown = 8.271806125530277e-25f, kUp = 1.2089258196146292e24f;  // 2^-80, 2^80

template <bool VEC>
__global__ void __launch_bounds__(256) ns_sumsq_kernel(const __grid_constant__ NsInput in, float* parts) {
  __shared__ float part[3][8];
  const int chunks = (in.cols + 7) / 8;
  const long long total = (long long)in.rows * chunks;
  float s[3] = {0.f, 0.f, 0.f};
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    float v[8];
    load8<VEC>(in, blockIdx.y * in.bstride + r * in.ld + c, in.cols - c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(v[j]);
      const float up = x > kBig ? x * kDown : 0.f, down = x < kSmall ? x * kUp : 0.f;
      const float mid = (x > kBig || x < kSmall) ? 0.f : x;  // NaN stays here
      s[0] = fmaf(mid, mid, s[0]);
      s[1] = fmaf(up, up, s[1]);
      s[2] = fmaf(down, down, s[2]);
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
    for (int j = 0; j < 8; ++j) x += part[threadIdx.x][j];
    parts[((long long)blockIdx.y * kNsParts + blockIdx.x) * 3 + threadIdx.x] = x;
  }
}

template <bool VEC>
__global__ void __launch_bounds__(256) ns_scale_kernel(const __grid_constant__ NsInput in, const float* parts,
                                                       int num_parts, float mul, float eps, uint16_t* hi, uint16_t* lo,
                                                       long long ld) {
  __shared__ double part[8];
  __shared__ float factor[3];
  // |G|_F in 64 bits, the parts added in a fixed order
  double s = 0.0;
  if (threadIdx.x < num_parts) {
    const float* p = parts + ((long long)blockIdx.y * kNsParts + threadIdx.x) * 3;
    s = (double)p[0] + (double)p[1] * 1.4615016373309029e48 + (double)p[2] * 6.8422776578360209e-49;  // 2^160, 2^-160
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int j = 0; j < 8; ++j) sum += part[j];
    const double norm = sqrt(sum) + (double)eps;
    const double inv = norm > 0.0 ? (double)mul / norm : 0.0;
    // inv = f 2^e, applied as two powers of two and f: in range for every norm
    int e = 0;
    const double f = frexp(inv, &e);
    factor[0] = ldexpf(1.f, e / 2);
    factor[1] = ldexpf(1.f, e - e / 2);
    factor[2] = (float)f;
  }
  __syncthreads();
  const float f0 = factor[0], f1 = factor[1], f2 = factor[2];
  const int chunks = (in.cols + 7) / 8;
  const long long total = (long long)in.rows * chunks;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const long long r = i / chunks;
    const int c = (int)(i - r * chunks) * 8;
    float v[8];
    load8<VEC>(in, blockIdx.y * in.bstride + r * in.ld + c, in.cols - c, v);
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = ((v[2 * j] * f0) * f1) * f2, y = ((v[2 * j + 1] * f0) * f1) * f2;
      h[j] = pack_half2(x, y);
      const float2 b = unpack_half2(h[j]);
      l[j] = pack_half2(x - b.x, y - b.y);
    }
    // rows are padded to a multiple of 64 elements: whole 16-byte pieces
    const long long o = ((long long)blockIdx.y * in.rows + r) * ld + c;
    *reinterpret_cast<uint4*>(hi + o) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + o) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

bool rows_aligned(const NsInput& in) {
  const int es = in.dtype == RA_F32 ? 4 : 2;
  return (reinterpret_cast<uintptr_t>(in.g) & 15) == 0 && (in.ld * es) % 16 == 0 && (in.bstride * es) % 16 == 0;
}

int ns_blocks(const NsInput& in, int per_thread) {
  const long long chunks = (long long)in.rows * ((in.cols + 7) / 8);
  const long long n = (chunks + 256ll * per_thread - 1) / (256ll * per_thread);
  return (int)(n < 1 ? 1 : n);
}

}  // namespace

cudaError_t launch_xent_finish(const float2* stats, int parts, const float* target_logit, const long long* targets,
                               long long ignore, long long V, long long T, float* loss, float* lse, int* status,
                               cudaStream_t st) {
  xent_finish_kernel<<<(unsigned)((T + 31) / 32), 256, 0, st>>>(stats, parts, target_logit, targets, ignore, V, T, loss,
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

cudaError_t launch_ns_sumsq(const NsInput& in, float* parts, cudaStream_t st) {
  const int n = ns_blocks(in, 2);
  const dim3 grid(n < kNsParts ? n : kNsParts, in.batch);
  if (rows_aligned(in)) ns_sumsq_kernel<true><<<grid, 256, 0, st>>>(in, parts);
  else ns_sumsq_kernel<false><<<grid, 256, 0, st>>>(in, parts);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_ns_scale(const NsInput& in, const float* parts, float mul, float eps, uint16_t* hi, uint16_t* lo,
                            long long ld, cudaStream_t st) {
  const int n = ns_blocks(in, 2);
  const int num_parts = n < kNsParts ? n : kNsParts;
  const dim3 grid(n < 1216 ? n : 1216, in.batch);
  if (rows_aligned(in)) ns_scale_kernel<true><<<grid, 256, 0, st>>>(in, parts, num_parts, mul, eps, hi, lo, ld);
  else ns_scale_kernel<false><<<grid, 256, 0, st>>>(in, parts, num_parts, mul, eps, hi, lo, ld);
  count_launch();
  return cudaGetLastError();
}

}  // namespace ra
