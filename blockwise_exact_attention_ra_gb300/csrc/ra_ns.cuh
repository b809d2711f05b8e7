// What the Newton-Schulz kernels share: reading a gradient, and its norm.
#pragma once

#include <math.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

__device__ __forceinline__ float load_as_f32(const void* p, int dtype, long long i) {
  if (dtype == RA_F32) return static_cast<const float*>(p)[i];
  if (dtype == RA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

constexpr int kNsBatch = 4;  // groups of eight in flight per thread

// Eight consecutive elements of a row (fewer at its end; the rest read as zero).
__device__ __forceinline__ void load8(const NsInput& in, long long off, int left, float* v) {
  if (in.vec && left >= 8) {
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
__device__ __forceinline__ void ns_add_square(float x, float* s) {
  x = fabsf(x);
  const float up = x > kBig ? x * kDown : 0.f, down = x < kSmall ? x * kUp : 0.f;
  const float mid = (x > kBig || x < kSmall) ? 0.f : x;  // NaN stays here
  s[0] = fmaf(mid, mid, s[0]);
  s[1] = fmaf(up, up, s[1]);
  s[2] = fmaf(down, down, s[2]);
}

// mul / (|G|_F + eps) as f 2^e0 2^e1 (in range for every norm), by one warp; the parts
// are added in a fixed order, in 64 bits.
__device__ __forceinline__ void ns_factor(const float* parts, int num_parts, float mul, float eps, float* f) {
  double s = 0.0;
  for (int i = lane_id(); i < num_parts; i += 32) {
    const float* p = parts + 3 * i;
    s += (double)p[0] + (double)p[1] * 1.4615016373309029e48 + (double)p[2] * 6.8422776578360209e-49;  // 2^160, 2^-160
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const double norm = sqrt(s) + (double)eps;
  const double inv = norm > 0.0 ? (double)mul / norm : 0.0;
  int e = 0;
  f[2] = (float)frexp(inv, &e);
  f[0] = ldexpf(1.f, e / 2);
  f[1] = ldexpf(1.f, e - e / 2);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
  if (bf16) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&t);
  }
  return pack_half2(lo, hi);
}

// N (a multiple of 8) columns of the result's row from column cc on, those below cols.
template <int N>
__device__ __forceinline__ void ns_write_row(void* out, int dtype, bool vec, long long o, int cc, int cols,
                                             const float* v) {
  if (cc >= cols) return;
  if (vec && cc + N <= cols) {
    if (dtype == RA_F32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
#pragma unroll
      for (int j = 0; j < N / 4; ++j) q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o);
      const int bf = dtype == RA_BF16;
#pragma unroll
      for (int j = 0; j < N / 8; ++j)
        q[j] = make_uint4(pack16(v[8 * j], v[8 * j + 1], bf), pack16(v[8 * j + 2], v[8 * j + 3], bf),
                          pack16(v[8 * j + 4], v[8 * j + 5], bf), pack16(v[8 * j + 6], v[8 * j + 7], bf));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (cc + j < cols) {
      if (dtype == RA_F32) static_cast<float*>(out)[o + j] = v[j];
      else if (dtype == RA_BF16) static_cast<__nv_bfloat16*>(out)[o + j] = __float2bfloat16_rn(v[j]);
      else static_cast<__half*>(out)[o + j] = __float2half_rn(v[j]);
    }
  }
}

}  // namespace ra
