// What the Newton-Schulz kernels share: reading a gradient, and its norm.
#pragma once

#include <math.h>

#include "ra_device.cuh"
#include "ra_internal.h"

namespace ra {

constexpr int kNsBatch = 4;  // groups of eight in flight per thread; eight run no faster

// One element as its bits, and as a number.  Loading and converting are apart so that a
// thread's loads are all in flight before the first is used.
__device__ __forceinline__ uint32_t load_bits(const NsInput& in, long long i) {
  return in.dtype == RA_F32 ? static_cast<const uint32_t*>(in.g)[i] : static_cast<const uint16_t*>(in.g)[i];
}
__device__ __forceinline__ float bits_value(const NsInput& in, uint32_t u) {
  if (in.dtype == RA_F32) return __uint_as_float(u);
  if (in.dtype == RA_BF16) return __uint_as_float(u << 16);
  return __half2float(__ushort_as_half((unsigned short)u));
}

// Eight consecutive elements of a row (fewer at its end; the rest read as zero), as
// loaded: fp32, or 16-bit in x.
struct NsRaw {
  uint4 x, y;
};
__device__ __forceinline__ NsRaw load8(const NsInput& in, long long off, int left) {
  NsRaw r{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (in.vec && left >= 8) {
    if (in.dtype == RA_F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(in.g) + off);
      r.x = p[0];
      r.y = p[1];
    } else {
      r.x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(in.g) + off);
    }
  } else if (left > 0) {
    uint32_t w[8];
    if (in.dtype == RA_F32) {
      const uint32_t* p = static_cast<const uint32_t*>(in.g) + off;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < left ? p[j] : 0u;
      r.y = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(in.g) + off;
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = j < left ? p[j] : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = h[2 * j] | h[2 * j + 1] << 16;
    }
    r.x = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}
__device__ __forceinline__ void unpack8(const NsInput& in, const NsRaw& r, float* v) {
  const uint32_t w[8] = {r.x.x, r.x.y, r.x.z, r.x.w, r.y.x, r.y.y, r.y.z, r.y.w};
  if (in.dtype == RA_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = in.dtype == RA_BF16 ? make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u))
                                           : unpack_half2(w[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
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
// are added in a fixed order, in 64 bits.  With `shift`, times the power of two that brings
// |G|_F / (|G|_F + eps) to 1/2 ... 1, if it is less: 2^*shift.
__device__ __forceinline__ void ns_factor(const float* parts, int num_parts, float mul, float eps, float* f,
                                          int* shift = nullptr) {
  double s = 0.0;
  for (int i = lane_id(); i < num_parts; i += 32) {
    const float* p = parts + 3 * i;
    s += (double)p[0] + (double)p[1] * 1.4615016373309029e48 + (double)p[2] * 6.8422776578360209e-49;  // 2^160, 2^-160
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const double own = sqrt(s), norm = own + (double)eps;
  double inv = norm > 0.0 ? (double)mul / norm : 0.0;
  int e = 0;
  if (shift) {
    *shift = 0;
    if (own > 0.0 && own < 0.5 * norm) {  // neither 0 nor NaN
      (void)frexp(own / norm, &e);
      *shift = -e;
      inv = ldexp(inv, -e);
    }
  }
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

// 32 rows of N (32 or 64) columns of the result by one warp, a row's values in each lane; o:
// element of the first row and column.  Rows that start on 16-byte boundaries are written
// by their lanes, 16 bytes at a time.  Others go through shared memory (32 N floats of the
// warp's own, in rotated rows), so that a row's elements are stored by neighbouring lanes: a
// lane that stores its row's elements one by one took 38 us for the last 256 x 256 tile of a
// chain, against 5.
template <int N, typename T>
__device__ __forceinline__ void ns_store_rows(T* out, long long ld, int rows, int cols, const float* stage) {
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
#pragma unroll
    for (int h = 0; h < N; h += 32) {
      const int c = h + (int)lane_id();
      if (c < cols) out[r * ld + c] = from_f32<T>(stage[r * N + ((c + r) & (N - 1))]);
    }
  }
}
template <int N>
__device__ __forceinline__ void ns_write_rows(void* out, int dtype, bool vec, long long o, long long ld, int rows,
                                              int cols, const float* v, float* stage) {
  const int lane = (int)lane_id();
  if (vec && cols >= N) {
    if (lane >= rows) return;
    o += lane * ld;
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
  __syncwarp();
#pragma unroll
  for (int j = 0; j < N; ++j) stage[lane * N + ((j + lane) & (N - 1))] = v[j];
  __syncwarp();
  rows = min(rows, 32);
  if (dtype == RA_F32) ns_store_rows<N>(static_cast<float*>(out) + o, ld, rows, cols, stage);
  else if (dtype == RA_BF16) ns_store_rows<N>(static_cast<__nv_bfloat16*>(out) + o, ld, rows, cols, stage);
  else ns_store_rows<N>(static_cast<__half*>(out) + o, ld, rows, cols, stage);
  __syncwarp();
}

}  // namespace ra
