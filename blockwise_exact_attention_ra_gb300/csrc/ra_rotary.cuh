// What the forward and the backward kernel of the rotary positions (with or without the
// norm of each head) share: angles, and the exchange between the two columns of a pair.
//
// Mathematics.  Pair i of a row at position p is turned by the angle p f_i:
//   (x, y) -> A (x cos - y sin, x sin + y cos),
// columns (i, i + rot/2) or (2i, 2i+1).  A frequency is held as F = round(2^64 f / 2 pi),
// the 64-bit fixed-point fraction of a turn per position; p F mod 2^64 is the phase, so
// that whole turns fall away by the wrap-around of an integer product and positions of any
// size keep an error of at most |p| 2^-54 f / 2 pi turns (that of f itself, a double) plus
// 2^-33.  No table is read.
//
// Organisation.  G lanes (d / 8 of them, rounded up to a power of two) hold one row, eight
// columns (16 bytes of a 16-bit type) each; a warp holds 32 / G rows, of as many tokens,
// and goes through their heads, so that the angles of a token are formed once, by the warp
// that uses them, and stay in registers.  The kernels are bound by reading and writing the
// rows.
#pragma once

#include "ra_device.cuh"

namespace ra {

constexpr int kRotThreads = 256, kRotWarps = kRotThreads / 32;
constexpr int kRotMaxD = kRotMaxHead;

// How the other column of a pair is reached: within the thread; in a lane rot/16 further
// (rot a multiple of 16); through shared memory.
enum RotExchange { ROT_THREAD = 0, ROT_SHUFFLE = 1, ROT_STAGE = 2 };

// Eight columns of one row as they are in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, bool there) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    r.v[i] = there ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = to_f32(e[j]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    __align__(16) T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = from_f32<T>(f[j]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> shuffle8(const Raw8<T>& r, int lane) {
  Raw8<T> o;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    o.v[i].x = __shfl_sync(0xffffffffu, r.v[i].x, lane);
    o.v[i].y = __shfl_sync(0xffffffffu, r.v[i].y, lane);
    o.v[i].z = __shfl_sync(0xffffffffu, r.v[i].z, lane);
    o.v[i].w = __shfl_sync(0xffffffffu, r.v[i].w, lane);
  }
  return o;
}

__device__ __forceinline__ float load_any(const void* p, int dtype, int i) {
  return dtype == RA_F32    ? static_cast<const float*>(p)[i]
         : dtype == RA_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i])
                            : to_f32(static_cast<const __half*>(p)[i]);
}

// cos and sin of the phase (top 32 bits of position x frequency), times `amplitude`.  The
// phase is brought within an eighth of a turn in integers, so that its conversion to fp32
// loses nothing that matters.  FAST, for rows of 16-bit types: the hardware's sine and
// cosine, within 5e-7 there, a five-hundredth of fp16's rounding.
template <bool FAST>
__device__ __forceinline__ float2 turn(unsigned long long freq, long long pos, float amplitude) {
  const unsigned long long phase = (unsigned long long)pos * freq + 0x80000000ull;
  const uint32_t p = (uint32_t)(phase >> 32);
  const uint32_t quadrant = (p + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(p - (quadrant << 30));
  float s, c;
  if (FAST) {
    const float x = r * 1.4629180792671596e-9f;  // 2 pi / 2^32
    s = __sinf(x);
    c = __cosf(x);
  } else {
    sincospif(r * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
  }
  const float a = quadrant & 1u ? -s : c, b = quadrant & 1u ? c : s;
  return quadrant & 2u ? make_float2(-a * amplitude, -b * amplitude) : make_float2(a * amplitude, b * amplitude);
}

// F of a frequency in radians per position.
__device__ __forceinline__ unsigned long long fixed_turns(double f) {
  const double t = f * 0.15915494309189535;  // 1 / 2 pi
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ long long rot_position(const RotaryArgs& a, long long b, long long n) {
  if (a.positions) return __ldg(a.positions + b * a.pos_bstride + n);
  if (a.striped) {
    const long long host = n / a.S;
    n = (n - host * a.S) * a.P + host;
  }
  return a.pos_off + n;
}

// Sum over the G lanes of a row.
__device__ __forceinline__ float group_sum(float v, int G) {
  for (int o = G >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp's place: lane c of group g, which holds the row of token t0 + g.
struct RotLane {
  int g, c, partner;   // partner: lane that holds the pairs' other columns (ROT_SHUFFLE)
  bool column;         // this lane holds columns of the row
  uint32_t turned;     // bit j: column 8 c + j belongs to a pair
};
template <int EX>
__device__ __forceinline__ RotLane rot_lane(const RotaryArgs& a) {
  RotLane l;
  const int lane = (int)lane_id();
  l.g = lane / a.G;
  l.c = lane - l.g * a.G;
  l.column = l.c * 8 < a.d;
  const int left = a.rot - 8 * l.c;
  l.turned = left >= 8 ? 0xffu : left > 0 ? (1u << left) - 1u : 0u;
  l.partner = lane;
  if (EX == ROT_SHUFFLE && left > 0) l.partner = l.c * 16 < a.rot ? lane + a.rot / 16 : lane - a.rot / 16;
  return l;
}

// The other columns of the pairs of this lane's eight (0 for columns of no pair, whose
// factor is -0: x 1 + 0 (-0) is x, whatever the neighbour holds).  `stage`: 8 x 33 floats
// of the warp; column p of a group's row sits at [p % 8][g G + p / 8], so that neither the
// writes nor the reads, at any distance, meet in a bank.
template <int EX, typename T>
__device__ __forceinline__ void other_columns(const RotaryArgs& a, const RotLane& l, const Raw8<T>& raw,
                                              const float (&f)[8], float (&p)[8], float* stage) {
  if constexpr (EX == ROT_THREAD) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (l.turned >> j) & 1u ? f[j ^ 1] : 0.f;
  } else if constexpr (EX == ROT_SHUFFLE) {
    unpack8(shuffle8(raw, l.partner), p);
    if (!l.turned) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = 0.f;
    }
  } else {
    const int lane = (int)lane_id(), half = a.rot / 2;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) stage[j * 33 + lane] = f[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = 8 * l.c + j, at = e < half ? e + half : e - half;
      p[j] = (l.turned >> j) & 1u ? stage[(at & 7) * 33 + l.g * a.G + (at >> 3)] : 0.f;
    }
  }
}

// Factors of this lane's columns and of their pairs' other columns.  DIR: 1 turns by the
// angle, -1 by its opposite (the transpose, for gradients).
template <int EX, int DIR>
__device__ __forceinline__ void rot_factors(const RotaryArgs& a, const RotLane& l, const float2* cs, float (&C)[8],
                                            float (&S)[8]) {
  const int half = a.rot / 2;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = 8 * l.c + j;
    C[j] = 1.f;
    S[j] = -0.f;
    if ((l.turned >> j) & 1u) {
      const bool second = EX == ROT_THREAD ? j & 1 : e >= half;
      const float2 t = cs[l.g * half + (EX == ROT_THREAD ? e >> 1 : second ? e - half : e)];
      C[j] = t.x;
      S[j] = (second ? DIR : -DIR) * t.y;
    }
  }
}

// The column that shares a pair with column e.
template <int EX>
__device__ __forceinline__ int other_column(const RotaryArgs& a, int e) {
  if (EX == ROT_THREAD) return e ^ 1;
  return e < a.rot / 2 ? e + a.rot / 2 : e - a.rot / 2;
}

// cos and sin of every pair of the warp's tokens.
template <bool FAST>
__device__ __forceinline__ void rot_angles(const RotaryArgs& a, const unsigned long long* freq, long long t0,
                                           float2* cs) {
  const int half = a.rot / 2, rows = 32 / a.G;
  __syncwarp();
  if (half)
    for (int i = (int)lane_id(); i < rows * half; i += 32) {
      const int g = i / half;
      const long long t = t0 + g;
      if (t < a.tokens) {
        const long long b = t / a.N;
        cs[i] = turn<FAST>(freq[i - g * half], rot_position(a, b, t - b * a.N), a.amplitude);
      }
    }
  __syncwarp();
}

// Heads [first, last) of part `part` of `parts`.
__device__ __forceinline__ void rot_heads(int H, int part, int parts, int* first, int* last) {
  *first = (int)((long long)H * part / parts);
  *last = (int)((long long)H * (part + 1) / parts);
}

// 2^-70 where the sum of squares left fp32's range (or is NaN), else 1.
__device__ __forceinline__ float rot_scale(float sum) { return sum < 1e37f ? 1.f : 8.470329472543003e-22f; }

}  // namespace ra
