// What the forward and the backward kernel of the rotary positions (with or without the
// norm of each head) share: angles, the layout of rows in a warp, and the exchange between
// the two columns of a pair.
//
// Mathematics.  Pair i of a row at position p is turned by the angle p f_i:
//   (x, y) -> A (x cos - y sin, x sin + y cos),
// columns (i, i + rot/2) or (2i, 2i+1).  A frequency is held as F = round(2^64 f / 2 pi),
// the 64-bit fixed-point fraction of a turn per position; p F mod 2^64 is the phase, so
// that whole turns fall away by the wrap-around of an integer product.  f / 2 pi is formed in two
// doubles, so that F is off by its own rounding alone: the angle of position p by |p| 2^-64
// turns, and by 2^-28 for the phase's rounding to fp32.  No table is read.
//
// Organisation.  A lane holds two pieces of eight columns (16 bytes of a 16-bit type) of a
// row, so chosen that they hold whole pairs where rot/2 is a multiple of 8 (or pairs are
// neighbours): the two columns of a pair meet in a thread, without an exchange.  G lanes
// (d / 16, rounded up to a power of two) hold a row, a warp 32 / G rows: `heads` heads of a
// token next to each other (of several tokens where there are fewer heads), and it goes
// through the token's heads.  What the angles, and the norm's weights, do to a row is a
// factor for each column and one for the column that shares its pair; a warp forms them
// once for a token, in shared memory, from where each row's lanes read them: held in
// registers they took a third of those, and of the warps that cover DRAM's latency.
// Arithmetic is on pairs of fp32 (packed operations).  The kernels are bound by reading and
// writing the rows, those of the norm by the warps that cover DRAM's latency (half of the issue
// slots stay free).
#pragma once

#include "ra_device.cuh"

namespace ra {

constexpr int kRotThreads = 256, kRotWarps = kRotThreads / 32;
constexpr int kRotMaxD = kRotMaxHead;
constexpr int kRotSmemSm = 227 * 1024;  // shared memory of an SM that blocks may have

// Where the other column of a pair is: in the same piece; in the lane's other piece (rot a
// multiple of 16); anywhere in the row, reached through shared memory.
enum RotExchange { ROT_PIECE = 0, ROT_OTHER = 1, ROT_STAGE = 2 };

// Dynamic shared memory of a block: frequencies | weights | per warp: the factors of its
// tokens' columns, C then S (tile d floats each), and where q and k have weights of their own
// another pair; staged rows (ROT_STAGE); sums of the weights' gradients (backward).
template <int EX, bool BWD>
struct RotSmem {
  static constexpr int kWeights = kRotMaxD / 2 * 8;
  static constexpr int kWarps = kWeights + 2 * kRotMaxD * 4;
  static constexpr int kStageRow = 65;  // floats of one column in eight
  int stage, sums, warp, bytes;         // in a warp's part; a warp's part; a block's
  __host__ __device__ RotSmem(const RotaryArgs& a, int sides) {
    stage = sides * 2 * a.tile * a.d * 4;
    sums = stage + (EX == ROT_STAGE ? 8 * kStageRow * 4 + 32 : 0);  // 2112: a multiple of 16
    warp = sums + (BWD ? 2 * (32 / a.G) * a.d * 4 : 0);
    bytes = kWarps + kRotWarps * warp;
  }
};

// Eight columns of one row as they are in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
// What is not there keeps what r held.
template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* p, bool there) {
  if (there) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
}
template <typename T>
__device__ __forceinline__ void zero8(Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ float2 pair_of(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(uint32_t v, __half) { return unpack_half2(v); }
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float2 (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = make_float2(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
      f[2 * i + 1] = make_float2(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
    }
  } else {
    f[0] = pair_of(r.v[0].x, T());
    f[1] = pair_of(r.v[0].y, T());
    f[2] = pair_of(r.v[0].z, T());
    f[3] = pair_of(r.v[0].w, T());
  }
}
__device__ __forceinline__ uint32_t pack_pair(float2 f, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_pair(float2 f, __half) { return pack_half2(f.x, f.y); }
template <typename T>
__device__ __forceinline__ void pack8(Raw8<T>& r, const float2 (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y), __float_as_uint(f[2 * i + 1].x),
                          __float_as_uint(f[2 * i + 1].y));
  } else {
    r.v[0] = make_uint4(pack_pair(f[0], T()), pack_pair(f[1], T()), pack_pair(f[2], T()), pack_pair(f[3], T()));
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float2 (&f)[4]) {
  Raw8<T> r;
  pack8(r, f);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

__device__ __forceinline__ float load_any(const void* p, int dtype, int i) {
  return dtype == RA_F32    ? static_cast<const float*>(p)[i]
         : dtype == RA_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i])
                            : to_f32(static_cast<const __half*>(p)[i]);
}

// cos and sin of the phase (top 32 bits of position x frequency), times `amplitude`.  The
// phase is brought within an eighth of a turn in integers, so that its conversion to fp32
// is off by 2^-28 turns at most.  FAST, for results of 16-bit types: the hardware's sine and
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

// F of a frequency in radians per position: f times 1 / 2 pi in two doubles, whole turns of
// each taken away, the upper 32 bits of the fraction, then the lower ones with what the product lost.
__device__ __forceinline__ unsigned long long fixed_turns(double f) {
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;  // 1 / 2 pi
  const double hi = f * kInv, lo = fma(f, kInv, -hi) + f * kInvLow;
  const double turns = (hi - rint(hi)) * 4294967296.0, upper = rint(turns);
  const double lower = rint((turns - upper + (lo - rint(lo)) * 4294967296.0) * 4294967296.0);
  return ((unsigned long long)(long long)upper << 32) + (unsigned long long)(long long)lower;
}

__device__ __forceinline__ long long rot_position(const RotaryArgs& a, long long b, int n) {
  if (a.positions) return __ldg(a.positions + b * a.pos_bstride + n);
  if (a.striped) {
    const int host = n / a.S;
    n = (n - host * a.S) * a.P + host;
  }
  return a.pos_off + n;
}

// Sum over the G lanes of a row.
__device__ __forceinline__ float group_sum(float v, int G) {
#pragma unroll
  for (int o = 8; o; o >>= 1)
    if (o < G) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's place: group g holds the row of a token (t0 + token) and a head (h + head), this
// lane its columns e[0] .. + 8 and e[1] .. + 8 where they are there.
struct RotLane {
  int g, s, token, head;
  int e[2];
  bool there[2];
  uint32_t turned[2];  // bit j: column e + j belongs to a pair
};
template <int EX>
__device__ __forceinline__ RotLane rot_lane(const RotaryArgs& a) {
  RotLane l;
  const int lane = (int)lane_id(), pieces = a.d / 8;
  l.g = lane / a.G;
  l.s = lane - l.g * a.G;
  l.token = l.g / a.heads;
  l.head = l.g - l.token * a.heads;
  int p[2];
  const int pairs = EX == ROT_OTHER ? a.rot / 16 : 0;  // lanes that hold pairs of pieces
  if (l.s < pairs) {
    p[0] = l.s;
    p[1] = l.s + pairs;
  } else {
    const int rest = pieces - 2 * pairs, step = (rest + 1) / 2;
    p[0] = 2 * pairs + l.s - pairs;
    p[1] = p[0] + step;
    if (l.s - pairs >= step) p[0] = p[1] = pieces;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l.there[i] = p[i] < pieces;
    l.e[i] = 8 * p[i];
    const int left = a.rot - l.e[i];
    l.turned[i] = !l.there[i] || left <= 0 ? 0u : left >= 8 ? 0xffu : (1u << left) - 1u;
  }
  return l;
}

// The other columns of the pairs of this lane's columns; 0 for columns of no pair, whose
// factor is -0 (x 1 + 0 (-0) is x, whatever the neighbour holds).  ALL: every column
// belongs to a pair.  `stage`: column p of a group's row sits at [p % 8][g 2G + p / 8], so
// that neither the writes nor the reads, at any distance, meet in a bank.
template <int EX, bool ALL>
__device__ __forceinline__ void other_columns(const RotaryArgs& a, const RotLane& l, const float2 (&f)[2][4],
                                              float2 (&p)[2][4], float* stage) {
  if constexpr (EX == ROT_STAGE) {
    constexpr int R = RotSmem<EX, false>::kStageRow;
    const int half = a.rot / 2, row = l.g * 2 * a.G;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (l.there[i]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          stage[2 * j * R + row + l.e[i] / 8] = f[i][j].x;
          stage[(2 * j + 1) * R + row + l.e[i] / 8] = f[i][j].y;
        }
      }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = l.e[i] + j, at = e < half ? e + half : e - half;
        const float v = (l.turned[i] >> j) & 1u ? stage[(at & 7) * R + row + (at >> 3)] : 0.f;
        if (j & 1) p[i][j / 2].y = v;
        else p[i][j / 2].x = v;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 o = EX == ROT_OTHER ? f[1 - i][j] : make_float2(f[i][j].y, f[i][j].x);
        const bool turned = ALL || ((EX == ROT_OTHER ? l.turned[i] : l.turned[i] >> (2 * j)) & 1u);
        p[i][j] = turned ? o : make_float2(0.f, 0.f);
      }
  }
}

// Column c of a token's factors: the first four of each eight, then the others, so that the
// lanes' reads of four lie beside each other.
__device__ __forceinline__ int rot_column(int d, int c) { return (c & 4 ? d / 2 : 0) + (c >> 3) * 4 + (c & 3); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight columns' values: at p, and `half` floats further.
__device__ __forceinline__ void columns8(float2 (&v)[4], const float* p, int half) {
  const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + half);
  v[0] = make_float2(x.x, x.y);
  v[1] = make_float2(x.z, x.w);
  v[2] = make_float2(y.x, y.y);
  v[3] = make_float2(y.z, y.w);
}

// Batch entry and row of a token.
__device__ __forceinline__ void rot_token(const RotaryArgs& a, long long t, long long* b, long long* n) {
  if (a.N == a.tokens) {
    *b = 0;
    *n = t;
  } else if (a.tokens < (1ll << 31)) {
    const uint32_t q = (uint32_t)t / (uint32_t)a.N;
    *b = q;
    *n = (uint32_t)t - q * (uint32_t)a.N;
  } else {
    *b = t / a.N;
    *n = t - *b * a.N;
  }
}

// Offset of row (token t, head h); t = b N + n.
__device__ __forceinline__ long long rot_offset(const RotaryArgs& a, const Lay& L, long long t, long long b, long long n, int h) {
  return a.flat ? t * L.rs + h * L.hs : lay_at(L, b, n, h);
}

// The columns of a pair.
template <int EX>
__device__ __forceinline__ void rot_pair(const RotaryArgs& a, int pair, int* x, int* y) {
  *x = EX == ROT_PIECE ? 2 * pair : pair;
  *y = EX == ROT_PIECE ? 2 * pair + 1 : pair + a.rot / 2;
}

// The factors of a warp's tokens t0, t0 + 1, ...: C of each column, S of the column that
// shares its pair (1 and -0 where none does).  With WEIGHTS those of q, then those of k, times
// the weights (w, w + d) of the columns that they multiply.  DIR: 1 turns by the angle, -1 by
// its opposite (the transpose, for gradients).
template <int EX, bool FAST, int DIR, bool WEIGHTS>
__device__ __forceinline__ void rot_factors(const RotaryArgs& a, const unsigned long long* freq, const float* w, long long t0,
                                            float* factors) {
  const int half = a.rot / 2, S = a.tile * a.d;
  __syncwarp();
  for (int g = 0; g < a.tile && t0 + g < a.tokens; ++g, factors += a.d) {
    if (half) {
      long long b, n;
      rot_token(a, t0 + g, &b, &n);
      const long long pos = rot_position(a, b, (int)n);
      for (int j = (int)lane_id(); j < half; j += 32) {
        const float2 t = turn<FAST>(freq[j], pos, a.amplitude);
        int x, y;
        rot_pair<EX>(a, j, &x, &y);
        float* const fx = factors + rot_column(a.d, x);
        float* const fy = factors + rot_column(a.d, y);
#pragma unroll
        for (int side = 0; side < (WEIGHTS ? 2 : 1); ++side) {
          const float wx = WEIGHTS ? w[side * a.d + x] : 1.f, wy = WEIGHTS ? w[side * a.d + y] : 1.f;
          fx[2 * side * S] = t.x * wx;
          fy[2 * side * S] = t.x * wy;
          fx[(2 * side + 1) * S] = -DIR * t.y * wy;
          fy[(2 * side + 1) * S] = DIR * t.y * wx;
        }
      }
    }
    for (int c = a.rot + (int)lane_id(); c < a.d; c += 32) {
      float* const f = factors + rot_column(a.d, c);
#pragma unroll
      for (int side = 0; side < (WEIGHTS ? 2 : 1); ++side) {
        f[2 * side * S] = WEIGHTS ? w[side * a.d + c] : 1.f;
        f[(2 * side + 1) * S] = -0.f;
      }
    }
  }
  __syncwarp();
}

// Heads [first, last) of part `part` of a.parts, whole steps of a warp but for the last.
__device__ __forceinline__ void rot_heads(const RotaryArgs& a, int H, int part, int* first, int* last) {
  const int steps = (H + a.heads - 1) / a.heads;
  *first = a.parts == 1 ? 0 : steps * part / a.parts * a.heads;
  *last = a.parts == 1 ? H : min(H, steps * (part + 1) / a.parts * a.heads);
}

// A row whose sum of squares left fp32's range (or is NaN) is scaled, and its sum formed again:
// by 2^-70, or by 2^100 where the squares may have vanished and eps would not hide it.
__device__ __forceinline__ float rot_least(const RotaryArgs& a) { return a.eps < 1e-30f ? 1e-30f : 0.f; }
__device__ __forceinline__ float rot_scale(float sum, float least) {
  return sum < least ? 1.2676506002282294e30f : sum < 1e37f ? 1.f : 8.470329472543003e-22f;
}

}  // namespace ra
