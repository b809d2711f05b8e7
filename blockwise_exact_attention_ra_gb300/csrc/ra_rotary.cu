// Rotary positions of queries and keys, alone or with the norm of each head in the same
// pass, forward (and the gradient of the rotation, which is the rotation back).
//   r = (mean x^2 + eps)^-1/2,   y = R(x r w)
// What the weights and the rotation do to a row is one pair of factors for each column,
// formed once for a token and a tensor: y_c = r (x_c C_c + x_c' S_c), c' the pair's other
// column, C_c = w_c A cos, S_c = -+ w_c' A sin.
#include <type_traits>

#include "ra_rotary.cuh"

namespace ra {
namespace {

template <typename T, typename TO, bool NORM, int EX, int DIR>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ unsigned long long freq[kRotMaxD / 2];
  __shared__ float weight[NORM ? 2 : 1][NORM ? kRotMaxD : 1];
  __shared__ float2 angles[kRotWarps][kRotMaxD / 2];
  __shared__ float stages[EX == ROT_STAGE ? kRotWarps : 1][EX == ROT_STAGE ? 8 * 33 : 1];
  constexpr int U = sizeof(T) == 4 ? 2 : 4;  // rows in flight
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.rot / 2; i += kRotThreads) freq[i] = fixed_turns(a.freq[i]);
  if (NORM)
    for (int i = threadIdx.x; i < 2 * a.d; i += kRotThreads) {
      const int side = i >= a.d, c = i - side * a.d;
      weight[side][c] = a.side[side].w ? load_any(a.side[side].w, a.w_dtype, c) : 1.f;
    }
  __syncthreads();
  const RotLane l = rot_lane<EX>(a);
  float2* cs = angles[warp];
  float* stage = stages[EX == ROT_STAGE ? warp : 0];
  const float inv_d = 1.f / (float)a.d;
  const long long first = (long long)blockIdx.x * kRotWarps + warp, step = (long long)gridDim.x * kRotWarps;
  for (long long unit = first; unit < a.units; unit += step) {
    const long long tile = unit / a.parts;
    const int part = (int)(unit - tile * a.parts);
    const long long t0 = tile * (32 / a.G), t = t0 + l.g;
    rot_angles<sizeof(TO) == 2>(a, freq, t0, cs);
    const bool there = l.column && t < a.tokens;
    const long long b = t / a.N, n = t - b * a.N;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const RotarySide& s = a.side[side];
      int h0, h1;
      rot_heads(s.H, part, a.parts, &h0, &h1);
      if (h0 == h1) continue;
      float C[8], S[8];
      rot_factors<EX, DIR>(a, l, cs, C, S);
      if (NORM && l.column) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * l.c + j;
          C[j] *= weight[side][e];
          if ((l.turned >> j) & 1u) S[j] *= weight[side][other_column<EX>(a, e)];
        }
      }
      const T* in = static_cast<const T*>(s.x) + lay_at(s.xl, b, n, 0) + 8 * l.c;
      TO* out = static_cast<TO*>(s.y) + lay_at(s.yl, b, n, 0) + 8 * l.c;
      for (int h = h0; h < h1; h += U) {
        Raw8<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load8(in + (h + u) * s.xl.hs, there && h + u < h1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u >= h1) break;
          float f[8], p[8], y[8], r = 1.f;
          unpack8(raw[u], f);
          other_columns<EX>(a, l, raw[u], f, p, stage);
          if (NORM) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
            sum = group_sum(sum, a.G);
            float eps = a.eps;
            if (__any_sync(0xffffffffu, !(sum < 1e37f))) {
              const float sc = rot_scale(sum);
              sum = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                f[j] *= sc;
                p[j] *= sc;
                sum = fmaf(f[j], f[j], sum);
              }
              sum = group_sum(sum, a.G);
              eps *= sc * sc;
            }
            r = rsqrtf(fmaf(sum, inv_d, eps));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[j] = fmaf(f[j], C[j], p[j] * S[j]);
            if (NORM) y[j] *= r;
          }
          if (there) store8(out + (h + u) * s.yl.hs, y);
        }
      }
    }
  }
}

template <typename T, typename TO, bool NORM, int DIR>
cudaError_t run(const RotaryArgs& a, int exchange, int sms, cudaStream_t st) {
  auto go = [&](auto kernel) {
    const long long blocks = (a.units + kRotWarps - 1) / kRotWarps, most = (long long)sms * 8;
    kernel<<<(unsigned)(blocks < most ? blocks : most), kRotThreads, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
  };
  if (exchange == ROT_THREAD) return go(rotary_kernel<T, TO, NORM, ROT_THREAD, DIR>);
  if (exchange == ROT_SHUFFLE) return go(rotary_kernel<T, TO, NORM, ROT_SHUFFLE, DIR>);
  return go(rotary_kernel<T, TO, NORM, ROT_STAGE, DIR>);
}

}  // namespace

int rot_exchange(int rot, int interleaved) {
  return interleaved || rot == 0 ? ROT_THREAD : rot % 16 == 0 ? ROT_SHUFFLE : ROT_STAGE;
}

// A warp takes the tokens of its groups; where that leaves SMs without work (few tokens),
// the heads of a tile of tokens are split over several warps.
void rot_units(RotaryArgs& a, int sms) {
  a.G = 1;
  while (a.G * 8 < a.d) a.G *= 2;
  const long long tiles = (a.tokens + 32 / a.G - 1) / (32 / a.G);
  const int most = a.side[0].H > a.side[1].H ? a.side[0].H : a.side[1].H;
  a.parts = 1;
  while (2 * a.parts <= most && tiles * a.parts < (long long)sms * kRotWarps) a.parts *= 2;
  a.units = tiles * a.parts;
}

cudaError_t launch_rotary(RotaryArgs& a, int interleaved, int dtype, int out_dtype, int norm, int grad, int sms,
                          cudaStream_t st) {
  rot_units(a, sms);
  const int ex = rot_exchange(a.rot, interleaved);
  if (norm) {
    if (grad || dtype != out_dtype) return cudaErrorInvalidValue;
    return dtype == RA_F32    ? run<float, float, true, 1>(a, ex, sms, st)
           : dtype == RA_BF16 ? run<__nv_bfloat16, __nv_bfloat16, true, 1>(a, ex, sms, st)
                              : run<__half, __half, true, 1>(a, ex, sms, st);
  }
  auto way = [&](auto dir) {
    constexpr int DIR = decltype(dir)::value;
    if (dtype == RA_BF16 && out_dtype == RA_BF16) return run<__nv_bfloat16, __nv_bfloat16, false, DIR>(a, ex, sms, st);
    if (dtype == RA_F16 && out_dtype == RA_F16) return run<__half, __half, false, DIR>(a, ex, sms, st);
    if (dtype != RA_F32) return cudaErrorInvalidValue;
    if (out_dtype == RA_F32) return run<float, float, false, DIR>(a, ex, sms, st);
    if constexpr (DIR < 0)
      return out_dtype == RA_BF16 ? run<float, __nv_bfloat16, false, DIR>(a, ex, sms, st)
                                  : run<float, __half, false, DIR>(a, ex, sms, st);
    return cudaErrorInvalidValue;
  };
  return grad ? way(std::integral_constant<int, -1>{}) : way(std::integral_constant<int, 1>{});
}

}  // namespace ra
