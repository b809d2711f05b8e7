// Gradients of the norm of each head with the rotation behind it, y = R(x r w):
//   g = R^T dy,  n = x r,  dw_c = sum over rows of g_c n_c,
//   dx = r (g w - n mean(g w n)).
// r is formed again from x, which has to be read anyway.  Each block writes its sums of dw
// to the workspace and a second kernel adds the blocks' sums in order: the results do not
// vary from run to run.  Bound by reading x and dy and writing dx.
#include <type_traits>

#include "ra_rotary.cuh"

namespace ra {
namespace {

template <typename T, typename TG, typename TO, int EX>
__global__ void __launch_bounds__(kRotThreads, 2) norm_rotary_bwd_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ unsigned long long freq[kRotMaxD / 2];
  __shared__ float weight[2][kRotMaxD];
  __shared__ float2 angles[kRotWarps][kRotMaxD / 2];
  __shared__ float stages[EX == ROT_STAGE ? kRotWarps : 1][EX == ROT_STAGE ? 8 * 33 : 1];
  __shared__ float sums[kRotWarps][kRotMaxD];
  constexpr int U = 2;  // rows in flight
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.rot / 2; i += kRotThreads) freq[i] = fixed_turns(a.freq[i]);
  for (int i = threadIdx.x; i < 2 * a.d; i += kRotThreads) {
    const int side = i >= a.d, c = i - side * a.d;
    weight[side][c] = a.side[side].w ? load_any(a.side[side].w, a.w_dtype, c) : 1.f;
  }
  __syncthreads();
  const RotLane l = rot_lane<EX>(a);
  float2* cs = angles[warp];
  float* stage = stages[EX == ROT_STAGE ? warp : 0];
  const float inv_d = 1.f / (float)a.d;
  float dw[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
  const long long first = (long long)blockIdx.x * kRotWarps + warp, step = (long long)gridDim.x * kRotWarps;
  for (long long unit = first; unit < a.units; unit += step) {
    const long long tile = unit / a.parts;
    const int part = (int)(unit - tile * a.parts);
    const long long t0 = tile * (32 / a.G), t = t0 + l.g;
    rot_angles<sizeof(T) == 2>(a, freq, t0, cs);
    const bool there = l.column && t < a.tokens;
    const long long b = t / a.N, n = t - b * a.N;
    float C[8], S[8];
    rot_factors<EX, -1>(a, l, cs, C, S);
    auto rows = [&](const RotarySide& s, const float* ws, float (&dws)[8]) {
      int h0, h1;
      rot_heads(s.H, part, a.parts, &h0, &h1);
      if (h0 == h1) return;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = l.column ? ws[8 * l.c + j] : 0.f;
      const T* x = static_cast<const T*>(s.x) + lay_at(s.xl, b, n, 0) + 8 * l.c;
      const TG* dy = static_cast<const TG*>(s.dy) + lay_at(s.dyl, b, n, 0) + 8 * l.c;
      TO* out = static_cast<TO*>(s.y) + lay_at(s.yl, b, n, 0) + 8 * l.c;
      for (int h = h0; h < h1; h += U) {
        Raw8<T> rx[U];
        Raw8<TG> rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u] = load8(x + (h + u) * s.xl.hs, there && h + u < h1);
          rg[u] = load8(dy + (h + u) * s.dyl.hs, there && h + u < h1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u >= h1) break;
          float f[8], g[8], p[8], dx[8];
          unpack8(rg[u], g);
          other_columns<EX>(a, l, rg[u], g, p, stage);
          unpack8(rx[u], f);
          float sum = 0.f, dot = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            g[j] = fmaf(g[j], C[j], p[j] * S[j]);
            sum = fmaf(f[j], f[j], sum);
            dot = fmaf(g[j] * w[j], f[j], dot);
          }
          sum = group_sum(sum, a.G);
          dot = group_sum(dot, a.G);
          float eps = a.eps, sc = 1.f;
          if (__any_sync(0xffffffffu, !(sum < 1e37f))) {
            sc = rot_scale(sum);
            sum = dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] *= sc;
              sum = fmaf(f[j], f[j], sum);
              dot = fmaf(g[j] * w[j], f[j], dot);
            }
            sum = group_sum(sum, a.G);
            dot = group_sum(dot, a.G);
            eps *= sc * sc;
          }
          const float r = rsqrtf(fmaf(sum, inv_d, eps)), along = dot * r * inv_d, rs = r * sc;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float normed = f[j] * r;
            dws[j] = fmaf(g[j], normed, dws[j]);
            dx[j] = rs * fmaf(-normed, along, g[j] * w[j]);
          }
          if (there) store8(out + (h + u) * s.yl.hs, dx);
        }
      }
    };
    rows(a.side[0], weight[0], dw[0]);
    rows(a.side[1], weight[1], dw[1]);
  }
  // the block's sums: over the rows of a warp, then over its warps, in order
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = dw[side][j];
      for (int o = a.G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (l.g == 0 && l.column) sums[warp][8 * l.c + j] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kRotThreads) {
      float v = sums[0][c];
      for (int i = 1; i < kRotWarps; ++i) v += sums[i][c];
      a.dw_parts[((long long)side * gridDim.x + blockIdx.x) * a.d + c] = v;
    }
    __syncthreads();
  }
}

// dw = the sum of the blocks' sums, 32 columns a block: warp w adds up the blocks' sums w,
// w + 32, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) rotary_dw_kernel(const float* parts, int blocks, int d, float* dwq, float* dwk) {
  __shared__ float part[32][33];
  const int per = gridDim.x / 2, side = (int)blockIdx.x / per;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = ((int)blockIdx.x - side * per) * 32 + lane;
  float* out = side ? dwk : dwq;
  if (!out) return;
  pdl_wait();
  float v = 0.f;
  if (c < d)
    for (int b = w; b < blocks; b += 32) v += parts[((long long)side * blocks + b) * d + c];
  part[w][lane] = v;
  __syncthreads();
  if (w) return;
  for (int i = 1; i < 32; ++i) v += part[i][lane];
  if (c < d) out[c] = v;
}

template <typename T, typename TG, typename TO>
cudaError_t run(const RotaryArgs& a, int exchange, float* dwq, float* dwk, int sms, cudaStream_t st) {
  auto go = [&](auto kernel) {
    const long long want = (a.units + kRotWarps - 1) / kRotWarps, most = 2ll * sms < kRotParts ? 2ll * sms : kRotParts;
    const int blocks = (int)(want < most ? want : most);
    kernel<<<blocks, kRotThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_pdl(rotary_dw_kernel, (a.d + 31) / 32 * 2, 1024, 0, st, a.dw_parts, blocks, a.d, dwq, dwk);
    if (e == cudaSuccess) count_launch(2);
    return e;
  };
  if (exchange == ROT_THREAD) return go(norm_rotary_bwd_kernel<T, TG, TO, ROT_THREAD>);
  if (exchange == ROT_SHUFFLE) return go(norm_rotary_bwd_kernel<T, TG, TO, ROT_SHUFFLE>);
  return go(norm_rotary_bwd_kernel<T, TG, TO, ROT_STAGE>);
}

}  // namespace

cudaError_t launch_norm_rotary_bwd(RotaryArgs& a, int interleaved, int dtype, int g_dtype, int grad_dtype, float* dwq,
                                   float* dwk, int sms, cudaStream_t st) {
  rot_units(a, sms);
  const int ex = rot_exchange(a.rot, interleaved);
  auto types = [&](auto x) {
    using T = decltype(x);
    if (g_dtype == RA_F32)
      return grad_dtype == RA_F32 ? run<T, float, float>(a, ex, dwq, dwk, sms, st)
                                  : run<T, float, T>(a, ex, dwq, dwk, sms, st);
    return grad_dtype == RA_F32 ? run<T, T, float>(a, ex, dwq, dwk, sms, st) : run<T, T, T>(a, ex, dwq, dwk, sms, st);
  };
  // the gradients are of the rows' own type or fp32
  if ((g_dtype != dtype && g_dtype != RA_F32) || (grad_dtype != dtype && grad_dtype != RA_F32))
    return cudaErrorInvalidValue;
  if (dtype == RA_F32) return run<float, float, float>(a, ex, dwq, dwk, sms, st);
  return dtype == RA_BF16 ? types(__nv_bfloat16{}) : types(__half{});
}

}  // namespace ra
