// Rotary positions of queries and keys, alone or with the norm of each head in the same
// pass, forward (and the gradient of the rotation, which is the rotation back).
//   r = (mean x^2 + eps)^-1/2,   y = R(x r w)
// A row: y_c = r (x_c C_c + x_c' S_c), c' the pair's other column, C_c = w_c A cos,
// S_c = -+ w_c' A sin.
#include <type_traits>

#include "ra_rotary.cuh"

namespace ra {
namespace {

// Blocks of an SM: 64 registers a thread.  (131072 tokens of 16 + 4 heads of 128, bf16: 216 us,
// with the norm 258 us; with three 226 and 276, with two 248 and 323.)
constexpr int kBlocks = 4;

template <typename T, typename TO, bool NORM, int EX, bool ALL>
__device__ __forceinline__ void rotate_rows(const RotaryArgs& a, const RotLane& l, const RotarySide& side, const float* factors,
                                            const T* in, TO* out, bool token, int h0, int h1, float* stage) {
  const long long in_step = a.heads * side.xl.hs, out_step = a.heads * side.yl.hs;
  const float inv_d = 1.f / (float)a.d, least = rot_least(a);
  const float* C[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) C[i] = factors + l.token * a.d + (l.there[i] ? l.e[i] / 2 : 0);
  Raw8<T> raw[2];  // what is not there: zeros, or rows before
  zero8(raw[0]);
  zero8(raw[1]);
  for (int h = h0; h < h1; h += a.heads, in += in_step, out += out_step) {
    const bool row = token && h + l.head < h1;
#pragma unroll
    for (int i = 0; i < 2; ++i) load8(raw[i], in + l.e[i], row && l.there[i]);
    float2 f[2][4], p[2][4], r = both(1.f);
    unpack8(raw[0], f[0]);
    unpack8(raw[1], f[1]);
    if (NORM) {
      float2 s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(f[i][j], f[i][j], s2);
      float sum = group_sum(s2.x + s2.y, a.G), eps = a.eps;
      if (__any_sync(0xffffffffu, !(sum < 1e37f && sum >= least))) {
        const float sc = rot_scale(sum, least);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[i][j] = __fmul2_rn(f[i][j], both(sc));
            sum = fmaf(f[i][j].y, f[i][j].y, fmaf(f[i][j].x, f[i][j].x, sum));
          }
        sum = group_sum(sum, a.G);
        eps = eps * sc * sc;
      }
      r = both(rsqrtf(fmaf(sum, inv_d, eps)));
    }
    other_columns<EX, ALL>(a, l, f, p, stage);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 y[4], c[4], sn[4];
      columns8(c, C[i], a.d / 2);
      columns8(sn, C[i] + a.tile * a.d, a.d / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = __ffma2_rn(f[i][j], c[j], __fmul2_rn(p[i][j], sn[j]));
        if (NORM) y[j] = __fmul2_rn(y[j], r);
      }
      if (row && l.there[i]) store8(out + l.e[i], y);
    }
  }
}

// ALL: every column belongs to a pair.
template <typename T, typename TO, bool NORM, int EX, int DIR, bool ALL>
__global__ void __launch_bounds__(kRotThreads, kBlocks) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  using Smem = RotSmem<EX, false>;
  const Smem L(a, NORM ? 2 : 1);
  extern __shared__ __align__(16) uint8_t smem[];
  unsigned long long* freq = reinterpret_cast<unsigned long long*>(smem);
  float* weight = reinterpret_cast<float*>(smem + Smem::kWeights);
  const int warp = threadIdx.x >> 5;
  float* factors = reinterpret_cast<float*>(smem + Smem::kWarps + warp * L.warp);
  float* stage = reinterpret_cast<float*>(smem + Smem::kWarps + warp * L.warp + L.stage);
  for (int i = threadIdx.x; i < a.rot / 2; i += kRotThreads) freq[i] = fixed_turns(a.freq[i]);
  if (NORM)
    for (int i = threadIdx.x; i < 2 * a.d; i += kRotThreads) {
      const int side = i >= a.d, c = i - side * a.d;
      weight[i] = a.side[side].w ? load_any(a.side[side].w, a.w_dtype, c) : 1.f;
    }
  __syncthreads();
  const RotLane l = rot_lane<EX>(a);
  const long long first = (long long)blockIdx.x * kRotWarps + warp, step = (long long)gridDim.x * kRotWarps;
  for (long long unit = first; unit < a.units; unit += step) {
    const long long tile = a.parts == 1 ? unit : unit / a.parts;
    const int part = (int)(unit - tile * a.parts);
    const long long t0 = tile * a.tile;
    const bool token = t0 + l.token < a.tokens;
    const long long t = token ? t0 + l.token : t0;
    long long b, n;
    rot_token(a, t, &b, &n);
    rot_factors<EX, sizeof(TO) == 2, DIR, NORM>(a, freq, weight, t0, factors);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const RotarySide& s = a.side[side];
      int h0, h1;
      rot_heads(a, s.H, part, &h0, &h1);
      if (h0 == h1) continue;
      const float* const own = factors + (NORM ? side * 2 * a.tile * a.d : 0);
      const T* in = static_cast<const T*>(s.x) + rot_offset(a, s.xl, t, b, n, h0 + l.head);
      TO* out = static_cast<TO*>(s.y) + rot_offset(a, s.yl, t, b, n, h0 + l.head);
      rotate_rows<T, TO, NORM, EX, ALL>(a, l, s, own, in, out, token, h0, h1, stage);
    }
  }
}

template <typename T, typename TO, bool NORM, int DIR>
cudaError_t run(const RotaryArgs& a, int exchange, int sms, cudaStream_t st) {
  auto go = [&](auto kernel, int smem) {
    const int fit = kRotSmemSm / (smem + 1024);  // 3 where a warp's rows are of many tokens
    const long long blocks = (a.units + kRotWarps - 1) / kRotWarps, most = (long long)sms * (fit < kBlocks ? fit : kBlocks);
    cudaError_t e = smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(blocks < most ? blocks : most), kRotThreads, smem, st>>>(a);
    count_launch();
    return cudaGetLastError();
  };
  constexpr int sides = NORM ? 2 : 1;
  const int piece = RotSmem<ROT_PIECE, false>(a, sides).bytes, other = RotSmem<ROT_OTHER, false>(a, sides).bytes;
  if (exchange == ROT_PIECE)
    return a.rot == a.d ? go(rotary_kernel<T, TO, NORM, ROT_PIECE, DIR, true>, piece)
                        : go(rotary_kernel<T, TO, NORM, ROT_PIECE, DIR, false>, piece);
  if (exchange == ROT_OTHER)
    return a.rot == a.d ? go(rotary_kernel<T, TO, NORM, ROT_OTHER, DIR, true>, other)
                        : go(rotary_kernel<T, TO, NORM, ROT_OTHER, DIR, false>, other);
  return go(rotary_kernel<T, TO, NORM, ROT_STAGE, DIR, false>, RotSmem<ROT_STAGE, false>(a, sides).bytes);
}

}  // namespace

int rot_exchange(int rot, int interleaved) {
  return interleaved || rot == 0 ? ROT_PIECE : rot % 16 == 0 ? ROT_OTHER : ROT_STAGE;
}

// Where the tokens leave SMs without work (a few of them), their heads are split over
// several warps.
void rot_units(RotaryArgs& a, int sms) {
  a.G = 1;
  while (a.G * 16 < a.d) a.G *= 2;
  const int most = a.side[0].H > a.side[1].H ? a.side[0].H : a.side[1].H;
  a.heads = 1;
  while (a.heads * 2 <= 32 / a.G && a.heads * 2 <= a.side[0].H) a.heads *= 2;
  a.tile = 32 / a.G / a.heads;
  const long long tiles = (a.tokens + a.tile - 1) / a.tile;
  a.parts = 1;
  while (2 * a.parts * a.heads <= most && tiles * a.parts < (long long)sms * kRotWarps) a.parts *= 2;
  a.units = tiles * a.parts;
  a.flat = 1;
  if (a.N != a.tokens)
    for (const RotarySide& s : a.side)
      for (const Lay* L : {&s.xl, &s.dyl, &s.yl})
        if (s.H && L->bs != (long long)a.N * L->rs) a.flat = 0;
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
