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

// Blocks of an SM: 128 registers a thread.  (131072 tokens of 16 + 4 heads of 128, bf16: 466
// us with the sum of dw's parts, 4.3 TB/s; with three, whose 80 registers spill, 593.)
constexpr int kBlocks = 2;

template <typename T, typename TG, typename TO, int EX, bool ALL>
__device__ __forceinline__ void gradient_rows(const RotaryArgs& a, const RotLane& l, const RotarySide& side, const float* weight,
                                              const float* factors, const T* x, const TG* dy,
                                              TO* out, bool token, int h0, int h1, float* stage, float* sums) {
  const long long x_step = a.heads * side.xl.hs, dy_step = a.heads * side.dyl.hs, out_step = a.heads * side.yl.hs;
  const float inv_d = 1.f / (float)a.d, least = rot_least(a);
  float2 dw[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = both(0.f);
  int at[2];  // columns that are there
  const float *C[2], *W[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at[i] = l.there[i] ? l.e[i] : 0;
    C[i] = factors + l.token * a.d + at[i] / 2;
    W[i] = weight + at[i];
  }
  for (int h = h0; h < h1; h += a.heads, x += x_step, dy += dy_step, out += out_step) {
    const bool row = token && h + l.head < h1;
    // x stays as it was read, in half the registers, and is unpacked twice.  A head that is
    // not there reads the step's first.
    Raw8<T> rx[2];
    Raw8<TG> rg[2];
    const T* px = x;
    const TG* pg = dy;
    if (h + a.heads > h1 && h + l.head >= h1) {
      px -= l.head * side.xl.hs;
      pg -= l.head * side.dyl.hs;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load8(rx[i], px + at[i], true);
      load8(rg[i], pg + at[i], true);
    }
    float2 g[2][4], s2[2], d2[2];
    {
      float2 y[2][4], p[2][4];
      unpack8(rg[0], y[0]);
      unpack8(rg[1], y[1]);
      other_columns<EX, ALL>(a, l, y, p, stage);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 c[4], sn[4];
        columns8(c, C[i], a.d / 2);
        columns8(sn, C[i] + a.tile * a.d, a.d / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[i][j] = __ffma2_rn(y[i][j], c[j], __fmul2_rn(p[i][j], sn[j]));
      }
    }
    // the sums for the norm's factor
    auto sums_of = [&] {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 f[4], w[4];
        unpack8(rx[i], f);
        columns8(w, W[i], 4);
        s2[i] = d2[i] = both(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i] = __ffma2_rn(f[j], f[j], s2[i]);
          d2[i] = __ffma2_rn(__fmul2_rn(g[i][j], w[j]), f[j], d2[i]);
        }
      }
    };
    sums_of();
    auto of_row = [&](const float2 (&v)[2]) {
      return group_sum((l.there[0] ? v[0].x + v[0].y : 0.f) + (l.there[1] ? v[1].x + v[1].y : 0.f), a.G);
    };
    float sum = of_row(s2), dot = of_row(d2), eps = a.eps, sc = 1.f;
    if (__any_sync(0xffffffffu, !(sum < 1e37f && sum >= least))) {
      // x in place, in its type: a power of two loses only what is 2^-100 of the row's largest
      // (fp16 rows get here with zeros, infinities and NaN only)
      sc = rot_scale(sum, least);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 f[4];
        unpack8(rx[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], both(sc));
        pack8(rx[i], f);
      }
      sums_of();
      sum = of_row(s2);
      dot = of_row(d2);
      eps = eps * sc * sc;
    }
    const float r = rsqrtf(fmaf(sum, inv_d, eps));
    const float2 rs = both(r * sc), along = both(-dot * r * inv_d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 f[4], w[4], dx[4];
      unpack8(rx[i], f);
      columns8(w, W[i], 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 normed = __fmul2_rn(f[j], both(r));
        if (row) dw[i][j] = __ffma2_rn(g[i][j], normed, dw[i][j]);
        dx[j] = __fmul2_rn(rs, __ffma2_rn(normed, along, __fmul2_rn(g[i][j], w[j])));
      }
      if (row && l.there[i]) store8(out + l.e[i], dx);
    }
  }
  // this lane's own sums in shared memory
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (l.there[i]) {
      float4* p = reinterpret_cast<float4*>(sums + l.g * a.d + l.e[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float4 v = p[j];
        v.x += dw[i][2 * j].x;
        v.y += dw[i][2 * j].y;
        v.z += dw[i][2 * j + 1].x;
        v.w += dw[i][2 * j + 1].y;
        p[j] = v;
      }
    }
}

template <typename T, typename TG, typename TO, int EX, bool ALL>
__global__ void __launch_bounds__(kRotThreads, kBlocks) norm_rotary_bwd_kernel(const __grid_constant__ RotaryArgs a) {
  using Smem = RotSmem<EX, true>;
  const Smem L(a, 1);
  extern __shared__ __align__(16) uint8_t smem[];
  unsigned long long* freq = reinterpret_cast<unsigned long long*>(smem);
  float* weight = reinterpret_cast<float*>(smem + Smem::kWeights);
  const int warp = threadIdx.x >> 5, groups = 32 / a.G;
  auto of_warp = [&](int w, int at) { return smem + Smem::kWarps + w * L.warp + at; };
  float* factors = reinterpret_cast<float*>(of_warp(warp, 0));
  float* stage = reinterpret_cast<float*>(of_warp(warp, L.stage));
  float* sums = reinterpret_cast<float*>(of_warp(warp, L.sums));  // [side][group][d]
  const RotLane l = rot_lane<EX>(a);
  const long long first = (long long)blockIdx.x * kRotWarps + warp, step = (long long)gridDim.x * kRotWarps;
  for (int i = threadIdx.x; i < a.rot / 2; i += kRotThreads) freq[i] = fixed_turns(a.freq[i]);
  for (int i = threadIdx.x; i < 2 * a.d; i += kRotThreads) {
    const int side = i >= a.d, c = i - side * a.d;
    weight[i] = a.side[side].w ? load_any(a.side[side].w, a.w_dtype, c) : 1.f;
  }
  for (int i = (int)lane_id(); i < 2 * groups * a.d; i += 32) sums[i] = 0.f;
  __syncthreads();
  for (long long unit = first; unit < a.units; unit += step) {
    const long long tile = a.parts == 1 ? unit : unit / a.parts;
    const int part = (int)(unit - tile * a.parts);
    const long long t0 = tile * a.tile;
    rot_factors<EX, sizeof(TO) == 2, -1, false>(a, freq, nullptr, t0, factors);
    const bool token = t0 + l.token < a.tokens;
    const long long t = token ? t0 + l.token : t0;
    long long b, n;
    rot_token(a, t, &b, &n);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const RotarySide& s = a.side[side];
      int h0, h1;
      rot_heads(a, s.H, part, &h0, &h1);
      if (h0 == h1) continue;
      const T* x = static_cast<const T*>(s.x) + rot_offset(a, s.xl, t, b, n, h0 + l.head);
      const TG* dy = static_cast<const TG*>(s.dy) + rot_offset(a, s.dyl, t, b, n, h0 + l.head);
      TO* out = static_cast<TO*>(s.y) + rot_offset(a, s.yl, t, b, n, h0 + l.head);
      gradient_rows<T, TG, TO, EX, ALL>(a, l, s, weight + side * a.d, factors, x, dy, out, token, h0, h1, stage,
                                        sums + side * groups * a.d);
    }
  }
  // the block's sums, over groups and warps in order
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.d; i += kRotThreads) {
    const int side = i >= a.d, c = i - side * a.d;
    float v = 0.f;
    for (int w = 0; w < kRotWarps; ++w) {
      const float* from = reinterpret_cast<const float*>(of_warp(w, L.sums)) + side * groups * a.d + c;
      for (int g = 0; g < groups; ++g) v += from[g * a.d];
    }
    a.dw_parts[((long long)side * gridDim.x + blockIdx.x) * a.d + c] = v;
  }
}

// dw = the sum of the blocks' sums, 32 columns a block: warp w adds up the blocks' sums w,
// w + 32, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) rotary_dw_kernel(const float* parts, int blocks, int d, float* dwq, float* dwk) {
  __shared__ float part[32][33];
  const int per = gridDim.x / 2, side = (int)blockIdx.x / per;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = ((int)blockIdx.x - side * per) * 32 + lane;
  float* out = side ? dwk : dwq;
  pdl_wait();  // in every block: what comes after may wait for this kernel alone
  if (!out) return;
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
  auto go = [&](auto kernel, int smem) {
    const long long want = (a.units + kRotWarps - 1) / kRotWarps, most = (long long)kBlocks * sms < kRotParts ? (long long)kBlocks * sms : kRotParts;
    const int blocks = (int)(want < most ? want : most);
    cudaError_t e = smem > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    kernel<<<blocks, kRotThreads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_pdl(rotary_dw_kernel, (a.d + 31) / 32 * 2, 1024, 0, st, a.dw_parts, blocks, a.d, dwq, dwk);
    if (e == cudaSuccess) count_launch(2);
    return e;
  };
  const int piece = RotSmem<ROT_PIECE, true>(a, 1).bytes, other = RotSmem<ROT_OTHER, true>(a, 1).bytes;
  if (exchange == ROT_PIECE)
    return a.rot == a.d ? go(norm_rotary_bwd_kernel<T, TG, TO, ROT_PIECE, true>, piece)
                        : go(norm_rotary_bwd_kernel<T, TG, TO, ROT_PIECE, false>, piece);
  if (exchange == ROT_OTHER)
    return a.rot == a.d ? go(norm_rotary_bwd_kernel<T, TG, TO, ROT_OTHER, true>, other)
                        : go(norm_rotary_bwd_kernel<T, TG, TO, ROT_OTHER, false>, other);
  return go(norm_rotary_bwd_kernel<T, TG, TO, ROT_STAGE, false>, RotSmem<ROT_STAGE, true>(a, 1).bytes);
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
