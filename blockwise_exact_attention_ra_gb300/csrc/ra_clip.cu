// The global norm of the gradients of many tensors, and their clipping by it:
//   n = (sum over all tensors of g^2)^1/2,  c = min(1, max_norm / (n + eps)),  out = c g.
// The tensors' addresses and sizes go with the launch (the kernel's parameters), so that
// nothing is copied to the device beforehand and a captured call holds them.  A tensor is
// cut into chunks that start on 16-byte boundaries; the blocks take chunks in turn, in an
// order that depends on the sizes alone, and each leaves its sum in the workspace, where
// the second kernel's blocks add them up in order: the results do not vary from run to run.
//
// Squares are summed in fp32 over the at most 64 elements that a thread holds, and from
// there in fp64.  Where such a sum is outside [1e-30, 1e30) (elements whose squares leave
// fp32's range) the elements are squared and summed in fp64, so that gradients of any size
// have their norm.
//
// Bound by reading the gradients twice (the factor depends on all of them) and writing
// them once.  The second pass goes through the chunks from the last to the first: what the
// first one read last is still in L2.  Its chunks are small, a block each: what the GPU has
// open at a time then lies close together, for which a block of its own forms the factor.
// Few chunks are taken by blocks that form it each: a launch less.
// Measured: 2^29 bf16 elements, 8 tensors: 158 us for the sums (6.8 TB/s), 318 us for the
// second pass (6.75 TB/s; 460 us with 608 blocks that each go through chunks of 128 KB, 420 us
// with all pairs of types in one kernel).
#include <math.h>

#include <type_traits>

#include "ra_device.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;       // 16-byte vectors a thread holds while it sums
constexpr int kScaleBatch = 4;  // and while it scales

// A chunk: elements [lo, hi) of a tensor; those from `body` on sit on 16-byte boundaries.
struct Chunk {
  int tensor;
  long long lo, body, hi;
};

template <int MAX>
__device__ __forceinline__ Chunk find_chunk(const GradList<MAX>& a, int chunk) {
  int l = 0, r = a.count;  // first[l] <= chunk < first[r]
  while (r - l > 1) {
    const int m = (l + r) >> 1;
    if (a.first[m] <= chunk) l = m; else r = m;
  }
  Chunk c;
  c.tensor = l;
  const int size = (a.types[l] & 15) == RA_F32 ? 4 : 2;
  const long long n = a.n[l], k = chunk - a.first[l];
  const long long lead = (long long)((16u - (unsigned)((uintptr_t)a.in[l] & 15u)) & 15u) / size;
  c.body = lead + k * a.chunk;
  c.hi = c.body + a.chunk;
  if (c.body > n) c.body = n;
  c.lo = k ? c.body : 0;
  if (c.hi > n) c.hi = n;
  return c;
}

__device__ __forceinline__ void vector_of(const uint4& v, float (&f)[8], float) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
template <typename T>
__device__ __forceinline__ void vector_of(const uint4& v, float (&f)[8], T) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = to_f32(e[j]);
}

// Sum of squares of the vectors that a thread holds.
template <typename T>
__device__ __forceinline__ double batch_squares(const uint4 (&v)[kBatch]) {
  constexpr int E = 16 / sizeof(T);
  float s[2] = {0.f, 0.f};
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    float f[8];
    vector_of(v[i], f, T());
#pragma unroll
    for (int j = 0; j < E; ++j) s[j & 1] = fmaf(f[j], f[j], s[j & 1]);
    any |= v[i].x | v[i].y | v[i].z | v[i].w;
  }
  const float sum = s[0] + s[1];
  if (sum >= 1e-30f && sum < 1e30f) return sum;
  if (!(any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu))) return 0.;
  double d = 0.;
#pragma unroll 1
  for (int i = 0; i < kBatch; ++i) {
    float f[8];
    uint4 x = v[0];
#pragma unroll
    for (int k = 1; k < kBatch; ++k)
      if (i == k) x = v[k];
    vector_of(x, f, T());
#pragma unroll
    for (int j = 0; j < E; ++j) d += (double)f[j] * f[j];
  }
  return d;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, const Chunk& c) {
  constexpr int E = 16 / sizeof(T);
  double sum = 0.;
  const long long vectors = (c.hi - c.body) / E, rest = c.body + vectors * E;
  const uint4* q = reinterpret_cast<const uint4*>(p + c.body);
  for (long long i = threadIdx.x; i < vectors; i += kThreads * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      v[k] = i + k * kThreads < vectors ? q[i + k * kThreads] : make_uint4(0u, 0u, 0u, 0u);
    sum += batch_squares<T>(v);
  }
  // fewer elements than a vector before and behind
  const int head = (int)(c.body - c.lo), tail = (int)(c.hi - rest);
  if ((int)threadIdx.x < head + tail) {
    const long long i = (int)threadIdx.x < head ? c.lo + threadIdx.x : rest + ((int)threadIdx.x - head);
    const double x = to_f32(p[i]);
    sum += x * x;
  }
  return sum;
}

// Sum over the block's threads, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ GradList<MAX> a, double* parts) {
  pdl_trigger();
  pdl_wait();
  double sum = 0.;
  for (int chunk = blockIdx.x; chunk < a.first[a.count]; chunk += gridDim.x) {
    const Chunk c = find_chunk(a, chunk);
    const int t = a.types[c.tensor] & 15;
    const void* p = a.in[c.tensor];
    sum += t == RA_F32    ? chunk_squares(static_cast<const float*>(p), c)
           : t == RA_BF16 ? chunk_squares(static_cast<const __nv_bfloat16*>(p), c)
                          : chunk_squares(static_cast<const __half*>(p), c);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The norm from the blocks' sums, in every thread.
__device__ __forceinline__ double norm_of(const double* parts, int count) {
  __shared__ double all;
  double v = 0.;
  for (int i = threadIdx.x; i < count; i += kThreads) v += parts[i];
  v = block_sum(v);
  if (threadIdx.x == 0) all = sqrt(v);
  __syncthreads();
  return all;
}

template <typename TO>
__device__ __forceinline__ void store_vector(TO* out, const float (&f)[8], int E) {
  if constexpr (sizeof(TO) == 4) {
    __stcs(reinterpret_cast<float4*>(out), make_float4(f[0], f[1], f[2], f[3]));
    if (E == 8) __stcs(reinterpret_cast<float4*>(out) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __align__(16) TO e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = from_f32<TO>(f[j]);
    if (E == 8) __stcs(reinterpret_cast<uint4*>(out), *reinterpret_cast<const uint4*>(e));
    else __stcs(reinterpret_cast<uint2*>(out), *reinterpret_cast<const uint2*>(e));
  }
}

// factor(): the factor, asked for once a first batch is on its way.
template <typename T, typename TO, typename F>
__device__ __forceinline__ void scale_chunk(const T* p, TO* out, const Chunk& c, F factor) {
  constexpr int E = 16 / sizeof(T);
  constexpr unsigned kAlign = E * sizeof(TO) < 16 ? E * sizeof(TO) : 16;
  if (reinterpret_cast<uintptr_t>(out + c.body) & (kAlign - 1)) {  // the outputs do not lie as the inputs do
    const float2 mul = factor();
    for (long long i = c.lo + threadIdx.x; i < c.hi; i += kThreads) out[i] = from_f32<TO>(to_f32(p[i]) * mul.x * mul.y);
    return;
  }
  const int vectors = (int)((c.hi - c.body) / E);
  const uint4* q = reinterpret_cast<const uint4*>(p + c.body) + threadIdx.x;
  TO* o = out + c.body + (int)threadIdx.x * E;
  float2 mul = make_float2(0.f, 0.f);
  for (int i = 0; i == 0 || i < vectors; i += kThreads * kScaleBatch) {
    uint4 v[kScaleBatch];
#pragma unroll
    for (int k = 0; k < kScaleBatch; ++k)
      if (i + k * kThreads + (int)threadIdx.x < vectors) v[k] = q[i + k * kThreads];
    if (i == 0) mul = factor();
#pragma unroll
    for (int k = 0; k < kScaleBatch; ++k) {
      if (i + k * kThreads + (int)threadIdx.x >= vectors) break;
      float f[8];
      vector_of(v[k], f, T());
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] = f[j] * mul.x * mul.y;
      store_vector(o + (i + k * kThreads) * E, f, E);
    }
  }
  const long long rest = c.body + (long long)vectors * E;
  const int head = (int)(c.body - c.lo), tail = (int)(c.hi - rest);
  if ((int)threadIdx.x < head + tail) {
    const long long i = (int)threadIdx.x < head ? c.lo + threadIdx.x : rest + ((int)threadIdx.x - head);
    out[i] = from_f32<TO>(to_f32(p[i]) * mul.x * mul.y);
  }
}

template <typename T, typename F>
__device__ __forceinline__ void scale_to(const T* p, void* out, int type, const Chunk& c, F factor) {
  if (type == RA_F32) scale_chunk(p, static_cast<float*>(out), c, factor);
  else if (type == RA_BF16) scale_chunk(p, static_cast<__nv_bfloat16*>(out), c, factor);
  else scale_chunk(p, static_cast<__half*>(out), c, factor);
}

// The factor, in two steps: one below fp32's smallest normal number would lose its digits.
// A norm that is infinite gives 0 and one that is NaN gives NaN.
__device__ __forceinline__ float2 factor_of(double norm, float max_norm, float eps) {
  const double factor = (double)max_norm / (norm + (double)eps);
  return factor >= 1.     ? make_float2(1.f, 1.f)
         : factor < 1e-30 ? make_float2(9.094947017729282e-13f, (float)(factor * 1099511627776.))
                          : make_float2((float)factor, 1.f);
}

// factor NULL: from the parts; else what grad_norm_kernel left there.  T, TO: the types of
// all tensors and their outputs, void: each has its own (nine cases in one kernel, which takes
// a third more time).
template <int MAX, typename T, typename TO>
__global__ void __launch_bounds__(kThreads, std::is_void<T>::value ? 4 : 6) grad_scale_kernel(const __grid_constant__ GradList<MAX> a, const double* parts,
                                                              int count, float max_norm, float eps, float* norm,
                                                              const float2* factor) {
  pdl_trigger();
  pdl_wait();
  float2 mul = make_float2(0.f, 0.f);
  if (!factor) {
    const double n = norm_of(parts, count);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    mul = factor_of(n, max_norm, eps);
  }
  for (int k = blockIdx.x; k < a.first[a.count]; k += gridDim.x) {
    const Chunk c = find_chunk(a, a.first[a.count] - 1 - k);
    const void* p = a.in[c.tensor];
    void* out = a.out[c.tensor];
    // gradients that are clipped in place and need not be are not touched
    if (out == p && (factor ? *factor : mul).x == 1.f) continue;
    auto get = [&] { return factor ? *factor : mul; };
    if constexpr (std::is_void<T>::value) {
      const int t = a.types[c.tensor] & 15, to = a.types[c.tensor] >> 4;
      if (t == RA_F32) scale_to(static_cast<const float*>(p), out, to, c, get);
      else if (t == RA_BF16) scale_to(static_cast<const __nv_bfloat16*>(p), out, to, c, get);
      else scale_to(static_cast<const __half*>(p), out, to, c, get);
    } else {
      scale_chunk(static_cast<const T*>(p), static_cast<TO*>(out), c, get);
    }
  }
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* parts, int count, float max_norm, float eps,
                                                             float* norm, float2* factor) {
  pdl_trigger();
  pdl_wait();
  const double n = norm_of(parts, count);
  if (threadIdx.x) return;
  *norm = (float)n;
  if (factor) *factor = factor_of(n, max_norm, eps);
}

template <int MAX>
int grid_of(const GradList<MAX>& a, int sms) {
  const int chunks = a.first[a.count];
  const int most = sms * 4 < kClipParts ? sms * 4 : kClipParts;
  return chunks < most ? chunks : most;
}

}  // namespace

template <int MAX>
cudaError_t launch_grad_squares(const GradList<MAX>& a, double* parts, int* used, int sms, cudaStream_t st) {
  *used = grid_of(a, sms);
  const cudaError_t e = launch_pdl(grad_squares_kernel<MAX>, *used, kThreads, 0, st, a, parts);
  if (e == cudaSuccess) count_launch();
  return e;
}
template <int MAX>
cudaError_t launch_grad_scale(const GradList<MAX>& a, const double* parts, int count, float max_norm, float eps,
                              float* norm, const float2* factor, int sms, cudaStream_t st) {
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, factor ? a.first[a.count] : grid_of(a, sms), kThreads, 0, st, a, parts, count, max_norm, eps,
                      norm, factor);
  };
  int kind = a.types[0];
  for (int i = 1; i < a.count; ++i)
    if (a.types[i] != kind) kind = -1;
  cudaError_t e;
  switch (kind) {
    case RA_F32 * 17: e = run(grad_scale_kernel<MAX, float, float>); break;
    case RA_BF16 * 17: e = run(grad_scale_kernel<MAX, __nv_bfloat16, __nv_bfloat16>); break;
    case RA_F16 * 17: e = run(grad_scale_kernel<MAX, __half, __half>); break;
    case RA_F32 + 16 * RA_BF16: e = run(grad_scale_kernel<MAX, float, __nv_bfloat16>); break;
    case RA_F32 + 16 * RA_F16: e = run(grad_scale_kernel<MAX, float, __half>); break;
    default: e = run(grad_scale_kernel<MAX, void, void>);
  }
  if (e == cudaSuccess) count_launch();
  return e;
}
cudaError_t launch_grad_norm(const double* parts, int count, float max_norm, float eps, float* norm, float2* factor,
                             cudaStream_t st) {
  const cudaError_t e = launch_pdl(grad_norm_kernel, 1, kThreads, 0, st, parts, count, max_norm, eps, norm, factor);
  if (e == cudaSuccess) count_launch();
  return e;
}

template cudaError_t launch_grad_squares(const GradList<kClipFew>&, double*, int*, int, cudaStream_t);
template cudaError_t launch_grad_squares(const GradList<kClipSome>&, double*, int*, int, cudaStream_t);
template cudaError_t launch_grad_squares(const GradList<kClipMany>&, double*, int*, int, cudaStream_t);
template cudaError_t launch_grad_scale(const GradList<kClipFew>&, const double*, int, float, float, float*, const float2*, int, cudaStream_t);
template cudaError_t launch_grad_scale(const GradList<kClipSome>&, const double*, int, float, float, float*, const float2*, int, cudaStream_t);
template cudaError_t launch_grad_scale(const GradList<kClipMany>&, const double*, int, float, float, float*, const float2*, int, cudaStream_t);

}  // namespace ra
