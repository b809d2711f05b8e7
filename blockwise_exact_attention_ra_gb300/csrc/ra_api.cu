// C-ABI front end of libra: argument validation, workspace layout, tensor
// map encoding and kernel dispatch.  Every entry point only enqueues work on
// the caller's stream; nothing here allocates device memory.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "ra_internal.h"

// One status word per device (module-global storage, not an allocation).
__device__ int g_ra_status_word;

namespace ra {

static std::atomic<unsigned long long> g_launches{0};
void count_launch(unsigned n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

namespace {

thread_local std::string t_err;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_err = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;

struct DeviceCache {
  std::mutex mu;
  int* status[kMaxDevices] = {};
  int sms[kMaxDevices] = {};
  int cc_major[kMaxDevices] = {};
  int cc_minor[kMaxDevices] = {};
};
DeviceCache& cache() {
  static DeviceCache c;
  return c;
}

int current_device(int* dev) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (*dev < 0 || *dev >= kMaxDevices) return fail(RA_ERR_UNSUPPORTED, "device ordinal %d", *dev);
  return RA_OK;
}

// Address of this device's status word, looked up once per device.
int status_ptr(int** out) {
  int dev;
  int rc = current_device(&dev);
  if (rc) return rc;
  DeviceCache& c = cache();
  std::lock_guard<std::mutex> lk(c.mu);
  if (!c.status[dev]) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_ra_status_word);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status word)");
    c.status[dev] = static_cast<int*>(p);
    cudaDeviceGetAttribute(&c.sms[dev], cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&c.cc_major[dev], cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&c.cc_minor[dev], cudaDevAttrComputeCapabilityMinor, dev);
  }
  *out = c.status[dev];
  return RA_OK;
}

int device_sms() {
  int dev = 0;
  cudaGetDevice(&dev);
  return cache().sms[dev] > 0 ? cache().sms[dev] : 1;
}

bool device_is_sm103() {
  int dev = 0;
  cudaGetDevice(&dev);
  return cache().cc_major[dev] == 10 && cache().cc_minor[dev] == 3;
}

unsigned long long wait_limit_ns() {
  static unsigned long long v = [] {
    const char* s = getenv("RA_WAIT_TIMEOUT_MS");
    unsigned long long ms = s ? strtoull(s, nullptr, 10) : 10000ull;
    if (ms == 0) ms = 10000ull;
    return ms * 1000000ull;
  }();
  return v;
}

// -------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

int encoder(EncodeTiledFn* fn) {
  static EncodeTiledFn f = nullptr;
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                           &q);
    if (err == cudaSuccess && q == cudaDriverEntryPointSuccess) f = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (!f) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(err));
  *fn = f;
  return RA_OK;
}

// [B, N, H, d] 16-bit tensor with layout L (elements): dims (d, H, N, B),
// box (64, 1, 128, 1), 128-byte swizzle; rows past N read as zeros.
int make_map(CUtensorMap* m, const void* base, int is_bf16, int B, int N, int H, int d,
             const Lay& L) {
  EncodeTiledFn fn;
  int rc = encoder(&fn);
  if (rc) return rc;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)N, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)L.hs * 2, (cuuint64_t)L.rs * 2, (cuuint64_t)L.bs * 2};
  cuuint32_t box[4] = {64, 1, 128, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return RA_OK;
}

// Packed fp32 [B, N, H, d] tensor: box (32, 1, 32, 1), 128-byte swizzle (one
// warp's 32 rows of a 32-column slab).
int make_map_f32(CUtensorMap* m, void* base, int B, int N, int H, int d) {
  EncodeTiledFn fn;
  int rc = encoder(&fn);
  if (rc) return rc;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)N, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)d * 4, (cuuint64_t)H * d * 4, (cuuint64_t)N * H * d * 4};
  cuuint32_t box[4] = {32, 1, 32, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled (fp32) failed (%d)", (int)r);
  return RA_OK;
}

}  // namespace

// Row-major 16-bit matrix [rows, cols] with leading dimension ld (elements):
// dims (cols, rows), box (64, box_rows), 128-byte swizzle.
int make_map_2d(CUtensorMap* m, const void* base, int is_bf16, long long rows, long long cols,
                long long ld, int box_rows) {
  EncodeTiledFn fn;
  int rc = encoder(&fn);
  if (rc) return rc;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled (2-D) failed (%d)", (int)r);
  return RA_OK;
}

namespace {

// Batch of row-major matrices [batch, rows, cols]: dims (cols, rows, batch), boxes of
// 128-byte rows with the 128-byte swizzle; cols and rows may be of any size, ld and
// bstride (elements) are multiples of 16 bytes.
int make_map_3d(CUtensorMap* m, const void* base, int dtype, long long cols, long long rows, long long batch,
                long long ld, long long bstride, int box_cols, int box_rows) {
  EncodeTiledFn fn;
  int rc = encoder(&fn);
  if (rc) return rc;
  const cuuint64_t es = dtype == RA_F32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  cuuint64_t strides[2] = {(cuuint64_t)ld * es, (cuuint64_t)(batch > 1 ? bstride : ld) * es};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, dtype == RA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                     : dtype == RA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled (3-D) failed (%d)", (int)r);
  return RA_OK;
}

// -------------------------------------------------------------- validation
size_t dtype_size(int dt) { return dt == RA_F32 ? 4 : 2; }
bool valid_dtype(int dt) { return dt == RA_F32 || dt == RA_BF16 || dt == RA_F16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Shape {
  int B, Nq, Nkv, Hq, Hkv, d;
  Lay ql, kvl;  // q, o, dO, dq; k, v, dk, dv
};

// The layout of one group: zero strides take their packed defaults; rows of
// d elements at n * rs + h * hs must not overlap (the smaller of the two
// strides steps past a row, the larger past the whole inner axis), nor may
// one batch overlap the next.
int group_layout(const char* name, int N, int H, int d, long long bs, long long rs, long long hs, Lay* out) {
  if (bs < 0 || rs < 0 || hs < 0) return fail(RA_ERR_INVALID_ARG, "%s strides must be >= 0", name);
  if (rs == 0) rs = (long long)H * d;
  if (hs == 0) hs = d;
  long long s1 = rs, n1 = N, s2 = hs, n2 = H;
  if (s1 > s2) {
    long long t = s1; s1 = s2; s2 = t;
    t = n1; n1 = n2; n2 = t;
  }
  const long long inner = (n1 - 1) * s1 + d;
  if ((n1 > 1 && s1 < d) || (n2 > 1 && s2 < inner))
    return fail(RA_ERR_INVALID_ARG, "%s row and head strides (%lld, %lld) make rows of %d elements overlap", name,
                rs, hs, d);
  const long long extent = (long long)(N - 1) * rs + (long long)(H - 1) * hs + d;
  if (bs == 0) bs = extent;
  if (bs < extent)
    return fail(RA_ERR_INVALID_ARG, "%s batch stride %lld is smaller than one batch (%lld elements)", name, bs,
                extent);
  *out = Lay{bs, rs, hs};
  return RA_OK;
}

int check_shape(const ra_shape& s, Shape* out) {
  if (s.B < 1 || s.N_q < 1 || s.N_kv < 1 || s.Hq < 1 || s.Hkv < 1 || s.d < 1)
    return fail(RA_ERR_INVALID_ARG, "shape has a non-positive extent (B=%d N_q=%d N_kv=%d Hq=%d Hkv=%d d=%d)",
                s.B, s.N_q, s.N_kv, s.Hq, s.Hkv, s.d);
  if (s.Hq % s.Hkv) return fail(RA_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", s.Hq, s.Hkv);
  if (s.N_q >= (1 << 30) || s.N_kv >= (1 << 30) || s.Hq > 4096 || s.d > 4096)
    return fail(RA_ERR_INVALID_ARG, "shape extent too large");
  const long long big = 1ll << 50;  // keeps every offset product far from overflow
  if (s.q_bstride > big || s.kv_bstride > big || s.q_rstride > big || s.q_hstride > big || s.kv_rstride > big ||
      s.kv_hstride > big)
    return fail(RA_ERR_INVALID_ARG, "stride too large");
  Shape r{s.B, s.N_q, s.N_kv, s.Hq, s.Hkv, s.d, {}, {}};
  int rc;
  if ((rc = group_layout("q", s.N_q, s.Hq, s.d, s.q_bstride, s.q_rstride, s.q_hstride, &r.ql)) ||
      (rc = group_layout("kv", s.N_kv, s.Hkv, s.d, s.kv_bstride, s.kv_rstride, s.kv_hstride, &r.kvl)))
    return rc;
  *out = r;
  return RA_OK;
}

bool is_packed(const Lay& L, long long N, long long H, long long d) {
  return L.rs == H * d && L.hs == d;
}

int check_ptr(const void* p, const char* name) {
  if (!p) return fail(RA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(RA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return RA_OK;
}

int check_scale(float scale) {
  if (!(scale > 0.f) || !isfinite(scale))
    return fail(RA_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", (double)scale);
  return RA_OK;
}

// Tensor-core path prerequisites (d, strides, device).
int check_tc(const Shape& s, int dtype) {
  if (s.d != 64 && s.d != 128)
    return fail(RA_ERR_UNSUPPORTED, "tensor-core path supports d in {64, 128} (got %d)", s.d);
  for (const Lay* L : {&s.ql, &s.kvl})
    if ((L->bs % 8) || (L->rs % 8) || (L->hs % 8))
      return fail(RA_ERR_INVALID_ARG, "16-bit tensor-core inputs need strides that are multiples of 8 elements");
  if (!device_is_sm103())
    return fail(RA_ERR_UNSUPPORTED, "tensor-core kernels are built for sm_103a only");
  (void)dtype;
  return RA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// ------------------------------------------------------------ kernel timing
struct KernelTimer {
  std::mutex mu;
  bool on = false;
  std::vector<std::pair<cudaEvent_t, cudaEvent_t>> ev[RA_KERNEL_COUNT];
};
KernelTimer& ktimer() {
  static KernelTimer t;
  return t;
}
void ktimer_clear(KernelTimer& t) {
  for (auto& v : t.ev) {
    for (auto& p : v) {
      cudaEventDestroy(p.first);
      cudaEventDestroy(p.second);
    }
    v.clear();
  }
}

// Brackets one launch with events when timing is on.
struct TimedLaunch {
  int id;
  cudaStream_t st;
  cudaEvent_t a = nullptr, b = nullptr;
  TimedLaunch(int kid, cudaStream_t s) : id(kid), st(s) {
    KernelTimer& t = ktimer();
    std::lock_guard<std::mutex> lk(t.mu);
    if (!t.on) return;
    if (cudaEventCreate(&a) != cudaSuccess || cudaEventCreate(&b) != cudaSuccess) {
      a = b = nullptr;
      return;
    }
    cudaEventRecord(a, st);
  }
  ~TimedLaunch() {
    if (!a) return;
    cudaEventRecord(b, st);
    KernelTimer& t = ktimer();
    std::lock_guard<std::mutex> lk(t.mu);
    t.ev[id].emplace_back(a, b);
  }
};

}  // namespace

int set_error(int code, const char* msg) {
  t_err = msg;
  return code;
}

namespace {
// The debug visit log set by ra_debug_visit_log (process-wide; off by default).
std::mutex g_log_mu;
VisitLog g_log{nullptr, nullptr, 0};
VisitLog visit_log() {
  std::lock_guard<std::mutex> lk(g_log_mu);
  return g_log;
}
}  // namespace

}  // namespace ra

using namespace ra;

extern "C" {
#pragma GCC visibility push(default)

const char* ra_last_error(void) { return t_err.c_str(); }

unsigned long long ra_launch_count(void) { return g_launches.load(); }

int ra_debug_visit_log(unsigned int* entries, size_t capacity, unsigned int* count) {
  if (entries && (!count || capacity == 0))
    return fail(RA_ERR_INVALID_ARG, "a visit log needs a count word and a capacity > 0");
  if (entries && ((reinterpret_cast<uintptr_t>(entries) & 15u) || (reinterpret_cast<uintptr_t>(count) & 3u)))
    return fail(RA_ERR_INVALID_ARG, "visit log entries must be 16-byte aligned and the count word 4-byte aligned");
  std::lock_guard<std::mutex> lk(g_log_mu);
  if (entries)
    g_log = VisitLog{reinterpret_cast<uint4*>(entries), count, (unsigned long long)capacity};
  else
    g_log = VisitLog{nullptr, nullptr, 0};
  return RA_OK;
}

int ra_kernel_timing(int enable) {
  KernelTimer& t = ktimer();
  std::lock_guard<std::mutex> lk(t.mu);
  ktimer_clear(t);
  t.on = enable != 0;
  return RA_OK;
}

int ra_kernel_timing_read(int kernel, double* total_ms, unsigned long long* launches) {
  if (kernel < 0 || kernel >= RA_KERNEL_COUNT || !total_ms || !launches)
    return fail(RA_ERR_INVALID_ARG, "bad kernel id or NULL output");
  KernelTimer& t = ktimer();
  std::lock_guard<std::mutex> lk(t.mu);
  double sum = 0.0;
  for (auto& p : t.ev[kernel]) {
    cudaError_t e = cudaEventSynchronize(p.second);
    if (e != cudaSuccess) return cuda_fail(e, "cudaEventSynchronize");
    float ms = 0.f;
    e = cudaEventElapsedTime(&ms, p.first, p.second);
    if (e != cudaSuccess) return cuda_fail(e, "cudaEventElapsedTime");
    sum += ms;
  }
  *total_ms = sum;
  *launches = t.ev[kernel].size();
  return RA_OK;
}

int ra_sync_status(void* stream) {
  int* st;
  int rc = status_ptr(&st);
  if (rc) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int v = 0;
  e = cudaMemcpyFromSymbol(&v, g_ra_status_word, sizeof v);
  if (e != cudaSuccess) return cuda_fail(e, "read status word");
  if (v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_ra_status_word, &zero, sizeof zero);
    if (e != cudaSuccess) return cuda_fail(e, "clear status word");
    return fail(v, v == RA_ERR_RANGE ? "an operand exceeded the fp16 range"
                                     : v == RA_ERR_TIMEOUT ? "a bounded wait on the device gave up"
                                     : v == RA_ERR_INVALID_ARG ? "a target lies outside the vocabulary"
                                                           : "device reported status %d",
                v);
  }
  t_err.clear();
  return RA_OK;
}

int ra_selftest_timeout(unsigned int timeout_us, void* stream) {
  int* st;
  int rc = status_ptr(&st);
  if (rc) return rc;
  if (timeout_us == 0 || timeout_us > 10000000u)
    return fail(RA_ERR_INVALID_ARG, "timeout_us must be in (0, 1e7]");
  cudaError_t e = launch_selftest_timeout(timeout_us, st, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "selftest_timeout launch");
}

int ra_acc_init(float* o_acc, float* m_acc, float* l_acc, ra_shape shape, void* stream) {
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if ((rc = check_ptr(o_acc, "o_acc")) || (rc = check_ptr(m_acc, "m_acc")) || (rc = check_ptr(l_acc, "l_acc")))
    return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaError_t e = launch_acc_init(o_acc, m_acc, l_acc, s.B, s.Nq, s.Hq, s.d,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "acc_init launch");
}

int ra_merge(float* o_a, float* m_a, float* l_a, const float* o_b, const float* m_b,
             const float* l_b, ra_shape shape, void* stream) {
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if ((rc = check_ptr(o_a, "o_a")) || (rc = check_ptr(m_a, "m_a")) || (rc = check_ptr(l_a, "l_a")) ||
      (rc = check_ptr(o_b, "o_b")) || (rc = check_ptr(m_b, "m_b")) || (rc = check_ptr(l_b, "l_b")))
    return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaError_t e = launch_merge(o_a, m_a, l_a, o_b, m_b, l_b, s.B, s.Nq, s.Hq, s.d,
                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "merge launch");
}

int ra_finalize(const float* o_acc, const float* m_acc, const float* l_acc, void* o_out,
                ra_dtype o_dtype, float* lse, ra_shape shape, void* stream) {
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if (!valid_dtype(o_dtype)) return fail(RA_ERR_INVALID_ARG, "bad o_dtype %d", (int)o_dtype);
  if ((rc = check_ptr(o_acc, "o_acc")) || (rc = check_ptr(m_acc, "m_acc")) || (rc = check_ptr(l_acc, "l_acc")) ||
      (rc = check_ptr(o_out, "o_out")) || (rc = check_ptr(lse, "lse")))
    return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaError_t e = launch_finalize(o_acc, m_acc, l_acc, o_out, o_dtype, s.ql, lse, s.B, s.Nq,
                                  s.Hq, s.d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "finalize launch");
}

size_t ra_block_fwd_workspace_bytes(ra_dtype dtype, ra_shape shape) {
  if (dtype != RA_BF16 || shape.B < 1 || shape.N_kv < 1 || shape.Hkv < 1 || shape.d < 1) return 0;
  return align256((size_t)shape.B * shape.N_kv * shape.Hkv * shape.d * 2);
}

int ra_block_fwd(const void* q, const void* k_blk, const void* v_blk, ra_dtype dtype,
                 float* o_acc, float* m_acc, float* l_acc, ra_shape shape, long long q_off,
                 long long kv_off, int flags, float scale, void* workspace, size_t ws_bytes,
                 void* stream) {
  const int causal = (flags & RA_CAUSAL) != 0, precise = (flags & RA_PRECISE) != 0;
  if (flags & ~(RA_CAUSAL | RA_PRECISE)) return fail(RA_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if (!valid_dtype(dtype)) return fail(RA_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
  if ((rc = check_scale(scale))) return rc;
  if ((rc = check_ptr(q, "q")) || (rc = check_ptr(k_blk, "k_blk")) || (rc = check_ptr(v_blk, "v_blk")) ||
      (rc = check_ptr(o_acc, "o_acc")) || (rc = check_ptr(m_acc, "m_acc")) || (rc = check_ptr(l_acc, "l_acc")))
    return rc;
  if (q_off < 0 || kv_off < 0) return fail(RA_ERR_INVALID_ARG, "offsets must be >= 0");
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == RA_F32) {
    if (s.d != 32 && s.d != 64 && s.d != 128)
      return fail(RA_ERR_UNSUPPORTED, "fp32 path supports d in {32, 64, 128} (got %d)", s.d);
    SimtFwdArgs a{};
    a.q = static_cast<const float*>(q);
    a.k = static_cast<const float*>(k_blk);
    a.v = static_cast<const float*>(v_blk);
    a.B = s.B; a.Nq = s.Nq; a.Nkv = s.Nkv; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
    a.ql = s.ql; a.kvl = s.kvl;
    a.scale = scale; a.causal = causal; a.q_off = q_off; a.kv_off = kv_off;
    a.P = 0; a.S = 0;
    a.o_acc = o_acc; a.m_acc = m_acc; a.l_acc = l_acc;
    TimedLaunch tl(RA_KERNEL_FWD_F32, cs);
    cudaError_t e = launch_simt_fwd(a, cs);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "fp32 block forward launch");
  }
  if ((rc = check_tc(s, dtype))) return rc;
  const void* v16 = v_blk;
  if (dtype == RA_BF16) {
    const size_t need = ra_block_fwd_workspace_bytes(dtype, shape);
    if (!workspace || ws_bytes < need)
      return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
    if ((rc = check_ptr(workspace, "workspace"))) return rc;
    cudaError_t e = launch_to_f16(v_blk, RA_BF16, s.kvl, workspace, s.B, s.Nkv, s.Hkv, s.d, st, cs);
    if (e != cudaSuccess) return cuda_fail(e, "v -> fp16 launch");
    v16 = workspace;
  }
  TcFwdArgs a;
  memset(&a, 0, sizeof a);
  const int bf = dtype == RA_BF16;
  if ((rc = make_map(&a.tm_q, q, bf, s.B, s.Nq, s.Hq, s.d, s.ql))) return rc;
  if ((rc = make_map(&a.tm_k, k_blk, bf, s.B, s.Nkv, s.Hkv, s.d, s.kvl))) return rc;
  if ((rc = make_map(&a.tm_v, v16, 0, s.B, s.Nkv, s.Hkv, s.d,
                     dtype == RA_BF16 ? packed_lay(s.Nkv, s.Hkv, s.d) : s.kvl)))
    return rc;
  a.qk_bf16 = bf;
  a.B = s.B; a.Nq = s.Nq; a.Nkv = s.Nkv; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal; a.q_off = q_off; a.kv_off = kv_off; a.precise = precise;
  a.ring_P = 0; a.ring_S = 0; a.T_m = 0; a.mode = 1;
  a.o_acc = o_acc; a.m_acc = m_acc; a.l_acc = l_acc;
  a.status = st;
  a.wait_limit_ns = wait_limit_ns();
  a.log = visit_log();
  const int nqt = (s.Nq + 127) / 128;
  a.num_units = s.B * s.Hq * ((nqt + 1) / 2);
  TimedLaunch tl(RA_KERNEL_FWD_TC, cs);
  cudaError_t e = launch_tc_fwd(a, device_sms(), cs);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "tensor-core block forward launch");
}

// Ring forward workspace (16-bit dtypes): unit counter (256 bytes) | fp16
// copy of V [B,N,Hkv,d] (bf16 inputs).
size_t ra_ring_fwd_workspace_bytes(ra_dtype dtype, ra_shape shape, int P) {
  (void)P;
  if ((dtype != RA_BF16 && dtype != RA_F16) || shape.B < 1 || shape.N_kv < 1 || shape.Hkv < 1 || shape.d < 1)
    return 0;
  if (dtype == RA_F16) return 256;
  return 256 + align256((size_t)shape.B * shape.N_kv * shape.Hkv * shape.d * 2);
}

static int check_ring(const Shape& s, int P, int dtype) {
  if (s.Nq != s.Nkv) return fail(RA_ERR_INVALID_ARG, "ring attention needs N_q == N_kv (%d vs %d)", s.Nq, s.Nkv);
  if (P < 1 || s.Nq % P) return fail(RA_ERR_INVALID_ARG, "P=%d must divide N=%d", P, s.Nq);
  if (dtype != RA_F32 && (s.Nq / P) % 128)
    return fail(RA_ERR_UNSUPPORTED, "tensor-core ring needs a host block N/P that is a multiple of 128 (got %d)",
                s.Nq / P);
  return RA_OK;
}

static int ring_fwd_impl(const void* q, const void* k, const void* v, ra_dtype dtype, ra_shape shape,
                         int P, int flags, float scale, void* o, ra_dtype o_dtype, float* lse,
                         void* workspace, size_t ws_bytes, void* stream, const int* host_len) {
  const int causal = (flags & RA_CAUSAL) != 0, precise = (flags & RA_PRECISE) != 0;
  const int striped = causal && (flags & RA_STRIPED) != 0;
  if (flags & ~(RA_CAUSAL | RA_PRECISE | RA_STRIPED))
    return fail(RA_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  if (host_len && striped)
    return fail(RA_ERR_INVALID_ARG, "RA_STRIPED does not combine with per-host lengths");
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if (!valid_dtype(dtype) || !valid_dtype(o_dtype)) return fail(RA_ERR_INVALID_ARG, "bad dtype");
  if ((rc = check_scale(scale))) return rc;
  if ((rc = check_ring(s, P, dtype))) return rc;
  if ((rc = check_ptr(q, "q")) || (rc = check_ptr(k, "k")) || (rc = check_ptr(v, "v")) ||
      (rc = check_ptr(o, "o")) || (rc = check_ptr(lse, "lse")))
    return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == RA_F32) {
    if (s.d != 32 && s.d != 64 && s.d != 128)
      return fail(RA_ERR_UNSUPPORTED, "fp32 path supports d in {32, 64, 128} (got %d)", s.d);
    SimtFwdArgs a{};
    a.q = static_cast<const float*>(q);
    a.k = static_cast<const float*>(k);
    a.v = static_cast<const float*>(v);
    a.B = s.B; a.Nq = s.Nq; a.Nkv = s.Nkv; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
    a.ql = s.ql; a.kvl = s.kvl;
    a.scale = scale; a.causal = causal;
    a.P = P; a.S = s.Nq / P; a.striped = striped; a.host_len = host_len;
    a.o_out = o; a.o_dtype = o_dtype; a.lse = lse;
    TimedLaunch tl(RA_KERNEL_FWD_F32, cs);
    cudaError_t e = launch_simt_fwd(a, cs);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "fp32 ring forward launch");
  }
  if ((rc = check_tc(s, dtype))) return rc;
  const size_t need = ra_ring_fwd_workspace_bytes(dtype, shape, P);
  if (!workspace || ws_bytes < need)
    return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if ((rc = check_ptr(workspace, "workspace"))) return rc;
  unsigned int* sched = static_cast<unsigned int*>(workspace);
  cudaError_t me = cudaMemsetAsync(sched, 0, 256, cs);
  if (me != cudaSuccess) return cuda_fail(me, "zero unit counter");
  const void* v16 = v;
  if (dtype == RA_BF16) {
    void* vcopy = static_cast<char*>(workspace) + 256;
    cudaError_t e = launch_to_f16(v, RA_BF16, s.kvl, vcopy, s.B, s.Nkv, s.Hkv, s.d, st, cs);
    if (e != cudaSuccess) return cuda_fail(e, "v -> fp16 launch");
    v16 = vcopy;
  }
  TcFwdArgs a;
  memset(&a, 0, sizeof a);
  const int bf = dtype == RA_BF16;
  if ((rc = make_map(&a.tm_q, q, bf, s.B, s.Nq, s.Hq, s.d, s.ql))) return rc;
  if ((rc = make_map(&a.tm_k, k, bf, s.B, s.Nkv, s.Hkv, s.d, s.kvl))) return rc;
  if ((rc = make_map(&a.tm_v, v16, 0, s.B, s.Nkv, s.Hkv, s.d,
                     dtype == RA_BF16 ? packed_lay(s.Nkv, s.Hkv, s.d) : s.kvl)))
    return rc;
  a.qk_bf16 = bf;
  a.B = s.B; a.Nq = s.Nq; a.Nkv = s.Nkv; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal;
  a.ring_P = P; a.ring_S = s.Nq / P; a.T_m = div_magic((unsigned)(a.ring_S / 128)); a.mode = 0; a.precise = precise; a.striped = striped;
  a.host_len = host_len;
  if (host_len) {  // padded rows: O = 0, LSE = -inf (the kernel skips them)
    cudaError_t fe = launch_fill_padding(o, o_dtype, s.ql, s.B, s.Nq, s.Hq, s.d, P, host_len, lse, cs);
    if (fe != cudaSuccess) return cuda_fail(fe, "padding fill launch");
  }
  a.o_out = o; a.o_dtype = o_dtype; a.ol = s.ql; a.lse = lse;
  a.status = st;
  a.wait_limit_ns = wait_limit_ns();
  a.log = visit_log();
  const int T = a.ring_S / 128;
  a.num_units = s.B * s.Hq * P * ((T + 1) / 2);
  a.sched = sched;
  TimedLaunch tl(RA_KERNEL_FWD_TC, cs);
  cudaError_t e = launch_tc_fwd(a, device_sms(), cs);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "tensor-core ring forward launch");
}

// Backward workspace: D [B,Hq,N] fp32 | LSE*log2e [B,Hq,N] fp32 |
// dq_acc [B,N,Hq,d] fp32 | unit counter (256 bytes, zeroed with dq_acc) |
// fp16 copies of q, k, v, dO (16-bit dtypes that are not already fp16).
struct BwdWs {
  size_t D, lse2, dq, sched, q16, k16, v16, do16, total;
};
static BwdWs bwd_layout(int dtype, const ra_shape& sh) {
  BwdWs w{};
  const size_t qel = (size_t)sh.B * sh.N_q * sh.Hq * sh.d;
  const size_t kvel = (size_t)sh.B * sh.N_kv * sh.Hkv * sh.d;
  size_t off = 0;
  w.D = off; off += align256((size_t)sh.B * sh.Hq * sh.N_q * 4);
  if (dtype != RA_F32) {
    w.lse2 = off; off += align256((size_t)sh.B * sh.Hq * sh.N_q * 4);
    w.dq = off; off += align256(qel * 4);
    w.sched = off; off += 256;
    if (dtype == RA_BF16) {
      w.q16 = off; off += align256(qel * 2);
      w.k16 = off; off += align256(kvel * 2);
      w.v16 = off; off += align256(kvel * 2);
      w.do16 = off; off += align256(qel * 2);
    }
  }
  w.total = off;
  return w;
}

size_t ra_ring_bwd_workspace_bytes(ra_dtype dtype, ra_dtype grad_dtype, ra_shape shape, int P) {
  (void)grad_dtype;
  (void)P;
  if (shape.B < 1 || shape.N_q < 1 || shape.N_kv < 1 || shape.Hq < 1 || shape.Hkv < 1 || shape.d < 1) return 0;
  return bwd_layout(dtype, shape).total;
}

static int ring_bwd_impl(const void* q, const void* k, const void* v, const void* o, ra_dtype o_dtype,
                         const void* dO, const float* lse, ra_dtype dtype, ra_shape shape, int P,
                         int flags, float scale, void* dq, void* dk, void* dv, ra_dtype grad_dtype,
                         void* workspace, size_t ws_bytes, void* stream, const int* host_len) {
  const int causal = (flags & RA_CAUSAL) != 0, precise = (flags & RA_PRECISE) != 0;
  const int striped = causal && (flags & RA_STRIPED) != 0;
  if (flags & ~(RA_CAUSAL | RA_PRECISE | RA_STRIPED))
    return fail(RA_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  if (host_len && striped)
    return fail(RA_ERR_INVALID_ARG, "RA_STRIPED does not combine with per-host lengths");
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if (!valid_dtype(dtype) || !valid_dtype(o_dtype) || !valid_dtype(grad_dtype))
    return fail(RA_ERR_INVALID_ARG, "bad dtype");
  if ((rc = check_scale(scale))) return rc;
  if ((rc = check_ring(s, P, dtype))) return rc;
  if ((rc = check_ptr(q, "q")) || (rc = check_ptr(k, "k")) || (rc = check_ptr(v, "v")) ||
      (rc = check_ptr(o, "o")) || (rc = check_ptr(dO, "dO")) || (rc = check_ptr(lse, "lse")) ||
      (rc = check_ptr(dq, "dq")) || (rc = check_ptr(dk, "dk")) || (rc = check_ptr(dv, "dv")))
    return rc;
  const BwdWs w = bwd_layout(dtype, shape);
  if (!workspace || ws_bytes < w.total)
    return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", w.total, ws_bytes);
  if ((rc = check_ptr(workspace, "workspace"))) return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float* Dv = reinterpret_cast<float*>(ws + w.D);
  if (dtype == RA_F32) {
    if (s.d != 32 && s.d != 64 && s.d != 128)
      return fail(RA_ERR_UNSUPPORTED, "fp32 path supports d in {32, 64, 128} (got %d)", s.d);
    cudaError_t e = launch_bwd_dot(dO, RA_F32, o, o_dtype, s.ql, Dv, nullptr, nullptr, s.B, s.Nq,
                                   s.Hq, s.d, cs);
    if (e != cudaSuccess) return cuda_fail(e, "bwd D launch");
    SimtBwdArgs a{};
    a.q = static_cast<const float*>(q);
    a.k = static_cast<const float*>(k);
    a.v = static_cast<const float*>(v);
    a.dO = static_cast<const float*>(dO);
    a.lse = lse;
    a.Dvec = Dv;
    a.B = s.B; a.N = s.Nq; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
    a.ql = s.ql; a.kvl = s.kvl;
    a.scale = scale; a.causal = causal;
    a.P = P; a.S = s.Nq / P; a.striped = striped; a.host_len = host_len;
    a.dq = dq; a.dk = dk; a.dv = dv; a.grad_dtype = grad_dtype;
    {
      TimedLaunch tl(RA_KERNEL_BWD_F32, cs);
      e = launch_simt_bwd(a, cs);
    }
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "fp32 ring backward launch");
  }
  if ((rc = check_tc(s, dtype))) return rc;
  float* lse2 = reinterpret_cast<float*>(ws + w.lse2);
  cudaError_t e = launch_bwd_dot(dO, dtype, o, o_dtype, s.ql, Dv, lse, lse2, s.B, s.Nq, s.Hq,
                                 s.d, cs);
  if (e != cudaSuccess) return cuda_fail(e, "bwd D launch");
  const void *q16 = q, *k16 = k, *v16 = v, *do16 = dO;
  Lay q16_l = s.ql, kv16_l = s.kvl;
  if (dtype == RA_BF16) {
    q16 = ws + w.q16; k16 = ws + w.k16; v16 = ws + w.v16; do16 = ws + w.do16;
    q16_l = packed_lay(s.Nq, s.Hq, s.d);
    kv16_l = packed_lay(s.Nkv, s.Hkv, s.d);
    if ((e = launch_to_f16(q, RA_BF16, s.ql, ws + w.q16, s.B, s.Nq, s.Hq, s.d, st, cs)) != cudaSuccess ||
        (e = launch_to_f16(k, RA_BF16, s.kvl, ws + w.k16, s.B, s.Nkv, s.Hkv, s.d, st, cs)) != cudaSuccess ||
        (e = launch_to_f16(v, RA_BF16, s.kvl, ws + w.v16, s.B, s.Nkv, s.Hkv, s.d, st, cs)) != cudaSuccess ||
        (e = launch_to_f16(dO, RA_BF16, s.ql, ws + w.do16, s.B, s.Nq, s.Hq, s.d, st, cs)) != cudaSuccess)
      return cuda_fail(e, "fp16 operand copy launch");
  }
  float* dq_acc = reinterpret_cast<float*>(ws + w.dq);
  e = cudaMemsetAsync(dq_acc, 0, w.sched + 256 - w.dq, cs);  // and the unit counter
  if (e != cudaSuccess) return cuda_fail(e, "zero dq accumulator");
  TcBwdArgs a;
  memset(&a, 0, sizeof a);
  if ((rc = make_map(&a.tm_q, q16, 0, s.B, s.Nq, s.Hq, s.d, q16_l)) ||
      (rc = make_map(&a.tm_do, do16, 0, s.B, s.Nq, s.Hq, s.d, q16_l)) ||
      (rc = make_map(&a.tm_k, k16, 0, s.B, s.Nkv, s.Hkv, s.d, kv16_l)) ||
      (rc = make_map(&a.tm_v, v16, 0, s.B, s.Nkv, s.Hkv, s.d, kv16_l)) ||
      (rc = make_map_f32(&a.tm_dq, dq_acc, s.B, s.Nq, s.Hq, s.d)))
    return rc;
  a.B = s.B; a.N = s.Nq; a.Hq = s.Hq; a.Hkv = s.Hkv; a.d = s.d;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal;
  a.ring_P = P; a.ring_S = s.Nq / P; a.T_m = div_magic((unsigned)(a.ring_S / 128)); a.P_m = div_magic((unsigned)P);
  a.precise = precise; a.striped = striped;
  a.host_len = host_len;
  if (host_len) {  // padded key rows: dK = dV = 0 (the kernel skips wholly padded key tiles)
    cudaError_t fe = launch_fill_padding(dk, grad_dtype, s.kvl, s.B, s.Nkv, s.Hkv, s.d, P, host_len, nullptr, cs);
    if (fe == cudaSuccess)
      fe = launch_fill_padding(dv, grad_dtype, s.kvl, s.B, s.Nkv, s.Hkv, s.d, P, host_len, nullptr, cs);
    if (fe != cudaSuccess) return cuda_fail(fe, "padding fill launch");
  }
  a.lse = lse2; a.Dvec = Dv; a.dq_acc = dq_acc;
  a.dk = dk; a.dv = dv; a.grad_dtype = grad_dtype; a.kvl = s.kvl;
  a.status = st;
  a.wait_limit_ns = wait_limit_ns();
  a.log = visit_log();
  a.num_units = s.B * s.Hkv * (s.Nkv / 128);
  a.sched = reinterpret_cast<unsigned int*>(ws + w.sched);
  {
    TimedLaunch tl(RA_KERNEL_BWD_TC, cs);
    e = launch_tc_bwd(a, device_sms(), cs);
  }
  if (e != cudaSuccess) return cuda_fail(e, "tensor-core ring backward launch");
  e = launch_f32_to(dq_acc, dq, grad_dtype, s.ql, s.B, s.Nq, s.Hq, s.d, scale, cs);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "dq conversion launch");
}

int ra_ring_fwd(const void* q, const void* k, const void* v, ra_dtype dtype, ra_shape shape,
                int P, int flags, float scale, void* o, ra_dtype o_dtype, float* lse,
                void* workspace, size_t ws_bytes, void* stream) {
  return ring_fwd_impl(q, k, v, dtype, shape, P, flags, scale, o, o_dtype, lse, workspace, ws_bytes,
                       stream, nullptr);
}

int ra_ring_bwd(const void* q, const void* k, const void* v, const void* o, ra_dtype o_dtype,
                const void* dO, const float* lse, ra_dtype dtype, ra_shape shape, int P,
                int flags, float scale, void* dq, void* dk, void* dv, ra_dtype grad_dtype,
                void* workspace, size_t ws_bytes, void* stream) {
  return ring_bwd_impl(q, k, v, o, o_dtype, dO, lse, dtype, shape, P, flags, scale, dq, dk, dv,
                       grad_dtype, workspace, ws_bytes, stream, nullptr);
}

int ra_ring_fwd_varlen(const void* q, const void* k, const void* v, ra_dtype dtype, ra_shape shape,
                       int P, const int* host_len, int flags, float scale, void* o, ra_dtype o_dtype,
                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if (!host_len || (reinterpret_cast<uintptr_t>(host_len) & 3u))
    return fail(RA_ERR_INVALID_ARG, "host_len must be a non-NULL, 4-byte aligned device array");
  return ring_fwd_impl(q, k, v, dtype, shape, P, flags, scale, o, o_dtype, lse, workspace, ws_bytes,
                       stream, host_len);
}

int ra_ring_bwd_varlen(const void* q, const void* k, const void* v, const void* o, ra_dtype o_dtype,
                       const void* dO, const float* lse, ra_dtype dtype, ra_shape shape, int P,
                       const int* host_len, int flags, float scale, void* dq, void* dk, void* dv,
                       ra_dtype grad_dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!host_len || (reinterpret_cast<uintptr_t>(host_len) & 3u))
    return fail(RA_ERR_INVALID_ARG, "host_len must be a non-NULL, 4-byte aligned device array");
  return ring_bwd_impl(q, k, v, o, o_dtype, dO, lse, dtype, shape, P, flags, scale, dq, dk, dv,
                       grad_dtype, workspace, ws_bytes, stream, host_len);
}

#pragma GCC visibility pop
}  // extern "C"

// ------------------------------------------------ blockwise feed-forward layer
namespace ra {
namespace {

struct FfnShape {
  long long T;
  int dm, dh, block;
};

int check_ffn(ra_dtype dtype, long long T, int d_model, int d_hidden, int block, FfnShape* out) {
  if (dtype != RA_BF16 && dtype != RA_F16)
    return fail(RA_ERR_UNSUPPORTED, "the feed-forward path takes bf16 or fp16 operands");
  if (T < 1 || d_model < 1 || d_hidden < 1 || block < 1)
    return fail(RA_ERR_INVALID_ARG, "non-positive feed-forward size (T=%lld d_model=%d d_hidden=%d block=%d)", T,
                d_model, d_hidden, block);
  if (d_model % 256 || d_hidden % 256)
    return fail(RA_ERR_UNSUPPORTED, "d_model and d_hidden must be multiples of 256 (got %d, %d)", d_model, d_hidden);
  if (T % 128 || block % 128)
    return fail(RA_ERR_UNSUPPORTED, "T and block must be multiples of 128 (got %lld, %d)", T, block);
  if (T >= (1ll << 31) || d_model > 65536 || d_hidden > 262144)
    return fail(RA_ERR_INVALID_ARG, "feed-forward size too large");
  *out = FfnShape{T, d_model, d_hidden, (int)(block < T ? block : T)};
  return RA_OK;
}

// per-block 16-bit scratch: hidden activations a, GELU'(h), dH
struct FfnWs {
  size_t a, g, dh, total;
};
FfnWs ffn_layout(const FfnShape& s, bool bwd) {
  FfnWs w{};
  const size_t blk = align256((size_t)s.block * s.dh * 2);
  w.a = 0;
  w.g = blk;
  w.dh = 2 * blk;
  w.total = bwd ? 3 * blk : blk;
  return w;
}

struct GemmPlan {
  int rc = RA_OK;
  cudaStream_t st;
  int bf16;
  int* status;
  int sms;
  // a second problem run in the same launch (same K, majorness and epilogue)
  struct Second {
    const void* A;
    long long a_rows, a_cols;
    const void* B;
    long long b_rows, b_cols;
    int M, N;
    void* c;
    long long ldc;
  };
  // C[M, N] = epi(A B^T); a_rows/b_rows are the row counts of the stored matrices
  int run(const void* A, long long a_rows, long long a_cols, int a_mn, const void* B, long long b_rows,
          long long b_cols, int b_mn, int M, int N, int K, int epi, void* c, long long ldc, int c_dtype,
          void* c2 = nullptr, const void* aux = nullptr, const Second* second = nullptr) {
    if (rc) return rc;
    GemmArgs g;
    memset(&g, 0, sizeof g);
    if ((rc = make_map_2d(&g.tm_a, A, bf16, a_rows, a_cols, a_cols, a_mn ? 64 : 128)) ||
        (rc = make_map_2d(&g.tm_b, B, bf16, b_rows, b_cols, b_cols, b_mn ? 64 : 256)))
      return rc;
    g.M = M; g.N = N; g.K = K;
    g.a_mn = a_mn; g.b_mn = b_mn; g.ab_bf16 = bf16;
    g.epi = epi; g.c = c; g.ldc = ldc; g.c_dtype = c_dtype; g.c2 = c2; g.aux = aux;
    g.groups = 1;
    if (second) {
      g.groups = 2;
      if ((rc = make_map_2d(&g.tm_a2, second->A, bf16, second->a_rows, second->a_cols, second->a_cols,
                            a_mn ? 64 : 128)) ||
          (rc = make_map_2d(&g.tm_b2, second->B, bf16, second->b_rows, second->b_cols, second->b_cols,
                            b_mn ? 64 : 256)))
        return rc;
      g.M2 = second->M; g.N2 = second->N; g.c_g2 = second->c; g.ldc_g2 = second->ldc;
    }
    g.status = status;
    g.wait_limit_ns = wait_limit_ns();
    cudaError_t e;
    {
      TimedLaunch tl(RA_KERNEL_GEMM_TC, st);
      e = launch_tc_gemm(g, sms, st);
    }
    if (e != cudaSuccess) rc = cuda_fail(e, "tensor-core GEMM launch");
    return rc;
  }
};

int ffn_common(const void* x, const void* w1, const void* w2, ra_dtype dtype, long long T, int d_model,
               int d_hidden, int block, void* workspace, size_t ws_bytes, bool bwd, FfnShape* s, FfnWs* w,
               int** st) {
  int rc;
  if ((rc = check_ffn(dtype, T, d_model, d_hidden, block, s))) return rc;
  if ((rc = check_ptr(x, "x")) || (rc = check_ptr(w1, "w1")) || (rc = check_ptr(w2, "w2"))) return rc;
  *w = ffn_layout(*s, bwd);
  if (!workspace || ws_bytes < w->total)
    return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", w->total, ws_bytes);
  if ((rc = check_ptr(workspace, "workspace"))) return rc;
  if ((rc = status_ptr(st))) return rc;
  if (!device_is_sm103()) return fail(RA_ERR_UNSUPPORTED, "tensor-core kernels are built for sm_103a only");
  return RA_OK;
}

}  // namespace
}  // namespace ra

extern "C" {
#pragma GCC visibility push(default)

size_t ra_ffn_workspace_bytes(ra_dtype dtype, long long T, int d_model, int d_hidden, int block, int backward) {
  FfnShape s;
  if (check_ffn(dtype, T, d_model, d_hidden, block, &s)) return 0;
  return ffn_layout(s, backward != 0).total;
}

int ra_ffn_fwd(const void* x, const void* w1, const void* w2, ra_dtype dtype, long long T, int d_model,
               int d_hidden, int block, void* y, ra_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream) {
  FfnShape s;
  FfnWs w;
  int* st;
  int rc = ffn_common(x, w1, w2, dtype, T, d_model, d_hidden, block, workspace, ws_bytes, false, &s, &w, &st);
  if (rc) return rc;
  if (!valid_dtype(y_dtype)) return fail(RA_ERR_INVALID_ARG, "bad y dtype");
  if ((rc = check_ptr(y, "y"))) return rc;
  GemmPlan g;
  g.st = static_cast<cudaStream_t>(stream);
  g.bf16 = dtype == RA_BF16;
  g.status = st;
  g.sms = device_sms();
  char* ws = static_cast<char*>(workspace);
  const size_t es = 2, ys = dtype_size(y_dtype);
  for (long long t0 = 0; t0 < s.T && !g.rc; t0 += s.block) {
    const int Mb = (int)(s.T - t0 < s.block ? s.T - t0 : s.block);
    const char* xb = static_cast<const char*>(x) + (size_t)t0 * s.dm * es;
    // a = GELU(x W1^T) for this block of tokens only
    g.run(xb, Mb, s.dm, 0, w1, s.dh, s.dm, 0, Mb, s.dh, s.dm, GEMM_GELU, ws + w.a, s.dh, dtype);
    // y = a W2^T
    g.run(ws + w.a, Mb, s.dh, 0, w2, s.dm, s.dh, 0, Mb, s.dm, s.dh, GEMM_STORE,
          static_cast<char*>(y) + (size_t)t0 * s.dm * ys, s.dm, y_dtype);
  }
  return g.rc;
}

int ra_ffn_bwd(const void* x, const void* w1, const void* w2, const void* dy, ra_dtype dtype, long long T,
               int d_model, int d_hidden, int block, void* dx, ra_dtype dx_dtype, float* dw1, float* dw2,
               void* workspace, size_t ws_bytes, void* stream) {
  FfnShape s;
  FfnWs w;
  int* st;
  int rc = ffn_common(x, w1, w2, dtype, T, d_model, d_hidden, block, workspace, ws_bytes, true, &s, &w, &st);
  if (rc) return rc;
  if (!valid_dtype(dx_dtype)) return fail(RA_ERR_INVALID_ARG, "bad dx dtype");
  if ((rc = check_ptr(dy, "dy")) || (rc = check_ptr(dx, "dx")) || (rc = check_ptr(dw1, "dw1")) ||
      (rc = check_ptr(dw2, "dw2")))
    return rc;
  GemmPlan g;
  g.st = static_cast<cudaStream_t>(stream);
  g.bf16 = dtype == RA_BF16;
  g.status = st;
  g.sms = device_sms();
  char* ws = static_cast<char*>(workspace);
  const size_t es = 2, xs = dtype_size(dx_dtype);
  cudaError_t e = cudaMemsetAsync(dw1, 0, (size_t)s.dh * s.dm * 4, g.st);
  if (e == cudaSuccess) e = cudaMemsetAsync(dw2, 0, (size_t)s.dm * s.dh * 4, g.st);
  if (e != cudaSuccess) return cuda_fail(e, "zero weight gradients");
  for (long long t0 = 0; t0 < s.T && !g.rc; t0 += s.block) {
    const int Mb = (int)(s.T - t0 < s.block ? s.T - t0 : s.block);
    const char* xb = static_cast<const char*>(x) + (size_t)t0 * s.dm * es;
    const char* dyb = static_cast<const char*>(dy) + (size_t)t0 * s.dm * es;
    // recompute the block's hidden activations: a = GELU(h), g = GELU'(h), h = x W1^T
    g.run(xb, Mb, s.dm, 0, w1, s.dh, s.dm, 0, Mb, s.dh, s.dm, GEMM_GELU2, ws + w.a, s.dh, dtype, ws + w.g);
    // dH = (dy W2) * GELU'(h)   (W2 [dm, dh] read as a [K, N] matrix: MN-major)
    g.run(dyb, Mb, s.dm, 0, w2, s.dm, s.dh, 1, Mb, s.dh, s.dm, GEMM_MUL, ws + w.dh, s.dh, dtype, nullptr,
          ws + w.g);
    // dx = dH W1   (W1 [dh, dm] as [K, N]: MN-major)
    g.run(ws + w.dh, Mb, s.dh, 0, w1, s.dh, s.dm, 1, Mb, s.dm, s.dh, GEMM_STORE,
          static_cast<char*>(dx) + (size_t)t0 * s.dm * xs, s.dm, dx_dtype);
    // dW2 += dy^T a   (M = d_model, N = d_hidden, K = the block's tokens; both operands MN-major)
    // and, in the same launch, dW1 += dH^T x   (M = d_hidden, N = d_model): each alone has
    // too few 128 x 256 tiles to keep the last wave of SMs busy
    const GemmPlan::Second dw1_prob{ws + w.dh, Mb, s.dh, xb, Mb, s.dm, s.dh, s.dm, dw1, s.dm};
    g.run(dyb, Mb, s.dm, 1, ws + w.a, Mb, s.dh, 1, s.dm, s.dh, Mb, GEMM_ACC, dw2, s.dh, RA_F32, nullptr, nullptr,
          &dw1_prob);
  }
  return g.rc;
}

#pragma GCC visibility pop
}  // extern "C"

// ----------------------------------------------------- one step from host memory
namespace ra {
namespace {

// Device workspace of ra_ring_step_host: device copies of the inputs and
// outputs (packed [B, N, H, d]; LSE [B, Hq, N]) and the forward and backward
// workspaces.
struct HostWs {
  size_t q, k, v, dO, o, lse, dq, dk, dv, fwd, bwd, total;
};
HostWs host_layout(int dtype, int o_dtype, int grad_dtype, const ra_shape& sh, int P) {
  HostWs w{};
  const size_t qel = (size_t)sh.B * sh.N_q * sh.Hq * sh.d, kvel = (size_t)sh.B * sh.N_kv * sh.Hkv * sh.d;
  ra_shape packed = sh;
  packed.q_bstride = packed.q_rstride = packed.q_hstride = 0;
  packed.kv_bstride = packed.kv_rstride = packed.kv_hstride = 0;
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  const size_t es = dtype_size(dtype), gs = dtype_size(grad_dtype);
  w.q = take(qel * es);
  w.k = take(kvel * es);
  w.v = take(kvel * es);
  w.dO = take(qel * es);
  w.o = take(qel * dtype_size(o_dtype));
  w.lse = take((size_t)sh.B * sh.Hq * sh.N_q * 4);
  w.dq = take(qel * gs);
  w.dk = take(kvel * gs);
  w.dv = take(kvel * gs);
  w.fwd = take(ra_ring_fwd_workspace_bytes((ra_dtype)dtype, packed, P));
  w.bwd = take(ra_ring_bwd_workspace_bytes((ra_dtype)dtype, (ra_dtype)grad_dtype, packed, P));
  w.total = off;
  return w;
}

// Side streams of ra_ring_step_host, one pair per device, created on first
// use and kept for the life of the process.
struct SideStreams {
  std::mutex mu;
  cudaStream_t in[kMaxDevices] = {}, out[kMaxDevices] = {};
};
SideStreams& side_streams() {
  static SideStreams s;
  return s;
}
int get_side_streams(cudaStream_t* in, cudaStream_t* out) {
  int dev;
  int rc = current_device(&dev);
  if (rc) return rc;
  SideStreams& s = side_streams();
  std::lock_guard<std::mutex> lk(s.mu);
  if (!s.in[dev]) {
    cudaError_t e = cudaStreamCreateWithFlags(&s.in[dev], cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&s.out[dev], cudaStreamNonBlocking);
    if (e != cudaSuccess) {
      s.in[dev] = s.out[dev] = nullptr;
      return cuda_fail(e, "create side streams");
    }
  }
  *in = s.in[dev];
  *out = s.out[dev];
  return RA_OK;
}

// Copies B batches of `batch` elements between a buffer with batch stride
// `src_bs` and one with batch stride `dst_bs` (elements of `es` bytes).
cudaError_t copy_batches(void* dst, long long dst_bs, const void* src, long long src_bs, int B,
                         long long batch, size_t es, cudaStream_t st) {
  if (dst_bs == batch && src_bs == batch)
    return cudaMemcpyAsync(dst, src, (size_t)B * batch * es, cudaMemcpyDefault, st);
  for (int b = 0; b < B; ++b) {
    cudaError_t e = cudaMemcpyAsync(static_cast<char*>(dst) + (size_t)b * dst_bs * es,
                                    static_cast<const char*>(src) + (size_t)b * src_bs * es,
                                    (size_t)batch * es, cudaMemcpyDefault, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

struct Events {
  cudaEvent_t e[4] = {};
  ~Events() {
    for (cudaEvent_t x : e)
      if (x) cudaEventDestroy(x);  // released once the recorded work completes
  }
};

}  // namespace
}  // namespace ra

extern "C" {
#pragma GCC visibility push(default)

size_t ra_ring_step_host_workspace_bytes(ra_dtype dtype, ra_dtype o_dtype, ra_dtype grad_dtype,
                                         ra_shape shape, int P) {
  if (shape.B < 1 || shape.N_q < 1 || shape.N_kv < 1 || shape.Hq < 1 || shape.Hkv < 1 || shape.d < 1 ||
      !valid_dtype(dtype) || !valid_dtype(o_dtype) || !valid_dtype(grad_dtype))
    return 0;
  return host_layout(dtype, o_dtype, grad_dtype, shape, P).total;
}

int ra_ring_step_host(const void* q, const void* k, const void* v, const void* dO, ra_dtype dtype,
                      ra_shape shape, int P, int flags, float scale, void* o, ra_dtype o_dtype,
                      float* lse, void* dq, void* dk, void* dv, ra_dtype grad_dtype, void* workspace,
                      size_t ws_bytes, void* stream) {
  // everything the forward and backward would reject is rejected before any
  // copy is enqueued
  if (flags & ~(RA_CAUSAL | RA_PRECISE | RA_STRIPED))
    return fail(RA_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
  Shape s;
  int rc;
  if ((rc = check_shape(shape, &s))) return rc;
  if (!valid_dtype(dtype) || !valid_dtype(o_dtype) || !valid_dtype(grad_dtype))
    return fail(RA_ERR_INVALID_ARG, "bad dtype");
  if ((rc = check_scale(scale))) return rc;
  if ((rc = check_ring(s, P, dtype))) return rc;
  const void* ins[4] = {q, k, v, dO};
  const char* in_names[4] = {"q", "k", "v", "dO"};
  for (int i = 0; i < 4; ++i)
    if (!ins[i]) return fail(RA_ERR_INVALID_ARG, "%s is NULL", in_names[i]);
  if (!o || !lse || !dq || !dk || !dv) return fail(RA_ERR_INVALID_ARG, "an output pointer is NULL");
  if (!is_packed(s.ql, s.Nq, s.Hq, s.d) || !is_packed(s.kvl, s.Nkv, s.Hkv, s.d))
    return fail(RA_ERR_UNSUPPORTED,
                "ra_ring_step_host takes host tensors with packed rows (row stride H*d, head stride d); "
                "batch strides may be any");
  const HostWs w = host_layout(dtype, o_dtype, grad_dtype, shape, P);
  if (!workspace || ws_bytes < w.total)
    return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", w.total, ws_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(RA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  if (dtype == RA_F32) {
    if (s.d != 32 && s.d != 64 && s.d != 128)
      return fail(RA_ERR_UNSUPPORTED, "fp32 path supports d in {32, 64, 128} (got %d)", s.d);
  } else {
    Shape packed = s;
    packed.ql = packed_lay(s.Nq, s.Hq, s.d);
    packed.kvl = packed_lay(s.Nkv, s.Hkv, s.d);
    if ((rc = check_tc(packed, dtype))) return rc;
  }
  cudaStream_t main_st = static_cast<cudaStream_t>(stream), in_st, out_st;
  if ((rc = get_side_streams(&in_st, &out_st))) return rc;
  Events ev;
  for (cudaEvent_t& e : ev.e) {
    cudaError_t err = cudaEventCreateWithFlags(&e, cudaEventDisableTiming);
    if (err != cudaSuccess) return cuda_fail(err, "cudaEventCreateWithFlags");
  }
  char* ws = static_cast<char*>(workspace);
  const long long qel = (long long)s.Nq * s.Hq * s.d, kvel = (long long)s.Nkv * s.Hkv * s.d;
  const size_t es = dtype_size(dtype), gs = dtype_size(grad_dtype);
  ra_shape packed = shape;
  packed.q_bstride = packed.q_rstride = packed.q_hstride = 0;
  packed.kv_bstride = packed.kv_rstride = packed.kv_hstride = 0;
  cudaError_t e;
  // dO travels on the input side stream while q, k, v go up and the forward runs
  if ((e = cudaEventRecord(ev.e[0], main_st)) != cudaSuccess ||
      (e = cudaStreamWaitEvent(in_st, ev.e[0], 0)) != cudaSuccess)
    return cuda_fail(e, "dO upload");
  {
    TimedLaunch tl(RA_COPY_H2D, in_st);
    if ((e = copy_batches(ws + w.dO, qel, dO, s.ql.bs, s.B, qel, es, in_st)) != cudaSuccess)
      return cuda_fail(e, "dO upload");
  }
  if ((e = cudaEventRecord(ev.e[1], in_st)) != cudaSuccess) return cuda_fail(e, "dO upload");
  {
    TimedLaunch tl(RA_COPY_H2D, main_st);
    if ((e = copy_batches(ws + w.q, qel, q, s.ql.bs, s.B, qel, es, main_st)) != cudaSuccess ||
        (e = copy_batches(ws + w.k, kvel, k, s.kvl.bs, s.B, kvel, es, main_st)) != cudaSuccess ||
        (e = copy_batches(ws + w.v, kvel, v, s.kvl.bs, s.B, kvel, es, main_st)) != cudaSuccess)
      return cuda_fail(e, "q, k, v upload");
  }
  rc = ring_fwd_impl(ws + w.q, ws + w.k, ws + w.v, dtype, packed, P, flags, scale, ws + w.o, o_dtype,
                     reinterpret_cast<float*>(ws + w.lse), ws + w.fwd, w.bwd - w.fwd, stream, nullptr);
  if (rc) return rc;
  // O and LSE travel down on the output side stream while the backward runs
  if ((e = cudaEventRecord(ev.e[2], main_st)) != cudaSuccess ||
      (e = cudaStreamWaitEvent(out_st, ev.e[2], 0)) != cudaSuccess)
    return cuda_fail(e, "O, LSE download");
  {
    TimedLaunch tl(RA_COPY_D2H, out_st);
    if ((e = copy_batches(o, s.ql.bs, ws + w.o, qel, s.B, qel, dtype_size(o_dtype), out_st)) != cudaSuccess ||
        (e = cudaMemcpyAsync(lse, ws + w.lse, (size_t)s.B * s.Hq * s.Nq * 4, cudaMemcpyDefault, out_st)) !=
            cudaSuccess)
      return cuda_fail(e, "O, LSE download");
  }
  if ((e = cudaEventRecord(ev.e[3], out_st)) != cudaSuccess) return cuda_fail(e, "O, LSE download");
  if ((e = cudaStreamWaitEvent(main_st, ev.e[1], 0)) != cudaSuccess) return cuda_fail(e, "join dO upload");
  rc = ring_bwd_impl(ws + w.q, ws + w.k, ws + w.v, ws + w.o, o_dtype, ws + w.dO,
                     reinterpret_cast<const float*>(ws + w.lse), dtype, packed, P, flags, scale, ws + w.dq,
                     ws + w.dk, ws + w.dv, grad_dtype, ws + w.bwd, w.total - w.bwd, stream, nullptr);
  if (rc) return rc;
  {
    TimedLaunch tl(RA_COPY_D2H, main_st);
    if ((e = copy_batches(dq, s.ql.bs, ws + w.dq, qel, s.B, qel, gs, main_st)) != cudaSuccess ||
        (e = copy_batches(dk, s.kvl.bs, ws + w.dk, kvel, s.B, kvel, gs, main_st)) != cudaSuccess ||
        (e = copy_batches(dv, s.kvl.bs, ws + w.dv, kvel, s.B, kvel, gs, main_st)) != cudaSuccess)
      return cuda_fail(e, "gradient download");
  }
  if ((e = cudaStreamWaitEvent(main_st, ev.e[3], 0)) != cudaSuccess) return cuda_fail(e, "join O download");
  return RA_OK;
}

#pragma GCC visibility pop
}  // extern "C"

// ------------------------------------------------ cross entropy of a vocabulary
namespace ra {
namespace {

// How one product is cut up.  A CTA pair works on a tile of 256 rows by 256 or 128
// columns; GB300 has 76 pairs, and the cut is made for that number whatever the device,
// so that workspaces and results do not depend on it.
//   - Where the result may be a sum of fp32 planes and wide tiles fill less than half the
//     pairs, K is split over the idle ones.  A k-slab (64) of a wide tile takes about
//     0.33 us; planes cost another launch that adds them up, 5 us in all.
//   - A narrow tile takes as long as a wide one (measured: 0.98 against 1.86 PFLOP/s on
//     8192 x 131072 x 2048), only its epilogue is shorter: it is taken where even the
//     narrow tiles find a pair each.
constexpr int kPairs = 76;
struct Cut {
  int bn, splits;
};
Cut cut_product(long long M, long long N, long long K, bool may_split) {
  const long long tm = (M + 255) / 256, wide = tm * ((N + 255) / 256), narrow = tm * ((N + 127) / 128);
  if (may_split && wide * 2 <= kPairs) {
    const long long by_k = (K + 255) / 256, by_pairs = kPairs / wide;
    const int splits = (int)(by_k < by_pairs ? by_k : by_pairs);
    const double whole = 0.33 * (double)((K + 63) / 64);
    if (splits > 1 && whole / splits + 5.0 < whole) return Cut{256, splits};
  }
  return Cut{narrow <= kPairs ? 128 : 256, 1};
}

// CTA-pair products of the cross entropy, one or two in a launch.
struct PairPlan {
  cudaStream_t st;
  int* status;
  int sms;
  struct Operand {  // a matrix of rows x cols as stored, or several, one after the other
    const void* p;
    long long rows, cols, ld;
    int count = 1;
  };
  // q: M, N, K, the majornesses and the output; sets the operands' maps and the cut
  int problem(PairProblem& q, Cut cut, const Operand& A, const Operand& B, int dtype) const {
    int rc;
    // few rows: only those are loaded (whole boxes would fill in zeros, which costs as much
    // as data)
    q.a_rows = !q.a_mn && q.M < 128 ? (q.M + 7) / 8 * 8 : 128;
    if ((rc = make_map_3d(&q.tm_a, A.p, dtype, A.cols, A.rows, A.count, A.ld, A.rows * A.ld, 64,
                          q.a_mn ? 64 : q.a_rows)) ||
        (rc = make_map_3d(&q.tm_b, B.p, dtype, B.cols, B.rows, 1, B.ld, 0, 64, q.b_mn ? 64 : cut.bn / 2)))
      return rc;
    q.bn = cut.bn;
    q.splits = cut.splits;
    // the pairs at work together cover all columns of a few tile rows, or 16 tile
    // rows where the columns are many
    const int tn = (q.N + cut.bn - 1) / cut.bn;
    q.group_m = tn < 5 ? (kPairs + tn - 1) / tn : 16;
    return RA_OK;
  }
  int launch(PairArgs& a, int dtype) const {
    a.ab_bf16 = dtype == RA_BF16;
    a.status = status;
    a.wait_limit_ns = wait_limit_ns();
    TimedLaunch tl(RA_KERNEL_PAIR_TC, st);
    const cudaError_t e = launch_xent_pair(a, sms, st);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "cross-entropy product launch");
  }
  int launch_few(const XentFewArgs& f) const {
    TimedLaunch tl(RA_KERNEL_PAIR_TC, st);
    const cudaError_t e =
        f.T == 1 && f.D * 4 <= kXentTokenSmem ? launch_xent_token(f, st) : launch_xent_few(f, st);
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "cross-entropy launch for few tokens");
  }
};

struct XentShape {
  long long T, xs, ws;
  int D, V, block;
};

int check_xent(ra_dtype dtype, long long T, int D, int V, long long x_rstride, long long w_rstride, int block,
               XentShape* out) {
  if (dtype != RA_BF16 && dtype != RA_F16)
    return fail(RA_ERR_UNSUPPORTED, "the cross entropy takes bf16 or fp16 operands");
  if (T < 1 || D < 1 || V < 1 || block < 1)
    return fail(RA_ERR_INVALID_ARG, "non-positive cross-entropy size (T=%lld D=%d V=%d block=%d)", T, D, V, block);
  if (D % 8) return fail(RA_ERR_UNSUPPORTED, "D must be a multiple of 8 (got %d)", D);
  if (T > (1 << 30) || V > (1 << 30) || D > (1 << 20)) return fail(RA_ERR_INVALID_ARG, "cross-entropy size too large");
  if (x_rstride == 0) x_rstride = D;
  if (w_rstride == 0) w_rstride = D;
  if (x_rstride < D || w_rstride < D || x_rstride > (1ll << 32) || w_rstride > (1ll << 32))
    return fail(RA_ERR_INVALID_ARG, "row strides (%lld, %lld) must be 0 or at least D=%d", x_rstride, w_rstride, D);
  if (x_rstride % 8 || w_rstride % 8)
    return fail(RA_ERR_INVALID_ARG, "row strides must be multiples of 8 elements (got %lld, %lld)", x_rstride, w_rstride);
  // a block whose gradient takes less than 256 MB is widened to that: narrower ones are
  // bound by launches and leave SMs idle at their ends (4096 tokens, D 2048, V 32768: 1193
  // us in blocks of 64 MB, 1021 us in one of 256 MB)
  const long long least = ((256ll << 20) / (2 * T)) / 256 * 256;
  const long long wide = block > least ? block : least;
  *out = XentShape{T, x_rstride, w_rstride, D, V, (int)(wide < V ? wide : V)};
  return RA_OK;
}

// Whether the kernels for few tokens take a call, and their blocks (and so parts) for V
// entries: a single token 16 entries a block and turn, eight blocks per SM at most;
// several tokens units of 16 entries, four at a time.
bool single_token(const XentShape& s) { return s.T == 1 && s.D * 4 <= kXentTokenSmem; }
bool few_tokens(const XentShape& s) { return single_token(s) || xent_few(s.T, s.D); }
int few_blocks(const XentShape& s, int V) {
  const int n = (V + 15) / 16, turns = (n + 3) / 4;
  if (single_token(s)) return n < 16 * kPairs ? n : 16 * kPairs;
  return turns < 2 * kPairs ? turns : 2 * kPairs;
}
XentFewArgs few_args(const XentShape& s, const void* x, const void* w, int dtype, const long long* targets,
                     long long ignore, int V) {
  XentFewArgs f;
  memset(&f, 0, sizeof f);
  f.x = x; f.w = w; f.bf16 = dtype == RA_BF16;
  f.T = (int)s.T; f.D = s.D; f.V = V;
  f.blocks = few_blocks(s, V);
  f.xs = s.xs; f.ws = s.ws;
  f.targets = targets; f.ignore = ignore; f.vocab = s.V;
  return f;
}

// forward: target logits [T] fp32 | statistics [column parts][T] (max, sum); the
// tensor-core tiles' parts and those of few tokens are at most ceil(V / 64)
struct XentFwdWs {
  size_t target, stats, total;
};
XentFwdWs xent_fwd_layout(const XentShape& s) {
  XentFwdWs w{};
  w.stats = align256((size_t)s.T * 4);
  const int tiles = (s.V + 63) / 64, token = single_token(s) ? few_blocks(s, s.V) : 0;
  w.total = w.stats + align256((size_t)(tiles > token ? tiles : token) * s.T * 8);
  return w;
}

// Up to so many tokens the logits' gradient is kept as two 16-bit terms, a matrix each: both
// fit the tiles that one would take.
constexpr int kTwoTerms = 64;  // one k-slab of dw = d^T x

// backward: scale (256 bytes) | gradient of one block's logits [terms][T][ld] 16-bit | fp32
// sum of dx: its splits' planes (of both terms' products, one below the other), or [T, D]
// where dx is 16-bit and there is more than one block | planes of one block's dw where its
// product is split
struct XentBwdWs {
  size_t scale, d, acc, dw, total;
  long long ld;
  int terms;
  Cut dx_cut, dw_cut;
};
XentBwdWs xent_bwd_layout(const XentShape& s, int dx_dtype) {
  XentBwdWs w{};
  w.ld = (s.block + 63) / 64 * 64;
  w.terms = s.T <= kTwoTerms ? 2 : 1;
  w.dx_cut = cut_product(s.T * w.terms, s.D, s.block, true);
  w.dw_cut = cut_product(s.block, s.D, s.T, true);
  w.d = 256;
  w.acc = w.d + align256((size_t)s.T * w.terms * w.ld * 2);
  w.dw = w.acc;
  if (w.dx_cut.splits > 1) w.dw += align256((size_t)w.dx_cut.splits * w.terms * s.T * s.D * 4);
  else if (dx_dtype != RA_F32 && s.block < s.V) w.dw += align256((size_t)s.T * s.D * 4);
  w.total = w.dw;
  if (w.dw_cut.splits > 1) w.total += align256((size_t)w.dw_cut.splits * s.block * s.D * 4);
  return w;
}

int check_targets(const long long* targets) {
  if (!targets || (reinterpret_cast<uintptr_t>(targets) & 7u))
    return fail(RA_ERR_INVALID_ARG, "targets must be a non-NULL, 8-byte aligned device array of 64-bit integers");
  return RA_OK;
}
int check_floats(const void* p, const char* name) {
  if (!p || (reinterpret_cast<uintptr_t>(p) & 3u))
    return fail(RA_ERR_INVALID_ARG, "%s must be a non-NULL, 4-byte aligned device array", name);
  return RA_OK;
}
int check_workspace(const void* workspace, size_t ws_bytes, size_t need) {
  if (!workspace || ws_bytes < need)
    return fail(RA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(RA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  return RA_OK;
}

}  // namespace
}  // namespace ra

extern "C" {
#pragma GCC visibility push(default)

size_t ra_xent_fwd_workspace_bytes(ra_dtype dtype, long long T, int D, int V) {
  XentShape s;
  if (check_xent(dtype, T, D, V, 0, 0, V, &s)) return 0;
  return xent_fwd_layout(s).total;
}

size_t ra_xent_bwd_workspace_bytes(ra_dtype dtype, ra_dtype dx_dtype, long long T, int D, int V, int block) {
  XentShape s;
  if (check_xent(dtype, T, D, V, 0, 0, block, &s) || !valid_dtype(dx_dtype)) return 0;
  return xent_bwd_layout(s, dx_dtype).total;
}

int ra_xent_fwd(const void* x, const void* w, ra_dtype dtype, long long T, int D, int V, long long x_rstride,
                long long w_rstride, const long long* targets, long long ignore_index, float* loss, float* lse,
                void* workspace, size_t ws_bytes, void* stream) {
  XentShape s;
  int rc;
  if ((rc = check_xent(dtype, T, D, V, x_rstride, w_rstride, V, &s))) return rc;
  if ((rc = check_ptr(x, "x")) || (rc = check_ptr(w, "w")) || (rc = check_targets(targets)) ||
      (rc = check_floats(loss, "loss")) || (rc = check_floats(lse, "lse")))
    return rc;
  const XentFwdWs l = xent_fwd_layout(s);
  if ((rc = check_workspace(workspace, ws_bytes, l.total))) return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  if (!device_is_sm103()) return fail(RA_ERR_UNSUPPORTED, "tensor-core kernels are built for sm_103a only");
  char* base = static_cast<char*>(workspace);
  PairPlan plan{static_cast<cudaStream_t>(stream), st, device_sms()};
  PairArgs a;
  memset(&a, 0, sizeof a);
  a.epi = PAIR_STATS;
  a.problems = 1;
  a.q[0].M = (int)s.T; a.q[0].N = s.V; a.q[0].K = s.D;
  a.targets = targets;
  a.ignore = ignore_index;
  a.vocab = s.V;
  a.stats = reinterpret_cast<float2*>(base + l.stats);
  a.target_logit = reinterpret_cast<float*>(base);
  int parts = 0;
  cudaError_t e;
  if (few_tokens(s)) {
    XentFewArgs f = few_args(s, x, w, dtype, targets, ignore_index, s.V);
    parts = f.blocks;
    f.stats = a.stats;
    f.target_logit = a.target_logit;
    if ((rc = plan.launch_few(f))) return rc;
  } else {
    const Cut cut = cut_product(s.T, s.V, s.D, false);
    if ((rc = plan.problem(a.q[0], cut, {x, s.T, s.D, s.xs}, {w, s.V, s.D, s.ws}, dtype)) ||
        (rc = plan.launch(a, dtype)))
      return rc;
    parts = (s.V + cut.bn / 2 - 1) / (cut.bn / 2);
  }
  e = launch_xent_finish(a.stats, parts, a.target_logit, targets, ignore_index, s.V, s.T, loss, lse, st, plan.st);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cross-entropy reduction launch");
}

int ra_xent_bwd(const void* x, const void* w, ra_dtype dtype, long long T, int D, int V, long long x_rstride,
                long long w_rstride, const long long* targets, long long ignore_index, const float* lse,
                const float* dloss, int block, void* dx, ra_dtype dx_dtype, void* dw, ra_dtype dw_dtype,
                void* workspace, size_t ws_bytes, void* stream) {
  XentShape s;
  int rc;
  if ((rc = check_xent(dtype, T, D, V, x_rstride, w_rstride, block, &s))) return rc;
  if (!valid_dtype(dx_dtype) || !valid_dtype(dw_dtype)) return fail(RA_ERR_INVALID_ARG, "bad gradient dtype");
  if ((rc = check_ptr(x, "x")) || (rc = check_ptr(w, "w")) || (rc = check_targets(targets)) ||
      (rc = check_floats(lse, "lse")) || (rc = check_floats(dloss, "dloss")) || (rc = check_ptr(dx, "dx")) ||
      (rc = check_ptr(dw, "dw")))
    return rc;
  const XentBwdWs l = xent_bwd_layout(s, dx_dtype);
  if ((rc = check_workspace(workspace, ws_bytes, l.total))) return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  if (!device_is_sm103()) return fail(RA_ERR_UNSUPPORTED, "tensor-core kernels are built for sm_103a only");
  char* base = static_cast<char*>(workspace);
  PairPlan plan{static_cast<cudaStream_t>(stream), st, device_sms()};
  float* scale = nullptr;
  if (dtype == RA_F16) {
    scale = reinterpret_cast<float*>(base);
    const cudaError_t e = launch_xent_scale(dloss, targets, ignore_index, s.V, s.T, scale, plan.st);
    if (e != cudaSuccess) return cuda_fail(e, "gradient scale launch");
  }
  void* d = base + l.d;
  float* planes = reinterpret_cast<float*>(base + l.acc);
  float* dw_planes = reinterpret_cast<float*>(base + l.dw);
  const bool dx_split = l.dx_cut.splits > 1, dw_split = l.dw_cut.splits > 1;
  for (int v0 = 0; v0 < s.V; v0 += s.block) {
    const int C = s.V - v0 < s.block ? s.V - v0 : s.block;
    const bool first = v0 == 0, last = v0 + C == s.V;
    const char* wb = static_cast<const char*>(w) + (size_t)v0 * s.ws * 2;
    const PairPlan::Operand W{wb, C, s.D, s.ws}, X{x, s.T, s.D, s.xs}, Dl{d, s.T, C, l.ld, l.terms};
    const int k_slabs = (C + 63) / 64;
    PairArgs a;
    memset(&a, 0, sizeof a);
    a.scale = scale;
    // d = gradient of this block's logits, recomputed from x and w
    if (few_tokens(s)) {
      XentFewArgs f = few_args(s, x, wb, dtype, targets, ignore_index, C);
      f.col_off = v0;
      f.lse = lse;
      f.grad = dloss;
      f.scale = scale;
      f.d = d;
      f.ld = l.ld;
      if ((rc = plan.launch_few(f))) return rc;
    } else {
      a.epi = PAIR_DLOGITS;
      a.problems = 1;
      a.q[0].M = (int)s.T; a.q[0].N = C; a.q[0].K = s.D;
      a.targets = targets;
      a.ignore = ignore_index;
      a.vocab = s.V;
      a.col_off = v0;
      a.lse = lse;
      a.grad = dloss;
      a.two_terms = l.terms == 2;
      if ((rc = make_map_3d(&a.q[0].tm_c, d, dtype, C, s.T, l.terms, l.ld, s.T * l.ld, 64, 32)) ||
          (rc = plan.problem(a.q[0], cut_product(s.T, C, s.D, false), X, W, dtype)) || (rc = plan.launch(a, dtype)))
        return rc;
    }
    // dx += d W  (W's rows as [K, N]: MN-major), summed over blocks in fp32, and in the
    // same launch this block's dw = d^T x  (both MN-major); the longer units first.  Two
    // terms of d are further rows of a split dx, whose planes are added up anyway; otherwise
    // they follow each other along K, x or W being read again.
    a.epi = PAIR_STORE;
    a.problems = 2;
    const bool dx_first = C / l.dx_cut.splits >= s.T / l.dw_cut.splits;
    PairProblem &qx = a.q[dx_first ? 0 : 1], &qw = a.q[dx_first ? 1 : 0];
    const long long dx_rows = dx_split ? s.T * l.terms : s.T;
    qx.M = (int)dx_rows; qx.N = s.D; qx.K = C;
    if (l.terms == 2 && !dx_split) {
      qx.fold = k_slabs;
      qx.K = 2 * k_slabs * 64;
    }
    qx.a_mn = 0;
    qx.b_mn = 1;
    qx.c_dtype = dx_split || dx_dtype == RA_F32 || !last ? RA_F32 : dx_dtype;
    void* c = dx_split || (qx.c_dtype == RA_F32 && dx_dtype != RA_F32) ? (void*)planes : dx;
    qx.c_accumulate = qx.c_dtype == RA_F32 && !first;
    qx.c_add = qx.c_dtype != RA_F32 && !first ? planes : nullptr;
    // the last block may be too short for as many splits: its planes are fewer, the
    // others keep what they hold
    Cut cut = l.dx_cut;
    if (cut.splits > k_slabs) cut.splits = k_slabs;
    qw.M = C; qw.N = s.D; qw.K = (int)s.T;
    if (l.terms == 2) {
      qw.fold = 1;
      qw.K = 2 * 64;
    }
    qw.a_mn = qw.b_mn = 1;
    qw.c_dtype = dw_split ? RA_F32 : dw_dtype;
    qw.c_accumulate = 0;
    qw.c_add = nullptr;
    void* dwb = static_cast<char*>(dw) + (size_t)v0 * s.D * dtype_size(dw_dtype);
    const PairPlan::Operand rows{d, dx_rows, C, l.ld};
    if ((rc = make_map_3d(&qx.tm_c, c, qx.c_dtype, s.D, dx_rows, dx_split ? l.dx_cut.splits : 1, s.D, dx_rows * s.D,
                          qx.c_dtype == RA_F32 ? 32 : 64, 32)) ||
        (rc = plan.problem(qx, cut, dx_split ? rows : Dl, W, dtype)) ||
        (rc = make_map_3d(&qw.tm_c, dw_split ? dw_planes : dwb, qw.c_dtype, s.D, C, l.dw_cut.splits, s.D,
                          (long long)C * s.D, qw.c_dtype == RA_F32 ? 32 : 64, 32)) ||
        (rc = plan.problem(qw, l.dw_cut, Dl, X, dtype)) || (rc = plan.launch(a, dtype)))
      return rc;
    if (dw_split) {
      const cudaError_t e = launch_sum_planes(dw_planes, l.dw_cut.splits, (long long)C * s.D, dwb, dw_dtype, plan.st);
      if (e != cudaSuccess) return cuda_fail(e, "dw sum launch");
    }
  }
  if (dx_split) {
    const cudaError_t e = launch_sum_planes(planes, l.dx_cut.splits * l.terms, s.T * s.D, dx, dx_dtype, plan.st);
    if (e != cudaSuccess) return cuda_fail(e, "dx sum launch");
  }
  return RA_OK;
}

#pragma GCC visibility pop
}  // extern "C"

// ------------------------------------------------ Newton-Schulz orthogonalisation
namespace ra {
namespace {

struct NsShape {
  int batch, rows, cols, m;  // m: the smaller side
  long long ld, ldm;         // padded rows of X and of the m x m matrices
  double sx, sa, sb;         // powers of two by which X, A' and B' are held in fp16
  double growth;             // log2 of the most by which a step lets a singular value grow
};

// The largest |p(s)| over s in [0, top], p(s) = a s + b s^3 + c s^5: at top or at a
// root of p'(s) = a + 3 b s^2 + 5 c s^4.
double ns_bound(double a, double b, double c, double top) {
  auto p = [&](double s) { return fabs(s * (a + s * s * (b + c * s * s))); };
  double best = p(top);
  double roots[2] = {-1.0, -1.0};
  if (c == 0.0) {
    if (b != 0.0) roots[0] = -a / (3.0 * b);
  } else {
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (disc >= 0.0) {
      roots[0] = (-3.0 * b + sqrt(disc)) / (10.0 * c);
      roots[1] = (-3.0 * b - sqrt(disc)) / (10.0 * c);
    }
  }
  for (double r : roots)
    if (r > 0.0 && r < top * top && p(sqrt(r)) > best) best = p(sqrt(r));
  return best;
}
// The largest |p(s) / s| over s in [0, top]: at an end or where a + b t + c t^2 turns, t = s^2.
double ns_growth(double a, double b, double c, double top) {
  auto q = [&](double t) { return fabs(a + t * (b + c * t)); };
  double best = q(0.0) > q(top * top) ? q(0.0) : q(top * top);
  const double turn = c != 0.0 ? -b / (2.0 * c) : -1.0;
  if (turn > 0.0 && turn < top * top && q(turn) > best) best = q(turn);
  return best;
}
double pow2_below(double x) { return ldexp(1.0, ilogb(x)); }

int check_ns(int batch, int rows, int cols, const float* coeffs, int steps, float eps, NsShape* out) {
  if (batch < 1 || rows < 1 || cols < 1 || steps < 1)
    return fail(RA_ERR_INVALID_ARG, "non-positive Newton-Schulz size (batch=%d rows=%d cols=%d steps=%d)", batch, rows,
                cols, steps);
  if (rows > 65536 || cols > 65536 || batch > 65535 || steps > 100)
    return fail(RA_ERR_INVALID_ARG, "Newton-Schulz size too large (batch=%d rows=%d cols=%d steps=%d)", batch, rows,
                cols, steps);
  if (!coeffs) return fail(RA_ERR_INVALID_ARG, "coeffs is NULL");
  for (int i = 0; i < 3; ++i)
    if (!isfinite(coeffs[i])) return fail(RA_ERR_INVALID_ARG, "coeffs must be finite");
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(RA_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", (double)eps);
  NsShape s{};
  s.batch = batch; s.rows = rows; s.cols = cols;
  s.m = rows < cols ? rows : cols;
  s.ld = (cols + 63) / 64 * 64;
  s.ldm = (s.m + 63) / 64 * 64;
  // Singular values start at or below 1 and stay below `top`; from that follow the
  // largest entries of X, A' and B', which must fit fp16 times their powers of two.
  const double a = coeffs[0], b = coeffs[1], c = coeffs[2];
  double top = 1.0, cur = 1.0, growth = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double g = ns_growth(a, b, c, cur);
    if (g > growth) growth = g;
    cur = ns_bound(a, b, c, cur);
    if (!(cur < 64.0))
      return fail(RA_ERR_UNSUPPORTED, "coeffs (%g, %g, %g) let singular values grow past 64", a, b, c);
    if (cur > top) top = cur;
  }
  s.growth = log2(growth) * (1.0 + 1e-6);
  const double t2 = top * top, room = 32768.0;
  const double bmax = (fabs(b) + 2.0 * fabs(c) * t2) * t2 + fabs(c) * t2 * t2;
  s.sa = pow2_below(room / t2);
  s.sb = pow2_below(room / (bmax > 1.0 ? bmax : 1.0));
  const double most = pow2_below(room / top), want = pow2_below(sqrt((double)rows * cols));
  s.sx = want < most ? want : most;
  *out = s;
  return RA_OK;
}

// Matrices with a side of at most 128 and the other at most 4096 go to clusters of CTAs
// that hold them whole: slices of 64 columns on up to 8 CTAs or of 128 on up to 16 (the
// largest cluster) where the SMs suffice for the batch, of 256 otherwise.  Measured with
// cold caches, code among what is cold: 97 x
// 1757 63 us with 16 slices of 128, 100 with 8 of 256; 120 x 1000 49 with 8 of 128, 51
// with 16 of 64; 12 of 128 x 2000 92 with slices of 256, 115 with 128 in two rounds; 120 x
// 4000 105 with 256, 182 in the general chain.
bool ns_small_cut(const NsShape& s, int* slice, int* cluster) {
  const int n = s.rows > s.cols ? s.rows : s.cols;
  if (s.m > 128 || n > 4096) return false;
  auto ctas = [&](int c) {
    int g = 1;
    while (g * c < n) g *= 2;
    return g;
  };
  int c = 64;
  while (c < 256 && (ctas(c) > (c == 64 ? 8 : 16) || (long long)s.batch * ctas(c) > 2 * kPairs)) c *= 2;
  *slice = c;
  *cluster = ctas(c);
  return true;
}

// The cut of one phase: the tile's width as for the cross entropy's products; K may be
// split for every phase, over at most as many pairs as run at once.  A k-slab of a wide
// tile takes about 0.33 us; exchanging the splits' sums takes 5 us and 1.5 us more for each
// split past the second.  (2600 x 400: 180 us in all, 191 with splits taken for 4 us and 0.3
// us each; 16 of 256 x 1024: 158 without splits, 178 with them.)  Wide tiles only.
Cut ns_cut(const NsArgs& a, int kind, int pairs) {
  const long long K = kind == NS_GRAM && !a.tall ? a.cols : kind == NS_GRAM ? a.rows : a.m;
  const long long wide = (long long)a.batch * ns_phase_tiles(a, kind, 256);
  const long long narrow = (long long)a.batch * ns_phase_tiles(a, kind, 128);
  const long long by_pairs = pairs / wide;
  const double whole = 0.33 * (double)((K + 63) / 64);
  int best = 1;
  double best_us = whole;
  for (int s = 2; s <= by_pairs && s <= K / 256; ++s) {
    const double us = whole / s + 5.0 + 1.5 * (s - 2);
    if (us < best_us) {
      best_us = us;
      best = s;
    }
  }
  if (best > 1) return Cut{256, best};
  return Cut{narrow <= pairs ? 128 : 256, 1};
}

// words, flags, counts and shifts | norm parts | sums of X's squares (two buffers) | X high terms
// (two buffers) | X low terms | A' | B' | sums of splits
struct NsWs {
  size_t words, parts, sums[2], hi[2], lo, a, b, partials, total;
};
// 16 partial sums per unit of the update; narrow tiles bound their number, or pairs where
// tiles are split
size_t ns_sums(const NsShape& s) {
  const size_t tiles = (size_t)((s.rows + 255) / 256) * ((s.cols + 127) / 128);
  return 16 * (tiles > kPairs ? tiles : kPairs);
}
NsWs ns_layout(const NsShape& s) {
  NsWs w{};
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  const size_t x = (size_t)s.batch * s.rows * s.ld * 2, g = (size_t)s.batch * s.m * s.ldm * 2;
  w.words = take(((size_t)kNsWords + 2 * s.batch) * 4);
  w.parts = take((size_t)s.batch * kNsParts * 3 * 4);
  for (size_t& at : w.sums) at = take((size_t)s.batch * ns_sums(s) * 4);
  w.hi[0] = take(x);
  w.hi[1] = take(x);
  w.lo = take(x);
  w.a = take(g);
  w.b = take(g);
  NsArgs a;
  memset(&a, 0, sizeof a);
  a.batch = s.batch; a.rows = s.rows; a.cols = s.cols; a.m = s.m; a.tall = s.rows > s.cols;
  size_t units = 0;
  for (int k = NS_GRAM; k <= NS_UPDATE; ++k) {
    const int splits = ns_cut(a, k, kPairs).splits;
    if (splits > 1) units += (size_t)splits * s.batch * ns_phase_tiles(a, k, 256);
  }
  w.partials = take(units * 2 * 8 * 128 * 32 * 4);
  w.total = off;
  return w;
}

}  // namespace
}  // namespace ra

extern "C" {
#pragma GCC visibility push(default)

size_t ra_newton_schulz_workspace_bytes(int batch, int rows, int cols) {
  NsShape s;
  const float none[3] = {1.f, 0.f, 0.f};
  if (check_ns(batch, rows, cols, none, 1, 0.f, &s)) return 0;
  return ns_layout(s).total;
}

int ra_newton_schulz(const void* g, ra_dtype g_dtype, int batch, int rows, int cols, long long g_bstride,
                     long long g_rstride, const float* coeffs, int steps, float eps, void* out, ra_dtype out_dtype,
                     long long out_bstride, long long out_rstride, void* workspace, size_t ws_bytes, void* stream) {
  NsShape s;
  int rc;
  if ((rc = check_ns(batch, rows, cols, coeffs, steps, eps, &s))) return rc;
  if (!valid_dtype(g_dtype) || !valid_dtype(out_dtype)) return fail(RA_ERR_INVALID_ARG, "bad dtype");
  struct Side {
    const char* name;
    const void* p;
    int dtype;
    long long *bs, *rs;
  };
  for (const Side& d : {Side{"g", g, g_dtype, &g_bstride, &g_rstride}, Side{"out", out, out_dtype, &out_bstride, &out_rstride}}) {
    if (!d.p || (reinterpret_cast<uintptr_t>(d.p) & (dtype_size(d.dtype) - 1)))
      return fail(RA_ERR_INVALID_ARG, "%s is NULL or not aligned to its elements", d.name);
    if (*d.rs == 0) *d.rs = cols;
    const long long extent = (long long)(rows - 1) * *d.rs + cols;
    if (*d.bs == 0) *d.bs = extent;
    // one matrix after the other, or all matrices' rows between two rows of one
    const bool apart = *d.bs >= extent, between = *d.bs >= cols && *d.bs <= (1ll << 45) &&
                                                  *d.rs >= (batch - 1) * *d.bs + cols;
    if (*d.rs < cols || *d.rs > (1ll << 40) || *d.bs > (1ll << 45) || !(apart || between))
      return fail(RA_ERR_INVALID_ARG, "%s strides (%lld, %lld) make rows or matrices overlap", d.name, *d.bs, *d.rs);
  }
  const NsWs l = ns_layout(s);
  if ((rc = check_workspace(workspace, ws_bytes, l.total))) return rc;
  int* st;
  if ((rc = status_ptr(&st))) return rc;
  if (!device_is_sm103()) return fail(RA_ERR_UNSUPPORTED, "tensor-core kernels are built for sm_103a only");
  const long long gs = (long long)dtype_size(g_dtype), os = (long long)dtype_size(out_dtype);
  const NsInput in{g, g_dtype, batch, rows, cols, g_rstride, g_bstride,
                   aligned16(g) && (g_rstride * gs) % 16 == 0 && (g_bstride * gs) % 16 == 0};
  const bool out_vec = aligned16(out) && (out_rstride * os) % 16 == 0 && (out_bstride * os) % 16 == 0;
  int slice = 0, cluster = 0;
  if (ns_small_cut(s, &slice, &cluster)) {
    NsSmallArgs a;
    memset(&a, 0, sizeof a);
    a.in = in;
    a.m = s.m;
    a.n = rows > cols ? rows : cols;
    a.tall = rows > cols;
    a.steps = steps;
    a.ca = coeffs[0]; a.cb = coeffs[1]; a.cc = coeffs[2];
    a.sx = (float)s.sx; a.sa = (float)s.sa; a.sb = (float)s.sb; a.inv_sb = (float)(1.0 / s.sb); a.eps = eps;
    a.alpha_mul = (float)(1.0 / (s.sx * s.sx * s.m));
    a.gram_acc = (float)(s.sa / (s.sx * s.sx));
    a.square_acc = (float)(coeffs[2] * s.sb / (s.sa * s.sa));
    a.square_lin = (float)(s.sb / s.sa);
    a.out_mul = (float)(1.0 / s.sx);
    a.out = out; a.out_dtype = out_dtype; a.out_vec = out_vec; a.out_ld = out_rstride; a.out_bstride = out_bstride;
    a.status = st;
    a.wait_limit_ns = wait_limit_ns();
    TimedLaunch tl(RA_KERNEL_PAIR_TC, static_cast<cudaStream_t>(stream));
    const cudaError_t e = launch_ns_small(a, slice, cluster, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RA_OK : cuda_fail(e, "Newton-Schulz launch");
  }
  char* base = static_cast<char*>(workspace);
  NsArgs a;
  memset(&a, 0, sizeof a);
  a.batch = batch; a.rows = rows; a.cols = cols; a.m = s.m; a.tall = rows > cols;
  a.steps = steps;
  a.in = in;
  a.ca = coeffs[0]; a.cb = coeffs[1]; a.cc = coeffs[2];
  a.sx = (float)s.sx; a.sa = (float)s.sa; a.eps = eps;
  a.alpha_mul = (float)(1.0 / (s.sx * s.sx * s.m));
  a.gram_acc = (float)(s.sa / (s.sx * s.sx));
  a.square_acc = (float)(coeffs[2] * s.sb / (s.sa * s.sa));
  a.square_lin = (float)(s.sb / s.sa);
  a.update_acc = (float)(1.0 / s.sb);
  a.out_mul = (float)(1.0 / s.sx);
  a.words = reinterpret_cast<unsigned int*>(base + l.words);
  a.flags = a.words + 64;
  a.partials = reinterpret_cast<float*>(base + l.partials);
  a.parts = reinterpret_cast<float*>(base + l.parts);
  for (int i = 0; i < 2; ++i) a.sums[i] = reinterpret_cast<float*>(base + l.sums[i]);
  a.sums_ld = (long long)ns_sums(s);
  a.counts = a.words + kNsWords;
  a.shifts = reinterpret_cast<int*>(a.counts + batch);
  a.growth = (float)s.growth;
  uint16_t* hi[2] = {reinterpret_cast<uint16_t*>(base + l.hi[0]), reinterpret_cast<uint16_t*>(base + l.hi[1])};
  a.hi0 = hi[0];
  a.lo = reinterpret_cast<uint16_t*>(base + l.lo);
  a.ld = s.ld;
  a.out = out; a.out_dtype = out_dtype; a.out_ld = out_rstride; a.out_bstride = out_bstride;
  a.out_vec = out_vec;
  a.status = st;
  a.wait_limit_ns = wait_limit_ns();
  int pairs = 0;
  cudaError_t e = ns_max_pairs(&pairs);
  if (e != cudaSuccess) return cuda_fail(e, "Newton-Schulz occupancy");
  if (pairs > kPairs) pairs = kPairs;
  static_assert(3 * kPairs * 16 <= kNsFlags, "16 flags per pair and phase");
  // as many pairs as the widest phase has units, and enough to read G at 32 KB or so
  // per CTA
  long long most = ((long long)batch * rows * cols + 16383) / 16384;
  for (int k = NS_GRAM; k <= NS_UPDATE; ++k) {
    const Cut cut = ns_cut(a, k, pairs);
    a.bn[k] = cut.bn;
    a.splits[k] = cut.splits;
    a.per[k] = ns_phase_tiles(a, k, cut.bn);
    if (k < NS_UPDATE) a.split_base[k + 1] = a.split_base[k] + (cut.splits > 1 ? cut.splits * batch * a.per[k] : 0);
    const long long units = (long long)batch * a.per[k] * cut.splits;
    if (units > 0x3fffffff) return fail(RA_ERR_INVALID_ARG, "Newton-Schulz batch too large");
    if (units > most) most = units;
  }
  if (most < pairs) pairs = (int)most;
  const int tn = (cols + a.bn[NS_UPDATE] - 1) / a.bn[NS_UPDATE];
  a.group_m = tn < 5 ? (kPairs + tn - 1) / tn : 16;
  const long long xb = (long long)rows * s.ld, gb = (long long)s.m * s.ldm;
  void *A = base + l.a, *B = base + l.b;
  auto xmap = [&](CUtensorMap* m, const void* p, int box_cols, int box_rows) {
    return make_map_3d(m, p, RA_F16, cols, rows, batch, s.ld, xb, box_cols, box_rows);
  };
  auto gmap = [&](CUtensorMap* m, const void* p, int box_cols, int box_rows) {
    return make_map_3d(m, p, RA_F16, s.m, s.m, batch, s.ldm, gb, box_cols, box_rows);
  };
  for (int i = 0; i < 2; ++i)
    if ((rc = xmap(&a.x_k[i], hi[i], 64, 128)) || (rc = xmap(&a.x_kb[i], hi[i], 64, a.bn[NS_GRAM] / 2)) ||
        (rc = xmap(&a.x_mn[i], hi[i], 64, 64)) || (rc = xmap(&a.hi_io[i], hi[i], 64, 32)))
      return rc;
  if ((rc = xmap(&a.lo_io, a.lo, 64, 32)) || (rc = gmap(&a.a_row, A, 64, 128)) ||
      (rc = gmap(&a.a_col, A, 64, a.bn[NS_SQUARE] / 2)) || (rc = gmap(&a.a_mn, A, 64, 64)) ||
      (rc = gmap(&a.a_io, A, 64, 32)) || (rc = gmap(&a.b_row, B, 64, 128)) ||
      (rc = gmap(&a.b_col, B, 64, a.bn[NS_UPDATE] / 2)) || (rc = gmap(&a.b_mn, B, 64, 64)) ||
      (rc = gmap(&a.b_io, B, 64, 32)))
    return rc;
  TimedLaunch tl(RA_KERNEL_PAIR_TC, static_cast<cudaStream_t>(stream));
  e = launch_ns(a, pairs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "Newton-Schulz launch");
}

#pragma GCC visibility pop
}  // extern "C"
