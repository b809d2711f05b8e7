// Internal interface between the C-ABI front end (ra_api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ra.h"

namespace ra {

// Division by a divisor that is fixed for a launch or a work unit, done as a
// multiply and a shift (the invariant-divisor method of Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication", 1994):
// with m = floor(2^40 / d) + 1, floor(n * m / 2^40) = floor(n / d) for all
// 0 <= n < 2^20 and 1 <= d < 2^20, because the excess n * (m - 2^40 / d) / 2^40
// stays below 2^-20 < 1 / d.  Tile and iteration indices stay far below 2^20.
__host__ __device__ inline unsigned long long div_magic(unsigned d) { return (1ull << 40) / d + 1; }
__host__ __device__ inline int div_by(int n, unsigned long long m) {
  return (int)(((unsigned long long)(unsigned)n * m) >> 40);
}

// Layout of a [B, N, H, d] tensor with d contiguous: element (b, n, h, c)
// sits at b * bs + n * rs + h * hs + c (elements).  Packed: rs = H * d,
// hs = d, bs = N * H * d.
struct Lay {
  long long bs, rs, hs;
};
__host__ __device__ inline long long lay_at(const Lay& L, long long b, long long n, long long h) {
  return b * L.bs + n * L.rs + h * L.hs;
}
inline Lay packed_lay(long long N, long long H, long long d) { return Lay{N * H * d, H * d, d}; }

// ---------------------------------------------------------------------------
// fp32 CUDA-core path
// ---------------------------------------------------------------------------
struct SimtFwdArgs {
  const float* q;
  const float* k;
  const float* v;
  int B, Nq, Nkv, Hq, Hkv, d;
  Lay ql, kvl;              // q; k and v
  float scale;
  int causal;
  long long q_off, kv_off;  // block mode: global positions of row 0
  int P, S;                 // ring mode: P hosts of S rows; P == 0 -> block mode
  int striped;              // ring mode, causal: rows in striped order (position l*P + host)
  const int* host_len;      // ring mode, optional: valid rows per host (device, P entries)
  float* o_acc;             // block mode state (read + written)
  float* m_acc;
  float* l_acc;
  void* o_out;              // ring mode outputs (layout ql)
  int o_dtype;
  float* lse;
};

struct SimtBwdArgs {
  const float* q;
  const float* k;
  const float* v;
  const float* dO;
  const float* lse;
  const float* Dvec;  // [B, Hq, N]
  int B, N, Hq, Hkv, d;
  Lay ql, kvl;        // q, dO, dq; k, v, dk, dv
  float scale;
  int causal;
  int P, S;
  int striped;
  const int* host_len;
  void* dq;
  void* dk;
  void* dv;
  int grad_dtype;
};

cudaError_t launch_simt_fwd(const SimtFwdArgs& a, cudaStream_t st);
cudaError_t launch_simt_bwd(const SimtBwdArgs& a, cudaStream_t st);

// ---------------------------------------------------------------------------
// Elementwise / row kernels (any path)
// ---------------------------------------------------------------------------
cudaError_t launch_acc_init(float* o, float* m, float* l, int B, int N, int H, int d,
                            cudaStream_t st);
cudaError_t launch_merge(float* oa, float* ma, float* la, const float* ob,
                         const float* mb, const float* lb, int B, int N, int H, int d,
                         cudaStream_t st);
cudaError_t launch_finalize(const float* o, const float* m, const float* l, void* out,
                            int out_dtype, Lay out_l, float* lse, int B, int N,
                            int H, int d, cudaStream_t st);
// dst (packed fp16 [B, N, H, d]) <- src (dtype, layout src_l; rows 16-byte
// aligned, d % 8 == 0); values beyond the fp16 range set RA_ERR_RANGE in *status.
cudaError_t launch_to_f16(const void* src, int src_dtype, Lay src_l, void* dst,
                          int B, int N, int H, int d, int* status, cudaStream_t st);
// D[b, h, n] = sum_c dO[b, n, h, c] * O[b, n, h, c].  When lse2 is given (the
// tensor-core backward) both come out negated: D[b, h, n] = -sum(...) and
// lse2[b, h, n] = -lse[b, h, n] * log2(e), the terms that kernel adds.
cudaError_t launch_bwd_dot(const void* dO, int do_dtype, const void* o, int o_dtype,
                           Lay ql, float* D, const float* lse, float* lse2, int B,
                           int N, int H, int d, cudaStream_t st);
// out (dtype, layout out_l) <- mul * src (packed fp32 [B, N, H, d])
cudaError_t launch_f32_to(const float* src, void* out, int out_dtype, Lay out_l,
                          int B, int N, int H, int d, float mul, cudaStream_t st);
// Padded rows of a [B, N, H, d] tensor (row l of host i with l >= host_len[i],
// S = N / P rows per host) are set to zero, and lse[b, h, row] to -inf when
// lse is given.
cudaError_t launch_fill_padding(void* t, int dtype, Lay l, int B, int N, int H, int d,
                                int P, const int* host_len, float* lse, cudaStream_t st);
cudaError_t launch_selftest_timeout(unsigned int timeout_us, int* status,
                                    cudaStream_t st);

// Debug record of the tiles the tensor-core kernels bring in (see
// ra_debug_visit_log in ra.h): entries of four uint32, appended through an
// atomic cursor; entries past `capacity` are counted but not stored.
struct VisitLog {
  uint4* entries;
  unsigned int* count;
  unsigned long long capacity;
};

// ---------------------------------------------------------------------------
// tcgen05 tensor-core path (d = 64 or 128, fp16/bf16 operands)
// ---------------------------------------------------------------------------
struct TcFwdArgs {
  // Tensor maps over [B, N, H, d] (dims d, H, N, B), 64-element boxes of 128
  // rows, 128-byte swizzle.  q/k in qk_dtype, v in fp16.
  CUtensorMap tm_q, tm_k, tm_v;
  int qk_bf16;  // 1: q, k are bf16; 0: fp16
  int precise;  // two-term fp16 P in the P V product
  int B, Nq, Nkv, Hq, Hkv, d;
  float scale_log2;  // scale * log2(e)
  int causal;
  long long q_off, kv_off;
  int ring_P, ring_S;  // ring mode when ring_P > 0 (Nq == Nkv == P*S, S % 128 == 0)
  unsigned long long T_m;  // ring mode: div_magic(ring_S / 128)
  int striped;         // ring mode, causal: rows are in striped order (position l*P + host)
  const int* host_len; // ring mode, optional: valid rows per host (device, P entries)
  // outputs
  // cross attention: queries against keys of another length (ring_P 0, causal 0)
  int cross, splits;   // parts of the keys
  int bf16_p;          // P as two bf16 terms, v in bf16
  const int* kv_len;   // optional: keys per batch entry (device)
  int mode;         // 0: finalise, 1: block (read/write state), 2: cross: write the parts' states
  float* o_acc;     // block mode: [B, Nq, Hq, d] fp32
  float* m_acc;     // [B, Hq, Nq] (natural-log units)
  float* l_acc;
  void* o_out;      // ring mode: [B, Nq, Hq, d] in o_dtype, layout ol
  int o_dtype;
  Lay ol;
  float* lse;       // [B, Hq, Nq]
  int* status;
  unsigned long long wait_limit_ns;
  int num_units;    // work units (pairs of 128-row query tiles)
  unsigned int* sched;  // unit counter the CTAs draw from, zero at launch; NULL: CTA c takes units c, c + grid, ...
  VisitLog log;     // debug record of the key/value tiles loaded (off when log.entries is NULL)
};
cudaError_t launch_tc_fwd(TcFwdArgs& a, int num_sms, cudaStream_t st);

struct TcBwdArgs {
  // fp16 operands: q, dO over [B, N, Hq, d]; k, v over [B, N, Hkv, d]
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
  // the fp32 dQ accumulator [B, N, Hq, d]: 32-column boxes of 128 rows,
  // 128-byte swizzle, written by TMA reduce-add
  CUtensorMap tm_dq;
  int B, N, Hq, Hkv, d;
  float scale;
  float scale_log2;
  int causal;
  int precise;  // two-term fp16 dS in the dK product
  int ring_P, ring_S;
  unsigned long long T_m;  // div_magic(ring_S / 128)
  unsigned long long P_m;  // div_magic(ring_P)
  int striped;  // causal, rows in striped order (position l*P + host)
  const int* host_len;  // optional: valid rows per host (device, P entries)
  // cross attention: N query rows, Nkv key rows, lse and Dvec with rows of Np (a multiple
  // of 128, -inf and 0 from N on); units (head, part of the query tiles, key tile)
  int cross, Nkv, Np, q_splits;
  const int* kv_len;    // optional: keys per batch entry (device)
  float* parts;         // q_splits > 1: dK then dV [q_splits][B, Nkv, Hkv, d]
  const int2* range;    // cross_scale's [B, Hkv]: lse is larger by kCrossP, Dvec and dS times powers of two
  int bf16_in;          // of the inputs' type, before the copies
  const float* lse;   // [B, Hq, N]: -LSE * log2(e)
  const float* Dvec;  // [B, Hq, N]: -D
  float* dq_acc;      // packed fp32 [B, N, Hq, d], pre-zeroed, reduce-added
  void* dk;           // [B, N, Hkv, d] in grad_dtype, layout kvl
  void* dv;
  int grad_dtype;
  Lay kvl;
  int* status;
  unsigned long long wait_limit_ns;
  int num_units;
  unsigned int* sched;  // unit counter the CTAs draw from; zero at launch
  VisitLog log;     // debug record of the query tiles loaded (off when log.entries is NULL)
};
cudaError_t launch_tc_bwd(TcBwdArgs& a, int num_sms, cudaStream_t st);

// -------------------------------------------- cross attention
// A few queries (Nq * Hq / Hkv <= kCrossFewRows) on warp-level products: bound by reading
// K and V.  Results, or with splits > cluster the clusters' states.
struct CrossState {   // [splits][B, Nq, Hq, d], [splits][B, Hq, Nq] (natural-log units)
  float *o, *m, *l;
};
constexpr int kCrossFewRows = 32;
constexpr int kCrossP = 12;  // backward: P is held times 2^kCrossP
// Backward: bounds of the norms of the rows of dO (x) and of v (y) that a key head of a batch
// entry meets, as 16 log2 rounded up; kCrossNone: all are zero.
constexpr int kCrossNone = (int)0x80808080;  // what bytes of 0x80 are
struct CrossRangeArgs {
  struct Side {
    const void* x;
    Lay l;
    int H;
    int heads, chunks;  // set by the launch: heads of a block, and blocks that share their rows
  } side[2];            // dO, v
  int bf16, B, Nq, Nkv, Hkv, d;
  const int* kv_len;
  int2* range;  // [B, Hkv], kCrossNone before
  int blocks;   // of dO; set by the launch
};
cudaError_t launch_cross_range(CrossRangeArgs& a, cudaStream_t st);
struct CrossFewArgs {
  const void *q, *k, *v;
  int bf16, B, Nq, Nkv, Hq, Hkv, d;
  Lay ql, kvl, ol;
  float scale_log2;
  const int* kv_len;
  int splits, cluster;  // parts of the keys, and how many of them a cluster joins
  CrossState part;
  void* o;
  int o_dtype;
  float* lse;
};
cudaError_t launch_cross_few(const CrossFewArgs& a, cudaStream_t st);
// o, lse <- the parts' states joined
cudaError_t launch_cross_join(const CrossState& part, int splits, int B, int Nq, int Hq, int d, void* o, int o_dtype,
                              Lay ol, float* lse, cudaStream_t st);
// k16, v16 (packed fp16; NULL: not wanted) <- k, v (16-bit), rows from kv_len[b] on zero;
// values beyond the fp16 range set RA_ERR_RANGE in *status
struct CrossKeysArgs {
  const void *k, *v;
  void *k16, *v16;
  int bf16, B, Nkv, Hkv, d;
  Lay kvl;
  const int* kv_len;
  int* status;
};
cudaError_t launch_cross_keys(const CrossKeysArgs& a, cudaStream_t st);
// what the backward kernel needs of the query side: lse2 = kCrossP - lse log2(e), D = -dO . O
// times its power of two (rows of Np; -inf and 0 where there is no row or it saw no key), fp16 copies of q
// and, times another, of dO (bf16 inputs), dq_acc = 0 and the unit counter; and the key side as above
// where k16 is not NULL
struct CrossRowsArgs {
  const void *q, *dO, *o;
  const float* lse;
  int bf16, o_dtype, B, Nq, Np, Hq, Hkv, d;
  Lay ql;
  const int2* range;
  void *q16, *do16;  // NULL for fp16 inputs
  float *D, *lse2, *dq_acc;
  unsigned int* sched;
  int* status;
};
cudaError_t launch_cross_prepare(const CrossRowsArgs& a, const CrossKeysArgs& keys, cudaStream_t st);
// D (as above) <- -sum_j P_ij dO_i . v_j for the rows of batch entries with up to max_keys keys
struct CrossDotArgs {
  const void *q, *k, *v, *dO;
  const float* lse;
  int bf16, B, Nq, Nkv, Np, Hq, Hkv, d, max_keys;
  Lay ql, kvl;
  float scale_log2;
  const int2* range;
  const int* kv_len;
  float* D;
};
cudaError_t launch_cross_dot(const CrossDotArgs& a, cudaStream_t st);
// dk, dv <- sums of the parts' planes
cudaError_t launch_cross_sum(const float* parts, int splits, int B, int Nkv, int Hkv, int d, void* dk, void* dv, int dtype,
                             Lay kvl, cudaStream_t st);
// dq (dtype, layout) <- dq_acc (packed fp32) times scale, without the head's power of two
cudaError_t launch_cross_dq(const float* dq_acc, float scale, const int2* range, int bf16, int B, int Nq, int Hq, int Hkv, int d,
                            void* dq, int dtype, Lay ql, cudaStream_t st);

// Counts kernel launches (ra_launch_count).
void count_launch(unsigned n = 1);

// Records `msg` as the calling thread's ra_last_error() message; returns code.
int set_error(int code, const char* msg);

// Row-major 16-bit matrix [rows, cols], leading dimension ld (elements):
// tensor map with box (64 columns, box_rows rows), 128-byte swizzle.
int make_map_2d(CUtensorMap* m, const void* base, int is_bf16, long long rows, long long cols,
                long long ld, int box_rows);

// ----------------------------------------------------------------- GEMM
// C[M, N] = epilogue(sum_k A(m, k) B(n, k)) on the tensor cores, 16-bit
// operands, fp32 accumulation.  A is K-major (a row-major [M, K] matrix) or
// MN-major (a row-major [K, M] matrix); B likewise with N.  Tiles 128 x 256.
enum GemmEpi {
  GEMM_STORE = 0,   // c = acc (c_dtype)
  GEMM_GELU = 1,    // c = GELU(acc) (16-bit)
  GEMM_GELU2 = 2,   // c = GELU(acc), c2 = GELU'(acc) (16-bit)
  GEMM_MUL = 3,     // c = acc * aux (16-bit aux and c)
  GEMM_ACC = 4,     // c += acc (fp32)
};
struct GemmArgs {
  CUtensorMap tm_a;   // K-major: box (64, 128); MN-major: box (64, 64)
  CUtensorMap tm_b;   // K-major: box (64, 256); MN-major: box (64, 64)
  int M, N, K;
  int a_mn, b_mn;
  int ab_bf16;        // operand type: bf16 (1) or fp16 (0)
  int epi;
  void* c;            // row-major [M, N], leading dimension ldc
  long long ldc;
  int c_dtype;        // ra_dtype of c
  void* c2;           // GEMM_GELU2: second output, same layout and type as c
  const void* aux;    // GEMM_MUL: row-major [M, N], leading dimension ldc, 16-bit
  // optional second problem of the same kind in the same launch (same K,
  // operand types and epilogue): its tiles follow the first problem's
  int groups;         // 1 or 2
  CUtensorMap tm_a2, tm_b2;
  int M2, N2;
  void* c_g2;
  long long ldc_g2;
  int* status;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_tc_gemm(GemmArgs& a, int num_sms, cudaStream_t st);

// -------------------------------------------- vocabulary cross entropy
// C[M, N] = epilogue(sum_k A(m, k) B(n, k)) on pairs of CTAs; operands K-major or
// MN-major, sizes of any value.  The epilogues:
enum PairEpi {
  PAIR_STATS = 0,    // softmax statistics of each row's columns and the target's logit
  PAIR_DLOGITS = 1,  // gradient of the logits, 16-bit, rounded or as two terms
  PAIR_STORE = 2,    // C, 16-bit or fp32, fp32 optionally added to what is there
};
struct PairProblem {
  // operands: K-major: boxes of 64 x a_rows (A), 64 x bn/2 (B); MN-major: 64 x 64
  CUtensorMap tm_a, tm_b;
  CUtensorMap tm_c;   // output: boxes of 64 x 32 (16-bit) or 32 x 32 (fp32), 128-byte swizzle
  int M, N, K;
  int a_mn, b_mn;
  int fold;           // > 0: A is matrices of `fold` k-slabs each, all multiplied with one B
  int a_rows;         // rows of a K-major A a CTA loads: 128, or all of them (M < 128, multiple of 8)
  int bn;             // tile columns: 128 or 256
  int splits;         // PAIR_STORE, fp32: K is split, split s writes plane s of C
  int group_m;        // tile rows taken together
  // PAIR_STORE
  int c_dtype;
  int c_accumulate;   // fp32: add to C
  const float* c_add; // 16-bit: packed fp32 [M, N] added to the product
};
struct PairArgs {
  PairProblem q[2];   // one launch works on one problem, PAIR_STORE on one or two
  int problems;
  int ab_bf16;
  int epi;
  int two_terms;             // PAIR_DLOGITS: matrix 1 of tm_c gets what rounding takes from matrix 0
  int* status;
  unsigned long long wait_limit_ns;
  const long long* targets;  // [M]
  long long ignore;          // target of rows without loss
  long long vocab;           // V
  long long col_off;         // vocabulary entry of column 0
  const float* lse;          // [M]
  const float* grad;         // [M]: gradient of each row's loss
  const float* scale;        // {2^k, 2^-k} on the device, or NULL: {1, 1}
  float2* stats;             // [column parts][M]: (max, sum of exponentials) of bn / 2 columns
  float* target_logit;       // [M]
};
cudaError_t launch_xent_pair(const PairArgs& a, int num_sms, cudaStream_t st);
// The logits of few tokens: statistics (d NULL; a part per block), or the gradient of V
// entries from col_off on.
struct XentFewArgs {
  const void *x, *w;
  int bf16, T, D, V, blocks;
  long long xs, ws;
  const long long* targets;
  long long ignore, vocab, col_off;
  float2* stats;
  float* target_logit;
  const float *lse, *grad, *scale;  // as in PairArgs
  void* d;                          // [2 T] rows at ld elements: rounded, and the rest
  long long ld;
};
// A single token (D kXentTokenSmem / 4 or less), on the CUDA cores.
constexpr int kXentTokenSmem = 32768;
cudaError_t launch_xent_token(const XentFewArgs& a, cudaStream_t st);
bool xent_few(long long T, int D);  // whether the next kernel takes such a call
cudaError_t launch_xent_few(const XentFewArgs& a, cudaStream_t st);
// loss and lse from the column parts' statistics; a target outside [0, V) that is
// not `ignore` gives loss = NaN and RA_ERR_INVALID_ARG in *status.
cudaError_t launch_xent_finish(const float2* stats, int parts, const float* target_logit, const long long* targets,
                               long long ignore, long long V, long long T, float* loss, float* lse, int* status,
                               cudaStream_t st);
// scale = {2^k, 2^-k} with 2^k max |grad| in [2^13, 2^14) over the rows with a loss, infinities
// left out; k at most 126 (max |grad| from 2^-113 on).
cudaError_t launch_xent_scale(const float* grad, const long long* targets, long long ignore, long long V, long long T,
                              float* scale, cudaStream_t st);
// out (dtype) <- the sum of `planes` fp32 planes of n elements each (n a multiple of 8)
cudaError_t launch_sum_planes(const float* planes, int count, long long n, void* out, int dtype, cudaStream_t st);

// -------------------------------------------- rotary positions, norms of heads
struct RotarySide {  // queries, or keys
  const void* x;
  const void* dy;    // backward
  void* y;           // result, or gradient of x
  const void* w;     // weights of the norm [d], or NULL: ones
  Lay xl, dyl, yl;
  int H;             // 0: there are none
};
struct RotaryArgs {
  RotarySide side[2];
  long long tokens;  // B N
  int N, d, rot;
  const double* freq;          // [rot / 2], radians per position
  const long long* positions;  // [B or 1, N], or NULL: pos_off + row
  long long pos_bstride, pos_off;
  int striped, P, S;           // row i S + l holds position l P + i
  float amplitude, eps;
  int w_dtype;
  float* dw_parts;             // [2][blocks][d], backward
  // set by the launch
  int flat;                   // every tensor's token t is at t rs
  int G, heads, tile, parts;  // lanes of a row; heads and tokens of a warp's rows; parts of the heads
  long long units;            // tiles of tokens x parts
};
constexpr int kRotMaxHead = 256;
constexpr int kRotParts = 608;  // blocks of the backward kernel
cudaError_t launch_rotary(RotaryArgs& a, int interleaved, int dtype, int out_dtype, int norm, int grad, int sms,
                          cudaStream_t st);
cudaError_t launch_norm_rotary_bwd(RotaryArgs& a, int interleaved, int dtype, int g_dtype, int grad_dtype, float* dwq,
                                   float* dwk, int sms, cudaStream_t st);
int rot_exchange(int rot, int interleaved);
void rot_units(RotaryArgs& a, int sms);

// -------------------------------------------- norm and clipping of many tensors
constexpr int kClipFew = 48, kClipSome = 320, kClipMany = 1024;  // tensors a launch takes
constexpr int kClipParts = 608;                 // blocks of a launch
template <int MAX>
struct GradList {
  int count, chunk;        // tensors; elements of a chunk, a multiple of 8
  const void* in[MAX];
  void* out[MAX];
  long long n[MAX];        // at least 1
  int first[MAX + 1];      // a tensor's first chunk
  unsigned char types[MAX];  // dtype of in + 16 times that of out
};
template <int MAX>
cudaError_t launch_grad_squares(const GradList<MAX>& a, double* parts, int* used, int sms, cudaStream_t st);
template <int MAX>
cudaError_t launch_grad_scale(const GradList<MAX>& a, const double* parts, int count, float max_norm, float eps,
                              float* norm, const float2* factor, int sms, cudaStream_t st);
// norm, and the factor where it is not NULL
cudaError_t launch_grad_norm(const double* parts, int count, float max_norm, float eps, float* norm, float2* factor,
                             cudaStream_t st);

// -------------------------------------------- Newton-Schulz
struct NsInput {
  const void* g;
  int dtype, batch, rows, cols;
  long long ld, bstride;
  int vec;  // rows start on 16-byte boundaries
};
constexpr int kNsParts = 304;     // partial sums of G's squares per batch entry
constexpr int kNsFlags = 3 * 16 * 128;  // 16 per unit of split tiles, three phases
constexpr int kNsWords = 64 + kNsFlags;  // mark of a launch that gave up, flags; counts per matrix follow
enum NsPhase { NS_GRAM = 0, NS_SQUARE = 1, NS_UPDATE = 2 };
struct NsArgs {
  // operands of X's two buffers: K-major boxes for A and for B, MN-major boxes
  CUtensorMap x_k[2], x_kb[2], x_mn[2];
  // A' and B' as A (boxes of 64 x 128), as B (64 x bn/2) and MN-major (64 x 64)
  CUtensorMap a_row, a_col, a_mn, b_row, b_col, b_mn;
  // what the epilogues read and write: boxes of 64 x 32, 128-byte swizzle
  CUtensorMap hi_io[2], lo_io, a_io, b_io;
  NsInput in;
  int batch, rows, cols, m, tall;  // m: the smaller side; tall: rows > cols
  int steps;
  int bn[3];      // tile columns of each phase
  int per[3];     // tiles per matrix of each phase
  int splits[3];  // parts of K of each phase; above 1 only with a pair for every part
  int split_base[3];  // units of split tiles in the phases before
  int group_m;    // NS_UPDATE: tile rows taken together
  float ca, cb, cc;                                            // coefficients
  float sx, sa, eps, alpha_mul;                                // scales of X and A'; alpha = alpha_mul sum x^2
  float gram_acc, square_acc, square_lin, update_acc, out_mul;  // factors of accumulators, of A', of the result
  float* parts;
  int num_parts;
  float* sums[2];  // [batch][16 per unit], read by a step and written for the next one
  long long sums_ld;
  uint16_t *hi0, *lo;
  long long ld;    // X's padded rows
  void* out;
  int out_dtype, out_vec;
  long long out_ld, out_bstride;
  unsigned int* words;  // zeroed at first: the mark of a launch that gave up, the flags, the counts
  unsigned int* counts; // per matrix: warps that have scaled it and halves of tiles written
  int* shifts;          // per matrix: X is held times 2^shift at first
  float growth;         // log2 of the most by which a step lets X grow: what the shift falls by
  unsigned int* flags;  // per warp of a split: the last phase whose sums for the others it has written
  float* partials;      // sums that splits leave each other, [unit][CTA][warp][128 columns][32 rows]
  int* status;
  unsigned long long wait_limit_ns;
};
// Matrices whose smaller side m is at most 128: a cluster of CTAs per matrix (a power of
// two, at most 16), each with a slice of 64, 128 or 256 of the n columns of X (rows of a
// tall gradient).
struct NsSmallArgs {
  NsInput in;
  int m, n, tall, steps;
  float ca, cb, cc;
  float sx, sa, sb, inv_sb, eps, alpha_mul;
  float gram_acc, square_acc, square_lin, out_mul;
  void* out;
  int out_dtype, out_vec;
  long long out_ld, out_bstride;
  int* status;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_ns_small(const NsSmallArgs& a, int slice, int cluster, cudaStream_t st);
// Pairs of CTAs that can run at the same time on the current device.
cudaError_t ns_max_pairs(int* pairs);
int ns_phase_tiles(const NsArgs& a, int kind, int bn);  // per batch entry
cudaError_t launch_ns(NsArgs& a, int pairs, cudaStream_t st);

}  // namespace ra
