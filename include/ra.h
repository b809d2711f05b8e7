/*
 * ra.h -- C ABI of the blockwise exact attention library (libra.so), sm_103a.
 *
 * Exact softmax attention computed blockwise, as in "Ring Attention with
 * Blockwise Transformers for Near-Infinite Context" (arXiv 2310.01889,
 * Abstract: blockwise self-attention over key/value blocks that travel
 * around a ring of hosts, with no approximation).  On one GPU the ring is
 * emulated: P virtual hosts own contiguous row blocks of Q, K, V in device
 * memory and host i computes against key/value block (i - step) mod P at
 * each step ("Ring Attention: Train 1M Tokens on 8GB GPUs in 2026", section
 * "Ring Attention: Partition Sequence Length, Not Batch").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout.  q, k, v, o, dO, dq, dk, dv are [B, N, H, d] with d contiguous; by
 *   default packed with heads at stride d (the pages' [seq, heads, head_dim]
 *   layout with a batch axis; "Building Ring Attention in PyTorch: The
 *   200-Line Version"), and any batch, row and head strides through ra_shape
 *   (see there), so [B, H, N, d] tensors and slices of a fused projection
 *   need no copy.  Row blocks of a larger tensor are plain pointer offsets.
 *   The fp32 running state is o_acc [B, N_q, Hq, d] (packed) and m_acc,
 *   l_acc, lse [B, Hq, N_q] (packed).
 * Scores.  s_ij = scale * q_i . k_j; scale is usually d^-0.5 (same section).
 *   With RA_CAUSAL in `flags` key j is visible to query i iff
 *   kv_pos(j) <= q_pos(i), positions being global row indices (q_off /
 *   kv_off added for blocks).
 * State.  (m, l, o) is the triple the pages carry between ring steps
 *   (max_score, exp_sum, weighted_output; "Gotchas and Failure Modes"):
 *   l = sum_j exp(s_j - m), o = sum_j exp(s_j - m) v_j, m in natural-log
 *   units of the scaled scores.  m is a reference point, not necessarily
 *   the exact row maximum (kernels may defer rescaling while the maximum
 *   grows by less than 8 in log2 units); the represented quantities o/l and
 *   m + log(l) are what the state means.  A row that has seen no key has
 *   m = -inf, l = 0, o = 0.
 * Grouped heads.  Hq % Hkv == 0; query head h reads key/value head
 *   h / (Hq / Hkv).
 * Streams.  `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream).  Every call only enqueues work and returns; it holds no pointer
 *   after it returns and allocates no device memory: the caller owns every
 *   buffer, including the workspace.  A call's work (kernels and the
 *   cudaMemsetAsync that zeroes its workspace's counters and accumulators)
 *   all goes to `stream`, so calls can be captured into a CUDA graph and
 *   replayed, provided one call has run on the device beforehand (the first
 *   call looks up the library's device status word).
 * Errors.  The return value reports argument validation and launch errors
 *   (ra_status).  Errors found on the device (a value out of fp16 range in a
 *   bf16 -> fp16 operand copy, a bounded wait that ran out) are recorded in a
 *   device status word; ra_sync_status() synchronises the stream and returns
 *   and clears it.  ra_last_error() gives a message for the last failure on
 *   the calling thread.
 * Precision.  RA_F32 inputs run in fp32 CUDA-core arithmetic (exact fp32
 *   products and sums).  RA_BF16 / RA_F16 inputs with d in {64, 128} run on
 *   the tcgen05 tensor cores with fp32 accumulation; the probabilities P
 *   (and dS in the backward pass) are rounded to fp16 for the second
 *   product, and bf16 operands of those products are copied to fp16 in the
 *   workspace first (exact for |x| in [2^-14, 65504]; larger values set
 *   RA_ERR_RANGE in the status word; smaller ones become fp16 subnormals,
 *   rounded to a multiple of 2^-24 without any status error).
 * Requirements.  Pointers 16-byte aligned; for ra_ring_fwd / ra_ring_bwd on
 *   tensor cores the host block N/P is a multiple of 128 rows; violations
 *   return RA_ERR_INVALID_ARG or RA_ERR_UNSUPPORTED.  Nothing falls back to
 *   another implementation.
 */
#ifndef RA_H_
#define RA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RA_F32 = 0, RA_BF16 = 1, RA_F16 = 2 } ra_dtype;

/* Bits of the `flags` argument.
 * RA_CAUSAL   key j is visible to query i only if kv_pos(j) <= q_pos(i).
 * RA_PRECISE  16-bit inputs: the operand rounded to fp16 for the second
 *             product (P in P V; dS in dS^T Q) is carried as two fp16 terms
 *             hi + lo, taking its rounding from 2^-12 to about 2^-24
 *             relative at the cost of one more MMA per tile.  Needed when
 *             logits are large and values have outliers (e.g. |q| ~ 4 N(0,1)
 *             with +-50 entries in V); ignored for RA_F32.
 * RA_STRIPED  ring entry points with RA_CAUSAL: the rows of q, k, v, o, dO,
 *             dq, dk, dv, lse are in striped order -- host i's local row l
 *             (tensor row i*S + l) holds sequence position l*P + i -- so every
 *             host has the same share of the causal triangle (load-balanced
 *             ordering; "Striped Attention" is named beside Ring Attention on
 *             "Ring Attention: Train 1M Tokens on 8GB GPUs in 2026", section
 *             "How Does This Compare to Other Long-Context Methods?").  The
 *             ring order is unchanged; every host visits every block, and in a
 *             (query host i, key host j) pair local key row lk is visible to
 *             local query row lq iff lk < lq, or lk == lq and j <= i.  In the
 *             backward pass a key tile's gradients go round the ring once per
 *             local query tile they meet (each lap in ring order), which keeps
 *             the query tiles that concurrent work units read in cache; only
 *             rounding depends on that order.  Ignored without RA_CAUSAL.
 *             Also taken by the rotary entry points, for rows in that order.
 * RA_INTERLEAVED  rotary entry points: pairs are columns (2i, 2i + 1). */
enum { RA_CAUSAL = 1, RA_PRECISE = 2, RA_STRIPED = 4, RA_INTERLEAVED = 8 };

typedef enum {
  RA_OK = 0,
  RA_ERR_INVALID_ARG = 1, /* bad pointer, size, stride or alignment */
  RA_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. d = 96) */
  RA_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
  RA_ERR_RANGE = 4,       /* device: operand outside fp16 range */
  RA_ERR_TIMEOUT = 5      /* device: a bounded wait gave up */
} ra_status;

/* Sizes and strides.  The q group (q, o, dO, dq) and the kv group (k, v, dk,
 * dv) each share one layout: element (b, n, h, c) of a q-group tensor sits at
 * b * q_bstride + n * q_rstride + h * q_hstride + c (elements; d is always
 * contiguous), and likewise for the kv group.  A stride of 0 takes its packed
 * default: row stride H*d, head stride d, batch stride the extent of one
 * batch ((N-1)*rstride + (H-1)*hstride + d).  So zeroed strides describe the
 * pages' [seq, heads, head_dim] rows with a batch axis, and
 *   [B, H, N, d] tensors:  rstride = d, hstride = N*d, bstride = H*N*d;
 *   a slice of a fused [B, N, 3, H, d] projection: rstride = 3*H*d,
 *   hstride = d, bstride = N*3*H*d (outputs of the group need the same
 *   strides).
 * Strides must not make two (n, h) rows overlap, nor one batch overlap the
 * next; for 16-bit inputs on the tensor cores every stride is a multiple of 8
 * elements (16 bytes).  The fp32 running state o_acc/m_acc/l_acc and lse are
 * always packed.  Violations return RA_ERR_INVALID_ARG. */
typedef struct {
  int B;                /* batch */
  int N_q;              /* query rows covered by the call */
  int N_kv;             /* key/value rows covered by the call */
  int Hq;               /* query heads */
  int Hkv;              /* key/value heads (divides Hq) */
  int d;                /* head dimension */
  long long q_bstride;  /* elements between batches of q/o/dO/dq; 0 = packed */
  long long kv_bstride; /* elements between batches of k/v/dk/dv; 0 = packed */
  long long q_rstride;  /* elements between rows (positions) of q/o/dO/dq; 0 = Hq*d */
  long long q_hstride;  /* elements between heads of q/o/dO/dq; 0 = d */
  long long kv_rstride; /* elements between rows of k/v/dk/dv; 0 = Hkv*d */
  long long kv_hstride; /* elements between heads of k/v/dk/dv; 0 = d */
} ra_shape;

/* Set the running state to "nothing seen": o_acc = 0, m_acc = -inf,
 * l_acc = 0 (the ring loop's zero accumulators, "Building Ring Attention in
 * PyTorch: The 200-Line Version").  Uses shape.B, N_q, Hq, d. */
int ra_acc_init(float* o_acc, float* m_acc, float* l_acc, ra_shape shape,
                void* stream);

/* One ring step: fold the scores of a query block against one key/value
 * block into the running state (o_acc, m_acc, l_acc) with the online-softmax
 * rescale ("Gotchas and Failure Modes": keep (max, exp_sum,
 * weighted_output) and rescale on merge; online normaliser of Milakov and
 * Gimelshein cited by the arXiv 2310.01889 page).
 *   q      [B, N_q, Hq, d]  query block, global row position q_off + r
 *   k_blk, v_blk [B, N_kv, Hkv, d]  key/value block at positions kv_off + c
 *   dtype  type of q, k_blk, v_blk
 *   o_acc, m_acc, l_acc  state of the query block, read and updated
 *   flags  RA_CAUSAL / RA_PRECISE; key/value tiles wholly after a query
 *          tile are skipped, rows left with no visible key keep their state
 *   scale  score scale (> 0)
 *   workspace, ws_bytes  at least ra_block_fwd_workspace_bytes(dtype, shape)
 * Any N_q, N_kv >= 1 (ragged tiles are masked); tensor-core dtypes need
 * d in {64, 128}, RA_F32 d in {32, 64, 128}. */
int ra_block_fwd(const void* q, const void* k_blk, const void* v_blk,
                 ra_dtype dtype, float* o_acc, float* m_acc, float* l_acc,
                 ra_shape shape, long long q_off, long long kv_off, int flags,
                 float scale, void* workspace, size_t ws_bytes, void* stream);
size_t ra_block_fwd_workspace_bytes(ra_dtype dtype, ra_shape shape);

/* a <- merge(a, b) for two states of the same query rows: m = max(m_a, m_b),
 * l = l_a e^{m_a - m} + l_b e^{m_b - m}, o likewise; a side with m = -inf
 * has weight 0 ("Gotchas and Failure Modes").  Uses shape.B, N_q, Hq, d. */
int ra_merge(float* o_a, float* m_a, float* l_a, const float* o_b,
             const float* m_b, const float* l_b, ra_shape shape, void* stream);

/* Final normalisation of the state: O = o / l ("output / softmax_denom" at
 * the end of the ring loop) written as o_dtype, and lse = m + ln l (natural
 * log, saved for the backward pass).  Rows with l = 0 give O = 0 and
 * lse = -inf.  o_out has the q layout of `shape` (q_bstride honoured). */
int ra_finalize(const float* o_acc, const float* m_acc, const float* l_acc,
                void* o_out, ra_dtype o_dtype, float* lse, ra_shape shape,
                void* stream);

/* Whole forward ring in one call: P virtual hosts of S = N/P rows; host i
 * visits key/value blocks (i - s) mod P for s = 0..P-1, skipping blocks
 * wholly in its causal future, merges each block into its state and
 * normalises at the end ("Ring Attention: Partition Sequence Length, Not
 * Batch"; the loop of "Building Ring Attention in PyTorch: The 200-Line
 * Version" with the rescaled merge).
 *   q [B, N, Hq, d], k, v [B, N, Hkv, d] with N = shape.N_q = shape.N_kv
 *   o [B, N, Hq, d] in o_dtype; lse [B, Hq, N] fp32 (natural log)
 *   workspace: device memory, 256-byte aligned, at least
 *   ra_ring_fwd_workspace_bytes() bytes: for bf16/fp16 a 256-byte counter
 *   from which the kernel's CTAs draw their work (zeroed by each call), for
 *   bf16 also the fp16 copy of V; fp32 needs none (NULL allowed).  It must
 *   not be in use by work that overlaps the call on the GPU.
 * Tensor-core dtypes need S a multiple of 128. */
int ra_ring_fwd(const void* q, const void* k, const void* v, ra_dtype dtype,
                ra_shape shape, int P, int flags, float scale, void* o,
                ra_dtype o_dtype, float* lse, void* workspace, size_t ws_bytes,
                void* stream);
size_t ra_ring_fwd_workspace_bytes(ra_dtype dtype, ra_shape shape, int P);

/* Backward ring: gradients of L = sum(O * dO).  Probabilities are recomputed
 * from the saved lse (activation recomputation; "Building Ring Attention in
 * PyTorch" notes production code needs gradient checkpointing), and the
 * gradients of each key/value block travel with it around the ring: block
 * j visits hosts (j + s) mod P ("Gotchas and Failure Modes": gradients flow
 * backwards through the ring).
 *   D_i = dO_i . O_i; P_ij = exp(s_ij - lse_i); dV_j = sum_i P_ij dO_i;
 *   dS_ij = P_ij (dO_i . v_j - D_i); dQ_i = scale sum_j dS_ij k_j;
 *   dK_j = scale sum_i dS_ij q_i (summed over the query heads of a group).
 *   o in o_dtype, dO in dtype, lse from ra_ring_fwd; dq [B,N,Hq,d],
 *   dk, dv [B,N,Hkv,d] written in grad_dtype (fully overwritten).
 *   workspace: device memory, 256-byte aligned, at least
 *   ra_ring_bwd_workspace_bytes() bytes: D and LSE*log2(e) per row, for
 *   16-bit dtypes the fp32 dQ accumulator and the counter the kernel's CTAs
 *   draw their work from (both zeroed by each call), and for bf16 the fp16
 *   copies of q, k, v, dO.  It must not be in use by work that overlaps the
 *   call on the GPU. */
int ra_ring_bwd(const void* q, const void* k, const void* v, const void* o,
                ra_dtype o_dtype, const void* dO, const float* lse,
                ra_dtype dtype, ra_shape shape, int P, int flags, float scale,
                void* dq, void* dk, void* dv, ra_dtype grad_dtype,
                void* workspace, size_t ws_bytes, void* stream);
size_t ra_ring_bwd_workspace_bytes(ra_dtype dtype, ra_dtype grad_dtype,
                                   ra_shape shape, int P);

/* ra_ring_fwd for callers that cannot allocate device memory: code that runs
 * where cudaMalloc is not available or not allowed (inside a host callback
 * or a custom allocator's own hooks, under a framework that owns every
 * device allocation, or with a fixed memory budget set at start-up) cannot
 * provide the workspace ra_ring_fwd asks for.  This entry point takes the
 * same arguments minus the workspace and uses a scratch buffer that is part
 * of the library itself: a device array of 32 MiB + 256 bytes per GPU that
 * loads the library, held until the process exits.  It allocates nothing.  The pages
 * describe no counterpart; it is a packaging of the same computation.
 *   Limit: shapes whose ra_ring_fwd_workspace_bytes() exceeds that size
 *   (the 256-byte work counter plus, for bf16 inputs, the fp16 copy of V,
 *   B*N*Hkv*d*2 bytes, at most 32 MiB) are rejected with RA_ERR_INVALID_ARG;
 *   fp16 inputs use only the counter, fp32 inputs no scratch.
 *   When the memory is taken: the array sits in a device module of its own
 *   (no kernel shares it).  Under CUDA's lazy module loading (the default
 *   since CUDA 12.2) a device reserves the 32 MiB at this entry point's
 *   first call there, when its address is looked up; with eager loading
 *   (CUDA_MODULE_LOADING=EAGER) every device the process creates a context
 *   on reserves them as soon as the library is loaded, whether or not this
 *   entry point is ever called.
 *   The first call on each device looks up the buffer's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.
 *   All calls share the one buffer per device and it keeps whatever the last
 *   call left there (each call zeroes the counter and overwrites the part it
 *   uses).  Calls whose work overlaps on the GPU (different streams,
 *   or threads without ordering between them) race on it. */
int ra_ring_fwd_noalloc(const void* q, const void* k, const void* v, ra_dtype dtype,
                        ra_shape shape, int P, int flags, float scale, void* o,
                        ra_dtype o_dtype, float* lse, void* stream);

/* Ring forward / backward with variable per-host lengths ("FAQ" of "Ring
 * Attention: Train 1M Tokens on 8GB GPUs in 2026": instead of computing on
 * padding, each host tracks which of its positions are valid and masks the
 * scores).  host_len is a device array of P int32: host i's first
 * host_len[i] rows (of S = N/P) hold its tokens, the rest is padding (values
 * are clamped to [0, S]).  The sequence is the valid rows in order, so a
 * causal mask keeps its block structure; padded keys are never visible,
 * padded query rows give O = 0, LSE = -inf, and padded rows get zero dQ, dK,
 * dV.  Key/value tiles or query tiles wholly in padding are skipped.  Other
 * arguments as in ra_ring_fwd / ra_ring_bwd; RA_STRIPED is not accepted. */
int ra_ring_fwd_varlen(const void* q, const void* k, const void* v, ra_dtype dtype,
                       ra_shape shape, int P, const int* host_len, int flags, float scale,
                       void* o, ra_dtype o_dtype, float* lse, void* workspace,
                       size_t ws_bytes, void* stream);
int ra_ring_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                       ra_dtype o_dtype, const void* dO, const float* lse, ra_dtype dtype,
                       ra_shape shape, int P, const int* host_len, int flags, float scale,
                       void* dq, void* dk, void* dv, ra_dtype grad_dtype, void* workspace,
                       size_t ws_bytes, void* stream);

/* One forward + backward step with the tensors in HOST memory: the work of
 * ra_ring_fwd followed by ra_ring_bwd, with the uploads and downloads it
 * needs.  The pages keep every block resident on its host and only move KV
 * between hosts; this call is for callers whose batches live in host memory
 * (a data loader, a CPU-side training loop).
 *   Inputs q, dO [B,N,Hq,d] and k, v [B,N,Hkv,d] in dtype; outputs o (o_dtype),
 *   lse [B,Hq,N] fp32 (packed), dq, dk, dv (grad_dtype); batch strides from
 *   `shape` apply to the host buffers.  All ten pointers are host pointers.
 *   workspace: device memory, 256-byte aligned, at least
 *   ra_ring_step_host_workspace_bytes() bytes; it holds the device copies and
 *   the forward and backward workspaces.
 *   Order: on `stream`, q, k, v go up, the forward runs, the backward runs,
 *   dq, dk, dv come down.  dO goes up on a library-owned side stream while the
 *   forward runs, and o and lse come down on a second one while the backward
 *   runs; both are joined back into `stream` with events, so the outputs are
 *   complete once `stream` has completed.  Pinned host memory (cudaHostAlloc,
 *   cudaHostRegister) makes every copy asynchronous; pageable memory works,
 *   but the copies then block the calling thread.  Two calls on two streams
 *   with two workspaces overlap one step's copies with the other's kernels.
 *   The workspace must not be in use by work that is not ordered before this
 *   call on `stream`.  The side streams are created on the first call on
 *   each device (make that call before any stream capture).
 *   Errors: everything ra_ring_fwd or ra_ring_bwd would reject is rejected
 *   before anything is enqueued; flags as for ra_ring_fwd. */
int ra_ring_step_host(const void* q, const void* k, const void* v, const void* dO,
                      ra_dtype dtype, ra_shape shape, int P, int flags, float scale,
                      void* o, ra_dtype o_dtype, float* lse, void* dq, void* dk, void* dv,
                      ra_dtype grad_dtype, void* workspace, size_t ws_bytes, void* stream);
size_t ra_ring_step_host_workspace_bytes(ra_dtype dtype, ra_dtype o_dtype,
                                         ra_dtype grad_dtype, ra_shape shape, int P);

/* Blockwise feed-forward layer ("Ring Attention with Blockwise Transformers
 * for Near-Infinite Context", Abstract: self-attention and the feedforward
 * network are both computed blockwise).  The layer is the Transformer's
 * position-wise feedforward
 *     y = GELU(x W1^T) W2^T,   GELU(u) = u Phi(u)  (exact, erf form),
 * computed one block of `block` tokens at a time so that only one block's
 * hidden activations [block, d_hidden] exist at once; the result is the same
 * as the unblocked layer.
 *   x, y [T, d_model] row-major (tokens of all batches); W1 [d_hidden, d_model],
 *   W2 [d_model, d_hidden] (output x input); x, W1, W2 (and dy) in `dtype`
 *   (RA_BF16 or RA_F16), y in y_dtype; fp32 accumulation on the tensor cores.
 *   Sizes: d_model and d_hidden multiples of 256, T and block multiples of 128
 *   (the last block may be shorter); else RA_ERR_UNSUPPORTED.
 *   workspace: device memory of ra_ffn_workspace_bytes() bytes (backward != 0
 *   for ra_ffn_bwd), 16-byte aligned; it holds the block's hidden activations.
 *   Ownership and errors as for ra_ring_fwd. */
size_t ra_ffn_workspace_bytes(ra_dtype dtype, long long T, int d_model, int d_hidden,
                              int block, int backward);
int ra_ffn_fwd(const void* x, const void* w1, const void* w2, ra_dtype dtype, long long T,
               int d_model, int d_hidden, int block, void* y, ra_dtype y_dtype,
               void* workspace, size_t ws_bytes, void* stream);

/* Backward of the blockwise feed-forward layer: gradients of L = sum(y * dy).
 * Each block recomputes its hidden activations h = x W1^T (no activation is
 * kept from the forward), then
 *     dH = (dy W2) * GELU'(h),  dx = dH W1,  dW2 += dy^T GELU(h),  dW1 += dH^T x.
 *   dx [T, d_model] in dx_dtype (fully overwritten); dw1 [d_hidden, d_model] and
 *   dw2 [d_model, d_hidden] fp32, zeroed by the call and summed over blocks.
 *   GELU(h), GELU'(h) and dH are rounded to `dtype` before they enter a
 *   product (they are tensor-core operands). */
int ra_ffn_bwd(const void* x, const void* w1, const void* w2, const void* dy, ra_dtype dtype,
               long long T, int d_model, int d_hidden, int block, void* dx, ra_dtype dx_dtype,
               float* dw1, float* dw2, void* workspace, size_t ws_bytes, void* stream);

/* Softmax cross entropy of a large vocabulary, the loss at the head of a model:
 *     z_tv = x_t . w_v,   lse_t = ln sum_v e^{z_tv},   loss_t = lse_t - z_{t, y_t}
 * without the logits z ever being held: the forward keeps, per token, a (max,
 * sum) pair for each tile of the vocabulary; the backward recomputes the logits
 * of `block` vocabulary entries at a time, so that only one block's gradient
 * [T, block] exists at once (the vocabulary's counterpart of the feed-forward
 * layer's blocks of tokens).
 *   x [T, D] hidden states (tokens of all batches), w [V, D] the vocabulary's
 *   weights, both in `dtype` (RA_BF16 or RA_F16), rows at x_rstride / w_rstride
 *   elements (0 = D; multiples of 8); targets [T] 64-bit integers.  D is a multiple
 *   of 8; T, V and block are of any size >= 1 (blocks that are multiples of 256 fill
 *   the tiles; a block whose gradient takes less than 256 MB is widened to that).
 *   A token whose target equals ignore_index has loss 0 and no gradient (its lse is
 *   still written, and its x, multiplied by exact zeros in dw, has to be finite).  Any
 *   other target outside [0, V) gives loss NaN, no gradient, and RA_ERR_INVALID_ARG in
 *   the status word.
 *   loss, lse [T] fp32.  Products accumulate in fp32; the softmax's maxima and sums
 *   are fp32.  +inf and NaN among the logits give NaN; a logit of -inf is an entry of
 *   probability zero; a row whose logits are all -inf has lse = -inf and loss NaN.
 *   workspace: device memory, 256-byte aligned, of the size given (about T V / 8
 *   bytes for the forward; 2 T block bytes (4 for up to 64 tokens), 4 T D where dx is
 *   16-bit and there is more than one block, and up to 20 MB each for dx and dw where
 *   their products are split, for the backward).  It must not be in use by work that overlaps the call on the
 *   GPU.  Outputs overlap neither each other nor the inputs or the workspace. */
size_t ra_xent_fwd_workspace_bytes(ra_dtype dtype, long long T, int D, int V);
int ra_xent_fwd(const void* x, const void* w, ra_dtype dtype, long long T, int D, int V,
                long long x_rstride, long long w_rstride, const long long* targets,
                long long ignore_index, float* loss, float* lse, void* workspace, size_t ws_bytes,
                void* stream);

/* Backward of ra_xent_fwd: gradients of L = sum_t dloss_t loss_t,
 *     d_tv = dloss_t (e^{z_tv - lse_t} - [v = y_t]),   dx = d W,   dW = d^T x.
 *   lse from ra_xent_fwd of the same x, w, targets; dloss [T] fp32 (1 / T for a mean;
 *   values at ignored tokens are not used).
 *   dx [T, D] in dx_dtype and dw [V, D] in dw_dtype, packed, fully overwritten.  d is
 *   rounded to `dtype` before the two products (it is a tensor-core operand: by up to
 *   2^-8 relative for bf16, 2^-11 for fp16, whose values are brought into range by a power
 *   of two from the largest finite |dloss|, 2^-113 at least), and kept as two such terms
 *   for up to 64 tokens, where no sum averages its roundings out.  The logits are those of
 *   the forward bit for bit, so that tokens the model is sure of keep their gradients.  The
 *   sums, over blocks too, are fp32; the tensor core's round towards zero, which over
 *   131072 tokens took up to 9e-5 of dw (x of one sign; 2e-5 otherwise).  The results do
 *   not vary from run to run, nor dx with the type of dw or dw with that of dx. */
size_t ra_xent_bwd_workspace_bytes(ra_dtype dtype, ra_dtype dx_dtype, long long T, int D, int V,
                                   int block);
int ra_xent_bwd(const void* x, const void* w, ra_dtype dtype, long long T, int D, int V,
                long long x_rstride, long long w_rstride, const long long* targets,
                long long ignore_index, const float* lse, const float* dloss, int block, void* dx,
                ra_dtype dx_dtype, void* dw, ra_dtype dw_dtype, void* workspace, size_t ws_bytes,
                void* stream);

/* Orthogonalises a weight gradient by Newton-Schulz products, as optimisers do that
 * make the update of a hidden layer's matrix orthogonal (the dW1 and dW2 of
 * ra_ffn_bwd, for instance):
 *     X = G / (|G|_F + eps);   `steps` times:  A = X X^T (X^T X where rows > cols),
 *     X <- a X + (b A + c A^2) X
 * with (a, b, c) = coeffs[0..2], read on the host; (3.4445, -4.7750, 2.0315) and five
 * steps bring every singular value that is not tiny near 1.  (The iteration: Kovarik 1970,
 * Bjorck and Bowie 1971; these coefficients: K. Jordan et al., "Muon: An optimizer for
 * hidden layers in neural networks", 2024.)
 *   g [batch, rows, cols] in any dtype, out [batch, rows, cols] in any dtype; rows and
 *   matrices at the strides given (elements, 0 = packed): matrices one after the other, or
 *   rows of all of them between two rows of one ([rows, batch, cols]).  out may be g
 *   itself where dtype and strides agree.  Sizes of any value up to 65536; each matrix of
 *   the batch is orthogonalised by itself.
 *   The products run on the tensor cores with fp16 operands (held times powers of two
 *   that follow from the size and the coefficients, so that nothing leaves fp16's
 *   range) and fp32 sums; X is carried as two fp16 terms, and the Gram matrix without
 *   the mean of its diagonal, which enters in fp32, so that its rounding is no common
 *   factor of the result.  What the operands' roundings leave along directions of zero or
 *   tiny singular values is multiplied by up to a per step.  With (3.4445, -4.7750, 2.0315)
 *   and five steps the result is within (relative, 2-norm, m the smaller side)
 *     2.5e-3 of exact arithmetic for singular values that are spread (Gaussian, or decaying
 *            to a thousandth) and m >= 32,
 *     0.12 / sqrt(m) for any others: for ranks of an eighth to a quarter of m, the worst,
 *            8e-3 was measured at m = 32, 4e-3 at 128, 3e-3 at 256 and 8e-2 at 2.
 *   Norms far below eps lose nothing.  G = 0 gives 0; infinities and NaN in a matrix give
 *   NaN.  Coefficients that let the singular values grow past 64 return
 *   RA_ERR_UNSUPPORTED.
 *   workspace: device memory, 256-byte aligned, about 6 bytes per element of g, 4 per
 *   element of a square matrix of the smaller side, and up to 20 MB for each of the
 *   three products that is split.  It must not be in use by work that overlaps the call
 *   on the GPU.  (A matrix with a side of at most 128 and the other of at most 4096 needs
 *   none of it; the size asked for is the same.) */
size_t ra_newton_schulz_workspace_bytes(int batch, int rows, int cols);
int ra_newton_schulz(const void* g, ra_dtype g_dtype, int batch, int rows, int cols,
                     long long g_bstride, long long g_rstride, const float* coeffs, int steps,
                     float eps, void* out, ra_dtype out_dtype, long long out_bstride,
                     long long out_rstride, void* workspace, size_t ws_bytes, void* stream);

/* Attention of queries to the keys and values of another sequence of any length (cross
 * attention to an encoder's states):
 *     s_ij = scale q_i . k_j,   P = softmax over j < kv_len[b],   o = P v,
 *     lse_i = ln sum_j e^{s_ij}.
 *   q, o [B, N_q, Hq, d], k, v [B, N_kv, Hkv, d], any N_q, N_kv >= 1, in `dtype` (RA_BF16 or
 *   RA_F16), d 64 or 128; o in o_dtype, lse [B, Hq, N_q] fp32.  Strides as in ra_shape.
 *   kv_len  device array of B int32 (clamped to [0, N_kv]), or NULL: every key is there.
 *     Keys and values from kv_len[b] on may hold anything (infinities and NaN too).  A batch
 *     entry without keys has o = 0, lse = -inf.  So has a row whose scores are all -inf (a key with
 *     one counts as not there); one with a score of +inf or NaN is NaN in o and lse.
 *   flags   RA_PRECISE (P and dS in two terms, which the backward pass of fp16 inputs takes
 *     anyway).
 *   A few queries (N_q Hq / Hkv <= 32; single tokens) run on a kernel bound by reading k
 *   and v once; where there are few query tiles the keys are split over the SMs and the parts
 *   joined.  P is rounded to fp16 (two terms with RA_PRECISE) against v in fp16 (bf16 v
 *   copied, with RA_ERR_RANGE, as for the ring), or enters as two terms of the inputs' type (a few
 *   queries, and bf16 where the copy would take longer than the products).
 *   workspace: device memory, 256-byte aligned, ra_cross_fwd_workspace_bytes() bytes.  It
 *   must not be in use by work that overlaps the call on the GPU.  o overlaps no input. */
size_t ra_cross_fwd_workspace_bytes(ra_dtype dtype, ra_shape shape, int flags);
int ra_cross_fwd(const void* q, const void* k, const void* v, ra_dtype dtype, ra_shape shape,
                 const int* kv_len, int flags, float scale, void* o, ra_dtype o_dtype, float* lse,
                 void* workspace, size_t ws_bytes, void* stream);

/* Gradients of L = sum(o * dO): dq [B, N_q, Hq, d], dk, dv [B, N_kv, Hkv, d] in grad_dtype,
 * fully overwritten (rows from kv_len[b] on with zeros), by the formulas of ra_ring_bwd; o in
 * o_dtype, dO in dtype, lse from ra_cross_fwd with the same kv_len and scale.  q, k and v are
 * copied to fp16 as for ra_ring_bwd (those past kv_len[b] as zeros), dO times a power of two.
 * dO . o of an o in 16 bits is formed from q, k and v again for batch entries of up to 4 d keys
 * (with RA_PRECISE of any number): the rounding of o would be the larger part of the errors of
 * rows that few keys share, and stays in those of longer ones (pass o in RA_F32 to be without it).
 * P and dS are rounded to fp16 times powers of two.  Those of dO and dS follow, for each batch
 * entry and key head, the largest rows of dO and v, so that dO may have any size (the largest
 * rows' norm from 2^-72 to 2^100) and no element overflows; rows of dO far below the largest lose
 * digits of their own dq, from 2^-8 at N_kv = 131072 (2^-15 at 1024) on.  dq is summed over the
 * key tiles in fp32 in an order that varies; dk and dv do not vary from run to run.  dk and dv
 * overlap none of q, k, v and dO, and no gradient another. */
size_t ra_cross_bwd_workspace_bytes(ra_dtype dtype, ra_shape shape);
int ra_cross_bwd(const void* q, const void* k, const void* v, const void* o, ra_dtype o_dtype,
                 const void* dO, const float* lse, ra_dtype dtype, ra_shape shape,
                 const int* kv_len, int flags, float scale, void* dq, void* dk, void* dv,
                 ra_dtype grad_dtype, void* workspace, size_t ws_bytes, void* stream);

/* Rotary positions.  Row (b, n, h) of q and of k at position p has its first `rot` columns
 * turned in pairs, pair i by the angle p freq[i]:
 *     (x, y) -> amplitude (x cos - y sin, x sin + y cos),
 * pair i being columns (i, i + rot / 2), or (2i, 2i + 1) with RA_INTERLEAVED; columns from
 * rot on are copied.  q and k of one call go through one launch, between the projections
 * and ra_ring_fwd (backward: between ra_ring_bwd and the projections' gradients).
 *   freq       device array of rot / 2 doubles, radians per position (ra_rotary_frequencies
 *              makes some); angles keep an error of at most 2^-28 + |p| 2^-64 turns.
 *   positions  device array of 64-bit integers, element (b, n) at b * pos_bstride + n (0:
 *              every batch has the same N), any values (pos_off is 0); or NULL: row n is at pos_off + n,
 *              or with RA_STRIPED, where row i S + l (S = N / P) is the l-th of virtual host
 *              i, at pos_off + l P + i.  (Per-host lengths: pass positions.)
 *   P          with RA_STRIPED the number of hosts, which divides N; ignored otherwise. */
typedef struct {
  int rot;                    /* even, 0 (no rotation) to d */
  const double* freq;
  const long long* positions; /* 8-byte aligned, or NULL */
  long long pos_bstride;
  long long pos_off;
  int P;
  float amplitude;            /* 1, or what a scaling method multiplies cos and sin by */
} ra_rotary;

/* How ra_rotary_frequencies stretches frequencies to `scale` times the trained length.
 * With f = base^(-2i / rot):
 * RA_ROTARY_LINEAR  f / scale (positions interpolated).
 * RA_ROTARY_BASE    the same with base scale^(rot / (rot - 2)) base: the fastest pair keeps its
 *                   frequency, the slowest is divided by scale.  rot > 2.
 * RA_ROTARY_PARTS   by the turns t = trained f / 2 pi that a pair makes in the trained length:
 *                   f from `fast` turns on, f / scale up to `slow` turns, in between the mean
 *                   of both with weights that go linearly with t ("YaRN: Efficient Context
 *                   Window Extension of Large Language Models", Peng et al. 2023, section 3.2,
 *                   which also multiplies cos and sin by 1 + 0.1 ln scale: `amplitude`). */
enum { RA_ROTARY_LINEAR = 0, RA_ROTARY_BASE = 1, RA_ROTARY_PARTS = 2 };

/* freq[0 .. rot / 2) (host memory) of a method.  base > 1, scale >= 1; trained > 0 and
 * fast > slow >= 0 for RA_ROTARY_PARTS (ignored otherwise). */
int ra_rotary_frequencies(int rot, double base, double scale, int method, double trained,
                          double fast, double slow, double* freq);

/* q [B, N, Hq, d], k [B, N, Hkv, d] (shape.N_q = shape.N_kv = N) -> q_out, k_out, same type,
 * at the strides of out_shape (whose extents are those of shape).  k and k_out may both be
 * NULL: q alone.  q_out may be q itself (and k_out k) where the strides agree; otherwise
 * outputs overlap no input, nor each other.  (Refused; tensors of different strides or
 * types that lie within each other count as overlapping.)  flags: RA_INTERLEAVED, RA_STRIPED.
 *   Sizes: d a multiple of 8 up to 256; rows start on 16-byte boundaries.  Any dtype; sums
 *   and products fp32, rounded once; sine and cosine to fp32's last bits for results in fp32,
 *   within 5e-7 for results (backward: dq, dk) in 16 bits.  Columns from rot on are copied, bit for bit
 *   but for what a NaN holds. */
int ra_rotary_fwd(const void* q, const void* k, ra_dtype dtype, ra_shape shape, ra_rotary rotary,
                  int flags, void* q_out, void* k_out, ra_shape out_shape, void* stream);

/* Gradients of ra_rotary_fwd: dq, dk from the gradients dq_out, dk_out of its results (in
 * dtype, at the strides of shape), written in grad_dtype (dtype, or any type where dtype is
 * RA_F32) at the strides of grad_shape.  In place as above. */
int ra_rotary_bwd(const void* dq_out, const void* dk_out, ra_dtype dtype, ra_shape shape,
                  ra_rotary rotary, int flags, void* dq, void* dk, ra_dtype grad_dtype,
                  ra_shape grad_shape, void* stream);

/* Norm of each head and rotary positions in one pass over q and k:
 *     r = (mean_c x_c^2 + eps)^-1/2,   y = rotate(x r w)
 * for each row (b, n, h), the mean over all d columns, w q_weight or k_weight [d] in
 * w_dtype (NULL: ones).  rotary.rot = 0 norms without a rotation (for queries and keys of
 * cross attention, say).  eps >= 0; rows whose squares leave fp32's range, up or down, are
 * scaled first.
 * Other arguments as for ra_rotary_fwd. */
int ra_norm_rotary_fwd(const void* q, const void* k, ra_dtype dtype, ra_shape shape,
                       const void* q_weight, const void* k_weight, ra_dtype w_dtype, float eps,
                       ra_rotary rotary, int flags, void* q_out, void* k_out, ra_shape out_shape,
                       void* stream);

/* Gradients of ra_norm_rotary_fwd, with g = rotate^T(dy) and n = x r:
 *     dx = r (g w - n mean_c(g_c w_c n_c)),   dw_c = sum over rows of g_c n_c.
 *   q, k the inputs of the forward pass (dtype, shape); dq_out, dk_out the gradients of its
 *   results in dout_dtype (dtype or RA_F32) at the strides of dout_shape; dq, dk in
 *   grad_dtype (dtype or RA_F32) at the strides of grad_shape, which may be dq_out, dk_out
 *   (or q, k) themselves where type and strides agree, and otherwise overlap none; dq_weight, dk_weight [d] fp32,
 *   overwritten, NULL where not wanted.  Results do not vary from run to run.
 *   workspace: device memory, 256-byte aligned, ra_norm_rotary_bwd_workspace_bytes(d)
 *   bytes.  It must not be in use by work that overlaps the call on the GPU. */
size_t ra_norm_rotary_bwd_workspace_bytes(int d);
int ra_norm_rotary_bwd(const void* q, const void* k, ra_dtype dtype, ra_shape shape,
                       const void* dq_out, const void* dk_out, ra_dtype dout_dtype,
                       ra_shape dout_shape, const void* q_weight, const void* k_weight,
                       ra_dtype w_dtype, float eps, ra_rotary rotary, int flags, void* dq, void* dk,
                       ra_dtype grad_dtype, ra_shape grad_shape, float* dq_weight,
                       float* dk_weight, void* workspace, size_t ws_bytes, void* stream);

/* The norm of the gradients of many tensors taken together, n = (sum g^2)^1/2 over all
 * elements of all of them, and their clipping by it ("Ring Attention: Train 1M Tokens on 8GB
 * GPUs in 2026", section "Gotchas and Failure Modes", clips gradients through the ring):
 *     c = min(1, max_norm / (n + eps)),   out = c g.
 *   grads, sizes, dtypes, outs, out_dtypes  host arrays of `count` entries, read during the
 *   call: device addresses (aligned to an element), numbers of elements (0 allowed), types;
 *   a tensor's elements are contiguous.  outs NULL: in place (where c = 1 nothing is
 *   written); an entry of outs may be that of grads where the types agree; otherwise no
 *   output overlaps another tensor.  A tensor that is listed twice counts twice, and cannot
 *   be written twice.
 *   norm [1] fp32 on the device.  Sums are fp64 (fp32 over up to 64 elements): gradients of
 *   any size, from fp32's smallest to its largest, have their norm.  An infinite n gives
 *   c = 0 and NaN gives NaN, as the formula says: read norm to skip such a step.  The
 *   results do not vary from run to run.
 *   max_norm >= 0, eps >= 0 (with both 0 and n = 0, c is NaN).
 *   workspace: device memory, 256-byte aligned, ra_grad_workspace_bytes(count) bytes.  It
 *   must not be in use by work that overlaps the call on the GPU. */
size_t ra_grad_workspace_bytes(int count);
int ra_grad_norm(const void* const* grads, const long long* sizes, const int* dtypes, int count,
                 float* norm, void* workspace, size_t ws_bytes, void* stream);
int ra_grad_clip(const void* const* grads, const long long* sizes, const int* dtypes, int count,
                 float max_norm, float eps, void* const* outs, const int* out_dtypes, float* norm,
                 void* workspace, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then return and clear the device status word
 * (RA_OK, RA_ERR_RANGE, RA_ERR_TIMEOUT, or RA_ERR_INVALID_ARG for a target outside
 * the vocabulary), or RA_ERR_CUDA if the stream
 * itself reports an error. */
int ra_sync_status(void* stream);

/* Message for the last non-OK return on the calling thread ("" if none). */
const char* ra_last_error(void);

/* Number of kernels this library has launched in this process. */
unsigned long long ra_launch_count(void);

/* Debug record of the ring schedule (off by default).  The pages debug a real
 * ring with one log file per rank that records what each step received
 * ("Ring Attention: Train 1M Tokens on 8GB GPUs in 2026", section "Debugging
 * Ring Transfers with Rank-Specific Logs"); here one process runs every
 * virtual host, and this log records, per tile the tensor-core kernels bring
 * into shared memory, which host's work it serves:
 *   entries  device array of `capacity` records of four uint32
 *            {kind, head, query tile, key tile}, 16-byte aligned:
 *            kind 0 -- the forward (ra_ring_fwd*, ra_block_fwd) loaded key/value
 *              tile `key tile` for the unit whose first query tile is
 *              `query tile` (128-row tiles, tensor row / 128);
 *            kind 1 -- the backward (ra_ring_bwd*) loaded query tile
 *              `query tile` for the unit of key/value tile `key tile`;
 *            head = b * Hq + (query head).
 *   count    device uint32 the kernels advance atomically (the caller zeroes
 *            it); records past `capacity` are counted but not stored.
 * One thread per CTA writes a unit's records, so they appear in the order the
 * unit visits its tiles (records of different units interleave).  Tiles that
 * are skipped (blocks in a query tile's causal future, tiles wholly in
 * padding) leave no record.  The setting is process-wide and applies to every
 * launch until ra_debug_visit_log(NULL, 0, NULL) turns it off; the buffers
 * must stay valid until then.  Logging costs one atomic per tile. */
int ra_debug_visit_log(unsigned int* entries, size_t capacity, unsigned int* count);

/* Kernel timing.  While enabled, every launch of the kernels below is
 * bracketed by CUDA events recorded on the stream it is launched on;
 * ra_kernel_timing_read() waits for those events and returns the summed
 * device time (ms) and the number of launches since timing was enabled.
 * ra_kernel_timing(1) enables and resets, ra_kernel_timing(0) disables and
 * releases the events.  Used by the benchmark to time the dominant kernel.
 * The two copy entries time ra_ring_step_host's transfers the same way: each
 * group of copies on one stream (q, k, v up; dO up; O and LSE down; dQ, dK,
 * dV down) is bracketed by events on that stream, so the sums are the time
 * the copies themselves took, whatever kernels ran beside them. */
typedef enum {
  RA_KERNEL_FWD_TC = 0,   /* tensor-core forward (ring and block step) */
  RA_KERNEL_BWD_TC = 1,   /* tensor-core backward */
  RA_KERNEL_FWD_F32 = 2,  /* fp32 CUDA-core forward */
  RA_KERNEL_BWD_F32 = 3,  /* fp32 CUDA-core backward (both kernels) */
  RA_KERNEL_GEMM_TC = 4,  /* tensor-core GEMM of the feed-forward layer (every launch) */
  RA_COPY_H2D = 5,        /* ra_ring_step_host uploads (two groups per call) */
  RA_COPY_D2H = 6,        /* ra_ring_step_host downloads (two groups per call) */
  RA_KERNEL_PAIR_TC = 7,  /* tensor-core CTA-pair products (cross entropy, Newton-Schulz) */
  RA_KERNEL_COUNT = 8
} ra_kernel_id;
int ra_kernel_timing(int enable);
int ra_kernel_timing_read(int kernel, double* total_ms, unsigned long long* launches);

/* Self-test of the bounded wait: launches one CTA that waits on an mbarrier
 * nobody arrives at, with a limit of timeout_us microseconds; the kernel must
 * give up, record RA_ERR_TIMEOUT in the status word and return.  Returns the
 * launch status; read the outcome with ra_sync_status(). */
int ra_selftest_timeout(unsigned int timeout_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RA_H_ */
