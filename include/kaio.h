/*
 * kaio.h -- C ABI of the MI355X (gfx950) W4A16 fused-QKV library.
 *
 * Each operation is asynchronous on the caller's HIP stream, one launch unless
 * noted:
 *
 *   kaio_qkv_w4a16          W4A16 group-quantized fused tri-output QKV projection
 *   kaio_qkv_w8a16          its W8A16 sibling (INT8 weights, same contract)
 *                           (kaio_qkv_plan: which kernel form a call of given sizes runs)
 *   kaio_gemm_f16f32        dense f16 x f16 -> f32 matmul
 *   kaio_gemm_f16f32_bwd    its backward: f16 gradients of A and B (three launches)
 *                           (kaio_gemm_f16f32_bwd_noalloc: the same without a workspace)
 *   kaio_dequant_group_bwd  straight-through per-group dequant backward
 *   kaio_linear_w4a16       W4A16 product with bias, activation and residual
 *   kaio_rope_append        rotary positions on Q and K, K and V written to a
 *                           paged cache
 *   kaio_paged_attention    attention of new tokens over that cache (two
 *                           launches where the keys of a row are split)
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 * - Pointers are DEVICE pointers (memory the HIP runtime allocated on the
 *   current device).  The caller owns every buffer; the library never
 *   allocates, frees, copies to the host or synchronizes.  Inputs are never
 *   written.  Outputs are fully overwritten (no pre-zeroing needed).
 * - All tensors are dense, row-major, zero-offset.  Base pointers must be
 *   16-byte aligned.  Outputs must not overlap any input or each other.
 * - `stream` is a hipStream_t passed as void* (NULL = the null stream).  The
 *   launch is queued on it and the call returns; a fault inside a kernel is
 *   reported by the caller's next synchronizing HIP call, not here.
 * - Validation happens on the host, in the order listed per entry point;
 *   the first failure wins and nothing is launched.  An empty problem
 *   (no outputs) returns KAIO_OK without touching the device.
 * - On failure kaio_last_error() returns "kaio::<op>: <reason>" for the
 *   calling thread.
 * - The device must be an AMD gfx950 (MI355X); anything else returns
 *   KAIO_ERR_DEVICE.  There is no CPU fallback.
 */
#ifndef KAIO_H
#define KAIO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kaio_status {
  KAIO_OK = 0,
  KAIO_ERR_INVALID_ARGUMENT = 1, /* null, misaligned or overlapping pointer             */
  KAIO_ERR_INVALID_PROBLEM = 2,  /* sizes the operation does not define                 */
  KAIO_ERR_UNSUPPORTED = 3,      /* defined, but not offered (group size, dtype)        */
  KAIO_ERR_DEVICE = 4,           /* no HIP device, or the current device is not gfx950 */
  KAIO_ERR_LAUNCH = 5            /* the HIP runtime refused the launch                  */
} kaio_status;

typedef enum kaio_dtype {
  KAIO_DTYPE_F32 = 0,
  KAIO_DTYPE_BF16 = 1,
  KAIO_DTYPE_F16 = 2,
  KAIO_DTYPE_F64 = 3
} kaio_dtype;

/*
 * W4A16 fused tri-output QKV projection.
 * Defined by: kaio-candle 0.2.0, src/qkv_project_int4.rs -- module doc (one
 * launch, seven inputs, group size locked at 128, K a multiple of 128) and
 * the doc comment of qkv_project_int4 (operand shapes, f16 outputs converted
 * from f32 inside the kernel).
 *
 *   For p in {q, k, v}:
 *     Y_p[m, n] = sum_k x[m, k] * int4(W_p, k, n) * S_p[k / 128, n]
 *
 *   x        f16[m, k]       activations, shared by the three projections
 *   w_q/k/v  u32[k/8, n]     packed INT4 weights: word (r, n) at offset r*n_cols + n;
 *                            nibble i (bits 4i..4i+3, low first) holds k = 8r + i as a
 *                            signed two's-complement value in [-8, 7], no zero point
 *   s_q/k/v  f16[k/128, n]   one scale per 128 consecutive k of each column
 *   q, k_out, v  f16[m, n]   outputs, f32 accumulation rounded once to f16 (RNE)
 *   group_size  must be 128
 *
 * Validation order: group_size != 128 -> UNSUPPORTED; k % 128 != 0 ->
 * INVALID_PROBLEM; m == 0 or n == 0 -> OK (nothing launched); sizes too
 * large for one launch (n >= 2^26, k >= 2^24, any tensor of 2^62 bytes or
 * more, or more than 2^24 - 1 workgroups) -> INVALID_PROBLEM; null pointer (weights/scales/x
 * only when k > 0) -> INVALID_ARGUMENT; misaligned pointer ->
 * INVALID_ARGUMENT; an output overlapping an input or another output ->
 * INVALID_ARGUMENT; device -> DEVICE; launch -> LAUNCH.  k == 0 writes
 * zeros.  m <= 64 runs the memory-bound split-K kernel (decode and batched
 * decode), larger m the MFMA tile kernel (up to m = 128 with one output per
 * workgroup, and so from m = 33 when k / 128 is a multiple of 4); all obey
 * this contract.
 */
kaio_status kaio_qkv_w4a16(const void* x,
                           const uint32_t* w_q, const uint32_t* w_k, const uint32_t* w_v,
                           const void* s_q, const void* s_k, const void* s_v,
                           void* q, void* k_out, void* v,
                           uint32_t m, uint32_t n, uint32_t k, uint32_t group_size,
                           void* stream);

/*
 * W8A16 fused tri-output QKV projection: the INT8 sibling of kaio_qkv_w4a16.
 * Named by: kaio-candle 0.2.0, src/qkv_project_int4.rs -- module doc (the
 * INT4 op follows the same direct-call pattern as qkv_project_int8, whose
 * weight layout the pages do not print).  This library's reading of it is the
 * 8-bit analogue of the INT4 packing:
 *
 *   For p in {q, k, v}:
 *     Y_p[m, n] = sum_k x[m, k] * int8(W_p, k, n) * S_p[k / 128, n]
 *
 *   x        f16[m, k]       activations, shared by the three projections
 *   w_q/k/v  u32[k/4, n]     packed INT8 weights: word (r, n) at offset r*n_cols + n;
 *                            byte i (bits 8i..8i+7, low first) holds k = 4r + i as a
 *                            signed two's-complement value in [-128, 127], no zero point
 *   s_q/k/v  f16[k/128, n]   one scale per 128 consecutive k of each column
 *   q, k_out, v  f16[m, n]   outputs, f32 accumulation rounded once to f16 (RNE)
 *   group_size  must be 128
 *
 * Validation order, limits and error behaviour: exactly as kaio_qkv_w4a16;
 * m <= 64 runs the split-K kernel, larger m the tile kernel.
 */
kaio_status kaio_qkv_w8a16(const void* x,
                           const uint32_t* w_q, const uint32_t* w_k, const uint32_t* w_v,
                           const void* s_q, const void* s_k, const void* s_v,
                           void* q, void* k_out, void* v,
                           uint32_t m, uint32_t n, uint32_t k, uint32_t group_size,
                           void* stream);

/*
 * Dense f16 x f16 -> f32 matmul, C = A . B (C is overwritten, not accumulated).
 * Defined by: kaio-candle 0.2.0, src/matmul_tc_async.rs -- module doc
 * (f16 x f16 -> f32 matmul) and MatmulTcAsyncOp::cuda_fwd (A [m, k],
 * B [k, n], a zeroed [m, n] f32 output written by the kernel).
 *
 *   a  f16[m, k]   b  f16[k, n]   c  f32[m, n]
 *
 * Validation order: m == 0 or n == 0 -> OK (nothing launched); sizes too
 * large for one launch -> INVALID_PROBLEM; null pointer (a, b only when
 * k > 0) -> INVALID_ARGUMENT; misaligned -> INVALID_ARGUMENT; c overlapping
 * a or b -> INVALID_ARGUMENT; device -> DEVICE; launch -> LAUNCH.  k == 0
 * writes zeros.
 */
kaio_status kaio_gemm_f16f32(const void* a, const void* b, float* c,
                             uint32_t m, uint32_t n, uint32_t k, void* stream);

/*
 * Backward of kaio_gemm_f16f32 for an f32 output gradient g [m, n]:
 *   g16    = f16(g)                                (round to nearest even)
 *   grad_a = f16( g16 . b^T )     f16[m, k]
 *   grad_b = f16( a^T . g16 )     f16[k, n]
 * each product accumulated in f32 and rounded once to f16 (nearest even).
 * Defined by: kaio-candle 0.2.0, src/matmul_tc_async.rs --
 * MatmulTcAsyncOp::bwd (the gradient cast to f16, dA = grad . B^T and
 * dB = A^T . grad by the forward kernel, both results cast to f16).
 *
 *   a  f16[m, k]   b  f16[k, n]   grad  f32[m, n]
 *   grad_a  f16[m, k]   grad_b  f16[k, n]
 *   workspace  device scratch for g16: at least
 *              kaio_gemm_f16f32_bwd_workspace_size(m, n) bytes, 16-byte
 *              aligned, overlapping nothing else; its contents on return
 *              are unspecified.  Calls on one workspace must not overlap.
 *
 * Validation order: sizes too large for one launch -> INVALID_PROBLEM;
 * k == 0 -> OK (both gradients are empty, nothing launched); null output
 * -> INVALID_ARGUMENT; m == 0 or n == 0 -> both gradients are the empty
 * sum: zeros are written (a, b, grad and workspace are not read and may be
 * null); null input or workspace, or workspace_bytes too small ->
 * INVALID_ARGUMENT; misaligned -> INVALID_ARGUMENT; overlapping buffers ->
 * INVALID_ARGUMENT; device -> DEVICE; launch -> LAUNCH.
 */
kaio_status kaio_gemm_f16f32_bwd(const void* a, const void* b, const float* grad,
                                 void* grad_a, void* grad_b,
                                 uint32_t m, uint32_t n, uint32_t k,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes kaio_gemm_f16f32_bwd needs for an [m, n] gradient: m * n * 2. */
size_t kaio_gemm_f16f32_bwd_workspace_size(uint32_t m, uint32_t n);

/*
 * kaio_gemm_f16f32_bwd without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  f16(grad) is staged in a static device
 * buffer of KAIO_GEMM_BWD_NOALLOC_MAX_BYTES bytes that the library's code
 * object holds on every device it is loaded on, until the process ends; this
 * call allocates and frees nothing.  Results are bit-identical to
 * kaio_gemm_f16f32_bwd with a caller workspace (same kernels).
 *
 * Every call on a device shares that device's buffer: calls that overlap in
 * time on one device (other streams, concurrently replayed graphs) race and
 * must be serialized by the caller.  Nothing in the buffer needs to be
 * cleared between calls (the cast overwrites what the products read).
 *
 * Validation order: as kaio_gemm_f16f32_bwd, without the workspace checks,
 * plus m * n * 2 > KAIO_GEMM_BWD_NOALLOC_MAX_BYTES -> UNSUPPORTED (right
 * after the size check; nothing launched).
 */
#define KAIO_GEMM_BWD_NOALLOC_MAX_BYTES (64ull << 20)
kaio_status kaio_gemm_f16f32_bwd_noalloc(const void* a, const void* b, const float* grad,
                                         void* grad_a, void* grad_b,
                                         uint32_t m, uint32_t n, uint32_t k, void* stream);

/*
 * Straight-through per-group dequant backward:
 *   dq[i, j] = dy[i, j] * scale[i, j / group_size]     (one rounded multiply)
 * Defined by: baracuda-kernels 0.0.1-alpha.68,
 * src/quantize/dequantize_per_group_backward.rs -- module doc (the formula),
 * DequantizePerGroupBackwardArgs (shapes), DequantizePerGroupBackwardPlan::select
 * (dtype and size rules), ::workspace_size (none) and ::run (empty problem
 * returns without work).  Results are bit-exact: the correctly rounded
 * product in the dtype, identical on every run.
 *
 *   dtype      element type of dy, scale and dq (F32, BF16, F16, F64)
 *   dy         [outer, axis]              upstream gradient
 *   scale      [outer, axis / group_size] saved scales
 *   dq         [outer, axis]              output gradient
 *   workspace, workspace_bytes   accepted and ignored (no workspace is used)
 *
 * Pointers need only element alignment here; 16-byte alignment and
 * group_size % (16 / element size) == 0 select the vector path.
 *
 * Validation order: dtype unknown -> UNSUPPORTED; outer < 0 or axis < 0 ->
 * INVALID_PROBLEM; group_size <= 0 -> INVALID_PROBLEM; axis % group_size != 0
 * -> INVALID_PROBLEM; outer * axis == 0 -> OK (nothing launched); sizes
 * too large -> INVALID_PROBLEM; null pointer -> INVALID_ARGUMENT; misaligned (element) -> INVALID_ARGUMENT;
 * dq overlapping dy or scale -> INVALID_ARGUMENT; device -> DEVICE; launch
 * -> LAUNCH.
 */
kaio_status kaio_dequant_group_bwd(kaio_dtype dtype, int32_t outer, int32_t axis,
                                   int32_t group_size,
                                   const void* dy, const void* scale, void* dq,
                                   void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Which kernel form a kaio_qkv_w4a16 (bits 4) or kaio_qkv_w8a16 (bits 8)
 * call of these sizes runs, for tests and tuning; host only, no device
 * touched, nothing launched.  On KAIO_OK:
 *   plan[0]  0: the split-K kernel, 1: the tile kernel (each workgroup
 *            computes its tile of Q, K and V), 2: the tile kernel with one
 *            output per workgroup (three times the workgroups)
 *   plan[1]  tile kernel: waves per set; split-K: 0
 *   plan[2]  tile kernel: rows of x per tile; split-K: columns per strip
 *   plan[3]  tile kernel: sets of waves per workgroup (2: the 128-k groups
 *            are split in halves over two sets); split-K: 1
 *   plan[4]  workgroups the launch has
 * m == 0 or n == 0 is an empty call (plan[0..4] = 0).  bits other than 4 or
 * 8, or a null plan -> INVALID_ARGUMENT; k % 128 != 0 -> INVALID_PROBLEM.
 */
kaio_status kaio_qkv_plan(uint32_t m, uint32_t n, uint32_t k, uint32_t bits, uint32_t plan[5]);

/* Activations of kaio_linear_w4a16's epilogue. */
typedef enum kaio_activation {
  KAIO_ACT_NONE = 0,
  KAIO_ACT_RELU = 1,      /* max(y, 0), NaN kept                                      */
  KAIO_ACT_GELU = 2,      /* y (1 + erf(y / sqrt 2)) / 2                              */
  KAIO_ACT_GELU_TANH = 3, /* y (1 + tanh(sqrt(2 / pi) (y + 0.044715 y^3))) / 2        */
  KAIO_ACT_SILU = 4       /* y / (1 + exp(-y))                                        */
} kaio_activation;

/*
 * W4A16 product with an epilogue, the projection after attention and the
 * products of a feed-forward block on the same packed weights as the QKV
 * projection:
 *
 *   y[m, n] = act( sum_k x[m, k] * int4(W, k, n) * S[k / 128, n] + b[n] ) + r[m, n]
 *
 *   x  f16[m, k]   w  u32[k/8, n] and s  f16[k/128, n] as kaio_qkv_w4a16
 *   bias      f16[n] or NULL        residual  f16[m, n] or NULL
 *   y         f16[m, n]; may be the residual's buffer itself (updated in place)
 *   group_size  must be 128
 *
 * The sum, the bias, the activation and the residual are in f32, rounded once
 * to f16 (RNE).
 *
 * Validation order: group_size != 128 -> UNSUPPORTED; unknown activation ->
 * UNSUPPORTED; k % 128 != 0 -> INVALID_PROBLEM; m == 0 or n == 0 -> OK
 * (nothing launched); too large (limits of kaio_qkv_w4a16) ->
 * INVALID_PROBLEM; null pointer (x, w and s only when k > 0) ->
 * INVALID_ARGUMENT; misaligned (16 bytes) -> INVALID_ARGUMENT; y overlapping
 * an input (other than residual == y) -> INVALID_ARGUMENT; device -> DEVICE;
 * launch -> LAUNCH.  k == 0: the product is zero, the epilogue still runs.
 */
kaio_status kaio_linear_w4a16(const void* x, const uint32_t* w, const void* s,
                              const void* bias, const void* residual, void* y,
                              uint32_t m, uint32_t n, uint32_t k, uint32_t group_size,
                              kaio_activation activation, void* stream);

/*
 * A paged key/value cache and the batch that uses it.  The struct itself is in
 * host memory and read during the call; the pointers are device pointers.
 *
 * Sequence s has the new tokens of rows q_start[s] .. q_start[s+1]-1 and
 * lens[s] tokens in the cache with the new ones last: row t of it is at
 * position lens[s] - (q_start[s+1] - t).  The token at position c lies in slot
 * c % page_size of page page_table[s][c / page_size].
 *
 * The contents of page_table, q_start and lens are read on the device and may
 * change from call to call (a captured graph sees them at replay).  A page id
 * outside [0, pages), -1 by custom, is a page that is not there: a released
 * page or one not needed yet.  Its positions are not visible, and nothing is
 * written to it; so are positions past table_width * page_size.  Rows of q in
 * no sequence (a batch padded past q_start[seqs]) see nothing.
 * Calls read and write the cache only through present pages.  No two
 * sequences may write to one page.
 */
typedef struct kaio_paged_kv {
  void* k_cache;              /* [pages, page_size, kv_heads, head_dim] */
  void* v_cache;              /* the same shape                         */
  const int32_t* page_table;  /* [seqs, table_width]                    */
  const int32_t* q_start;     /* [seqs + 1], ascending                  */
  const int32_t* lens;        /* [seqs]                                 */
  int32_t dtype;              /* KAIO_DTYPE_F16 or KAIO_DTYPE_BF16: cache and q, k, v, outputs */
  uint32_t pages, page_size, kv_heads, head_dim;
  uint32_t seqs, table_width;
} kaio_paged_kv;

/*
 * Rotary positions on Q and K, K and V written to the paged cache.
 *
 * Pair j < half of every head of q and k (elements 2j and 2j+1 when
 * interleaved, else j and j + half) is turned by the angle
 * a = positions[axis(j)][t] * inv_freq[j], taken in 64 bits:
 *   (x, y) -> (x cos a - y sin a, x sin a + y cos a)
 * in f32, rounded once.  sections[i] consecutive pairs belong to axis i; half
 * is their sum.  Elements past 2 * half pass through.  The turned K and V of
 * row t go to the slot of its position.
 *
 *   q  [tokens, q_heads, head_dim]   k, v  [tokens, kv_heads, head_dim]
 *   positions  i32[axes, tokens]     inv_freq  f64[half]
 *   sections   u32[axes], in HOST memory
 *   q_out      as q; may be q itself (turned in place)
 *
 * Validation order: kv null -> INVALID_ARGUMENT; dtype -> UNSUPPORTED; axes
 * not in [1, 8], head_dim > 1024 -> UNSUPPORTED; page_size, kv_heads or
 * head_dim zero, 2 * half > head_dim -> INVALID_PROBLEM; tokens == 0 -> OK
 * (nothing launched); too large (2^31 slots, 2^24 - 1 workgroups, 2^62 bytes)
 * -> INVALID_PROBLEM; null, misaligned (16 bytes; integers and inv_freq by
 * element) or overlapping pointer -> INVALID_ARGUMENT; device -> DEVICE;
 * launch -> LAUNCH.
 */
kaio_status kaio_rope_append(const kaio_paged_kv* kv, const void* q, const void* k, const void* v,
                             const int32_t* positions, const double* inv_freq,
                             const uint32_t* sections, uint32_t axes, int32_t interleaved,
                             void* q_out, uint32_t tokens, uint32_t q_heads, void* stream);

/*
 * Attention of the new tokens over the paged cache: decode, chunks of prompts
 * and whole prompts, causal, with grouped heads (q head h reads K/V head
 * h / (q_heads / kv_heads)).
 *
 *   out[t, h] = sum_c softmax_c(scale * q[t, h] . K[c]) V[c]
 *
 * over the visible positions c of the row at position pos: c <= pos, c <
 * lens[s], its page there, and, with window > 0, c > pos - window or c < sinks.
 * A row that sees nothing is zero.  Scores, maxima, sums and the output's
 * accumulation are f32.  The weights are rounded to the cache's type for the
 * product with V at head_dim 64 and 128 (half a step each; the sum is taken of
 * the rounded ones), and stay f32 at other sizes.  Invisible positions are not
 * read into the result, whatever they hold; a visible value that is not finite
 * shows in the result however small its weight.  Scores of a magnitude past 2^26,
 * where f32's steps exceed the weights' range, may make their row NaN.
 *
 * Speed follows from what the host knows, the lengths not among it: a table
 * not much wider than the sequences need lets short calls run in one launch,
 * one workgroup per tile, where a wide one splits the keys and joins the
 * pieces (512 / 1024 / 4096 new tokens of 32 heads over 8, 128 columns: 18 / 30
 * / 160 us against 32 / 47 / 231 us with room for 131072 tokens).  Keys are
 * never split in calls of many tiles, and one long sequence among short ones
 * then takes its own time: a tile is 128 rows (tokens times heads of a group),
 * or 16 where max_new * group is at most 16, every sequence counts one more,
 * and many are more than 512, or 2048 and more over all K/V heads.  With tiles
 * of 128 rows a cache tensor past 4 GiB, or a page_size that is no multiple of
 * 4 (128 columns) or 8 (64), costs 1.4 times the time.  Head sizes other than
 * 64 and 128 run a simple kernel, tens of times slower.
 *
 *   q, out  [tokens, q_heads, head_dim]
 *   max_new    the most new tokens a sequence has (it chooses the kernel; a
 *              larger number in q_start is still served correctly)
 *   window     0: none                sinks  first tokens that stay visible
 *   workspace  device scratch of at least kaio_paged_attention_workspace_size
 *              bytes, 16-byte aligned (NULL when that is 0); unspecified on
 *              return.  Calls on one workspace must not overlap in time.
 *
 * Results are deterministic for given sizes and contents of lens and q_start.
 *
 * Validation order: kv null -> INVALID_ARGUMENT; dtype -> UNSUPPORTED;
 * page_size, kv_heads or head_dim zero, q_heads not a multiple of kv_heads,
 * scale not finite -> INVALID_PROBLEM; head_dim > 256 -> UNSUPPORTED; tokens
 * == 0 or q_heads == 0 -> OK; max_new == 0 or too large -> INVALID_PROBLEM; null,
 * misaligned or overlapping pointer, workspace too small ->
 * INVALID_ARGUMENT; device -> DEVICE; launch -> LAUNCH.
 */
kaio_status kaio_paged_attention(const kaio_paged_kv* kv, const void* q, void* out,
                                 uint32_t tokens, uint32_t q_heads, uint32_t max_new,
                                 float scale, uint32_t window, uint32_t sinks,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes kaio_paged_attention needs for these sizes (0 for sizes it refuses). */
size_t kaio_paged_attention_workspace_size(const kaio_paged_kv* kv, uint32_t tokens, uint32_t q_heads,
                                           uint32_t max_new);

/* Message of the calling thread's most recent failed call ("" after a success). */
const char* kaio_last_error(void);

/* Library version string, e.g. "kaio-mi355x 0.1.0 gfx950". */
const char* kaio_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KAIO_H */
