/*
 * dynconv.h: C ABI of the dynamic short convolution library (libdynconv.so), gfx950.
 *
 * The operation, from "Dynamic Short Convolutions Improve Transformers" (reading note),
 * section "Parameterization":
 *
 *   eq. 2 + eq. 3:   y[b,t,d] = x[b,t,d] + sum_{k=0}^{W-1} w[b,t,g(d),k] * x[b,t-k,d]
 *
 * with x[b,t,d] = 0 for t < 0 in every sequence b, g(d) = d / H (one filter shared by H
 * consecutive channels: H = 1 is the per-channel form, H > 1 the head-wise form), and a
 * static filter (eq. 1) as the case where w does not depend on (b, t). In the low-rank
 * form (same section, and "Efficient training (Triton kernels)") the filters are
 * generated on the GPU from z (B x T x R) and the second projection U (R x (D/H)*W)
 * plus a bias b: w[b,t,g,k] = sum_r z[b,t,r] U[r, g*W+k] + b[g*W+k], and are never
 * written to memory.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers. The caller owns every buffer, including
 *   the workspace; the library never allocates or frees device memory, never
 *   synchronises, and keeps no mutable global state (thread-safe) apart from the
 *   per-device address of dynconv_bwd_ex_noalloc's scratch array (set once, under a lock).
 * - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream) and the call
 *   returns without waiting.
 * - Strides are in ELEMENTS, int64, in PyTorch .stride() order. Activation-shaped tensors
 *   (x, y, dy, dx) are [B, T, D] with strides s[0..2], s[2] == 1. Filter-shaped tensors
 *   (w, dw) are [B, T, D/H, W] with strides s[0..3], s[3] == 1 and s[2] == W (the W taps
 *   of one group are contiguous). w with s[0] == s[1] == 0 is a static filter [D/H, W].
 *   z and dz are [B, T, R] with strides s[0..2], s[2] == 1.
 * - Element types: x, w, z, U, bias, y, dy, dx, dw (per token) and dz all have `dtype`
 *   (float32, bfloat16 or float16). Reduced parameter gradients (static dw, dU, db) are
 *   always float32 and contiguous.
 * - Arithmetic is float32 (products and sums), 16-bit results are rounded to nearest even.
 *   The fast low-rank kernels serve bfloat16 and float16; float32 takes the general ones.
 * - Validation happens before any HIP call; invalid input returns a status, never aborts.
 *   B == 0 or T == 0 or D == 0 is a no-op returning DYNCONV_OK.
 * - Supported parameters: 1 <= W <= 8; H any divisor of D, with
 *   H / VEC <= 64 for the materialised and static forms, where VEC (channels per lane) is,
 *   in 16-bit storage, 2m when H = m * 2^k with m = 3 or 5 and k >= 1 and H itself when H is
 *   3 or 5, and otherwise the largest power of two that divides H and is at most the widest
 *   lane vector allowed by the alignment below / element size (so with 16-byte aligned
 *   activations: powers of two up to 512 in 16-bit storage and 256 in float32; H = 3 * 2^k up
 *   to 384 and H = 5 * 2^k up to 640 in 16-bit storage, 192 and 160 in float32; other odd H
 *   up to 63); low-rank form: 1 <= R <= 128.
 * - Alignment: base pointers of activation-shaped tensors and their s[0], s[1] (in bytes)
 *   must be multiples of 4 bytes (bf16: D even); wider lane vectors (8 or 16 bytes) are
 *   used when every activation-shaped tensor of the call allows them. Filters: base and
 *   s[0], s[1] multiples of 4 bytes for H == 1, and for H > 1 when the W taps of a group
 *   fill whole 32-bit words (float32, or bf16 with W even); element alignment otherwise.
 *   Violations return DYNCONV_ERR_UNSUPPORTED.
 * - An output pointer equal to any input pointer returns DYNCONV_ERR_INVALID_ARG
 *   (in-place use would corrupt the time halo); partial overlap is undefined behaviour.
 * - A failed kernel launch returns DYNCONV_ERR_HIP; dynconv_last_hip_error() then gives
 *   the hipError_t of the calling thread's last failure.
 */
#ifndef DYNCONV_H
#define DYNCONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type codes and status codes are plain 32-bit integers, so that any value a caller
 * passes is well defined (an unknown dtype code is refused with DYNCONV_ERR_INVALID_ARG). */
typedef int32_t dynconv_dtype;
enum { DYNCONV_F32 = 0, DYNCONV_BF16 = 1, DYNCONV_F16 = 2 };

typedef int32_t dynconv_status;
enum {
  DYNCONV_OK = 0,
  DYNCONV_ERR_INVALID_ARG = 1, /* null / negative / inconsistent argument, aliasing */
  DYNCONV_ERR_UNSUPPORTED = 2, /* valid per the equations but outside this library's limits */
  DYNCONV_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the size query */
  DYNCONV_ERR_HIP = 4          /* a HIP launch failed */
};

/* Human-readable name of a status code (static storage). */
const char* dynconv_status_string(dynconv_status s);

/* hipError_t (as int) of the calling thread's last DYNCONV_ERR_HIP, 0 if none. */
int dynconv_last_hip_error(void);

/*
 * Forward, eq. 2 + eq. 3 (eq. 1 when w is static).
 *   x  [B,T,D]      input activations (read once)
 *   w  [B,T,D/H,W]  per-token filters, or static [D/H,W] given by ws[0] == ws[1] == 0
 *   y  [B,T,D]      output, y = x + conv(x) (written once)
 */
dynconv_status dynconv_fwd(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                           void* y, const int64_t* ys, int64_t B, int64_t T, int64_t D, int32_t W,
                           int32_t H, dynconv_dtype dtype, void* stream);

/*
 * Backward of dynconv_fwd given dy = dL/dy (the exact adjoint of eq. 2 + eq. 3):
 *   dx[b,s,d]   = dy[b,s,d] + sum_k w[b,s+k,g(d),k] * dy[b,s+k,d]        (s + k < T)
 *   dw[b,t,g,k] = sum_{d : g(d) = g} dy[b,t,d] * x[b,t-k,d]              (0 for t < k)
 * x and w are independent inputs (the filters are generated from another tensor), so dx
 * has no term through w.
 *   dx  [B,T,D] or NULL to skip.
 *   dw  per-token filters: [B,T,D/H,W] with strides dws, dtype `dtype`, or NULL to skip.
 *       static w: float32 [D/H, W] contiguous, the sum over all (b, t); dws is ignored.
 * At least one of dx, dw must be non-NULL. A static w needs a workspace of
 * dynconv_bwd_workspace_size(...) bytes when dw is requested (per-tile partial sums,
 * reduced in a fixed order, so results are run-to-run deterministic).
 */
dynconv_status dynconv_bwd(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                           const void* dy, const int64_t* dys, void* dx, const int64_t* dxs, void* dw,
                           const int64_t* dws, int64_t B, int64_t T, int64_t D, int32_t W, int32_t H,
                           dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes needed by dynconv_bwd (0 unless the filter is static). */
size_t dynconv_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int is_static,
                                  dynconv_dtype dtype);

/*
 * Low-rank forward: filters w[b,t,g,k] = sum_r z[b,t,r] U[r, g*W+k] + bias[g*W+k] are
 * formed on the GPU (matrix cores, float32 accumulation) and applied at once; they are
 * never written to memory. Then y = x + conv(x) as in dynconv_fwd.
 *   z     [B,T,R] with strides zs
 *   U     [R, (D/H)*W] with row stride ldu (elements), column j = g*W + k
 *   bias  [(D/H)*W] or NULL (zero bias)
 * Row strides (xs[1], zs[1], ys[1], ldu; and dys[1], dxs[1] of the backward) must be below
 * 2^24 elements (DYNCONV_ERR_UNSUPPORTED otherwise).
 */
dynconv_status dynconv_lowrank_fwd(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                   const void* U, int64_t ldu, const void* bias, void* y, const int64_t* ys,
                                   int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int32_t R,
                                   dynconv_dtype dtype, void* stream);

/*
 * Low-rank backward. With g[b,t,j] = dw[b,t,g,k] (j = g*W + k) the per-token filter
 * gradient of dynconv_bwd (never written to memory):
 *   dx = as in dynconv_bwd with the generated filters,
 *   dz[b,t,r] = sum_j g[b,t,j] U[r,j],
 *   dU[r,j]   = sum_{b,t} z[b,t,r] g[b,t,j]   (float32 [R, (D/H)*W] contiguous, overwritten),
 *   db[j]     = sum_{b,t} g[b,t,j]            (float32 [(D/H)*W], overwritten; NULL to skip).
 * dx, dz and dU are required. Needs dynconv_lowrank_bwd_workspace_size(...) bytes of
 * workspace for fixed-order partial sums (run-to-run deterministic, no float atomics).
 */
dynconv_status dynconv_lowrank_bwd(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                   const void* U, int64_t ldu, const void* bias, const void* dy,
                                   const int64_t* dys, void* dx, const int64_t* dxs, void* dz,
                                   const int64_t* dzs, float* dU, float* db, int64_t B, int64_t T, int64_t D,
                                   int32_t W, int32_t H, int32_t R, dynconv_dtype dtype, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Workspace bytes needed by dynconv_lowrank_bwd. */
size_t dynconv_lowrank_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int32_t R,
                                          dynconv_dtype dtype);

/*
 * Inference: decoding one token at a time (the reading note lists inference among the
 * things it left unoptimised). A sequence keeps its last W-1 inputs in a rolling cache
 *   cache [B, W-1, D] with strides cs[0..2] (cs[2] == 1), dtype `dtype`,
 * where token s sits in slot s mod (W-1) and the slots of positions before 0 hold zeros
 * (the zero padding before t = 0). The cache is read and written in place. W == 1 needs
 * no cache (it may be NULL).
 */

/*
 * After a prompt of T tokens (y from dynconv_fwd or dynconv_lowrank_fwd on x [B,T,D]):
 * slot s mod (W-1) of each sequence receives x[b, s] for s = T-W+1 .. T-1, and zero for
 * s < 0 (so T == 0 empties the cache). Decoding then continues at t = T.
 */
dynconv_status dynconv_cache_fill(const void* x, const int64_t* xs, void* cache, const int64_t* cs, int64_t B,
                                  int64_t T, int64_t D, int32_t W, dynconv_dtype dtype, void* stream);

/*
 * One decoding step at token index t >= 0 (the same for every sequence of the batch):
 *   y[b,d] = x[b,d] + sum_{k<W} w[b,g(d),k] * x_{t-k}[b,d],   x_{t-k} from the cache for k >= 1,
 * after which x[b, :] is stored in slot t mod (W-1). Equal to row t of dynconv_fwd over the
 * whole sequence.
 *   x  [B, D] with strides xs[0..1] (xs[1] == 1)
 *   w  [B, D/H, W] with strides ws[0..2] (ws[2] == 1, ws[1] == W), or a static filter
 *      [D/H, W] given by ws[0] == 0
 *   y  [B, D] with strides ys[0..1] (ys[1] == 1); y may not be x, w or the cache.
 */
dynconv_status dynconv_decode_step(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                                   void* cache, const int64_t* cs, void* y, const int64_t* ys, int64_t t,
                                   int64_t B, int64_t D, int32_t W, int32_t H, dynconv_dtype dtype, void* stream);

/*
 * Low-rank decoding step: the filters of the new token, w[b,g,k] = sum_r z[b,r] U[r, g*W+k]
 * + bias[g*W+k], are formed on the GPU (float32) and applied as in dynconv_decode_step.
 *   z  [B, R] with strides zs[0..1] (zs[1] == 1); U, ldu, bias as in dynconv_lowrank_fwd.
 * 1 <= R <= 128, W <= 8.
 */
dynconv_status dynconv_lowrank_decode_step(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                           const void* U, int64_t ldu, const void* bias, void* cache,
                                           const int64_t* cs, void* y, const int64_t* ys, int64_t t, int64_t B,
                                           int64_t D, int32_t W, int32_t H, int32_t R, dynconv_dtype dtype,
                                           void* stream);

/*
 * Packed sequences (several documents in one row of x): the same calls with a segment id
 * per token,
 *   seq_idx  int32 [B,T] with strides ss[0..1] >= 0 (elements), 4-byte aligned,
 * after which tap k of token t is present only when seq_idx[b,t-k] == seq_idx[b,t]: a
 * document never reads the inputs of the one before it (the RubiConv page's point that
 * a convolution over packed sequences must not cross a document start). Documents are
 * normally contiguous runs of equal ids; any ids work, the test is equality. Gradients
 * are those of the masked forward. The bf16 fast low-rank kernels take packed calls whose
 * id rows are contiguous, 16-byte aligned and T % 4 == 0; others take the general kernels.
 * seq_idx == NULL returns DYNCONV_ERR_INVALID_ARG; every other argument is as in the call
 * without the suffix.
 */
dynconv_status dynconv_fwd_varlen(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                                  const int32_t* seq_idx, const int64_t* ss, void* y, const int64_t* ys, int64_t B,
                                  int64_t T, int64_t D, int32_t W, int32_t H, dynconv_dtype dtype, void* stream);

dynconv_status dynconv_bwd_varlen(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                                  const int32_t* seq_idx, const int64_t* ss, const void* dy, const int64_t* dys,
                                  void* dx, const int64_t* dxs, void* dw, const int64_t* dws, int64_t B, int64_t T,
                                  int64_t D, int32_t W, int32_t H, dynconv_dtype dtype, void* workspace,
                                  size_t workspace_bytes, void* stream);

dynconv_status dynconv_lowrank_fwd_varlen(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                          const void* U, int64_t ldu, const void* bias, const int32_t* seq_idx,
                                          const int64_t* ss, void* y, const int64_t* ys, int64_t B, int64_t T,
                                          int64_t D, int32_t W, int32_t H, int32_t R, dynconv_dtype dtype,
                                          void* stream);

dynconv_status dynconv_lowrank_bwd_varlen(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                          const void* U, int64_t ldu, const void* bias, const int32_t* seq_idx,
                                          const int64_t* ss, const void* dy, const int64_t* dys, void* dx,
                                          const int64_t* dxs, void* dz, const int64_t* dzs, float* dU, float* db,
                                          int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int32_t R,
                                          dynconv_dtype dtype, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * Optional convolution bias (the Conv1D module of the convolution technical report: a
 * per-channel bias c added to every output, y = x + conv(x) + c), together with optional
 * segment ids (seq_idx == NULL: one document per row, ss ignored):
 *   conv_bias   [D] of `dtype`, contiguous, 4-byte aligned, or NULL
 *   dconv_bias  [D] float32, overwritten with sum over (b, t) of dy (NULL to skip)
 * The backward's workspace then holds float32 partial sums of dy per (sequence, time
 * chunk) after those of a static filter: size it with dynconv_bwd_ex_workspace_size.
 * Materialised, static and head-wise forms (the low-rank form: dynconv_lowrank_*_ex below);
 * the decoding step adds c to its output.
 */
dynconv_status dynconv_fwd_ex(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                              const int32_t* seq_idx, const int64_t* ss, const void* conv_bias, void* y,
                              const int64_t* ys, int64_t B, int64_t T, int64_t D, int32_t W, int32_t H,
                              dynconv_dtype dtype, void* stream);

size_t dynconv_bwd_ex_workspace_size(int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int is_static,
                                     int want_dconv_bias, dynconv_dtype dtype);

dynconv_status dynconv_bwd_ex(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                              const int32_t* seq_idx, const int64_t* ss, const void* dy, const int64_t* dys, void* dx,
                              const int64_t* dxs, void* dw, const int64_t* dws, float* dconv_bias, int64_t B,
                              int64_t T, int64_t D, int32_t W, int32_t H, dynconv_dtype dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

dynconv_status dynconv_decode_step_ex(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                                      const void* conv_bias, void* cache, const int64_t* cs, void* y,
                                      const int64_t* ys, int64_t t, int64_t B, int64_t D, int32_t W, int32_t H,
                                      dynconv_dtype dtype, void* stream);

/*
 * The same optional convolution bias on the low-rank form (y = x + conv(x) + c with the
 * generated filters), together with optional segment ids (seq_idx == NULL: one document
 * per row, ss ignored); every other argument is as in dynconv_lowrank_{fwd,bwd} and
 * dynconv_lowrank_decode_step.
 *   conv_bias   [D] of `dtype`, contiguous, 4-byte aligned (decoding step: element
 *               aligned), or NULL
 *   dconv_bias  [D] float32, 4-byte aligned, overwritten with sum over (b, t) of dy (NULL
 *               to skip); its float32 partial sums per (sequence, chunk of tokens) take
 *               workspace after those of dU and db: size the workspace with
 *               dynconv_lowrank_bwd_ex_workspace_size(..., want_dconv_bias = 1, ...).
 * The bias gradient reads dy once more (one extra pass over B*T*D elements).
 */
dynconv_status dynconv_lowrank_fwd_ex(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                      const void* U, int64_t ldu, const void* bias, const int32_t* seq_idx,
                                      const int64_t* ss, const void* conv_bias, void* y, const int64_t* ys, int64_t B,
                                      int64_t T, int64_t D, int32_t W, int32_t H, int32_t R, dynconv_dtype dtype,
                                      void* stream);

size_t dynconv_lowrank_bwd_ex_workspace_size(int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, int32_t R,
                                             int want_dconv_bias, dynconv_dtype dtype);

dynconv_status dynconv_lowrank_bwd_ex(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                      const void* U, int64_t ldu, const void* bias, const int32_t* seq_idx,
                                      const int64_t* ss, const void* dy, const int64_t* dys, void* dx,
                                      const int64_t* dxs, void* dz, const int64_t* dzs, float* dU, float* db,
                                      float* dconv_bias, int64_t B, int64_t T, int64_t D, int32_t W, int32_t H,
                                      int32_t R, dynconv_dtype dtype, void* workspace, size_t workspace_bytes,
                                      void* stream);

dynconv_status dynconv_lowrank_decode_step_ex(const void* x, const int64_t* xs, const void* z, const int64_t* zs,
                                              const void* U, int64_t ldu, const void* bias, const void* conv_bias,
                                              void* cache, const int64_t* cs, void* y, const int64_t* ys, int64_t t,
                                              int64_t B, int64_t D, int32_t W, int32_t H, int32_t R,
                                              dynconv_dtype dtype, void* stream);

/*
 * The convolution in the epilogue of the producing projection (the reading note's
 * end-to-end throughput section, closing analysis: fusing the dynamic convolution into
 * the matmul epilogue removes memory traffic; its "Parameterization" section puts the
 * convolution on the QKV projection's outputs). One kernel computes
 *   X = A W_p^T          (the projection; X is never written to memory)
 *   y = X + conv(X)      (eq. 2 + eq. 3 on X, zeros before t = 0 of every sequence)
 * with float32 accumulation (X is not rounded before the convolution).
 *   A   [B,T,K] activations with strides as[0..2], as[2] == 1
 *   Wp  [N,K] projection weight (a linear layer's out x in layout), rows ldw apart
 *   y   [B,T,N] with strides ys[0..2], ys[2] == 1
 * dynconv_gemm_fwd takes per-token filters w [B,T,N/H,W] (strides ws, ws[3] == 1,
 * ws[2] == W; ws[0] == ws[1] == 0: a static [N/H,W] filter); dynconv_gemm_lowrank_fwd
 * forms them as w = z U + bias on the matrix cores (z [B,T,R] strides zs, zs[2] == 1;
 * U [R,(N/H)*W] rows ldu apart, column g*W + k; bias [(N/H)*W] or NULL).
 * Limits (DYNCONV_ERR_UNSUPPORTED otherwise): bfloat16 or float16; 1 <= W <= 5;
 * H in {1, 2, 4, 8, 16}; K a positive multiple of 64; N a multiple of 128; B*T < 2^31;
 * A and W_p rows 16-byte aligned (base, as[0], as[1], ldw); low-rank: R <= 128 with
 * W * (32 ceil(R/32) + 8) <= 552 (R <= 128 at W <= 4, R <= 96 at W = 5).
 * y may not be any input (DYNCONV_ERR_INVALID_ARG). Forward only.
 */
dynconv_status dynconv_gemm_fwd(const void* A, const int64_t* as, const void* Wp, int64_t ldw, const void* w,
                                const int64_t* ws, void* y, const int64_t* ys, int64_t B, int64_t T, int64_t N,
                                int64_t K, int32_t W, int32_t H, dynconv_dtype dtype, void* stream);

dynconv_status dynconv_gemm_lowrank_fwd(const void* A, const int64_t* as, const void* Wp, int64_t ldw, const void* z,
                                        const int64_t* zs, const void* U, int64_t ldu, const void* bias, void* y,
                                        const int64_t* ys, int64_t B, int64_t T, int64_t N, int64_t K, int32_t W,
                                        int32_t H, int32_t R, dynconv_dtype dtype, void* stream);

/*
 * Allocation-free backward, for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc). The same
 * operation and arguments as dynconv_bwd_ex, without a workspace: the float32 partial
 * sums of a static filter's dw and of dconv_bias go to a scratch array that the library
 * holds in device memory, DYNCONV_NOALLOC_SCRATCH_BYTES per GPU, kept from the library's
 * load until the process ends. Calls that need no partial sums (per-token filters without
 * dconv_bias) do not touch it.
 *   - A call whose partial sums need more than DYNCONV_NOALLOC_SCRATCH_BYTES (the bytes
 *     dynconv_bwd_ex_workspace_size reports) returns DYNCONV_ERR_WORKSPACE.
 *   - The scratch array of the CURRENT device is used: `stream` must belong to it. Its
 *     device address is resolved on the first call on each device (hipGetSymbolAddress),
 *     so that first call must not be made during a graph capture.
 *   - Every call on a GPU shares that GPU's array: calls that overlap in time on one GPU
 *     (on different streams, or from different threads without ordering) race and give
 *     wrong sums. Calls ordered on one stream are safe; each call overwrites every
 *     partial it later reads, so nothing has to start at zero.
 *   - No hipMalloc, hipFree or allocating library routine is called.
 */
#define DYNCONV_NOALLOC_SCRATCH_BYTES (16u << 20)

dynconv_status dynconv_bwd_ex_noalloc(const void* x, const int64_t* xs, const void* w, const int64_t* ws,
                                      const int32_t* seq_idx, const int64_t* ss, const void* dy, const int64_t* dys,
                                      void* dx, const int64_t* dxs, void* dw, const int64_t* dws, float* dconv_bias,
                                      int64_t B, int64_t T, int64_t D, int32_t W, int32_t H, dynconv_dtype dtype,
                                      void* stream);

/*
 * Cache fill after a packed prompt: decoding continues the document of token T-1, so the
 * slots of tokens with another segment id than token T-1 are zero (the start of that
 * document). T == 0 empties the cache as in dynconv_cache_fill.
 */
dynconv_status dynconv_cache_fill_varlen(const void* x, const int64_t* xs, const int32_t* seq_idx, const int64_t* ss,
                                         void* cache, const int64_t* cs, int64_t B, int64_t T, int64_t D, int32_t W,
                                         dynconv_dtype dtype, void* stream);

/*
 * Gated delta rule: the recurrence that consumes the convolved q, k, v in linear-attention
 * models (the reading note's linear-attention experiments put the dynamic convolution in
 * Gated DeltaNet). Per sequence b and value head h, with a_t = exp(g[b,t,h]), the key head
 * h / (Hv/Hk) shared by Hv/Hk consecutive value heads, and a float32 state S [dk, dv]:
 *   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,
 *   o_t = scale S_t^T q_t.
 *   q, k   [B,T,Hk,dk], v, o [B,T,Hv,dv] of `dtype`, strides s[0..3], s[3] == 1
 *   beta   [B,T,Hv] of `dtype`, g float32 [B,T,Hv] (log decay, normally <= 0), strides s[0..2]
 *   qk_norm_eps >= 0: q and k are divided by sqrt(|.|^2 + qk_norm_eps) first (the sum of squares
 *            in float32; with 0 a row of zeros is 0 / 0); < 0: as given; NaN is refused
 *   seq_idx  int32 [B,T] (strides ss[0..1]) or NULL: the state is reset to zero before a
 *            token whose id differs from the token's before it (document starts of packed
 *            rows); the initial state belongs to the first document of a row, the final
 *            state to the last
 *   state_in   float32 [B,Hv,dk,dv] (strides [0..3], last 1) or NULL (zero)
 *   state_out  the same, overwritten with the state after token T-1, or NULL; may be
 *              state_in itself (same strides). T == 0 copies the state.
 * A token with beta = 0 and g = 0 leaves the state as it is (padding behind a sequence, whose
 * q, k, v have to be finite, and q and k not zero when qk_norm_eps is 0).
 * A g whose exp is 0 in float32 (below -103.97) is a decay to exactly zero. Tokens are worked
 * on 64 at a time: a NaN or infinity among a head's inputs can reach every output of its
 * 64-token chunk and of what follows, other documents included; other heads keep theirs.
 * Limits (DYNCONV_ERR_UNSUPPORTED otherwise): dk <= 128, dv <= 65536; strides >= 0, token
 * strides (s[1]) of q, k, v, o and their gradients below 2^22 elements (with T == 1 they are not
 * used), B Hv ceil(dv/32) below 2^23. With another size than T of 0 nothing is read or written.
 * Inputs and outputs need element alignment; rows of q, k that allow 16-byte loads are read so.
 * Needs dynconv_delta_fwd_workspace_size(...) bytes of workspace. Run-to-run deterministic.
 */
dynconv_status dynconv_delta_fwd(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                 const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                 const int64_t* bs, const int32_t* seq_idx, const int64_t* ss, const float* state_in,
                                 const int64_t* sis, void* o, const int64_t* os, float* state_out, const int64_t* sos,
                                 int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale,
                                 float qk_norm_eps, dynconv_dtype dtype, void* workspace, size_t workspace_bytes,
                                 void* stream);

size_t dynconv_delta_fwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                        dynconv_dtype dtype);

/*
 * Backward of dynconv_delta_fwd given dO = dL/do [B,T,Hv,dv] and, optionally, the gradient of
 * the final state (dstate_out float32 [B,Hv,dk,dv], or NULL): the exact adjoints
 *   dq, dk    [B,T,Hk,dk] (through the normalisation; summed over the value heads of a key head)
 *   dv        [B,T,Hv,dv], dbeta [B,T,Hv] of `dtype`
 *   dg        float32 [B,T,Hv] (0 at a document start and where exp(g) is 0)
 *   dstate_in float32 [B,Hv,dk,dv], the gradient of the initial state, or NULL to skip.
 * States are recomputed from the inputs; nothing is kept from the forward. Needs
 * dynconv_delta_bwd_workspace_size(...) bytes (per 64 tokens and value head 20 KiB +
 * (8 dk' + 528) dv, with dk rounded up to dk' = 64 or 128 and dv to a multiple of 16, and what
 * the segments of long sequences take). T == 0 is a no-op.
 */
dynconv_status dynconv_delta_bwd(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                 const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                 const int64_t* bs, const int32_t* seq_idx, const int64_t* ss, const float* state_in,
                                 const int64_t* sis, const void* dO, const int64_t* dos, const float* dstate_out,
                                 const int64_t* dsos, void* dq, const int64_t* dqs, void* dk_, const int64_t* dks,
                                 void* dv_, const int64_t* dvs, float* dg, const int64_t* dgs, void* dbeta,
                                 const int64_t* dbs, float* dstate_in, const int64_t* dsis, int64_t B, int64_t T,
                                 int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale, float qk_norm_eps,
                                 dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_delta_bwd_workspace_size(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                        dynconv_dtype dtype);

/*
 * One decoding step of the gated delta rule: one token of every sequence, the state updated
 * in place (equal to dynconv_delta_fwd with T = 1).
 *   q, k [B,Hk,dk], v, o [B,Hv,dv] strides s[0..2] (s[2] == 1), g, beta [B,Hv] strides
 *   s[0..1], state float32 [B,Hv,dk,dv] strides sts[0..3] (sts[3] == 1).
 */
dynconv_status dynconv_delta_step(const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                                  const int64_t* vs, const float* g, const int64_t* gs, const void* beta,
                                  const int64_t* bs, float* state, const int64_t* sts, void* o, const int64_t* os,
                                  int64_t B, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, float scale,
                                  float qk_norm_eps, dynconv_dtype dtype, void* stream);

/*
 * RMS norm over the last dimension with a weight, a SiLU gate and a scaled residual: the norm
 * behind the gated delta rule (per head, gated) and the norms before and after a block.
 *   n = x / sqrt(mean(x^2) + eps),  y = n * weight * silu(gate)
 * With a residual and residual_after == 0 (the norm before a block, fused with the addition):
 *   h = residual + residual_scale * x, rounded to `dtype` and written, takes x's place.
 * With a residual and residual_after != 0 (the norm after a block):
 *   y = residual + residual_scale * n * weight * silu(gate).
 *   x, gate, residual, y, h  [n0,n1,n2,D] of `dtype`, strides s[0..3] (elements, >= 0, s[3] == 1);
 *                            gate and residual may be NULL; h is required (and only used)
 *                            with a residual before
 *   weight                   [D] of `dtype`, contiguous, or NULL (ones)
 * Any D up to 2^24; element alignment (rows that allow 16-byte accesses use them). Sums are
 * held to float32 accuracy for any D. y and h may not be an input or each other (DYNCONV_ERR_INVALID_ARG).
 */
dynconv_status dynconv_norm_fwd(const void* x, const int64_t* xs, const void* weight, const void* gate,
                                const int64_t* gs, const void* residual, const int64_t* rs, int32_t residual_after,
                                float residual_scale, void* y, const int64_t* ys, void* h, const int64_t* hs, int64_t n0,
                                int64_t n1, int64_t n2, int64_t D, float eps, dynconv_dtype dtype, void* stream);

enum { DYNCONV_NORM_NO_RESIDUAL = 0, DYNCONV_NORM_RESIDUAL_BEFORE = 1, DYNCONV_NORM_RESIDUAL_AFTER = 2 };

/*
 * Backward of dynconv_norm_fwd given dy:
 *   x          what was normalised: the forward's x, or its h with the residual before
 *   dh         gradient of h from its other uses, or NULL (residual before only)
 *   dx         gradient of the forward's x
 *   dresidual  gradient of the residual (before only), or NULL to skip. With the residual
 *              after it is dy itself and not written.
 *   dweight    float32 [D], overwritten, or NULL to skip; needs
 *              dynconv_norm_bwd_workspace_size(...) bytes of workspace (fixed-order partial
 *              sums, run-to-run deterministic). Without rows it is zero.
 *   dgate      gradient of the gate; required with a gate
 */
dynconv_status dynconv_norm_bwd(const void* x, const int64_t* xs, const void* weight, const void* gate,
                                const int64_t* gs, const void* dy, const int64_t* dys, const void* dh,
                                const int64_t* dhs, int32_t residual_at, float residual_scale, void* dx,
                                const int64_t* dxs, void* dresidual, const int64_t* drs, float* dweight, void* dgate,
                                const int64_t* dgs, int64_t n0, int64_t n1, int64_t n2, int64_t D, float eps,
                                dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_norm_bwd_workspace_size(int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype);

/*
 * Gated linear scan: the recurrence per channel that a linear-recurrent layer puts behind its
 * convolution. With s_t = sigmoid(decay_t):
 *   a_t = exp(-rate s_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t,  y_t = h_t.
 *   x, decay, gate, y  [B,T,D] of `dtype`, strides s[0..2] (elements, >= 0, s[2] == 1); gate may be
 *             NULL (a factor of 1)
 *   rate      float32 [D], contiguous, >= 0 (a negative one gives NaN)
 *   seq_idx   int32 [B,T] (strides ss[0..1]) or NULL: the state restarts from zero at a token whose id
 *             differs from the one's before it; the initial state belongs to a row's first document,
 *             the final state to its last
 *   state_in  float32 [B,D] (strides [0..1], last 1) or NULL (zero)
 *   state_out the same, overwritten with the state after token T-1, or NULL; may be state_in itself
 *             (same strides). T == 0 copies the state.
 *   chunks    float32 [B, ceil(T/128), D], contiguous, overwritten with the state before every 128th
 *             token (0, 128, ...), for the backward; or NULL
 * The states are float32 whatever the `dtype`. A NaN or infinity stays in its channel and document.
 * Limits (DYNCONV_ERR_UNSUPPORTED otherwise): D <= 2^24, B ceil(D/64) < 2^22; token strides below 2^22
 * elements (with T == 1 they are not used). Element alignment; 16-bit types go two channels at a time where
 * D and all strides are even and the pointers aligned to two elements.
 * Few channels and long sequences need dynconv_scan_fwd_workspace_size(...) bytes of workspace
 * (aligned to 8; 0 for most calls). Run-to-run deterministic.
 */
dynconv_status dynconv_scan_fwd(const void* x, const int64_t* xs, const void* decay, const int64_t* as, const void* gate,
                                const int64_t* gs, const float* rate, const int32_t* seq_idx, const int64_t* ss,
                                const float* state_in, const int64_t* sis, void* y, const int64_t* ys, float* state_out,
                                const int64_t* sos, float* chunks, int64_t B, int64_t T, int64_t D, dynconv_dtype dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, dynconv_dtype dtype);

/*
 * Backward of dynconv_scan_fwd given dy [B,T,D] and, optionally, the gradient of the final state
 * (dstate_out float32 [B,D], or NULL):
 *   x, decay, gate  the forward's; or, with scales, int8 codes of them as dynconv_pack writes them
 *              (x_scales, decay_scales and, with a gate, gate_scales: uint8 [B,T,ceil(D/64)], strides
 *              [0..2], last 1; all or none): the gradients are then those at the values the codes stand for
 *   chunks     what the forward wrote, or NULL: the states are then recomputed from the inputs (one
 *              more reading of x, decay and gate; state_in is only used here). NULL with scales
 *              (DYNCONV_ERR_INVALID_ARG otherwise): the forward's states are of other inputs
 *   dx, ddecay, dgate  [B,T,D] of `dtype`; dgate is required with a gate
 *   drate      float32 [D], overwritten (sums in 64 bits in a fixed order)
 *   dstate_in  float32 [B,D], the gradient of the initial state, or NULL to skip
 * Where 1 - a^2 is below 2^-126 (rate or s of nearly 0) it counts as 0, here as in the other calls, and the
 * derivative of its root as 0. Without tokens drate is zero and dstate_in a copy of dstate_out. Needs
 * dynconv_scan_bwd_workspace_size(...) bytes (aligned to 8; with_chunks: whether chunks are given).
 */
dynconv_status dynconv_scan_bwd(const void* x, const int64_t* xs, const void* decay, const int64_t* as, const void* gate,
                                const int64_t* gs, const uint8_t* x_scales, const int64_t* xcs,
                                const uint8_t* decay_scales, const int64_t* acs, const uint8_t* gate_scales,
                                const int64_t* gcs, const float* rate, const int32_t* seq_idx, const int64_t* ss,
                                const float* state_in, const int64_t* sis, const float* chunks, const void* dy,
                                const int64_t* dys, const float* dstate_out, const int64_t* dsos, void* dx,
                                const int64_t* dxs, void* ddecay, const int64_t* das, float* drate, void* dgate,
                                const int64_t* dgs, float* dstate_in, const int64_t* dsis, int64_t B, int64_t T,
                                int64_t D, dynconv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int32_t with_chunks, dynconv_dtype dtype);

/*
 * One decoding step of the gated linear scan: one token of every sequence, the state updated in
 * place. x, decay, gate, y [B,D] of `dtype`, strides s[0..1] (s[1] == 1); state float32 [B,D].
 */
dynconv_status dynconv_scan_step(const void* x, const int64_t* xs, const void* decay, const int64_t* as,
                                 const void* gate, const int64_t* gs, const float* rate, float* state,
                                 const int64_t* sts, void* y, const int64_t* ys, int64_t B, int64_t D,
                                 dynconv_dtype dtype, void* stream);

/*
 * Activations in 8 bits: what a training step keeps for its backward pass. Every 64 channels of a row
 * share a step, the power of two 2^(floor(log2 max|x|) - 6) (at least 2^-126); a value is an integer code
 * of -127 to 127 (nearest, ties to even) times the step. Off by at most 2^-7 of the group's largest
 * value; a group with a NaN or infinity reads back as NaN, whole.
 *   x       [n0,n1,n2,D] of `dtype`, strides s[0..3] (s[3] == 1)
 *   codes   int8 of the same shape, strides cs[0..3] (cs[3] == 1)
 *   scales  uint8 [n0,n1,n2,ceil(D/64)], strides ss[0..3] (ss[3] == 1): the step's float32 exponent field
 * dynconv_unpack writes code times step, which `dtype` holds exactly when it is the type that was
 * packed (or float32). Backward calls that take scales read the codes themselves.
 */
dynconv_status dynconv_pack(const void* x, const int64_t* xs, int8_t* codes, const int64_t* cs, uint8_t* scales,
                             const int64_t* ss, int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype,
                             void* stream);

dynconv_status dynconv_unpack(const int8_t* codes, const int64_t* cs, const uint8_t* scales, const int64_t* ss, void* y,
                               const int64_t* ys, int64_t n0, int64_t n1, int64_t n2, int64_t D, dynconv_dtype dtype,
                               void* stream);

/*
 * Group norm, channels last, with weight, bias, SiLU and a SiLU gate:
 *   n = (x - mean) / sqrt(var + eps),  y = act(n weight + bias) silu(gate)
 * The mean and the variance run over the C/groups neighbouring channels of a group: of each token, or
 * (over_sequence != 0) of all tokens of a sequence. act is SiLU with silu != 0, else nothing.
 *   x, gate, y    [B,T,C] of `dtype`, strides s[0..2] (elements, >= 0, s[2] == 1); gate may be NULL (1)
 *   weight, bias  [C] of `dtype`, contiguous, or NULL (ones, zeros)
 *   lengths       int32 [B], contiguous, or NULL (T); over sequences only: the tokens of a sequence,
 *                 cut to 0..T. Tokens behind them are not in the statistics, and their y is 0.
 *   stats         float32 [B,groups,2], overwritten with mean and 1 / sqrt(var + eps) (0, 0 for a
 *                 sequence without tokens) for the backward, or NULL; over sequences only
 * The statistics' sums over a sequence are held in 64 bits, those over a token's group in 32 (in 64 for groups longer
 * than the registers take). C up to 2^19, B below 2^23, B T below 2^31. Element alignment; 16 bytes at a time where
 * C/groups, all strides and pointers allow it. Over sequences needs
 * dynconv_groupnorm_fwd_workspace_size(...) bytes (aligned to 8), per token none. Run-to-run deterministic.
 */
dynconv_status dynconv_groupnorm_fwd(const void* x, const int64_t* xs, const void* weight, const void* bias,
                                     const void* gate, const int64_t* gs, const int32_t* lengths, void* y,
                                     const int64_t* ys, float* stats, int64_t B, int64_t T, int64_t C, int64_t groups,
                                     int32_t over_sequence, int32_t silu, float eps, dynconv_dtype dtype,
                                     void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_groupnorm_fwd_workspace_size(int64_t B, int64_t T, int64_t C, int64_t groups, int32_t over_sequence,
                                            int32_t with_stats, dynconv_dtype dtype);

/*
 * Backward of dynconv_groupnorm_fwd given dy:
 *   x        the forward's, or, with x_scales (uint8 [B,T,ceil(C/64)], strides xcs[0..2], last 1), its int8
 *            codes as dynconv_pack writes them: the gradients are then those at the values they stand for
 *   stats    what the forward wrote, or NULL: recomputed from x (over sequences only). NULL with x_scales
 *            (DYNCONV_ERR_INVALID_ARG otherwise): the forward's are of another x
 *   dx       [B,T,C] of `dtype`; 0 behind a sequence's tokens
 *   dweight, dbias  float32 [C], overwritten, or NULL to skip (without tokens zero)
 *   dgate    required with a gate; 0 behind a sequence's tokens
 * The sums over tokens, from which over sequences the groups' means of the gradient follow too, are held in 32 bits
 * over a workgroup's tokens, at most 512 of each lane, and in 64 over the workgroups.
 * Needs dynconv_groupnorm_bwd_workspace_size(...) bytes (aligned to 8; per token only for dweight or dbias).
 */
dynconv_status dynconv_groupnorm_bwd(const void* x, const int64_t* xs, const uint8_t* x_scales, const int64_t* xcs,
                                     const void* weight, const void* bias, const void* gate, const int64_t* gs,
                                     const int32_t* lengths, const float* stats, const void* dy, const int64_t* dys,
                                     void* dx, const int64_t* dxs, float* dweight, float* dbias, void* dgate,
                                     const int64_t* dgs, int64_t B, int64_t T, int64_t C, int64_t groups,
                                     int32_t over_sequence, int32_t silu, float eps, dynconv_dtype dtype,
                                     void* workspace, size_t workspace_bytes, void* stream);

size_t dynconv_groupnorm_bwd_workspace_size(int64_t B, int64_t T, int64_t C, int64_t groups, int32_t over_sequence,
                                            int32_t with_stats, dynconv_dtype dtype);

#ifdef __cplusplus
}
#endif

#endif /* DYNCONV_H */
