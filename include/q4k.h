/*
 * q4k — matrix products against GGUF Q4_K block-quantized weights on GB300 (sm_103a).
 *
 * The operation.  A GGUF serving target "dequantizes Q4_K into the matrix-multiply
 * operand" on every prefill pass, a fixed cost that dominates at 128 tokens and is
 * amortized by 4k (sparkinfer-server README, "Serve a GGUF instead of NVFP4").
 * Decode runs the same projections with one token per lane, and speculative
 * verification with 1 + draft tokens per lane (ninfer serving docs, "Start the
 * server": --draft-tokens N, MTP 1..5, DFlash 1..15; "Determinism": decode kernels
 * are chosen by the step's token count).  A routed MoE layer ends in a weighted
 * combine of its experts' down projections (sparkinfer-server README,
 * "Determinism").  This library computes exactly those products:
 *
 *     y[m][n] = sum_k x[m][k] * w[n][k]
 *
 * with w an N x K matrix stored as GGUF Q4_K blocks, x bf16 activations and y fp32.
 *
 * Q4_K block (144 bytes, 256 consecutive weights of one row; public GGUF format):
 *     [0,2) d (fp16)  [2,4) dmin (fp16)  [4,16) scales[12]  [16,144) qs[128]
 *     eight 6-bit (sc_j, m_j) pairs:  j < 4: sc = scales[j] & 63, m = scales[j+4] & 63
 *                 j >= 4: sc = (scales[j+4] & 15) | (scales[j-4] >> 6) << 4
 *                          m = (scales[j+4] >> 4) | (scales[j]   >> 6) << 4
 *     qs[32g+l]: low nibble = code of weight 64g+l, high nibble = weight 64g+32+l
 *     weight 32s+l = d*sc_s*q - dmin*m_s
 *
 * Matrix layout.  Row n of w (output feature n) is K/256 consecutive blocks;
 * rows are consecutive, so row n starts at byte n*q4k_row_bytes(K).  K must be a
 * positive multiple of 256.  x is row-major [M][ldx] bf16 (uint16 bit patterns),
 * y is row-major [M][ldy] fp32.
 *
 * Conventions for every call.
 *   - All data pointers are DEVICE pointers owned by the caller.  The library keeps
 *     no pointer after it returns.  Scratch memory, where a call needs it, is the
 *     caller's `ws` buffer; no call allocates device memory.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL is
 *     the legacy default stream) and enqueue their kernels in order on it.
 *   - Outputs are overwritten (never accumulated into).
 *   - Arguments are validated on the host before anything is launched; a call that
 *     returns an error has enqueued nothing.  Q4K_ERR_NULL: a required pointer is
 *     NULL.  Q4K_ERR_SHAPE: a size is out of range (K % 256 != 0, N or M < 1,
 *     ldx < K, ldy < N, ...).  Q4K_ERR_ALIGN: a pointer or leading dimension breaks
 *     the alignment stated for it.  Q4K_ERR_WORKSPACE: ws is smaller than the size
 *     query returns.  Q4K_ERR_DEVICE: the current device is not compute capability
 *     10.3.  Q4K_ERR_CUDA: a CUDA runtime call failed (q4k_last_cuda_error() gives
 *     the cudaError_t, per thread).
 *   - Faults inside a kernel surface at the caller's next synchronization, as with
 *     any CUDA library.  No kernel spins without a bound: a wait that runs past
 *     its limit records Q4K_ERR_TIMEOUT in a device status word and the kernel
 *     returns; q4k_check_device() reports and clears it.
 *   - Every result is run-to-run deterministic: no floating-point atomics, fixed
 *     reduction orders.
 */
#ifndef Q4K_H
#define Q4K_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    Q4K_OK = 0,
    Q4K_ERR_NULL = 1,
    Q4K_ERR_SHAPE = 2,
    Q4K_ERR_ALIGN = 3,
    Q4K_ERR_WORKSPACE = 4,
    Q4K_ERR_DEVICE = 5,
    Q4K_ERR_CUDA = 6,
    Q4K_ERR_TIMEOUT = 7,
    Q4K_ERR_ROUTING = 8,
    Q4K_ERR_INDEX = 10 /* 9 is not assigned */
} q4k_status;

/* Static English text for a status code; never NULL. */
const char *q4k_status_string(int status);

/* The cudaError_t behind this thread's most recent Q4K_ERR_CUDA (0 if none). */
int q4k_last_cuda_error(void);

/* Bytes of one Q4_K row of K weights: K/256*144; 0 if K is not a positive
 * multiple of 256. */
size_t q4k_row_bytes(int64_t K);

/* Library version as major*10000 + minor*100 + patch. */
int q4k_version(void);

/* Synchronizes `stream`, then reads and clears the device status word that the
 * kernels set when a bounded wait gives up (Q4K_ERR_TIMEOUT) or when a call of
 * q4k_moe_grouped_gemm_reuse_routing found no routing for its shape in its
 * workspace (Q4K_ERR_ROUTING), or when a call on a paged cache read an index from
 * device memory that is out of range (Q4K_ERR_INDEX).  The first of these, in this
 * order, that was recorded since the last check is reported.  Returns Q4K_OK, one
 * of those three, or Q4K_ERR_CUDA if the synchronization itself failed. */
q4k_status q4k_check_device(void *stream);

/* Declares whether the weight matrices read by the small-M calls (q4k_gemv,
 * q4k_gemm with M <= 16, q4k_gemm_x8, q4k_nvfp4_gemm with M <= 16, and the down
 * projection of q4k_moe_ffn with at most 16 items) are static: never written by
 * the kernel enqueued on the same stream immediately before the call.  Every kernel of the library is
 * launched so that it may start while the previous kernel on its stream drains,
 * and it waits for that kernel to finish before it touches memory.  With static
 * weights on, the small-M kernels already copy their first weight blocks into
 * shared memory during that wait, which hides part of each call's start-up
 * (about 1.5 us on a 50 MB GEMV).  In q4k_moe_ffn the down projection then also
 * reads topk_ids early; its gate/up kernel has already waited for the ids' writer
 * by then.  That is the usual inference setting: weights
 * are uploaded once, by copies, and only read afterwards.  Keep it off (the
 * default) when a kernel may write a weight buffer right before a q4k call reads
 * it, for example a fill or an on-device quantization kernel: the early copies
 * could then see the old contents.  Activations and outputs are never touched
 * early.  Process-wide; applies to calls enqueued after it returns.  Returns the
 * previous setting (0 or 1). */
int q4k_set_static_weights(int enable);

/* Batch-invariant mode.  The pages' serving engines pick their decode kernels by
 * the step's token count, so a token's logits can change with how many tokens
 * share the step; their deterministic mode removes that for a small cost
 * (sparkinfer-server README, "Determinism").  Here every call is run-to-run
 * deterministic in either mode; this switch is about batch invariance:
 *   off (default): M = 1 runs the decode GEMV kernel (sub-blocks in the MMA
 *       columns: the fastest one-token form), whose rounding differs from the
 *       2..16-token kernel's (both within the small-M bar).  Rows of calls with
 *       2 <= M <= 16 tokens equal each other bit for bit.
 *   on: M = 1 runs the 2..16-token kernel as well, so row m of any call with
 *       M <= 16 equals the one-token call on row m bit for bit.  Calls with
 *       M > 16 (the tensor-core path of q4k_gemm and q4k_nvfp4_gemm) split K
 *       in two or not at all, as the weight shape alone dictates (never by M),
 *       and split off no last-wave launch, so a token's row has the same bits
 *       in every call of 17 tokens or more, wherever it sits in the batch.  The
 *       two K halves are summed over a thread-block cluster pair, half 0 plus
 *       half 1.
 *       Cost: none where the weight rows fill the GPU without a K split (the
 *       K 5120 -> N 17408 prefill shape); on the narrow K 17408 -> N 5120 shape
 *       about +34 % time at 128 tokens, +25 % at 1024, +22 % at 4096 on one
 *       GB300.
 * The boundary between the two paths stays: rows of calls with M <= 16 and
 * M > 16 differ in rounding (different kernels, each within its bar).
 * Of the operators between the products, q4k_norm_residual and q4k_norm_residual_x8
 * follow the mode (about 0.15 us for a few rows); q4k_kv_append, q4k_kv_evict, q4k_sample
 * and q4k_batch_plan (whole numbers) give a token or sequence the same bits in either; a
 * row of q4k_lora_add depends in either on T, not on the other rows' content; q4k_attn_decode and
 * q4k_attn_chunk are not batch-invariant in either: they split their work by all lengths
 * of the batch.
 * Process-wide; applies to calls enqueued after it returns.  Returns the previous
 * setting (0 or 1). */
int q4k_set_batch_invariant(int enable);

/* Failure-detection test hook (no counterpart on the pages).  Every wait inside
 * the kernels is bounded (2 s); a wait that runs out makes its kernel abandon
 * its work, wait for its own copies in flight, reach all of its barriers and
 * set a device status word that q4k_check_device reports as Q4K_ERR_TIMEOUT.
 * This sets the limit of the decode GEMV's main-loop waits (q4k_gemv, and
 * q4k_gemm with M = 1 outside batch-invariant mode) and of q4k_norm_residual's and
 * q4k_norm_residual_x8's waits for their ring of rows to `ns`, so that a test can make
 * those paths run out without faulting or hanging anything; 0 restores the standard limit.  Under
 * 1000 ns a wait tests its copy once, without blocking, and gives up at once if it
 * has not landed.  A call whose wait ran out leaves its outputs undefined.
 * Process-wide; applies to calls enqueued after it returns.  Returns the
 * previous setting (0 = standard). */
unsigned long long q4k_set_gemv_wait_limit_ns(unsigned long long ns);

/* ----------------------------------------------------------------- dequant --
 * Standalone dequantization of an N x K Q4_K matrix:
 *     out[n][k] = d*sc_s*q - dmin*m_s   (fp32, computed as fp32 multiplies and one
 *                                        final fp32 subtraction: bit-exact)
 * q4k_dequant_bf16 stores the round-to-nearest-even bf16 of that fp32 value.
 * This is the "dequantize Q4_K into the matrix-multiply operand" step of the
 * sparkinfer-server README ("Serve a GGUF instead of NVFP4") on its own.
 *   w    device, N*q4k_row_bytes(K) bytes, 16-byte aligned
 *   out  device, N*K elements, row-major, 16-byte aligned
 * Errors: NULL, SHAPE (N < 1, bad K), ALIGN, DEVICE, CUDA. */
q4k_status q4k_dequant(const void *w, int64_t N, int64_t K, float *out, void *stream);
q4k_status q4k_dequant_bf16(const void *w, int64_t N, int64_t K, uint16_t *out, void *stream);

/* -------------------------------------------------------------------- GEMV --
 * Decode projection, one token:  y[n] = sum_k x[k] * w[n][k]   (n < N, k < K)
 * Same as q4k_gemm with M = 1 and the same bits.  The decode path of the pages
 * carries no floating-point atomics (sparkinfer-server README, "Determinism");
 * neither does this one.  Activations must be finite and below 2^63 in
 * magnitude (the kernel scales them by 2^64 inside its tensor-core operands);
 * magnitudes below 2^-56 lose relative precision there.
 *   w  device Q4_K blocks, 16-byte aligned;  x  device bf16[K], 16-byte aligned;
 *   y  device fp32[N], 4-byte aligned.
 * Errors: NULL, SHAPE, ALIGN, DEVICE, CUDA. */
q4k_status q4k_gemv(const void *w, int64_t N, int64_t K, const uint16_t *x, float *y, void *stream);

/* -------------------------------------------------------------------- GEMM --
 * y[m][n] = sum_k x[m*ldx + k] * w[n][k]  for m < M, n < N; y[m*ldy + n].
 *   M <= 16 : the small-M path (decode and speculative verification, 1 + drafts
 *             tokens per lane; ninfer serving docs "Determinism"): exact integer
 *             tensor-core products per 32-weight sub-block, fp32 scaling and
 *             accumulation.  M = 1 is the decode GEMV (q4k_gemv).  For 2 <= M <=
 *             16, row m of the result does not depend on M; with
 *             q4k_set_batch_invariant(1) that holds for M = 1 too.
 *   M >  16 : the prefill path (sparkinfer-server README, "Serve a GGUF instead of
 *             NVFP4"): each weight tile is dequantized to bf16 in shared memory and
 *             multiplied on the tcgen05 tensor cores with fp32 accumulation in
 *             tensor memory.
 *   w   device Q4_K blocks, 16-byte aligned
 *   x   device bf16, 16-byte aligned, ldx >= K and ldx % 8 == 0
 *   y   device fp32, ldy >= N; 4-byte aligned for M <= 16, 16-byte aligned with
 *       ldy % 4 == 0 for M > 16
 *   ws  device scratch of at least q4k_gemm_workspace_size(M, N, K) bytes,
 *       256-byte aligned (may be NULL when that size is 0).  Its contents need not
 *       be initialized and are garbage afterwards.
 * Errors: NULL, SHAPE (M < 1, N < 1, bad K, ldx < K, ldy < N), ALIGN, WORKSPACE,
 * DEVICE, CUDA. */
size_t q4k_gemm_workspace_size(int64_t M, int64_t N, int64_t K);
q4k_status q4k_gemm(const void *w, int64_t N, int64_t K, const uint16_t *x, int64_t M, int64_t ldx, float *y,
                    int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* -------------------------------------------------------- int8 activations --
 * The pages' serving pipeline requantizes activations to int8 at each layer
 * (sparkinfer-server README, "Determinism"); their format is not given.  The
 * reading taken: blocks of 32 consecutive elements of a row (one Q4_K
 * sub-block's span), in fp32: a = max |x|, s = a / 127, q = rint(x / s) with
 * ties to even, and q = 0, s = 0 for an all-zero block.
 *
 * q4k_quantize_x8: x -> (q, s).
 *   x  device bf16 [M][ldx], ldx >= K, 4-byte aligned
 *   q  device int8 [M][K], dense, 16-byte aligned
 *   s  device fp32 [M][K/32], dense, 16-byte aligned
 * Bit-exact: every q and s follows from the IEEE round-to-nearest divisions
 * above.  Errors: NULL, SHAPE (M < 1, K not a positive multiple of 256,
 * ldx < K), ALIGN, DEVICE, CUDA. */
q4k_status q4k_quantize_x8(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int8_t *q, float *s, void *stream);

/* q4k_gemm_x8: y = xh . W^T, where xh[m][k] = s[m][k/32] * q[m][k] are the
 * int8 activations (layouts as q4k_quantize_x8).
 *   M <= 16: the integer dot products of each 32-weight sub-block are exact; the
 *            scaling and accumulation are fp32.  Row m of the result does not
 *            depend on M.  No workspace.
 *   M >  16 (prefill, where the pages requantize the next layer's input): the
 *            activation scale changes every 32 elements of K, which an MMA
 *            accumulating over K cannot apply, so a pre-pass writes
 *            bf16(s * q) (the fp32 product rounded to nearest-even bf16) into
 *            the workspace and the tcgen05 prefill GEMM multiplies it like bf16
 *            activations (within the tensor-core bar, 1e-2).
 *   y   fp32 [M][ldy], ldy >= N; 4-byte aligned for M <= 16, 16-byte aligned with
 *       ldy % 4 == 0 for M > 16
 *   ws  device scratch of at least q4k_gemm_x8_workspace_size(M, K) bytes (M*K*2
 *       for M > 16, else 0), 256-byte aligned; garbage afterwards
 * Errors: NULL, SHAPE (M < 1, N < 1, bad K, ldy < N), ALIGN, WORKSPACE, DEVICE,
 * CUDA. */
size_t q4k_gemm_x8_workspace_size(int64_t M, int64_t K);
q4k_status q4k_gemm_x8(const void *w, int64_t N, int64_t K, const int8_t *q, const float *s, int64_t M, float *y,
                       int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------- NVFP4 weights --
 * The pages serve NVFP4 checkpoints as well as GGUF Q4_K (sparkinfer-server
 * README, "Serve a GGUF instead of NVFP4"); they do not spell the format out.
 * Reading taken: NVIDIA's NVFP4, w = g * e4m3 * e2m1 - 4-bit e2m1 values
 * (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit), one e4m3 scale per 16
 * consecutive weights of a row, one fp32 scale g per tensor.  Byte layout (this
 * library's): a row is K/256 blocks of 144 bytes (q4k_row_bytes(K)), each 16
 * e4m3 scale bytes (scale j covers weights 16j..16j+15) followed by 128 bytes
 * of e2m1 pairs (weight 2i in the low nibble of byte i, 2i+1 in the high one).
 *
 * q4k_nvfp4_dequant: out[N][K] fp32 = g * (e4m3 * e2m1), the product exact and
 * the multiplication by g rounded once: bit-exact.  w and out 16-byte aligned.
 * q4k_nvfp4_gemm: y[M][ldy] = x[M][ldx] . W^T for any M >= 1, on the tcgen05
 * tensor cores: each weight enters the MMA as the exact bf16 value e4m3 * e2m1,
 * the fp32 accumulator is multiplied by g in the epilogue.  x 16-byte aligned,
 * ldx % 8 == 0; y 4-byte aligned.  Deterministic (no atomics).
 * Errors: NULL, SHAPE (M or N < 1, K not a positive multiple of 256, ldx < K,
 * ldy < N), ALIGN, DEVICE, CUDA. */
q4k_status q4k_nvfp4_dequant(const void *w, float g, int64_t N, int64_t K, float *out, void *stream);
q4k_status q4k_nvfp4_gemm(const void *w, float g, int64_t N, int64_t K, const uint16_t *x, int64_t M, int64_t ldx,
                          float *y, int64_t ldy, void *stream);

/* --------------------------------------------------------------------- MoE --
 * Routed-expert layer over E experts, each an N x K Q4_K matrix; the pages' MoE
 * models route each token to its top-k experts and combine the experts' outputs
 * weighted by the gates (sparkinfer-server README, "Determinism": the routed MoE
 * down-projection combine, done there with fp32 atomicAdd; here in slot order,
 * with no atomics).
 *
 * q4k_moe_route: stable counting sort of the T*topk (token t, slot j) items by
 * expert id.  Item i = t*topk + j.
 *   topk_ids  device int32[T*topk]
 *   offsets   device int32[E+1]: items of expert e are perm[offsets[e] .. offsets[e+1])
 *   perm      device int32[T*topk]: item indices, grouped by expert, increasing
 *             within an expert.  Items whose id is outside [0,E) are left out
 *             (offsets[E] counts the valid items; perm beyond it is -1).
 * This is the routing step of q4k_moe_grouped_gemm exposed on its own.
 * Errors: NULL, SHAPE (T < 1, topk < 1, E < 1 or E > 1024, topk > E,
 * T*topk >= 2^31), ALIGN (a pointer not 4-byte aligned), DEVICE, CUDA. */
q4k_status q4k_moe_route(const int32_t *topk_ids, int64_t T, int32_t topk, int32_t n_experts, int32_t *offsets,
                         int32_t *perm, void *stream);

typedef enum {
    Q4K_MOE_X_PER_TOKEN = 0, /* x is [T][K]: every slot of token t multiplies x[t] */
    Q4K_MOE_X_PER_SLOT = 1   /* x is [T][topk][K]: slot (t,j) multiplies x[t][j] */
} q4k_moe_x_mode;

typedef enum {
    Q4K_MOE_Y_PER_SLOT = 0, /* y is [T][topk][N]: y[t][j] = x_row . w_{ids[t][j]}^T */
    Q4K_MOE_Y_COMBINE = 1   /* y is [T][N]: y[t] = sum_{j=0..topk-1} gates[t][j] * out[t][j],
                               summed in increasing j */
} q4k_moe_y_mode;

/* q4k_moe_grouped_gemm: every (token, slot) item multiplies its activation row by
 * its expert's matrix; one call covers all experts.
 *   w_experts  device, E*N*q4k_row_bytes(K) bytes: expert e's matrix starts at byte
 *              e*N*q4k_row_bytes(K); 16-byte aligned
 *   x          device bf16 rows of K (dense, ld = K), 16-byte aligned
 *   topk_ids   device int32[T][topk]; ids outside [0,E) give zero output rows and
 *              are not an error (they cannot be checked without a synchronization)
 *   gates      device fp32[T][topk]; required for Q4K_MOE_Y_COMBINE, else ignored
 *   y          device fp32, dense, 16-byte aligned
 *   ws         device scratch, >= q4k_moe_workspace_size(...) bytes, 256-byte aligned;
 *              holds the routing permutation and, for Q4K_MOE_Y_COMBINE, the
 *              per-slot fp32 rows; contents need not be initialized
 * Errors: NULL, SHAPE (as q4k_moe_route, plus N < 1, bad K, E*N >= 2^31, an
 * unknown mode, N % 4 != 0 with Q4K_MOE_Y_COMBINE), ALIGN, WORKSPACE, DEVICE,
 * CUDA.  q4k_moe_workspace_size returns 0 for arguments that would give SHAPE.
 * It takes the output mode as well as the shape (an addition to the plain
 * shape query): only Q4K_MOE_Y_COMBINE needs room for the per-slot rows. */
size_t q4k_moe_workspace_size(int32_t n_experts, int64_t N, int64_t K, int64_t T, int32_t topk, int y_mode);
q4k_status q4k_moe_grouped_gemm(const void *w_experts, int32_t n_experts, int64_t N, int64_t K, const uint16_t *x,
                                int x_mode, const int32_t *topk_ids, const float *gates, int64_t T, int32_t topk,
                                float *y, int y_mode, void *ws, size_t ws_bytes, void *stream);

/* q4k_moe_grouped_gemm_reuse_routing: q4k_moe_grouped_gemm without the routing
 * step.  The gate, up and down projections of one routed layer share the same
 * top-k ids (sparkinfer-server README, "Determinism": discrete top-k expert
 * routing), so after one q4k_moe_grouped_gemm call has sorted the items into
 * `ws`, the layer's other projections can use that sort instead of repeating it.
 * Same arguments, results and errors as q4k_moe_grouped_gemm (same bits), under
 * these conditions:
 *   - `ws` holds the routing written by the last q4k_moe_grouped_gemm call that
 *     used it (calls to this function leave it unchanged, so any number of them
 *     may follow one routing call), ordered before this call on the GPU;
 *   - that call had the same n_experts and the same number of items T*topk, and
 *     topk_ids has not changed since.
 * The routing records the (n_experts, T*topk) it was made for, and the kernels
 * check it on the GPU before reading any of it: a workspace holding a routing
 * for another shape, or none, makes the call write nothing, and the next
 * q4k_check_device reports Q4K_ERR_ROUTING.  (With at most 16 items no routing
 * is used at all.)  That topk_ids is unchanged is not checked: changed ids give
 * wrong results, not an error.  N, K, x, x_mode, gates, y and y_mode may differ
 * from the routing call; ws_bytes must cover this call
 * (q4k_moe_workspace_size), and the routing part of the workspace depends only
 * on (n_experts, T, topk). */
q4k_status q4k_moe_grouped_gemm_reuse_routing(const void *w_experts, int32_t n_experts, int64_t N, int64_t K,
                                              const uint16_t *x, int x_mode, const int32_t *topk_ids,
                                              const float *gates, int64_t T, int32_t topk, float *y, int y_mode,
                                              void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------- routed expert FFN layer --
 * One routed SwiGLU feed-forward layer of the pages' MoE models (sparkinfer-server
 * README, "Determinism": discrete top-k expert routing and the routed MoE
 * down-projection combine).  For every token t and slot j with a valid expert
 * e = topk_ids[t][j]:
 *   g = x[t] . Wg_e^T,  u = x[t] . Wu_e^T                     (fp32, H values)
 *   h = bf16(silu(g) * u), silu(g) = g / (1 + e^-g)           (rounded to nearest even)
 *   o = h . Wd_e^T                                            (fp32, D values)
 *   y[t] = sum_{j=0..topk-1} gates[t][j] * o[t][j], summed in increasing j.
 * Slots whose id is outside [0,E) contribute nothing (a token whose ids are all
 * invalid gets a zero row).  The routing is computed once for the three
 * projections; the up projection's epilogue applies SwiGLU to the gate
 * projection's output and stores h in bf16, so u is never written out.
 *   w_gate, w_up  device, E*H*q4k_row_bytes(D) bytes each: expert e's H x D matrix
 *                 starts at byte e*H*q4k_row_bytes(D); 16-byte aligned
 *   w_down        device, E*D*q4k_row_bytes(H) bytes: expert e's D x H matrix at
 *                 byte e*D*q4k_row_bytes(H); 16-byte aligned
 *   x             device bf16 [T][D], dense, 16-byte aligned
 *   topk_ids      device int32 [T][topk];  gates  device fp32 [T][topk]
 *   y             device fp32 [T][D], dense, 16-byte aligned
 *   ws            device scratch, >= q4k_moe_ffn_workspace_size(...) bytes,
 *                 256-byte aligned, contents need not be initialized: the
 *                 routing, g (4*T*topk*H bytes), h (2*T*topk*H), the per-slot
 *                 outputs o (4*T*topk*D) and, from 32*E items on, the
 *                 expert-sorted copy of x (2*T*topk*D)
 * Errors: NULL, SHAPE (E < 1 or E > 1024, topk < 1 or topk > E, T < 1,
 * T*topk >= 2^31, H or D not a positive multiple of 256, E*H or E*D >= 2^31),
 * ALIGN, WORKSPACE, DEVICE, CUDA.  q4k_moe_ffn_workspace_size returns 0 for
 * arguments that would give SHAPE. */
size_t q4k_moe_ffn_workspace_size(int32_t n_experts, int64_t H, int64_t D, int64_t T, int32_t topk);
q4k_status q4k_moe_ffn(const void *w_gate, const void *w_up, const void *w_down, int32_t n_experts, int64_t H,
                       int64_t D, const uint16_t *x, const int32_t *topk_ids, const float *gates, int64_t T,
                       int32_t topk, float *y, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------- allocation-free MoE --
 * No counterpart on the pages: an addition for callers that cannot provide a
 * workspace - code that must not call cudaMalloc/cudaFree (they synchronize the
 * whole device), engines that hand all device memory to their own pools at
 * start-up, and foreign-language callers that only pass buffers they own.
 *
 * q4k_moe_grouped_gemm_noalloc computes exactly what q4k_moe_grouped_gemm
 * computes (same arguments, same kernels, same bits) but takes no workspace:
 * its scratch is a fixed array of Q4K_MOE_NOALLOC_SCRATCH_BYTES inside the
 * library, which every GPU that loads the library keeps allocated until the
 * process exits.  It allocates nothing itself.
 *   - The first call on a device looks up that device's scratch address
 *     (cudaGetSymbolAddress, with the device current), and so does the first
 *     call in a context of that device created since (cudaDeviceReset destroys
 *     the context the address belonged to).  Make that first call before
 *     capturing a stream into a CUDA graph.
 *   - Every call on a device shares the one array.  Calls whose kernels can
 *     overlap on the GPU (different streams without ordering between them) race
 *     on it and give wrong results; order them on one stream.
 *   - The array keeps the last call's contents; nothing in it needs to start at
 *     zero, because each call writes every scratch byte it later reads.
 *   - A request whose scratch need, q4k_moe_workspace_size(n_experts, N, K, T,
 *     topk, y_mode), exceeds Q4K_MOE_NOALLOC_SCRATCH_BYTES fails with
 *     Q4K_ERR_WORKSPACE before anything is launched.  With Q4K_MOE_Y_PER_SLOT and
 *     fewer than 32*E items the need is only the routing (about 4*(E + T*topk)
 *     bytes); Q4K_MOE_Y_COMBINE adds 4*T*topk*N bytes (for example T = 64,
 *     topk = 8, N = 2048 needs 4 MiB), and from 32*E items on, where the experts
 *     run on the tensor cores, the gathered activation rows add 2*T*topk*K bytes.
 * Other errors are those of q4k_moe_grouped_gemm. */
#define Q4K_MOE_NOALLOC_SCRATCH_BYTES (8u << 20)
q4k_status q4k_moe_grouped_gemm_noalloc(const void *w_experts, int32_t n_experts, int64_t N, int64_t K,
                                        const uint16_t *x, int x_mode, const int32_t *topk_ids, const float *gates,
                                        int64_t T, int32_t topk, float *y, int y_mode, void *stream);

/* ---------------------------------------------------------------------------
 * The operators between a decode step's weight products: closing one block and
 * opening the next (q4k_norm_residual), writing new keys and values into a paged
 * cache (q4k_kv_append), attention of the new tokens over that cache
 * (q4k_attn_decode), shrinking a cache to a budget (q4k_kv_evict) and drawing the
 * next tokens (q4k_sample).  Their fp32 inputs are what the weight products write,
 * and their bf16 outputs what those read.
 *
 * A sequence's cache is a list of SLOTS 0 .. len - 1, one per cached token, kept in
 * pages of page_size slots.  Slot j of sequence b lies in page
 * page_table[b*ld_table + j / page_size] at row j % page_size; the D values of KV
 * head h there start at element
 *     page*page_stride + h*head_stride + (j % page_size)*slot_stride
 * of both pools, which covers [page][head][slot][D], [page][slot][head][D] and pools
 * that interleave keys and values.  Slots carry no order: rotary positions are in
 * the keys, and the caller may keep each slot's position (and the attention weight
 * it received) in the arrays `positions` and `weights` [batch][n_kv_heads][ld_meta].
 *
 * Indices read from device memory are checked in the kernels: a page id outside
 * [0, n_pages), a length above max_pages*page_size, a sequence, slot or position out
 * of range records Q4K_ERR_INDEX for q4k_check_device, and the slot or token that it
 * belongs to is left out (a length counts as clamped to what the table or the
 * metadata can hold). Negative lengths count as 0. Two sequences may share pages
 * that neither writes. */

#define Q4K_KV_BF16 0 /* cache of bf16 */
#define Q4K_KV_E4M3 1 /* cache of e4m3 (fp8): the value stands for itself times k_scale or v_scale */

typedef struct {
    void *k, *v;               /* pools: 16-byte aligned device pointers */
    const int32_t *page_table; /* device, [batch][ld_table] */
    int64_t ld_table;          /* >= max_pages */
    int64_t n_pages;           /* pages in each pool */
    int64_t page_stride, head_stride, slot_stride; /* in elements, >= 1, multiples of 16 bytes */
    int32_t batch;             /* sequences, 1 .. 65535 */
    int32_t max_pages;         /* table entries per sequence; max_pages*page_size < 2^31 */
    int32_t page_size;         /* slots per page, >= 1 */
    int32_t n_kv_heads;        /* 1 .. 1024; batch*n_kv_heads <= 2^24 */
    int32_t head_dim;          /* D: 64, 128 or 256 */
    int32_t dtype;             /* Q4K_KV_BF16 or Q4K_KV_E4M3 */
    float k_scale, v_scale;    /* > 0 and finite; 1 for a plain cache */
} q4k_kv_cache;

#define Q4K_ROPE_HALF 0  /* value i pairs with value i + rope_dim/2 */
#define Q4K_ROPE_PAIRS 1 /* value 2i pairs with value 2i + 1 */

/* Rotary embedding of T new tokens' queries and keys, and the write of their keys
 * and values into the cache: for token t of sequence seq[t], slot slot[t],
 *     (a, b) -> (a*cos - b*sin, b*cos + a*sin)   over the first rope_dim values of
 * each q and k head, each product and sum rounded to fp32, cos and sin from row
 * pos[t] of `rope`; q is rounded once to bf16 into q_out, k/k_scale and v/v_scale
 * (computed as a product with the fp32 reciprocal) once to the cache's type.  For
 * e4m3, values beyond +-448 become +-448 and NaN stays NaN.
 *   q [T][ldq], k [T][ldk], v [T][ldv]: fp32, heads consecutive in a row, 4-byte
 *     aligned.  They may be columns of one product's output.
 *   seq, slot, pos: int32 [T]; no two tokens with the same (seq, slot).
 *   rope: fp32 [n_pos][rope_dim], row = rope_dim/2 cosines, then rope_dim/2 sines;
 *     rope_dim even, 0 .. D; 0: no rotation (rope may be NULL, pos is then only
 *     written to positions).  With rope_dim > 0, pos[t] must be in [0, n_pos).
 *   q_out bf16 [T][ldqo].  q and q_out may both be NULL (keys and values only).
 *   weights, positions (each may be NULL): slot[t]'s entry of every head becomes
 *     0 and pos[t]; with either, slot[t] must be < ld_meta.
 * T < 2^31; n_heads 1 .. 65536.
 * A token with an index out of range is recorded (Q4K_ERR_INDEX) and leaves the
 * cache, weights and positions alone; its q_out row becomes 0. */
q4k_status q4k_kv_append(const q4k_kv_cache *cache, int64_t T, int32_t n_heads, const float *q, int64_t ldq,
                         const float *k, int64_t ldk, const float *v, int64_t ldv, const int32_t *seq,
                         const int32_t *slot, const int32_t *pos, const float *rope, int64_t n_pos, int32_t rope_dim,
                         int rope_mode, uint16_t *q_out, int64_t ldqo, float *weights, int32_t *positions,
                         int64_t ld_meta, void *stream);

/* Attention of the last n_q tokens of every sequence over its cache.
 *   s[r][j] = scale * k_scale * q[r] . k[j]   (with softcap c > 0: c*tanh(s/c))
 *   o[r]    = v_scale * sum_j softmax_j(s[r])[j] * v[j]
 * Row r is query token i (0 <= i < n_q) and head hq of sequence b; it reads KV head
 * hq / (n_heads/n_kv_heads) at slots [max(0, e - window), e), e = len - n_q + 1 + i
 * (window 0: all of [0, e)).  len = seq_lens[b] counts the n_q tokens themselves
 * (q4k_kv_append writes them first).  A row that reads nothing (e <= 0) gives 0.  A slot outside a
 * row's range has no part in it, whatever its key and value hold.
 *   q, o: bf16 [batch*n_q][ldq], [batch*n_q][ldo], row b*n_q + i, heads of D
 *     consecutive; 16-byte aligned, ldq and ldo multiples of 8.
 *   n_heads: a multiple of n_kv_heads; n_q 1 .. 64; rows of a KV head, n_q * n_heads /
 *     n_kv_heads, 1 .. 1024.  (With many sequences, batch * n_kv_heads * D * these rows,
 *     rounded up to whole tiles of 8, 16 or 32, must be below 2^38.)
 *   weights (may be NULL): fp32 [batch][n_kv_heads][ld_weights], updated for every
 *     slot j < len:  weights[b][h][j] = decay*weights[b][h][j] + sum of
 *     softmax(s[r])[j] over the rows r of head h.  len must be <= ld_weights.
 *     (A slot left out for its page: decay*weights alone.)
 * Products are exact and sums, maxima and the joined softmax fp32.  (For an e4m3 cache
 * a value of q below 2^-31 of the largest of its row is taken to 2^-39 of that one.)
 * The weights p enter the product with v as the sum of two bf16 values (to 2^-16), for
 * an e4m3 cache of two f16 values (to 2^-22, and to 2^-32 of the largest), while the sum
 * that divides them is that of the fp32 values; o is rounded once.  The length is split
 * over the whole GPU by the lengths of the batch, and the parts are joined in slot
 * order: the same call repeats its bits, but a sequence's last bits may depend on the
 * other lengths of its batch, also in batch-invariant mode.
 * Workspace: q4k_attn_decode_workspace_size(cache, n_heads, n_q, ld_weights, or 0
 * without weights) bytes, 256-byte aligned; 0 is returned for arguments that the call
 * would refuse. */
size_t q4k_attn_decode_workspace_size(const q4k_kv_cache *cache, int32_t n_heads, int32_t n_q, int64_t ld_weights);
q4k_status q4k_attn_decode(const q4k_kv_cache *cache, const int32_t *seq_lens, const uint16_t *q, int64_t ldq,
                           int32_t n_heads, int32_t n_q, float scale, float softcap, int64_t window, uint16_t *o,
                           int64_t ldo, float *weights, int64_t ld_weights, float decay, void *ws, size_t ws_bytes,
                           void *stream);

/* Eviction: every sequence longer than `budget` slots is cut to budget, each KV head
 * by its own weights.  Of a head's slots, the len - budget ones with the smallest
 * weight go (equal weights: the lowest slot first; NaN counts as larger than all),
 * among those that are not protected; protected are positions < sinks and positions
 * > newest - recent, newest being the head's largest position.  (Should more than
 * budget slots be protected, protected ones go too, by the same order.)  The slots
 * freed below budget are filled, in increasing order, with the kept slots at or above
 * it, in increasing order; the other kept slots stay where they are.  So pages from
 * ceil(budget/page_size) on are free afterwards, and pages must not be shared between
 * sequences below that.
 * A move from or to a page whose id is out of range is not made: the hole keeps the
 * token that was to go, with its own weight and position, and the kept one is lost.
 *   weights, positions: [batch][n_kv_heads][ld_meta]; weights_out and positions_out
 *     receive the entries of the slots < new length (each may be the input array;
 *     otherwise they must not overlap it).
 *   new_lens[b] = min(len, budget); may be seq_lens.  len must be <= ld_meta.
 *   1 <= budget; 0 <= sinks, recent; sinks + recent <= budget.
 * Workspace: q4k_kv_evict_workspace_size(cache, ld_meta) bytes, 256-byte aligned. */
size_t q4k_kv_evict_workspace_size(const q4k_kv_cache *cache, int64_t ld_meta);
q4k_status q4k_kv_evict(const q4k_kv_cache *cache, const int32_t *seq_lens, int32_t *new_lens, int64_t budget,
                        int64_t sinks, int64_t recent, const float *weights, const int32_t *positions,
                        float *weights_out, int32_t *positions_out, int64_t ld_meta, void *ws, size_t ws_bytes,
                        void *stream);

#define Q4K_NORM_NONE 0
#define Q4K_NORM_RMS 1   /* x / sqrt(mean(x^2) + eps) * w + b */
#define Q4K_NORM_LAYER 2 /* the same of x - mean(x) */
#define Q4K_RES_FP32 0
#define Q4K_RES_BF16 1

/* The end of one block and the start of the next, for M rows of D values:
 *     h = r_in + scale * gate * post(y)      r_out = h      x = bf16(pre(h))
 * post and pre are norms over a row (kinds above); y fp32 [M][ldy], may be NULL (h =
 * r_in).  *_w and *_b fp32 [D], each may be NULL (1 and 0); not read for
 * Q4K_NORM_NONE.  gate fp32 [M][ld_gate], or one row for all with ld_gate = 0, or
 * NULL (1).  r_in and r_out [M][ldr] of type r_dtype; r_out may be r_in, or NULL (not
 * kept).  x bf16 [M][ldx], may be NULL if r_out is not (pre is then not computed).
 * Everything is fp32 until r_out and x are rounded once each; x comes from h before
 * r_out's rounding.  1 <= M < 2^31; 1 <= D <= 2^20; pointers aligned to their element.  A row's last
 * bits depend on D, on how pointers and strides are aligned, and on whether M is below
 * the number of SMs, but with q4k_set_batch_invariant(1) not on M. */
q4k_status q4k_norm_residual(int64_t M, int64_t D, const float *y, int64_t ldy, int post, const float *post_w,
                             const float *post_b, float post_eps, const float *gate, int64_t ld_gate, float scale,
                             const void *r_in, void *r_out, int64_t ldr, int r_dtype, int pre, const float *pre_w,
                             const float *pre_b, float pre_eps, uint16_t *x, int64_t ldx, void *stream);

/* Draws token[m] from row m of logits [M][ldl] (fp32, V values) with the given random
 * number u[m] in [0, 1).  Per row: temperature, top_k, top_p and min_p (device arrays
 * [M]; each may be NULL: 1, off, off, off).
 *   NaN logits count as -inf.  Tokens are ranked by logit, equal ones by index.
 *   Weights are whole numbers, so that every sum and comparison below is exact and the
 *   token depends on no order of summation: with z the largest logit and
 *     d = (z - logit) * ((1/temperature) * log2(e)) in fp32, left to right,
 *     w = floor(P(d) * 2^40), where 2^-d = 2^-n 2^-f, n = floor(d), and P is 2^-n times
 *   the fp32 Horner form of the series of 2^-f about f = 1/2 to the 7th power (each
 *   product and sum rounded); w = 0 from d >= 41 on.
 *   top_k > 0 keeps the top_k first in rank.  top_p < 1 keeps the shortest run of
 *   these, in rank, whose weights reach floor(S*floor(top_p*2^24)/2^24), S the sum of what top_k
 *   kept, and at least one.  min_p > 0 keeps the tokens whose weight is at least
 *   floor(W*floor(min_p*2^24)/2^24), W the largest weight.  Over the kept tokens by
 *   index, token is the first whose running sum exceeds floor(S'*floor(u*2^24)/2^24),
 *   S' being their sum.  prob[m] (may be NULL) = w/S'.
 *   temperature <= 0 or NaN: the first in rank, prob 1.  A row without any logit above
 *   -inf: token -1, prob 0.  top_p and min_p are clamped to [0, 1], u to [0, 1 -
 *   2^-24]; NaN counts as off (0 for u).
 * 1 <= M <= 2^24, 1 <= V <= 2^22, ldl >= V; pointers aligned to their element. */
q4k_status q4k_sample(const float *logits, int64_t M, int64_t V, int64_t ldl, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *token,
                      float *prob, void *stream);

/* ---------------------------------------------------------------------------
 * The operators of a step that runs chunks of prompts and decode tokens of many
 * requests together: pages and slots for the new tokens (q4k_batch_plan), the norm
 * between two blocks with 8-bit activations for the next product
 * (q4k_norm_residual_x8), the requests' low-rank adapters beside a shared projection
 * (q4k_lora_add) and the attention of chunks of any length over the paged cache
 * (q4k_attn_chunk). */

/* Gives every request of a batch its pages and every new token its slot.  Request b
 * holds held[b] pages (the first entries of its row of cache->page_table, which this
 * call writes) and seq_lens[b] slots in them, and brings n_new[b] tokens; a negative
 * n_new[b] says that the request is over.  In this order, every sum over requests running
 * in their order:
 *   1. A request whose slots and tokens exceed max_pages*page_size brings none
 *      (Q4K_ERR_INDEX is recorded).  Then those with which the running sum of tokens
 *      exceeds T bring none in this step.
 *   2. want = ceil((seq_lens[b] + tokens) / page_size), 0 for a request that is over.
 *      Entries want .. held - 1 (after an eviction, or at the end) go back onto the free
 *      list free_pages[0 .. *free_count), in order.
 *   3. A request with want > held takes want - held pages from the list's end, if the
 *      running sum of what requests lack, itself included, is at most what the list
 *      holds now; otherwise it brings no tokens and keeps what it holds.
 * Outputs: the table's entries, held_out[b], *count_out (the list's new length),
 * after_lens[b] = seq_lens[b] + its tokens (0 if over), starts[0 .. batch] = running sum
 * of tokens, and for each token t < starts[batch] its seq, slot and position pos[t] =
 * first_pos[b] + i for the request's i-th (first_pos NULL: the slot): the inputs of
 * q4k_kv_append and q4k_attn_chunk.  For starts[batch] <= t < T, seq = -1, slot = pos = 0.
 *   All arrays int32 on the device, 4-byte aligned: seq_lens, n_new, first_pos, held,
 *   held_out, after_lens [batch]; free_pages [n_pages]; seq, slot, pos [T]; starts
 *   [batch + 1].  after_lens may be seq_lens, held_out held, count_out free_count; other
 *   outputs overlap nothing.  1 <= T < 2^31.
 * Lengths and held pages out of range count as clamped and are recorded, as is a page id
 * out of range that changes hands (it is passed on as it is) and a page that the list
 * (of n_pages entries) has no room for (it is dropped).
 * Workspace: q4k_batch_plan_workspace_size(cache) bytes, 256-byte aligned. */
size_t q4k_batch_plan_workspace_size(const q4k_kv_cache *cache);
q4k_status q4k_batch_plan(const q4k_kv_cache *cache, const int32_t *seq_lens, const int32_t *n_new,
                          const int32_t *first_pos, const int32_t *held, int32_t *held_out, int32_t *free_pages,
                          const int32_t *free_count, int32_t *count_out, int64_t T, int32_t *after_lens,
                          int32_t *starts, int32_t *seq, int32_t *slot, int32_t *pos, void *ws, size_t ws_bytes,
                          void *stream);

/* q4k_norm_residual whose output is (also) 8 bits wide, the input of q4k_gemm_x8: with
 * v = pre(h) in fp32, for each 32 consecutive values of a row a = max |v|, s = a / 127,
 * q = rint(v / s) (ties to even, at most 127 in magnitude), and q = 0, s = 0 where all
 * are zero or a is so small that a / 127 is 0 (q4k_quantize_x8's rule, applied to the fp32
 * values instead of their bf16 roundings).  A block with a NaN gets s = NaN and q = 0, one with
 * an infinity s = infinity and q = +-127 where |v| is infinite, 0 elsewhere.
 *   q  int8 [M][D], dense, 4-byte aligned;  s  fp32 [M][D/32], dense
 *   D a multiple of 32; x (bf16, for the other readers of v) and r_out may be NULL
 * Everything else, the rows' bits included, is as in q4k_norm_residual. */
q4k_status q4k_norm_residual_x8(int64_t M, int64_t D, const float *y, int64_t ldy, int post, const float *post_w,
                                const float *post_b, float post_eps, const float *gate, int64_t ld_gate, float scale,
                                const void *r_in, void *r_out, int64_t ldr, int r_dtype, int pre, const float *pre_w,
                                const float *pre_b, float pre_eps, uint16_t *x, int64_t ldx, int8_t *q, float *s,
                                void *stream);

/* Adds to a projection's output what each token's low-rank adapter contributes:
 *     y[t][n] += scales[a] * sum_{r < ranks[a]} b[a][n][r] * (sum_k a[a][r][k] * x[t][k]),
 * a = ids[t].  Rows of tokens with a negative id are not touched (no adapter), nor those
 * with an id >= n_adapters (Q4K_ERR_INDEX is recorded).  What lies beyond an adapter's
 * rank has no part in it.
 *   a  bf16 [n_adapters][R][K], b bf16 [n_adapters][N][R]: dense, 16-byte aligned
 *   ranks  int32 [n_adapters] (NULL: R), clamped to 0 .. R;  scales  fp32 [n_adapters] (NULL: 1)
 *   ids  int32 [T], in any order;  x  bf16 [T][ldx], 16-byte aligned, ldx % 8 == 0
 *   y  fp32 [T][ldy], 4-byte aligned
 *   1 <= n_adapters <= 1024; R a multiple of 8, 8 .. 128; K a multiple of 8; N, K <= 2^21;
 *   T <= 2^23
 * Products are exact and sums fp32; the inner sums, times the scale, enter the second
 * product as the sum of three bf16 values, exactly; a value of b that is not finite adds its own
 * product with the inner sum.  A row's last bits do not depend on the
 * other rows' adapters, but on K, R, T and n_adapters.
 * Workspace: q4k_lora_add_workspace_size(...) bytes, 256-byte aligned; 0 is returned for
 * arguments that the call would refuse. */
size_t q4k_lora_add_workspace_size(int32_t n_adapters, int64_t N, int64_t K, int32_t R, int64_t T);
q4k_status q4k_lora_add(int32_t n_adapters, int64_t N, int64_t K, int32_t R, const uint16_t *a, const uint16_t *b,
                        const int32_t *ranks, const float *scales, const int32_t *ids, const uint16_t *x, int64_t T,
                        int64_t ldx, float *y, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* Attention of a chunk of new tokens of every sequence over its cache: q4k_attn_decode's
 * definition with a number of new tokens n_b = starts[b+1] - starts[b] of each sequence's
 * own, from none to whole prompts.
 *   s[r][j] = scale * k_scale * q[r] . k[j]   (with softcap c > 0: c*tanh(s/c))
 *   o[r]    = v_scale * sum_j softmax_j(s[r])[j] * v[j]
 * Row r is head hq of token i (0 <= i < n_b) of sequence b, which is row starts[b] + i of
 * q and o; it reads KV head hq / (n_heads/n_kv_heads) at slots [max(0, e - window), e),
 * e = seq_lens[b] - n_b + 1 + i (window 0: all of [0, e)).  seq_lens[b] counts the new
 * tokens, which q4k_kv_append has written.  A row that reads nothing (e <= 0) gives 0; a
 * slot outside a row's range has no part in it, whatever its key and value hold.
 *   q, o: bf16 [T][ldq], [T][ldo], heads of D consecutive; 16-byte aligned, ldq and ldo
 *     multiples of 8; they do not overlap.  Rows of o that belong to no sequence are not touched.
 *   starts: int32 [batch + 1], not decreasing, 0 .. T; one that is out of order or range is recorded
 *     (Q4K_ERR_INDEX) and counts as the nearest that is not.  starts[0] need not be 0.
 *   n_heads: a multiple of n_kv_heads, n_heads / n_kv_heads <= 1024; T * n_heads < 2^31.
 * Products are exact, sums and softmax fp32.  The weights enter the second product
 * rounded to bf16 (each off by 2^-8 at most; for an e4m3 cache, whose values are exact in
 * f16, to f16: by 2^-11, and 2^-32 of the largest), while the sum that divides them is that of the fp32 values: their
 * errors, which add up at random, are of the size of o's own rounding.  (For an e4m3 cache a value of
 * q below 2^-31 of the largest of its row is taken to 2^-39 of that one.)  A softcap may have any
 * size; beyond its own fp32 roundings a capped score is off by 1.5e-4 at most (e4m3 cache: 2e-5), and by
 * less for small caps.  The work is split over the whole GPU by all
 * lengths, and split rows are joined in slot order: the same call repeats its bits, but a
 * row's last bits may depend on the rest of the batch, also in batch-invariant mode.
 * Workspace: q4k_attn_chunk_workspace_size(cache, T, n_heads) bytes, 256-byte aligned; 0
 * is returned for arguments that the call would refuse. */
size_t q4k_attn_chunk_workspace_size(const q4k_kv_cache *cache, int64_t T, int32_t n_heads);
q4k_status q4k_attn_chunk(const q4k_kv_cache *cache, const int32_t *starts, const int32_t *seq_lens, const uint16_t *q,
                          int64_t T, int64_t ldq, int32_t n_heads, float scale, float softcap, int64_t window,
                          uint16_t *o, int64_t ldo, void *ws, size_t ws_bytes, void *stream);

/* The nine calls above for callers whose foreign-function interface converts every
 * argument on its own (from Python that takes longer than the rest of a small call on
 * the host): `slots` holds the arguments of the call of the same name, in its order, 8
 * bytes each in the machine's byte order - integers and addresses as int64 (a smaller
 * integer parameter takes the low bits), floats as double, rounded to fp32.  The same
 * checks, results and errors; slots = NULL gives Q4K_ERR_NULL. */
q4k_status q4k_kv_append_slots(const void *slots);
q4k_status q4k_attn_decode_slots(const void *slots);
q4k_status q4k_kv_evict_slots(const void *slots);
q4k_status q4k_norm_residual_slots(const void *slots);
q4k_status q4k_sample_slots(const void *slots);
q4k_status q4k_batch_plan_slots(const void *slots);
q4k_status q4k_norm_residual_x8_slots(const void *slots);
q4k_status q4k_lora_add_slots(const void *slots);
q4k_status q4k_attn_chunk_slots(const void *slots);

#ifdef __cplusplus
}
#endif
#endif /* Q4K_H */
