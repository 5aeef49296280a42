/*
 * nvfp4_mm.h -- C ABI of the batch-invariant NVFP4 weight matmul (GB300,
 * sm_103a), built into the same shared library as decode_attn.h and sharing
 * its status codes (DA_OK, DA_ERR_*).
 *
 * Why it exists.  "Greedy outputs depend on batch composition (NVFP4
 * GEMV/GEMM switch at 32 rows is a candidate)" (gllm issue #98, Candidate
 * cause) traces batch-dependent greedy decoding to a weight matmul whose
 * kernel is chosen by the number of activation rows n: a dequantizing GEMV
 * with f32 activations up to 32 rows, a bf16 tensor-core GEMM above.  The
 * same page (Next steps) proposes one activation precision, bf16, for both,
 * so the switch changes speed and not results.  This library goes one step
 * further: one arithmetic for every n, so a row's result is bitwise the same
 * whatever else shares the call.
 *
 * What it computes.  For activations x [n, K] and an NVFP4 weight W [N, K]:
 *
 *     xr[i, k]  = bf16(x[i, k])                      round to nearest even
 *     W[o, k]   = e4m3(scales[o, k / 16]) * e2m1(nibble(o, k))   (exact in bf16)
 *     P_c[i, o] = sum over k in chunk c of xr[i, k] * W[o, k]
 *                 (fp32 accumulation on the tensor cores, K ascending in
 *                  steps of 16; chunk c = k in [c * 1024, (c + 1) * 1024))
 *     y[i, o]   = global_scale * (((P_0 + P_1) + P_2) + ...)      fp32
 *     y_bf16    = bf16(y)                            round to nearest even
 *
 * The chunking (NVFP4_MM_K_CHUNK) and the order of every sum depend only on
 * K, never on n, on the other rows or on where row i sits in x.
 *
 * Weight format (the page names NVFP4 but not its layout; this is the
 * reading):
 *   codes   uint8 [N, K / 2]  two E2M1 codes per byte along K, element 2j of
 *                             a row in the low nibble of byte j.  E2M1: sign
 *                             bit 3, exponent bits 2..1 (bias 1), fraction
 *                             bit 0; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   scales  uint8 [N, K / 16] one E4M3 code (sign, 4 exponent bits with bias
 *                             7, 3 fraction bits; 0x7F / 0xFF are NaN) per 16
 *                             consecutive weights of a row.
 *   global_scale              one finite fp32 factor for the whole matrix.
 *
 * Conventions are those of decode_attn.h: device pointers owned by the
 * caller, `stream` a cudaStream_t passed as void*, no allocation, no host
 * synchronisation (except nvfp4_mm_read_error), DA_OK or a DA_ERR_* status
 * with nothing enqueued on error, no abort, trap or print.
 */
#ifndef NVFP4_MM_H
#define NVFP4_MM_H

#include <stddef.h>
#include <stdint.h>

#include "decode_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_MM_TILE_N 128   /* output features per tensor-core tile (MMA M) */
#define NVFP4_MM_ROW_TILE 32  /* activation rows per tile (MMA N)              */
#define NVFP4_MM_K_CHUNK 1024 /* K per partial sum P_c                         */

#define NVFP4_X_F32 0  /* activations given as fp32: rounded to bf16 on the device */
#define NVFP4_X_BF16 1 /* activations given as bf16: used as they are             */

/* Device workspace bytes for one call with n activation rows, N outputs and
 * reduction length K (0 when the shape is not supported).  It holds a 256-byte
 * header, one counter per output tile, the rounded activations (n rounded up
 * to NVFP4_MM_ROW_TILE rows) and, when K > NVFP4_MM_K_CHUNK, the fp32 partial
 * sums P_c.  Its contents need no initialisation. */
size_t nvfp4_mm_workspace_bytes(int32_t n, int32_t N, int32_t K);

/* y = global_scale * bf16(x) @ W^T as defined above.
 *   x       [n, K], fp32 (x_dtype NVFP4_X_F32) or bf16 (NVFP4_X_BF16),
 *           row-major, 16-byte aligned.
 *   codes   uint8 [N, K / 2], scales uint8 [N, K / 16], row-major; codes
 *           16-byte aligned, scales 4-byte aligned.
 *   y       fp32 [n, N], row-major, required.
 *   y_bf16  bf16 [n, N] or NULL; 8-byte aligned.
 *   ws      device workspace of at least nvfp4_mm_workspace_bytes(n, N, K)
 *           bytes, 256-byte aligned; reused by the next call only after this
 *           one's work on `stream` is ordered before it.
 * Supported shapes: n >= 0 (n = 0 enqueues nothing), N a positive multiple of
 * NVFP4_MM_TILE_N, K a positive multiple of 64; n * K and n * N below 2^31.
 * Errors: DA_ERR_INVALID_ARG (null or misaligned pointer, non-finite
 * global_scale, unknown x_dtype), DA_ERR_UNSUPPORTED (shape), DA_ERR_WORKSPACE,
 * DA_ERR_CUDA (a launch failed).  A pipeline wait inside the kernel that
 * hits its time limit records DA_DEVERR_TIMEOUT in the workspace header and
 * the kernel returns; y is then undefined. */
int nvfp4_mm(const void* x, int32_t x_dtype, const uint8_t* codes, const uint8_t* scales,
             float global_scale, int32_t n, int32_t N, int32_t K, float* y, void* y_bf16,
             void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then read the device error word (DA_DEVERR_* bits)
 * of the most recent nvfp4_mm call on workspace `ws` (each call clears it
 * when its first kernel starts; reading clears it too). */
int nvfp4_mm_read_error(void* ws, int32_t* code, void* stream);

/* ---- low-rank adapters of many requests ------------------------------- */

#define NVFP4_ADAPTER_MAX_RANK 128
#define NVFP4_ADAPTER_MAX_K (1 << 22)

/* Tests only: added to x_dtype of nvfp4_mm_adapters, one of them keeps the first stage
 * of every CTA of the first or second matmul kernel from ever getting full and bounds
 * waits to 2 ms, which drives that kernel's time-out path. */
#define NVFP4_X_TEST_STALL_DOWN 0x100
#define NVFP4_X_TEST_STALL_UP 0x200

/* Device workspace bytes of one nvfp4_mm_adapters call (0: shape not
 * supported): a 256-byte header, the plan (which rows make a tile with which
 * adapter) and the fp32 products t.  Needs no initialisation. */
size_t nvfp4_mm_adapters_workspace_bytes(int32_t n, int32_t N, int32_t K, int32_t n_adapters,
                                         int32_t max_rank);

/* Add each row's own low-rank adapter to the output of a matmul that all rows
 * share (nvfp4_mm's y):
 *
 *     t[i, r]   = sum_k bf16(x[i, k]) * A[id, r, k]                  (fp32)
 *     out[i, o] = y[i, o] + sum_{r < rank[id]} (scale[id] * t[i, r]) * B[id, o, r]
 *
 * with id = ids[i]; a row whose id is negative has no adapter, out = y.  Both
 * sums run on the tensor cores with fp32 accumulation over exact products: t
 * enters the second one as three bf16 terms that hold its 24 bits.  Orders are
 * fixed by K and the rank alone, so a row's bits depend only on its own x, y
 * and adapter, not on n, on its place or on the other rows.  Infinities, NaN and sums
 * that overflow follow the formulas: a result that does not come out finite is formed
 * again in plain fp32, in order of r.
 *   x       [n, K], fp32 or bf16 as x_dtype (NVFP4_X_*) says, 16-byte aligned.
 *   a       bf16 [n_adapters, max_rank, K], b  bf16 [n_adapters, N, max_rank],
 *           16-byte aligned.
 *   ranks   int32 [n_adapters] or NULL (all max_rank).  What a and b hold at or
 *           beyond an adapter's rank has no effect on the result.
 *   scales  fp32 [n_adapters] or NULL (all 1).
 *   ids     int32 [n].
 *   y, out  fp32 [n, N], 16-byte aligned; out may be y (rows without an adapter
 *           are then not touched).
 *   out_bf16  bf16 [n, N] or NULL, 16-byte aligned: out rounded to nearest even,
 *           all rows.  Otherwise out and out_bf16 overlap no other argument.
 *   ws      as for nvfp4_mm.
 * An id at or above n_adapters counts as none and sets DA_DEVERR_INDEX, a rank
 * outside [0, max_rank] is clamped and sets DA_DEVERR_LENGTH; a pipeline wait that
 * hits its time limit sets DA_DEVERR_TIMEOUT and the kernel returns, out and out_bf16
 * are then undefined.  Read the bits of the last call with nvfp4_mm_read_error(ws, ...);
 * a call with n = 0 clears them and does nothing else (ws may be NULL).
 * Supported shapes: n >= 0, N a positive multiple of NVFP4_MM_TILE_N, K a
 * positive multiple of 64 up to NVFP4_ADAPTER_MAX_K, max_rank a multiple of 16
 * up to NVFP4_ADAPTER_MAX_RANK, n_adapters >= 1; n * K, n * N below 2^31. */
int nvfp4_mm_adapters(const void* x, int32_t x_dtype, int32_t n, int32_t N, int32_t K,
                      const void* a, const void* b, int32_t n_adapters, int32_t max_rank,
                      const int32_t* ranks, const float* scales, const int32_t* ids,
                      const float* y, float* out, void* out_bf16, void* ws, size_t ws_bytes,
                      void* stream);

/* ---- logits ------------------------------------------------------------ */

/* Entries of a row's bias list at most: each of its tokens is looked for in it, so
 * that the work grows with the square (33 rows of 50001 tokens: 12 us with 40
 * entries, 49 with 400, 657 with 4096). */
#define NVFP4_LOGITS_MAX_BIAS 4096

/* What a decode step does to the logits of its vocabulary projection (nvfp4_mm's
 * y or y_bf16).  Plain data; a NULL list is an empty one; the three widths add
 * up to less than 2^29. */
typedef struct nvfp4_logits {
  int32_t batch;             /* B >= 0 rows                                    */
  int32_t vocab;             /* V tokens, 1 .. 2^30                              */
  int32_t x_dtype;           /* NVFP4_X_* of x                                 */
  const void* x;             /* [B, V], rows x_stride elements apart           */
  int64_t x_stride;          /* V .. 2^40 (one row: >= V)                       */
  const int32_t* prompt;     /* int32 [B, prompt_width]: the prompt's tokens   */
  const int32_t* prompt_lens; /* int32 [B]                                     */
  int32_t prompt_width;
  const int32_t* output;     /* int32 [B, output_width]: tokens generated      */
  const int32_t* output_lens; /* int32 [B]                                     */
  int32_t output_width;
  const float* repetition;   /* fp32 [B] or NULL (1): divides / multiplies     */
  const float* frequency;    /* fp32 [B] or NULL (0): per occurrence           */
  const float* presence;     /* fp32 [B] or NULL (0): once                     */
  const int32_t* bias_tokens; /* int32 [B, bias_width]                         */
  const float* bias_values;  /* fp32 [B, bias_width]                           */
  const int32_t* bias_lens;  /* int32 [B]                                      */
  int32_t bias_width;        /* <= NVFP4_LOGITS_MAX_BIAS                       */
  const uint32_t* mask;      /* [n_masks, ceil(V / 32)]: bit v % 32 of word    */
                             /* v / 32 set: token v may come                   */
  const int32_t* mask_ids;   /* int32 [B]: the row's mask, negative: none;     */
                             /* NULL: row b has mask b                         */
  int32_t n_masks;
  float* out;                /* fp32 [B, V], rows out_stride apart, or NULL    */
  int64_t out_stride;        /* V .. 2^40 (one row: >= V)                       */
  int32_t* tokens;           /* int32 [B] or NULL                              */
  int32_t* err;              /* device word for DA_DEVERR_* bits, or NULL      */
} nvfp4_logits;

/* For every row b and token v, in fp32 with one rounding for each operation:
 *
 *     l = x[b, v]
 *     v in the row's prompt or output:  l = l > 0 ? l / repetition : l * repetition
 *     v in its output, c times:         l = l - frequency * c;  l = l - presence
 *     v among its bias tokens:          l = l + (its bias values, added in order)
 *     the row's mask has v's bit clear: l = -inf
 *     out[b, v] = l
 *     tokens[b] = the lowest v among those with the largest l > -inf, or -1 if
 *                 there is none (every token masked, or -inf or NaN)
 *
 * A row's results depend on that row alone.  out may be x itself (fp32, same
 * stride); otherwise out and tokens overlap no other argument (rows of x and out that
 * lie in turn in one buffer need strides of the same size in bytes).  List entries at
 * or past a row's length are never read.  A length below 0 or above its width is clamped and
 * sets DA_DEVERR_LENGTH; a token outside [0, V) is skipped and a mask id at or
 * above n_masks counts as none, both set DA_DEVERR_INDEX.  Bits are OR-ed into
 * *err, never cleared.  Alignment: that of the element types; rows that start
 * on 16-byte boundaries (x, out) move in wider accesses.  One launch, no
 * workspace. */
int nvfp4_mm_logits(const nvfp4_logits* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MM_H */
