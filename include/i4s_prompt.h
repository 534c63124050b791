/*
 * i4s_prompt.h -- C ABI of libi4s, third part: a prompt's step.  A prompt
 * brings hundreds or thousands of tokens at once; the packed products of i4s.h
 * take 16.  Here are products of any number of tokens with weights in
 * microscaled 4-bit floating point, the quantization to that format, and
 * attention of whole prompts over their own 16-bit keys and values (which
 * i4s_kv_append of i4s_serve.h then writes into the cache).
 *
 * The conventions of i4s.h and i4s_serve.h hold: every pointer to tensor data
 * is a DEVICE pointer unless marked "host"; the caller owns all memory and the
 * library allocates nothing; `stream` is a hipStream_t passed as void*, and the
 * current device has to be the one that the stream and the buffers belong to;
 * all argument checks run before anything is enqueued; calls are asynchronous
 * and can be captured into a HIP graph.  Values that only the device knows
 * (where sequences begin) cannot be checked on the host: the kernels move them
 * into range and never read or write outside the buffers.
 *
 * MICROSCALED FORMAT (version 1).  A matrix [rows][cols], cols a multiple of
 *   32.  32 neighbouring columns of a row are a block with one scale:
 *     e = max(floor(log2(amax)) - 2, -127), -127 where amax is 0;
 *     scale byte e + 127 (e8m0);
 *     value = x / 2^e rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *         (e2m1; a tie goes to the even code, beyond 6 to 6), the sign kept;
 *         codes 0..7 in that order, sign bit 8.
 *   A block that holds an infinity or a NaN gets scale byte 255 and codes 0:
 *   every value of it reads as NaN, and so does every product with it.
 *   vals   : uint8 [ceil(rows/16)][2 * ceil(cols/256)][64 lanes][16].  Lane
 *            16 * b + r of a tile (16 rows x 128 columns) holds row r, columns
 *            32 b .. 32 b + 31; byte j its columns 2j (low four bits) and
 *            2j + 1.
 *   scales : uint8 [ceil(rows/16)][ceil(cols/512)][64 lanes][4].  Byte c of
 *            lane 16 * b + r is the scale of row r, columns 128 c + 32 b and
 *            on, of 512 columns.
 *   Columns past cols are held as 0 with scale byte 0; rows past rows may hold
 *   anything.  A matrix takes 4.25 bits a value.
 */
#ifndef I4S_PROMPT_H
#define I4S_PROMPT_H

#include <stddef.h>
#include <stdint.h>

#include "i4s.h"
#include "i4s_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

#define I4S_MX_FORMAT_VERSION 1

/* A matrix in the microscaled format.  Plain data, like i4s_packed.  A call
 * takes matrices of ceil(rows/16) * ceil(cols/512) <= 2^25 - 4, about 2^38
 * values. */
typedef struct i4s_mx {
  int32_t rows;    /* 0 .. 2^24                                              */
  int32_t cols;    /* a multiple of 32, 32 .. 2^20                           */
  uint8_t *vals;   /* each buffer 16-byte aligned                            */
  uint8_t *scales;
} i4s_mx;

/* Buffer sizes in bytes. */
typedef struct i4s_mx_buffers {
  uint64_t vals;
  uint64_t scales;
} i4s_mx_buffers;

/* Sizes of the buffers of a matrix.  Host-only and pure.  Errors:
 * I4S_ERR_INVALID_ARGUMENT for a size outside the ranges of i4s_mx, rows and
 * cols together included, or out == NULL. */
i4s_status i4s_mx_sizes(int32_t rows, int32_t cols, i4s_mx_buffers *out /* host */);

/* Quantizes x ([rows][cols] of dtype I4S_F16 or I4S_BF16; columns adjacent,
 * rows at `stride` elements, cols .. 2^40 and a multiple of 8, 16-byte
 * aligned) into out's buffers.  x must not overlap them.  One kernel launch.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_mx_quantize(const void *x, int32_t dtype, int64_t stride, const i4s_mx *out /* host */, void *stream);

/* Reads a matrix back: out [rows][cols] contiguous, 16-byte aligned, the held
 * values rounded once to dtype (I4S_F16, I4S_BF16 or I4S_F32; bf16 and fp32
 * hold all of them).  out must not overlap the matrix.  One kernel launch.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_mx_read(const i4s_mx *m /* host */, int32_t dtype, void *out, void *stream);

/* y = X W^T for tokens X [tokens][cols] and a weight W [rows][cols]:
 * y[t][n] = sum_k X[t][k] W[n][k], summed in fp32, rounded once to y_dtype.  A
 * sum that passes fp32's range on its way ends as an infinity (of its sign, if
 * its terms have one) or NaN; below the normal range it keeps subnormal numbers.
 * X is given in the microscaled format or as 16-bit values, which the call
 * quantizes as i4s_mx_quantize does; y is the same, bit for bit.
 * ceil(tokens/128) * ceil(rows/128) is at most 2^23 - 1, about 2^37 outputs, and
 * [tokens][cols] within the limit of i4s_mx. */
typedef struct i4s_mx_product_args {
  const i4s_mx *w;         /* host; the weight                               */
  const i4s_mx *x;         /* host; the tokens, or NULL: x_values            */
  const void *x_values;    /* [tokens][cols] 16-bit, 16-byte aligned         */
  int64_t x_stride;        /* of x_values, in elements: cols .. 2^40, a      */
                           /* multiple of 8                                  */
  int32_t x_dtype;         /* of x_values: I4S_F16 or I4S_BF16               */
  int32_t tokens;          /* 0 .. 2^24; x->rows where x is given            */
  void *y;                 /* [tokens][rows] at y_stride elements, aligned   */
  int64_t y_stride;        /* to its element; rows .. 2^40                   */
  int32_t y_dtype;         /* I4S_F16, I4S_BF16 or I4S_F32                   */
  int32_t reserved;        /* 0                                              */
  void *workspace;         /* 16-byte aligned; may be NULL if 0 bytes        */
  uint64_t workspace_bytes;
} i4s_mx_product_args;

/* Bytes of workspace that i4s_mx_product needs for these sizes (pointers are
 * not looked at, save w and whether x is NULL); may be 0.  Host-only and pure.
 * Errors: I4S_ERR_INVALID_ARGUMENT. */
i4s_status i4s_mx_product_workspace_size(const i4s_mx_product_args *a /* host */, uint64_t *bytes /* host */);

/* The call.  One or two kernel launches; results do not depend on the order
 * of blocks.  Calls that share a workspace must not overlap.  y and the
 * workspace must not overlap one another or an input.  Columns of y between
 * rows and y_stride are left as they were.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_WORKSPACE_TOO_SMALL,
 * I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_mx_product(const i4s_mx_product_args *a /* host */, void *stream);

/* Attention of packed sequences over their own keys and values.  Sequence i
 * has the query tokens q_start[i] .. q_start[i+1] of q and the keys k_start[i]
 * .. k_start[i+1] of k and v.  With `causal`, query token t of nq sees the keys
 * j <= nk - nq + t of its nk (the last token sees all; where nq > nk the first
 * ones see none); without it every token sees all keys:
 *   out = sum_j p_j v_j, p = softmax(scale * q . k_j).
 * A token that sees no key, or only scores of -inf, gets lse = -inf and, where
 * the values that it sees are finite, out = 0.  Query head h reads KV head
 * h / (q_heads / kv_heads).  What is in keys and values that a token does not
 * see does not matter to it, infinities and NaN included.  What it sees does,
 * whatever its probability: a NaN among the values, or infinities of both
 * signs, make that channel of its output NaN, other infinities make it that
 * infinity; a NaN among q . k_j, or one above fp32's range, makes all of its
 * output and lse NaN, and so may two whose difference is above it.  Scores,
 * softmax statistics and sums are held in fp32; probabilities are rounded to the
 * type of v before they multiply it (2^-8 of a probability for bf16; 2^-11 for
 * fp16, or 2^-32 of the row's largest where that is more). */
typedef struct i4s_prompt_args {
  const void *q;             /* [num_tokens][q_heads][D]; k, v               */
  const void *k;             /* [num_keys][kv_heads][D]: channels adjacent,  */
  const void *v;             /* 16-byte aligned                              */
  int64_t q_token_stride;    /* in elements, multiples of 8: 0 .. 2^23 from  */
  int64_t q_head_stride;     /* token to token, 0 .. 2^40 from head to head  */
  int64_t k_token_stride;
  int64_t k_head_stride;
  int64_t v_token_stride;
  int64_t v_head_stride;
  int32_t dtype;             /* of q, k, v and out: I4S_F16 or I4S_BF16      */
  int32_t head_dim;          /* D: 64, 128 or 256                            */
  int32_t q_heads;           /* a multiple of kv_heads, at most 65536        */
  int32_t kv_heads;          /* 1 .. 1024                                    */
  int32_t num_tokens;        /* rows of q and out, 0 .. 2^30                 */
  int32_t num_keys;          /* rows of k and v, 0 .. 2^30                   */
  int32_t num_seqs;          /* 0 .. 65535                                   */
  int32_t max_q;             /* largest number of query tokens of a          */
                             /* sequence, 1 .. 2^24; num_seqs * kv_heads     */
                             /* times its blocks of 128 rows (tokens x query */
                             /* heads of a KV head) below 2^23               */
  int32_t max_k;             /* largest number of keys of a sequence (0:     */
                             /* num_keys); sizes the launch                  */
  int32_t causal;            /* 0 or 1                                       */
  float scale;               /* > 0, finite                                  */
  int32_t reserved;          /* 0                                            */
  const int32_t *q_start;    /* [num_seqs+1], non-decreasing; both NULL: one */
  const int32_t *k_start;    /* sequence of all tokens and keys, num_seqs 1  */
  void *out;                 /* [num_tokens][q_heads][D] contiguous, 16-byte */
                             /* aligned                                      */
  float *lse;                /* [num_tokens][q_heads], natural logarithm of  */
                             /* the sum of exp(scale * q . k), or NULL       */
  void *workspace;           /* 16-byte aligned; may be NULL if 0 bytes      */
  uint64_t workspace_bytes;
} i4s_prompt_args;

/* Bytes of workspace that i4s_prompt_attention needs for these sizes (pointers
 * are not looked at); 0 when the call does not split the keys.  Host-only and
 * pure.  Errors: I4S_ERR_INVALID_ARGUMENT. */
i4s_status i4s_prompt_attention_workspace_size(const i4s_prompt_args *a /* host */, uint64_t *bytes /* host */);

/* The call.  Every row of out (and lse) that belongs to a sequence is written;
 * rows before q_start[0] and from q_start[num_seqs] on, and tokens of a
 * sequence past max_q, are left as they were.  A start outside [0, num_tokens]
 * (num_keys) is moved into it; a sequence that ends before it begins is empty,
 * and a row that two sequences claim then holds values of either.
 * max_k below a number of keys costs time, not correctness.  One kernel
 * launch, or two where the keys are split; results do not depend on the order
 * of blocks.  Calls that share a workspace must not overlap.  out, lse and
 * workspace must not overlap one another or an input.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_WORKSPACE_TOO_SMALL,
 * I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_prompt_attention(const i4s_prompt_args *a /* host */, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* I4S_PROMPT_H */
