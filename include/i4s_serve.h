/*
 * i4s_serve.h -- C ABI of libi4s, second part: what a decode or verification
 * step needs between the packed INT4 products of i4s.h.  A paged KV cache
 * held in 4 bits, the block tables and slot maps that address it, attention
 * over it, and the log probabilities of given tokens.
 *
 * The conventions of i4s.h hold: every pointer to tensor data is a DEVICE
 * pointer unless marked "host"; the caller owns all memory and the library
 * allocates nothing; `stream` is a hipStream_t passed as void*, and the
 * current device has to be the one that the stream and the buffers belong to;
 * all argument checks run before anything is enqueued; calls are asynchronous
 * and can be captured into a HIP graph.  Values that only the device knows
 * (lengths, page numbers, slots, token ids) cannot be checked on the host:
 * the kernels check them and never read or write outside the buffers, as said
 * at each call.
 *
 * CACHE FORMAT (version 1).  A page holds page_size tokens of every KV head.
 *   The D = head_dim values of a token's K (and of its V) in one head are
 *   quantized in groups of G = group_size neighbouring channels:
 *     s = min(round_to_nearest_even_fp16(amax / 7), 9352), the scale (9352 is
 *         the largest whose 7-fold is finite in fp16);
 *     q = clamp(round_half_even(x / s), -7, 7) with a correctly rounded
 *         division, 0 where s is 0; nibble u = q + 8.
 *   The cache holds finite values only: a NaN is stored as 0 and an infinity
 *   as the largest value of its sign (7 * 9352).
 *   k_vals   : uint8 [num_pages][kv_heads][page_size][D/2].  32-bit word
 *              w = (D/32)*a + j (a = 0..3) of a token holds channels
 *              32j + 8a + e, e = 0..7; nibble slot k (bits 4k..4k+3) holds
 *              e = (0,2,4,6,1,3,5,7)[k].
 *   v_vals   : uint8 [num_pages][kv_heads][page_size/4][D/8 words][4 tokens]
 *              of 32-bit words.  The 16-bit half h = i*(D/64) + c of a
 *              token's words (i = 0..15, c = 0..D/64-1; half h is the lower
 *              (h even) or upper (h odd) half of word h/2) holds channels
 *              64c + 16e + i, e = 0..3, at bits 4e..4e+3.
 *   k_scales, v_scales : fp16 [num_pages][kv_heads][page_size/4][D/G][4 tokens].
 *   Slot s = page * page_size + offset names a token's place in every head.
 */
#ifndef I4S_SERVE_H
#define I4S_SERVE_H

#include <stddef.h>
#include <stdint.h>

#include "i4s.h"

#ifdef __cplusplus
extern "C" {
#endif

#define I4S_KV_FORMAT_VERSION 1
#define I4S_KV_MAX_REQUESTS 4096 /* requests of one i4s_kv_extend call */
#define I4S_MAX_TOP_K 32         /* alternatives of one i4s_token_logprobs row */
#define I4S_MAX_VOCAB (1 << 23)  /* columns of one i4s_token_logprobs row */
#define I4S_MAX_TREE 64          /* candidate tokens a tree mask can name */

/* Element types of activations and logits. */
typedef enum i4s_dtype { I4S_F16 = 0, I4S_BF16 = 1, I4S_F32 = 2 } i4s_dtype;

/* A 4-bit paged KV cache.  Plain data, like i4s_packed. */
typedef struct i4s_kv_cache {
  int32_t num_pages;   /* >= 1; num_pages * page_size < 2^31                  */
  int32_t page_size;   /* tokens of a page: 16, 32, 64, 128 or 256            */
  int32_t kv_heads;    /* 1 .. 1024                                           */
  int32_t head_dim;    /* D: 64, 128 or 256                                   */
  int32_t group_size;  /* G: 32, 64 or 128, at most D                         */
  int32_t reserved;    /* 0                                                   */
  uint8_t *k_vals;     /* each buffer 16-byte aligned                         */
  uint8_t *v_vals;
  uint16_t *k_scales;  /* fp16 bits                                           */
  uint16_t *v_scales;
} i4s_kv_cache;

/* Buffer sizes of a cache in bytes: of k_vals and of v_vals, and of k_scales
 * and of v_scales. */
typedef struct i4s_kv_sizes {
  uint64_t vals;
  uint64_t scales;
} i4s_kv_sizes;

/* Sizes of the buffers of a cache.  Host-only and pure.  Errors:
 * I4S_ERR_INVALID_ARGUMENT for a size outside the ranges of i4s_kv_cache or
 * out == NULL. */
i4s_status i4s_kv_cache_sizes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                              int32_t group_size, i4s_kv_sizes *out /* host */);

/* Bits of the flags word that i4s_kv_extend writes. */
#define I4S_KV_BAD_LENGTH 1  /* a length is negative, or the sum passes 2^31 - 1  */
#define I4S_KV_ROW_FULL 2    /* a request needs more pages than its table row has */
#define I4S_KV_NO_PAGES 4    /* the free list has too few pages                   */
#define I4S_KV_NO_SLOTS 8    /* more new tokens than `capacity`                   */
#define I4S_KV_BAD_COUNT 16  /* free_count lies outside [0, free_entries]         */

/* Gives the new tokens of n requests their pages and slots.  Request i holds
 * lens[i] tokens and adds new_lens[i] (0 or more).  It keeps the pages that
 * it has, and takes ceil((lens+new)/page_size) - ceil(lens/page_size) new ones
 * from the end of the free list: the call's j-th new page, counted in request
 * order and then by position, is free_pages[free_count - 1 - j].
 *   table     : int32 [n][width], page numbers of every request in order of
 *               position; only the entries of new pages are written.
 *   free_pages: int32 [free_entries]; its first *free_count entries are free.
 *   lens_out  : int32 [n], lens + new_lens.
 *   q_start   : int32 [n+1], where the new tokens of each request begin.
 *   slots     : int32 [capacity], the slot of each new token in request order
 *               (table entry * page_size + position % page_size), then -1;
 *               also -1 where the page number is negative or its slots would
 *               pass 2^31 - 1.
 *   positions : int32 [capacity], the position of each new token in its
 *               request, then 0.
 *   free_count_out : int32, the free pages that are left.
 *   flags     : int32, 0 or the I4S_KV_* bits of what does not fit.  If any
 *               bit is set the call changes nothing: lens_out = lens,
 *               free_count_out = free_count, table unchanged, q_start all 0,
 *               slots all -1, positions all 0.
 * n is 0 .. I4S_KV_MAX_REQUESTS, width 1 or more, page_size 16, 32, 64, 128 or
 * 256, capacity and free_entries 0 or more.  Every pointer 4-byte aligned; none may be
 * NULL but table, lens, new_lens and lens_out when n is 0, slots and positions
 * when capacity is 0, and free_pages when free_entries is 0.  No output may
 * overlap an input or another output: the new lengths and the new count go
 * into buffers of their own, which serve as the inputs of the next call.
 * One kernel launch.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_kv_extend(int32_t *table, int32_t n, int32_t width, int32_t page_size, const int32_t *lens,
                         const int32_t *new_lens, const int32_t *free_pages, int32_t free_entries,
                         const int32_t *free_count, int32_t capacity, int32_t *lens_out, int32_t *q_start,
                         int32_t *slots, int32_t *positions, int32_t *free_count_out, int32_t *flags,
                         void *stream);

/* Quantizes the K and V of `tokens` tokens into their slots.
 *   k, v   : [tokens][kv_heads][D] of dtype I4S_F16 or I4S_BF16; the channels
 *            of a head lie next to each other, tokens and heads at the given
 *            strides (in elements, 0 .. 2^40, multiples of 8); 16-byte aligned.
 *   slots  : int32 [tokens], 4-byte aligned.  A token whose slot is outside
 *            [0, num_pages * page_size) is not stored (-1 marks padding).  A
 *            slot may be named once: what is stored for a slot named twice is
 *            a mix of the two.
 * k, v and slots must not overlap the cache; kv_heads * (D * tokens + 2048) is
 * below 2^34.  One kernel launch.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_kv_append(const i4s_kv_cache *cache /* host */, const void *k, const void *v, int32_t dtype,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                         int64_t v_head_stride, const int32_t *slots, int32_t tokens, void *stream);

/* Reads tokens back: k_out, v_out = s * q, rounded once to dtype (I4S_F16,
 * I4S_BF16 or I4S_F32), [tokens][kv_heads][D] contiguous, 16-byte aligned.  A
 * token whose slot is outside the cache gives zeros.  The outputs must not
 * overlap the cache, slots or one another; kv_heads * (D * tokens + 2048) is
 * below 2^34.  One kernel launch.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_kv_read(const i4s_kv_cache *cache /* host */, const int32_t *slots, int32_t tokens,
                       int32_t dtype, void *k_out, void *v_out, void *stream);

/* Attention of query tokens over the 4-bit cache.  Sequence i holds lens[i]
 * tokens, the last q_start[i+1] - q_start[i] of which are its query tokens
 * (already appended); ctx = lens[i] - that number are before them.  Query
 * token t of a sequence sees the keys at positions up to ctx + t, or with a
 * tree mask the keys before ctx and those at ctx + b for each bit b set in
 * its mask (its ancestors and itself; only positions below lens[i]):
 *   out = sum_j p_j v_j, p = softmax(scale * q . k_j).
 * A token that sees no key gets out = 0 and lse = -inf.  Query head h reads
 * KV head h / (q_heads / kv_heads).  Scores, softmax statistics and sums are
 * held in fp32; a score is off by about 2^-24 scale sum |q| (|k| + 24 s), s K's
 * scales.  A probability times V's scale is exact to 2^-16 of itself.  With many
 * rows and groups (D/G >= 8, or D = 128, G = 32 and more than 16 query rows of a
 * KV head) a probability times a value is exact to 2^-21 for fp16 and 2^-10 for
 * bf16 outputs, and where the probability is below 2^-21 of the row's largest it
 * is off by up to 2^-32 of that largest one instead. */
typedef struct i4s_attention_args {
  const i4s_kv_cache *cache; /* host                                          */
  const void *q;             /* [num_tokens][q_heads][D], channels adjacent,  */
                             /* 16-byte aligned                               */
  int64_t q_token_stride;    /* in elements, 0 .. 2^40, multiples of 8        */
  int64_t q_head_stride;
  int32_t dtype;             /* of q and out: I4S_F16 or I4S_BF16             */
  int32_t q_heads;           /* a multiple of kv_heads, at most 65536         */
  int32_t num_tokens;        /* rows of q and out, 0 or more                  */
  int32_t num_seqs;          /* 0 .. 65535                                    */
  const int32_t *table;      /* [num_seqs][table_width] page numbers          */
  int32_t table_width;       /* 1 or more, times page_size at most 2^30       */
  const int32_t *lens;       /* [num_seqs]                                    */
  const int32_t *q_start;    /* [num_seqs+1], non-decreasing, or NULL: one    */
                             /* token each, num_tokens == num_seqs            */
  int32_t max_q;             /* largest number of query tokens of a sequence, */
                             /* 1 .. 2^20, times q_heads below 2^23           */
  int32_t max_len;           /* largest length (0: table_width * page_size);  */
                             /* sizes the launch                              */
  float scale;               /* > 0, finite                                   */
  const int64_t *tree_mask;  /* [num_tokens], 8-byte aligned, or NULL; needs  */
                             /* max_q <= I4S_MAX_TREE                         */
  void *out;                 /* [num_tokens][q_heads][D] contiguous, 16-byte  */
                             /* aligned                                       */
  float *lse;                /* [num_tokens][q_heads], natural logarithm of   */
                             /* the sum of exp(scale * q . k), or NULL        */
  void *workspace;           /* 16-byte aligned; may be NULL if 0 bytes       */
  uint64_t workspace_bytes;
} i4s_attention_args;

/* Bytes of workspace that i4s_attention needs for these sizes (the pointers
 * are not looked at, save cache); 0 when the call does not split the keys.
 * Host-only and pure.  Errors: I4S_ERR_INVALID_ARGUMENT. */
i4s_status i4s_attention_workspace_size(const i4s_attention_args *a /* host */, uint64_t *bytes /* host */);

/* The call.  Every row of out (and lse) that belongs to a sequence is
 * written; rows from q_start[num_seqs] on, and tokens of a sequence past
 * max_q, are left as they were.  A length below 0 counts as 0, one beyond
 * table_width * page_size as that; a q_start outside [0, num_tokens] is moved
 * into it; the keys of a page number outside [0, num_pages) are read from the
 * nearest page inside.  max_len below a length costs time, not correctness.
 * One kernel launch, or two where the keys are split; results do not depend
 * on the order of blocks.  Calls that share a workspace must not overlap.
 * out, lse and workspace must not overlap one another or an input.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_WORKSPACE_TOO_SMALL,
 * I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_attention(const i4s_attention_args *a /* host */, void *stream);

/* Log probabilities of given tokens, the entropy of each row's distribution
 * and its top alternatives, over logits [rows][vocab] (row r at r * stride
 * elements, rows below 2^23): with m = max_j x_j and l = sum_j exp(x_j - m),
 *   logprobs[r] = x[tokens[r]] - m - ln l            (fp32)
 *   entropy[r]  = ln l - sum_j (x_j - m) exp(x_j - m) / l   (fp32, nats)
 *   top_ids[r][i], top_logprobs[r][i], i < top_k: the largest logits in
 *                 falling order, among equal ones the lower index first (-0
 *                 equals 0, a NaN counts as +inf), int32 and fp32.
 *   logits  : dtype I4S_F16, I4S_BF16 or I4S_F32, aligned to its element;
 *             stride vocab .. 2^40; vocab 1 .. I4S_MAX_VOCAB.
 *   tokens  : int64 [rows], 8-byte aligned; one outside [0, vocab) gives NaN.
 *   top_k   : 0 .. min(I4S_MAX_TOP_K, vocab); top_ids and top_logprobs may be
 *             NULL when it is 0.
 * -inf marks a token that cannot occur (probability 0).  A row of nothing but
 * -inf has no distribution: its log probabilities are -inf and its entropy 0.
 * A row with a NaN or +inf gives NaN log probabilities and entropy.
 * workspace: as i4s_token_logprobs_workspace_size says, 16-byte aligned.  One
 * launch, or two where rows are split.  Outputs 4-byte aligned; they and the
 * workspace must not overlap one another or an input.
 * Errors: I4S_ERR_INVALID_ARGUMENT, I4S_ERR_WORKSPACE_TOO_SMALL,
 * I4S_ERR_UNSUPPORTED, I4S_ERR_DEVICE. */
i4s_status i4s_token_logprobs(const void *logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t stride,
                              const int64_t *tokens, int32_t top_k, float *logprobs, float *entropy,
                              int32_t *top_ids, float *top_logprobs, void *workspace,
                              uint64_t workspace_bytes, void *stream);

/* Bytes of workspace of such a call; may be 0.  Host-only and pure.  Errors:
 * I4S_ERR_INVALID_ARGUMENT. */
i4s_status i4s_token_logprobs_workspace_size(int32_t dtype, int32_t rows, int32_t vocab, int32_t top_k,
                                             uint64_t *bytes /* host */);

#ifdef __cplusplus
}
#endif

#endif /* I4S_SERVE_H */
