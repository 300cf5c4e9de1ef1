/*
 * qpn_prompt.h - C ABI of libqpn.so for a prompt's step, where qpn.h and
 * qpn_decode.h serve steps of up to 16 rows: products of any number of rows
 * with weights of 8 bits and a scale for each block of 128, attention of a
 * chunk of new tokens over the 4-bit paged cache, and the log-probabilities of
 * given tokens.
 *
 * The conventions of qpn.h hold: device pointers, caller-owned buffers, work
 * enqueued on `stream` (NULL = the default stream) without waiting, arguments
 * checked on the host before any HIP call, no memory allocated here, no
 * global state. Every call may be captured into a HIP graph; lengths, tables
 * and tokens are read on the device, so a replay follows their contents. A
 * workspace's contents need no preparation and carry nothing to the next
 * call; calls that may run at once need one each.
 */
#ifndef QPN_PROMPT_H
#define QPN_PROMPT_H

#include "qpn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The type of x in a block product that is E4M3 codes already. */
#define QPN_DT_E4M3 4

/* Quantizes x [rows][k] of `dtype` (F16, BF16 or F32, rows `stride` elements
 * apart) to E4M3 codes with a scale for each 128 columns and `block_rows` rows
 * (1: activations; 128: weights): the least power of two s >= 2^-126 with
 * amax <= 448 s, 1 for a block of zeros. code = E4M3(x / s), nearest with ties
 * to even; the quotient is exact, so each code is the nearest there is. inf
 * and NaN get the NaN code and do not count for amax. k may be any number; the
 * last block of a row (and of the rows) may be short.
 *   codes   [rows][k], rows code_stride bytes apart
 *   scales  [ceil(rows / block_rows)][ceil(k / 128)] by strides in elements */
qpn_status qpn_fp8_block_quantize(const void* x_dev, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                  int32_t block_rows, uint8_t* codes_dev, int64_t code_stride, float* scales_dev,
                                  int64_t scale_row_stride, int64_t scale_block_stride, void* stream);

/* y[m][n] = sum over k of (x code * x scale)[m][k] * (w code * w scale)[n][k],
 * x with a scale for each row and 128 columns, w with one for each 128 rows
 * and 128 columns (any fp32 scales). A block's sum is scaled and added to the
 * others' in fp32, and y is rounded once. For y of F32 the products of codes are
 * exact and their sums fp32. For y of F16 or BF16 a block is summed by the 8-bit
 * matrix instruction, which keeps its products to about 2^-11 of the block's
 * largest: a result of random blocks is 1.4e-5 of itself off by that, a tenth
 * and less of its rounding, but where large products of a block cancel it is off by
 * 2^-11 of what has cancelled (an fp32 y is not). With x of F16, BF16 or F32 it is quantized first, as
 * by qpn_fp8_block_quantize with block_rows 1, into the workspace. NaN codes
 * make the outputs that they enter NaN. */
typedef struct {
  const void* x;          /* device: [m][k] of x_dtype, rows x_stride elements apart */
  const float* x_scales;  /* device: E4M3 x: [m][ceil(k / 128)] by strides; else NULL */
  const uint8_t* w;       /* device: [n][k] E4M3 codes, 16-byte aligned */
  const float* w_scales;  /* device: [ceil(n / 128)][ceil(k / 128)] by strides */
  void* y;                /* device: [m][n] of y_dtype, rows y_stride elements apart */
  int64_t x_stride;       /* E4M3 x: a multiple of 16, and x 16-byte aligned */
  int64_t x_scale_row_stride;
  int64_t x_scale_block_stride;
  int64_t w_stride;       /* bytes, a multiple of 16 */
  int64_t w_scale_row_stride;
  int64_t w_scale_block_stride;
  int64_t y_stride;       /* >= n */
  int64_t m;              /* 0 .. 2^22 */
  int64_t n;              /* 0 .. 2^24 */
  int64_t k;              /* 0 .. 2^20, a multiple of 16 */
  int32_t x_dtype;        /* F16, BF16, F32 or E4M3 */
  int32_t y_dtype;        /* F16, BF16 or F32 */
} qpn_fp8_block_gemm_args;

/* Workspace of a call with these sizes, whatever the type of x (0 for sizes
 * that are refused, and where none is needed). */
size_t qpn_fp8_block_workspace_bytes(int64_t m, int64_t n, int64_t k);

qpn_status qpn_fp8_block_gemm(const qpn_fp8_block_gemm_args* args, void* workspace_dev, size_t workspace_bytes,
                              void* stream);

/* Attention of chunks of new tokens over their sequences' cached tokens and
 * themselves. Sequence b has kv_len[b] tokens in the 4-bit cache, in pages
 * table[b * table_stride + t / page_size], and the new tokens q_start[b] ..
 * q_start[b + 1] - 1 (q_start NULL: max_q_len each) with rows of q, k and v;
 * their keys and values are read from k and v as they are, and need not have
 * been appended. Row i sits at position kv_len + i and sees the cached tokens
 * (position t) and the new ones up to itself, with window > 0 those at
 * positions above its own less window. Query head h reads kv head
 * h / (heads / kv_heads).
 *   out[row][head] = sum_t softmax_t(scale * q . k_t) v_t      (dtype of q)
 *   lse[row][head] = log sum_t exp(scale * q . k_t)            (fp32, may be NULL)
 * A page index outside the pool holds no tokens: its positions are not seen.
 * Tokens that a row does not see have no effect on it, whatever k, v or the
 * cache hold there. Rows that no sequence has are not written.
 * All sums are fp32. Rounded to fewer bits are: the softmax weights before
 * their product with the values, to fp16 for cached tokens and to the type of q
 * for new ones (each is off by at most half a step of that type, or, in fp16, by 2^-33 of
 * the row's largest); and, for the cached tokens, q of bf16, which is scaled by
 * a power of two that takes a row's largest element to 2^15 and then held in
 * fp16 (elements keep their 8 bits down to 2^-32 of the largest). lse sums the
 * weights unrounded. Scores are to be below 2^26 in magnitude. */
typedef struct {
  const void* q;           /* device: [rows][heads][head_dim] by strides */
  const void* k;           /* device: [rows][kv_heads][head_dim] by strides */
  const void* v;
  void* out;               /* device: contiguous, 16-byte aligned */
  float* lse;              /* device: [rows][heads], or NULL */
  const int32_t* table;    /* device: page indices */
  const int32_t* kv_len;   /* device: [batch], each 0 .. max_kv_len */
  const int32_t* q_start;  /* device: [batch + 1] from 0 to rows, or NULL */
  int64_t q_token_stride;  /* elements */
  int64_t q_head_stride;
  int64_t k_token_stride;
  int64_t k_head_stride;
  int64_t v_token_stride;
  int64_t v_head_stride;
  int64_t table_stride;    /* entries a sequence, table_stride * page_size >= max_kv_len */
  int32_t dtype;           /* F16 or BF16, of q, k, v and out */
  int32_t layer;
  int32_t heads;           /* a multiple of kv_heads */
  int32_t batch;
  int32_t rows;            /* all sequences' new tokens */
  int32_t max_q_len;       /* no sequence has more new tokens */
  int32_t max_kv_len;      /* no sequence has more cached tokens; longer ones are cut there */
  int32_t window;          /* 0: none */
  float scale;             /* finite and > 0 */
  int32_t reserved;        /* 0 */
} qpn_kv4_chunk_args;

/* Workspace of a call (its pointers may be NULL; 0: none is needed). */
size_t qpn_kv4_chunk_workspace_bytes(const qpn_kv4_cache* cache, const qpn_kv4_chunk_args* args);

qpn_status qpn_kv4_chunk_attention(const qpn_kv4_cache* cache, const qpn_kv4_chunk_args* args, void* workspace_dev,
                                   size_t workspace_bytes, void* stream);

/* Log-probabilities of given tokens. With x a row's logits, t its temperature
 * and p = softmax(x / t):
 *   logprobs[row]     = log p[token]
 *   entropy[row]      = -sum p log p
 *   rank[row]         = how many tokens come before the given one
 *   top_tokens[row]   = the first `top` tokens, and top_logprobs their log p
 * where tokens with larger logits come first, equal ones in the order of their
 * index. A token outside 0 .. vocab - 1 gives 0 and a rank of -1. NaN logits
 * count as -inf. Infinite logits share p = 1 among themselves; a row of -inf
 * alone gives log p = -inf and an entropy of 0. A temperature that is 0, below
 * or NaN counts as 1. Sums are fp32 over at most 128 elements of a row and 64
 * bits beyond. */
typedef struct {
  const void* logits;        /* device: [rows][vocab], rows row_stride elements apart */
  const int32_t* tokens;     /* device: [rows], or NULL with logprobs and rank NULL */
  const float* temperature;  /* device: [rows], or NULL (1) */
  float* logprobs;           /* device: [rows], may be NULL */
  float* entropy;            /* device: [rows], may be NULL */
  int32_t* rank;             /* device: [rows], may be NULL */
  int32_t* top_tokens;       /* device: [rows][top], NULL only if top is 0 */
  float* top_logprobs;       /* device: [rows][top], NULL only if top is 0 */
  int64_t row_stride;        /* elements */
  int32_t dtype;             /* F16, BF16 or F32 */
  int32_t rows;              /* 0 .. 2^20 */
  int32_t vocab;             /* 1 .. 2^24 */
  int32_t top;               /* 0 .. 64, at most vocab */
} qpn_logprobs_args;

/* Workspace of a call with these sizes (0: none is needed, or refused sizes). */
size_t qpn_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top);

qpn_status qpn_token_logprobs(const qpn_logprobs_args* args, void* workspace_dev, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QPN_PROMPT_H */
