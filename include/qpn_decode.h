/*
 * qpn_decode.h - C ABI of libqpn.so for what a verify step does between and
 * after its weight products (qpn.h): the keys and values of the step's tokens
 * enter a paged cache held in 4 bits, the step's rows attend to it, the
 * drafted tokens are verified against the target's probabilities, and pages
 * are copied when sequences fork or the pool is compacted.
 *
 * The conventions of qpn.h hold: device pointers, caller-owned buffers, work
 * enqueued on `stream` (NULL = the default stream) without waiting, arguments
 * checked on the host before any HIP call, no memory allocated here, no
 * global state. Every call may be captured into a HIP graph; lengths, tables,
 * slots and counts are read on the device, so a replay follows their
 * contents.
 *
 * The 4-bit cache. data holds [layers][pages][page_bytes] bytes. A page keeps
 * page_size tokens; kv head h has the segment of
 *   segment = page_size * head_dim * 9 / 8 bytes at h * segment,
 * made of four arrays in this order (D = head_dim):
 *   K codes   [page_size][D / 2]             byte j: elements 2j (low nibble), 2j + 1
 *   V codes   [page_size / 4][16][4][D / 32] token t: [t / 4][i][t % 4] holds its
 *                                            elements [i * D / 16, (i + 1) * D / 16)
 *   K scales  [page_size][D / 16]            an E4M3 byte per 16 elements
 *   V scales  [page_size / 4][D / 16][4]     token t: [t / 4][block][t % 4]
 * and an element is E2M1(code) * E4M3(block scale) * k_scale (or v_scale): the
 * NVFP4 format of qpn.h. Offset o of page p is slot p * page_size + o.
 */
#ifndef QPN_DECODE_H
#define QPN_DECODE_H

#include "qpn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QPN_DT_F16 = 1, QPN_DT_BF16 = 2, QPN_DT_F32 = 3 } qpn_dtype;

typedef struct {
  void* data;        /* device, 16-byte aligned */
  int64_t pages;     /* 0 .. 2^31 - 1 */
  int32_t layers;    /* >= 1 */
  int32_t page_size; /* tokens a page: 16, 32, 64, 128 or 256 */
  int32_t kv_heads;  /* 1 .. 1024 */
  int32_t head_dim;  /* 64, 128 or 256 */
  float k_scale;     /* tensor scales, finite and > 0 */
  float v_scale;
} qpn_kv4_cache;

/* Bytes of one page (0 for sizes the cache does not take). */
size_t qpn_kv4_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim);

/* Quantizes k and v ([tokens][kv_heads][head_dim] of `dtype`, F16 or BF16, the
 * strides in elements, a head's elements contiguous) into slots[t] of one
 * layer. A block's scale is E4M3(min(448, amax / 6 / tensor scale)) and its
 * codes E2M1(x / (scale * tensor scale)), in fp32, nearest with ties to even:
 * the rule of qpn_quantize_nvfp4. +-inf is held as the largest value of its
 * block, NaN as 0 (the cache has no code for them). A slot outside the pool
 * is skipped. No slot may be given twice in one call: its blocks would be those
 * of either token, codes of one under scales of the other among them. */
qpn_status qpn_kv4_append(const qpn_kv4_cache* cache, int32_t layer, const void* k_dev, const void* v_dev,
                          int32_t dtype, int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                          int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots_dev, void* stream);

/* The values that slots[t] of one layer stand for, as [tokens][kv_heads]
 * [head_dim] of `dtype` (F16, BF16 or F32; rounded once, F16 saturating);
 * zeros for a slot outside the pool. */
qpn_status qpn_kv4_read(const qpn_kv4_cache* cache, int32_t layer, const int64_t* slots_dev, int64_t tokens,
                        int32_t dtype, void* k_dev, void* v_dev, void* stream);

/* Copies page src[i] onto page dst[i] in every layer, for all i at once: no
 * page may be both a source and a destination, or twice a destination. A pair
 * with a page outside the pool is skipped. */
qpn_status qpn_kv4_copy_pages(const qpn_kv4_cache* cache, const int32_t* src_dev, const int32_t* dst_dev,
                              int64_t count, void* stream);

/* Attention of each sequence's last rows over its cached tokens.
 * Sequence b has kv_len[b] tokens (the rows' own among them; append first), in
 * pages table[b * table_stride + t / page_size], and its rows are
 * q_start[b] .. q_start[b + 1] - 1 of q (q_start NULL: max_q_len rows each).
 * Row i of n sits at position kv_len - n + i and sees tokens t with
 *   t <= position, and with window > 0 also t > position - window.
 * Query head h reads kv head h / (heads / kv_heads).
 *   out[row][head] = sum_t softmax_t(scale * q . k_t) v_t      (dtype of q)
 *   lse[row][head] = log sum_t exp(scale * q . k_t)            (fp32, may be NULL)
 * A row that sees no token (a length of 0, a position below 0) gets zeros and
 * -inf. A page index outside the pool holds no tokens: its positions are not
 * seen. Rows that no sequence has are not written. Cached values enter the
 * products exactly, all sums are fp32, and two factors are rounded to fp16:
 *  - q of bf16, scaled by a power of two that takes a row's largest element to
 *    2^15: elements keep their 8 bits down to 2^-32 of it, smaller ones are off
 *    by at most 2^-40 of it;
 *  - the softmax weights before their product with v: each is off by at most
 *    2^-11 of itself or 2^-33 of the row's largest. lse sums them unrounded.
 * Scores (scale * q . k) are to be below 2^26 in magnitude, which fp32 holds to a
 * few units: beyond 2^27 a row may come out as NaN, zeros or -inf. */
typedef struct {
  const void* q;           /* device: [rows][heads][head_dim] by strides */
  void* out;               /* device: contiguous, 16-byte aligned */
  float* lse;              /* device: [rows][heads], or NULL */
  const int32_t* table;    /* device: page indices */
  const int32_t* kv_len;   /* device: [batch], each 0 .. max_kv_len */
  const int32_t* q_start;  /* device: [batch + 1] from 0 to rows, or NULL */
  int64_t q_token_stride;  /* elements */
  int64_t q_head_stride;
  int64_t table_stride;    /* entries a sequence, table_stride * page_size >= max_kv_len */
  int32_t dtype;           /* F16 or BF16 */
  int32_t layer;
  int32_t heads;           /* a multiple of kv_heads */
  int32_t batch;
  int32_t rows;            /* all sequences' rows */
  int32_t max_q_len;       /* no sequence has more rows */
  int32_t max_kv_len;      /* no sequence has more tokens; longer ones are cut there */
  int32_t window;          /* 0: none */
  float scale;             /* finite and > 0 */
  int32_t reserved;        /* 0 */
} qpn_kv4_attention_args;

/* Workspace of a call (its pointers may be NULL; 0: none is needed). Its
 * contents need no preparation and carry nothing to the next call. */
size_t qpn_kv4_attention_workspace_bytes(const qpn_kv4_cache* cache, const qpn_kv4_attention_args* args);

qpn_status qpn_kv4_attention(const qpn_kv4_cache* cache, const qpn_kv4_attention_args* args, void* workspace_dev,
                             size_t workspace_bytes, void* stream);

/* Verification of drafted tokens by speculative sampling. Sequence b has
 * num_draft[b] <= drafts drafted tokens (NULL: drafts each). With p the
 * target's and q the draft's probabilities at a place, draft d is accepted
 * where u_accept * q(d) < p(d) (draft NULL: the drafts were chosen without
 * chance, q(d) = 1). The first that is not accepted is replaced by the token
 * that u_sample picks from max(p - q, 0) (draft NULL: from p without d); after
 * a block that is accepted whole it picks from the p of the next row. u picks
 * the smallest token whose running sum exceeds u times the sum.
 *   tokens[b]   = the accepted drafts, the picked token, then -1  (drafts + 1)
 *   accepted[b] = the number of accepted drafts
 *   logprobs[b] = log p of each given token, then 0               (may be NULL)
 * Logits: p = softmax(logits / temperature[b]) (NULL: 1); at a temperature of
 * 0 (or below, or NaN) sequence b is greedy: a draft is accepted where it is
 * the row's largest logit, the picked token is the largest logit (ties to the
 * lowest index), draft and numbers are not used, and logprobs are those at
 * temperature 1. NaN logits count as -inf, NaN and negative probabilities as
 * 0. A draft token outside 0 .. vocab - 1 is not accepted. If nothing is left
 * over, the token is picked from p; if p is all zero, it is -1.
 * Probabilities (probabilities = 1): fp32 p and q are taken as they are.
 * From logits, the row sums behind the accept tests and logprobs add 32-bit
 * exponentials in 64 bits: p and q are good to about 2^-21 of themselves, and a
 * test closer to its border than that may go either way. The token is picked
 * with 64-bit exponentials and sums. */
typedef struct {
  const void* target;           /* device: [batch][drafts + 1][vocab] by strides */
  const void* draft;            /* device: [batch][drafts][vocab] by strides, same dtype, or NULL */
  const int32_t* draft_tokens;  /* device: [batch][drafts] */
  const int32_t* num_draft;     /* device: [batch], or NULL */
  const float* temperature;     /* device: [batch], or NULL */
  const float* u_accept;        /* device: [batch][drafts], in [0, 1) */
  const float* u_sample;        /* device: [batch], in [0, 1) */
  int32_t* tokens;              /* device: [batch][drafts + 1] */
  int32_t* accepted;            /* device: [batch] */
  float* logprobs;              /* device: [batch][drafts + 1], or NULL */
  int64_t target_batch_stride;  /* elements */
  int64_t target_row_stride;
  int64_t draft_batch_stride;
  int64_t draft_row_stride;
  int32_t dtype;                /* F16, BF16 or F32 */
  int32_t probabilities;        /* 0: logits, 1: probabilities (F32) */
  int32_t batch;
  int32_t drafts;               /* 0 .. 64 */
  int32_t vocab;                /* 1 .. 2^24 */
  int32_t reserved;             /* 0 */
} qpn_verify_args;

/* Workspace of a call with these sizes (0 for sizes that are refused: more
 * rows and chunks of 4096 tokens than a launch has workgroups for). Its
 * contents need no preparation and carry nothing to the next call. */
size_t qpn_verify_workspace_bytes(int32_t batch, int32_t drafts, int32_t vocab);

qpn_status qpn_verify(const qpn_verify_args* args, void* workspace_dev, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QPN_DECODE_H */
