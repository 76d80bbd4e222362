/*
 * dsv4_gqa.h - C ABI of the grouped-query operators of libdsv4: layers that keep keys and values per
 * head (draft models for multi-token decoding, plain attention layers beside the compressed ones).
 *
 *   dsv4_gqa_append     rotates the new tokens' keys (and queries) and stores keys and values into
 *                       paged caches, bf16 or e4m3 with one power-of-two scale per page and head
 *   dsv4_gqa_attention  softmax attention of one or many new tokens a sequence over those caches, with
 *                       causal / prefix / document / window masks, capped scores, distance bias, sink
 *
 * The conventions of dsv4.h hold (device pointers, caller-owned memory, asynchronous on `stream`,
 * graph-capturable, struct_size, host validation before any launch, device range checks that skip the
 * access and raise dsv4_read_device_flags() bits, bounded waits: where one may last through a block of
 * queries, 50 us longer for each 128 rows that the call's bounds let a CTA go through).  Both calls wait for the
 * kernel before them on the stream.  Further:
 *  - Batches are ragged: q_start[B + 1] holds the first flat token of each sequence; sequence b has
 *    n_b = q_start[b+1] - q_start[b] new tokens, and kv_len[b] rows INCLUDING them, so its token i is
 *    at position kv_len[b] - n_b + i.  n_b = 0 and kv_len[b] = 0 are allowed.  Tokens from q_start[B] on
 *    (the padding of a fixed-size batch) are not written, and what they hold does not matter.
 *  - A sequence with q_start not in 0 <= q_start[b] <= q_start[b+1] <= T, n_b > max_q_len,
 *    kv_len[b] < n_b or kv_len[b] over 2^30 or the call's bound is skipped (its outputs stay as they were) and
 *    flagged (bit 0).
 *  - Caches are [num_pages, kv_heads, page_size, head_dim] in any order of the first three (element
 *    strides are given; head_dim is contiguous).  Row j of sequence b lies in page
 *    block_table[b][j / page_size], row j % page_size.  A table entry outside [0, num_pages) is flagged
 *    (bit 0); its rows are not stored, or take no part.
 *  - DSV4_E4M3_PAGE caches hold e4m3fn codes; k_exp / v_exp [num_pages, kv_heads] hold one UE8M0 byte
 *    per page and head, value = code * 2^(byte - 127).
 */
#ifndef DSV4_GQA_H
#define DSV4_GQA_H

#include "dsv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache dtype beside DSV4_BF16: e4m3fn codes with one UE8M0 exponent per page and head. */
#define DSV4_E4M3_PAGE 5

/* ---------------------------------------------------------------------------------------------
 * dsv4_gqa_append: for every new token t of sequence b at position p,
 *   k row = rotate(k_new[t], p), v row = v_new[t], stored at row p of the sequence for every kv head;
 *   q_out[t] = rotate(q[t], p) when q is given (bf16, round to nearest even).
 * rotate turns the pairs of the rope_dim dims from rope_first on by cos_sin[p] (cos in the first half
 * of the row, sin in the second), in fp32 with each product and sum rounded:
 *   a' = a cos - b sin,  b' = b cos + a sin,
 * pair i being dims (2i, 2i + 1) of the range (GPT-J), or (i, i + rope_dim / 2) with rope_halves.
 * bf16 caches: round to nearest even.  E4M3_PAGE: let m be the largest |x| the call stores into a
 * (page, head), in fp32, and e the smallest integer in [-127, 127] with 448 * 2^e >= m (-127 for
 * m = 0).  When the call stores row 0 of the page, its exponent becomes e (what the page held before
 * is forgotten); else it becomes the larger of e and the old one, and when it grew the rows before the
 * call's first one are re-encoded: code' = RNE(code * 2^(old - new)), exact unless the result is
 * subnormal.  Then code = RNE(x * 2^-exponent).  NaN stays NaN; +-Inf saturates at code +-448 (and
 * sets the exponent to 120).
 * A call must not store into one page twice, for two sequences or two table entries of one (its contents
 * would be unspecified).
 * ------------------------------------------------------------------------------------------- */
typedef struct dsv4_gqa_append_params {
  uint32_t struct_size;
  const void* k_new;           /* [T, kv_heads, head_dim] bf16, 16-byte aligned */
  const void* v_new;           /* the same */
  int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;  /* elements, multiples of 8 */
  const void* q;               /* [T, q_heads, head_dim] bf16, 16-byte aligned, or NULL: no queries */
  void* q_out;                 /* bf16, 16-byte aligned, strides > 0; q itself (same strides: in place) or apart */
  int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
  void* k_cache;               /* 16-byte aligned, in cache_dtype */
  void* v_cache;
  int64_t k_page_stride, k_cache_head_stride, k_row_stride;  /* elements; multiples of 16 bytes */
  int64_t v_page_stride, v_cache_head_stride, v_row_stride;
  uint8_t* k_exp;              /* [num_pages, kv_heads] (E4M3_PAGE only) */
  uint8_t* v_exp;
  int32_t cache_dtype;         /* DSV4_BF16 or DSV4_E4M3_PAGE */
  int32_t T, B, q_heads, kv_heads, head_dim;  /* T <= 2^30; B <= 65535; heads 1 .. 1024; head_dim 64 or 128 */
  int32_t page_size;           /* 16, 32, 64, 128 or 256 */
  int64_t num_pages;           /* < 2^31 */
  const int32_t* block_table;  /* [B, max_pages_per_seq] */
  int32_t max_pages_per_seq;
  const int32_t* q_start;      /* [B + 1] */
  const int32_t* kv_len;       /* [B] */
  int32_t max_q_len;           /* host bound on n_b, >= 1 */
  const float* cos_sin;        /* [max_pos, rope_dim], 16-byte aligned, or NULL: nothing is rotated */
  int32_t max_pos;             /* bound on kv_len when cos_sin is given */
  int32_t rope_first, rope_dim;  /* rope_first a multiple of 8, rope_dim of 16, within head_dim */
  int32_t rope_halves;
} dsv4_gqa_append_params;

int dsv4_gqa_append(const dsv4_gqa_append_params* p, dsv4_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * dsv4_gqa_attention: for token t of sequence b at position p and query head h (kv head
 * h / (q_heads / kv_heads)), over the visible rows j:
 *   z_j = softmax_scale * (q[t][h] . k_j);  if softcap > 0: z_j = softcap * tanh(z_j / softcap);
 *   if slopes: z_j -= slopes[h] * |p - j|
 *   out[t][h] = sum_j e^(z_j - m) v_j / (sum_j e^(z_j - m) + e^(sink[h] - m))
 *   lse[t][h] = m + log(denominator),  m = max(max_j z_j, sink[h])
 * Row j is visible when  j < kv_len[b],  causal == 0 or j <= p or j < prefix_len[b],
 * window == 0 or j > p - window,  and j >= kv_start[t].  A token that sees no row gets out = 0 and
 * lse = sink[h] (-inf without a sink).
 * What rows from kv_len on, rows of other pages and rows before the first one that any of the sequence's
 * tokens sees hold never matters, NaN included; nor do the table entries of pages with no other rows.  The
 * rows from that one on must hold finite values, as bf16 (e4m3: code times scale): a NaN or Inf among them
 * may also reach tokens that do not see it.
 * Sums over the rows are fp32 and divided at the end: |v| times the rows seen has to stay below 2^100, and
 * weights below 2^-100 of a token's total may count as zeros (with softcap: below 2^-60, and values below
 * 2^-40 may lose bits).
 * Calls of more than 8192 blocks of 256 rows (token, head of the group; B ceil(max_q_len group / 256)) add up
 * a token's rows in one run, whose rounding takes about rows * 2^-29 of an output.
 * Weights are rounded before their product with V whatever out_dtype is: to bf16 (2^-8 of themselves), or, over
 * e4m3 caches with at most 32 rows (token, head of the group) a sequence, to two e4m3 terms (2^-8 of
 * themselves, or 2^-19 of the largest among 32 neighbouring ones).  Their sum is that of the unrounded ones.
 * max_q_len and max_kv_len choose the kernels, the grid and the workspace for the whole call.  Over e4m3
 * caches, a step that mixes prompt chunks with single tokens is better made as two calls, one for each kind
 * (512 tokens beside 31 single ones over up to 8k rows: 151 us for 337, and 61 MB of workspace for 1.1 GB).
 * The workspace of an e4m3 call with more than 32 rows (token, head of the group) a sequence has room for
 * bf16 copies of the batch's rows: 4 B kv_heads max_kv_len head_dim bytes, lengths rounded up to 128.
 * ------------------------------------------------------------------------------------------- */
typedef struct dsv4_gqa_attention_params {
  uint32_t struct_size;
  const void* q;               /* [T, q_heads, head_dim] bf16, 16-byte aligned */
  int64_t q_token_stride, q_head_stride;       /* elements, multiples of 8 */
  const void* k_cache;         /* as in dsv4_gqa_append_params */
  const void* v_cache;
  int64_t k_page_stride, k_cache_head_stride, k_row_stride;
  int64_t v_page_stride, v_cache_head_stride, v_row_stride;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  int32_t cache_dtype;
  int32_t T, B, q_heads, kv_heads, head_dim, page_size;  /* q_heads a multiple of kv_heads */
  int64_t num_pages;
  const int32_t* block_table;  /* [B, max_pages_per_seq] */
  int32_t max_pages_per_seq;
  const int32_t* q_start;      /* [B + 1] */
  const int32_t* kv_len;       /* [B] */
  int32_t max_q_len;           /* host bound on n_b, >= 1 (choose the kernels and the grid) */
  int32_t max_kv_len;          /* host bound on kv_len[b], 0 .. 2^30 */
  float softmax_scale;         /* 4 softmax_scale finite */
  int32_t causal;              /* 1: rows after the token are hidden (but for the prefix), 0: all visible */
  const int32_t* prefix_len;   /* [B] rows visible to every token of the sequence, or NULL */
  const int32_t* kv_start;     /* [T] first visible row of each token, or NULL */
  int32_t window;              /* 0: none */
  float softcap;               /* 0: none; at most 1024 (logits are off by up to softcap * 2^-20), and
                                  4 / softcap and 4 softmax_scale / softcap finite */
  const float* slopes;         /* [q_heads] or NULL */
  const float* sink;           /* [q_heads], finite or -inf, or NULL (= -inf) */
  void* out;                   /* [T, q_heads, head_dim] contiguous, out_dtype BF16 or F32, 16-byte aligned */
  int32_t out_dtype;
  float* lse;                  /* [T, q_heads] or NULL */
  void* workspace;             /* dsv4_gqa_attention_workspace_bytes() bytes, 256-byte aligned; what it
                                  holds before and after a call is of no account, but calls that may
                                  overlap on the GPU need workspaces of their own */
  size_t workspace_bytes;
} dsv4_gqa_attention_params;

size_t dsv4_gqa_attention_workspace_bytes(const dsv4_gqa_attention_params* p);
int dsv4_gqa_attention(const dsv4_gqa_attention_params* p, dsv4_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSV4_GQA_H */
