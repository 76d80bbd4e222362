/*
 * dsv4_loop.h - C ABI of the operators of libdsv4 that surround the layers of a decode step with drafted tokens:
 * what the layers' calls take as positions, block tables, slots and rotary tables, and which drafted tokens stand.
 *
 *   dsv4_draft_verify   which drafted tokens of every sequence stand against the target's probabilities, and
 *                       the token that follows them, from given random numbers
 *   dsv4_batch_plan     pages given back and taken, block tables, slots, positions, q_start and kv_len of the
 *                       next step, from every request's rows and new tokens
 *   dsv4_rope           rows of queries and keys turned by their tokens' positions (and back)
 *   dsv4_rope_table     the cos_sin table that the layers' calls take
 *   dsv4_rope_freqs     (host) the frequencies of both, scaled for long contexts
 *
 * One step of a loop over fixed buffers, with no host synchronisation, so that a CUDA graph can hold it:
 *   dsv4_batch_plan (ctx += n_out of the last step) -> the layers (dsv4_gqa_append / dsv4_gqa_attention, dsv4_kv_insert
 *   ...) over its positions, slots and tables -> logits -> dsv4_draft_verify (n_out, out_tokens).
 *
 * The conventions of dsv4.h and, for ragged batches, of dsv4_gqa.h hold: device pointers, caller-owned memory,
 * asynchronous on `stream`, capturable, struct_size, host validation before any launch, device range checks that skip
 * and raise bit 0 of dsv4_read_device_flags(); every call waits for the kernel before it on the stream.  No call
 * needs a workspace.  Results do not depend on the order in which the GPU runs the call's blocks.
 */
#ifndef DSV4_LOOP_H
#define DSV4_LOOP_H

#include "dsv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * dsv4_rope_freqs (a pure host function; `freqs` is HOST memory): the frequency of every pair i < rope_dim / 2,
 * in radians a position f_i = theta^(-2 i / rope_dim), scaled by
 *   DSV4_ROPE_LINEAR  f_i / factor
 *   DSV4_ROPE_BASE    theta * factor^(rope_dim / (rope_dim - 2)) in the place of theta
 *   DSV4_ROPE_YARN    f_i (r_i / factor + 1 - r_i),  r_i = clamp((i - low) / max(high - low, 0.001), 0, 1),
 *                     low = max(floor(c(beta_fast)), 0), high = min(ceil(c(beta_slow)), rope_dim - 1),
 *                     c(b) = rope_dim ln(original_len / (2 pi b)) / (2 ln theta)
 *   DSV4_ROPE_BANDS   f_i ((1 - m_i) / factor + m_i),
 *                     m_i = clamp((original_len f_i / (2 pi) - low_turns) / (high_turns - low_turns), 0, 1)
 * freqs[i] = f_i / (2 pi) as a binary fraction of 64 bits, cut: position * freqs[i] mod 2^64 is the angle, reduced to one
 * turn without a rounding, so an angle is off by position * (k theta^(-2 i / rope_dim) 2^-53 + 2 pi 2^-64) at most, whatever
 * the position, with k = 2 ln(theta) + 8 (theta as it is used; BANDS: times 1 + high_turns / (high_turns - low_turns)): the
 * roundings of f_i in fp64, and a step of the fraction, which is the larger part for small frequencies.
 * ------------------------------------------------------------------------------------------- */
#define DSV4_ROPE_NONE 0
#define DSV4_ROPE_LINEAR 1
#define DSV4_ROPE_BASE 2
#define DSV4_ROPE_YARN 3
#define DSV4_ROPE_BANDS 4

typedef struct dsv4_rope_freqs_params {
  uint32_t struct_size;
  int32_t rope_dim;            /* even, 2 .. 1024 (BASE: from 4 on) */
  int32_t scaling;             /* DSV4_ROPE_* */
  double theta;                /* over 1, finite */
  double factor;               /* 1 or more, finite */
  double original_len;         /* rows trained on, over 0 (YARN, BANDS) */
  double beta_fast, beta_slow; /* over 0 (YARN; usually 32 and 1) */
  double low_turns, high_turns; /* high over low (BANDS; usually 1 and 4) */
} dsv4_rope_freqs_params;

int dsv4_rope_freqs(const dsv4_rope_freqs_params* p, uint64_t* freqs);

/* ---------------------------------------------------------------------------------------------
 * dsv4_rope: for every token t at position p = positions[t], head h and pair i of the rope_dim dims from
 * rope_first on, with the angle w = p f_i:
 *   a' = scale (a cos w - b sin w),  b' = scale (b cos w + a sin w)      (inverse: -w for w)
 * pair i being dims (2i, 2i + 1) of the range, or (i, i + rope_dim / 2) with rope_halves; the other dims are
 * copied.  fp32 arithmetic, rounded once to the type (bf16: nearest even).  The inverse call with the same scale is
 * the gradient of the forward one: it turns the gradient of y into that of x.
 * A token with a negative position is skipped: its rows of y stay as they are.
 * A second tensor (the keys beside the queries) is turned in the same launch when x2 is given.
 * y is x itself (same strides: in place) or lies apart from x, x2 and y2, and y2 likewise; rows of one buffer may
 * alternate.  Calls where they meet are refused where extents, or equal strides, tell.  Rows of y, and of y2, lie apart from
 * one another (else refused).  Strides of x may be 0 (a row for several heads or tokens).
 * ------------------------------------------------------------------------------------------- */
typedef struct dsv4_rope_params {
  uint32_t struct_size;
  const void* x;               /* [T, heads, head_dim] in dtype, 16-byte aligned */
  void* y;
  int64_t x_token_stride, x_head_stride, y_token_stride, y_head_stride; /* elements, multiples of 8; y's head_dim or more */
  const void* x2;              /* [T, heads2, head_dim] or NULL */
  void* y2;
  int64_t x2_token_stride, x2_head_stride, y2_token_stride, y2_head_stride;
  int32_t heads, heads2;       /* 1 .. 1024 (heads2: read with x2 only) */
  int32_t dtype;               /* DSV4_F32 or DSV4_BF16 */
  int32_t T, head_dim;         /* T <= 2^30; head_dim a multiple of 8, up to 1024 */
  const int32_t* positions;    /* [T] */
  const uint64_t* freqs;       /* [rope_dim / 2] of dsv4_rope_freqs, in device memory, 16-byte aligned */
  int32_t rope_first, rope_dim; /* rope_first a multiple of 8, rope_dim of 16, within head_dim */
  int32_t rope_halves, inverse; /* 0 or 1 */
  float scale;                 /* finite (YaRN: 0.1 ln(factor) + 1, or 1) */
} dsv4_rope_params;

int dsv4_rope(const dsv4_rope_params* p, dsv4_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * dsv4_rope_table: row r of table = scale cos(w_i) for every pair i, then scale sin(w_i), w_i = (first_position + r)
 * f_i: the cos_sin operand of dsv4_kv_insert, dsv4_qnorm_rope_kv_insert, dsv4_compress_update and dsv4_gqa_append.
 * ------------------------------------------------------------------------------------------- */
typedef struct dsv4_rope_table_params {
  uint32_t struct_size;
  float* table;                /* [rows, rope_dim], 16-byte aligned */
  int32_t rows;                /* >= 0; first_position + rows <= 2^31 - 1 */
  int32_t rope_dim;            /* a multiple of 8, up to 1024 */
  int32_t first_position;      /* >= 0 */
  float scale;
  const uint64_t* freqs;       /* [rope_dim / 2], device memory, 16-byte aligned */
} dsv4_rope_table_params;

int dsv4_rope_table(const dsv4_rope_table_params* p, dsv4_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * dsv4_batch_plan: the next step of B requests, request b keeping c_b = ctx[b] + ctx_add[b] rows and bringing
 * n_new[b] tokens, over 1 .. 4 paged caches.  A cache holds e = floor(rows / ratio) entries of a request, in table
 * entries first_b .. held_b - 1 (first_b = 0 without a window); free_pages[0 .. free_count - 1] is its stack of pages
 * that nobody holds.
 *  1. Given back.  What a request does not need any more is pushed onto the stack, in the order of the
 *     requests (of one request: front pages, then back pages, in order): the table entries from
 *     max(ceil(e_b / page_size), first_b) on, e_b = floor((c_b + n_b) / ratio), and, with a window, those before
 *     floor(max(0, c_b - window + 1) / page_size), whose rows no token of this step or a later one sees.  A request
 *     with c_b + n_b = 0 (one that has ended) gives back all it holds, and holds nothing from entry 0 on.
 *  2. Taken.  A request that needs more pages than it holds pops them, in the order of the requests.  It gets its
 *     tokens only if, in every cache that it takes pages of, the pages taken by all requests up to and
 *     including it fit what the stack holds then, and if the tokens of all up to it fit T; requests that are left out
 *     count like the others.  One that is left out (or has n_b = 0) has no token in this step, and
 *     takes no page; it can be brought again in the next.
 *  3. Written.  With n_b the tokens that run: q_start[b + 1] = sum n, kv_len[b] = c_b + n_b, ctx_out[b] = c_b; for
 *     token i of request b at flat index t = q_start[b] + i: positions[t] = c_b + i, token_seq[t] = b, and for each
 *     cache slots[t] = page * page_size + row of entry j = floor(position / ratio), which the token completes
 *     ((position + 1) % ratio = 0), else -1.  From q_start[B] to T: -1 in all of them (dsv4_kv_insert skips
 *     such slots, dsv4_rope such positions).  Table entries that are given back stay as they were.
 * Every *_out may be its input (in place) or lie apart; apart from its input, the same call can be made again with
 * the same result.  What the call writes of a cache (table, held_out, first_out, stack, free_count_out, slots) belongs to
 * no other: two that name the same, or one that reads what is written of another, are refused.
 * A request with ctx, ctx_add or n_new that gives c_b < 0, n_b < 0 or c_b + n_b over 2^30, more pages than
 * max_pages_per_seq, first and held not in 0 <= first <= held <= max_pages_per_seq, or a window that reaches rows before
 * first is flagged (bit 0) and left alone: no token, kv_len 0, ctx_out = ctx, nothing given back or taken.  A
 * free_count outside [0, num_pages] is taken as the nearest bound and flagged; pages pushed beyond num_pages are lost
 * and flagged; a page outside [0, num_pages) that is popped goes into the table and is flagged (its slots are -1).
 * ------------------------------------------------------------------------------------------- */
#define DSV4_PLAN_MAX_CACHES 4
#define DSV4_PLAN_MAX_REQUESTS 4096
#define DSV4_PLAN_MAX_TOKENS (1 << 19)

typedef struct dsv4_plan_cache {
  int32_t page_size, ratio;    /* 1 .. 65536 rows, 1 .. 65536 */
  int32_t window;              /* 0: none; > 0: only the last window rows before a token are seen (ratio 1 only) */
  int32_t max_pages_per_seq;   /* 1 .. 2^19 */
  int64_t num_pages;           /* 0 .. 2^31 - 1: page ids and the stack's capacity */
  int32_t* block_table;        /* [B, max_pages_per_seq] */
  const int32_t* held;         /* [B] end of each request's table entries */
  int32_t* held_out;
  const int32_t* first;        /* [B] begin of each request's table entries (window only; else NULL) */
  int32_t* first_out;
  int32_t* free_pages;         /* [num_pages] */
  const int32_t* free_count;   /* [1] */
  int32_t* free_count_out;
  int64_t* slots;              /* [T], 16-byte aligned, or NULL */
} dsv4_plan_cache;

typedef struct dsv4_batch_plan_params {
  uint32_t struct_size;
  int32_t B;                   /* 0 .. DSV4_PLAN_MAX_REQUESTS */
  int32_t T;                   /* tokens that the step has room for, 0 .. DSV4_PLAN_MAX_TOKENS */
  int32_t num_caches;          /* 1 .. DSV4_PLAN_MAX_CACHES */
  const int32_t* ctx;          /* [B] rows that each request held before */
  const int32_t* ctx_add;      /* [B] added to ctx (the n_out of dsv4_draft_verify), or NULL */
  const int32_t* n_new;        /* [B] */
  int32_t* ctx_out;            /* [B] or NULL */
  int32_t* q_start;            /* [B + 1] */
  int32_t* kv_len;             /* [B] */
  int32_t* positions;          /* [T], 16-byte aligned, or NULL */
  int32_t* token_seq;          /* the same */
  dsv4_plan_cache caches[DSV4_PLAN_MAX_CACHES];
} dsv4_batch_plan_params;

int dsv4_batch_plan(const dsv4_batch_plan_params* p, dsv4_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * dsv4_draft_verify: sequence b brought n_b = q_start[b+1] - q_start[b] tokens to the target: its last token, then
 * n_b - 1 drafted ones.  Target row t = q_start[b] + i says how token t + 1 is distributed:
 *   logits         p = softmax(row / temperature[b])
 *   target_probs   p = row
 * and draft row of token t + 1 (draft_row[t + 1]; when draft_row is NULL, t less the number of sequences before b that
 * brought tokens: the drafted tokens' rows in order, sequences without tokens having none) the distribution q that it was
 * drawn from, likewise; without a draft, q is 1 at the token (drafts that were not drawn).  For i = 0, 1, ... the drafted token x = tokens[t + 1] stands if
 *   u[t + 1] q(x) < p(x)
 * up to the first that does not; that one is replaced by argmax_x max(p(x) - q(x), 0) / noise[b][x] (without a
 * draft: of p(x) / noise[b][x] over the others), and when all stand, argmax_x p(x) / noise[b][x] of the last row
 * follows: with u uniform on [0, 1) and noise of independent Exp(1) variates, the tokens are distributed as if
 * drawn from p.  Where p <= q everywhere, the race runs over p.  Equal numbers: the lowest index.
 * Greedy sequences (temperature not over 0, or a call without u and noise): x stands if it is the row's first
 * maximum, which else takes its place, or follows; u, noise and draft are not read.
 *   n_out[b] = drafted tokens that stand + 1;  out_tokens[b] = these tokens, then -1;
 *   logp[b] = log p of each (greedy: temperature 1), then 0.
 * A NaN or -inf logit has probability 0, as has a NaN or negative probability, and one below 2^-126 may count as
 * 0; +inf counts as the type's largest value.  Temperatures count as within [1e-30, 1e30].  A row that leaves no
 * token its probability lets no drafted token stand, and -1 takes its place, which n_out does not count.  A
 * drafted token outside [0, vocab), or with a draft row outside [0, draft_rows), falls and is flagged (bit 0; then the race
 * runs over p in the latter case).  n_b = 0 gives n_out = 0.  A sequence with q_start not in
 * 0 <= q_start[b] <= q_start[b+1] <= T or n_b > max_q_len is skipped (its outputs stay) and flagged.
 * Rows after the first drafted token that falls do not matter, nor do the draft rows of greedy sequences.
 * ------------------------------------------------------------------------------------------- */
typedef struct dsv4_draft_verify_params {
  uint32_t struct_size;
  const void* target;          /* [T, vocab] in target_dtype, rows target_stride elements apart */
  int64_t target_stride;       /* >= vocab */
  int32_t target_dtype;        /* DSV4_F32 or DSV4_BF16 */
  int32_t target_probs;        /* 0: logits, 1: probabilities */
  const void* draft;           /* [draft_rows, vocab] in draft_dtype, or NULL */
  int64_t draft_stride, draft_rows;
  int32_t draft_dtype, draft_probs;
  const int32_t* draft_row;    /* [T] or NULL */
  const int32_t* tokens;       /* [T] */
  const int32_t* q_start;      /* [B + 1] */
  int32_t T, B, vocab;         /* T <= 2^30; B <= 65535; vocab 1 .. 2^24 */
  int32_t max_q_len;           /* host bound on n_b, >= 1; columns of out_tokens and logp */
  const float* temperature;    /* [B] or NULL (1 for every sequence) */
  const float* u;              /* [T], and noise [B, vocab] with rows noise_stride apart, positive; or both NULL */
  const float* noise;
  int64_t noise_stride;
  int32_t* out_tokens;         /* [B, max_q_len] */
  int32_t* n_out;              /* [B] */
  float* logp;                 /* [B, max_q_len] or NULL */
} dsv4_draft_verify_params;

int dsv4_draft_verify(const dsv4_draft_verify_params* p, dsv4_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSV4_LOOP_H */
