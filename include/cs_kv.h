/*
 * cs_kv.h -- C ABI of the paged key/value cache operators for GB300 (sm_103a),
 * in the same library as cs_chain.h.
 *
 * What it computes.  The attention chain of cs_chain.h runs whole prompts and
 * keeps no keys.  A serving program also keeps every layer's keys and values in
 * a cache of fixed-size pages, and each step (a) rotates the new tokens' queries
 * and keys by their positions and appends keys and values to the cache
 * (cs_kv_append), (b) attends from the new queries to the cached keys
 * (cs_kv_attention), or (c) does so for sequences that share one long prefix,
 * whose keys are read once for the whole batch (cs_kv_attention_shared).
 * cs_attn_cached_forward puts (a) and (b) between the QKV and output-projection
 * stages of an attention chain's plan.
 *
 * A batch.  Sequence b of a batch brings n = cu_q[b+1] - cu_q[b] new tokens,
 * rows cu_q[b] .. cu_q[b+1]-1 of every token-indexed tensor, and has
 * m = kv_lens[b] keys in the cache, the new tokens' keys being the last n of
 * them.  New token i has the position p = m - n + i; key j of the sequence lives
 * in page page_table[b][j / page_size], slot j % page_size.  n may be 0 (an idle
 * slot of the batch).  Rows at and behind cu_q[seqs] are padding: nothing
 * is written there.
 *
 * Conventions: those of cs_chain.h (cs_status everywhere, cs_last_error_string,
 * stream as void*, calls only enqueue).  The lengths, page tables and positions
 * are read on the device, so a captured call may be replayed with other ones as
 * long as they fit what the call was made with.  Ones that do not fit never
 * cause an access out of bounds, and cs_kv_status reports the device error.  A
 * sequence whose lengths do not fit is left out (its rows stay as they were),
 * and so is an appended token whose page or position does not.  What attention gives a
 * sequence with such a page means nothing, nor, where the prefix has one or the
 * lengths under a prefix do not fit, what it gives the batch.  A plan is not thread-safe and runs
 * on one stream at a time (its workspace is per plan): two captured graphs that
 * may run at the same time need a plan each.
 */
#ifndef CS_KV_H
#define CS_KV_H

#include "cs_chain.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CS_KV_ABI_VERSION 1

typedef struct cs_kv_s* cs_kv_t;

/* Layout of the K and V caches (each one contiguous tensor).
 *  TOKEN: [num_pages, page_size, kv_heads, head_dim]
 *  HEAD : [num_pages, kv_heads, page_size, head_dim]                           */
typedef enum cs_kv_layout { CS_KV_TOKEN = 0, CS_KV_HEAD = 1 } cs_kv_layout;

/* Which two of a head's first rotary_dim dimensions are rotated together:
 *  HALF    : (i, i + rotary_dim / 2)      ADJACENT: (2 i, 2 i + 1)             */
typedef enum cs_kv_pairing { CS_KV_HALF = 0, CS_KV_ADJACENT = 1 } cs_kv_pairing;

typedef struct cs_kv_desc {
  int dtype;           /* cs_dtype of Q, K, V, the cache and O */
  int heads;           /* query heads */
  int kv_heads;        /* key/value heads: query head h reads key head h / (heads / kv_heads);
                          divides heads, heads / kv_heads <= 128 */
  int head_dim;        /* 64 or 128 */
  int page_size;       /* positions per page: 16, 32, 64 or 128 */
  int num_pages;       /* pages of the pool (each of the K and the V cache) */
  int cache_layout;    /* cs_kv_layout */
  int max_tokens;      /* most rows of the token-indexed tensors of a call */
  int max_seqs;        /* most sequences of a call, at most 8192 */
  int rotary_dim;      /* dimensions of each head that cs_kv_append rotates: 0 (none) or a
                          multiple of 16 up to head_dim */
  int rotary_pairing;  /* cs_kv_pairing */
  int window;          /* 0: token p sees keys 0..p.  w > 0: keys p-w+1..p and the first `sinks` */
  int sinks;           /* first keys of every sequence that stay visible under a window */
  float scale;         /* factor of the scores; 0 = 1 / sqrt(head_dim) */
  int shared;          /* 1: the plan also runs cs_kv_attention_shared (its workspace holds
                          max_tokens x heads x (head_dim + 1) floats more); needs window 0 */
  int num_sms;         /* SMs used; 0 = every SM of the device */
} cs_kv_desc;

/* Fill *desc with defaults (f16, 128-wide heads, pages of 16, TOKEN, HALF, the rest 0). */
cs_status cs_kv_desc_init(cs_kv_desc* desc);

/* Make a plan on the current device: validates, allocates the workspace. */
cs_status cs_kv_plan(const cs_kv_desc* desc, cs_kv_t* out);

/* Free everything the plan owns.  NULL-safe.  Synchronises the device first. */
cs_status cs_kv_destroy(cs_kv_t plan);

/* One batch, shared by the calls of a step.  All pointers are device memory. */
typedef struct cs_kv_batch {
  int tokens;                 /* rows of the token-indexed tensors, padding included; <= max_tokens */
  int seqs;                   /* <= max_seqs */
  int max_q;                  /* no sequence brings more new tokens than this (it chooses the kernel) */
  int table_cols;             /* columns of the page table; table_cols * page_size <= 2^22.  The width also
                                 chooses how prompts are divided: with a table no wider than the longest
                                 sequence needs, short ones take about two thirds of the time */
  const int32_t* cu_q;        /* [seqs + 1], not decreasing, within 0 .. tokens */
  const int32_t* kv_lens;     /* [seqs], within n .. table_cols * page_size (below n: the tokens before
                                 position 0 see no key) */
  const int32_t* page_table;  /* [seqs, table_cols]; entries behind a sequence's last page, and those of
                                 pages that no new token sees, are not used */
} cs_kv_batch;

typedef struct cs_kv_append_args {
  const void* qkv;            /* rows of [Q: heads | K: kv_heads | V: kv_heads] x head_dim */
  long long qkv_stride;       /* elements between rows; 0 = (heads + 2 kv_heads) * head_dim */
  void* q_out;                /* rows of heads * head_dim: the rotated queries; may be the Q part of
                                 qkv itself (rotation in place), else must not overlap it */
  long long q_stride;         /* elements between rows of q_out; 0 = heads * head_dim */
  void* k_cache;              /* the caches overlap neither each other nor qkv nor q_out */
  void* v_cache;
  const float* rope;          /* [rope_rows, rotary_dim]: row p = rotary_dim / 2 cosines, then as many
                                 sines, of position p's angles.  Unused with rotary_dim 0 */
  int rope_rows;
  const int32_t* positions;   /* [tokens]: the position whose angles rotate each token; NULL: its place
                                 p in its sequence */
} cs_kv_append_args;

/* Rotate Q and K of the batch's new tokens (in 32 bits, rounded once to the
 * dtype), write Q to q_out and K, V to their places in the cache.  Pairs
 * (a, b) become (a cos - b sin, b cos + a sin).  The pages that new tokens fall in
 * must belong to one sequence each: two tokens sent to one slot leave either's
 * values there.  A new token before position 0 (kv_lens[b] < n) is left out. */
cs_status cs_kv_append(cs_kv_t plan, const cs_kv_batch* batch, const cs_kv_append_args* args, void* stream);

typedef struct cs_kv_attn_args {
  const void* q;              /* rows of heads * head_dim */
  long long q_stride;         /* elements between rows; 0 = heads * head_dim */
  const void* k_cache;
  const void* v_cache;
  void* out;                  /* rows of heads * head_dim; must not overlap q or a cache */
  long long out_stride;       /* elements between rows; 0 = heads * head_dim */
  float* lse;                 /* NULL, or [tokens, heads]: log of the sum of exp(score); overlaps nothing else */
} cs_kv_attn_args;

/* O = softmax(scale Q K^T over the visible keys) V for every new token and head,
 * scores, sums and O in 32 bits (the weights enter the product with V rounded to
 * the dtype).  A token that sees no key (before position 0) gets O = 0 and
 * lse = -inf, and so does one whose scores are all -infinity.  With more than 16 rows per key
 * head a row whose scores lie beyond 9e7 (f16) or 1.4e9 (bf16) from 0 is NaN.  Nothing that the cache holds at hidden keys changes a result. */
cs_status cs_kv_attention(cs_kv_t plan, const cs_kv_batch* batch, const cs_kv_attn_args* args, void* stream);

/* The same where every sequence's keys follow one common prefix of prefix_len
 * keys, key j of it in page prefix_pages[j / page_size] (device memory): the
 * new tokens see the whole prefix and their own sequence's keys up to themselves.
 * kv_lens, positions p and the page table count the sequences' own keys only.
 * The prefix is attended to once for all tokens of the batch; the two parts are
 * joined by their row maxima and sums. */
cs_status cs_kv_attention_shared(cs_kv_t plan, const cs_kv_batch* batch, const int32_t* prefix_pages, int prefix_len,
                                 const cs_kv_attn_args* args, void* stream);

/* An attention chain's forward over the cache: QKV = X Wqkv (stage 0 of `chain`,
 * a plan of kind CS_CHAIN_ATTN), append with rotation (in place in the chain's
 * QKV), attention over the cache into the chain's O, Y = O Wo (stage 2).  The
 * plans' devices and dtypes agree, heads = kv_heads = the chain's heads, head_dim 128, and
 * batch->tokens = the chain's M; the chain's plan must not split K (split_k = 1,
 * sk_tiles = -1).  append->qkv, qkv_stride, q_out and q_stride are not used.
 * Rows of Y behind the last sequence are not meaningful. */
cs_status cs_attn_cached_forward(cs_chain_t chain, cs_kv_t plan, const cs_kv_batch* batch, const cs_attn_args* args,
                                 const cs_kv_append_args* append, void* stream);

/* After the caller has synchronised the stream: CS_OK, or the first device error
 * since the plan was made or reset: CS_ERR_INVALID_ARG (lengths, pages or
 * positions that do not fit; the message names them), CS_ERR_WATCHDOG (internal).
 * From then on the plan's calls return CS_ERR_NEEDS_RESET.  Blocking. */
cs_status cs_kv_status(cs_kv_t plan);

/* Clear the device error and the workspace's counters (blocking). */
cs_status cs_kv_reset(cs_kv_t plan);

int cs_kv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CS_KV_H */
