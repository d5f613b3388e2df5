/*
 * cs_kv4.h -- C ABI of the paged key/value cache held in 4 bits, for GB300
 * (sm_103a), in the same library as cs_kv.h.
 *
 * What it computes.  The operators of cs_kv.h over a cache that takes 0.266 of the
 * memory (and, for single tokens, of the bytes that attention has to bring):
 * cs_kv4_append rotates and quantises as it writes, cs_kv4_attention and
 * cs_kv4_attention_shared attend to what the cache stands for, cs_kv4_read
 * gives it back in 16 bits, cs_attn_cached4_forward is an attention layer over it.
 * Plans, batches, page tables, windows, sinks, status and conventions are those of cs_kv.h: any
 * plan of cs_kv_plan serves caches of either kind, its dtype is that of Q, O and the
 * values, its cache_layout that of the codes.
 *
 * The format.  A group is 32 consecutive dimensions of one key (or value) of one
 * head, and has
 *   a scale s: an unsigned byte of 5 exponent bits (bias 15) and 3 mantissa bits, so that
 *     the half whose bits are the byte << 7 is s: steps of 2^-17 below 2^-14, at most
 *     61440 (0xF7); 0xF8 .. 0xFF stand for no number, and every value of the group is
 *     NaN (infinite scales make infinite values or NaN);
 *   32 codes c + 8 of 4 bits, c in -7 .. 7 (-8 is never written, and is read as -8).
 * The value is s c, a number of both 16-bit types: reading rounds nothing.  (Caches that are
 * not written here may hold values beyond f16's 65504; a plan of that type may give infinities, or NaN, for them and
 * to rows that see them.)
 * Written: s = the scale nearest to max |x| / 7 (ties to the even byte), c = x / s rounded to
 * the nearest (ties to even), within -7 .. 7, where x is what cs_kv_append would
 * have stored.  So |x - s c| <= 0.54 s while 2^-14 <= max |x| / 7 <= 61440; below, the
 * scale's own rounding (2^-18) counts up to 7 times more, above, values are cut off at
 * +-430080.  A group with a value that is not finite gets scale 0xFF.
 * Codes: [num_pages, page_size, kv_heads, head_dim / 2] bytes (TOKEN) or
 * [num_pages, kv_heads, page_size, head_dim / 2] (HEAD); of the 8 values in a (little
 * endian) 32-bit word, value 2 j lies at bit 4 j and value 2 j + 1 at bit 16 + 4 j.
 * Scales: [num_pages, kv_heads, page_size, head_dim / 32] bytes in both layouts.
 */
#ifndef CS_KV4_H
#define CS_KV4_H

#include "cs_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A K or V cache: device memory, both parts 16-byte aligned. */
typedef struct cs_kv4_cache {
  void* codes;
  void* scales;
} cs_kv4_cache;

typedef struct cs_kv4_append_args {
  const void* qkv;            /* as in cs_kv_append_args */
  long long qkv_stride;
  void* q_out;
  long long q_stride;
  cs_kv4_cache k;             /* the caches' parts overlap neither each other nor qkv nor q_out */
  cs_kv4_cache v;
  const float* rope;
  int rope_rows;
  const int32_t* positions;
} cs_kv4_append_args;

/* cs_kv_append into a cache in 4 bits.  The rotation rounds each product and each sum
 * to 32 bits (no fused multiply-add) and the result to the dtype, and what is
 * quantised is that result: the same inputs give the same bytes.  Two tokens sent to one
 * slot leave a mixture of their codes and scales there. */
cs_status cs_kv4_append(cs_kv_t plan, const cs_kv_batch* batch, const cs_kv4_append_args* args, void* stream);

typedef struct cs_kv4_read_args {
  cs_kv4_cache k;             /* used where its output is asked for */
  cs_kv4_cache v;
  void* k_out;                /* rows of kv_heads * head_dim, or NULL (not both); overlap nothing else */
  long long k_stride;         /* elements between rows; 0 = kv_heads * head_dim */
  void* v_out;
  long long v_stride;
} cs_kv4_read_args;

/* The values of the batch's new tokens' keys, as the cache holds them, into the tokens' rows:
 * the inverse of the append.  A batch whose cu_q counts whole sequences (n = kv_lens[b]) reads
 * whole sequences.  Rows of tokens before position 0 and of padding stay as they were. */
cs_status cs_kv4_read(cs_kv_t plan, const cs_kv_batch* batch, const cs_kv4_read_args* args, void* stream);

typedef struct cs_kv4_attn_args {
  const void* q;              /* as in cs_kv_attn_args */
  long long q_stride;
  cs_kv4_cache k;
  cs_kv4_cache v;
  void* out;
  long long out_stride;
  float* lse;
} cs_kv4_attn_args;

/* cs_kv_attention (cs_kv_attention_shared) over a cache in 4 bits: scores, sums and
 * O in 32 bits of the exact values, the weights rounded to the dtype for the product with V.  (f16 has
 * no weights below 2^-25 of a row's largest, with at most 16 rows per key head 2^-32.  There lse is too small where a row's
 * largest query times the scale is beyond 2^134, scores that nearly always overflow.) */
cs_status cs_kv4_attention(cs_kv_t plan, const cs_kv_batch* batch, const cs_kv4_attn_args* args, void* stream);
cs_status cs_kv4_attention_shared(cs_kv_t plan, const cs_kv_batch* batch, const int32_t* prefix_pages, int prefix_len,
                                  const cs_kv4_attn_args* args, void* stream);

/* cs_attn_cached_forward over a cache in 4 bits.  append->qkv, qkv_stride, q_out and
 * q_stride are not used. */
cs_status cs_attn_cached4_forward(cs_chain_t chain, cs_kv_t plan, const cs_kv_batch* batch, const cs_attn_args* args,
                                  const cs_kv4_append_args* append, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CS_KV4_H */
