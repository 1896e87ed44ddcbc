/*
 * mi_kv8 — a paged key/value cache in 8 bits and the attention that reads it,
 * for gfx950 (MI355X).  Part of libmi_topk.so.
 *
 * The cache.  k_cache and v_cache are arrays of pages [num_pages, HK,
 * block_size, D] of OCP e4m3 codes, k_scale and v_scale fp32 [num_pages, HK]:
 * a code c of page p and key head h stands for c * scale[p][h].  Block b of
 * sequence i (its tokens [b * block_size, (b + 1) * block_size)) lies in page
 * block_table[i][b]; lengths[i] is the number of its tokens.  The queries or
 * new tokens of a call are packed as in mi_block_attention.h: those of sequence
 * i are [cu[i], cu[i + 1]) and they are its last ones (token r of n stands at
 * position lengths[i] - n + r); cu NULL means one for each sequence.
 *
 * Entries of the block table outside [0, num_pages) are pages that are not
 * there: nothing is stored for them, and attention sees none of their keys.
 * A sequence holds block_table_cols * block_size tokens at most; positions
 * from there on are ignored, and so are negative ones.
 *
 * All pointers are device pointers owned by the caller; nothing is allocated or
 * synchronised, all work is enqueued on `stream`, results do not change from
 * run to run, and the values in cu, lengths, block_table and blocks are read on
 * the device only.  Status codes as in mi_block_attention.h.
 */
#ifndef MI_KV8_H
#define MI_KV8_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "attention/mi_block_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Stores the new tokens' keys and values.  A page's scale is the smallest power
 * of two, 2^-60 at least, that brings its largest finite value to 448 or less;
 * with a power of two a value's quotient by its scale is exact, and a code is
 * that quotient rounded to nearest even.  A page that a call finds empty (its
 * first token is new) takes the scale of the new tokens.  In a page that holds
 * tokens the scale can only grow: if the new tokens need a larger one, the
 * codes that are there are rounded again under it; a scale that is no power of
 * two grows to the next one.  Infinite values become
 * +-448 * scale, NaN stays NaN.  A call may store into a page
 * through one entry of one sequence's row only.
 *
 * k_mean (NULL, or fp32 [num_pages, HK, D]) receives, for each page that got
 * new tokens, the mean of the keys that the page holds then, as their codes
 * stand for them: the `means` of block_scores().
 *
 *   k, v  [total, HK, D] of `dtype`, strides as in mi_block_attention.h.
 */
typedef struct mi_kv8_append_args {
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  float* k_mean;
  const int32_t* block_table;
  const int32_t* lengths;
  const int32_t* cu;
  int64_t k_stride_t, k_stride_h, v_stride_t, v_stride_h;
  int64_t total, num_pages, block_table_stride;
  int32_t block_table_cols, dtype, num_seqs, kv_heads, dim, block_size;
} mi_kv8_append_args;

int kv8_append(const mi_kv8_append_args* args, hipStream_t stream);

/*
 * Attention of each sequence's last tokens over its cache: causal, over all
 * blocks (blocks NULL) or, for each query and key head, over those that
 * blocks[t][c][0..select) names (as in block_attention()).  out and lse as
 * there.  max_length is the caller's bound of the lengths: the work is split
 * by it, longer sequences are computed right but slowly.
 *
 *   q          [total_q, H, D] of `dtype`, strides as in mi_block_attention.h.
 *   out        [total_q, H, D] of `dtype`, contiguous; lse fp32 [total_q, H].
 *   scales     positive and finite; V scales count as between 2^-80 and 2^100.
 *              Where those that one query sees lie more than 2^100 apart, keys
 *              under the smaller ones lose their share of the weights' sum.
 *   workspace  kv8_attention_workspace() bytes, 16-byte aligned, need not be
 *              cleared; calls that overlap in time need one each.  At most 2^19
 *              rows of D + 2 floats, or about 32 rows for each token and head where
 *              sequences have few tokens.
 */
typedef struct mi_kv8_attention_args {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* lengths;
  const int32_t* cu;
  const int32_t* blocks;
  void* out;
  float* lse;
  void* workspace;
  uint64_t workspace_bytes;
  int64_t q_stride_t, q_stride_h;
  int64_t total_q, num_pages, block_table_stride, max_length;
  int32_t block_table_cols, dtype, num_seqs, heads, kv_heads, dim, block_size, select;
  float scale;
} mi_kv8_attention_args;

uint64_t kv8_attention_workspace(const mi_kv8_attention_args* args);
int kv8_attention(const mi_kv8_attention_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_KV8_H */
