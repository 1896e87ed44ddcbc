/*
 * mi_chunk — attention of a chunk of new tokens behind a paged 8-bit cache, for
 * gfx950 (MI355X).  Part of libmi_topk.so.
 *
 * Sequence i has lengths[i] tokens, of which the last n_i are the chunk's own,
 * packed as in mi_kv8.h: rows [cu[i], cu[i + 1]) of q, k and v (cu NULL: one
 * each).  The lengths[i] - n_i tokens before them, its context, lie in pages
 * (mi_kv8.h gives their layout); the new tokens' keys and values are those of k
 * and v, in 16 bits, and need not be in the cache.  Token r of the chunk sees
 * the context and the new tokens up to itself:
 *
 *   out = sum_j p_j v_j,  p = softmax(scale q . k_j),  lse = log sum exp(scale q . k_j)
 *
 * Pages outside [0, num_pages), and context from block_table_cols * block_size
 * tokens on, are not there: nothing is seen of them.  Where a chunk is longer
 * than its sequence the tokens that would stand before its start see nothing and
 * are not seen.  A query that sees no key, and a row behind the last sequence,
 * has out 0 and lse -inf.  Infinities and NaN count where they are visible only;
 * those among the values then count whatever their weight, also one that is 0 in
 * 32 bits.
 *
 * All pointers are device pointers owned by the caller; nothing is allocated or
 * synchronised, all work is enqueued on `stream`, results do not change from
 * run to run, and the values in cu, lengths and block_table are read on the
 * device only.  Status codes as in mi_block_attention.h.
 */
#ifndef MI_CHUNK_H
#define MI_CHUNK_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "attention/mi_block_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   q          [total][H][D] of `dtype`, k and v [total][HK][D], strides as in
 *              mi_block_attention.h (k's and v's token strides likewise below
 *              MI_ATTN_MAX_STRIDE).
 *   out        [total][H][D] of `dtype`, contiguous; lse fp32 [total][H].
 *   scales     positive and finite; V scales count as between 2^-80 and 2^100.
 *              Where those that one query sees (new tokens: 1) lie more than 2^100
 *              apart, keys under the smaller ones lose their share of the
 *              weights' sum.  fp16 weights are kept to 2^-37 of a row's largest
 *              where V scales lie in [2^-15, 2^8); below, what is lost is less
 *              than half of fp16's least step for up to 2^18 keys; from 2^8 on,
 *              where full codes pass fp16's range, it is 2^-37 of the largest
 *              product of a weight and its scale.
 *   max_length the caller's bound of the lengths: the work is split by it, longer
 *              sequences are computed right but slowly, and so are few tokens of
 *              sequences that are far shorter.
 *   workspace  chunk_attention_workspace() bytes, 16-byte aligned, need not be
 *              cleared; calls that overlap in time need one each.
 */
typedef struct mi_chunk_attention_args {
  const void* q;
  const void* k;
  const void* v;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* lengths;
  const int32_t* cu;
  void* out;
  float* lse;
  void* workspace;
  uint64_t workspace_bytes;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h;
  int64_t total, num_pages, block_table_stride, max_length;
  int32_t block_table_cols, dtype, num_seqs, heads, kv_heads, dim, block_size;
  float scale;
} mi_chunk_attention_args;

uint64_t chunk_attention_workspace(const mi_chunk_attention_args* args);
int chunk_attention(const mi_chunk_attention_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_CHUNK_H */
