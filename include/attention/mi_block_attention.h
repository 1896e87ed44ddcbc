/*
 * mi_block_attention — what stands on both sides of the selection in block
 * sparse attention, for gfx950 (MI355X).  Part of libmi_topk.so.
 *
 *   block_means / block_scores   a cheap score of every key block for every
 *       query and key head: the fp32 logits rows that topk_indices() selects
 *       from;
 *   block_attention / block_attention_backward   attention over the selected
 *       blocks and its gradient.
 *
 * Sequences are packed: token t of q, dout, out is row t; sequence i holds the
 * queries [cu_q[i], cu_q[i+1]) and the keys [cu_k[i], cu_k[i+1]).  Query r of a
 * sequence with n queries and m keys stands at position m - n + r: the last
 * query at the last key.  H query heads share HK key heads in groups of
 * G = H / HK consecutive ones.  Block b of a sequence is its keys
 * [b * block_size, (b + 1) * block_size).
 *
 * blocks[t][c][s] (int32) are the blocks that token t selects for key head c,
 * in any order; an entry that is negative or names no block of the sequence
 * selects nothing, a block named twice counts once.  Key j is visible to query
 * t under head c if its block is selected and, with `causal`, j <= position.
 *
 *   out[t][h] = sum_j p_j v_j,  p_j = exp(scale q.k_j - lse),
 *   lse[t][h] = log sum_j exp(scale q.k_j)     over the visible keys j.
 *
 * Infinities and NaN count where they are visible and nowhere else (the
 * workgroups that meet any go over their keys a second time, one by one).
 * A query without visible keys, and a row behind the last sequence, has out 0
 * and lse -inf, and its gradient is 0.  Keys that no query sees, and keys
 * behind the last sequence, have gradient 0.
 *
 * Pointers are device pointers owned by the caller.  Nothing is allocated or
 * synchronised, all work is enqueued on `stream`, and every result is the same
 * from run to run (no floating-point atomics).  cu_q and cu_k are read on the
 * device only; they must start at 0 and not decrease.  Calls that overlap in
 * time need workspaces of their own; a workspace needs no clearing.
 */
#ifndef MI_BLOCK_ATTENTION_H
#define MI_BLOCK_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MI_ATTN_OK 0
#define MI_ATTN_EINVAL 1     /* bad argument; nothing was launched        */
#define MI_ATTN_EWORKSPACE 2 /* workspace_bytes below what the call needs */
#define MI_ATTN_ELAUNCH 3    /* a kernel launch failed                    */

#define MI_ATTN_BF16 0
#define MI_ATTN_FP16 1

/* Largest number of selected blocks per query and key head. */
#define MI_ATTN_MAX_SELECT 1024

/* Token strides of k and v in attention are below this many elements. */
#define MI_ATTN_MAX_STRIDE (1 << 23)

/*
 * Mean of the keys of each block, fp32 [rows, HK, D] with
 * rows = total_k / block_size + num_seqs: block b of sequence i is row
 * cu_k[i] / block_size + i + b.  Rows that are no block are set to 0.
 *
 *   k            [total_k, HK, D] of `dtype`, unit stride along D,
 *                k_stride_t / k_stride_h elements between tokens / heads
 *                (multiples of 8), 16-byte aligned.
 *   cu_k         int32 [num_seqs + 1], or NULL for one sequence.
 *   block_size   16, 32, 64 or 128.  D is 64 or 128.
 */
int block_means(int32_t dtype, const void* k, int64_t k_stride_t, int64_t k_stride_h, int64_t total_k,
                int32_t kv_heads, int32_t dim, int32_t block_size, const int32_t* cu_k, int32_t num_seqs,
                float* means, hipStream_t stream);

/*
 * Scores of blocks:  scores[t][c][b] = scale * max over the G heads h of group
 * c of q[t][h] . mean of block b, for the blocks b < max_blocks that hold a
 * position up to the query's; counts[t][c] is the number of those.  The first
 * `first` of them and the last `last` of them are forced: their score is +inf.
 * Scores from counts[t][c] on are -inf.  Rows of queries without blocks, and
 * rows behind the last sequence, are -inf with count 0.  A NaN among a
 * block's products makes its score NaN.
 *
 * The means are those of block_means() (block_table NULL; cu_k as there), or
 * of a paged cache: block_table int32 [num_seqs, max_pages >= max_blocks],
 * block_table_stride entries between rows; block b of sequence i is row
 * block_table[i][b] of `means` and the sequence holds lengths[i] keys.  An
 * entry outside [0, mean_rows), like a packed block behind the rows, makes the
 * block's score -inf.
 *
 *   q       [total_q, H, D] of `dtype`, strides as for k above.
 *   total_k keys of the one sequence where cu_k is NULL (packed form).
 *   scores  fp32 [total_q, HK, max_blocks];  counts int32 [total_q, HK].
 *   cu_q    int32 [num_seqs + 1] or NULL: one sequence (packed form), one
 *           query for each sequence (paged form).
 */
typedef struct mi_block_scores_args {
  const void* q;
  const float* means;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* lengths;
  const int32_t* block_table;
  float* scores;
  int32_t* counts;
  int64_t q_stride_t, q_stride_h;
  int64_t total_q, total_k, mean_rows, block_table_stride;
  int32_t dtype, num_seqs, heads, kv_heads, dim, block_size;
  int32_t max_blocks, first, last;
  float scale;
} mi_block_scores_args;

int block_scores(const mi_block_scores_args* args, hipStream_t stream);

/*
 * Attention over the selected blocks (the operation above) and its gradient.
 *
 *   q, k, v, dout  of `dtype`, unit stride along D, strides in elements
 *                  (multiples of 8; token strides of k and v below
 *                  MI_ATTN_MAX_STRIDE), 16-byte aligned; D 64 or 128; H a multiple
 *                  of HK with H / HK <= 128.
 *   blocks         int32 [total_q, HK, select], contiguous, 1 <= select <=
 *                  MI_ATTN_MAX_SELECT.
 *   out, dq        [total_q, H, D] contiguous; dk, dv [total_k, HK, D]
 *                  contiguous; lse fp32 [total_q, H].
 *   rest           NULL, or like out: what the rounding of out leaves out.  The
 *                  forward computes out more exactly then; the backward takes it
 *                  in where it is given (bf16: dq 3 times nearer to the exact
 *                  one).
 *   scale          positive and finite.
 * block_attention_backward() takes out, rest and lse as block_attention()
 * gave them and a workspace of block_attention_workspace() bytes (16-byte aligned):
 * a bit for each token, key head and block, of one sequence or another, so it
 * grows with the square of the tokens, and fp32 sums of block_size x D keys and
 * values for every block and every 2048 rows (tokens x H / HK) that select.
 */
typedef struct mi_block_attention_args {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* blocks;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  void* rest;
  float* lse;
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  void* workspace;
  uint64_t workspace_bytes;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h, dout_stride_t, dout_stride_h;
  int64_t total_q, total_k;
  int32_t dtype, num_seqs, heads, kv_heads, dim, block_size, select, causal;
  float scale;
} mi_block_attention_args;

int block_attention(const mi_block_attention_args* args, hipStream_t stream);

uint64_t block_attention_workspace(const mi_block_attention_args* args);
int block_attention_backward(const mi_block_attention_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_BLOCK_ATTENTION_H */
