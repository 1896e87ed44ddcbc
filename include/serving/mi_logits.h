/*
 * mi_logits — what a sampler changes in rows of logits before it ranks them:
 * penalties for repeated tokens, biases and a grammar's mask, for gfx950
 * (MI355X).  Part of libmi_topk.so.
 *
 * Row i, id j:
 *   x = logits[i][j]
 *   if j is among tokens[i][0 .. lengths[i]):  x = x > 0 ? x / r : x * r
 *   x = x - f * n - (n > 0 ? p : 0),  n the number of times that j is among the
 *       generated tokens, tokens[i][prompt_lengths[i] .. lengths[i])
 *   x = x + bias[i][e],  bias_ids[i][e] == j (the last such e)
 *   out[i][j] = bit j % 32 of mask[i][j / 32] ? x : -inf
 * with r = repetition[i], f = frequency[i], p = presence[i], in 32 bits.
 *
 * Tokens and bias ids outside [0, vocab) are none.  Lengths count as between 0
 * and token_cols, prompt lengths as between 0 and the row's length.  A row whose
 * mask allows nothing is -inf all over.  NaN stays NaN where it is allowed.
 *
 * All pointers are device pointers owned by the caller; nothing is allocated or
 * synchronised, all work is enqueued on `stream`, and results do not change from
 * run to run.  Status codes as in attention/mi_block_attention.h.
 */
#ifndef MI_LOGITS_H
#define MI_LOGITS_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { MI_LOGITS_BF16 = 0, MI_LOGITS_FP16 = 1, MI_LOGITS_FP32 = 2 };

#define MI_LOGITS_MAX_TOKENS ((1 << 21) - 1)
#define MI_LOGITS_MAX_BIAS 1023

/*
 *   logits   [rows][vocab] of `dtype`; out fp32 [rows][vocab]; rows
 *            logits_stride and out_stride elements apart.  out may be logits
 *            itself (fp32, the same stride), else they do not overlap.
 *   tokens   int32 [rows][token_cols], NULL where token_cols is 0; lengths and
 *            prompt_lengths int32 [rows] (NULL: token_cols, and 0).
 *   repetition, frequency, presence  fp32 [rows], NULL: 1, 0 and 0.
 *   bias_ids, bias  int32 and fp32 [rows][bias_cols], rows bias_stride apart.
 *   mask     int32 [rows][(vocab + 31) / 32], NULL: everything is allowed.
 */
typedef struct mi_penalize_args {
  const void* logits;
  float* out;
  const int32_t* tokens;
  const int32_t* lengths;
  const int32_t* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias;
  const int32_t* mask;
  int64_t rows, vocab, logits_stride, out_stride, tokens_stride, bias_stride, mask_stride;
  int32_t token_cols, bias_cols, dtype;
} mi_penalize_args;

int logits_penalize(const mi_penalize_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_LOGITS_H */
