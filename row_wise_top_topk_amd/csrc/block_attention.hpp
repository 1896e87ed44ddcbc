// What the forward and the backward of the block sparse attention share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"

#define MI_ATTN_EXPORT extern "C" __attribute__((visibility("default")))

namespace miattn {

struct Args {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* blocks;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  float* lse;
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, do_t, do_h;
  int64_t total_q, total_k, slots;
  int32_t num_seqs, heads, kv_heads, group, bs, lb, select, causal, tokens_per;
  float scale;
};

int make_args(const mi_block_attention_args* a, Args& p);

}  // namespace miattn
