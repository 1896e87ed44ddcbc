// Penalties, biases and masks on rows of logits.
//
// A workgroup takes a stretch of a row's ids and counts the row's tokens that
// fall into it in LDS, one word an id:
//   bits 0..20   how often the id was generated
//   bit 21       it stands in the prompt
//   bits 22..31  1 + the place of its bias
// so that one pass over the logits finds all that changes an id, and the counts
// are the same whatever order the atomics come in.  Every stretch of a row reads
// all of the row's tokens (from the caches but for the first).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"
#include "serving/mi_logits.h"

#define MI_LOGITS_EXPORT extern "C" __attribute__((visibility("default")))

namespace miattn {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kSaid = (1u << 21) - 1, kPrompt = 1u << 21;
constexpr int kBiasBit = 22;

struct Fp32 {};

struct LogitArgs {
  const char* logits;
  float* out;
  const int32_t* tokens;
  const int32_t* lengths;
  const int32_t* prompts;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias;
  const int32_t* mask;
  int64_t rows, vocab, logits_stride, out_stride, tokens_stride, bias_stride, mask_stride;
  int32_t token_cols, bias_cols, stretch, stretches;
};

// Eight logits, from an address that is a multiple of their size only.
template <typename T>
__device__ __forceinline__ void load8(const char* from, float (&x)[8]) {
  if constexpr (__is_same(T, Fp32)) {
    __builtin_memcpy(x, from, 32);
  } else {
    uint32_t w[4];
    __builtin_memcpy(w, from, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = T::lo(w[i]);
      x[2 * i + 1] = T::hi(w[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ float load1(const char* from) {
  if constexpr (__is_same(T, Fp32)) return *reinterpret_cast<const float*>(from);
  else return T::lo(*reinterpret_cast<const uint16_t*>(from));
}

// kCount: there are tokens or biases.
template <typename T, bool kCount>
__global__ void __launch_bounds__(kThreads) penalize_kernel(LogitArgs p) {
  extern __shared__ uint32_t words[];
  constexpr int kSize = __is_same(T, Fp32) ? 4 : 2;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / p.stretches;
  const int64_t first = static_cast<int64_t>(blockIdx.x % p.stretches) * p.stretch;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.stretch), p.vocab - first));
  const float* bias = p.bias + row * p.bias_stride;
  if constexpr (kCount) {
    for (int i = tid; i < p.stretch; i += kThreads) words[i] = 0;
    __syncthreads();
    if (p.bias_cols > 0) {
      for (int e = tid; e < p.bias_cols; e += kThreads) {
        const int64_t at = p.bias_ids[row * p.bias_stride + e] - first;
        if (at >= 0 && at < n) atomicMax(&words[at], static_cast<uint32_t>(e + 1) << kBiasBit);
      }
      __syncthreads();
    }
    if (p.token_cols > 0) {
      int len = p.lengths == nullptr ? p.token_cols : p.lengths[row];
      len = max(0, min(len, p.token_cols));
      const int prompt = p.prompts == nullptr ? 0 : p.prompts[row];
      const int32_t* tokens = p.tokens + row * p.tokens_stride;
      for (int i0 = 0; i0 < len; i0 += kThreads * 8) {
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + j * kThreads + tid;
          id[j] = i < len ? tokens[i] : -1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t at = id[j] - first;
          if (id[j] >= 0 && at >= 0 && at < n) {
            if (i0 + j * kThreads + tid < prompt) atomicOr(&words[at], kPrompt);
            else atomicAdd(&words[at], 1u);
          }
        }
      }
    }
    __syncthreads();
  }
  const float r = p.repetition == nullptr ? 1.f : p.repetition[row];
  const float f = p.frequency == nullptr ? 0.f : p.frequency[row], pr = p.presence == nullptr ? 0.f : p.presence[row];
  auto one = [&](float x, uint32_t w) {
    if constexpr (kCount) {
      if (w != 0) {
        const uint32_t said = w & kSaid, place = w >> kBiasBit;
        if ((w & (kSaid | kPrompt)) != 0) x = x > 0.f ? x / r : x * r;
        if (said != 0) x = x - f * static_cast<float>(said) - pr;
        if (place != 0) x += bias[place - 1];
      }
    }
    return x;
  };
  const char* from = p.logits + (row * p.logits_stride + first) * kSize;
  float* to = p.out + row * p.out_stride + first;
  const int32_t* mask = p.mask == nullptr ? nullptr : p.mask + row * p.mask_stride + (first >> 5);
  for (int i = tid * 8; i < n; i += kThreads * 8) {
    const uint32_t allowed = mask == nullptr ? 0xffu : static_cast<uint32_t>(mask[i >> 5]) >> (i & 31);
    if (i + 8 <= n) {
      float x[8];
      load8<T>(from + static_cast<int64_t>(i) * kSize, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = one(x[j], kCount ? words[i + j] : 0);
        if (!((allowed >> j) & 1)) x[j] = -kInf;
      }
      __builtin_memcpy(to + i, x, 32);
    } else {
      for (int j = 0; i + j < n; ++j) {
        const float x = one(load1<T>(from + static_cast<int64_t>(i + j) * kSize), kCount ? words[i + j] : 0);
        to[i + j] = (allowed >> j) & 1 ? x : -kInf;
      }
    }
  }
}

template <typename T>
int launch_penalize(const LogitArgs& p, hipStream_t stream) {
  const int64_t grid = p.rows * p.stretches;
  if (grid > INT32_MAX) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
  if (p.token_cols > 0 || p.bias_cols > 0) penalize_kernel<T, true><<<g, b, p.stretch * 4, stream>>>(p);
  else penalize_kernel<T, false><<<g, b, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

bool odd(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_LOGITS_EXPORT int logits_penalize(const mi_penalize_args* a, hipStream_t stream) {
  if (a == nullptr || a->dtype < MI_LOGITS_BF16 || a->dtype > MI_LOGITS_FP32 || a->rows < 0 || a->rows > INT32_MAX || a->vocab < 0 ||
      a->vocab > INT32_MAX || a->token_cols < 0 || a->token_cols > MI_LOGITS_MAX_TOKENS || a->bias_cols < 0 ||
      a->bias_cols > MI_LOGITS_MAX_BIAS || a->logits_stride < 0 || a->tokens_stride < 0 || a->bias_stride < 0 || a->mask_stride < 0 ||
      (a->rows > 1 && a->out_stride < a->vocab))
    return MI_ATTN_EINVAL;
  if (odd(a->logits, a->dtype == MI_LOGITS_FP32 ? 4 : 2)) return MI_ATTN_EINVAL;
  const void* words[] = {a->out, a->tokens, a->lengths, a->prompt_lengths, a->repetition, a->frequency, a->presence, a->bias_ids, a->bias, a->mask};
  for (const void* x : words)
    if (odd(x, 4)) return MI_ATTN_EINVAL;
  if (a->rows == 0 || a->vocab == 0) return MI_ATTN_OK;
  if (a->logits == nullptr || a->out == nullptr || (a->token_cols > 0 && a->tokens == nullptr) ||
      (a->bias_cols > 0 && (a->bias_ids == nullptr || a->bias == nullptr)))
    return MI_ATTN_EINVAL;
  if (a->logits == a->out && (a->dtype != MI_LOGITS_FP32 || (a->rows > 1 && a->logits_stride != a->out_stride))) return MI_ATTN_EINVAL;
  LogitArgs p;
  p.logits = static_cast<const char*>(a->logits); p.out = a->out; p.tokens = a->tokens; p.lengths = a->lengths; p.prompts = a->prompt_lengths;
  p.repetition = a->repetition; p.frequency = a->frequency; p.presence = a->presence;
  p.bias_ids = a->bias_ids; p.bias = a->bias; p.mask = a->mask;
  p.rows = a->rows; p.vocab = a->vocab; p.logits_stride = a->logits_stride; p.out_stride = a->out_stride;
  p.tokens_stride = a->tokens_stride; p.bias_stride = a->bias_stride; p.mask_stride = a->mask_stride;
  p.token_cols = a->token_cols; p.bias_cols = a->bias_cols;
  p.stretch = 8192;
  p.stretches = static_cast<int>((p.vocab + p.stretch - 1) / p.stretch);
  if (a->dtype == MI_LOGITS_BF16) return launch_penalize<Bf16>(p, stream);
  if (a->dtype == MI_LOGITS_FP16) return launch_penalize<Fp16>(p, stream);
  return launch_penalize<Fp32>(p, stream);
}
