// Penalties, biases and masks on rows of logits.
//
// A workgroup takes a stretch of a row's ids and counts the row's tokens that
// fall into it in LDS, one word an id:
//   bits 0..20   how often the id was generated
//   bit 21       it stands in the prompt
//   bits 22..31  1 + the place of its bias
// so that one pass over the logits finds all that changes an id, and the counts
// are the same whatever order the atomics come in.  Every stretch of a row reads
// all of the row's tokens (from the caches but for the first), so stretches are
// long where there are enough of them.
//
// Measured (in a graph): 64 rows of 128256, bf16, 300 to 8000 tokens, 20 biases and
// a mask: 13.8 us, 51 MB at 3.7 TB/s; 256 x 32000, up to 500 tokens: 12.6 us, 49 MB.
// A lane takes four ids, so that the stores of a wavefront are whole lines: with
// eight ids a lane they took 17 and 16 us.  32 rows of 151937 behind 50000 to 100000
// tokens: 19.3 us, 9.9 behind 500: thirteen stretches look at 75000 tokens each, 8
// instructions a token.  3 x 32000: 3.8 us, the chain from the lengths over the
// tokens to the logits.  Slower: the logits loaded before the tokens (18 us for the
// first: loads come back in order), results written by a pass of their own.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"
#include "serving/mi_logits.h"

#define MI_LOGITS_EXPORT extern "C" __attribute__((visibility("default")))

namespace miattn {
namespace {

constexpr uint32_t kSaid = (1u << 21) - 1, kPrompt = 1u << 21;
constexpr int kBiasBit = 22;
constexpr int kThreads = 1024;
constexpr uint32_t kDies = 8;

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
  int32_t token_cols, bias_cols, stretches;
};

// Four logits from an address that is a multiple of their size only, the n that
// there are.
template <typename T>
__device__ __forceinline__ void load4(const char* from, int n, float (&x)[4]) {
  if constexpr (__is_same(T, Fp32)) {
    if (n >= 4) {
      __builtin_memcpy(x, from, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = j < n ? reinterpret_cast<const float*>(from)[j] : 0.f;
    }
  } else {
    if (n >= 4) {
      uint32_t w[2];
      __builtin_memcpy(w, from, 8);
      x[0] = T::lo(w[0]);
      x[1] = T::hi(w[0]);
      x[2] = T::lo(w[1]);
      x[3] = T::hi(w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = T::lo(j < n ? reinterpret_cast<const uint16_t*>(from)[j] : 0);
    }
  }
}

// Calls count(place) for the tokens [from, to) that are ids first + place, place < n.
// A wavefront behind the last token leaves at once: with short rows of tokens the
// instructions of all wavefronts would cost more than the loads.
template <typename F>
__device__ __forceinline__ void each_token(const int32_t* tokens, int from, int to, uint32_t first, uint32_t n, F count) {
  constexpr int kAtOnce = 4, kStep = kThreads * 4;
  auto take = [&](const int32_t (&id)[4]) {
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const uint32_t at = static_cast<uint32_t>(id[z]) - first;  // negative ids lie behind any n
      if (at < n) count(at);
    }
  };
  const int mine = static_cast<int>(threadIdx.x) * 4;
  for (; to - from >= kAtOnce * kStep; from += kAtOnce * kStep) {
    int32_t id[kAtOnce][4];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) __builtin_memcpy(id[j], tokens + from + j * kStep + mine, 16);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) take(id[j]);
  }
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x)) * 4;
  for (; from + wave < to; from += kStep) {
    const int i = from + mine;
    int32_t id[4];
    if (i + 4 <= to) {
      __builtin_memcpy(id, tokens + i, 16);
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z) id[z] = i + z < to ? tokens[i + z] : -1;
    }
    take(id);
  }
}

// kCount: there are tokens or biases.
template <typename T, bool kCount, int kUnits>
__global__ void __launch_bounds__(kThreads) penalize_kernel(LogitArgs p) {
  constexpr int kStretch = kThreads * 4 * kUnits;
  __shared__ __attribute__((aligned(16))) uint32_t words[kCount ? kStretch : 4];
  constexpr int kSize = __is_same(T, Fp32) ? 4 : 2;
  const int tid = threadIdx.x;
  // The dies take workgroups in turn and have a cache each: a die works on consecutive
  // rows, so that a row's tokens come into one cache (32 rows of 151937 behind 75000
  // tokens: 25 us with a row's stretches over all dies, 21 so).
  const uint32_t at = blockIdx.x % kDies * (gridDim.x / kDies) + blockIdx.x / kDies;
  const int64_t row = at / p.stretches;
  if (row >= p.rows) return;
  const int64_t first = static_cast<int64_t>(at % p.stretches) * kStretch;
  const int n = static_cast<int>(min(static_cast<int64_t>(kStretch), p.vocab - first));
  const char* from = p.logits + (row * p.logits_stride + first) * kSize;
  const int32_t* mask = p.mask == nullptr ? nullptr : p.mask + row * p.mask_stride + (first >> 5);
  if constexpr (kCount) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) *reinterpret_cast<uint4*>(words + (u * kThreads + tid) * 4) = uint4{0, 0, 0, 0};
    __syncthreads();
    if (p.bias_cols > 0) {
      for (int e = tid; e < p.bias_cols; e += kThreads) {
        const uint32_t at = static_cast<uint32_t>(p.bias_ids[row * p.bias_stride + e]) - static_cast<uint32_t>(first);
        if (at < static_cast<uint32_t>(n)) atomicMax(&words[at], static_cast<uint32_t>(e + 1) << kBiasBit);
      }
      __syncthreads();
    }
    if (p.token_cols > 0) {
      int len = p.lengths == nullptr ? p.token_cols : p.lengths[row];
      len = max(0, min(len, p.token_cols));
      const int prompt = p.prompts == nullptr ? 0 : max(0, min(p.prompts[row], len));
      const int32_t* tokens = p.tokens + row * p.tokens_stride;
      each_token(tokens, 0, prompt, static_cast<uint32_t>(first), n, [&](uint32_t at) { atomicOr(&words[at], kPrompt); });
      each_token(tokens, prompt, len, static_cast<uint32_t>(first), n, [&](uint32_t at) { atomicAdd(&words[at], 1u); });
    }
    __syncthreads();
  }
  const float r = p.repetition == nullptr ? 1.f : p.repetition[row];
  // (1 / r can be infinite where y / r is not)
  const float raise = fabsf(r) < 0x1p-126f ? 0x1p64f : 1.f, divisor = r * raise, inverse = 1.f / divisor;
  const float f = p.frequency == nullptr ? 0.f : p.frequency[row], pr = p.presence == nullptr ? 0.f : p.presence[row];
  const float* bias = p.bias + row * p.bias_stride;
  auto changed = [&](float y, uint32_t w) {
    // y / r: a quotient that one step of Newton's rounds to nearest
    const float z = y * raise, q = z * inverse, near = fmaf(fmaf(-q, divisor, z), inverse, q);
    const float up = fabsf(near) < kInf ? near : q;
    y = (w << (32 - kBiasBit)) != 0 ? (y > 0.f ? up : y * r) : y;
    const uint32_t said = w & kSaid;
    y = said != 0 ? y - f * static_cast<float>(said) - pr : y;
    if ((w >> kBiasBit) != 0) y += bias[(w >> kBiasBit) - 1];
    return y;
  };
  float* to = p.out + row * p.out_stride + first;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int i = (u * kThreads + tid) * 4;
    if (i >= n) break;
    float y[4];
    load4<T>(from + static_cast<int64_t>(i) * kSize, n - i, y);
    const uint32_t allowed = mask == nullptr ? 0xfu : static_cast<uint32_t>(mask[i >> 5]) >> (i & 31);
    if constexpr (kCount) {
      uint32_t w[4];
      __builtin_memcpy(w, __builtin_assume_aligned(words + i, 16), 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (w[j] != 0) y[j] = changed(y[j], w[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // a bit that is not set makes it -inf
      const uint32_t on = static_cast<uint32_t>(static_cast<int32_t>(allowed << (31 - j)) >> 31);
      y[j] = __uint_as_float((__float_as_uint(y[j]) & on) | (0xff800000u & ~on));
    }
    if (i + 4 <= n) {
      __builtin_memcpy(to + i, y, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) to[i + j] = y[j];
    }
  }
}

int64_t workgroups(const LogitArgs& p, int units) { return p.rows * ((p.vocab + kThreads * 4 * units - 1) / (kThreads * 4 * units)); }

template <typename T, int kUnits>
int launch_as(LogitArgs p, hipStream_t stream) {
  const int64_t all = workgroups(p, kUnits), grid = (all + kDies - 1) / kDies * kDies;
  p.stretches = static_cast<int>(all / p.rows);
  if (grid > UINT32_MAX / kThreads) return MI_ATTN_EINVAL;  // a launch has less than 2^32 threads
  const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
  if (p.token_cols > 0 || p.bias_cols > 0) penalize_kernel<T, true, kUnits><<<g, b, 0, stream>>>(p);
  else penalize_kernel<T, false, kUnits><<<g, b, 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

// Stretches of one to four times 4096 ids.  512 workgroups run at once, two on a
// compute unit, and a round of them takes about as long as their units and one more
// for what comes before; the longest stretch of the cheapest, which reads the tokens
// least often.  Measured (us in a graph, 1 to 4 units): 3 x 32000: 4.0, 4.5, 4.8, 5.4;
// 8 x 128256: 5.3, 6.0, 6.9, 7.8; 20 x 128256: 9.3, 8.4, 8.0, 8.8; 32 x 151937: 13.4,
// 12.0, 10.5, 11.8; behind 60000 tokens: 22.8, 18.5, 15.4, 16.4; 48 x 128256: 16.7,
// 15.0, 15.5, 12.9; 64 x 128256: 24, 18.7, 17.6, 14.1; 300 x 32000: 26.1, 20.8, 19.1,
// 20.2.
template <typename T>
int launch_penalize(const LogitArgs& p, hipStream_t stream) {
  int units = 1;
  int64_t least = INT64_MAX;
  for (int u = 1; u <= 4; ++u) {
    const int64_t cost = (workgroups(p, u) + 511) / 512 * (u + 1);
    if (cost <= least) {
      least = cost;
      units = u;
    }
  }
  if (units == 1) return launch_as<T, 1>(p, stream);
  if (units == 2) return launch_as<T, 2>(p, stream);
  return units == 3 ? launch_as<T, 3>(p, stream) : launch_as<T, 4>(p, stream);
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
  p.stretches = 0;
  if (a->dtype == MI_LOGITS_BF16) return launch_penalize<Bf16>(p, stream);
  if (a->dtype == MI_LOGITS_FP16) return launch_penalize<Fp16>(p, stream);
  return launch_penalize<Fp32>(p, stream);
}
