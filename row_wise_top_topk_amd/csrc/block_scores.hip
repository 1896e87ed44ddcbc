// Block means and block scores: the fp32 rows that the top-k selection of
// blocks reads.
//
//   mean_b = (1 / |b|) sum of the keys of block b
//   score  = scale * max over the group's heads h of q_h . mean_b
//
// The means are read in fp32 and the scores are held in fp32 throughout: a
// product q . mean runs on the 16-bit matrix cores with the mean as a sum of
// three bf16 terms (8 bits each, 24 together), or, for fp16 queries, of two
// fp16 terms (11 bits each and the sign of the second) of the block's mean
// scaled by a power of two to below 1.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

struct MeanArgs {
  const void* k;
  const int32_t* cu_k;
  float* means;
  int64_t k_t, k_h, total_k, rows;
  int32_t num_seqs, kv_heads, bs;
};

// One wavefront per block and key head; D / 8 lanes read a key's chunks, the
// others the keys beside it.  Bound by the read of k, below some thousand blocks
// by its start (8192 tokens, 4 heads of 128: 8.4 MB in 4.4 us).
template <typename T, int D>
__global__ void __launch_bounds__(256) block_means_kernel(MeanArgs p) {
  constexpr int kChunks = D / 8, kKeys = 64 / kChunks;
  const int lane = threadIdx.x & 63;
  const uint32_t item = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = item / p.kv_heads;
  const int hk = static_cast<int>(item % p.kv_heads);
  if (row >= p.rows) return;
  const Place at = place_of(p.cu_k, p.num_seqs, p.total_k, row, p.bs);
  int n = 0;
  if (at.seq < p.num_seqs && at.first < at.end) n = static_cast<int>(at.end - at.first < p.bs ? at.end - at.first : p.bs);
  const int chunk = lane % kChunks, sub = lane / kChunks;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n > 0) {
    const char* from = static_cast<const char*>(p.k) + (at.first * p.k_t + hk * p.k_h + chunk * 8) * 2;
#pragma unroll 4
    for (int j = sub; j < n; j += kKeys) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(from + j * p.k_t * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[2 * e] += T::lo(x[e]);
        sum[2 * e + 1] += T::hi(x[e]);
      }
    }
  }
#pragma unroll
  for (int d = kChunks; d < 64; d <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], d);
  if (sub == 0) {
    const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
    float* to = p.means + (row * p.kv_heads + hk) * D + chunk * 8;
    *reinterpret_cast<f32x4*>(to) = f32x4{sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv};
    *reinterpret_cast<f32x4*>(to + 4) = f32x4{sum[4] * inv, sum[5] * inv, sum[6] * inv, sum[7] * inv};
  }
}

struct ScoreArgs {
  const void* q;
  const float* means;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* lengths;
  const int32_t* table;
  float* scores;
  int32_t* counts;
  int64_t q_t, q_h, total_q, total_k, mean_rows, table_stride, slots;
  int32_t num_seqs, heads, kv_heads, group, bs, lb, max_blocks, first, last, tokens_per, chunk;
  float scale;
};

// Splits 8 floats into bf16 terms: x = t0 + t1 + t2 up to 2^-24 of x.
__device__ __forceinline__ void split3(const float* x, u32x4* t) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      t[i][e] = Bf16::pack(a, b);
      a -= Bf16::lo(t[i][e]);
      b -= Bf16::hi(t[i][e]);
    }
  }
}

// Splits 8 floats below 1 into fp16 terms: x = t0 + 2^-11 t1 up to 2^-23.
__device__ __forceinline__ void split2(const float* x, u32x4* t) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = Fp16::pack(x[2 * e], x[2 * e + 1]);
    const float a = (x[2 * e] - Fp16::lo(w)) * 2048.f, b = (x[2 * e + 1] - Fp16::hi(w)) * 2048.f;
    t[0][e] = w;
    t[1][e] = Fp16::pack(a, b);
  }
}

// The best score of a group's heads, product by product: the terms of an
// infinity have a NaN among them, so where the sum of them is one it is none of
// theirs yet.
template <typename T, int D>
__device__ __noinline__ float best_again(const ScoreArgs& p, const float* mean, const char* q) {
  float s = -kInf;
  for (int g = 0; g < p.group && s == s; ++g) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q + g * p.q_h * 2);
    float x = 0.f;
    for (int d = 0; d < D / 2; ++d) x = fmaf(T::hi(w[d]), mean[2 * d + 1], fmaf(T::lo(w[d]), mean[2 * d], x));
    s = x > s || x != x ? x : s;
  }
  return s;
}

// A workgroup takes RT * 16 rows (the group's heads of consecutive tokens) of
// one key head and `chunk` blocks, a wavefront 16 blocks at a time: the queries
// stay in registers, the means go from memory to registers and are split
// there, once for all RT row tiles.  The maximum over the heads crosses lanes
// through LDS, since a group need not divide a tile.
//
// Measured: 8192 tokens, 32/4 heads of 128, 128 blocks: 43 us, of which the
// vector unit is busy for half (the split of the means, the conversion's cost),
// the matrix units for a seventh.
// 128 rows a workgroup would split the means half as often, but leave two
// wavefronts a SIMD: 53 us.  64 queries of 64/8 heads over up to 60000 keys: 29
// us, 128 MB of means at 4.4 TB/s: the read bounds it.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(256, RT == 8 ? 2 : 4) block_scores_kernel(ScoreArgs p) {
  constexpr bool kHalf = __is_same(T, Fp16);
  constexpr int kPad = 20;
  __shared__ __attribute__((aligned(16))) float s_best[4][RT * 16 * kPad];
  __shared__ __attribute__((aligned(1024))) char s_q[RT * 32 * D];
  const int hk = blockIdx.x % p.kv_heads;
  const int64_t slot = static_cast<int>(blockIdx.x / p.kv_heads);
  int32_t x0, x1;
  const Place at = place_of(p.cu_q, p.num_seqs, p.total_q, slot, p.tokens_per, [&](int i) {
    if (p.table == nullptr) return cu_at(p.cu_k, p.num_seqs, p.total_k, i);
    return i < p.num_seqs ? p.lengths[i] : 0;
  }, x0, x1);
  const int64_t left = at.end - at.first;
  const int tokens = static_cast<int>(left < 0 ? 0 : (left < p.tokens_per ? left : p.tokens_per));
  if (tokens == 0) return;
  int64_t len = 0, base = 0;
  if (at.seq < p.num_seqs) {
    if (p.table != nullptr) {
      len = x0;
    } else {
      len = x1 - x0;
      base = (x0 >> p.lb) + at.seq;
    }
    if (len < 0) len = 0;
  }
  const int64_t pos0 = len - (at.end - at.begin) + (at.first - at.begin);  // position of the first token
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto count_of = [&](int tl) {
    const int64_t pos = pos0 + tl;
    if (at.seq >= p.num_seqs || len == 0 || pos < 0) return 0;
    const int64_t n = (pos >> p.lb) + 1;
    return static_cast<int>(n < p.max_blocks ? n : p.max_blocks);
  };
  // means of no rows hold no block, and nothing is read of them
  const int seen = p.mean_rows > 0 ? count_of(tokens - 1) : 0;  // positions ascend
  if (blockIdx.y == 0)
    for (int tl = threadIdx.x; tl < tokens; tl += 256) p.counts[(at.first + tl) * p.kv_heads + hk] = count_of(tl);

  const int kg = lane >> 4;
  // the rows' queries go through LDS: read once and whole for the four
  // wavefronts, which all need all of them (read by each from memory: 55 us
  // instead of 42 for 8192 tokens of 32 heads)
  u32x4 q[RT][D / 32];
  if (seen > 0) {
    constexpr int kLanes = D / 8;
#pragma unroll
    for (int e = threadIdx.x; e < RT * 16 * kLanes; e += 256) {
      const int row = e / kLanes, tl = row / p.group;
      u32x4 x = {0, 0, 0, 0};
      if (tl < tokens)
        x = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.q) +
            ((at.first + tl) * p.q_t + (hk * p.group + row % p.group) * p.q_h + (e % kLanes) * 8) * 2);
      *reinterpret_cast<u32x4*>(s_q + tile_at<D>(row, e % kLanes)) = x;
    }
    __syncthreads();
    const uint32_t from = lds_offset(s_q) + tile_at<D>(lane & 15, kg);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) q[t][i] = lds_read16((from ^ (i * 64)) + t * 32 * D);
  }
  float* best = s_best[wave];
  const int end = min(p.max_blocks, (static_cast<int>(blockIdx.y) + 1) * p.chunk);
  for (int b0 = blockIdx.y * p.chunk + wave * 16; b0 < end; b0 += 64) {
    bool bad = p.mean_rows == 0;
    if (b0 < seen) {
      const int b = min(b0 + (lane & 15), seen - 1);
      int64_t row = base + b;
      if (p.table != nullptr) row = p.table[at.seq * p.table_stride + b];
      bad = row < 0 || row >= p.mean_rows;
      const float* from = p.means + ((bad ? 0 : row) * p.kv_heads + hk) * D + kg * 8;
      float x[D / 32][8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        *reinterpret_cast<f32x4*>(x[i]) = *reinterpret_cast<const f32x4*>(from + i * 32);
        *reinterpret_cast<f32x4*>(x[i] + 4) = *reinterpret_cast<const f32x4*>(from + i * 32 + 4);
      }
      f32x4 acc[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (kHalf) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[i][e]));
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        const int ex = most < kInf ? __builtin_amdgcn_frexp_expf(most) : 0;
        f32x4 low[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) low[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = ldexpf(x[i][e], -ex);
          u32x4 a[2];
          split2(x[i], a);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            low[t] = T::mfma16(a[1], q[t][i], low[t]);
            acc[t] = T::mfma16(a[0], q[t][i], acc[t]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int er = __shfl(ex, 4 * kg + r);
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t][r] = ldexpf(fmaf(low[t][r], 1.f / 2048.f, acc[t][r]), er);
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          u32x4 a[3];
          split3(x[i], a);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            acc[t] = T::mfma16(a[2], q[t][i], acc[t]);
            acc[t] = T::mfma16(a[1], q[t][i], acc[t]);
            acc[t] = T::mfma16(a[0], q[t][i], acc[t]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t)
        *reinterpret_cast<f32x4*>(best + (t * 16 + (lane & 15)) * kPad + 4 * kg) = acc[t];
    }
    // lane: block b0 + (lane & 15), tokens lane >> 4, + 4, ...; with one token the
    // four lanes of a block share its heads (128 of them: 279 us -> 200 for 8192
    // tokens, 64: 93 -> 77)
    const int b = b0 + (lane & 15);
    const bool shared = tokens == 1;
    for (int tl = shared ? 0 : kg; tl < tokens; tl += 4) {
      const int n = count_of(tl);
      float s = -kInf;
      if (b < n && !bad) {
        if (b < p.first || b >= n - p.last) {
          s = kInf;
        } else {
          const float* from = best + tl * p.group * kPad + (lane & 15);
          for (int g = shared ? kg : 0; g < p.group; g += shared ? 4 : 1) {
            const float x = from[g * kPad];
            s = x > s || x != x ? x : s;
          }
        }
      }
      if (shared)
#pragma unroll
        for (int d = 16; d < 64; d <<= 1) {
          const float x = __shfl_xor(s, d);
          s = x > s || x != x ? x : s;
        }
      if (__any(s != s) && s != s) {
        const int64_t row = p.table == nullptr ? base + b : p.table[at.seq * p.table_stride + b];
        s = best_again<T, D>(p, p.means + (row * p.kv_heads + hk) * D,
                             static_cast<const char*>(p.q) + ((at.first + tl) * p.q_t + hk * p.group * p.q_h) * 2);
      }
      if (b < end && (!shared || kg == 0))
        p.scores[((at.first + tl) * p.kv_heads + hk) * static_cast<int64_t>(p.max_blocks) + b] = s * p.scale;
    }
  }
}

template <typename T, int D>
int launch_scores(const ScoreArgs& p0, bool few, hipStream_t stream) {
  ScoreArgs p = p0;
  const int64_t grid = p.slots * p.kv_heads;
  const int64_t chunks = (p.max_blocks + p.chunk - 1) / p.chunk;
  if (grid > INT32_MAX || chunks > 65535) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(chunks));
  if (few) block_scores_kernel<T, D, 1><<<g, dim3(256), 0, stream>>>(p);
  else if (p.group <= 64) block_scores_kernel<T, D, 4><<<g, dim3(256), 0, stream>>>(p);
  else block_scores_kernel<T, D, 8><<<g, dim3(256), 0, stream>>>(p);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

bool bad_block_size(int32_t bs) { return bs != 16 && bs != 32 && bs != 64 && bs != 128; }

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT int block_means(int32_t dtype, const void* k, int64_t k_stride_t, int64_t k_stride_h, int64_t total_k,
                               int32_t kv_heads, int32_t dim, int32_t block_size, const int32_t* cu_k, int32_t num_seqs,
                               float* means, hipStream_t stream) {
  if ((dtype != MI_ATTN_BF16 && dtype != MI_ATTN_FP16) || (dim != 64 && dim != 128) || bad_block_size(block_size) ||
      kv_heads < 1 || total_k < 0 || total_k > INT32_MAX || num_seqs < 0 || k_stride_t < 0 || k_stride_h < 0 ||
      ((k_stride_t | k_stride_h) & 7) || (cu_k == nullptr && num_seqs != 1) || (reinterpret_cast<uintptr_t>(k) & 15u) ||
      (reinterpret_cast<uintptr_t>(means) & 15u) || (reinterpret_cast<uintptr_t>(cu_k) & 3u))
    return MI_ATTN_EINVAL;
  MeanArgs p{k, cu_k, means, k_stride_t, k_stride_h, total_k, total_k / block_size + num_seqs, num_seqs, kv_heads, block_size};
  if (p.rows == 0) return MI_ATTN_OK;
  if (means == nullptr || (total_k > 0 && k == nullptr)) return MI_ATTN_EINVAL;
  const int64_t grid = (p.rows * kv_heads + 3) / 4;
  if (grid > INT32_MAX / 4) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid));
  if (dtype == MI_ATTN_BF16) {
    if (dim == 128) block_means_kernel<Bf16, 128><<<g, dim3(256), 0, stream>>>(p);
    else block_means_kernel<Bf16, 64><<<g, dim3(256), 0, stream>>>(p);
  } else {
    if (dim == 128) block_means_kernel<Fp16, 128><<<g, dim3(256), 0, stream>>>(p);
    else block_means_kernel<Fp16, 64><<<g, dim3(256), 0, stream>>>(p);
  }
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

MI_ATTN_EXPORT int block_scores(const mi_block_scores_args* a, hipStream_t stream) {
  if (a == nullptr) return MI_ATTN_EINVAL;
  if ((a->dtype != MI_ATTN_BF16 && a->dtype != MI_ATTN_FP16) || (a->dim != 64 && a->dim != 128) ||
      bad_block_size(a->block_size) || a->kv_heads < 1 || a->heads < a->kv_heads || a->heads % a->kv_heads ||
      a->heads / a->kv_heads > 128 || a->total_q < 0 || a->total_q > INT32_MAX || a->num_seqs < 0 || a->max_blocks < 1 ||
      a->first < 0 || a->last < 0 || !(a->scale > 0.f) || !(a->scale < kInf) || a->q_stride_t < 0 || a->q_stride_h < 0 ||
      ((a->q_stride_t | a->q_stride_h) & 7) || a->mean_rows < 0 || a->total_k < 0 || a->total_k > INT32_MAX)
    return MI_ATTN_EINVAL;
  const bool paged = a->block_table != nullptr;
  if (paged && (a->lengths == nullptr || a->block_table_stride < a->max_blocks || (a->cu_q == nullptr && a->total_q != a->num_seqs)))
    return MI_ATTN_EINVAL;
  if (!paged && ((a->cu_q == nullptr) != (a->cu_k == nullptr) || (a->cu_q == nullptr && a->num_seqs != 1))) return MI_ATTN_EINVAL;
  if (!paged && a->cu_k == nullptr && a->mean_rows < a->total_k / a->block_size + 1) return MI_ATTN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(a->q) & 15u) || (reinterpret_cast<uintptr_t>(a->means) & 15u)) return MI_ATTN_EINVAL;
  const void* words[] = {a->cu_q, a->cu_k, a->lengths, a->block_table, a->scores, a->counts};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MI_ATTN_EINVAL;
  if (a->total_q == 0) return MI_ATTN_OK;
  if (a->q == nullptr || a->scores == nullptr || a->counts == nullptr || (a->mean_rows > 0 && a->means == nullptr)) return MI_ATTN_EINVAL;
  ScoreArgs p;
  p.q = a->q; p.means = a->means; p.cu_q = a->cu_q; p.cu_k = a->cu_k; p.lengths = a->lengths; p.table = a->block_table;
  p.scores = a->scores; p.counts = a->counts; p.q_t = a->q_stride_t; p.q_h = a->q_stride_h;
  p.total_q = a->total_q; p.total_k = a->cu_k == nullptr ? a->total_k : INT32_MAX; p.mean_rows = a->mean_rows; p.table_stride = a->block_table_stride;
  p.num_seqs = a->num_seqs; p.heads = a->heads; p.kv_heads = a->kv_heads; p.group = a->heads / a->kv_heads;
  p.bs = a->block_size; p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size)); p.max_blocks = a->max_blocks; p.first = a->first; p.last = a->last; p.scale = a->scale;
  // Few rows for each sequence (a decode batch): tiles of 16 rows, and the
  // blocks are split over workgroups; many: tiles of 64 rows, or of 128 where a
  // group needs them.
  const bool few = a->total_q * p.group <= static_cast<int64_t>(a->num_seqs) * 16 && p.group <= 16;
  p.tokens_per = (few ? 16 : (p.group <= 64 ? 64 : 128)) / p.group;
  if (a->cu_q == nullptr && paged) p.tokens_per = 1;  // one query a sequence
  p.slots = slots_of(p.total_q, p.num_seqs, p.tokens_per);
  p.chunk = few ? 128 : 1024;
  if (a->dtype == MI_ATTN_BF16)
    return a->dim == 128 ? launch_scores<Bf16, 128>(p, few, stream) : launch_scores<Bf16, 64>(p, few, stream);
  return a->dim == 128 ? launch_scores<Fp16, 128>(p, few, stream) : launch_scores<Fp16, 64>(p, few, stream);
}
