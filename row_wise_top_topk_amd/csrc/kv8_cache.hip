// The 8-bit paged cache: storing new tokens.
//
//   scale = 2^ceil(log2(max|x| / 448)) of a page and head,  code = e4m3(x / scale)
//
// One workgroup per touched page, head and side (keys or values).  The page's
// new rows are read once and stay in registers between the maximum and the
// rounding; the codes that are there already are read only for the mean of the
// keys and where the scale grows.
//
// Measured: 64 single tokens of 8 heads of 128 with the mean: 11 us, which is the
// chain of its loads (lengths, table, scale and rows, mean); 2 x 8191 tokens: 26
// us, 102 MB at 3.9 TB/s, near what a copy reaches.  All 128 rows of a page in
// registers cost 65 of them; seven wavefronts a SIMD remain to cover the loads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention/mi_kv8.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

struct AppendArgs {
  const void* x[2];
  uint8_t* cache[2];
  float* scale[2];
  float* mean;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* cu;
  int64_t x_t[2], x_h[2];
  int64_t total, num_pages, table_stride;
  int32_t table_cols, num_seqs, kv_heads;
  uint32_t bs, lb;
};

// The smallest power of two that brings `most` to 448 or less: with
// most = f 2^x, 1 <= f < 2, and 448 = 1.75 * 2^8 it is 2^(x - 8), or twice
// that where f > 1.75.
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t bits = __float_as_uint(most);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < -60 ? -60 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float into_range(float x) {
  const float y = fminf(fmaxf(x, -448.f), 448.f);
  return x != x ? x : y;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(into_range(a), into_range(b), 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(into_range(c), into_range(d), w, true));
}

__device__ __forceinline__ f32x4 values4(uint32_t w) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  return f32x4{a[0], a[1], b[0], b[1]};
}

template <typename T, int D>
__global__ void __launch_bounds__(256, 4) kv8_append_kernel(AppendArgs p) {
  constexpr int kChunks = D / 8;            // 8 elements each
  constexpr int kRowsPer = 256 / kChunks;   // rows of the page in one step
  constexpr int kSteps = 128 / kRowsPer;    // of a page of 128 rows
  __shared__ float s_most[4];
  __shared__ float s_sum[4][D];
  const int side = blockIdx.x & 1;
  const uint32_t item = blockIdx.x >> 1;
  const int hk = static_cast<int>(item % p.kv_heads);
  const uint32_t slot = item / p.kv_heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  // sequence i owns the slots [cu[i] / bs + 2 i, cu[i + 1] / bs + 2 i + 2): n
  // tokens from any place of a page touch ceil(n / bs) + 1 pages at most
  int seq = 0;
  int64_t from = 0, n = 0, j = 0, len = 0;
  if (p.cu == nullptr) {
    seq = static_cast<int>(slot);
    from = slot;
    n = 1;
    len = p.lengths[seq];
  } else {
    int before = 0, last = 0;
    int32_t c = 0, next = 0, mine = 0;  // sequences whose first slot is not behind this one, 64 at a time
    for (int i0 = 0; i0 < p.num_seqs; i0 += 64) {
      const int i = i0 + lane;
      last = i0;
      c = cu_at(p.cu, p.num_seqs, p.total, i);
      next = cu_at(p.cu, p.num_seqs, p.total, i + 1);
      mine = i < p.num_seqs ? p.lengths[i] : 0;
      const bool yes = i < p.num_seqs && (static_cast<uint32_t>(c) >> p.lb) + 2u * i <= slot;
      const int some = __popcll(__ballot(yes));
      before += some;
      if (some < 64) break;
    }
    seq = __builtin_amdgcn_readfirstlane(before > 0 ? before - 1 : 0);
    if (seq >= last) {
      from = __builtin_amdgcn_readlane(c, seq - last);
      n = __builtin_amdgcn_readlane(next, seq - last) - from;
      len = __builtin_amdgcn_readlane(mine, seq - last);
    } else {  // the last of the 64 before
      from = cu_at(p.cu, p.num_seqs, p.total, seq);
      n = cu_at(p.cu, p.num_seqs, p.total, seq + 1) - from;
      len = p.lengths[seq];
    }
    j = slot - ((static_cast<uint32_t>(from) >> p.lb) + 2u * seq);
  }
  if (n <= 0) return;
  const int64_t start = len - n;
  if (len <= 0) return;
  j += (start < 0 ? 0 : start) >> p.lb;
  if ((j << p.lb) >= len || j >= p.table_cols) return;
  const int64_t page = p.table[seq * p.table_stride + j];
  if (page < 0 || page >= p.num_pages) return;
  const int64_t first = j << p.lb;
  const int held = static_cast<int>(start < first ? 0 : start - first);  // rows that were there
  const int there = static_cast<int>(len - first < p.bs ? len - first : p.bs);

  const int chunk = tid % kChunks, row0 = tid / kChunks;
  const char* x = static_cast<const char*>(p.x[side]) + ((from + first - start) * p.x_t[side] + hk * p.x_h[side] + chunk * 8) * 2;
  float* scale_at = p.scale[side] + page * p.kv_heads + hk;
  float old = *scale_at;  // read by all before the barrier, written by one behind it
  const bool wants_mean = side == 0 && p.mean != nullptr;
  uint8_t* cache = p.cache[side] + ((page * p.kv_heads + hk) * p.bs) * D + chunk * 8;
  u32x4 in[kSteps];
  float most = 0.f;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int row = row0 + s * kRowsPer;
    in[s] = u32x4{0, 0, 0, 0};
    if (row >= held && row < there) in[s] = *reinterpret_cast<const u32x4*>(x + row * p.x_t[side] * 2);
    // the mean needs the codes that are there: on their way with the new rows
    // rather than behind the barrier (11.1 us instead of 11.5 for 64 tokens)
    if (row < held && wants_mean) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(cache + row * D);
      in[s] = u32x4{w[0], w[1], 0, 0};
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (row0 + s * kRowsPer < held) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = fabsf(T::lo(in[s][e])), b = fabsf(T::hi(in[s][e]));
      most = fmaxf(most, a < kInf ? a : 0.f);
      most = fmaxf(most, b < kInf ? b : 0.f);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
  if (lane == 0) s_most[wave] = most;
  __syncthreads();
  most = fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3]));
  float scale = scale_for(most);
  if (held == 0) old = scale;
  if (!(old > 0.f && old < kInf)) old = scale_for(0.f);
  // a scale that somebody else left there is taken up to a power of two
  const uint32_t bits = __float_as_uint(old);
  scale = fmaxf(scale, __uint_as_float((bits + 0x7fffffu) & 0x7f800000u));
  const bool grows = scale > old;
  const float inv = 1.f / scale, shrink = old / scale;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int row = row0 + s * kRowsPer;
    if (row >= there) continue;
    u32x2* at = reinterpret_cast<u32x2*>(cache + row * D);
    u32x2 w;
    if (row >= held) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = T::lo(in[s][2 * h]), b = T::hi(in[s][2 * h]), c = T::lo(in[s][2 * h + 1]), d = T::hi(in[s][2 * h + 1]);
        w[h] = codes4(a * inv, b * inv, c * inv, d * inv);
      }
      *at = w;
    } else {
      if (!grows && !wants_mean) continue;
      w = wants_mean ? u32x2{in[s][0], in[s][1]} : *at;
      if (grows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 v = values4(w[h]);
          w[h] = codes4(v[0] * shrink, v[1] * shrink, v[2] * shrink, v[3] * shrink);
        }
        *at = w;
      }
    }
    if (wants_mean) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 v = values4(w[h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[4 * h + e] += v[e];
      }
    }
  }
  if (tid == 0) *scale_at = scale;
  if (!wants_mean) return;
#pragma unroll
  for (int d = kChunks; d < 64; d <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor(sum[e], d);
  if (lane < kChunks)
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[wave][chunk * 8 + e] = sum[e];
  __syncthreads();
  if (tid < D)
    p.mean[(page * p.kv_heads + hk) * D + tid] =
        (s_sum[0][tid] + s_sum[1][tid] + s_sum[2][tid] + s_sum[3][tid]) * scale / static_cast<float>(there);
}

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT int kv8_append(const mi_kv8_append_args* a, hipStream_t stream) {
  if (a == nullptr) return MI_ATTN_EINVAL;
  if ((a->dtype != MI_ATTN_BF16 && a->dtype != MI_ATTN_FP16) || (a->dim != 64 && a->dim != 128) ||
      (a->block_size != 16 && a->block_size != 32 && a->block_size != 64 && a->block_size != 128) || a->kv_heads < 1 ||
      a->total < 0 || a->total > INT32_MAX || a->num_pages < 0 || a->num_pages > INT32_MAX || a->num_seqs < 0 || a->block_table_cols < 0 ||
      a->block_table_stride < a->block_table_cols || (a->cu == nullptr && a->total != a->num_seqs))
    return MI_ATTN_EINVAL;
  const int64_t strides[] = {a->k_stride_t, a->k_stride_h, a->v_stride_t, a->v_stride_h};
  for (int64_t s : strides)
    if (s < 0 || (s & 7)) return MI_ATTN_EINVAL;
  if ((reinterpret_cast<uintptr_t>(a->k) | reinterpret_cast<uintptr_t>(a->v) | reinterpret_cast<uintptr_t>(a->k_cache) |
       reinterpret_cast<uintptr_t>(a->v_cache)) & 15u)
    return MI_ATTN_EINVAL;
  const void* words[] = {a->k_scale, a->v_scale, a->k_mean, a->block_table, a->lengths, a->cu};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MI_ATTN_EINVAL;
  if (a->total == 0 || a->num_pages == 0 || a->block_table_cols == 0 || a->num_seqs == 0) return MI_ATTN_OK;
  if (a->k == nullptr || a->v == nullptr || a->k_cache == nullptr || a->v_cache == nullptr || a->k_scale == nullptr ||
      a->v_scale == nullptr || a->block_table == nullptr || a->lengths == nullptr)
    return MI_ATTN_EINVAL;
  AppendArgs p;
  p.x[0] = a->k; p.x[1] = a->v;
  p.cache[0] = static_cast<uint8_t*>(a->k_cache); p.cache[1] = static_cast<uint8_t*>(a->v_cache);
  p.scale[0] = a->k_scale; p.scale[1] = a->v_scale; p.mean = a->k_mean;
  p.table = a->block_table; p.lengths = a->lengths; p.cu = a->cu;
  p.x_t[0] = a->k_stride_t; p.x_h[0] = a->k_stride_h; p.x_t[1] = a->v_stride_t; p.x_h[1] = a->v_stride_h;
  p.total = a->total; p.num_pages = a->num_pages; p.table_stride = a->block_table_stride; p.table_cols = a->block_table_cols;
  p.num_seqs = a->num_seqs; p.kv_heads = a->kv_heads; p.bs = a->block_size;
  p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size));
  const int64_t slots = a->cu == nullptr ? a->num_seqs : a->total / a->block_size + 2 * static_cast<int64_t>(a->num_seqs);
  const int64_t grid = slots * a->kv_heads * 2;
  if (grid > INT32_MAX) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid));
  if (a->dtype == MI_ATTN_BF16) {
    if (a->dim == 128) kv8_append_kernel<Bf16, 128><<<g, dim3(256), 0, stream>>>(p);
    else kv8_append_kernel<Bf16, 64><<<g, dim3(256), 0, stream>>>(p);
  } else {
    if (a->dim == 128) kv8_append_kernel<Fp16, 128><<<g, dim3(256), 0, stream>>>(p);
    else kv8_append_kernel<Fp16, 64><<<g, dim3(256), 0, stream>>>(p);
  }
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}
