// What the forward and the backward of the block sparse attention share: the
// arguments, and the walk of a workgroup's rows over the blocks they select.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"

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

constexpr int kRows = 128;        // rows of a workgroup
constexpr int kTile = 64;         // keys of a tile
constexpr int kMaskWords = 2048;  // words of token bits, window of block numbers x words per block

struct Select {
  uint32_t mask[kMaskWords];
  uint16_t list[kMaskWords];
  uint32_t wave_count[4];
};

// The tokens of one workgroup and how its rows map to them.
struct Group {
  int64_t t0, begin, tk0;  // first token; the sequence's first token and first key
  int64_t row0;            // number of its first block among the packed ones
  int32_t tokens;          // tokens of this workgroup
  int32_t len_k;
  int32_t shift;           // position of token t: t - begin + shift
  int32_t blocks;          // blocks that any of its rows can see
};

__device__ __forceinline__ Group group_of(const Args& p, int64_t slot, int tq) {
  const Place at = place_of(p.cu_q, p.num_seqs, p.total_q, slot, tq);
  Group g;
  g.t0 = at.first;
  g.begin = at.begin;
  const int64_t left = at.end - at.first;
  g.tokens = static_cast<int32_t>(left < 0 ? 0 : (left < tq ? left : tq));
  g.tk0 = 0;
  g.row0 = 0;
  g.len_k = 0;
  if (at.seq < p.num_seqs) {
    g.tk0 = cu_at(p.cu_k, p.num_seqs, p.total_k, at.seq);
    const int64_t n = cu_at(p.cu_k, p.num_seqs, p.total_k, at.seq + 1) - g.tk0;
    g.len_k = static_cast<int32_t>(n < 0 ? 0 : n);
    g.row0 = g.tk0 / p.bs + at.seq;
  }
  g.shift = g.len_k - static_cast<int32_t>(at.end - at.begin);
  int64_t seen = g.len_k;
  if (p.causal) {
    const int64_t last = at.first - at.begin + g.tokens - 1 + g.shift;
    if (last + 1 < seen) seen = last + 1 < 0 ? 0 : last + 1;
  }
  g.blocks = g.tokens > 0 ? static_cast<int32_t>((seen + p.bs - 1) >> p.lb) : 0;
  return g;
}

// Marks which tokens select each block of [w0, w0 + width) and lists the blocks
// that any does, ascending.  Returns their number.  Ends with a barrier.
__device__ __forceinline__ int list_window(const Args& p, const Group& g, int hk, int w0, int width, int nw, Select& s) {
  const int tid = threadIdx.x;
  __syncthreads();
  for (int i = tid; i < width * nw; i += 256) s.mask[i] = 0;
  __syncthreads();
  const int most = min(width, g.blocks - w0);
  const int32_t* rows = p.blocks + (g.t0 * p.kv_heads + hk) * static_cast<int64_t>(p.select);
  const int64_t stride = static_cast<int64_t>(p.kv_heads) * p.select;
  const int total = g.tokens * p.select;
  for (int i = tid; i < total; i += 256) {
    const int tl = i / p.select;
    const int b = rows[tl * stride + (i - tl * p.select)] - w0;
    if (b >= 0 && b < most) atomicOr(&s.mask[b * nw + (tl >> 5)], 1u << (tl & 31));
  }
  __syncthreads();
  // every thread has width / 256 consecutive blocks; counts are summed over
  // the lanes, then over the wavefronts
  const int each = (width + 255) >> 8;
  int mine = 0;
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    uint32_t any = 0;
    if (b < most)
      for (int w = 0; w < nw; ++w) any |= s.mask[b * nw + w];
    mine += any != 0;
  }
  int sum = mine;
  const int lane = tid & 63, wave = tid >> 6;
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 63) s.wave_count[wave] = sum;
  __syncthreads();
  int at = sum - mine;
  int count = 0;
  for (int w = 0; w < 4; ++w) {
    const int c = s.wave_count[w];
    if (w < wave) at += c;
    count += c;
  }
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    uint32_t any = 0;
    if (b < most)
      for (int w = 0; w < nw; ++w) any |= s.mask[b * nw + w];
    if (any != 0) s.list[at++] = static_cast<uint16_t>(b);
  }
  __syncthreads();
  return count;
}

// The four 16-key groups of a tile: first key of each in its sequence, or -1.
struct Keys {
  int32_t key[4];
  int32_t id[4];  // place of the block in the window
};

__device__ __forceinline__ Keys keys_of(const Select& s, int lb, int bs, int w0, int active, int tile) {
  Keys k;
  int id[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) id[i] = s.list[min((tile * kTile + 16 * i) >> lb, active - 1)];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = tile * kTile + 16 * i;
    k.id[i] = __builtin_amdgcn_readfirstlane(id[i]);
    k.key[i] = (a >> lb) < active ? ((w0 + k.id[i]) << lb) + (a & (bs - 1)) : -1;
  }
  return k;
}

// Half of a tile on its way from memory to LDS: 64 rows of D elements over 256
// threads, held in registers while the tile before it is worked on.
template <int D>
struct Half {
  static constexpr int kLanes = D / 8;           // threads of a row
  static constexpr int kRowsAt = 256 / kLanes;   // rows of one step
  static constexpr int kSteps = kTile / kRowsAt;
  u32x4 x[kSteps];

  // base + key * stride of a 16-key group is uniform; a thread adds its row and
  // chunk in 32 bits.  Rows behind the sequence's last key repeat it.
  __device__ __forceinline__ void load(const char* base, int64_t stride_bytes, const Keys& k, int len_k) {
    const int tid = threadIdx.x;
    const uint32_t chunk = (tid % kLanes) * 16;
    const int row = (tid / kLanes) & 15;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      int key;
      if constexpr (kRowsAt == 16) key = k.key[j];
      else key = __builtin_amdgcn_readfirstlane(tid) < 128 ? k.key[2 * j] : k.key[2 * j + 1];
      key = max(0, min(key, len_k - 1));  // a group may lie behind the last key of its block
      const char* from = base + key * stride_bytes;
      x[j] = *reinterpret_cast<const u32x4*>(from + (__umul24(min(row, len_k - 1 - key), static_cast<uint32_t>(stride_bytes)) + chunk));
    }
  }
  __device__ __forceinline__ void store(char* tile) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const uint32_t row = j * kRowsAt + tid / kLanes;
      *reinterpret_cast<u32x4*>(tile + tile_at<D>(row, tid % kLanes)) = x[j];
    }
  }
};

// Tells the scheduler to keep `ahead` products' operand reads (`reads`
// instructions each) before the product that uses them, for `products` in a row.
template <int products, int ahead, int reads>
__device__ __forceinline__ void read_ahead() {
  constexpr int first = ahead < products ? ahead : products;
  __builtin_amdgcn_sched_group_barrier(0x100, first * reads, 0);
#pragma unroll
  for (int i = 0; i < products - first; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, first, 0);
}

// What a lane's row may see of a tile: for each 16-key group the last visible
// offset (relative to the group's first key), negative for none.
struct Sight {
  int32_t last[4];
  bool any;      // some row of the wavefront sees something
  bool partial;  // some row sees a part of a group only
};

__device__ __forceinline__ Sight sight_of(const Select& s, const Keys& k, int nw, int word, int bit, int limit, bool valid) {
  Sight v;
  bool some = false, part = false;
  uint32_t bits[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) bits[i] = s.mask[k.id[i] * nw + word];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.last[i] = k.key[i] >= 0 && ((bits[i] >> bit) & 1u) ? limit - k.key[i] : -1;
    some |= v.last[i] >= 0;
    part |= v.last[i] >= 0 && v.last[i] < 15;
  }
  v.any = __any(valid && some);
  v.partial = __any(valid && part);
  return v;
}

// Where a lane reads a tile in LDS.  By rows: row lane & 31 of 32, 8 elements
// from 16 i + 8 (lane >> 5) on.  Transposed: rows 4 (lane >> 5) .. + 3 (x) and
// those 8 behind them (y) of 16, column 32 i + (lane & 31); the rows are the
// order in which the scores of 32 keys lie in a lane's registers.
template <int D>
struct Reads {
  uint32_t by_row, x, y;
  __device__ __forceinline__ Reads() {
    const uint32_t lane = threadIdx.x & 63, half = lane >> 5, li = lane & 15, dhalf = (lane >> 4) & 1;
    by_row = tile_at<D>(lane & 31, half);
    const uint32_t row = 4 * half + (li >> 2), chunk = dhalf * 2 + ((li & 3) >> 1);
    x = tile_at<D>(row, chunk) + (li & 1) * 8;
    y = tile_at<D>(row + 8, chunk) + (li & 1) * 8;
  }
  // operand i of the 32 rows from `rows` on (a multiple of 32)
  __device__ __forceinline__ u32x4 row(uint32_t tile, int rows, int i) const { return lds_read16((tile + (by_row ^ (i * 32))) + rows * (2 * D)); }
  // operand of the 16 rows from `rows` on (a multiple of 16), columns 32 i ..
  __device__ __forceinline__ u32x4 column(uint32_t tile, int rows, int i) const {
    const u32x2 a = lds_read_tr16((tile + (x ^ (i * 64))) + rows * (2 * D)), b = lds_read_tr16((tile + (y ^ (i * 64))) + rows * (2 * D));
    return u32x4{a[0], a[1], b[0], b[1]};
  }
};

}  // namespace miattn
