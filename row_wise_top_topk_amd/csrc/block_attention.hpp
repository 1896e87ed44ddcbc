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
  void* rest;
  float* lse;
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, do_t, do_h;
  int64_t total_q, total_k, slots;
  int32_t num_seqs, heads, kv_heads, group, bs, lb, select, causal, tokens_per;
  uint32_t select_magic;  // n / select = n * select_magic >> 32 for the entries of a workgroup, select above 1
  float scale;
};

int make_args(const mi_block_attention_args* a, Args& p);

// Few rows: 64 of them a workgroup instead of 128 are better where the card's 256
// compute units would get one workgroup each, or a little more.  There are twice
// as many, the union of their blocks is smaller and two wavefronts share a tile's
// keys; but each key is copied more often, the less neighbouring tokens differ
// (many heads a group: few tokens) the more in vain.  Measured, 128 rows against
// 64, with n workgroups of 128 (us): 8 heads a group, 128 columns: n 128: 29, 26;
// 256: 52, 47; 376: 75, 69; 4 heads, 752: 189, 231; one head, 376: 141, 122; 512:
// 200, 221.  64 columns, 4 heads: 256: 75, 53; 540: 70, 62; 750: 154, 151.  16
// heads: 188: 43, 44; 256: 61, 73.  The cuts lie where the two come within 3 % of
// each other, so next to them (64 columns at 750, 16 heads at 188) the other side
// can be ahead by that.
inline bool split_rows(Args& p, int dim) {
  const int64_t most = p.group > 8 ? 192 : (dim == 64 ? 640 : 384);
  if (p.slots * p.kv_heads > most || p.group > 64) return false;
  p.tokens_per = 64 / p.group;
  p.slots = slots_of(p.total_q, p.num_seqs, p.tokens_per);
  return true;
}

constexpr int kRows = 128;        // rows of a workgroup: 32 for each of four wavefronts
constexpr int kThreads = 256;
constexpr int kTile = 64;         // keys of a tile
constexpr int kMaskWords = 2048;  // words of token bits, window of block numbers x words per block

struct Select {
  uint32_t mask[kMaskWords];
  uint16_t list[kMaskWords];
  uint32_t wave_count[kThreads / 64];
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
  int32_t k0, k1;
  const Place at = place_of(p.cu_q, p.num_seqs, p.total_q, slot, tq, [&](int i) { return cu_at(p.cu_k, p.num_seqs, p.total_k, i); }, k0, k1);
  Group g;
  g.t0 = at.first;
  g.begin = at.begin;
  const int64_t left = at.end - at.first;
  g.tokens = static_cast<int32_t>(left < 0 ? 0 : (left < tq ? left : tq));
  g.tk0 = 0;
  g.row0 = 0;
  g.len_k = 0;
  if (at.seq < p.num_seqs) {
    g.tk0 = k0;
    g.len_k = k1 < k0 ? 0 : k1 - k0;
    g.row0 = (k0 >> p.lb) + at.seq;
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
  constexpr int kWaves = kThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int most = min(width, g.blocks - w0);
  const int32_t* rows = p.blocks + (g.t0 * p.kv_heads + hk) * static_cast<int64_t>(p.select);
  const int64_t stride = static_cast<int64_t>(p.kv_heads) * p.select;
  const int total = g.tokens * p.select;
  // entry i belongs to token i / select; the first of a thread's entries is on
  // its way while the words are cleared
  auto entry = [&](int i, int& tl) {
    tl = static_cast<int>(__umulhi(static_cast<uint32_t>(i), p.select_magic));
    if (p.select == 1) tl = i;
    return rows[tl * stride + (i - tl * p.select)] - w0;
  };
  int tl = 0, b = tid < total ? entry(tid, tl) : -1;
  __syncthreads();
  for (int i = tid; i < most * nw; i += kThreads) s.mask[i] = 0;
  __syncthreads();
  for (int i = tid; i < total; i += kThreads) {
    if (i != tid) b = entry(i, tl);
    if (b >= 0 && b < most) atomicOr(&s.mask[b * nw + (tl >> 5)], 1u << (tl & 31));
  }
  __syncthreads();
  // a wavefront lists a quarter of the window, 64 blocks at a time: counts
  // first, then the places
  const int share = ((most + 64 * kWaves - 1) / (64 * kWaves)) * 64;
  const int from = min(most, wave * share), to = min(most, from + share);
  auto taken = [&](int i) {
    uint32_t any = 0;
    if (i < to)
      for (int w = 0; w < nw; ++w) any |= s.mask[i * nw + w];
    return __ballot(any != 0);
  };
  int mine = 0;
  for (int i = from; i < to; i += 64) mine += __popcll(taken(i + lane));
  if (lane == 0) s.wave_count[wave] = mine;
  __syncthreads();
  int at = 0, count = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int n = s.wave_count[w];
    if (w < wave) at += n;
    count += n;
  }
  for (int i = from; i < to; i += 64) {
    const uint64_t has = taken(i + lane);
    if ((has >> lane) & 1) s.list[at + __popcll(has & ((1ull << lane) - 1))] = static_cast<uint16_t>(i + lane);
    at += __popcll(has);
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(count);
}

// The four 16-key groups of a tile: first key of each in its sequence, or -1.
// Wide: blocks of 64 keys or more, so that all four are of one block.
template <bool kWide>
struct Keys {
  static constexpr int kIds = kWide ? 1 : 4;
  int32_t key[4];
  int32_t id[kIds];  // place of the block in the window
};

template <bool kWide>
__device__ __forceinline__ Keys<kWide> keys_of(const Select& s, int lb, int bs, int w0, int active, int tile) {
  Keys<kWide> k;
  if constexpr (kWide) {
    const int a = tile * kTile;
    k.id[0] = __builtin_amdgcn_readfirstlane(s.list[min(a >> lb, active - 1)]);
    const int key = ((w0 + k.id[0]) << lb) + (a & (bs - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) k.key[i] = key + 16 * i;
  } else {
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = s.list[min((tile * kTile + 16 * i) >> lb, active - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = tile * kTile + 16 * i;
      k.id[i] = __builtin_amdgcn_readfirstlane(id[i]);
      k.key[i] = (a >> lb) < active ? ((w0 + k.id[i]) << lb) + (a & (bs - 1)) : -1;
    }
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
  template <bool kWide>
  __device__ __forceinline__ void load(const char* base, int64_t stride_bytes, const Keys<kWide>& k, int len_k) {
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

  // for a wavefront that takes the 32 keys from 32 * part on only
  __device__ __forceinline__ void from(int part) {
    last[0] = part != 0 ? last[2] : last[0];
    last[1] = part != 0 ? last[3] : last[1];
  }
};

template <bool kWide>
__device__ __forceinline__ Sight sight_of(const Select& s, const Keys<kWide>& k, int nw, int word, int bit, int limit, bool valid) {
  Sight v;
  if constexpr (kWide) {
    const uint32_t bits = s.mask[k.id[0] * nw + word];
    const int last = (bits >> bit) & 1u ? limit - k.key[0] : -64;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.last[i] = last - 16 * i;
    v.any = __any(valid && last >= 0);
    v.partial = __any(valid && last >= 0 && last < 63);
  } else {
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
  }
  return v;
}

// Whether a row sees group i, where what it sees a part of has been masked: with
// one block the first group stands for all.
template <bool kWide>
__device__ __forceinline__ bool sees(const Sight& v, int i) { return v.last[kWide ? 0 : i] >= 0; }

// Where a lane reads a tile in LDS.  By rows: row lane & 31 of 32, 8 elements
// from 16 i + 8 (lane >> 5) on.  Transposed: rows 4 (lane >> 5) .. + 3 (x) and
// those 8 behind them (y) of 16, column 32 i + (lane & 31); the rows are the
// order in which the scores of 32 keys lie in a lane's registers.
// The addresses are those of a tile at `base`; other tiles and rows are constants
// away, which the instructions add.
template <int D>
struct Reads {
  uint32_t r[D / 16], x[D / 32], y[D / 32];
  __device__ __forceinline__ explicit Reads(uint32_t base) {
    const uint32_t lane = threadIdx.x & 63, half = lane >> 5, li = lane & 15, dhalf = (lane >> 4) & 1;
    const uint32_t row = 4 * half + (li >> 2), chunk = dhalf * 2 + ((li & 3) >> 1);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) r[i] = keep(base + (tile_at<D>(lane & 31, half) ^ (i * 32)));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[i] = keep(base + ((tile_at<D>(row, chunk) + (li & 1) * 8) ^ (i * 64)));
      y[i] = keep(base + ((tile_at<D>(row + 8, chunk) + (li & 1) * 8) ^ (i * 64)));
    }
  }
  static __device__ __forceinline__ uint32_t keep(uint32_t v) {  // in a register, not worked out again
    asm volatile("" : "+v"(v));
    return v;
  }
  // operand i of the 32 rows from `rows` on (a multiple of 32) of the tile `at` bytes on
  __device__ __forceinline__ u32x4 row(int at, int rows, int i) const { return lds_read16(r[i] + (at + rows * 2 * D)); }
  // operand of the 16 rows from `rows` on (a multiple of 16), columns 32 i ..
  __device__ __forceinline__ u32x4 column(int at, int rows, int i) const {
    const u32x2 a = lds_read_tr16(x[i] + (at + rows * 2 * D)), b = lds_read_tr16(y[i] + (at + rows * 2 * D));
    return u32x4{a[0], a[1], b[0], b[1]};
  }
};

}  // namespace miattn
