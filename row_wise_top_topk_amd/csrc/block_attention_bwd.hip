// The gradient of block sparse attention.
//
//   p_j = exp(scale q.k_j - lse),  delta = dout . out,  ds_j = p_j (dout.v_j - delta)
//   dq = scale sum_j ds_j k_j,  dk_j = scale sum_q ds_j q,  dv_j = sum_q p_j dout
//
// The ds_j of a row add up to 0, so what keys have in common cancels in dq and
// roundings show: there ds is multiplied as two 16-bit terms, and delta takes
// out with what its rounding left out.  dk and dv round p and ds once.
//
// dq goes over the rows as the forward does.  dk and dv go over the key blocks:
// a bit matrix [key head][block][token] says which tokens selected a block
// (atomic OR and integer counts: nothing depends on their order), a block's tokens
// are cut into pieces of equal length, and a workgroup takes one piece: the
// sink and the own blocks, which every token selects, become many pieces.  A
// block of one piece is written at once; the others' pieces are summed in order
// by a last kernel, so the result is the same from run to run.
//
// Measured on 8192 tokens, 32/2 heads of 128, 16 blocks of 64: dq 510 to 540 us,
// dk and dv 400 to 425 us, the sums of pieces 27 us, the bits and pieces 10 us.
// The matrix units are busy for 27 % (dq) and 25 % (dk, dv): dq is bound as the
// forward is, by the union of its tokens' blocks and a tile's chain with two
// wavefronts a SIMD; dk and dv by LDS,
// whose reads (each row twice, by rows and transposed, for every 16 keys) take
// nine tenths of the time.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

constexpr int kPieceRows = 2048;  // rows (tokens x heads of a group) of a piece

struct BackArgs {
  Args a;
  float* delta;        // [total_q, heads]
  uint32_t* bits;      // [kv_heads][rows][words]
  int32_t* first;      // [kv_heads * rows + 1]: first piece of each block
  int32_t* counts;     // [kv_heads * rows]: tokens of each block
  int32_t* owner;      // [piece]: its block
  float* part;         // [piece][2][bs][D]
  int64_t rows;        // blocks of all sequences, and those of the keys behind them
  int64_t words;
  int32_t piece;       // tokens of a piece
  int32_t max_pieces;
  uint32_t group_magic;  // n / group = n * group_magic >> 32 for n below 2^24, group above 1
};

// Which tokens of the workgroup selected each listed block, into the bit matrix
// and the blocks' counts: tokens t0 .. t0 + 31 of mask word w lie in two words of a
// block's row.
__device__ __forceinline__ void mark_tokens(const BackArgs& b, const Group& g, int hk, int w0, int active, int nw, const Select& s) {
  for (int i = threadIdx.x; i < active * nw; i += 256) {
    const int id = s.list[i / nw], w = i % nw;
    const uint32_t x = s.mask[id * nw + w];
    if (x == 0) continue;
    const int64_t t = g.t0 + 32 * w;
    const int64_t entry = hk * b.rows + g.row0 + w0 + id;
    uint32_t* to = b.bits + entry * b.words + (t >> 5);
    const int up = static_cast<int>(t & 31);
    if (x << up) atomicOr(to, x << up);
    if (up > 0 && (x >> (32 - up))) atomicOr(to + 1, x >> (32 - up));
    atomicAdd(b.counts + entry, __popc(x));
  }
}

// ---- dq ----

template <typename T, int D>
struct QShared {
  char k[2][kTile * 2 * D];
  char v[2][kTile * 2 * D];
  Select sel;
};

// kSplit as in the forward: two wavefronts share 32 rows and take 32 keys of a tile each
template <typename T, int D, bool kWide, bool kSplit>
__global__ void __launch_bounds__(256, 2) block_attention_dq_kernel(BackArgs b) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  QShared<T, D>& sh = *reinterpret_cast<QShared<T, D>*>(smem);
  const Args& p = b.a;
  const int hk = blockIdx.x % p.kv_heads;
  const int64_t slot = p.slots - 1 - static_cast<int64_t>(blockIdx.x / p.kv_heads);
  const int tq = p.tokens_per;
  const Group g = group_of(p, slot, tq);
  if (g.tokens == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5;
  const int rows32 = kSplit ? wave & 1 : wave, keys32 = kSplit ? wave >> 1 : 0;
  const bool last = keys32 == 0;  // this wavefront stores its rows' results
  const int row = rows32 * 32 + (lane & 31);
  const int tl = row / p.group, head = hk * p.group + row % p.group;
  const bool valid = tl < g.tokens;
  const int64_t tok = g.t0 + (valid ? tl : 0);
  int limit = -1;
  if (valid) {
    const int64_t pos = tok - g.begin + g.shift;
    limit = p.causal ? static_cast<int>(pos < g.len_k ? pos : g.len_k - 1) : g.len_k - 1;
  }
  u32x4 q[D / 16], go[D / 16];
  float delta = 0.f, lse2 = kInf;
  {
    const char* from = static_cast<const char*>(p.q) + (tok * p.q_t + head * p.q_h) * 2 + half * 16;
    const char* gfrom = static_cast<const char*>(p.dout) + (tok * p.do_t + head * p.do_h) * 2 + half * 16;
    const int64_t o_at = (tok * p.heads + head) * (2 * D) + half * 16;
    const char* ofrom = static_cast<const char*>(p.out) + o_at;
    const char* rfrom = p.rest == nullptr ? nullptr : static_cast<const char*>(p.rest) + o_at;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      q[i] = go[i] = u32x4{0, 0, 0, 0};
      if (valid) {
        q[i] = *reinterpret_cast<const u32x4*>(from + i * 32);
        go[i] = *reinterpret_cast<const u32x4*>(gfrom + i * 32);
        const u32x4 o = *reinterpret_cast<const u32x4*>(ofrom + i * 32);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          delta = fmaf(T::lo(go[i][e]), T::lo(o[e]), delta);
          delta = fmaf(T::hi(go[i][e]), T::hi(o[e]), delta);
        }
        if (rfrom != nullptr) {
          const u32x4 z = *reinterpret_cast<const u32x4*>(rfrom + i * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            delta = fmaf(T::lo(go[i][e]), T::lo(z[e]), delta);
            delta = fmaf(T::hi(go[i][e]), T::hi(z[e]), delta);
          }
        }
      }
    }
    delta = half_sum(delta);
    if (valid) {
      const float l = p.lse[tok * p.heads + head];
      lse2 = l == -kInf ? kInf : l * kLog2e;
      if (half == 0 && last) b.delta[tok * p.heads + head] = delta;
    }
  }
  const char* kbase = static_cast<const char*>(p.k) + (g.tk0 * p.k_t + hk * p.k_h) * 2;
  const char* vbase = static_cast<const char*>(p.v) + (g.tk0 * p.v_t + hk * p.v_h) * 2;
  f32x16 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  const float c = p.scale * kLog2e;
  const int nw = (tq + 31) >> 5;
  const int width = kMaskWords / nw;
  const Reads<D> rd(lds_offset(sh.k[0]) + keys32 * (64 * D));
  constexpr int kBuf = kTile * 2 * D;  // from one buffer to the other; the values lie two behind the keys

  for (int w0 = 0; w0 < g.blocks; w0 += width) {
    const int active = list_window(p, g, hk, w0, width, nw, sh.sel);
    mark_tokens(b, g, hk, w0, active, nw, sh.sel);
    const int tiles = ((active << p.lb) + kTile - 1) / kTile;
    if (tiles == 0) continue;
    // Keys of the tile in LDS, of the one on its way and of the one behind it;
    // what a row sees of a tile is worked out one tile ahead.
    Keys<kWide> next = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, 0);
    Half<D> kin, vin;
    kin.load(kbase, p.k_t * 2, next, g.len_k);
    vin.load(vbase, p.v_t * 2, next, g.len_k);
    const int word = tl >> 5 < nw ? tl >> 5 : 0;
    auto sight = [&](const Keys<kWide>& k) {
      Sight v = sight_of(sh.sel, k, nw, word, tl & 31, limit, valid);
      if constexpr (kSplit) v.from(keys32);
      return v;
    };
    Sight ahead = sight(next);
    next = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, 1);
    auto step = [&](auto which, int tile) {
      constexpr int buf = decltype(which)::value;
      kin.store(sh.k[buf]);
      vin.store(sh.v[buf]);
      __syncthreads();
      const Sight see = ahead;
      if (tile + 1 < tiles) {
        kin.load(kbase, p.k_t * 2, next, g.len_k);
        vin.load(vbase, p.v_t * 2, next, g.len_k);
        ahead = sight(next);
        next = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, tile + 2);
      }
      if (!see.any) return;
#pragma unroll
      for (int mt = 0; mt < (kSplit ? 1 : 2); ++mt) {
        f32x16 s, dp;
        {
          u32x4 ka[D / 16], va[D / 16];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) ka[i] = rd.row(buf * kBuf, mt * 32, i);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) va[i] = rd.row((2 + buf) * kBuf, mt * 32, i);
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) s = T::mfma32(ka[i], q[i], s);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) dp = T::mfma32(va[i], go[i], dp);
          // four reads ahead of the products
          __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
          for (int i = 0; i < D / 8 - 4; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
          __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
        }
        u32x4 ds[2], low[2];
        if (see.partial) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (8 * ((r >> 2) & 1) + (r & 3) + 4 * half > see.last[2 * mt + (r >> 3)]) s[r] = -kInf;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float from = sees<kWide>(see, 2 * mt + i) ? lse2 : kInf;
#pragma unroll
          for (int r = 0; r < 8; r += 2) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) w[e] = exp2_fast(fmaf(s[8 * i + r + e], c, -from)) * (dp[8 * i + r + e] - delta);
            ds[i][r >> 1] = T::pack(w[0], w[1]);
            low[i][r >> 1] = T::pack(w[0] - T::lo(ds[i][r >> 1]), w[1] - T::hi(ds[i][r >> 1]));
          }
        }
        {
          u32x4 ka[D / 32][2];
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int st = 0; st < 2; ++st) ka[i][st] = rd.column(buf * kBuf, mt * 32 + 16 * st, i);
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              acc[i] = T::mfma32(ka[i][st], ds[st], acc[i]);
              acc[i] = T::mfma32(ka[i][st], low[st], acc[i]);
            }
          __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
          for (int i = 0; i < D / 16 - 4; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          }
          __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
        }
      }
    };
    for (int tile = 0; tile < tiles; tile += 2) {
      step(Int<0>{}, tile);
      if (tile + 1 < tiles) step(Int<1>{}, tile + 1);
    }
  }
  if constexpr (kSplit) {
    __syncthreads();
    float* box = reinterpret_cast<float*>(smem) + rows32 * 64 + lane;
    if (!last)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) box[(i * 16 + r) * 128] = acc[i][r];
    __syncthreads();
    if (last)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] += box[(i * 16 + r) * 128];
  }
  // as in the forward: what a row does not see must not reach it as 0 times an
  // infinity or NaN
  bool odd = false;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd |= !(fabsf(acc[i][r]) < kInf);
  if (__syncthreads_or(valid && last && odd)) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    for (int w0 = 0; w0 < g.blocks; w0 += width) {
      const int active = list_window(p, g, hk, w0, width, nw, sh.sel);
      const int word = tl >> 5 < nw ? tl >> 5 : 0;
      for (int e = 0; e < active; ++e) {
        const int id = __builtin_amdgcn_readfirstlane(sh.sel.list[e]);
        const bool mine = valid && ((sh.sel.mask[id * nw + word] >> (tl & 31)) & 1u);
        if (!__any(mine)) continue;
        const int from = (w0 + id) << p.lb, to = min(from + p.bs, g.len_k);
        for (int key = from; key < to; ++key) {
          const char* kr = kbase + key * (p.k_t * 2);
          const char* vr = vbase + key * (p.v_t * 2);
          float x = 0.f, y = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const u32x4 kv = *reinterpret_cast<const u32x4*>(kr + half * 16 + i * 32), vv = *reinterpret_cast<const u32x4*>(vr + half * 16 + i * 32);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              x = fmaf(T::hi(kv[z]), T::hi(q[i][z]), fmaf(T::lo(kv[z]), T::lo(q[i][z]), x));
              y = fmaf(T::hi(vv[z]), T::hi(go[i][z]), fmaf(T::lo(vv[z]), T::lo(go[i][z]), y));
            }
          }
          x = half_sum(x);
          y = half_sum(y);
          if (mine && key <= limit) {
            const float w = exp2_fast(fmaf(x, c, -lse2)) * (y - delta);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
              for (int r = 0; r < 16; r += 4) {
                const u32x2 kv = *reinterpret_cast<const u32x2*>(kr + half * 8 + i * 64 + (r >> 2) * 16);
                acc[i][r] = fmaf(w, T::lo(kv[0]), acc[i][r]);
                acc[i][r + 1] = fmaf(w, T::hi(kv[0]), acc[i][r + 1]);
                acc[i][r + 2] = fmaf(w, T::lo(kv[1]), acc[i][r + 2]);
                acc[i][r + 3] = fmaf(w, T::hi(kv[1]), acc[i][r + 3]);
              }
          }
        }
      }
    }
  }
  if (!valid || !last) return;
  char* to = static_cast<char*>(p.dq) + (tok * p.heads + head) * (2 * D) + half * 8;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      u32x2 w;
      w[0] = T::pack(acc[i][r] * p.scale, acc[i][r + 1] * p.scale);
      w[1] = T::pack(acc[i][r + 2] * p.scale, acc[i][r + 3] * p.scale);
      *reinterpret_cast<u32x2*>(to + i * 64 + (r >> 2) * 16) = w;
    }
}

// ---- the pieces of each block's tokens ----

__global__ void __launch_bounds__(256) clear_bits_kernel(BackArgs b) {
  const int64_t entries = b.a.kv_heads * b.rows, total = entries * b.words, step = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t i = first; i < total; i += step) b.bits[i] = 0;
  for (int64_t i = first; i < entries; i += step) b.counts[i] = 0;
}

// Pieces of each block (one at least, for the zeros of a block that nobody
// selected), their running number and whose they are; one workgroup.
__global__ void __launch_bounds__(1024) number_pieces_kernel(BackArgs b) {
  __shared__ int32_t s_wave[16];
  __shared__ int32_t s_base;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t total = b.a.kv_heads * b.rows;
  if (tid == 0) s_base = 0;
  __syncthreads();
  for (int64_t i0 = 0; i0 < total; i0 += 1024) {
    const int64_t e = i0 + tid;
    int n = 0;
    if (e < total) n = max(1, (b.counts[e] + b.piece - 1) / b.piece);
    int sum = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 63) s_wave[wave] = sum;
    __syncthreads();
    int at = s_base + sum - n;
    for (int w = 0; w < wave; ++w) at += s_wave[w];
    if (e < total) b.first[e] = at;
    for (int i = 0; i < n; ++i) b.owner[at + i] = static_cast<int32_t>(e);
    __syncthreads();
    if (tid == 1023) s_base = at + n;
    __syncthreads();
  }
  if (tid == 0) b.first[total] = s_base;
}

// ---- dk, dv ----

// Rows of a stage for each group of wavefronts that shares them: the more, the
// more of the loads' time is covered (8192 tokens, 32/2 heads of 128, 16 blocks of
// 64: 64 rows 410 us, 32 rows 600).
template <int KW>
constexpr int kStage = KW == 4 ? 64 : 32;

template <int D, int KW>
struct KvShared {
  static constexpr int kRowsAt = kStage<KW> * (4 / KW);  // rows staged at a time
  union {
    struct {
      char q[2][kRowsAt * 2 * D];
      char go[2][kRowsAt * 2 * D];
    };
    float join[4][16][D + 4];
  };
  float lse2[2][kRowsAt], delta[2][kRowsAt];
  int32_t pos[2][kRowsAt];
  int32_t list[kPieceRows];
  int32_t wave_count[4];
};

// KW wavefronts of 16 keys; 4 / KW of them share the keys and take different
// rows; a block of 128 keys is two workgroups'.  The keys and values stay in
// registers as operands, the rows' queries and output gradients are staged in
// LDS (the next ones wait in registers meanwhile) and read by rows for the
// scores, transposed for the gradients.  16 keys rather than 32 a wavefront:
// with 32 the accumulators leave one wavefront a SIMD, and its waits show
// (measured on 8192 tokens, 32/2 heads, 16 blocks of 64: 690 us).
template <typename T, int D, int KW>
__global__ void __launch_bounds__(256, 2) block_attention_dkv_kernel(BackArgs b) {
  using Sh = KvShared<D, KW>;
  constexpr int kRowsAt = Sh::kRowsAt, RW = 4 / KW;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  const Args& p = b.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int quad = lane >> 4;
  const int64_t entries = p.kv_heads * b.rows;
  const int parts = p.bs > 64 ? 2 : 1;  // workgroups of a piece
  const int piece = blockIdx.x / parts;
  const int key_first = (blockIdx.x % parts) * 64;  // this workgroup's first key within the block
  if (piece >= b.first[entries]) return;
  const int64_t entry = b.owner[piece];
  const int hk = static_cast<int>(entry / b.rows);
  const int64_t row = entry % b.rows;
  int32_t q0, q1;  // the sequence's queries
  const Place at = place_of(p.cu_k, p.num_seqs, p.total_k, row, p.bs, [&](int i) { return cu_at(p.cu_q, p.num_seqs, p.total_q, i); }, q0, q1);
  const int64_t left = at.end - at.first;
  const int keys = static_cast<int>(left < 0 ? 0 : (left < p.bs ? left : p.bs));
  if (keys <= key_first) return;
  const int pieces = b.first[entry + 1] - b.first[entry];
  const int part = piece - b.first[entry];
  const int count = b.counts[entry];
  const int tokens = max(0, min(b.piece, count - part * b.piece));

  // the piece's tokens: those of rank [part * piece, ..) in the block's bits
  int64_t shift = 0;
  if (at.seq >= p.num_seqs) {
    q0 = q1 = 0;
  } else {
    shift = (at.end - at.begin) - (q1 - q0) - q0;  // position of token t: t + shift
  }
  if (tokens > 0) {
    const uint32_t* bits = b.bits + entry * b.words;
    const int64_t w0 = q0 >> 5, w1 = (q1 + 31) >> 5;
    const int64_t each = (w1 - w0 + 255) / 256;
    const int64_t from = w0 + tid * each, to = from + each < w1 ? from + each : w1;
    int n = 0;
    for (int64_t w = from; w < to; ++w) n += __popc(bits[w]);
    int sum = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 63) sh.wave_count[wave] = sum;
    __syncthreads();
    int rank = sum - n - part * b.piece;
    for (int w = 0; w < wave; ++w) rank += sh.wave_count[w];
    for (int64_t w = from; w < to; ++w) {
      uint32_t x = bits[w];
      while (x != 0) {
        const int bit = __ffs(x) - 1;
        x &= x - 1;
        if (rank >= 0 && rank < tokens) sh.list[rank] = static_cast<int32_t>(w * 32 + bit);
        ++rank;
      }
    }
    __syncthreads();
  }

  const int kw = wave % KW, rwv = wave / KW;
  const int key0 = key_first + kw * 16;  // first key of this wavefront within the block
  const int mykey = key0 + (lane & 15);
  const bool haskey = mykey < keys;
  u32x4 kf[D / 32], vf[D / 32];
  {
    const char* kfrom = static_cast<const char*>(p.k) + ((at.first + (haskey ? mykey : 0)) * p.k_t + hk * p.k_h) * 2 + quad * 16;
    const char* vfrom = static_cast<const char*>(p.v) + ((at.first + (haskey ? mykey : 0)) * p.v_t + hk * p.v_h) * 2 + quad * 16;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      kf[i] = haskey ? *reinterpret_cast<const u32x4*>(kfrom + i * 64) : u32x4{0, 0, 0, 0};
      vf[i] = haskey ? *reinterpret_cast<const u32x4*>(vfrom + i * 64) : u32x4{0, 0, 0, 0};
    }
  }
  f32x4 dk[D / 16], dv[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) dk[i] = dv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float c = p.scale * kLog2e;
  const int keypos = static_cast<int>(at.first - at.begin) + mykey;  // position of this lane's key
  const int lastpos = static_cast<int>(at.first - at.begin) + min(keys, key0 + 16) - 1;
  const Reads16<D> rd;
  const int total = tokens * p.group;

  // rows on their way to LDS: thread t has chunk t % kLanes of the rows
  // t / kLanes, + kStep, ...  Rows behind the last one repeat it and weigh nothing.
  constexpr int kLanes = D / 8, kStep = 256 / kLanes, kIn = kRowsAt / kStep;
  u32x4 qin[kIn], gin[kIn];
  float lse_in = 0.f, delta_in = 0.f;
  int pos_in = 0;
  auto token_of = [&](int r, int& head) {
    const int t = p.group == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), b.group_magic));
    head = hk * p.group + r - t * p.group;
    return static_cast<uint32_t>(sh.list[t]);
  };
  const char* qbase = static_cast<const char*>(p.q) + (tid % kLanes) * 16;
  const char* gbase = static_cast<const char*>(p.dout) + (tid % kLanes) * 16;
  const uint64_t qt = p.q_t * 2, gt = p.do_t * 2, qh = p.q_h * 2, gh = p.do_h * 2;
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kIn; ++j) {
      int head;
      const uint32_t tok = token_of(min(r0 + j * kStep + tid / kLanes, total - 1), head);
      qin[j] = *reinterpret_cast<const u32x4*>(qbase + (tok * qt + static_cast<uint32_t>(head) * qh));
      gin[j] = *reinterpret_cast<const u32x4*>(gbase + (tok * gt + static_cast<uint32_t>(head) * gh));
    }
    if (tid < kRowsAt) {
      int head;
      const uint32_t tok = token_of(min(r0 + tid, total - 1), head);
      const int64_t at_row = static_cast<int64_t>(tok) * p.heads + head;
      const float l = p.lse[at_row];
      lse_in = l == -kInf || r0 + tid >= total ? kInf : l * kLog2e;
      delta_in = b.delta[at_row];
      pos_in = p.causal ? static_cast<int32_t>(tok + shift) : INT32_MAX;
    }
  };
  if (total > 0) load_rows(0);
  int buf = 0;
  for (int r0 = 0; r0 < total; r0 += kRowsAt, buf ^= 1) {
#pragma unroll
    for (int j = 0; j < kIn; ++j) {
      const uint32_t to = tile_at<D>(j * kStep + tid / kLanes, tid % kLanes);
      *reinterpret_cast<u32x4*>(sh.q[buf] + to) = qin[j];
      *reinterpret_cast<u32x4*>(sh.go[buf] + to) = gin[j];
    }
    if (tid < kRowsAt) {
      sh.lse2[buf][tid] = lse_in;
      sh.delta[buf][tid] = delta_in;
      sh.pos[buf][tid] = pos_in;
    }
    __syncthreads();
    if (r0 + kRowsAt < total) load_rows(r0 + kRowsAt);
    const uint32_t qs = lds_offset(sh.q[buf]), gs = lds_offset(sh.go[buf]);
#pragma unroll
    for (int sub = 0; sub < kStage<KW>; sub += 32) {
      const int first = rwv * kStage<KW> + sub;  // this wavefront's rows
      const bool masked = __any(sh.pos[buf][first + (lane & 31)] < lastpos);
      f32x4 s[2], dp[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t] = dp[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s[t] = T::mfma16(rd.row(qs, first + 16 * t, i), kf[i], s[t]);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) dp[t] = T::mfma16(rd.row(gs, first + 16 * t, i), vf[i], dp[t]);
      }
      read_ahead<D / 8, 6, 1>();
      u32x4 pw, sw;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r0 = first + 16 * t + 4 * quad;
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(&sh.lse2[buf][r0]);
        const f32x4 d4 = *reinterpret_cast<const f32x4*>(&sh.delta[buf][r0]);
        float pr[4], sr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = exp2_fast(fmaf(s[t][e], c, -l4[e]));
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sh.pos[buf][r0 + e] < keypos) pr[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sr[e] = pr[e] * (dp[t][e] - d4[e]);
        pw[2 * t] = T::pack(pr[0], pr[1]);
        pw[2 * t + 1] = T::pack(pr[2], pr[3]);
        sw[2 * t] = T::pack(sr[0], sr[1]);
        sw[2 * t + 1] = T::pack(sr[2], sr[3]);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        dv[i] = T::mfma16(pw, rd.column(gs, first, i), dv[i]);
        dk[i] = T::mfma16(sw, rd.column(qs, first, i), dk[i]);
      }
      read_ahead<D / 8, 4, 2>();
    }
  }

  // as in the forward: a row that does not see a key must not reach it as 0 times
  // an infinity or NaN.  Places behind the block's last key do not count: their
  // scores are 0, and e^(0 - lse) has no bound (where a sequence ends in a part of
  // a block and lse is below -11 in fp16 or -88 in bf16)
  bool odd = false;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) bad |= !(fabsf(dk[i][r]) < kInf) || !(fabsf(dv[i][r]) < kInf);
    odd |= bad && key0 + 4 * quad + r < keys;
  }
  if (__syncthreads_or(odd)) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) dk[i] = dv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int r = rwv; r < total; r += RW) {
      int head;
      const int64_t tok = token_of(r, head);
      const char* qr = static_cast<const char*>(p.q) + (tok * p.q_t + head * p.q_h) * 2;
      const char* gr = static_cast<const char*>(p.dout) + (tok * p.do_t + head * p.do_h) * 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const u32x4 qv = *reinterpret_cast<const u32x4*>(qr + quad * 16 + i * 64), gv = *reinterpret_cast<const u32x4*>(gr + quad * 16 + i * 64);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          x = fmaf(T::hi(kf[i][z]), T::hi(qv[z]), fmaf(T::lo(kf[i][z]), T::lo(qv[z]), x));
          y = fmaf(T::hi(vf[i][z]), T::hi(gv[z]), fmaf(T::lo(vf[i][z]), T::lo(gv[z]), y));
        }
      }
      x = quad_sum(x);
      y = quad_sum(y);
      const int64_t at_row = tok * p.heads + head;
      const float l = p.lse[at_row];
      const int64_t pos = p.causal ? tok + shift : INT32_MAX;
      const bool sees = haskey && keypos <= pos && l != -kInf;
      const float pr = sees ? exp2_fast(fmaf(x, c, -l * kLog2e)) : 0.f;
      const float ds = sees ? pr * (y - b.delta[at_row]) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = 4 * quad + j;  // the lane that has key 4 quad + j
        const bool seen = __shfl(static_cast<int>(sees), from) != 0;
        const float pj = __shfl(pr, from), dj = __shfl(ds, from);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float gx = T::lo(reinterpret_cast<const uint16_t*>(gr)[i * 16 + (lane & 15)]);
          const float qx = T::lo(reinterpret_cast<const uint16_t*>(qr)[i * 16 + (lane & 15)]);
          dv[i][j] = seen ? fmaf(pj, gx, dv[i][j]) : dv[i][j];
          dk[i][j] = seen ? fmaf(dj, qx, dk[i][j]) : dk[i][j];
        }
      }
    }
  }

  // Join the wavefronts that share keys, values first, then keys: lane l holds
  // column l & 15 of 16 and keys 4 (l >> 4) + r.
  const int64_t out0 = (at.first * p.kv_heads + hk) * D;
  const int here = min(keys - key_first, KW * 16);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh.join[wave][4 * quad + r][i * 16 + (lane & 15)] = side == 0 ? dv[i][r] : dk[i][r] * p.scale;
    __syncthreads();
    for (int e = tid; e < here * (D / 4); e += 256) {
      const int key = e / (D / 4), d = (e % (D / 4)) * 4;
      f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < RW; ++w) x += *reinterpret_cast<const f32x4*>(&sh.join[w * KW + key / 16][key % 16][d]);
      if (pieces == 1) {
        char* to = static_cast<char*>(side == 0 ? p.dv : p.dk) + (out0 + static_cast<int64_t>(key_first + key) * p.kv_heads * D + d) * 2;
        *reinterpret_cast<u32x2*>(to) = u32x2{T::pack(x[0], x[1]), T::pack(x[2], x[3])};
      } else {
        *reinterpret_cast<f32x4*>(b.part + ((static_cast<int64_t>(piece) * 2 + side) * p.bs + key_first + key) * D + d) = x;
      }
    }
  }
}

// Sums the pieces of the blocks that have several, in their order: one workgroup
// a block and 1024 of its 2 bs D values, eight pieces' loads in flight.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_pieces_kernel(BackArgs b) {
  const Args& p = b.a;
  const int64_t entry = blockIdx.x;
  const int first = b.first[entry], pieces = b.first[entry + 1] - first;
  if (pieces == 1) return;
  const int hk = static_cast<int>(entry / b.rows);
  const Place at = place_of(p.cu_k, p.num_seqs, p.total_k, entry % b.rows, p.bs);
  const int64_t left = at.end - at.first;
  const int keys = static_cast<int>(left < p.bs ? left : p.bs);
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
  const int side = e / (p.bs * D), key = e % (p.bs * D) / D, d = e % D;
  if (key >= keys) return;
  const float* from = b.part + static_cast<int64_t>(first) * 2 * p.bs * D + e;
  f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = 0; i < pieces; ++i) x += *reinterpret_cast<const f32x4*>(from + static_cast<int64_t>(i) * 2 * p.bs * D);
  char* to = static_cast<char*>(side == 0 ? p.dv : p.dk) + ((at.first + key) * p.kv_heads + hk) * static_cast<int64_t>(2 * D) + d * 2;
  *reinterpret_cast<u32x2*>(to) = u32x2{T::pack(x[0], x[1]), T::pack(x[2], x[3])};
}

// Sizes of the workspace's parts, 256-byte aligned.
struct Layout {
  uint64_t delta, bits, first, counts, owner, part, bytes;
};

uint64_t up256(uint64_t n) { return (n + 255) & ~uint64_t{255}; }

Layout lay_out(BackArgs& b, int dim) {
  const Args& p = b.a;
  b.rows = slots_of(p.total_k, p.num_seqs, p.bs);
  b.words = (p.total_q + 31) / 32;
  b.piece = kPieceRows / p.group;
  b.group_magic = static_cast<uint32_t>(((uint64_t{1} << 32) + p.group - 1) / p.group);
  const uint64_t entries = static_cast<uint64_t>(p.kv_heads) * b.rows;
  const uint64_t pairs = static_cast<uint64_t>(p.total_q) * p.select * p.kv_heads;
  const uint64_t pieces = entries + pairs / b.piece;
  b.max_pieces = pieces > INT32_MAX / 2 ? -1 : static_cast<int32_t>(pieces);
  Layout l;
  l.delta = 0;
  l.bits = up256(static_cast<uint64_t>(p.total_q) * p.heads * 4);
  l.first = l.bits + up256(entries * b.words * 4);
  l.counts = l.first + up256((entries + 1) * 4);
  l.owner = l.counts + up256(entries * 4);
  l.part = l.owner + up256(pieces * 4);
  l.bytes = l.part + pieces * 2 * p.bs * dim * 4;
  return l;
}

template <typename T, int D, int KW>
int launch_dkv(const BackArgs& b, hipStream_t stream) {
  block_attention_dkv_kernel<T, D, KW><<<dim3(static_cast<unsigned>(b.max_pieces) * (b.a.bs > 64 ? 2u : 1u)), dim3(256), sizeof(KvShared<D, KW>), stream>>>(b);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

template <typename T, int D, bool kSplit>
void launch_dq(const BackArgs& b, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(b.a.slots * b.a.kv_heads));
  if (b.a.lb >= 6) block_attention_dq_kernel<T, D, true, kSplit><<<grid, dim3(256), sizeof(QShared<T, D>), stream>>>(b);
  else block_attention_dq_kernel<T, D, false, kSplit><<<grid, dim3(256), sizeof(QShared<T, D>), stream>>>(b);
}

template <typename T, int D>
int launch_backward(const BackArgs& b, hipStream_t stream) {
  const Args& p = b.a;
  const int64_t grid = p.slots * p.kv_heads;
  const int64_t entries = p.kv_heads * b.rows;
  const int64_t pairs = p.total_q * p.kv_heads * p.select;
  if (grid > INT32_MAX || entries > INT32_MAX || b.max_pieces < 0) return MI_ATTN_EINVAL;
  const int64_t words = entries * b.words;
  if (entries > 0)
    clear_bits_kernel<<<dim3(static_cast<unsigned>(words / 1024 + 1 < 4096 ? words / 1024 + 1 : 4096)), dim3(256), 0, stream>>>(b);
  if (pairs > 0) {
    BackArgs few = b;
    if (split_rows(few.a, D)) launch_dq<T, D, true>(few, stream);
    else launch_dq<T, D, false>(b, stream);
  }
  if (p.total_k == 0) return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
  number_pieces_kernel<<<dim3(1), dim3(1024), 0, stream>>>(b);
  if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  const int st = p.bs >= 64 ? launch_dkv<T, D, 4>(b, stream) : (p.bs == 32 ? launch_dkv<T, D, 2>(b, stream) : launch_dkv<T, D, 1>(b, stream));
  if (st != MI_ATTN_OK) return st;
  join_pieces_kernel<T, D><<<dim3(static_cast<unsigned>(entries), 2 * p.bs * D / 1024), dim3(256), 0, stream>>>(b);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT uint64_t block_attention_workspace(const mi_block_attention_args* args) {
  BackArgs b;
  if (make_args(args, b.a) != MI_ATTN_OK) return 0;
  return lay_out(b, args->dim).bytes;
}

MI_ATTN_EXPORT int block_attention_backward(const mi_block_attention_args* args, hipStream_t stream) {
  BackArgs b;
  const int st = make_args(args, b.a);
  if (st != MI_ATTN_OK) return st;
  const Args& p = b.a;
  if (args->dout_stride_t < 0 || args->dout_stride_h < 0 || ((args->dout_stride_t | args->dout_stride_h) & 7)) return MI_ATTN_EINVAL;
  const void* wide[] = {args->dout, args->dq, args->dk, args->dv, args->workspace};
  for (const void* x : wide)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return MI_ATTN_EINVAL;
  if (p.total_q > 0 && (p.dout == nullptr || p.dq == nullptr)) return MI_ATTN_EINVAL;
  if (p.total_k > 0 && (p.dk == nullptr || p.dv == nullptr)) return MI_ATTN_EINVAL;
  if (p.total_q == 0 && p.total_k == 0) return MI_ATTN_OK;
  const Layout l = lay_out(b, args->dim);
  if (args->workspace == nullptr || args->workspace_bytes < l.bytes) return MI_ATTN_EWORKSPACE;
  char* ws = static_cast<char*>(args->workspace);
  b.delta = reinterpret_cast<float*>(ws + l.delta);
  b.bits = reinterpret_cast<uint32_t*>(ws + l.bits);
  b.first = reinterpret_cast<int32_t*>(ws + l.first);
  b.counts = reinterpret_cast<int32_t*>(ws + l.counts);
  b.owner = reinterpret_cast<int32_t*>(ws + l.owner);
  b.part = reinterpret_cast<float*>(ws + l.part);
  if (args->dtype == MI_ATTN_BF16)
    return args->dim == 128 ? launch_backward<Bf16, 128>(b, stream) : launch_backward<Bf16, 64>(b, stream);
  return args->dim == 128 ? launch_backward<Fp16, 128>(b, stream) : launch_backward<Fp16, 64>(b, stream);
}
