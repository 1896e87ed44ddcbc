// The gradient of block sparse attention.
//
//   p_j = exp(scale q.k_j - lse),  delta = dout . out,  ds_j = p_j (dout.v_j - delta)
//   dq = scale sum_j ds_j k_j,  dk_j = scale sum_q ds_j q,  dv_j = sum_q p_j dout
//
// dq goes over the rows as the forward does.  dk and dv go over the key blocks:
// a bit matrix [key head][block][token] says which tokens selected a block
// (atomic OR, so its content does not depend on their order), a block's tokens
// are cut into pieces of equal length, and a workgroup takes one piece: the
// sink and the own blocks, which every token selects, become many pieces.  A
// block of one piece is written at once; the others' pieces are summed in order
// by a last kernel, so the result is the same from run to run.
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
  float* part;         // [piece][2][bs][D]
  int64_t rows;        // blocks of all sequences, and those of the keys behind them
  int64_t words;
  int32_t piece;       // tokens of a piece
  int32_t max_pieces;
};

// ---- dq ----

template <typename T, int D>
struct QShared {
  char k[2][kTile * 2 * D];
  char v[2][kTile * 2 * D];
  Select sel;
};

template <typename T, int D>
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
  const int row = wave * 32 + (lane & 31);
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
    const char* ofrom = static_cast<const char*>(p.out) + (tok * p.heads + head) * (2 * D) + half * 16;
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
      }
    }
    delta = half_sum(delta);
    if (valid) {
      const float l = p.lse[tok * p.heads + head];
      lse2 = l == -kInf ? kInf : l * kLog2e;
      if (half == 0) b.delta[tok * p.heads + head] = delta;
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
  const uint32_t kread = (lane & 31) * (2 * D) + ((half ^ swizzle<D>(lane & 31)) << 4);
  const int li = lane & 15, dhalf = (lane >> 4) & 1;
  const uint32_t trow = 4 * half + (li >> 2);
  const uint32_t tchunk = dhalf * 2 + ((li & 3) >> 1);

  for (int w0 = 0; w0 < g.blocks; w0 += width) {
    const int active = list_window(p, g, hk, w0, width, nw, sh.sel);
    const int tiles = ((active << p.lb) + kTile - 1) / kTile;
    Keys next = keys_of(sh.sel, p.lb, p.bs, w0, active, 0);
    if (tiles > 0) {
      stage_tile<D>(sh.k[0], kbase, p.k_t * 2, next, g.len_k, wave, lane);
      stage_tile<D>(sh.v[0], vbase, p.v_t * 2, next, g.len_k, wave, lane);
    }
    for (int tile = 0; tile < tiles; ++tile) {
      const Keys keys = next;
      wait_loads();
      __syncthreads();
      const int buf = tile & 1;
      if (tile + 1 < tiles) {
        next = keys_of(sh.sel, p.lb, p.bs, w0, active, tile + 1);
        stage_tile<D>(sh.k[buf ^ 1], kbase, p.k_t * 2, next, g.len_k, wave, lane);
        stage_tile<D>(sh.v[buf ^ 1], vbase, p.v_t * 2, next, g.len_k, wave, lane);
      }
      const Sight see = sight_of(sh.sel, keys, nw, tl >> 5 < nw ? tl >> 5 : 0, tl & 31, limit, valid);
      if (!see.any) continue;
      const uint32_t ks = lds_offset(sh.k[buf]), vs = lds_offset(sh.v[buf]);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        f32x16 s, dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s = T::mfma32(lds_read16(ks + mt * 32 * 2 * D + (kread ^ (i * 32))), q[i], s);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) dp = T::mfma32(lds_read16(vs + mt * 32 * 2 * D + (kread ^ (i * 32))), go[i], dp);
        u32x4 ds[2];
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int off = 8 * (((r + e) >> 2) & 1) + ((r + e) & 3);
            w[e] = exp2_fast(fmaf(s[r + e], c, -lse2)) * (dp[r + e] - delta);
            if (!see.full && off + 4 * half > see.last[mt * 2 + (r >> 3)]) w[e] = 0.f;
          }
          ds[r >> 3][(r & 7) >> 1] = T::pack(w[0], w[1]);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t r0 = mt * 32 + 16 * st + trow;
            const u32x2 x = lds_read_tr16(ks + tile_at<D>(r0, 4 * i + tchunk) + (li & 1) * 8);
            const u32x2 y = lds_read_tr16(ks + tile_at<D>(r0 + 8, 4 * i + tchunk) + (li & 1) * 8);
            acc[i] = T::mfma32(u32x4{x[0], x[1], y[0], y[1]}, ds[st], acc[i]);
          }
      }
    }
  }
  if (!valid) return;
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

// ---- which tokens selected a block ----

__global__ void __launch_bounds__(256) clear_bits_kernel(BackArgs b) {
  const int64_t total = b.a.kv_heads * b.rows * b.words;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) b.bits[i] = 0;
}

// One thread per selected entry.
__global__ void __launch_bounds__(256) mark_bits_kernel(BackArgs b) {
  const Args& p = b.a;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.total_q * p.kv_heads * p.select) return;
  const int64_t tok = i / (static_cast<int64_t>(p.kv_heads) * p.select);
  const int hk = static_cast<int>((i / p.select) % p.kv_heads);
  const int blk = p.blocks[i];
  if (blk < 0) return;
  const Place at = place_of(p.cu_q, p.num_seqs, p.total_q, tok, 1);
  if (at.seq >= p.num_seqs) return;
  const int64_t k0 = cu_at(p.cu_k, p.num_seqs, p.total_k, at.seq), k1 = cu_at(p.cu_k, p.num_seqs, p.total_k, at.seq + 1);
  const int64_t pos = (k1 - k0) - (at.end - at.begin) + (tok - at.begin);
  const int64_t from = static_cast<int64_t>(blk) * p.bs;
  if (from >= k1 - k0 || (p.causal && from > pos)) return;
  const int64_t row = k0 / p.bs + at.seq + blk;
  atomicOr(b.bits + (hk * b.rows + row) * b.words + (tok >> 5), 1u << (tok & 31));
}

// Tokens of each block; one wavefront a block.
__global__ void __launch_bounds__(256) count_bits_kernel(BackArgs b) {
  const int lane = threadIdx.x & 63;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (e >= b.a.kv_heads * b.rows) return;
  const uint32_t* bits = b.bits + e * b.words;
  int n = 0;
  for (int64_t w = lane; w < b.words; w += 64) n += __popc(bits[w]);
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  if (lane == 0) b.counts[e] = n;
}

// Pieces of each block (one at least, for the zeros of a block that nobody
// selected) and their running number; one workgroup.
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
    __syncthreads();
    if (tid == 1023) s_base = at + n;
    __syncthreads();
  }
  if (tid == 0) b.first[total] = s_base;
}

// ---- dk, dv ----

template <int D, int KW>
struct KvShared {
  static constexpr int kRowsAt = 32 * (4 / KW < 2 ? 2 : 4 / KW);  // rows staged at a time
  union {
    struct {
      char q[kRowsAt * 2 * D];
      char go[kRowsAt * 2 * D];
    };
    float join[4][32][D + 1];
  };
  float lse2[kRowsAt], delta[kRowsAt];
  int32_t pos[kRowsAt];
  int32_t list[kPieceRows];
  int32_t wave_count[4];
};

// A block's keys: KW wavefronts of 32 keys (of 16 in a block of 16); 4 / KW
// wavefronts share the keys and take different rows.  The keys and values stay
// in registers as operands, the rows' queries and output gradients are staged
// in LDS and read by rows for the scores, transposed for the gradients.
template <typename T, int D, int KW>
__global__ void __launch_bounds__(256, 1) block_attention_dkv_kernel(BackArgs b) {
  using Sh = KvShared<D, KW>;
  constexpr int kRowsAt = Sh::kRowsAt, RW = 4 / KW;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  const Args& p = b.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, li = lane & 15, dhalf = (lane >> 4) & 1;
  const int64_t entries = p.kv_heads * b.rows;
  const int piece = blockIdx.x;
  if (piece >= b.first[entries]) return;
  int64_t lo = 0, hi = entries - 1;  // the last entry whose first piece is not behind this one
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= piece) lo = mid; else hi = mid - 1;
  }
  const int64_t entry = lo;
  const int hk = static_cast<int>(entry / b.rows);
  const int64_t row = entry % b.rows;
  const Place at = place_of(p.cu_k, p.num_seqs, p.total_k, row, p.bs);
  const int64_t left = at.end - at.first;
  const int keys = static_cast<int>(left < 0 ? 0 : (left < p.bs ? left : p.bs));
  if (keys == 0) return;
  const int pieces = b.first[entry + 1] - b.first[entry];
  const int part = piece - b.first[entry];
  const int count = b.counts[entry];
  const int tokens = max(0, min(b.piece, count - part * b.piece));

  // the piece's tokens: those of rank [part * piece, ..) in the block's bits
  int64_t q0 = 0, q1 = 0, shift = 0;
  if (at.seq < p.num_seqs) {
    q0 = cu_at(p.cu_q, p.num_seqs, p.total_q, at.seq);
    q1 = cu_at(p.cu_q, p.num_seqs, p.total_q, at.seq + 1);
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
  const int key0 = kw * 32;  // first key of this wavefront within the block
  const int mykey = key0 + (lane & 31);
  const bool haskey = mykey < keys;
  u32x4 kf[D / 16], vf[D / 16];
  {
    const char* kfrom = static_cast<const char*>(p.k) + ((at.first + (haskey ? mykey : 0)) * p.k_t + hk * p.k_h) * 2 + half * 16;
    const char* vfrom = static_cast<const char*>(p.v) + ((at.first + (haskey ? mykey : 0)) * p.v_t + hk * p.v_h) * 2 + half * 16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      kf[i] = haskey ? *reinterpret_cast<const u32x4*>(kfrom + i * 32) : u32x4{0, 0, 0, 0};
      vf[i] = haskey ? *reinterpret_cast<const u32x4*>(vfrom + i * 32) : u32x4{0, 0, 0, 0};
    }
  }
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[i][r] = dv[i][r] = 0.f;
  const float c = p.scale * kLog2e;
  const int64_t keypos = at.first - at.begin + mykey;  // position of this lane's key
  const int lastpos = static_cast<int>(at.first - at.begin) + min(keys, key0 + 32) - 1;
  const uint32_t aread = (lane & 31) * (2 * D) + ((half ^ swizzle<D>(lane & 31)) << 4);
  const uint32_t trow = 4 * half + (li >> 2);
  const uint32_t tchunk = dhalf * 2 + ((li & 3) >> 1);
  const uint32_t qs = lds_offset(sh.q), gs = lds_offset(sh.go);
  const int total = tokens * p.group;
  constexpr int kChunks = D / 8, kRowsPer = 64 / kChunks;

  for (int r0 = 0; r0 < total; r0 += kRowsAt) {
    __syncthreads();
    // stage the rows; those behind the last one repeat it and weigh nothing
#pragma unroll
    for (int j = 0; j < kRowsAt / (4 * kRowsPer); ++j) {
      const int base = (j * 4 + wave) * kRowsPer;
      const int rr = base + lane / kChunks, chunk = (lane % kChunks) ^ swizzle<D>(rr);
      const int at_row = min(r0 + rr, total - 1);
      const int64_t tok = sh.list[at_row / p.group];
      const int head = hk * p.group + at_row % p.group;
      __builtin_amdgcn_global_load_lds((const MI_GLOBAL void*)(static_cast<const char*>(p.q) + (tok * p.q_t + head * p.q_h + chunk * 8) * 2),
                                       (MI_LDS void*)(sh.q + base * 2 * D), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const MI_GLOBAL void*)(static_cast<const char*>(p.dout) + (tok * p.do_t + head * p.do_h + chunk * 8) * 2),
                                       (MI_LDS void*)(sh.go + base * 2 * D), 16, 0, 0);
    }
    if (tid < kRowsAt) {
      const int at_row = min(r0 + tid, total - 1);
      const int64_t tok = sh.list[at_row / p.group];
      const int64_t i = tok * p.heads + hk * p.group + at_row % p.group;
      const float l = p.lse[i];
      sh.lse2[tid] = l == -kInf || r0 + tid >= total ? kInf : l * kLog2e;
      sh.delta[tid] = b.delta[i];
      sh.pos[tid] = p.causal ? static_cast<int32_t>(tok + shift) : INT32_MAX;
    }
    wait_loads();
    __syncthreads();
    for (int sub = rwv; sub < kRowsAt / 32; sub += RW) {
      if (r0 + sub * 32 >= total) break;
      const uint32_t off = sub * 32 * 2 * D;
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) s = T::mfma32(lds_read16(qs + off + (aread ^ (i * 32))), kf[i], s);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) dp = T::mfma32(lds_read16(gs + off + (aread ^ (i * 32))), vf[i], dp);
      const bool masked = __any(sh.pos[sub * 32 + (lane & 31)] < lastpos);
      u32x4 pw[2], sw[2];
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int m = sub * 32 + 8 * (r >> 2) + 4 * half;
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(&sh.lse2[m]);
        const f32x4 d4 = *reinterpret_cast<const f32x4*>(&sh.delta[m]);
        float pr[4], sr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = exp2_fast(fmaf(s[r + e], c, -l4[e]));
          sr[e] = pr[e] * (dp[r + e] - d4[e]);
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sh.pos[m + e] < keypos) pr[e] = sr[e] = 0.f;
        }
        pw[r >> 3][(r & 7) >> 1] = T::pack(pr[0], pr[1]);
        pw[r >> 3][((r & 7) >> 1) + 1] = T::pack(pr[2], pr[3]);
        sw[r >> 3][(r & 7) >> 1] = T::pack(sr[0], sr[1]);
        sw[r >> 3][((r & 7) >> 1) + 1] = T::pack(sr[2], sr[3]);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint32_t t0 = sub * 32 + 16 * st + trow;
          const uint32_t a0 = tile_at<D>(t0, 4 * i + tchunk) + (li & 1) * 8, a1 = tile_at<D>(t0 + 8, 4 * i + tchunk) + (li & 1) * 8;
          const u32x2 x = lds_read_tr16(gs + a0), y = lds_read_tr16(gs + a1);
          dv[i] = T::mfma32(pw[st], u32x4{x[0], x[1], y[0], y[1]}, dv[i]);
          const u32x2 z = lds_read_tr16(qs + a0), w = lds_read_tr16(qs + a1);
          dk[i] = T::mfma32(sw[st], u32x4{z[0], z[1], w[0], w[1]}, dk[i]);
        }
    }
  }

  // Join the wavefronts that share keys, values first, then keys.
  const int64_t out0 = (at.first * p.kv_heads + hk) * D;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        sh.join[wave][8 * (r >> 2) + 4 * half + (r & 3)][i * 32 + (lane & 31)] = side == 0 ? dv[i][r] : dk[i][r] * p.scale;
    __syncthreads();
    for (int e = tid; e < keys * (D / 2); e += 256) {
      const int key = e / (D / 2), d = (e % (D / 2)) * 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < RW; ++w) {
        x += sh.join[w * KW + key / 32][key % 32][d];
        y += sh.join[w * KW + key / 32][key % 32][d + 1];
      }
      if (pieces == 1) {
        char* to = static_cast<char*>(side == 0 ? p.dv : p.dk) + (out0 + static_cast<int64_t>(key) * p.kv_heads * D + d) * 2;
        *reinterpret_cast<uint32_t*>(to) = T::pack(x, y);
      } else {
        float* to = b.part + ((static_cast<int64_t>(piece) * 2 + side) * p.bs + key) * D + d;
        to[0] = x;
        to[1] = y;
      }
    }
  }
}

// Sums the pieces of the blocks that have several: one workgroup a block.
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
  const int64_t out0 = (at.first * p.kv_heads + hk) * D;
  for (int e = threadIdx.x; e < 2 * keys * (D / 2); e += 256) {
    const int side = e / (keys * (D / 2)), f = e % (keys * (D / 2));
    const int key = f / (D / 2), d = (f % (D / 2)) * 2;
    float x = 0.f, y = 0.f;
    for (int i = 0; i < pieces; ++i) {
      const float* from = b.part + ((static_cast<int64_t>(first + i) * 2 + side) * p.bs + key) * D + d;
      x += from[0];
      y += from[1];
    }
    char* to = static_cast<char*>(side == 0 ? p.dv : p.dk) + (out0 + static_cast<int64_t>(key) * p.kv_heads * D + d) * 2;
    *reinterpret_cast<uint32_t*>(to) = T::pack(x, y);
  }
}

// Sizes of the workspace's parts, 256-byte aligned.
struct Layout {
  uint64_t delta, bits, first, counts, part, bytes;
};

uint64_t up256(uint64_t n) { return (n + 255) & ~uint64_t{255}; }

Layout lay_out(BackArgs& b, int dim) {
  const Args& p = b.a;
  b.rows = slots_of(p.total_k, p.num_seqs, p.bs);
  b.words = (p.total_q + 31) / 32;
  b.piece = kPieceRows / p.group;
  const uint64_t entries = static_cast<uint64_t>(p.kv_heads) * b.rows;
  const uint64_t pairs = static_cast<uint64_t>(p.total_q) * p.select * p.kv_heads;
  const uint64_t pieces = entries + pairs / b.piece;
  b.max_pieces = pieces > INT32_MAX ? -1 : static_cast<int32_t>(pieces);
  Layout l;
  l.delta = 0;
  l.bits = up256(static_cast<uint64_t>(p.total_q) * p.heads * 4);
  l.first = l.bits + up256(entries * b.words * 4);
  l.counts = l.first + up256((entries + 1) * 4);
  l.part = l.counts + up256(entries * 4);
  l.bytes = l.part + pieces * 2 * p.bs * dim * 4;
  return l;
}

template <typename T, int D, int KW>
int launch_dkv(const BackArgs& b, hipStream_t stream) {
  block_attention_dkv_kernel<T, D, KW><<<dim3(static_cast<unsigned>(b.max_pieces)), dim3(256), sizeof(KvShared<D, KW>), stream>>>(b);
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

template <typename T, int D>
int launch_backward(const BackArgs& b, hipStream_t stream) {
  const Args& p = b.a;
  const int64_t grid = p.slots * p.kv_heads;
  const int64_t entries = p.kv_heads * b.rows;
  const int64_t pairs = p.total_q * p.kv_heads * p.select;
  if (grid > INT32_MAX || entries > INT32_MAX || (pairs + 255) / 256 > INT32_MAX || b.max_pieces < 0) return MI_ATTN_EINVAL;
  const int64_t words = entries * b.words;
  if (words > 0)
    clear_bits_kernel<<<dim3(static_cast<unsigned>(words / 1024 + 1 < 4096 ? words / 1024 + 1 : 4096)), dim3(256), 0, stream>>>(b);
  if (pairs > 0) {
    mark_bits_kernel<<<dim3(static_cast<unsigned>((pairs + 255) / 256)), dim3(256), 0, stream>>>(b);
    block_attention_dq_kernel<T, D><<<dim3(static_cast<unsigned>(grid)), dim3(256), sizeof(QShared<T, D>), stream>>>(b);
  }
  if (p.total_k == 0) return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
  count_bits_kernel<<<dim3(static_cast<unsigned>((entries + 3) / 4)), dim3(256), 0, stream>>>(b);
  number_pieces_kernel<<<dim3(1), dim3(1024), 0, stream>>>(b);
  if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  const int st = p.bs == 128 ? launch_dkv<T, D, 4>(b, stream) : (p.bs == 64 ? launch_dkv<T, D, 2>(b, stream) : launch_dkv<T, D, 1>(b, stream));
  if (st != MI_ATTN_OK) return st;
  join_pieces_kernel<T, D><<<dim3(static_cast<unsigned>(entries)), dim3(256), 0, stream>>>(b);
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
  b.part = reinterpret_cast<float*>(ws + l.part);
  if (args->dtype == MI_ATTN_BF16)
    return args->dim == 128 ? launch_backward<Bf16, 128>(b, stream) : launch_backward<Bf16, 64>(b, stream);
  return args->dim == 128 ? launch_backward<Fp16, 128>(b, stream) : launch_backward<Fp16, 64>(b, stream);
}
