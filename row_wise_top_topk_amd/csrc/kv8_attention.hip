// Attention over the 8-bit paged cache.
//
//   out = sum_j p_j V_j s_v,  p_j = softmax(scale q.K_j s_k)   (s_k, s_v of j's page)
//
// A call of few tokens a sequence reads every visible code once, so it is bound
// by memory (many tokens: once for every 64 rows).  A workgroup
// takes the rows of one key head (tokens x the heads of its group, MT tiles of
// 16) and a chunk of the keys; its four wavefronts take 32 keys at a time in
// turn, each with its own running softmax, and are joined at the end.  A second
// kernel joins the chunks.  The codes become 16-bit elements exactly; a page's
// K scale multiplies its scores.  Its V scale joins the exponent: the running
// maximum is that of x = s + log2 s_v, the weights are 2^(x - max), and the sum
// of the probabilities adds a page's weights divided by s_v.
//
// Measured: 64 sequences of 500 to 32000 keys, 64/8 heads of 128, pages of 64:
// 400 us and 13 for the join, 2.13 GB at 5.2 TB/s, more than a large copy reaches;
// 3 x 3 tokens over 20011 keys: 10 + 6 us, 8 single tokens at 32 of 14000 blocks:
// 8 + 5 us: there the chain from the lengths over the table and the scales to the
// codes bounds it.  2048 new tokens over 32000 keys, 64/8 heads: 5.8 ms, 360
// TFLOP/s; each workgroup widens all codes again for its 64 rows, which has one
// wavefront a SIMD; at 32 selected blocks 1.0 ms, each token's blocks read alone.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_kv8.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

constexpr int kSeg = 256;          // blocks whose page numbers and scales are in LDS at a time
// V scales are held between these: 2^30 weights of up to 2^14, divided by the
// least, stay within fp32
constexpr float kLeast = 0x1p-80f, kMost = 0x1p100f;

struct DecodeArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* cu;
  const int32_t* blocks;
  void* out;
  float* lse;
  float* part;       // [item][split][R][D], then [item][split][R][2]
  float* part_ml;
  int64_t q_t, q_h, total_q, num_pages, table_stride, slots;
  int32_t table_cols, num_seqs, heads, kv_heads, group, bs, lb, select, tokens_per, head_chunks, splits, chunk;
  int32_t spread;  // splits is 2^spread, or -1
  float scale;
};

// The rows of a workgroup.
struct Rows {
  int seq, tokens, heads;  // sequence; tokens and heads of a group in this workgroup
  int64_t first;           // first token
  int64_t pos;             // position of the first token
  int hk, head0;
  int len;                 // keys of the sequence that the table can hold
};

__device__ __forceinline__ Rows rows_of(const DecodeArgs& p, uint32_t item, int rows) {
  Rows r;
  const int hc = static_cast<int>(item % p.head_chunks);
  const uint32_t rest = item / p.head_chunks;
  r.hk = static_cast<int>(rest % p.kv_heads);
  int32_t len, none;
  const Place at = place_of(p.cu, p.num_seqs, p.total_q, rest / p.kv_heads, p.tokens_per,
                            [&](int i) { return i < p.num_seqs ? p.lengths[i] : 0; }, len, none);
  r.seq = at.seq;
  r.first = at.first;
  const int64_t left = at.end - at.first;
  r.tokens = static_cast<int>(left < 0 ? 0 : (left < p.tokens_per ? left : p.tokens_per));
  const int per = p.head_chunks == 1 ? p.group : rows;
  r.head0 = r.hk * p.group + hc * per;
  r.heads = min(per, p.group - hc * per);
  r.len = 0;
  r.pos = -1;
  if (at.seq < p.num_seqs && r.tokens > 0) {
    const int64_t most = static_cast<int64_t>(p.table_cols) << p.lb;
    r.pos = len - (at.end - at.begin) + (at.first - at.begin);
    r.len = static_cast<int>(len < 0 ? 0 : (len < most ? len : most));
  }
  return r;
}

// Blocks that a workgroup's rows can see: those up to the last token's position.
__device__ __forceinline__ int blocks_seen(const DecodeArgs& p, const Rows& r) {
  int64_t seen = r.pos + r.tokens;
  if (seen > r.len) seen = r.len;
  return seen <= 0 ? 0 : static_cast<int>((seen + p.bs - 1) >> p.lb);
}

template <int D>
__device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t chunk) {  // 16-byte chunks of a row of D codes
  return D == 128 ? row * 128 + ((chunk ^ ((row >> 1) & 7u)) << 4) : row * 64 + ((chunk ^ ((row >> 2) & 3u)) << 4);
}

template <int D>
struct DecodeShared {
  union {
    char v[4][32 * D];
    float join[4][16][D + 4];
  };
  float ml[4][64][2];
  int32_t page[kSeg];  // -1: not there
  int32_t block[kSeg];
  float ks[kSeg], vs[kSeg];
  int32_t list[MI_ATTN_MAX_SELECT];
  int32_t count[4];
};

// The valid, different entries of a query's selection, in their order.
template <typename S>
__device__ __forceinline__ int list_selected(const DecodeArgs& p, const Rows& r, int nb, S& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t* from = p.blocks + (r.first * p.kv_heads + r.hk) * static_cast<int64_t>(p.select);
  int32_t mine[MI_ATTN_MAX_SELECT / 256];
  bool sorted = true;
#pragma unroll
  for (int i = 0; i < MI_ATTN_MAX_SELECT / 256; ++i) {
    const int e = i * 256 + tid;
    mine[i] = -1;
    if (e < p.select) {
      const int b = from[e];
      mine[i] = b >= 0 && b < nb ? b : -1;
      s.list[e] = mine[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MI_ATTN_MAX_SELECT / 256; ++i) {
    const int e = i * 256 + tid;
    if (e < p.select && e > 0 && mine[i] >= 0 && s.list[e - 1] >= mine[i]) sorted = false;
    if (e < p.select && e > 0 && mine[i] >= 0 && s.list[e - 1] < 0) sorted = false;  // an ascending row ends in its -1s
  }
  const bool clean = __syncthreads_and(sorted);
  if (!clean) {
#pragma unroll
    for (int i = 0; i < MI_ATTN_MAX_SELECT / 256; ++i) {
      const int e = i * 256 + tid;
      if (mine[i] >= 0)
        for (int f = 0; f < e; ++f)
          if (s.list[f] == mine[i]) { mine[i] = -1; break; }
    }
  }
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < MI_ATTN_MAX_SELECT / 256; ++i) {
    if (i * 256 >= p.select) break;
    const uint64_t has = __ballot(mine[i] >= 0);
    if (lane == 0) s.count[wave] = __popcll(has);
    __syncthreads();
    int at = base + __popcll(has & ((1ull << lane) - 1));
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += s.count[w];
      base += s.count[w];
    }
    if (mine[i] >= 0) s.list[at] = mine[i];
    __syncthreads();
  }
  return base;
}

// Four tiles of rows with 128 columns need more than 256 registers: one
// wavefront a SIMD there (16 sequences of 16000 keys, 64/4 heads, 4 tokens: 150
// us, with two 346; with 64 columns two are better, 62 and 91).
template <typename T, int D, int MT>
__global__ void __launch_bounds__(256, D == 128 ? (MT == 4 ? 1 : 2) : (MT == 4 ? 2 : 3)) kv8_attention_kernel(DecodeArgs p) {
  constexpr int R = MT * 16;
  __shared__ __attribute__((aligned(16))) DecodeShared<D> sh;
  // Consecutive workgroups go to the eight dies in turn, and on each to its four
  // engines.  The later chunks of a short sequence are empty: without the shift
  // an even number of chunks would give a die the same ones of every sequence (64
  // sequences of 500 to 32000 keys, 8 chunks: 413 us instead of 546, with the
  // join).  Few chunks (2^spread) are shifted by the bits of the item above those
  // that choose the engine.
  const uint32_t item = blockIdx.x / p.splits;
  uint32_t shift = item + (item >> 1) + (item >> 2);
  if (p.spread >= 0) {
    shift = item >> max(0, 5 - p.spread);
    shift ^= (shift >> p.spread) ^ (shift >> min(31, 2 * p.spread));
  }
  const int split = static_cast<int>((blockIdx.x + shift) % p.splits);
  const Rows rw = rows_of(p, item, R);
  if (rw.tokens == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int nb = blocks_seen(p, rw);
  // entries (blocks) of this chunk; the last chunk takes all that are left
  int entries = nb;
  if (p.blocks != nullptr) entries = nb > 0 ? list_selected(p, rw, nb, sh) : 0;
  const int e0 = split * p.chunk;
  const int e1 = split == p.splits - 1 ? entries : min(entries, e0 + p.chunk);
  if (e0 >= e1 && split > 0) {
    // nothing to add; a selection's chunks are all looked at by the join
    if (p.blocks != nullptr)
      for (int row = tid; row < rw.tokens * rw.heads; row += 256) {
        const int64_t at = (static_cast<int64_t>(item) * p.splits + split) * R + row;
        p.part_ml[at * 2] = -kInf;
        p.part_ml[at * 2 + 1] = 0.f;
      }
    return;
  }

  // rows: queries, limits
  u32x4 q[MT][D / 32];
  int limit[MT];
  int least = INT32_MAX;  // the smallest limit of the valid rows
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int row = t * 16 + n, tl = row / rw.heads, h = rw.head0 + row % rw.heads;
    const bool ok = tl < rw.tokens;
    const int64_t pos = rw.pos + tl;
    limit[t] = ok && rw.len > 0 ? static_cast<int>(pos < rw.len ? (pos < 0 ? -1 : pos) : rw.len - 1) : -1;
    if (ok) least = min(least, limit[t]);
    const char* from = static_cast<const char*>(p.q) + ((rw.first + (ok ? tl : 0)) * p.q_t + (ok ? h : rw.head0) * p.q_h + g * (D / 4)) * 2;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q[t][i] = ok ? *reinterpret_cast<const u32x4*>(from + i * 16) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) least = min(least, __shfl_xor(least, d));
  bool odd = false;  // NaNs of V were left out
  // the last key that any row sees
  const int most = static_cast<int>(rw.pos + rw.tokens - 1 < rw.len ? rw.pos + rw.tokens - 1 : rw.len - 1);

  // A weight is rounded once, to the type of q, relative to m: fp16 has no bits
  // below 2^-24, so there m stays 2^14 under the largest exponent and the weights
  // go up to 2^14 (bf16 has the exponents of fp32)
  constexpr float kRoom = __is_same(T, Fp16) ? 14.f : 0.f;
  f32x4 acc[MT][D / 16];
  float m[MT], sum[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    m[t] = -kInf;
    sum[t] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float c = p.scale * kLog2e;
  char* vt = sh.v[wave];
  const uint32_t vbase = lds_offset(vt);
  // transposing read: row (n >> 1) of the group's 8 keys, half row n & 1
  const uint32_t vrow = (n >> 1) < 4 ? 4 * g + (n >> 1) : 16 + 4 * g + (n >> 1) - 4;
  constexpr int kLoadsK = D / 64;              // 16-byte loads of a lane per 16 keys
  constexpr int kLoadsV = D / 32;              // of a lane per 32 keys
  constexpr int kLanesV = D / 16;              // lanes of a row of V

  struct Tile {
    u32x4 k[2][kLoadsK];
    u32x4 v[kLoadsV];
  };

  for (int s0 = e0; s0 < e1; s0 += kSeg) {
    const int ne = min(kSeg, e1 - s0);
    __syncthreads();
    if (tid < ne) {
      const int b = p.blocks != nullptr ? sh.list[s0 + tid] : s0 + tid;
      int pg = p.table[rw.seq * p.table_stride + b];
      if (pg < 0 || pg >= p.num_pages) pg = -1;
      const int64_t at = static_cast<int64_t>(pg < 0 ? 0 : pg) * p.kv_heads + rw.hk;
      sh.block[tid] = b;
      sh.page[tid] = pg;
      sh.ks[tid] = pg < 0 ? 0.f : p.k_scale[at];
      sh.vs[tid] = pg < 0 ? 1.f : fminf(fmaxf(p.v_scale[at], kLeast), kMost);
    }
    __syncthreads();
    const int tiles = ((ne << p.lb) + 31) >> 5;

    auto load = [&](int tile, Tile& x) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int a = tile * 32 + h * 16, e = min(a >> p.lb, ne - 1);
        const int64_t pg = max(0, sh.page[e]);
        const uint8_t* from = p.k + (((pg * p.kv_heads + rw.hk) << p.lb) + (a & (p.bs - 1)) + n) * D + g * (D / 4);
#pragma unroll
        for (int i = 0; i < kLoadsK; ++i) x.k[h][i] = *reinterpret_cast<const u32x4*>(from + i * 16);
      }
#pragma unroll
      for (int i = 0; i < kLoadsV; ++i) {
        const int row = i * (64 / kLanesV) + lane / kLanesV;
        const int a = tile * 32 + row, e = min(a >> p.lb, ne - 1);
        const int64_t pg = max(0, sh.page[e]);
        const uint8_t* from = p.v + (((pg * p.kv_heads + rw.hk) << p.lb) + (a & (p.bs - 1))) * D + (lane % kLanesV) * 16;
        x.v[i] = *reinterpret_cast<const u32x4*>(from);
      }
    };
    auto work = [&](int tile, const Tile& x) {
      // the two 16-key groups: first key, scales, whether they are there
      int key[2];
      float ck[2], lv[2], iv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int a = tile * 32 + h * 16, e = a >> p.lb;
        const bool there = e < ne && sh.page[min(e, ne - 1)] >= 0;
        const int ec = min(e, ne - 1);
        key[h] = there ? (sh.block[ec] << p.lb) + (a & (p.bs - 1)) : INT32_MAX - 64;
        ck[h] = sh.ks[ec] * c;
        const float vs = sh.vs[ec];
        lv[h] = __builtin_amdgcn_logf(vs);
        iv[h] = 1.f / vs;
      }
      const bool whole = max(key[0], key[1]) + 15 <= least;
      // V to LDS; codes that no row sees (behind the last token, never written,
      // or of a page that is not there) are set to 0, and so are NaNs that only
      // some rows see: 0 times them would reach the others
#pragma unroll
      for (int i = 0; i < kLoadsV; ++i) {
        const int row = i * (64 / kLanesV) + lane / kLanesV;
        u32x4 w = x.v[i];
        if (!whole) {
          const int at = (row < 16 ? key[0] : key[1]) + (row & 15);
          if (at > most) w = u32x4{0, 0, 0, 0};
          if (rw.tokens > 1 && at > rw.pos)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t nan = ((w[z] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              w[z] &= ~((nan >> 7) * 0xffu);
              odd |= nan != 0;
            }
        }
        *reinterpret_cast<u32x4*>(vt + v_at<D>(row, lane % kLanesV)) = w;
      }
      f32x4 s[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[t][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kLoadsK; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const u32x4 a = widen<T>(u32x2{x.k[h][i][2 * y], x.k[h][i][2 * y + 1]});
#pragma unroll
            for (int t = 0; t < MT; ++t) s[t][h] = T::mfma16(a, q[t][2 * i + y], s[t][h]);
          }
      u32x4 pr[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float top = -kInf;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float y = fmaf(s[t][h][r], ck[h], lv[h]);
            if (!whole && key[h] + 4 * g + r > limit[t]) y = -kInf;
            s[t][h][r] = y;
            top = fmaxf(top, y);
          }
        top = quad_max(top) - kRoom;
        if (__any(top > m[t])) {
          const float now = fmaxf(m[t], top);
          const float shrink = now == -kInf ? 1.f : exp2_fast(m[t] - now);
          m[t] = now;
          sum[t] *= shrink;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][i][r] *= shrink;
        }
        const float base = m[t] == -kInf ? 0.f : m[t];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = exp2_fast(s[t][h][r] - base);
          sum[t] = fmaf((w[0] + w[1]) + (w[2] + w[3]), iv[h], sum[t]);
          pr[t][2 * h] = T::pack(w[0], w[1]);
          pr[t][2 * h + 1] = T::pack(w[2], w[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t at = vbase + v_at<D>(vrow, i) + (n & 1) * 8;
        const u32x4 a = widen<T>(lds_read_tr8(at));
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t][i] = T::mfma16(a, pr[t], acc[t][i]);
      }
    };

    Tile x, y;
    int tile = wave;
    if (tile < tiles) load(tile, x);
    for (; tile < tiles; tile += 8) {
      if (tile + 4 < tiles) load(tile + 4, y);
      work(tile, x);
      if (tile + 4 < tiles) {
        if (tile + 8 < tiles) load(tile + 8, x);
        work(tile + 4, y);
      }
    }
  }

  // NaNs of V among the new tokens' keys that were left out: to the rows that see them
  if (rw.tokens > 1 && __syncthreads_or(odd) && wave == 0) {
    const int64_t to = min(static_cast<int64_t>(most), (static_cast<int64_t>(e1) << p.lb) - 1);
    for (int64_t key = max(max(rw.pos + 1, int64_t{0}), static_cast<int64_t>(e0) << p.lb); key <= to; ++key) {
      const int64_t pg = p.table[rw.seq * p.table_stride + (key >> p.lb)];
      if (pg < 0 || pg >= p.num_pages) continue;
      const uint8_t* from = p.v + (((pg * p.kv_heads + rw.hk) << p.lb) + (key & (p.bs - 1))) * D + 4 * g;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(from + i * 16);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (key <= limit[t] && ((w >> (8 * r)) & 0x7fu) == 0x7fu) acc[t][i][r] = __builtin_nanf("");
      }
    }
  }
  // Join the wavefronts: rows' maxima and sums, then 16 rows at a time.
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    sum[t] = quad_sum(sum[t]);
    if (g == 0) {
      sh.ml[wave][t * 16 + n][0] = m[t];
      sh.ml[wave][t * 16 + n][1] = sum[t];
    }
  }
  __syncthreads();
  const int rows = rw.tokens * rw.heads;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (t * 16 >= rows) break;
    float top = -kInf;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, sh.ml[w][t * 16 + n][0]);
    const float f = top == -kInf ? 0.f : exp2_fast(m[t] - top);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      *reinterpret_cast<f32x4*>(&sh.join[wave][n][i * 16 + 4 * g]) = f32x4{acc[t][i][0] * f, acc[t][i][1] * f, acc[t][i][2] * f, acc[t][i][3] * f};
    __syncthreads();
    for (int e = tid; e < 16 * D / 4; e += 256) {
      const int r = e / (D / 4), d = (e % (D / 4)) * 4, row = t * 16 + r;
      if (row >= rows) continue;
      f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
      float mm = -kInf, l = 0.f;
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sh.ml[w][row][0]);
      for (int w = 0; w < 4; ++w) {
        o += *reinterpret_cast<const f32x4*>(&sh.join[w][r][d]);
        l += sh.ml[w][row][1] * (mm == -kInf ? 0.f : exp2_fast(sh.ml[w][row][0] - mm));
      }
      if (p.splits > 1) {
        const int64_t at = (static_cast<int64_t>(item) * p.splits + split) * R + row;
        *reinterpret_cast<f32x4*>(p.part + at * D + d) = o;
        if (d == 0) {
          p.part_ml[at * 2] = mm;
          p.part_ml[at * 2 + 1] = l;
        }
      } else {
        const int64_t tok = rw.first + row / rw.heads, h = rw.head0 + row % rw.heads;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        u32x2 w2;
        w2[0] = T::pack(o[0] * inv, o[1] * inv);
        w2[1] = T::pack(o[2] * inv, o[3] * inv);
        *reinterpret_cast<u32x2*>(static_cast<char*>(p.out) + ((tok * p.heads + h) * D + d) * 2) = w2;
        if (d == 0) p.lse[tok * p.heads + h] = l == 0.f ? -kInf : (mm + __builtin_amdgcn_logf(l)) * kLn2;
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of a workgroup's rows: one wavefront a row (12300 rows of up
// to 8 chunks: 13 us), or four that share the chunks of a row and are added up in
// order (kFour; 90 rows of up to 157: 5.5 us, by one wavefront 9).
template <typename T, int D, bool kFour>
__global__ void __launch_bounds__(256) kv8_join_kernel(DecodeArgs p, int rows_per) {
  __shared__ float s_o[4][D], s_l[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t index = kFour ? blockIdx.x : blockIdx.x * 4 + wave;
  const int64_t item = index / rows_per;
  const int row = static_cast<int>(index % rows_per);
  if (item >= p.slots * p.kv_heads * p.head_chunks) return;
  const Rows rw = rows_of(p, item, rows_per);
  if (row >= rw.tokens * rw.heads) return;
  const int nb = blocks_seen(p, rw);
  // chunks that were written: all of a selection's, those of a sequence's blocks
  const int used = p.blocks != nullptr ? p.splits : min(p.splits, max(1, (nb + p.chunk - 1) / p.chunk));
  const int64_t at = item * p.splits * rows_per + row;
  float top = -kInf;
  for (int s = lane; s < used; s += 64) top = fmaxf(top, p.part_ml[(at + static_cast<int64_t>(s) * rows_per) * 2]);
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float from = top == -kInf ? 0.f : top;
  float l = 0.f, o[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) o[i] = 0.f;
  // 64 chunks at a time: a lane works out the weight of one, then all add the
  // chunks' values, eight loads in flight.  A chunk that added nothing may not
  // have written any (-1); one whose weight is 0 beside the others' has, and 0
  // times its NaN counts.
  const int share = kFour ? (used + 3) / 4 : used, end = min(used, (kFour ? wave + 1 : 1) * share);
  for (int s0 = kFour ? wave * share : 0; s0 < end; s0 += 64) {
    const int n = min(64, end - s0);
    float f = -1.f;
    if (lane < n) {
      const int64_t a = at + static_cast<int64_t>(s0 + lane) * rows_per;
      const float ll = p.part_ml[a * 2 + 1];
      f = ll == 0.f ? -1.f : exp2_fast(p.part_ml[a * 2] - from);
      l += ll * (ll == ll ? f : 1.f);
    }
    const float* values = p.part + (at + static_cast<int64_t>(s0) * rows_per) * D + lane * (D / 64);
    for (int s = 0; s < n; s += 8) {
      float x[8][D / 64];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) x[u][i] = values[static_cast<int64_t>(min(s + u, n - 1)) * rows_per * D + i];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s + u));  // -1 from n on
#pragma unroll
        for (int i = 0; i < D / 64; ++i) o[i] += fs < 0.f ? 0.f : x[u][i] * fs;
      }
    }
  }
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  if constexpr (kFour) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) s_o[wave][lane * (D / 64) + i] = o[i];
    if (lane == 0) s_l[wave] = l;
    __syncthreads();
    if (wave > 0) return;
    l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int d = lane * (D / 64) + i;
      o[i] = (s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d]);
    }
  }
  const int64_t tok = rw.first + row / rw.heads, h = rw.head0 + row % rw.heads;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* to = static_cast<char*>(p.out) + ((tok * p.heads + h) * D + lane * (D / 64)) * 2;
  if constexpr (D == 128) *reinterpret_cast<uint32_t*>(to) = T::pack(o[0] * inv, o[1] * inv);
  else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(T::pack(o[0] * inv, 0.f));
  if (lane == 0) p.lse[tok * p.heads + h] = l == 0.f ? -kInf : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int D>
int launch_decode(const DecodeArgs& p, int mt, hipStream_t stream) {
  const int64_t items = p.slots * p.kv_heads * p.head_chunks;
  const int64_t grid = items * p.splits;
  if (grid > INT32_MAX) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid));
  if (mt == 1) kv8_attention_kernel<T, D, 1><<<g, dim3(256), 0, stream>>>(p);
  else if (mt == 2) kv8_attention_kernel<T, D, 2><<<g, dim3(256), 0, stream>>>(p);
  else kv8_attention_kernel<T, D, 4><<<g, dim3(256), 0, stream>>>(p);
  if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  if (p.splits > 1) {
    const int64_t rows = items * mt * 16;
    const bool four = p.splits > 16;
    const int64_t joins = four ? rows : (rows + 3) / 4;
    if (joins > INT32_MAX / 4) return MI_ATTN_EINVAL;
    const dim3 jg(static_cast<unsigned>(joins));
    if (four) kv8_join_kernel<T, D, true><<<jg, dim3(256), 0, stream>>>(p, mt * 16);
    else kv8_join_kernel<T, D, false><<<jg, dim3(256), 0, stream>>>(p, mt * 16);
    if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  }
  return MI_ATTN_OK;
}

struct Plan {
  int mt, tokens_per, head_chunks, splits, chunk, spread;
  int64_t slots, items;
  uint64_t bytes;
};

// Rows: as many tiles of 16 as the rows that share their keys fill (all new
// tokens of a sequence where it reads its whole cache; one token's heads where
// each token selects its own blocks), 64 at most.  Chunks: about four
// workgroups for each of the 256 compute units, chunks of 128 keys at least
// and 4096 at most, so that long and short sequences of a batch even out; longer
// ones where the chunks' partial results would pass kMostRows rows: there are
// many workgroups then, and the results would outgrow the output many times
// (8192 tokens, 64/8 heads, a table for 131072 keys: 8.7 GB).
constexpr int64_t kMostRows = 1 << 19;

Plan make_plan(const mi_kv8_attention_args* a) {
  Plan p;
  const int group = a->heads / a->kv_heads;
  const bool sparse = a->blocks != nullptr;
  const int64_t tokens = sparse || a->num_seqs == 0 ? 1 : (a->total_q + a->num_seqs - 1) / a->num_seqs;
  const int64_t rows = tokens * group;
  p.mt = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  p.tokens_per = sparse || p.mt * 16 < group ? 1 : p.mt * 16 / group;
  if (a->cu == nullptr) p.tokens_per = 1;
  p.head_chunks = (group + p.mt * 16 - 1) / (p.mt * 16);
  p.slots = slots_of(a->total_q, a->num_seqs, p.tokens_per);
  p.items = p.slots * a->kv_heads * p.head_chunks;
  int64_t most = a->max_length / a->block_size + (a->max_length % a->block_size != 0);
  if (most > a->block_table_cols) most = a->block_table_cols;
  if (sparse && most > a->select) most = a->select;
  if (most < 1) most = 1;
  const int64_t least = 128 / a->block_size < 1 ? 1 : 128 / a->block_size, top = 4096 / a->block_size;
  const int64_t want = p.items > 0 ? (1024 + p.items - 1) / p.items : 1;  // chunks of an item
  int64_t chunk = (most + want - 1) / want;
  chunk = chunk < least ? least : (chunk > top ? top : chunk);
  // sequences of few tokens leave up to half of the slots empty: with a multiple of
  // 32 workgroups a slot those do not fall on the same engines
  int64_t splits_most = 1;
  if (p.tokens_per > 1 && p.slots < 8 * static_cast<int64_t>(a->num_seqs))
    while (splits_most < 32 && (a->kv_heads * p.head_chunks * splits_most) % 32 != 0) splits_most *= 2;
  while (p.items > 0 && p.items * p.mt * 16 * splits_most * 2 <= kMostRows) splits_most *= 2;
  p.spread = -1;
  if (chunk * splits_most < most) {
    chunk = (most + splits_most - 1) / splits_most;
    p.spread = (most + chunk - 1) / chunk == splits_most ? __builtin_ctz(static_cast<unsigned>(splits_most)) : -1;
  }
  p.chunk = static_cast<int>(chunk);
  p.splits = static_cast<int>((most + chunk - 1) / chunk);
  p.bytes = p.splits > 1 ? static_cast<uint64_t>(p.items) * p.splits * p.mt * 16 * (a->dim + 2) * 4 : 0;
  return p;
}

int check_decode(const mi_kv8_attention_args* a) {
  if (a == nullptr) return MI_ATTN_EINVAL;
  if ((a->dtype != MI_ATTN_BF16 && a->dtype != MI_ATTN_FP16) || (a->dim != 64 && a->dim != 128) ||
      (a->block_size != 16 && a->block_size != 32 && a->block_size != 64 && a->block_size != 128) || a->kv_heads < 1 ||
      a->heads < a->kv_heads || a->heads % a->kv_heads || a->heads / a->kv_heads > 128 || a->total_q < 0 ||
      a->total_q > INT32_MAX || a->num_pages < 0 || a->num_pages > INT32_MAX || a->num_seqs < 0 || a->block_table_cols < 0 ||
      a->block_table_stride < a->block_table_cols || (a->cu == nullptr && a->total_q != a->num_seqs) || a->max_length < 0 ||
      (static_cast<int64_t>(a->block_table_cols) * a->block_size >= (1 << 30)) || !(a->scale > 0.f) || !(a->scale < kInf) ||
      a->q_stride_t < 0 || a->q_stride_h < 0 || ((a->q_stride_t | a->q_stride_h) & 7) ||
      (a->blocks != nullptr && (a->select < 1 || a->select > MI_ATTN_MAX_SELECT)))
    return MI_ATTN_EINVAL;
  return MI_ATTN_OK;
}

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT uint64_t kv8_attention_workspace(const mi_kv8_attention_args* args) {
  return check_decode(args) == MI_ATTN_OK ? make_plan(args).bytes : 0;
}

MI_ATTN_EXPORT int kv8_attention(const mi_kv8_attention_args* a, hipStream_t stream) {
  const int st = check_decode(a);
  if (st != MI_ATTN_OK) return st;
  const void* wide[] = {a->q, a->k_cache, a->v_cache, a->out, a->workspace};
  for (const void* x : wide)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return MI_ATTN_EINVAL;
  const void* words[] = {a->k_scale, a->v_scale, a->block_table, a->lengths, a->cu, a->blocks, a->lse};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MI_ATTN_EINVAL;
  if (a->total_q == 0) return MI_ATTN_OK;
  if (a->q == nullptr || a->out == nullptr || a->lse == nullptr || (a->num_seqs > 0 && a->lengths == nullptr)) return MI_ATTN_EINVAL;
  if (a->num_seqs > 0 && a->block_table_cols > 0 && a->block_table == nullptr) return MI_ATTN_EINVAL;
  if (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr || a->k_scale == nullptr || a->v_scale == nullptr)) return MI_ATTN_EINVAL;
  const Plan plan = make_plan(a);
  if (plan.bytes > 0 && (a->workspace == nullptr || a->workspace_bytes < plan.bytes)) return MI_ATTN_EWORKSPACE;
  DecodeArgs p;
  p.q = a->q; p.k = static_cast<const uint8_t*>(a->k_cache); p.v = static_cast<const uint8_t*>(a->v_cache);
  p.k_scale = a->k_scale; p.v_scale = a->v_scale; p.table = a->block_table; p.lengths = a->lengths; p.cu = a->cu;
  p.blocks = a->blocks; p.out = a->out; p.lse = a->lse;
  p.part = static_cast<float*>(a->workspace);
  p.part_ml = p.part == nullptr ? nullptr : p.part + plan.items * plan.splits * plan.mt * 16 * a->dim;
  p.q_t = a->q_stride_t; p.q_h = a->q_stride_h; p.total_q = a->total_q; p.num_pages = a->num_pages;
  p.table_stride = a->block_table_stride; p.slots = plan.slots;
  // without pages nothing can be seen
  p.table_cols = a->num_pages > 0 ? a->block_table_cols : 0;
  p.num_seqs = a->num_seqs; p.heads = a->heads; p.kv_heads = a->kv_heads; p.group = a->heads / a->kv_heads;
  p.bs = a->block_size; p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size));
  p.select = a->select; p.tokens_per = plan.tokens_per; p.head_chunks = plan.head_chunks; p.splits = plan.splits;
  p.chunk = plan.chunk; p.spread = plan.spread; p.scale = a->scale;
  if (a->dtype == MI_ATTN_BF16)
    return a->dim == 128 ? launch_decode<Bf16, 128>(p, plan.mt, stream) : launch_decode<Bf16, 64>(p, plan.mt, stream);
  return a->dim == 128 ? launch_decode<Fp16, 128>(p, plan.mt, stream) : launch_decode<Fp16, 64>(p, plan.mt, stream);
}
