// Attention of a chunk of new tokens behind the 8-bit paged cache.
//
//   out = sum_j p_j v_j,  p = softmax(scale q . k_j)
//
// over the context's codes (k_j = code * k_scale of its page, v_j likewise) and
// the new tokens' own 16-bit rows.  A workgroup takes 32 rows a wavefront of one
// key head: consecutive tokens with the query heads that share the key head.  It
// walks over the keys 64 at a time: the context's codes become 16-bit elements
// exactly, once for the workgroup, on their way to LDS; the new tokens' rows are
// copied.  Where few rows leave the card empty the walk is split and a second
// kernel joins the parts.
//
// Scores are computed as K Q^T, so that a query's scores lie in two lanes and the
// weights are the second product's operand as they stand.  A page's K scale
// multiplies its scores; its V scale joins the exponent: the running maximum is
// that of x = s + log2 s_v, the weights are 2^(x - max), and the sum of the
// probabilities adds a page's weights divided by s_v.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_chunk.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

constexpr int kSeg = 256;     // blocks whose page numbers and scales are in LDS at a time
constexpr int kSplits = 64;   // parts of a walk, at most
// V scales are held between these: 2^30 weights of up to 2^15, divided by the
// least, stay within fp32
constexpr float kLeast = 0x1p-80f, kMost = 0x1p100f;

struct ChunkArgs {
  const char* q;
  const char* x[2];          // the new tokens' keys and values
  const uint8_t* cache[2];
  const float* scales[2];
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* cu;
  char* out;
  float* lse;
  float* part;               // [workgroup][row][D], then [workgroup][row][2]
  float* part_ml;
  int64_t q_t, q_h, x_t[2], x_h[2], total, num_pages, table_stride, slots;
  int32_t table_cols, num_seqs, heads, kv_heads, group, bs, lb, tokens_per, splits, chunk;
  float scale;
};

// The rows of a workgroup and the keys that they can see.
struct ChunkRows {
  int seq, tokens;    // sequence; tokens of this workgroup
  int n, r0;          // tokens of the chunk; the number of the first one here
  int64_t begin;      // the chunk's first row
  int context;        // keys in pages
  int hidden;         // new tokens that would stand before the sequence's start
  int tiles_context, first_new, tiles;  // tiles of 64 keys: of the context; the first of the new tokens; all
};

__device__ __forceinline__ ChunkRows rows_of(const ChunkArgs& p, int64_t slot) {
  int32_t len, none;
  const Place at = place_of(p.cu, p.num_seqs, p.total, slot, p.tokens_per, [&](int i) { return i < p.num_seqs ? p.lengths[i] : 0; }, len, none);
  ChunkRows r;
  r.seq = at.seq;
  r.begin = at.begin;
  const int64_t left = at.end - at.first;
  r.tokens = static_cast<int>(left < 0 ? 0 : (left < p.tokens_per ? left : p.tokens_per));
  r.n = static_cast<int>(at.end - at.begin);
  r.r0 = static_cast<int>(at.first - at.begin);
  int64_t context = static_cast<int64_t>(len) - r.n;
  if (at.seq >= p.num_seqs) context = -static_cast<int64_t>(r.n);  // rows behind the last sequence see nothing
  r.hidden = static_cast<int>(context < 0 ? (-context < r.n ? -context : r.n) : 0);
  const int64_t most = static_cast<int64_t>(p.table_cols) << p.lb;
  r.context = static_cast<int>(context < 0 ? 0 : (context < most ? context : most));
  r.tiles_context = (r.context + kTile - 1) / kTile;
  r.first_new = r.hidden / kTile;
  const int last = (r.r0 + r.tokens + kTile - 1) / kTile;
  r.tiles = r.tiles_context + (r.r0 + r.tokens > r.hidden ? last - r.first_new : 0);
  return r;
}

template <typename T>
__device__ __forceinline__ uint32_t finite_only(uint32_t w, bool& odd) {
  constexpr uint32_t e = __is_same(T, Bf16) ? 0x7f80u : 0x7c00u;
  if ((w & e) == e) {
    w &= 0xffff0000u;
    odd = true;
  }
  if ((w & (e << 16)) == (e << 16)) {
    w &= 0xffffu;
    odd = true;
  }
  return w;
}

// A tile of the context on its way to LDS: 64 keys' codes and 64 values' over
// NW wavefronts, in registers while the tile before it is worked on.
template <typename T, int D, int NW, bool kWide>
struct Codes {
  static constexpr int kThreads = NW * 64, kLanes = D / 16, kHalf = kTile * kLanes, kUnits = 2 * kHalf / kThreads;
  static_assert(kUnits * kThreads == 2 * kHalf, "");
  u32x4 x[kUnits];

  // `at`: the tile's first key, from the first of the ne blocks that pages[] is of;
  // blocks behind the last one stand for it.
  __device__ __forceinline__ void load(const ChunkArgs& p, int hk, const int32_t* pages, int ne, int at) {
    const int tid = threadIdx.x;
    int64_t base = 0;
    if constexpr (kWide) {
      const int64_t pg = max(0, __builtin_amdgcn_readfirstlane(pages[min(at >> p.lb, ne - 1)]));
      base = (((pg * p.kv_heads + hk) << p.lb) + (at & (p.bs - 1))) * D;
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = j * kThreads + tid, is_v = u / kHalf;
      const int row = (u / kLanes) % kTile, chunk = u % kLanes;
      if constexpr (!kWide) {
        const int a = at + row;
        const int64_t pg = max(0, pages[min(a >> p.lb, ne - 1)]);
        base = (((pg * p.kv_heads + hk) << p.lb) + ((a & (p.bs - 1)) - row)) * D;
      }
      x[j] = *reinterpret_cast<const u32x4*>(p.cache[is_v] + (base + (row * D + chunk * 16)));
    }
  }
  // `left`: keys of the tile that there are; the others, and those of pages that
  // are not there, become 0.
  __device__ __forceinline__ void store(const ChunkArgs& p, char* k, char* v, const int32_t* pages, int ne, int at, int left) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = j * kThreads + tid;
      const int row = (u / kLanes) % kTile, chunk = u % kLanes;
      u32x4 c = x[j];
      const int e = (at + (kWide ? 0 : row)) >> p.lb;
      if (row >= left || e >= ne || pages[min(e, ne - 1)] < 0) c = u32x4{0, 0, 0, 0};
      char* to = u / kHalf ? v : k;
      *reinterpret_cast<u32x4*>(to + tile_at<D>(row, 2 * chunk)) = widen<T>(u32x2{c[0], c[1]});
      *reinterpret_cast<u32x4*>(to + tile_at<D>(row, 2 * chunk + 1)) = widen<T>(u32x2{c[2], c[3]});
    }
  }
};

// A tile of the new tokens likewise.
template <typename T, int D, int NW>
struct Fresh {
  static constexpr int kThreads = NW * 64, kLanes = D / 8, kHalf = kTile * kLanes, kUnits = 2 * kHalf / kThreads;
  u32x4 x[kUnits];

  // rows behind the chunk's last one stand for it
  __device__ __forceinline__ void load(const ChunkArgs& p, int hk, const ChunkRows& rw, int first) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = j * kThreads + tid, is_v = u / kHalf;
      const int row = (u / kLanes) % kTile, chunk = u % kLanes;
      const int64_t token = rw.begin + min(first + row, rw.n - 1);
      x[j] = *reinterpret_cast<const u32x4*>(p.x[is_v] + (token * p.x_t[is_v] + hk * p.x_h[is_v]) * 2 + chunk * 16);
    }
  }
  // hide: some row does not see all of the tile, so that infinities and NaN among
  // the values become 0 and are marked
  __device__ __forceinline__ void store(char* k, char* v, bool hide, bool& odd) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = j * kThreads + tid;
      const int row = (u / kLanes) % kTile, chunk = u % kLanes;
      u32x4 c = x[j];
      if (hide && u / kHalf) {
#pragma unroll
        for (int z = 0; z < 4; ++z) c[z] = finite_only<T>(c[z], odd);
      }
      *reinterpret_cast<u32x4*>((u / kHalf ? v : k) + tile_at<D>(row, chunk)) = c;
    }
  }
};

template <int D>
struct ChunkShared {
  char k[2][kTile * 2 * D];
  char v[2][kTile * 2 * D];
  int32_t page[kSeg];  // -1: not there
  float ks[kSeg], lv[kSeg], iv[kSeg];
};

// A row's output from lane half `half`, which has the columns 32 i + 8 (r / 4) +
// 4 half + r % 4 in acc[i][r].
template <typename T, int D>
__device__ __forceinline__ void store_chunk_row(const ChunkArgs& p, int64_t tok, int head, int half, const f32x16 (&acc)[D / 32], float base, float sum, bool sees) {
  const float inv = sum == 0.f || !sees ? 0.f : 1.f / sum;
  char* to = p.out + (tok * p.heads + head) * (2 * D) + half * 8;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      u32x2 w;
      w[0] = T::pack(acc[i][r] * inv, acc[i][r + 1] * inv);
      w[1] = T::pack(acc[i][r + 2] * inv, acc[i][r + 3] * inv);
      *reinterpret_cast<u32x2*>(to + i * 64 + (r >> 2) * 16) = sees ? w : u32x2{0, 0};
    }
  if (half == 0) p.lse[tok * p.heads + head] = !sees || sum == 0.f ? -kInf : (base == kInf ? kInf : (base + __builtin_amdgcn_logf(sum)) * kLn2);
}

template <typename T, int D, bool kWide, int NW>
__global__ void __launch_bounds__(NW * 64, 2) chunk_attention_kernel(ChunkArgs p) {
  constexpr int kRowsHere = NW * 32;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  ChunkShared<D>& sh = *reinterpret_cast<ChunkShared<D>*>(smem);
  const int hk = blockIdx.x % p.kv_heads;
  const uint32_t rest = blockIdx.x / p.kv_heads;
  const int split = static_cast<int>(rest % p.splits);
  // later rows see more keys: they start first
  const int64_t slot = p.slots - 1 - static_cast<int64_t>(rest / p.splits);
  const ChunkRows rw = rows_of(p, slot);
  if (rw.tokens == 0) return;
  const int e0 = min(rw.tiles, split * p.chunk), e1 = split == p.splits - 1 ? rw.tiles : min(rw.tiles, e0 + p.chunk);
  if (e0 >= e1 && split > 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, row = wave * 32 + (lane & 31);
  const int tl = row / p.group, head = hk * p.group + row % p.group;
  const bool valid = tl < rw.tokens;
  const int mine = rw.r0 + (valid ? tl : 0);  // the row's token among the chunk's
  const bool sees = valid && mine >= rw.hidden;
  const int64_t tok = rw.begin + mine;

  u32x4 q[D / 16];
  {
    const char* from = p.q + (tok * p.q_t + (valid ? head : hk * p.group) * p.q_h) * 2 + half * 16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = valid ? *reinterpret_cast<const u32x4*>(from + i * 32) : u32x4{0, 0, 0, 0};
  }
  f32x16 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  float m = -kInf, sum = 0.f;
  const float c = p.scale * kLog2e;
  const Reads<D> rd(lds_offset(sh.k[0]));
  constexpr int kBuf = kTile * 2 * D;  // from one buffer to the other; the values lie two behind the keys
  // A weight is rounded once, to the type of q.  fp16 has no bits below 2^-24, so
  // there the weights are relative to a maximum 2^12 below the row's, and with the
  // 2^3 that this may lag behind they go up to 2^15 (bf16 has fp32's exponents)
  constexpr float kLag = __is_same(T, Fp16) ? 3.f : 8.f, kLower = __is_same(T, Fp16) ? 12.f : 0.f;
  constexpr int kScales = kWide ? 1 : 4;

  // One tile, in LDS buffer `buf`.  A row sees its keys low .. high, of the 16-key
  // groups whose bit is set in `groups`; `part`: some row sees a part only.
  auto work = [&](auto which, bool part, int low, int high, int groups, const float (&ck)[kScales], const float (&lv)[kScales],
                  const float (&iv)[kScales]) {
    constexpr int buf = decltype(which)::value;
    f32x16 s[2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[mt][r] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) s[mt] = T::mfma32(rd.row(buf * kBuf, mt * 32, i), q[i], s[mt]);
    }
    if (part) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int at = 32 * mt + 8 * (r >> 2) + (r & 3) + 4 * half;
          if (at < low || at > high || !((groups >> (2 * mt + (r >> 3))) & 1)) s[mt][r] = -kInf;
        }
    }
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t = s[i >> 1][8 * (i & 1)];
#pragma unroll
      for (int r = 1; r < 8; ++r) t = fmaxf(t, s[i >> 1][8 * (i & 1) + r]);
      if constexpr (!kWide) top = fmaxf(top, fmaf(t, ck[i], lv[i]));
      else top = fmaxf(top, t);
    }
    if constexpr (kWide) top = fmaf(top, ck[0], lv[0]);
    top = half_max(top);
    if (__any(top - m > kLag)) {
      const float now = fmaxf(m, top);
      const float shrink = now == -kInf ? 1.f : exp2_fast(m - now);
      m = now;
      sum *= shrink;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] *= shrink;
    }
    const float base = m == -kInf ? 0.f : m - kLower;
    u32x4 pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float cki = ck[kWide ? 0 : i], from = lv[kWide ? 0 : i] - base;
      float w[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = exp2_fast(fmaf(s[i >> 1][8 * (i & 1) + r], cki, from));
#pragma unroll
      for (int r = 0; r < 4; ++r) pr[i][r] = T::pack(w[2 * r], w[2 * r + 1]);
      sum = fmaf(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])), iv[kWide ? 0 : i], sum);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int st = 0; st < 4; ++st) acc[i] = T::mfma32(rd.column((2 + buf) * kBuf, 16 * st, i), pr[st], acc[i]);
  };

  // The context, kSeg blocks' tiles at a time.
  const int c1 = min(e1, rw.tiles_context);
  for (int s0 = e0; s0 < c1;) {
    // (a part can begin inside a block of 128 keys)
    const int block0 = (s0 * kTile) >> p.lb, shift = s0 * kTile - (block0 << p.lb);
    const int blocks = (rw.context + p.bs - 1) >> p.lb;
    const int s1 = min(c1, (((block0 + kSeg) << p.lb) / kTile));
    const int ne = min(kSeg, blocks - block0);
    __syncthreads();
    for (int b = tid; b < ne; b += NW * 64) {
      int pg = p.table[rw.seq * p.table_stride + block0 + b];
      if (pg < 0 || pg >= p.num_pages) pg = -1;
      const int64_t at = static_cast<int64_t>(max(0, pg)) * p.kv_heads + hk;
      const float vs = pg < 0 ? 1.f : fminf(fmaxf(p.scales[1][at], kLeast), kMost);
      sh.page[b] = pg;
      sh.ks[b] = pg < 0 ? 1.f : fmaxf(p.scales[0][at] * c, 0x1p-149f);
      sh.lv[b] = __builtin_amdgcn_logf(vs);
      sh.iv[b] = 1.f / vs;
    }
    __syncthreads();
    Codes<T, D, NW, kWide> in;
    auto at_of = [&](int t) { return (t - s0) * kTile + shift; };
    auto left_of = [&](int t) { return rw.context - t * kTile; };
    in.load(p, hk, sh.page, ne, at_of(s0));
    in.store(p, sh.k[0], sh.v[0], sh.page, ne, at_of(s0), left_of(s0));
    in.load(p, hk, sh.page, ne, at_of(min(s0 + 1, s1 - 1)));
    __syncthreads();
    auto step = [&](auto which, int t) {
      constexpr int buf = decltype(which)::value;
      float ck[kScales], lv[kScales], iv[kScales];
      int groups = 0;
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int e = min((at_of(t) + 16 * i) >> p.lb, ne - 1);
        ck[i] = sh.ks[e];
        lv[i] = sh.lv[e];
        iv[i] = sh.iv[e];
        groups |= (sh.page[e] >= 0 ? 1 : 0) << i;
      }
      groups = __builtin_amdgcn_readfirstlane(groups);
      if (kWide && groups) groups = 15;
      const int left = left_of(t), next = min(t + 1, s1 - 1);
      if (groups != 0) work(which, left < kTile || groups != 15, 0, left - 1, groups, ck, lv, iv);
      in.store(p, sh.k[buf ^ 1], sh.v[buf ^ 1], sh.page, ne, at_of(next), left_of(next));
      in.load(p, hk, sh.page, ne, at_of(min(t + 2, s1 - 1)));
    };
    for (int t = s0; t < s1; t += 2) {
      step(Int<0>{}, t);
      __syncthreads();
      if (t + 1 < s1) {
        step(Int<1>{}, t + 1);
        __syncthreads();
      }
    }
    s0 = s1;
  }

  // The new tokens.
  const int n0 = max(e0, rw.tiles_context);
  bool odd = false;
  const int least = max(rw.r0, rw.hidden);  // the first token here that sees anything
  auto first_of = [&](int t) { return (rw.first_new + t - rw.tiles_context) * kTile; };
  auto hides = [&](int t) { return first_of(t) + kTile - 1 > least || first_of(t) < rw.hidden; };
  if (n0 < e1) {
    Fresh<T, D, NW> in;
    in.load(p, hk, rw, first_of(n0));
    __syncthreads();
    in.store(sh.k[0], sh.v[0], hides(n0), odd);
    in.load(p, hk, rw, first_of(min(n0 + 1, e1 - 1)));
    __syncthreads();
    auto step = [&](auto which, int t) {
      constexpr int buf = decltype(which)::value;
      const float ones[4] = {1.f, 1.f, 1.f, 1.f}, zeros[4] = {0.f, 0.f, 0.f, 0.f}, cs[4] = {c, c, c, c};
      float ck[kScales], lv[kScales], iv[kScales];
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        ck[i] = cs[i];
        lv[i] = zeros[i];
        iv[i] = ones[i];
      }
      const int first = first_of(t), high = sees ? mine - first : -1, next = min(t + 1, e1 - 1);
      if (__any(high >= 0)) work(which, hides(t), rw.hidden - first, high, 15, ck, lv, iv);
      in.store(sh.k[buf ^ 1], sh.v[buf ^ 1], hides(next), odd);
      in.load(p, hk, rw, first_of(min(t + 2, e1 - 1)));
    };
    for (int t = n0; t < e1; t += 2) {
      step(Int<0>{}, t);
      __syncthreads();
      if (t + 1 < e1) {
        step(Int<1>{}, t + 1);
        __syncthreads();
      }
    }
  }
  // Infinities and NaN among the values that were left out, to the rows that see them
  if (__syncthreads_or(odd)) {
    for (int t = n0; t < e1; ++t) {
      if (!hides(t)) continue;
      const int from = max(first_of(t), rw.hidden), to = min(first_of(t) + kTile, rw.r0 + rw.tokens);
      for (int key = from; key < to; ++key) {
        const char* v = p.x[1] + ((rw.begin + key) * p.x_t[1] + hk * p.x_h[1]) * 2 + half * 8;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(v + i * 64 + (r >> 2) * 16 + (r & 2) * 2);
            const float a = T::lo(w), b = T::hi(w);
            if (sees && key <= mine) {
              if (!(fabsf(a) < kInf)) acc[i][r] += a;
              if (!(fabsf(b) < kInf)) acc[i][r + 1] += b;
            }
          }
      }
    }
  }
  sum = half_sum(sum);
  const float base = m - kLower;
  if (!valid) return;
  if (p.splits == 1) {
    store_chunk_row<T, D>(p, tok, head, half, acc, base, sum, sees);
    return;
  }
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kRowsHere + row;
  float* to = p.part + at * D + 4 * half;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<f32x4*>(to + i * 32 + 2 * r) = f32x4{acc[i][r], acc[i][r + 1], acc[i][r + 2], acc[i][r + 3]};
  if (half == 0) {
    p.part_ml[at * 2] = base;
    p.part_ml[at * 2 + 1] = sum;
  }
}

// Joins the parts of a row's walk: one wavefront a row.
template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkArgs p, int rows_per) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t index = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int64_t item = index / rows_per;  // slot (from the last one) and key head
  const int row = static_cast<int>(index % rows_per);
  if (item >= p.slots * p.kv_heads) return;
  const int hk = static_cast<int>(item % p.kv_heads);
  const int64_t from_last = item / p.kv_heads;
  const ChunkRows rw = rows_of(p, p.slots - 1 - from_last);
  const int tl = row / p.group, head = hk * p.group + row % p.group;
  if (tl >= rw.tokens) return;
  const bool sees = rw.r0 + tl >= rw.hidden;
  const int used = min(p.splits, max(1, (rw.tiles + p.chunk - 1) / p.chunk));
  auto at = [&](int s) { return ((from_last * p.splits + s) * p.kv_heads + hk) * rows_per + row; };
  float base = -kInf, l = 0.f;
  if (lane < used) {
    base = p.part_ml[at(lane) * 2];
    l = p.part_ml[at(lane) * 2 + 1];
  }
  float top = base;
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float f = base == -kInf ? 0.f : exp2_fast(base - top);
  l *= f;
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  float o[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) o[i] = 0.f;
  for (int s = 0; s < used; ++s) {
    const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] += p.part[at(s) * D + lane * (D / 64) + i] * fs;
  }
  const int64_t tok = rw.begin + rw.r0 + tl;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* to = p.out + ((tok * p.heads + head) * D + lane * (D / 64)) * 2;
  if constexpr (D == 128) *reinterpret_cast<uint32_t*>(to) = sees ? T::pack(o[0] * inv, o[1] * inv) : 0;
  else *reinterpret_cast<uint16_t*>(to) = sees ? static_cast<uint16_t>(T::pack(o[0] * inv, 0.f)) : 0;
  if (lane == 0) p.lse[tok * p.heads + head] = !sees || l == 0.f ? -kInf : (top == kInf ? kInf : (top + __builtin_amdgcn_logf(l)) * kLn2);
}

template <typename T, int D, int NW>
int launch_chunk(const ChunkArgs& p, hipStream_t stream) {
  const int64_t grid = p.slots * p.kv_heads * p.splits;
  if (grid > INT32_MAX) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid)), b(NW * 64);
  const size_t lds = sizeof(ChunkShared<D>);
  if (p.lb >= 6) chunk_attention_kernel<T, D, true, NW><<<g, b, lds, stream>>>(p);
  else chunk_attention_kernel<T, D, false, NW><<<g, b, lds, stream>>>(p);
  if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  if (p.splits > 1) {
    const int64_t joins = p.slots * p.kv_heads * NW * 8;
    if (joins > INT32_MAX) return MI_ATTN_EINVAL;
    chunk_join_kernel<T, D><<<dim3(static_cast<unsigned>(joins)), dim3(256), 0, stream>>>(p, NW * 32);
    if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  }
  return MI_ATTN_OK;
}

constexpr int kWaves = 4;

struct ChunkPlan {
  int tokens_per, splits, chunk;
  int64_t slots;
  uint64_t rows;  // rows of partial results
};

ChunkPlan plan_of(const mi_chunk_attention_args* a) {
  ChunkPlan p;
  p.tokens_per = a->cu == nullptr ? 1 : kWaves * 32 / (a->heads / a->kv_heads);
  p.slots = slots_of(a->total, a->num_seqs, p.tokens_per);
  const int64_t items = p.slots * a->kv_heads;
  int64_t most = (static_cast<int64_t>(a->block_table_cols) * a->block_size) + a->total;  // what a row can see
  if (a->max_length < most) most = a->max_length;
  const int64_t tiles = most / kTile + 2;
  int64_t splits = items > 0 ? 512 / items : 1;
  if (splits > kSplits) splits = kSplits;
  if (splits > tiles / 4) splits = tiles / 4;
  if (splits < 1) splits = 1;
  p.chunk = static_cast<int>((tiles + splits - 1) / splits);
  p.splits = static_cast<int>((tiles + p.chunk - 1) / p.chunk);
  p.rows = p.splits > 1 ? static_cast<uint64_t>(items) * p.splits * kWaves * 32 : 0;
  return p;
}

int check_chunk(const mi_chunk_attention_args* a) {
  if (a == nullptr) return MI_ATTN_EINVAL;
  if ((a->dtype != MI_ATTN_BF16 && a->dtype != MI_ATTN_FP16) || (a->dim != 64 && a->dim != 128) ||
      (a->block_size != 16 && a->block_size != 32 && a->block_size != 64 && a->block_size != 128) || a->kv_heads < 1 ||
      a->heads < a->kv_heads || a->heads % a->kv_heads || a->heads / a->kv_heads > 128 || a->total < 0 || a->total > INT32_MAX ||
      a->num_pages < 0 || a->num_pages > INT32_MAX || a->num_seqs < 0 || a->block_table_cols < 0 ||
      a->block_table_stride < a->block_table_cols || (a->cu == nullptr && a->total != a->num_seqs) || a->max_length < 0 ||
      a->max_length > INT32_MAX || (static_cast<int64_t>(a->block_table_cols) * a->block_size >= (1 << 30)) || !(a->scale > 0.f) ||
      !(a->scale < kInf))
    return MI_ATTN_EINVAL;
  const int64_t strides[] = {a->q_stride_t, a->q_stride_h, a->k_stride_t, a->k_stride_h, a->v_stride_t, a->v_stride_h};
  for (int64_t s : strides)
    if (s < 0 || (s & 7)) return MI_ATTN_EINVAL;
  return a->k_stride_t >= MI_ATTN_MAX_STRIDE || a->v_stride_t >= MI_ATTN_MAX_STRIDE ? MI_ATTN_EINVAL : MI_ATTN_OK;
}

}  // namespace
}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT uint64_t chunk_attention_workspace(const mi_chunk_attention_args* args) {
  return check_chunk(args) == MI_ATTN_OK ? plan_of(args).rows * (args->dim + 2) * 4 : 0;
}

MI_ATTN_EXPORT int chunk_attention(const mi_chunk_attention_args* a, hipStream_t stream) {
  const int st = check_chunk(a);
  if (st != MI_ATTN_OK) return st;
  const void* wide[] = {a->q, a->k, a->v, a->k_cache, a->v_cache, a->out, a->workspace};
  for (const void* x : wide)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return MI_ATTN_EINVAL;
  const void* words[] = {a->k_scale, a->v_scale, a->block_table, a->lengths, a->cu, a->lse};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MI_ATTN_EINVAL;
  if (a->total == 0) return MI_ATTN_OK;
  if (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->out == nullptr || a->lse == nullptr || (a->num_seqs > 0 && a->lengths == nullptr))
    return MI_ATTN_EINVAL;
  if (a->num_seqs > 0 && a->block_table_cols > 0 && a->block_table == nullptr) return MI_ATTN_EINVAL;
  if (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr || a->k_scale == nullptr || a->v_scale == nullptr)) return MI_ATTN_EINVAL;
  const ChunkPlan plan = plan_of(a);
  if (plan.rows > 0 && (a->workspace == nullptr || a->workspace_bytes < plan.rows * (a->dim + 2) * 4)) return MI_ATTN_EWORKSPACE;
  ChunkArgs p;
  p.q = static_cast<const char*>(a->q);
  p.x[0] = static_cast<const char*>(a->k);
  p.x[1] = static_cast<const char*>(a->v);
  p.cache[0] = static_cast<const uint8_t*>(a->k_cache);
  p.cache[1] = static_cast<const uint8_t*>(a->v_cache);
  p.scales[0] = a->k_scale;
  p.scales[1] = a->v_scale;
  p.table = a->block_table; p.lengths = a->lengths; p.cu = a->cu;
  p.out = static_cast<char*>(a->out);
  p.lse = a->lse;
  p.part = static_cast<float*>(a->workspace);
  p.part_ml = plan.rows == 0 ? nullptr : p.part + plan.rows * a->dim;
  p.q_t = a->q_stride_t; p.q_h = a->q_stride_h;
  p.x_t[0] = a->k_stride_t; p.x_h[0] = a->k_stride_h; p.x_t[1] = a->v_stride_t; p.x_h[1] = a->v_stride_h;
  p.total = a->total; p.num_pages = a->num_pages; p.table_stride = a->block_table_stride; p.slots = plan.slots;
  p.table_cols = a->num_pages > 0 ? a->block_table_cols : 0;  // without pages nothing can be seen of them
  p.num_seqs = a->num_seqs; p.heads = a->heads; p.kv_heads = a->kv_heads; p.group = a->heads / a->kv_heads;
  p.bs = a->block_size; p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size));
  p.tokens_per = plan.tokens_per; p.splits = plan.splits; p.chunk = plan.chunk; p.scale = a->scale;
  if (a->dtype == MI_ATTN_BF16) return a->dim == 128 ? launch_chunk<Bf16, 128, kWaves>(p, stream) : launch_chunk<Bf16, 64, kWaves>(p, stream);
  return a->dim == 128 ? launch_chunk<Fp16, 128, kWaves>(p, stream) : launch_chunk<Fp16, 64, kWaves>(p, stream);
}
