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
// probabilities adds a page's weights divided by s_v.  With fp16 the codes take the
// scale's power of two on their way to LDS, as far as they stay exact, and the
// exponent what is left of it: fp16 weights reach no further than 2^-36 of the
// largest, so that keys in pages of small scales would lose theirs beside new
// tokens, whose values have the scale 1 and may be as small (32000 keys of 2^-20
// beside one of value 0, a scale of 2^-17: 0 instead of 0.03 of the values).
//
// Measured (bf16, 128 columns unless said; cards differ by 7 %): 2048 tokens behind
// 32000 keys, 64/8 heads: 1.88 to 2.02 ms, 1100 to 1180 TFLOP/s, nine tenths of a
// large library product on the same card; fp16 1.98; 8192 alone, 32/4 heads: 0.50 to
// 0.54 ms, 1010 to 1090 (64 tiles a walk, of which each end costs one); 96 behind
// 100003, 32/2 heads: 157 us and 12 to join 21 parts; 64 columns, 2048 behind 16000,
// 32/4 heads: 0.32 to 0.37 ms, 770 to 890; 33 behind 500, 8/2 heads: 14 us, the chain
// of nine tiles.  In the first the matrix unit is busy for 59 % of the cycles, the
// vector unit (of 155 instructions a wavefront and tile 32 are exponentials) about as
// long, LDS for 70 %: two wavefronts a SIMD cover each other's chains, and the card's
// power holds the clock at 1.85 GHz, as in the library's product (69 %).  64 columns
// need the same exponentials for half the products.
//
// Slower (ms, the first two): four wavefronts a workgroup, 2.30 and 0.59: the codes
// are widened twice as often; the next tile's scores between this one's weights, in
// one wavefront, 2.05 and 0.58, by 32 keys 2.25 and 0.55; 64 rows a wavefront, which
// halve the reads of LDS, with one wavefront a SIMD, 2.96; operands read as they are
// needed instead of six products ahead, 2.53 and 0.87.  With 64 columns a third and
// fourth wavefront a SIMD spill.
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
// fp16 holds every code times these powers of two and those between: codes go from
// 2^-9 to 448, fp16 from 2^-24 to 65504
constexpr int kUpLeast = -15, kUpMost = 7;
template <typename T>
constexpr bool kUp = __is_same(T, Fp16);  // bf16 weights have fp32's exponents and need none

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

// Codes of a page that is not there.
__device__ u32x4 nothing[kTile * 128 / 16];

// A tile of the context on its way to LDS: 64 keys' codes and 64 values' over
// NW wavefronts, in registers while the tile before it is worked on; the pages of
// the tile behind it are looked up meanwhile.  A thread has 16 codes of each of
// kPer rows, kStep rows apart, of the keys and of the values (or of one of them).
// Values are multiplied by the power of two of their page.
template <typename T, int D, int NW, bool kWide>
struct Codes {
  static constexpr int kThreads = NW * 64, kLanes = D / 16, kUnits = 2 * kTile * kLanes / kThreads;
  static constexpr int kHalves = kUnits >= 2 ? 2 : 1, kPer = kUnits / kHalves, kStep = kThreads / kLanes;
  static constexpr int kPages = kWide ? 1 : kPer;
  static constexpr int kBuf = kTile * 2 * D;
  static_assert(kUnits * kThreads == 2 * kTile * kLanes && kStep % 16 == 0, "");
  u32x4 x[kHalves][kPer];
  int32_t page[kPages];
  uint32_t to;    // where the thread's first 8 elements go in the first buffer
  int row;        // its first row
  uint32_t lane;  // byte of its codes in a row

  __device__ __forceinline__ explicit Codes(uint32_t base) {
    // Eight lanes, whose stores go together, write every other chunk of 128 bytes of
    // two rows 8 apart, which the swizzle takes to different banks.
    const int tid = threadIdx.x, at = tid % (kTile * kLanes), piece = (at & 3) | (kLanes == 8 ? (at & 8) >> 1 : 0);
    row = at / (2 * kLanes) % 8 + at / (16 * kLanes) * 16 + (at & 4) * 2;
    lane = piece * 16;
    to = base + tile_at<D>(row, 2 * piece);
    if constexpr (kHalves == 1) to += tid / kLanes < kTile ? 0 : 2 * kBuf;
  }
  // `at`: the tile's first key, from the first of the ne blocks that pages[] is of;
  // blocks behind the last one stand for it.
  __device__ __forceinline__ void look(const ChunkArgs& p, const int32_t* pages, int ne, int at) {
#pragma unroll
    for (int j = 0; j < kPages; ++j) page[j] = pages[min((at + (kWide ? 0 : row + j * kStep)) >> p.lb, ne - 1)];
  }
  // The tile has `left` keys; rows behind them stand for the last one, which all
  // queries see.
  __device__ __forceinline__ void load(const ChunkArgs& p, int hk, int at, int left) {
    const int is_v = kHalves == 1 ? (__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x)) / kLanes < kTile ? 0 : 1) : 0;
    const uint8_t* base[kHalves];
    const int pg0 = __builtin_amdgcn_readfirstlane(page[0]);
    if constexpr (kWide) {
      const int64_t first = (((static_cast<int64_t>(pg0) * p.kv_heads + hk) << p.lb) + (at & (p.bs - 1))) * D;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) base[h] = pg0 < 0 ? reinterpret_cast<const uint8_t*>(nothing) : p.cache[is_v + h] + first;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = min(row + j * kStep, left - 1);
      if constexpr (kWide) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) x[h][j] = *reinterpret_cast<const u32x4*>(base[h] + (static_cast<uint32_t>(r) * D + lane));
      } else {
        const int64_t first = ((static_cast<int64_t>(page[j]) * p.kv_heads + hk) << p.lb) * D;
        const uint32_t off = static_cast<uint32_t>((at + r) & (p.bs - 1)) * D + lane;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          x[h][j] = *reinterpret_cast<const u32x4*>((page[j] < 0 ? reinterpret_cast<const uint8_t*>(nothing) : p.cache[is_v + h] + first) + off);
      }
    }
  }
  // The powers of two of the rows of the tile at `at`, as look() finds their pages.
  __device__ __forceinline__ void powers(const ChunkArgs& p, const float* ups, int ne, int at, float (&up)[kPages]) const {
#pragma unroll
    for (int j = 0; j < kPages; ++j) {
      up[j] = 1.f;
      if constexpr (kUp<T>) {
        const float of_page = ups[min((at + (kWide ? 0 : row + j * kStep)) >> p.lb, ne - 1)];
        if (kHalves == 2 || static_cast<int>(threadIdx.x) / kLanes >= kTile) up[j] = of_page;  // (else the thread has keys)
      }
    }
  }
  template <int buf>
  __device__ __forceinline__ void store(const float (&up)[kPages]) const {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        constexpr int kApart = kStep * 2 * D;
        const float by = kHalves == 2 && h == 0 ? 1.f : up[kWide ? 0 : j];
        *reinterpret_cast<MI_LDS u32x4*>(to + (2 * h + buf) * kBuf + j * kApart) = widen<T>(u32x2{x[h][j][0], x[h][j][1]}, by);
        *reinterpret_cast<MI_LDS u32x4*>((to ^ 16) + (2 * h + buf) * kBuf + j * kApart) = widen<T>(u32x2{x[h][j][2], x[h][j][3]}, by);
      }
  }
};

// A tile of the new tokens likewise.
template <typename T, int D, int NW>
struct Fresh {
  static constexpr int kThreads = NW * 64, kLanes = D / 8, kPer = kTile * kLanes / kThreads, kStep = kThreads / kLanes;
  static constexpr int kBuf = kTile * 2 * D;
  static_assert(kPer * kThreads == kTile * kLanes && kStep % 16 == 0, "");
  u32x4 x[2][kPer];
  uint32_t to, lane;
  int row;

  __device__ __forceinline__ explicit Fresh(uint32_t base) {
    const int tid = threadIdx.x;
    row = tid / kLanes;
    lane = (tid % kLanes) * 16;
    to = base + tile_at<D>(row, tid % kLanes);
  }
  // rows behind the chunk's last one stand for it
  __device__ __forceinline__ void load(const ChunkArgs& p, int hk, const ChunkRows& rw, int first) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* base = p.x[h] + ((rw.begin + first) * p.x_t[h] + hk * p.x_h[h]) * 2;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        x[h][j] = *reinterpret_cast<const u32x4*>(base + (__umul24(min(row + j * kStep, rw.n - 1 - first), static_cast<uint32_t>(p.x_t[h] * 2)) + lane));
    }
  }
  // kHide: some row does not see all of the tile, so that infinities and NaN among
  // the values become 0; whether there were any
  template <int buf, bool kHide>
  __device__ __forceinline__ bool store() const {
    bool odd = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        u32x4 c = x[h][j];
        if (kHide && h == 1) {
#pragma unroll
          for (int z = 0; z < 4; ++z) c[z] = finite_only<T>(c[z], odd);
        }
        *reinterpret_cast<MI_LDS u32x4*>(to + (2 * h + buf) * kBuf + j * (kStep * 2 * D)) = c;
      }
    return odd;
  }
};

template <typename T, int D>
struct ChunkShared {
  char k[2][kTile * 2 * D];
  char v[2][kTile * 2 * D];
  int32_t page[kSeg];  // -1: not there
  float ks[kSeg], lv[kSeg], iv[kSeg];
  float up[kUp<T> ? kSeg : 1];
  int32_t odd;         // an infinity or NaN is among the values that some row does not see
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
  ChunkShared<T, D>& sh = *reinterpret_cast<ChunkShared<T, D>*>(smem);
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

  u32x4 q[D / 16];
  {
    const char* from = p.q + ((rw.begin + mine) * p.q_t + (valid ? head : hk * p.group) * p.q_h) * 2 + half * 16;
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
  // A weight is rounded once, to the type of q, since the matrix unit takes no wider
  // operand at this rate (2^-8 of it at most with bf16, 2^-11 with fp16).  fp16 has no bits below 2^-24, so
  // there the weights are relative to a maximum 2^12 below the row's, and with the
  // 2^3 that this may lag behind they go up to 2^15 (bf16 has fp32's exponents)
  constexpr float kLag = __is_same(T, Fp16) ? 3.f : 8.f, kLower = __is_same(T, Fp16) ? 12.f : 0.f;
  constexpr int kScales = kWide ? 1 : 4;

  // One tile, in LDS buffer `buf`.  With kPart, if `part`, a row sees its keys low ..
  // high only.  put() writes the next tile to the other buffer (kWrites writes), get()
  // loads the one behind it: both are spread over the step.
  auto work = [&](auto which, auto parts, auto writes, bool part, int low, int high, const float (&ck)[kScales], const float (&lv)[kScales],
                  const float (&iv)[kScales], auto put, auto get) {
    constexpr int buf = decltype(which)::value, kWrites = decltype(writes)::value;
    constexpr bool kPart = decltype(parts)::value != 0;
    f32x16 s[2];
    {
      u32x4 ka[2][D / 16];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) ka[mt][i] = rd.row(buf * kBuf, mt * 32, i);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[mt][r] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s[mt] = T::mfma32(ka[mt][i], q[i], s[mt]);
      }
      put();
      // reads of the first products' operands, then a product and a read in turn,
      // then products and the other buffer's writes
      constexpr int kAhead = 6, kProducts = D / 8;
      __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
      for (int i = 0; i < kProducts - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, (kWrites + kAhead - 1) / kAhead, 0);
      }
    }
    if (kPart && part) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int at = 32 * mt + 8 * (r >> 2) + (r & 3);
          if (at < low - 4 * half || at > high - 4 * half) s[mt][r] = -kInf;
        }
    }
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t = s[i >> 1][8 * (i & 1)];
#pragma unroll
      for (int r = 1; r < 8; ++r) t = __builtin_elementwise_maximum(t, s[i >> 1][8 * (i & 1) + r]);
      if constexpr (!kWide) t = fmaf(t, ck[i], lv[i]);
      top = __builtin_elementwise_maximum(top, t);
    }
    if constexpr (kWide) top = fmaf(top, ck[0], lv[0]);
    top = half_max(top);
    if (__any(top - m > kLag)) {
      const float now = fmaxf(m, top);
      const float shrink = now == -kInf ? 1.f : exp2_fast(m - now);
      m = now;
      sum *= shrink;
      const float keeps = fmaxf(shrink, 0x1p-149f);  // an infinity stays one, nothing else does
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] *= keeps;
    }
    get();
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
    u32x4 va[D / 32][4];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int st = 0; st < 4; ++st) va[i][st] = rd.column((2 + buf) * kBuf, 16 * st, i);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int st = 0; st < 4; ++st) acc[i] = T::mfma32(va[i][st], pr[st], acc[i]);
    read_ahead<D / 8, 6, 2>();
  };

  // Number of the page of block `b` of the segment that begins with tile t; -1 where
  // there is none.
  auto page_at = [&](int t, int b) {
    const int block = ((t * kTile) >> p.lb) + b;
    if (b >= kSeg || block >= (rw.context + p.bs - 1) >> p.lb) return -1;
    const int pg = p.table[rw.seq * p.table_stride + block];
    return pg >= 0 && pg < p.num_pages ? pg : -1;
  };
  // on its way while the new tokens are worked on
  const int first_page = e0 < rw.tiles_context ? page_at(e0, tid) : -1;

  // The new tokens: tiles that all rows see, and tiles that some row sees a part of.
  const int n0 = max(e0, rw.tiles_context);
  if (tid == 0) sh.odd = 0;
  const int least = max(rw.r0, rw.hidden);  // the first token here that sees anything
  auto first_of = [&](int t) { return (rw.first_new + t - rw.tiles_context) * kTile; };
  auto hides = [&](int t) { return first_of(t) + kTile - 1 > least || first_of(t) < rw.hidden; };
  struct {
    float ck[kScales], lv[kScales], iv[kScales];
  } plain;
#pragma unroll
  for (int i = 0; i < kScales; ++i) {
    plain.ck[i] = c;
    plain.lv[i] = 0.f;
    plain.iv[i] = 1.f;
  }
  auto walk_part = [&](int from, int to) {
    Fresh<T, D, NW> in(lds_offset(sh.k[0]));
    in.load(p, hk, rw, first_of(from));
    for (int t = from; t < to; ++t) {
      __syncthreads();
      if (in.template store<0, true>()) sh.odd = 1;
      if (t + 1 < to) in.load(p, hk, rw, first_of(t + 1));
      __syncthreads();
      const int first = first_of(t), high = sees ? mine - first : -1;
      auto none = [] {};
      if (__any(high >= 0)) work(Int<0>{}, Int<1>{}, Int<0>{}, true, rw.hidden - first, high, plain.ck, plain.lv, plain.iv, none, none);
    }
    __syncthreads();
  };
  auto walk = [&](int from, int to) {
    Fresh<T, D, NW> in(lds_offset(sh.k[0]));
    in.load(p, hk, rw, first_of(from));
    __syncthreads();
    in.template store<0, false>();
    in.load(p, hk, rw, first_of(min(from + 1, to - 1)));
    __syncthreads();
    auto step = [&](auto which, int t) {
      constexpr int buf = decltype(which)::value;
      work(which, Int<0>{}, Int<2 * decltype(in)::kPer>{}, false, 0, 0, plain.ck, plain.lv, plain.iv,
           [&] { in.template store<buf ^ 1, false>(); }, [&] { in.load(p, hk, rw, first_of(min(t + 2, to - 1))); });
    };
    for (int t = from; t < to; t += 2) {
      step(Int<0>{}, t);
      __syncthreads();
      if (t + 1 < to) {
        step(Int<1>{}, t + 1);
        __syncthreads();
      }
    }
  };
  bool odd = false;  // the wavefront has met an infinity or NaN that all its rows see
  if (n0 < e1) {
    // the first tile can hold hidden tokens; the last ones are not seen by the first rows
    int from = n0, to = e1;
    while (from < to && hides(to - 1)) --to;
    if (from < to && hides(from)) {
      walk_part(from, from + 1);
      ++from;
    }
    if (from < to) {
      walk(from, to);
      // What is NaN here comes from an infinity or NaN among the values, which the end
      // adds, or from a score, and then the sum is NaN too: it starts anew, so that an
      // infinity of a weight that is 0 in 16 bits is one.
      float finite[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) finite[r & 3] = fmaf(acc[i][r], 0.f, finite[r & 3]);
      odd = __any((finite[0] + finite[1]) + (finite[2] + finite[3]) != 0.f);
      if (odd) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][r] = acc[i][r] != acc[i][r] ? 0.f : acc[i][r];
      }
    }
    if (to < e1) walk_part(to, e1);
  }

  // The context, kSeg blocks' tiles at a time.
  const int c1 = min(e1, rw.tiles_context);
  for (int s0 = e0; s0 < c1;) {
    // (a part can begin inside a block of 128 keys)
    const int block0 = (s0 * kTile) >> p.lb, shift = s0 * kTile - (block0 << p.lb);
    const int blocks = (rw.context + p.bs - 1) >> p.lb;
    const int s1 = min(c1, (((block0 + kSeg) << p.lb) / kTile));
    const int ne = min(kSeg, blocks - block0);
    const int pg = s0 == e0 ? first_page : page_at(s0, tid);
    __syncthreads();
    if (tid < ne) sh.page[tid] = pg;
    __syncthreads();
    Codes<T, D, NW, kWide> in(lds_offset(sh.k[0]));
    auto at_of = [&](int t) { return (min(t, s1 - 1) - s0) * kTile + shift; };
    auto left_of = [&](int t) { return rw.context - min(t, s1 - 1) * kTile; };
    in.look(p, sh.page, ne, at_of(s0));
    in.load(p, hk, at_of(s0), left_of(s0));
    if (tid < ne) {  // the scales come while the first codes do
      const int64_t at = static_cast<int64_t>(max(0, pg)) * p.kv_heads + hk;
      const float ks = p.scales[0][at];
      float vs = pg < 0 ? 1.f : fminf(fmaxf(p.scales[1][at], kLeast), kMost);
      if constexpr (kUp<T>) {
        const int e = max(kUpLeast, min(static_cast<int>(__float_as_uint(vs) >> 23) - 127, kUpMost));
        sh.up[tid] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        vs *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // what is left of it, exactly
      }
      sh.ks[tid] = pg < 0 ? 1.f : fmaxf(ks * c, 0x1p-149f);
      sh.lv[tid] = pg < 0 ? -kInf : __builtin_amdgcn_logf(vs);  // no weight
      sh.iv[tid] = 1.f / vs;
    }
    in.look(p, sh.page, ne, at_of(s0 + 1));
    if constexpr (kUp<T>) __syncthreads();
    float up[decltype(in)::kPages];
    in.powers(p, sh.up, ne, at_of(s0), up);
    in.template store<0>(up);
    in.load(p, hk, at_of(s0 + 1), left_of(s0 + 1));
    in.look(p, sh.page, ne, at_of(s0 + 2));
    __syncthreads();
    auto step = [&](auto which, int t) {
      constexpr int buf = decltype(which)::value;
      float ck[kScales], lv[kScales], iv[kScales];
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int e = min((at_of(t) + 16 * i) >> p.lb, ne - 1);
        ck[i] = sh.ks[e];
        lv[i] = sh.lv[e];
        iv[i] = sh.iv[e];
      }
      const int left = left_of(t);
      in.powers(p, sh.up, ne, at_of(t + 1), up);
      work(which, Int<1>{}, Int<2 * decltype(in)::kUnits>{}, left < kTile, 0, left - 1, ck, lv, iv, [&] { in.template store<buf ^ 1>(up); },
           [&] {
             in.load(p, hk, at_of(t + 2), left_of(t + 2));
             in.look(p, sh.page, ne, at_of(t + 3));
           });
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
  // Infinities and NaN among the new values, to the rows that see them, whatever their
  // weight.  A wavefront looks at 8 KB at a time; those that all rows see are added up
  // as they lie there, 8 columns a lane, the others' rows are gone over key by key.
  if (odd || (n0 < e1 && sh.odd != 0)) {
    constexpr int kLanes = D / 8, kRowsAt = 64 / kLanes, kAt = 8;
    const int at = static_cast<int>(__lane_id()), end = min(first_of(e1 - 1) + kTile, rw.r0 + rw.tokens);
    int from = n0, to = e1;  // the tiles that all rows see
    while (from < to && hides(to - 1)) --to;
    if (from < to && hides(from)) ++from;
    const char* base = p.x[1] + (rw.begin * p.x_t[1] + hk * p.x_h[1]) * 2;
    auto row_at = [&](int key) { return base + key * (p.x_t[1] * 2); };
    float added[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k0 = first_of(n0); k0 < end; k0 += kRowsAt * kAt) {
      const bool all = k0 >= first_of(from) && k0 < first_of(to);
      bool any = false;
#pragma unroll
      for (int j = 0; j < kAt; ++j) {  // (rows behind the last one stand for it)
        const u32x4 x = *reinterpret_cast<const u32x4*>(row_at(min(k0 + j * kRowsAt + at / kLanes, end - 1)) + at % kLanes * 16);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          finite_only<T>(x[z], any);
          const float a = T::lo(x[z]), b = T::hi(x[z]);
          added[2 * z] += all && !(fabsf(a) < kInf) ? a : 0.f;
          added[2 * z + 1] += all && !(fabsf(b) < kInf) ? b : 0.f;
        }
      }
      if (all || !__any(any)) continue;
#pragma unroll 1
      for (int key = k0; key < min(k0 + kRowsAt * kAt, end); ++key) {
        const char* v = row_at(key) + (at >> 5) * 8;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(v + i * 64 + (r >> 2) * 16);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float a = z & 1 ? T::hi(w[z >> 1]) : T::lo(w[z >> 1]);
              acc[i][r + z] += sees && key >= rw.hidden && key <= mine && !(fabsf(a) < kInf) ? a : 0.f;
            }
          }
      }
    }
#pragma unroll
    for (int z = 0; z < 8; ++z)
#pragma unroll
      for (int d = kLanes; d < 64; d <<= 1) added[z] += __shfl_xor(added[z], d);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float low = __shfl(added[r & 3], 4 * i + (r >> 2)), high = __shfl(added[4 + (r & 3)], 4 * i + (r >> 2));
        acc[i][r] += sees ? (at < 32 ? low : high) : 0.f;
      }
  }
  sum = half_sum(sum);
  const float base = m - kLower;
  if (!valid) return;
  if (p.splits == 1 || rw.tiles <= p.chunk) {  // the walk is in one part
    int token = mine;
    asm volatile("" : "+v"(token));  // (worked out again here: the walks need its registers)
    store_chunk_row<T, D>(p, rw.begin + token, head, half, acc, base, sum, sees);
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

// Joins the parts of the rows' walks: a wavefront takes four rows, 16 parts of each
// at a time to work out their weights, then adds the parts up in order.  21 parts of
// 96 tokens, 32 heads of 128: 34 MB in 12 us, the chain of three loads and memory.
constexpr int kJoin = 4;
template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkArgs p, int rows_per) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t index = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * kJoin;
  const int64_t item = index / rows_per;  // slot (from the last one) and key head
  const int row0 = static_cast<int>(index % rows_per);
  if (item >= p.slots * p.kv_heads) return;
  const int hk = static_cast<int>(item % p.kv_heads);
  const int64_t from_last = item / p.kv_heads;
  const int64_t first = (from_last * p.splits * p.kv_heads + hk) * rows_per + row0, step = static_cast<int64_t>(p.kv_heads) * rows_per;
  // maxima and sums are loaded before it is known which of them were written
  const float* ml = p.part_ml + (first + (lane >> 4)) * 2;  // the lane's row where weights are worked out
  f32x2 both[kSplits / 16];
#pragma unroll
  for (int c = 0; c < kSplits / 16; ++c) {
    const int s = c * 16 + (lane & 15);
    both[c] = s < p.splits ? *reinterpret_cast<const f32x2*>(ml + s * step * 2) : f32x2{-kInf, 0.f};
  }
  const ChunkRows rw = rows_of(p, p.slots - 1 - from_last);
  const int rows = rw.tokens * p.group;  // those there are
  if (row0 >= rows || rw.tiles <= p.chunk) return;  // (the latter is done)
  const int used = min(p.splits, (rw.tiles + p.chunk - 1) / p.chunk);
  float base[kSplits / 16], f[kSplits / 16], top = -kInf, l = 0.f;
#pragma unroll
  for (int c = 0; c < kSplits / 16; ++c) {
    const bool there = c * 16 + (lane & 15) < used;
    base[c] = there ? both[c][0] : -kInf;
    f[c] = there ? both[c][1] : 0.f;  // the sum, for now
    top = fmaxf(top, base[c]);
  }
  for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll
  for (int c = 0; c < kSplits / 16; ++c) {
    const float w = base[c] == -kInf ? 0.f : exp2_fast(base[c] - top);
    l += f[c] * w;
    f[c] = w == 0.f ? 0x1p-149f : w;  // (an infinity in a part of no weight stays one, nothing else does)
  }
  for (int d = 1; d < 16; d <<= 1) l += __shfl_xor(l, d);
  float o[kJoin][D / 64];
#pragma unroll
  for (int r = 0; r < kJoin; ++r)
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[r][i] = 0.f;
  const float* values = p.part + first * D + lane * (D / 64);
  constexpr int kAtOnce = 8;
#pragma unroll
  for (int c = 0; c < kSplits / 16; ++c) {
    if (c * 16 >= used) break;
    for (int s = c * 16; s < min(used, c * 16 + 16); s += kAtOnce) {
      float x[kAtOnce][kJoin][D / 64];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int r = 0; r < kJoin; ++r)
#pragma unroll
          for (int i = 0; i < D / 64; ++i) x[u][r][i] = values[(min(s + u, used - 1) * step + min(r, rows - 1 - row0)) * D + i];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int r = 0; r < kJoin; ++r) {
          const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f[c]), r * 16 + ((s + u) & 15)));
          if (s + u < used)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) o[r][i] += x[u][r][i] * w;
        }
    }
  }
#pragma unroll
  for (int r = 0; r < kJoin; ++r) {
    const int row = row0 + r;
    if (row >= rows) break;
    const int tl = row / p.group, head = hk * p.group + row % p.group;
    const bool sees = rw.r0 + tl >= rw.hidden;
    const float lr = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(l), r * 16));
    const float base_r = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(top), r * 16));
    const int64_t tok = rw.begin + rw.r0 + tl;
    const float inv = lr == 0.f ? 0.f : 1.f / lr;
    char* to = p.out + ((tok * p.heads + head) * D + lane * (D / 64)) * 2;
    if constexpr (D == 128) *reinterpret_cast<uint32_t*>(to) = sees ? T::pack(o[r][0] * inv, o[r][1] * inv) : 0;
    else *reinterpret_cast<uint16_t*>(to) = sees ? static_cast<uint16_t>(T::pack(o[r][0] * inv, 0.f)) : 0;
    if (lane == 0)
      p.lse[tok * p.heads + head] = !sees || lr == 0.f ? -kInf : (base_r == kInf ? kInf : (base_r + __builtin_amdgcn_logf(lr)) * kLn2);
  }
}

template <typename T, int D, int NW>
void launch_walk(const ChunkArgs& p, unsigned grid, hipStream_t stream) {
  const size_t lds = sizeof(ChunkShared<T, D>);
  if (p.lb >= 6) chunk_attention_kernel<T, D, true, NW><<<dim3(grid), dim3(NW * 64), lds, stream>>>(p);
  else chunk_attention_kernel<T, D, false, NW><<<dim3(grid), dim3(NW * 64), lds, stream>>>(p);
}

template <typename T, int D>
int launch_chunk(const ChunkArgs& p, int waves, hipStream_t stream) {
  const int64_t grid = p.slots * p.kv_heads * p.splits;
  if (grid > UINT32_MAX / (waves * 64)) return MI_ATTN_EINVAL;  // a launch has less than 2^32 threads
  if (waves == 8) launch_walk<T, D, 8>(p, static_cast<unsigned>(grid), stream);
  else launch_walk<T, D, 4>(p, static_cast<unsigned>(grid), stream);
  if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  if (p.splits > 1) {
    const int64_t joins = p.slots * p.kv_heads * waves * 8 / kJoin;
    if (joins > UINT32_MAX / 256) return MI_ATTN_EINVAL;
    chunk_join_kernel<T, D><<<dim3(static_cast<unsigned>(joins)), dim3(256), 0, stream>>>(p, waves * 32);
    if (hipGetLastError() != hipSuccess) return MI_ATTN_ELAUNCH;
  }
  return MI_ATTN_OK;
}

struct ChunkPlan {
  int waves, tokens_per, splits, chunk;
  int64_t slots;
  uint64_t rows;  // rows of partial results
};

// In how many parts, `most` at most, the walks of `items` workgroups over up to
// `tiles` tiles are cut.  `tiles` is that of the caller's bound, and a part has as many
// whatever the sequence's own length: behind a bound far above it a walk lies in few
// parts or one (96 tokens behind 8000, 32/8 heads: 39 us with its own length as bound,
// 195 with 131072; 96 behind 100003, 32/2 heads: 161, and 1140 with 2^20).  The 256 compute units take the workgroups in rounds (two
// small ones on a unit at once need as long as one after the other).  Where several
// sequences share the call their lengths differ: half of the work is counted, half
// a walk in which the card runs empty, and an eighth of the join's bytes, which
// passes over the parts that a sequence does not have.  A tile takes `tile` ns of a
// unit, `alone` at least; the join costs its launch (with the host's part) and the
// partial results' way through memory.  Measured: five sequences of 890 tokens behind
// up to 7000, 12/3 heads: 101 us in one part, 49 in 7, 45 in 11 to 20; four of 200
// behind 900, 16/4 heads: 23 in one, 28 in 4.
int parts_of(int64_t items, bool several, int64_t tiles, int64_t rows, int dim, int waves, int64_t most) {
  const int64_t tile = dim == 128 ? (waves == 8 ? 1900 : 1120) : (waves == 8 ? 1300 : 700), alone = dim == 128 ? tile : (waves == 8 ? tile : 950);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kSplits && (s == 1 || (s <= most && s <= tiles)); ++s) {
    const int64_t walk = (tiles + s - 1) / s, bytes = rows * s * (dim + 2) * 8;
    int64_t cost;
    if (several) cost = tile * items * s / 512 * walk + alone * walk / 2;
    else cost = tile * ((items * s + 255) / 256) * walk;
    if (cost < alone * walk) cost = alone * walk;
    if (s > 1) cost += several ? 14000 + 50 * s + bytes / 32000 : 10000 + 200 * s + bytes / 4000;  // (4 TB/s)
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

ChunkPlan plan_of(const mi_chunk_attention_args* a) {
  ChunkPlan p;
  const int group = a->heads / a->kv_heads;
  int64_t most = (static_cast<int64_t>(a->block_table_cols) * a->block_size) + a->total;  // what a row can see
  if (a->max_length < most) most = a->max_length;
  const int64_t tiles = most / kTile + 2;
  const int64_t seqs = a->total < a->num_seqs ? a->total : a->num_seqs;  // those that have tokens, at most
  auto with = [&](int waves) {
    p.waves = waves;
    p.tokens_per = a->cu == nullptr ? 1 : waves * 32 / group;
    p.slots = slots_of(a->total, a->num_seqs, p.tokens_per);
    // workgroups that have rows: of each sequence one more than whole ones, at most
    return (seqs <= 1 ? (a->total + p.tokens_per - 1) / p.tokens_per : a->total / p.tokens_per + seqs) * a->kv_heads;
  };
  // Eight wavefronts a workgroup widen the codes once for 256 rows; four start
  // quicker, leave fewer rows empty and with 64 columns run three workgroups on a unit
  // instead of one.  Eight where there are 4000 tiles or more to walk over, unless
  // there are several sequences, with 128 columns a third as many as whole workgroups
  // (half of a sequence's last workgroup is empty in the mean).  Measured (us, eight
  // against four, each with its best parts): 128 columns: 96 tokens behind 100003, 32/2
  // heads (18800 tiles): 190, 210; 512 behind 4000, 32/8 (4700): 61, 64; 2000 behind
  // 2000, 8/1 (4100): 56, 59; 300 behind 3000, 16/2 (1000): 37, 34; 128 behind 8000,
  // 8/8 (1000): 33, 30; 1000 alone, 16/4 (1100): 32, 25; 16 of 256 behind 2000, 32/8:
  // 163, 170; 30 of 100 behind 3000, 64/8: 398, 377; 64 single tokens and 512, 32/8:
  // 145, 95.  64 columns: 2048 behind 64000, 16/2: 715, 740; 8192 alone, 32/8: 350,
  // 335; 8 of 1000 behind 1000, 16/4: 95, 91; 64 of 128 behind 4000, 16/2: 235, 197;
  // five of 890 tokens, 12/3: 58, 46; 33 behind 500, 8/2: 17.6, 14.1.
  int64_t items = with(8);
  if (items * tiles < 4000 || (seqs > 1 && (a->dim == 64 || 3 * seqs > a->total / p.tokens_per))) items = with(4);
  // partial results of 2^17 rows at most (68 MB with 128 columns)
  const int64_t rows = p.slots * a->kv_heads * p.waves * 32;
  const int64_t splits = items > 0 ? parts_of(items, seqs > 1, tiles, a->total * a->heads, a->dim, p.waves, (int64_t{1} << 17) / rows) : 1;
  p.chunk = static_cast<int>((tiles + splits - 1) / splits);
  p.splits = static_cast<int>((tiles + p.chunk - 1) / p.chunk);
  p.rows = p.splits > 1 ? static_cast<uint64_t>(rows) * p.splits : 0;
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
  if (a->dtype == MI_ATTN_BF16) return a->dim == 128 ? launch_chunk<Bf16, 128>(p, plan.waves, stream) : launch_chunk<Bf16, 64>(p, plan.waves, stream);
  return a->dim == 128 ? launch_chunk<Fp16, 128>(p, plan.waves, stream) : launch_chunk<Fp16, 64>(p, plan.waves, stream);
}
