// Block sparse attention: forward, and the gradient of the queries.
//
//   out = sum_j p_j v_j over the keys j of the blocks that each query selects.
//
// A workgroup takes 128 rows of one key head: TQ = 128 / G consecutive tokens
// with the G query heads that share the key head, 32 rows a wavefront.  It
// walks over the blocks that any of its tokens selects, 64 keys at a time, so
// neighbouring tokens that select the same blocks read them once; each row
// masks what its own token did not select, and a wavefront none of whose rows
// selects a tile skips it.
//
// Scores are computed as K Q^T: a query's scores of a tile then lie in two
// lanes, so that the softmax crosses lanes once, and the weights are the second
// product's operand as they stand, with V read transposed from LDS in the order
// in which the scores lie.
//
// Measured (kernel, on a card that has run for 50 ms; 13 % longer before): 2048
// tokens over 65536 keys, 64/4 heads of 128, 32 blocks of 64: 467 us, 290 TFLOP/s
// of the selected keys' products, 2.6 TB/s from memory; 8192 tokens, 32/2 heads,
// 16 blocks, with the gradient's second terms: 347 us.  The matrix units are busy
// for 19 % and 30 % of that.  Two things bound it.  A workgroup walks the union of
// what its tokens select, 3.9 times (the second case 2.1 times) one token's blocks
// with 8 tokens, while a wavefront's two tokens need 1.6 (1.3) times one token's:
// in the other tiles it copies and waits.  And a tile's chain of product, maximum,
// exponentials and product has two wavefronts a SIMD to fill each other's gaps
// (192 registers of operands and sums leave no room for a third).  Below 1000
// tokens (517, 16/2 heads: 17 us) it is the start: 6 us to the list of blocks,
// then a tile's chain of about 1 us.  Tried and slower: 16 rows a
// wavefront (350 us where 32 took 311), 256 rows a workgroup (332 and 314; the
// first case 639 and 546), four wavefronts sharing the keys of 32 rows for few tokens
// (517 tokens: 21 us and 18).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "attn_device.hpp"
#include "block_attention.hpp"

namespace miattn {
namespace {

template <typename T, int D>
struct Shared {
  char k[2][kTile * 2 * D];
  char v[2][kTile * 2 * D];
  Select sel;
};

// A weight is rounded once, to the type of q.  fp16 has no bits below 2^-24, so
// there the weights are relative to a maximum 2^7 below the row's: with the 2^8
// that the maximum may lag behind they go up to 2^15 (bf16 has fp32's exponents).
template <typename T>
constexpr float kRoom = __is_same(T, Fp16) ? 7.f : 0.f;

// A row's output, divided by the sum of its weights: lane half `half` has the
// columns 32 i + 8 (r / 4) + 4 half + r % 4 in acc[i][r].  A weight of 1 counts
// as `one` in the sum.
template <typename T, int D, bool kRest>
__device__ __forceinline__ void store_row(const Args& p, int64_t tok, int head, int half, const f32x16 (&acc)[D / 32], float m, float sum, float one) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to_at = (tok * p.heads + head) * (2 * D) + half * 8;
  char* to = static_cast<char*>(p.out) + to_at;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      u32x2 w;
      w[0] = T::pack(acc[i][r] * inv, acc[i][r + 1] * inv);
      w[1] = T::pack(acc[i][r + 2] * inv, acc[i][r + 3] * inv);
      *reinterpret_cast<u32x2*>(to + i * 64 + (r >> 2) * 16) = w;
      if constexpr (kRest) {
        u32x2 z;
        z[0] = T::pack(acc[i][r] * inv - T::lo(w[0]), acc[i][r + 1] * inv - T::hi(w[0]));
        z[1] = T::pack(acc[i][r + 2] * inv - T::lo(w[1]), acc[i][r + 3] * inv - T::hi(w[1]));
        *reinterpret_cast<u32x2*>(static_cast<char*>(p.rest) + to_at + i * 64 + (r >> 2) * 16) = z;
      }
    }
  if (half == 0) p.lse[tok * p.heads + head] = sum == 0.f ? -kInf : (m == kInf ? kInf : m * p.scale + __logf(sum / one));
}

// The rows of the workgroup once more, key by key, with what a row does not see
// left out of its arithmetic: for the rare workgroup whose results are not
// finite.
template <typename T, int D, bool kRest>
__device__ __forceinline__ void one_by_one(const Args& p, Select& sel) {
  const int hk = blockIdx.x % p.kv_heads;
  const int64_t slot = p.slots - 1 - static_cast<int64_t>(blockIdx.x / p.kv_heads);
  const int tq = p.tokens_per;
  const Group g = group_of(p, slot, tq);
  const int lane = threadIdx.x & 63, half = lane >> 5, row = (threadIdx.x >> 6) * 32 + (lane & 31);
  const int tl = row / p.group, head = hk * p.group + row % p.group;
  const bool valid = tl < g.tokens;
  const int64_t tok = g.t0 + (valid ? tl : 0), pos = tok - g.begin + g.shift;
  const int64_t limit = p.causal && pos < g.len_k ? pos : g.len_k - 1;
  const char* q = static_cast<const char*>(p.q) + (tok * p.q_t + head * p.q_h) * 2 + half * 16;
  const char* kbase = static_cast<const char*>(p.k) + (g.tk0 * p.k_t + hk * p.k_h) * 2 + half * 16;
  const char* vbase = static_cast<const char*>(p.v) + (g.tk0 * p.v_t + hk * p.v_h) * 2 + half * 8;
  const float c = p.scale * kLog2e;
  f32x16 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  float m = -kInf, sum = 0.f;
  const int nw = (tq + 31) >> 5, width = kMaskWords / nw, word = tl >> 5 < nw ? tl >> 5 : 0;
  for (int w0 = 0; w0 < g.blocks; w0 += width) {
    const int active = list_window(p, g, hk, w0, width, nw, sel);
    for (int e = 0; e < active; ++e) {
      const int id = sel.list[e];
      const bool mine = valid && ((sel.mask[id * nw + word] >> (tl & 31)) & 1u);
      if (!__any(mine)) continue;
      const int from = (w0 + id) << p.lb, to = min(from + p.bs, g.len_k);
      for (int key = from; key < to; ++key) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(kbase + key * (p.k_t * 2) + i * 32), b = *reinterpret_cast<const u32x4*>(q + i * 32);
#pragma unroll
          for (int z = 0; z < 4; ++z) x = fmaf(T::hi(a[z]), T::hi(b[z]), fmaf(T::lo(a[z]), T::lo(b[z]), x));
        }
        x = half_sum(x);
        if (mine && key <= limit) {
          const float now = fmaxf(m, x), shift = now == -kInf ? 0.f : now;
          const float shrink = now == m ? 1.f : exp2_fast((m - now) * c), w = exp2_fast((x - shift) * c);
          m = now;
          sum = sum * shrink + w;
          const char* vr = vbase + key * (p.v_t * 2);
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const u32x2 v = *reinterpret_cast<const u32x2*>(vr + i * 64 + (r >> 2) * 16);
              acc[i][r] = fmaf(w, T::lo(v[0]), acc[i][r] * shrink);
              acc[i][r + 1] = fmaf(w, T::hi(v[0]), acc[i][r + 1] * shrink);
              acc[i][r + 2] = fmaf(w, T::lo(v[1]), acc[i][r + 2] * shrink);
              acc[i][r + 3] = fmaf(w, T::hi(v[1]), acc[i][r + 3] * shrink);
            }
        }
      }
    }
  }
  if (valid) store_row<T, D, kRest>(p, tok, head, half, acc, m, sum, 1.f);
}

// Called, it costs a short call nothing (inline: 20 us instead of 18 for 517
// tokens); with kRest the call's registers are missed in the loop, so there it
// is inline (440 us and 360 for 8192 tokens).
template <typename T, int D>
__device__ __noinline__ void one_by_one_called(const Args* args, Select* sel) {
  one_by_one<T, D, false>(*args, *sel);
}

// With kRest the weights of the second product have two terms (16 bits of 24)
// and the part of out that its own rounding leaves out is stored too: the
// gradient subtracts dout . out from terms that it nearly cancels.
// With kSplit, for few rows, a workgroup takes 64 rows and two wavefronts share
// 32 of them: each works on 32 keys of every tile, and they are joined at the end.
template <typename T, int D, bool kWide, bool kRest, bool kSplit>
__global__ void __launch_bounds__(256, D == 64 ? 3 : 2) block_attention_kernel(Args p) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Shared<T, D>& sh = *reinterpret_cast<Shared<T, D>*>(smem);
  const int hk = blockIdx.x % p.kv_heads;
  // later tiles see more blocks: they start first
  const int64_t slot = p.slots - 1 - static_cast<int64_t>(blockIdx.x / p.kv_heads);
  const int tq = p.tokens_per;
  const Group g = group_of(p, slot, tq);
  if (g.tokens == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5;
  const int rows32 = kSplit ? wave & 1 : wave, keys32 = kSplit ? wave >> 1 : 0;
  constexpr int kParts = kSplit ? 1 : 2;  // 32-key parts of a tile that a wavefront takes
  const int row = rows32 * 32 + (lane & 31);
  const int tl = row / p.group, head = hk * p.group + row % p.group;
  const bool valid = tl < g.tokens;
  const int64_t tok = g.t0 + (valid ? tl : 0);
  int limit = -1;
  if (valid) {
    const int64_t pos = tok - g.begin + g.shift;
    limit = p.causal ? static_cast<int>(pos < g.len_k ? pos : g.len_k - 1) : g.len_k - 1;
  }

  // the row's query: D / 16 operands of 8 elements
  u32x4 q[D / 16];
  {
    const char* from = static_cast<const char*>(p.q) + (tok * p.q_t + head * p.q_h) * 2 + half * 16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = valid ? *reinterpret_cast<const u32x4*>(from + i * 32) : u32x4{0, 0, 0, 0};
  }
  const char* kbase = static_cast<const char*>(p.k) + (g.tk0 * p.k_t + hk * p.k_h) * 2;
  const char* vbase = static_cast<const char*>(p.v) + (g.tk0 * p.v_t + hk * p.v_h) * 2;

  f32x16 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  float m = -kInf, sum = 0.f;
  const float c = p.scale * kLog2e;

  const int nw = (tq + 31) >> 5;
  const int width = kMaskWords / nw;
  const Reads<D> rd(lds_offset(sh.k[0]) + keys32 * (64 * D));
  constexpr int kBuf = kTile * 2 * D;  // from one buffer to the other; the values lie two behind the keys

  for (int w0 = 0; w0 < g.blocks; w0 += width) {
    const int active = list_window(p, g, hk, w0, width, nw, sh.sel);
    const int tiles = ((active << p.lb) + kTile - 1) / kTile;
    if (tiles == 0) continue;
    // While a tile is worked on, the next one goes to the other buffer and the
    // one behind it is on its way to registers; what a row sees of a tile is
    // worked out one tile ahead.  The copies are spread over the step, between
    // the products and the exponentials: in one place they wait for each other
    // (a step of 4061 cycles held 1177 of that, measured).  Behind the last
    // tile they copy it again.
    const int word = tl >> 5 < nw ? tl >> 5 : 0;
    Keys<kWide> next = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, 0);
    Half<D> kin, vin;
    kin.load(kbase, p.k_t * 2, next, g.len_k);
    vin.load(vbase, p.v_t * 2, next, g.len_k);
    auto sight = [&](const Keys<kWide>& k) {
      Sight v = sight_of(sh.sel, k, nw, word, tl & 31, limit, valid);
      if constexpr (kSplit) v.from(keys32);
      return v;
    };
    Sight ahead = sight(next);
    kin.store(sh.k[0]);
    vin.store(sh.v[0]);
    next = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, 1);
    kin.load(kbase, p.k_t * 2, next, g.len_k);
    vin.load(vbase, p.v_t * 2, next, g.len_k);
    Keys<kWide> after = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, 2);
    __syncthreads();
    auto step = [&](auto which, int tile) {
      constexpr int buf = decltype(which)::value;
      const Sight see = ahead;
      auto look_ahead = [&] {
        ahead = sight(next);
        next = after;
        after = keys_of<kWide>(sh.sel, p.lb, p.bs, w0, active, tile + 3);
      };
      if (!see.any) {
        kin.store(sh.k[buf ^ 1]);
        vin.store(sh.v[buf ^ 1]);
        kin.load(kbase, p.k_t * 2, after, g.len_k);
        vin.load(vbase, p.v_t * 2, after, g.len_k);
        look_ahead();
        return;
      }
      f32x16 s[kParts];
      {
        u32x4 ka[kParts][D / 16];
#pragma unroll
        for (int mt = 0; mt < kParts; ++mt)
#pragma unroll
          for (int i = 0; i < D / 16; ++i) ka[mt][i] = rd.row(buf * kBuf, mt * 32, i);
#pragma unroll
        for (int mt = 0; mt < kParts; ++mt) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[mt][r] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) s[mt] = T::mfma32(ka[mt][i], q[i], s[mt]);
        }
        kin.store(sh.k[buf ^ 1]);
        vin.store(sh.v[buf ^ 1]);
        // reads of the first 32 keys, then a product and a read of the others in
        // turn, then a product and a write
        __builtin_amdgcn_sched_group_barrier(0x100, D / 16, 0);
        if constexpr (!kSplit) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        }
      }
      if (see.partial) {
#pragma unroll
        for (int mt = 0; mt < kParts; ++mt)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int off = 8 * ((r >> 2) & 1) + (r & 3);
            if (off + 4 * half > see.last[mt * 2 + (r >> 3)]) s[mt][r] = -kInf;
          }
      }
      // a row sees all of a 16-key group, nothing of it, or what was just masked
      float top = -kInf;
#pragma unroll
      for (int i = 0; i < 2 * kParts; ++i) {
        float t = s[i >> 1][8 * (i & 1)];
#pragma unroll
        for (int r = 1; r < 8; ++r) t = fmaxf(t, s[i >> 1][8 * (i & 1) + r]);
        top = fmaxf(top, sees<kWide>(see, i) ? t : -kInf);
      }
      top = half_max(top);
      // The weights stay relative to an older maximum until it is passed by
      // 2^8: their sums are divided out at the end, and a weight keeps its bits.
      if (__any((top - m) * c > 8.f || (m == -kInf && top > m))) {
        const float now = fmaxf(m, top);
        const float shrink = now == -kInf ? 1.f : exp2_fast((m - now) * c);
        m = now;
        sum *= shrink;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][r] *= shrink;
      }
      kin.load(kbase, p.k_t * 2, after, g.len_k);
      vin.load(vbase, p.v_t * 2, after, g.len_k);
      const float base = m == -kInf ? 0.f : m * c - kRoom<T>;
      u32x4 pr[2 * kParts];
#pragma unroll
      for (int i = 0; i < 2 * kParts; ++i) {
        const float from = sees<kWide>(see, i) ? base : kInf;
        float w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = exp2_fast(fmaf(s[i >> 1][8 * (i & 1) + r], c, -from));
#pragma unroll
        for (int r = 0; r < 4; ++r) pr[i][r] = T::pack(w[2 * r], w[2 * r + 1]);
        sum += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        if constexpr (kRest) {
#pragma unroll
          for (int r = 0; r < 8; ++r) s[i >> 1][8 * (i & 1) + r] = w[r];
        }
      }
      {
        u32x4 va[D / 32][2 * kParts];
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int st = 0; st < 2 * kParts; ++st) va[i][st] = rd.column((2 + buf) * kBuf, 16 * st, i);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int st = 0; st < 2 * kParts; ++st) acc[i] = T::mfma32(va[i][st], pr[st], acc[i]);
        if constexpr (kRest) {
          // the second terms read V again: its operands do not fit beside them
#pragma unroll
          for (int st = 0; st < 2 * kParts; ++st) {
            u32x4 low;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              low[r] = T::pack(s[st >> 1][8 * (st & 1) + 2 * r] - T::lo(pr[st][r]), s[st >> 1][8 * (st & 1) + 2 * r + 1] - T::hi(pr[st][r]));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] = T::mfma32(rd.column((2 + buf) * kBuf, 16 * st, i), low, acc[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {  // the loads between the exponentials
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 64 * kParts / (D / 16), 0);
          }
          read_ahead<D / 16 * kParts, 4, 2>();
        }
      }
      look_ahead();
    };
    for (int tile = 0; tile < tiles; tile += 2) {
      step(Int<0>{}, tile);
      __syncthreads();
      if (tile + 1 < tiles) {
        step(Int<1>{}, tile + 1);
        __syncthreads();
      }
    }
  }
  sum = half_sum(sum);
  bool last = true;  // this wavefront has its rows' results
  if constexpr (kSplit) {
    last = keys32 == 0;
    float* box = reinterpret_cast<float*>(smem) + rows32 * 64 + lane;
    if (!last) {
      box[0] = m;
      box[128] = sum;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) box[(2 + i * 16 + r) * 128] = acc[i][r];
    }
    __syncthreads();
    if (last) {
      const float other = box[0], top = fmaxf(m, other);
      const float f = m == -kInf ? 0.f : exp2_fast((m - top) * c), fo = other == -kInf ? 0.f : exp2_fast((other - top) * c);
      m = top;
      sum = sum * f + box[128] * fo;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = acc[i][r] * f + box[(2 + i * 16 + r) * 128] * fo;
    }
  }
  // An infinity or NaN that a row does not see can have come in through the
  // products, as 0 times it
  bool odd = !(fabsf(sum) < kInf);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd |= !(fabsf(acc[i][r]) < kInf);
  if (__syncthreads_or(valid && last && odd)) {
    if constexpr (kRest) one_by_one<T, D, kRest>(p, sh.sel);
    else one_by_one_called<T, D>((const Args*)__builtin_amdgcn_kernarg_segment_ptr(), &sh.sel);
    return;
  }
  if (valid && last) store_row<T, D, kRest>(p, tok, head, half, acc, m, sum, kRoom<T> > 0.f ? 128.f : 1.f);
}

template <typename T, int D, bool kSplit>
int launch_as(const Args& p, hipStream_t stream) {
  const int64_t grid = p.slots * p.kv_heads;
  if (grid > INT32_MAX) return MI_ATTN_EINVAL;
  const dim3 g(static_cast<unsigned>(grid)), b(256);
  const size_t lds = sizeof(Shared<T, D>);
  if (p.lb >= 6) {
    if (p.rest != nullptr) block_attention_kernel<T, D, true, true, kSplit><<<g, b, lds, stream>>>(p);
    else block_attention_kernel<T, D, true, false, kSplit><<<g, b, lds, stream>>>(p);
  } else {
    if (p.rest != nullptr) block_attention_kernel<T, D, false, true, kSplit><<<g, b, lds, stream>>>(p);
    else block_attention_kernel<T, D, false, false, kSplit><<<g, b, lds, stream>>>(p);
  }
  return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH;
}

template <typename T, int D>
int launch(const Args& p, hipStream_t stream) {
  Args few = p;
  return split_rows(few, D) ? launch_as<T, D, true>(few, stream) : launch_as<T, D, false>(p, stream);
}

}  // namespace

// Checks what the forward and the backward share and fills the kernels' form.
int make_args(const mi_block_attention_args* a, Args& p) {
  if (a == nullptr) return MI_ATTN_EINVAL;
  if (a->total_q < 0 || a->total_q > INT32_MAX || a->total_k < 0 || a->total_k > INT32_MAX || a->num_seqs < 0) return MI_ATTN_EINVAL;
  if (a->dtype != MI_ATTN_BF16 && a->dtype != MI_ATTN_FP16) return MI_ATTN_EINVAL;
  if (a->dim != 64 && a->dim != 128) return MI_ATTN_EINVAL;
  if (a->block_size != 16 && a->block_size != 32 && a->block_size != 64 && a->block_size != 128) return MI_ATTN_EINVAL;
  if (a->kv_heads < 1 || a->heads < a->kv_heads || a->heads % a->kv_heads || a->heads / a->kv_heads > kRows) return MI_ATTN_EINVAL;
  if (a->select < 1 || a->select > MI_ATTN_MAX_SELECT) return MI_ATTN_EINVAL;
  if (!(a->scale > 0.f) || !(a->scale < kInf)) return MI_ATTN_EINVAL;
  if ((a->cu_q == nullptr || a->cu_k == nullptr) && (a->cu_q != a->cu_k || a->num_seqs != 1)) return MI_ATTN_EINVAL;
  const int64_t strides[] = {a->q_stride_t, a->q_stride_h, a->k_stride_t, a->k_stride_h, a->v_stride_t, a->v_stride_h};
  for (int64_t s : strides)
    if (s < 0 || (s & 7)) return MI_ATTN_EINVAL;
  if (a->k_stride_t >= MI_ATTN_MAX_STRIDE || a->v_stride_t >= MI_ATTN_MAX_STRIDE) return MI_ATTN_EINVAL;
  const bool some_q = a->total_q > 0, some_k = a->total_k > 0;
  if (some_q && (a->q == nullptr || a->blocks == nullptr || a->out == nullptr || a->lse == nullptr)) return MI_ATTN_EINVAL;
  if (some_k && (a->k == nullptr || a->v == nullptr)) return MI_ATTN_EINVAL;
  const void* wide[] = {a->q, a->k, a->v, a->out, a->rest};
  for (const void* x : wide)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return MI_ATTN_EINVAL;
  const void* words[] = {a->blocks, a->cu_q, a->cu_k, a->lse};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MI_ATTN_EINVAL;
  p.q = a->q; p.k = a->k; p.v = a->v; p.blocks = a->blocks; p.cu_q = a->cu_q; p.cu_k = a->cu_k;
  p.out = a->out; p.rest = a->rest; p.lse = a->lse; p.dout = a->dout; p.dq = a->dq; p.dk = a->dk; p.dv = a->dv;
  p.q_t = a->q_stride_t; p.q_h = a->q_stride_h; p.k_t = a->k_stride_t; p.k_h = a->k_stride_h;
  p.v_t = a->v_stride_t; p.v_h = a->v_stride_h; p.do_t = a->dout_stride_t; p.do_h = a->dout_stride_h;
  p.total_q = a->total_q; p.total_k = a->total_k;
  p.num_seqs = a->num_seqs; p.heads = a->heads; p.kv_heads = a->kv_heads; p.group = a->heads / a->kv_heads;
  p.bs = a->block_size; p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size));
  p.select = a->select; p.causal = a->causal != 0; p.scale = a->scale;
  p.tokens_per = kRows / p.group;
  p.select_magic = static_cast<uint32_t>(((uint64_t{1} << 32) + p.select - 1) / p.select);
  p.slots = slots_of(p.total_q, p.num_seqs, p.tokens_per);
  return MI_ATTN_OK;
}

}  // namespace miattn

using namespace miattn;

MI_ATTN_EXPORT int block_attention(const mi_block_attention_args* args, hipStream_t stream) {
  Args p;
  const int st = make_args(args, p);
  if (st != MI_ATTN_OK || p.total_q == 0) return st;
  if (args->dtype == MI_ATTN_BF16) return args->dim == 128 ? launch<Bf16, 128>(p, stream) : launch<Bf16, 64>(p, stream);
  return args->dim == 128 ? launch<Fp16, 128>(p, stream) : launch<Fp16, 64>(p, stream);
}
