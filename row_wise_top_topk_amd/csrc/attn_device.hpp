// Device helpers shared by the attention kernels for gfx950 (CDNA4): element
// types, matrix-core wrappers, LDS tiles and the packed-sequence lookup.
//
// Matrix layouts used here (64 lanes, l = lane):
//   32x32x16: A lane l holds row l & 31, k = (l >> 5) * 8 + j;  B lane l holds
//   column l & 31, k likewise;  C lane l holds column l & 31, rows
//   8 * (r >> 2) + 4 * (l >> 5) + (r & 3), r = 0..15.
//   16x16x32: A row / B column l & 15, k = (l >> 4) * 8 + j;  C column l & 15,
//   rows 4 * (l >> 4) + r, r = 0..3.
// Scores are computed transposed (keys as rows), so that a lane holds one
// query's scores: the softmax statistics stay within a lane and its partners,
// and the probabilities are already in the B layout of the second product up
// to a permutation of the keys, which the transposing LDS reads of V follow.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace miattn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define MI_LDS __attribute__((address_space(3)))
#define MI_GLOBAL __attribute__((address_space(1)))

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

template <int n>
struct Int {
  static constexpr int value = n;
};

struct Bf16 {
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  // two floats rounded to nearest even, packed (x in the low half)
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
};

struct Fp16 {
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), f16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t v) { return static_cast<float>(__builtin_bit_cast(f16x2, v)[0]); }
  static __device__ __forceinline__ float hi(uint32_t v) { return static_cast<float>(__builtin_bit_cast(f16x2, v)[1]); }
};

// 8 e4m3 codes, times the power of two `up`: exactly, but for what passes T's range.
template <typename T>
__device__ __forceinline__ u32x4 widen(u32x2 c, float up = 1.f) {
  u32x4 r;
  if constexpr (__is_same(T, Bf16)) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], up, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], up, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], up, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], up, true));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], up, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], up, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], up, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], up, true));
  }
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Address of a shared-memory byte as the LDS builtins take it.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const MI_LDS void*)p));
}

__device__ __forceinline__ u32x4 lds_read16(uint32_t at) {
  return *reinterpret_cast<const MI_LDS u32x4*>(at);
}

// Four rows of 16 elements transposed within each 16-lane group: lane i reads
// 8 bytes (row i >> 2, elements 4 (i & 3)..) and gets element i of the rows.
__device__ __forceinline__ u32x2 lds_read_tr16(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<MI_LDS s16x4*>(at)));
}

// Eight rows of 16 bytes transposed likewise: lane i reads 8 bytes (row i >> 1,
// half i & 1) and gets byte i of the rows.
__device__ __forceinline__ u32x2 lds_read_tr8(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<MI_LDS i32x2*>(at)));
}

// A tile of rows of D 16-bit elements in LDS: 16-byte chunks, chunk c of row r
// at place c ^ swizzle(r).  The swizzle takes rows within a group of four to
// different quarters of a row and rows four apart to different halves of a
// quarter, so that the row reads (16 lanes, 16 rows, one chunk) and the
// transposing reads (32 lanes: 4 rows of 4 chunks, or 8 rows of 2) touch every
// bank once.
template <int D>
__device__ __forceinline__ uint32_t swizzle(uint32_t row) {
  const uint32_t low = ((row >> 1) & 2u) | ((row >> 3) & 1u);
  return D == 128 ? ((row & 3u) << 2) | low : (((row >> 1) & 1u) << 2) | low;
}

template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t row, uint32_t chunk) {
  return row * (2 * D) + ((chunk ^ swizzle<D>(row)) << 4);
}

// Which packed sequence a tile slot belongs to.  Sequence i owns the slots
// [cu[i] / per + i, cu[i + 1] / per + i + 1), at least as many as it has tiles
// of `per` tokens (with one token a tile, exactly [cu[i], cu[i + 1])); sequence
// `num` stands for the rows behind the last one.  Without cu there is one
// sequence, or one token for each of several.
inline int64_t slots_of(int64_t total, int num, int per) { return per == 1 ? total : total / per + num + 1; }

struct Place {
  int seq;        // num for rows behind the last sequence
  int64_t first;  // first token of the tile
  int64_t end;    // end of the sequence
  int64_t begin;
};

// (totals are below 2^31: 32-bit arithmetic, 64-bit division is slow)
__device__ __forceinline__ int32_t cu_at(const int32_t* cu, int num, int64_t total64, int i) {
  const int32_t total = static_cast<int32_t>(total64);
  if (i > num) return total;
  if (cu == nullptr) return num == 1 ? (i == 0 ? 0 : total) : min(i, total);
  return max(0, min(cu[i], total));
}

// For a slot that is the same in the whole wavefront: 64 sequences are looked
// at together, and what belongs to them is loaded beside them, so that a search
// costs about one load's time for each 64 sequences up to the one it finds.
// also(i) is loaded for sequence i; what it gave for the one found, and for the
// next, come back in x0 and x1.
template <typename F>
__device__ __forceinline__ Place place_of(const int32_t* cu, int num, int64_t total, int64_t slot, int per, F also, int32_t& x0, int32_t& x1) {
  const uint32_t extra = per == 1 ? 0 : 1, wide = static_cast<uint32_t>(per);
  const int lane = static_cast<int>(__lane_id());
  int seq = -1, first = 0;  // the last i with first slot <= slot; the first of the 64 looked at
  int32_t c = 0, x = 0;
  for (int i0 = 0; i0 <= num; i0 += 64) {
    const int i = i0 + lane;
    first = i0;
    c = cu_at(cu, num, total, i);
    x = also(i);
    const bool before = i <= num && static_cast<uint32_t>(c) / wide + i * extra <= static_cast<uint32_t>(slot);
    const int n = __popcll(__ballot(before));
    seq += n;
    if (n < 64) break;
  }
  Place r;
  r.seq = __builtin_amdgcn_readfirstlane(seq < 0 ? 0 : seq);
  // the sequence lies among the last 64 looked at, or just before them
  auto pick = [&](int32_t mine, int i, auto value) {
    return i >= first && i < first + 64 ? __builtin_amdgcn_readlane(mine, i - first) : __builtin_amdgcn_readfirstlane(value(i));
  };
  auto at = [&](int i) { return cu_at(cu, num, total, i); };
  const uint32_t begin = pick(c, r.seq, at);
  r.begin = begin;
  r.end = pick(c, r.seq + 1, at);
  x0 = pick(x, r.seq, also);
  x1 = pick(x, r.seq + 1, also);
  r.first = r.begin + (slot - (begin / wide + r.seq * extra)) * per;
  return r;
}

__device__ __forceinline__ Place place_of(const int32_t* cu, int num, int64_t total, int64_t slot, int per) {
  int32_t x0, x1;
  return place_of(cu, num, total, slot, per, [](int) { return 0; }, x0, x1);
}

// Maximum and sum over a lane and its partner in the other half wavefront.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (those of one
// column of a 16x16 result): each gets it.
__device__ __forceinline__ float quad_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Where a lane reads a tile in LDS for 16x16x32 products.  By rows: row lane & 15
// of 16, 8 elements from 32 i + 8 (lane >> 4) on.  Transposed: of 32 rows, rows
// 4 (lane >> 4) .. + 3 and those 16 behind them, column 16 i + (lane & 15); that
// is the order in which two results of 16 rows lie in a lane's registers.
template <int D>
struct Reads16 {
  uint32_t by_row, by_column;
  __device__ __forceinline__ Reads16() {
    const uint32_t lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
    by_row = tile_at<D>(li, g);
    by_column = tile_at<D>(4 * g + (li >> 2), (li & 3) >> 1) + (li & 1) * 8;
  }
  // operand i of the 16 rows from `rows` on (a multiple of 16)
  __device__ __forceinline__ u32x4 row(uint32_t tile, int rows, int i) const { return lds_read16((tile + (by_row ^ (i * 64))) + rows * (2 * D)); }
  // operand of the 32 rows from `rows` on (a multiple of 16), columns 16 i ..
  __device__ __forceinline__ u32x4 column(uint32_t tile, int rows, int i) const {
    const uint32_t at = tile + (by_column ^ (i * 32));
    const u32x2 a = lds_read_tr16(at + rows * (2 * D)), b = lds_read_tr16(at + (rows + 16) * (2 * D));
    return u32x4{a[0], a[1], b[0], b[1]};
  }
};

}  // namespace miattn
