// The pages of a paged cache: forks, growth and compaction of a block table's
// rows, and the copies of pages that they ask for.
//
// A page is free where its count of holders is not above 0.  A first kernel turns
// the counts into one bit a page (a wavefront's ballot is a word) and a number of
// free pages for each 4096; F(p), the number of free pages below p, is then a sum
// of those numbers and of a few words' bits, so that the r-th free page is found
// by one wavefront in two scans, and a page's own rank by two loads.  No kernel
// waits for another workgroup, and only counts of holders and the least numbers of
// forks are changed by atomics (integers: their order does not matter).  What the rows
// before a row ask for is summed over groups of 1024 first, so that a call's work grows
// with the rows, and with their square by a thousandth of it only (2^20 rows that all
// ask: 1.9 ms to fork and 2.2 to grow, where sums row by row took 284 and 211).
//
// The bytes are few (512 rows of 1875 entries: 7 MB with the pages copied, 1.5 us at
// the rate of a large copy), so that these kernels are chains of loads, each behind
// the one before, and of launches: on the device 10.2 us for that fork, 15.3 us for
// 256 rows that end and are filled again, 9.8 us for the list of a compaction.
// What counts is that loads which do not depend on each other are in flight
// together: with a branch around each load of a count, a chunk's free bits took 6.8
// us instead of 4, and eight entries of a row at once instead of one made the fork's
// first kernel 4.9 us instead of 6.5.  A caller without a graph waits for the host:
// 8 us a call and 2.7 us for each further launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention/mi_block_attention.h"
#include "serving/mi_pages.h"

#define MI_PAGES_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kThreads = 256;
constexpr int kWords = 64;              // words of free bits of a chunk
constexpr int kChunk = kWords * 64;     // pages of a chunk
constexpr int64_t kMostBlocks = UINT32_MAX / kThreads;  // a launch has less than 2^32 threads
constexpr int kAtOnce = 8;              // entries of a row that a thread has in flight
constexpr int kGroup = 1024;            // rows whose asks are summed once for all rows behind them

struct PagesArgs {
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  const int32_t* in;
  int32_t* out;
  uint64_t* words;   // [chunks * kWords] bit set: the page is free
  int32_t* counts;   // [chunks] free pages
  int32_t* before;   // compact: [chunks * kWords] free pages below the word's first one
  int32_t* asks;     // fork, grow: [rows] pages that a row asks for
  int64_t* sums;     // fork, grow: [groups] pages that a group's rows ask for
  int32_t* first;    // fork of many rows: [rows] who keeps the row's last page: -1 the row itself, else the first fork
  int32_t* source;   // fork: [rows] page to copy, -1: none
  int32_t* length;   // fork: [rows] new lengths
  int32_t* rows_new; // fork: [rows][cols] new entries
  int64_t pages, stride, chunks;
  int32_t rows, cols, lb;
};

__device__ __forceinline__ int wave_scan(int x) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

template <typename N>
__device__ __forceinline__ N wave_sum(N x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

// Sums over the workgroup; every thread gets them.
template <typename T, int N>
__device__ __forceinline__ void block_sums(T (&x)[N], T (*box)[kThreads / 64]) {
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = wave_sum(x[i]);
    if ((threadIdx.x & 63) == 0) box[i][threadIdx.x >> 6] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) x[i] += box[i][w];
  }
}

__device__ __forceinline__ int block_sum(int x, int* box) {
  int all[1] = {x};
  block_sums(all, reinterpret_cast<int(*)[kThreads / 64]>(box));
  return all[0];
}

__device__ __forceinline__ int length_of(const PagesArgs& p, int row) {
  const int64_t most = static_cast<int64_t>(p.cols) << p.lb;
  const int n = p.lengths[row];
  return n < 0 ? 0 : (n < most ? n : static_cast<int>(most));
}

__device__ __forceinline__ int pages_of(const PagesArgs& p, int64_t tokens) { return static_cast<int>((tokens + (1 << p.lb) - 1) >> p.lb); }

// Free bits and their number of chunk `chunk`.
__device__ __forceinline__ void free_bits(const PagesArgs& p, int64_t chunk, int* box) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kMine = kWords / (kThreads / 64);
  const int64_t first = chunk * kChunk + wave * kMine * 64 + lane;
  int32_t held[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) held[i] = p.refs[min(first + i * 64, p.pages - 1)];  // (a branch here would wait for each load)
  uint64_t mine = 0;
  int count = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const uint64_t bits = __ballot(held[i] <= 0 && first + i * 64 < p.pages);
    if (lane == i) mine = bits;
    count += __popcll(bits);
  }
  if (lane < kMine) p.words[chunk * kWords + wave * kMine + lane] = mine;
  const int all = block_sum(lane == 0 ? count : 0, box);
  if (threadIdx.x == 0) p.counts[chunk] = all;
}

// The place of the free page with `rank` free ones before it: chunk, word and bit.
// For one wavefront, whose lanes agree on rank; chunk is p.chunks where there is none.
struct Spot {
  int64_t chunk;
  int word, bit;
};

__device__ __forceinline__ Spot find_free(const PagesArgs& p, int64_t rank) {
  const int lane = threadIdx.x & 63;
  Spot s{p.chunks, 0, 0};
  for (int64_t c0 = 0; c0 < p.chunks; c0 += 64) {
    const int n = c0 + lane < p.chunks ? p.counts[c0 + lane] : 0;
    const int upto = wave_scan(n);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (rank >= all) {
      rank -= all;
      continue;
    }
    const int at = __ffsll(static_cast<unsigned long long>(__ballot(rank < upto))) - 1;
    rank -= __builtin_amdgcn_readlane(upto - n, at);
    s.chunk = c0 + at;
    break;
  }
  if (s.chunk >= p.chunks) return s;
  const uint64_t word = p.words[s.chunk * kWords + lane];
  const int n = __popcll(word), upto = wave_scan(n);
  const uint64_t reach = __ballot(rank < upto);
  if (reach == 0) {  // the words are not those that were counted: another call wrote into this workspace
    s.chunk = p.chunks;
    return s;
  }
  s.word = __ffsll(static_cast<unsigned long long>(reach)) - 1;
  const int left = static_cast<int>(rank) - __builtin_amdgcn_readlane(upto - n, s.word);
  const uint64_t bits = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(word), s.word)) & 0xffffffffu;
  const uint64_t high = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(word >> 32), s.word)));
  const uint64_t both = bits | (high << 32);
  const bool it = ((both >> lane) & 1) && __popcll(both & ((1ull << lane) - 1)) == left;
  s.bit = __ffsll(static_cast<unsigned long long>(__ballot(it))) - 1;
  return s;
}

// Fork of many rows, before the first step: who keeps each row's last page.
__global__ void __launch_bounds__(kThreads) fork_clear_kernel(PagesArgs p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (row < p.rows) p.first[row] = p.rows;
}

__global__ void __launch_bounds__(kThreads) fork_first_kernel(PagesArgs p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (row >= p.rows) return;
  const int parent = p.in[row];
  if (parent >= 0 && parent < p.rows) atomicMin(p.first + parent, parent == row ? -1 : static_cast<int>(row));
}

// Fork, first step: what each row becomes, beside the table, since others may
// still read what it was.  One workgroup a row.
__global__ void __launch_bounds__(kThreads) fork_rows_kernel(PagesArgs p) {
  __shared__ int s_first;
  const int row = blockIdx.x, tid = threadIdx.x;
  const int parent = p.in[row];
  if (parent == row) {
    if (tid == 0) {
      p.asks[row] = 0;
      p.source[row] = -1;
    }
    return;
  }
  const bool ends = parent < 0 || parent >= p.rows;
  const int length = ends ? 0 : length_of(p, parent);
  const int whole = length >> p.lb;
  bool part = (length & ((1 << p.lb) - 1)) != 0, holds = false;
  int32_t* mine = p.table + row * p.stride;
  const int32_t* from = p.table + (ends ? row : parent) * p.stride;
  int source = -1;
  if (part) {
    source = from[whole];
    // who keeps the parent's last page: the parent, or the first of its forks
    if (p.first != nullptr) {
      holds = p.first[parent] == row;
    } else {
      if (tid == 0) s_first = p.in[parent] == parent ? -1 : row;
      __syncthreads();
      if (s_first >= 0) {
        for (int i = tid; i < row; i += kThreads)
          if (p.in[i] == parent) {
            atomicMin(&s_first, i);
            break;
          }
        __syncthreads();
      }
      holds = s_first == row;
    }
    if (source < 0 || source >= p.pages) {  // not there: handed on as it is
      holds = true;
      source = -1;
    }
  }
  const int had = pages_of(p, length_of(p, row)), has = whole + (part && holds ? 1 : 0);
  int32_t* next = p.rows_new + static_cast<int64_t>(row) * p.cols;
  for (int c0 = tid; c0 < p.cols; c0 += kThreads * kAtOnce) {
    int old[kAtOnce], now[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * kThreads;
      old[i] = c < had ? mine[c] : -1;
      now[i] = c < has ? from[c] : -1;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * kThreads;
      if (c < p.cols) next[c] = now[i];
      if (old[i] != now[i]) {  // forks of one parent share most of what they had
        if (old[i] >= 0 && old[i] < p.pages) atomicAdd(p.refs + old[i], -1);
        if (now[i] >= 0 && now[i] < p.pages) atomicAdd(p.refs + now[i], 1);
      }
    }
  }
  if (tid == 0) {
    p.asks[row] = part && !holds;
    p.source[row] = part && !holds ? source : -1;
    p.length[row] = length;
  }
}

// Fork, second step: the free pages, what the groups of rows (but the last) ask for,
// and the rows' new entries to the table.
__global__ void __launch_bounds__(kThreads) fork_write_kernel(PagesArgs p) {
  __shared__ int box[kThreads / 64];
  if (blockIdx.x < p.chunks) {
    free_bits(p, blockIdx.x, box);
    return;
  }
  const int64_t place = blockIdx.x - p.chunks;
  if (place >= p.rows) {
    const int32_t* asks = p.asks + (place - p.rows) * kGroup;
    int all = 0;
#pragma unroll
    for (int i = 0; i < kGroup / kThreads; ++i) all += asks[i * kThreads + threadIdx.x];
    all = block_sum(all, box);
    if (threadIdx.x == 0) p.sums[place - p.rows] = all;
    return;
  }
  const int row = static_cast<int>(place);
  if (p.in[row] == row) return;
  const int32_t* next = p.rows_new + static_cast<int64_t>(row) * p.cols;
  int32_t* mine = p.table + row * p.stride;
  for (int c0 = threadIdx.x; c0 < p.cols; c0 += kThreads * kAtOnce) {
    int now[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) now[i] = c0 + i * kThreads < p.cols ? next[c0 + i * kThreads] : 0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (c0 + i * kThreads < p.cols) mine[c0 + i * kThreads] = now[i];
  }
}

// Fork, third step: pages for the forks' last tokens, and lengths.  A wavefront a row.
__global__ void __launch_bounds__(kThreads) fork_last_kernel(PagesArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int parent = p.in[row], asks_here = p.asks[row], length_new = p.length[row], from = p.source[row];
  const bool stays = parent == row;  // (then it has no new length)
  int source = -1, page = -1, length = stays ? 0 : length_new;
  if (asks_here != 0) {
    source = from;
    int rank = 0;  // (no row asks for more than one)
    const int64_t group = row / kGroup;
    for (int64_t i0 = group * kGroup + lane; i0 < row; i0 += 64 * kAtOnce) {
      int asks[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) asks[i] = p.asks[min(i0 + i * 64, row)];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) rank += i0 + i * 64 < row ? asks[i] : 0;
    }
    for (int64_t g = lane; g < group; g += 64) rank += static_cast<int>(p.sums[g]);
    const Spot s = find_free(p, wave_sum(rank));
    const int whole = length >> p.lb;
    if (s.chunk < p.chunks) {
      page = static_cast<int>(s.chunk * kChunk + s.word * 64 + s.bit);
      if (lane == 0) {
        p.refs[page] = 1;
        p.table[row * p.stride + whole] = page;
      }
    } else {
      length = whole << p.lb;
    }
  }
  if (lane == 0) {
    if (!stays) p.lengths[row] = length;
    p.out[row * 2] = source;
    p.out[row * 2 + 1] = page;
  }
}

// Grow, first step: the free pages, what each row asks for (-1: its table is too
// narrow), and what a group of rows does.
__global__ void __launch_bounds__(kThreads) grow_ask_kernel(PagesArgs p) {
  __shared__ int box[kThreads / 64];
  __shared__ int64_t wide[1][kThreads / 64];
  if (blockIdx.x < p.chunks) {
    free_bits(p, blockIdx.x, box);
    return;
  }
  const int64_t group = blockIdx.x - p.chunks;
  constexpr int kMine = kGroup / kThreads;
  int given[kMine], lengths[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int row = static_cast<int>(min(group * kGroup + i * kThreads + threadIdx.x, static_cast<int64_t>(p.rows - 1)));
    given[i] = p.in[row];
    lengths[i] = length_of(p, row);
  }
  int64_t all[1] = {0};
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int64_t row = group * kGroup + i * kThreads + threadIdx.x;
    const int64_t more = given[i] < 0 ? 0 : given[i], want = (lengths[i] + more + (1 << p.lb) - 1) >> p.lb;
    const int asks = want > p.cols ? -1 : static_cast<int>(want) - pages_of(p, lengths[i]);
    if (row < p.rows) {
      p.asks[row] = asks;
      all[0] += max(0, asks);
    }
  }
  block_sums(all, wide);
  if (threadIdx.x == 0) p.sums[group] = all[0];
}

// Grow, second step: one workgroup a row, whose wavefronts share the pages that it
// asks for.
__global__ void __launch_bounds__(kThreads) grow_kernel(PagesArgs p) {
  __shared__ int64_t box[2][kThreads / 64];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int asks = p.asks[row], length = length_of(p, row), had = pages_of(p, length), given = p.in[row];
  int64_t rank = 0;
  bool fits = asks == 0;
  if (asks > 0) {
    int64_t all[2] = {0, 0};  // what the rows before it ask for (entries of a table can pass 32 bits), free pages
    const int64_t group = row / kGroup, first = group * kGroup, within = row - first;
    for (int64_t i = tid; i < max(max(group, within), p.chunks); i += kThreads) {
      const int64_t sum = p.sums[min(i, group)];
      const int ask = p.asks[first + min(i, within)], count = p.counts[min(i, p.chunks)];
      all[0] += (i < group ? sum : 0) + (i < within ? max(0, ask) : 0);
      all[1] += i < p.chunks ? count : 0;
    }
    block_sums(all, box);
    rank = all[0];
    fits = rank + asks <= all[1];
  }
  __syncthreads();  // all have read the length
  if (tid == 0) {
    const int more = given < 0 || !fits ? 0 : given;
    p.out[row] = more;
    if (more > 0) p.lengths[row] = length + more;
  }
  if (asks <= 0 || !fits) return;
  const int share = (asks + kThreads / 64 - 1) / (kThreads / 64);
  int at = wave * share;
  const int to = min(asks, at + share);
  if (at >= to) return;
  Spot s = find_free(p, rank + at);
  const int64_t words_end = p.chunks * kWords;
  int32_t* mine = p.table + row * p.stride + had;
  for (int64_t w0 = s.chunk * kWords + s.word; at < to && w0 < words_end; w0 += 64) {
    const uint64_t words = w0 + lane < words_end ? p.words[w0 + lane] : 0;
    for (int i = 0; i < 64 && at < to; ++i) {
      uint64_t bits = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(words), i))) |
                      static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(words >> 32), i))) << 32;
      bits &= ~0ull << s.bit;  // the first word from its place on
      s.bit = 0;
      const int mine_at = at + __popcll(bits & ((1ull << lane) - 1));
      if (((bits >> lane) & 1) && mine_at < to) {
        const int page = static_cast<int>((w0 + i) * 64 + lane);
        mine[mine_at] = page;
        p.refs[page] = 1;
      }
      at += __popcll(bits);
    }
  }
}

__global__ void __launch_bounds__(kThreads) free_kernel(PagesArgs p) {
  __shared__ int box[kThreads / 64];
  free_bits(p, blockIdx.x, box);
}

// Compact, second step: with n pages in use, page q >= n in use has the rank
// (q - F(q)) - (n - F(n)) among those that move, a free page q < n the rank F(q)
// among those that they move to: each writes its place in the list of moves.
__global__ void __launch_bounds__(kThreads) compact_list_kernel(PagesArgs p) {
  __shared__ int box[kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t chunk = blockIdx.x;
  int lower = 0, all = 0;
  for (int64_t c = tid; c < p.chunks; c += kThreads) {
    const int n = p.counts[c];
    all += n;
    if (c < chunk) lower += n;
  }
  all = block_sum(all, box);
  lower = block_sum(lower, box);
  const int64_t used = p.pages - all;
  const int64_t cut_chunk = used / kChunk;
  int below = 0;  // F(used)
  for (int64_t c = tid; c < cut_chunk; c += kThreads) below += p.counts[c];
  if (tid < kWords && cut_chunk < p.chunks) {
    const int64_t first = cut_chunk * kChunk + tid * 64;
    uint64_t bits = p.words[cut_chunk * kWords + tid];
    if (used <= first) bits = 0;
    else if (used < first + 64) bits &= (1ull << (used - first)) - 1;
    below += __popcll(bits);
  }
  below = block_sum(below, box);
  const int64_t still = used - below;  // in use and below the cut
  const uint64_t own = p.words[chunk * kWords + lane];
  const int count = __popcll(own), start = wave_scan(count) - count + lower;
  if (wave == 0) p.before[chunk * kWords + lane] = start;
  constexpr int kMine = kWords / (kThreads / 64);
  for (int i = 0; i < kMine; ++i) {
    const int w = wave * kMine + i;
    const uint64_t bits = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(own), w))) |
                          static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(own >> 32), w))) << 32;
    const int64_t q = chunk * kChunk + w * 64 + lane;
    const int64_t f = __builtin_amdgcn_readlane(start, w) + __popcll(bits & ((1ull << lane) - 1));
    const bool is_free = (bits >> lane) & 1;
    if (q < p.pages && !is_free && q >= used) p.out[(q - f - still) * 2] = static_cast<int>(q);
    if (q < used && is_free) p.out[f * 2 + 1] = static_cast<int>(q);
  }
  if (chunk == 0 && tid == 0) p.counts[p.chunks] = below;  // the number of moves
}

// Compact, third step: counts of holders, the list's end, and the rows' entries.
__global__ void __launch_bounds__(kThreads) compact_rows_kernel(PagesArgs p, int64_t pair_blocks) {
  const int tid = threadIdx.x;
  const int64_t moves = p.counts[p.chunks];
  if (blockIdx.x < pair_blocks) {
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + tid;
    if (i >= p.pages / 2) return;
    if (i >= moves) {
      p.out[i * 2] = p.out[i * 2 + 1] = -1;
      return;
    }
    const int from = p.out[i * 2], to = p.out[i * 2 + 1];
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
    return;
  }
  const int row = static_cast<int>(blockIdx.x - pair_blocks);
  if (moves == 0) return;
  const int n = pages_of(p, length_of(p, row));
  // the first page that moved, and its rank among the pages in use
  const int first = p.out[0];
  const int64_t still = first - p.before[first >> 6] - __popcll(p.words[first >> 6] & ((1ull << (first & 63)) - 1));
  for (int c = tid; c < n; c += kThreads) {
    const int q = p.table[row * p.stride + c];
    if (q < first || q >= p.pages) continue;
    const uint64_t word = p.words[q >> 6];
    if ((word >> (q & 63)) & 1) continue;  // named, but nothing counts it
    const int64_t f = p.before[q >> 6] + __popcll(word & ((1ull << (q & 63)) - 1));
    p.table[row * p.stride + c] = p.out[(q - f - still) * 2 + 1];
  }
}

// Small tables and caches: one workgroup does all of it, in one launch, with the
// free bits, their running numbers and what belongs to a row in LDS.
constexpr int kSmallThreads = 1024, kSmallRows = 1024, kSmallEntries = 4 * kSmallThreads, kSmallWords = 128;

struct Small {
  uint64_t words[kSmallWords];
  int before[kSmallWords];      // free pages below the word's first one
  int length[kSmallRows];       // as it was
  int parent[kSmallRows];
  int first[kSmallRows];        // fork: who keeps the row's last page: -1 the row itself, else the first fork
  int has[kSmallRows];          // fork: entries that it shares; grow: entries that it has
  int place[kSmallRows];        // fork: the page it gets, -1 for none; grow: the rank of its first new page, -1 for none
  int asks[kSmallRows];
  int box[kSmallThreads / 64 + 1];
};

// Exclusive sum over the workgroup's threads; `all`: the whole.
__device__ __forceinline__ int small_scan(int x, int* box, int& all) {
  const int upto = wave_scan(x), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (lane == 63) box[wave] = upto;
  __syncthreads();
  int lower = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 64; ++w) {
    const int n = box[w];
    if (w < wave) lower += n;
    all += n;
  }
  return lower + upto - x;
}

// The free bits and their running numbers; returns the number of free pages.
__device__ __forceinline__ int small_bits(const PagesArgs& p, Small& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kWaves = kSmallThreads / 64;
  const int pages = static_cast<int>(p.pages), words = (pages + 63) / 64;
  for (int w0 = wave * kAtOnce; w0 < words; w0 += kWaves * kAtOnce) {
    int32_t held[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      // (past the caches: other wavefronts' atomics have changed them)
      held[i] = __hip_atomic_load(p.refs + min((w0 + i) * 64 + lane, pages - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint64_t bits = __ballot(held[i] <= 0 && (w0 + i) * 64 + lane < pages);
      if (lane == 0 && w0 + i < words) s.words[w0 + i] = bits;
    }
  }
  __syncthreads();
  int all;
  const int mine = threadIdx.x < words ? __popcll(s.words[threadIdx.x]) : 0;
  const int lower = small_scan(mine, s.box, all);
  if (threadIdx.x < words) s.before[threadIdx.x] = lower;
  __syncthreads();
  return all;
}

// The free page with `rank` free ones before it, of those that there are.
__device__ __forceinline__ int small_find(const Small& s, int words, int rank) {
  int w = 0;
#pragma unroll
  for (int d = kSmallWords / 2; d > 0; d >>= 1)
    if (w + d < words && s.before[w + d] <= rank) w += d;
  uint64_t bits = s.words[w];
  int left = rank - s.before[w], at = 0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const int n = __popcll(bits & ((1ull << d) - 1));
    if (left >= n) {
      left -= n;
      bits >>= d;
      at += d;
    }
  }
  return w * 64 + at;
}

// Free pages below page q.
__device__ __forceinline__ int small_below(const Small& s, int q) { return s.before[q >> 6] + __popcll(s.words[q >> 6] & ((1ull << (q & 63)) - 1)); }

template <int op>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(PagesArgs p) {
  __shared__ Small s;
  const int tid = threadIdx.x, row = tid, words = static_cast<int>((p.pages + 63) / 64);
  const int bs = 1 << p.lb, entries = p.rows * p.cols;
  int length = 0, given = 0;
  if (row < p.rows) {
    length = length_of(p, row);
    if (op != MI_PAGES_COMPACT) given = p.in[row];
    s.length[row] = length;
  }
  if constexpr (op == MI_PAGES_FORK) {
    const int parent = given;
    const bool stays = row < p.rows && parent == row, ends = parent < 0 || parent >= p.rows;
    if (row < p.rows) {
      s.parent[row] = ends ? -1 : parent;
      s.first[row] = p.rows;
    }
    __syncthreads();
    if (row < p.rows && !ends) atomicMin(&s.first[parent], stays ? -1 : row);
    __syncthreads();
    // what the row becomes: its length, the entries that it shares, and a page that it asks for
    const int now = row < p.rows && !ends ? s.length[parent] : 0, whole = now >> p.lb;
    int source = -1;
    bool asks = false;
    if (row < p.rows) {
      bool holds = (now & (bs - 1)) != 0;
      if (holds && !stays && s.first[parent] != row) {
        source = p.table[parent * p.stride + whole];
        asks = source >= 0 && source < p.pages;  // not there: handed on as it is
        holds = !asks;
      }
      s.has[row] = whole + (holds ? 1 : 0);
    }
    __syncthreads();
    constexpr int kMost = kSmallEntries / kSmallThreads;
    int32_t old[kMost], next[kMost];
    const int turns = (entries + kSmallThreads - 1) / kSmallThreads;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      old[i] = next[i] = -1;
      const int e = i * kSmallThreads + tid;
      if (i < turns && e < entries) {
        const int r = e / p.cols, c = e - r * p.cols, from = s.parent[r];
        if (from != r && c < pages_of(p, s.length[r])) old[i] = p.table[r * p.stride + c];
        if (from != r && c < s.has[r]) next[i] = p.table[from * p.stride + c];
      }
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      if (old[i] != next[i]) {
        if (old[i] >= 0 && old[i] < p.pages) atomicAdd(p.refs + old[i], -1);
        if (next[i] >= 0 && next[i] < p.pages) atomicAdd(p.refs + next[i], 1);
      }
    __threadfence();
    __syncthreads();
    const int free = small_bits(p, s);
    int all;
    const int rank = small_scan(asks ? 1 : 0, s.box, all);
    if (row < p.rows) {
      int page = -1;
      if (asks && rank < free) {
        page = small_find(s, words, rank);
        p.refs[page] = 1;
      }
      s.place[row] = page;
      if (!stays) p.lengths[row] = asks && page < 0 ? whole << p.lb : now;
      p.out[row * 2] = asks ? source : -1;
      p.out[row * 2 + 1] = page;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int e = i * kSmallThreads + tid;
      if (i < turns && e < entries) {
        const int r = e / p.cols, c = e - r * p.cols;
        if (s.parent[r] != r) p.table[r * p.stride + c] = c == s.has[r] && s.place[r] >= 0 ? s.place[r] : next[i];
      }
    }
  } else if constexpr (op == MI_PAGES_GROW) {
    const int free = small_bits(p, s);
    const int64_t more = given < 0 ? 0 : given, want = (length + more + bs - 1) >> p.lb;
    const int had = pages_of(p, length);
    const bool wide = want <= p.cols;
    const int asks = row < p.rows && wide ? static_cast<int>(want) - had : 0;
    int all;
    const int rank = small_scan(asks, s.box, all);
    const bool fits = wide && (asks == 0 || rank + asks <= free);
    if (row < p.rows) {
      s.has[row] = had;
      s.asks[row] = fits ? asks : 0;
      s.place[row] = rank;
      p.out[row] = fits ? static_cast<int>(more) : 0;
      if (fits && more > 0) p.lengths[row] = length + static_cast<int>(more);
    }
    __syncthreads();
    for (int e = tid; e < entries; e += kSmallThreads) {
      const int r = e / p.cols, n = e - r * p.cols - s.has[r];
      if (n >= 0 && n < s.asks[r]) {
        const int page = small_find(s, words, s.place[r] + n);
        p.table[r * p.stride + s.has[r] + n] = page;
        p.refs[page] = 1;
      }
    }
  } else {
    const int free = small_bits(p, s), used = static_cast<int>(p.pages) - free;
    // pages in use below the cut stay; F(used) pages move
    const int moves = used < p.pages ? small_below(s, used) : 0, still = used - moves;
    auto place_of_page = [&](int q) { return q - small_below(s, q) - still; };  // its rank among those that move
    for (int e = tid; e < entries; e += kSmallThreads) {
      const int r = e / p.cols, c = e - r * p.cols;
      if (c >= pages_of(p, s.length[r])) continue;
      const int q = p.table[r * p.stride + c];
      if (q < used || q >= p.pages || ((s.words[q >> 6] >> (q & 63)) & 1)) continue;
      p.table[r * p.stride + c] = small_find(s, words, place_of_page(q));
    }
    for (int q = used + tid; q < p.pages; q += kSmallThreads) {
      if ((s.words[q >> 6] >> (q & 63)) & 1) continue;
      const int i = place_of_page(q), to = small_find(s, words, i);
      p.out[i * 2] = q;
      p.out[i * 2 + 1] = to;
      p.refs[to] = p.refs[q];
      p.refs[q] = 0;
    }
    for (int64_t i = moves + tid; i < p.pages / 2; i += kSmallThreads) p.out[i * 2] = p.out[i * 2 + 1] = -1;
  }
}

// Whether one workgroup does the call: a launch instead of three (two to grow), which
// saves the host 7 us.  Measured on the device (us in a graph, one workgroup against
// several): 64 rows of 55 entries, 2230 pages: fork 10.4, 10.0, grow 6.2, 6.5, compact
// 4.6, 8.9; 4 rows of 32: fork 8.1, 8.7; 256 rows of 55, 10124 pages: fork 15.9, 9.9.
bool is_small(const mi_pages_args* a) {
  return a->rows <= kSmallRows && static_cast<int64_t>(a->rows) * a->block_table_cols <= kSmallEntries && a->num_pages <= kSmallWords * 64;
}

struct CopyArgs {
  char *k, *v;
  float *k_scale, *v_scale;
  float* mean;
  const int32_t* copies;
  int64_t num, pages, page_bytes;
  int32_t heads, mean_floats, parts;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// `parts` workgroups share a pair, and go on to the pair `gridDim / parts` behind it.
// Bound by memory: 5140 pages of 132 KB, read and written, in 266 us (5.1 TB/s; 277 us
// with pointers and bounds looked up between the loads).
__global__ void __launch_bounds__(kThreads) copy_kernel(CopyArgs p) {
  const int tid = threadIdx.x, part = blockIdx.x % p.parts;
  const int64_t step = gridDim.x / p.parts;
  const int64_t each = (2 * p.page_bytes / 16 + p.parts - 1) / p.parts;  // 16-byte pieces of keys and values of a part
  for (int64_t i = blockIdx.x / p.parts; i < p.num; i += step) {
    const int from = p.copies[2 * i], to = p.copies[2 * i + 1];
    if (from < 0 || from >= p.pages || to < 0 || to >= p.pages) continue;
    const int64_t per = p.page_bytes / 16, end = min((part + 1) * each, 2 * per);
    char* to_k = p.k + to * p.page_bytes;
    char* to_v = p.v + to * p.page_bytes;
    const char* from_k = p.k + from * p.page_bytes;
    const char* from_v = p.v + from * p.page_bytes;
    for (int64_t a = part * each + tid; a < end; a += kThreads * 4) {
      u32x4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = min(a + j * kThreads, end - 1);  // (a branch here would wait for each load)
        x[j] = *reinterpret_cast<const u32x4*>((at < per ? from_k : from_v) + (at < per ? at : at - per) * 16);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = a + j * kThreads;
        if (at < end) *reinterpret_cast<u32x4*>((at < per ? to_k : to_v) + (at < per ? at : at - per) * 16) = x[j];
      }
    }
    if (part == 0) {
      for (int h = tid; h < 2 * p.heads; h += kThreads) {
        float* s = h < p.heads ? p.k_scale : p.v_scale;
        const int64_t k = h < p.heads ? h : h - p.heads;
        s[static_cast<int64_t>(to) * p.heads + k] = s[static_cast<int64_t>(from) * p.heads + k];
      }
      for (int d = tid; d < p.mean_floats; d += kThreads)
        p.mean[static_cast<int64_t>(to) * p.mean_floats + d] = p.mean[static_cast<int64_t>(from) * p.mean_floats + d];
    }
  }
}

// Up to so many rows a workgroup looks for a parent's first fork among the rows
// before it; beyond, two launches more find those of all rows at once.  Measured (us
// in a graph, four forks of each parent, 55 entries a row, the scan against the
// launches): 4200 rows: 24.8, 20.0 where no parent goes on, 16.6, 19.5 where all do;
// 8192: 48.5, 26.8 and 25.6, 25.6.  Below, the launches cost 4 us of 11 to 15.
constexpr int kScan = 4096;

bool block_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check(const mi_pages_args* a) {
  if (a == nullptr || !block_ok(a->block_size) || a->op < MI_PAGES_FORK || a->op > MI_PAGES_COMPACT || a->rows < 0 ||
      a->block_table_cols < 0 || a->block_table_stride < a->block_table_cols || a->num_pages < 0 || a->num_pages > INT32_MAX ||
      static_cast<int64_t>(a->block_table_cols) * a->block_size >= (1 << 30))
    return MI_ATTN_EINVAL;
  return MI_ATTN_OK;
}

int64_t chunks_of(const mi_pages_args* a) { return (a->num_pages + kChunk - 1) / kChunk; }

uint64_t up16(uint64_t n) { return (n + 15) & ~uint64_t{15}; }

// Lays the workspace out from `at` (which may be null); returns its size.
uint64_t lay_out(const mi_pages_args* a, char* at, PagesArgs* p) {
  if (is_small(a)) return 0;
  const uint64_t chunks = chunks_of(a), rows = a->rows;
  uint64_t n = 0;
  auto take = [&](uint64_t bytes) {
    char* x = at == nullptr ? nullptr : at + n;
    n += up16(bytes);
    return x;
  };
  PagesArgs none;
  PagesArgs& q = p == nullptr ? none : *p;
  q.words = reinterpret_cast<uint64_t*>(take(chunks * kWords * 8));
  q.counts = reinterpret_cast<int32_t*>(take((chunks + 1) * 4));
  q.before = nullptr;
  q.asks = q.first = q.source = q.length = q.rows_new = nullptr;
  q.sums = nullptr;
  if (a->op == MI_PAGES_COMPACT) q.before = reinterpret_cast<int32_t*>(take(chunks * kWords * 4));
  else q.asks = reinterpret_cast<int32_t*>(take(rows * 4)), q.sums = reinterpret_cast<int64_t*>(take((rows + kGroup - 1) / kGroup * 8));
  if (a->op == MI_PAGES_FORK) {
    q.source = reinterpret_cast<int32_t*>(take(rows * 4));
    q.length = reinterpret_cast<int32_t*>(take(rows * 4));
    q.rows_new = reinterpret_cast<int32_t*>(take(rows * a->block_table_cols * 4));
    if (a->rows > kScan) q.first = reinterpret_cast<int32_t*>(take(rows * 4));
  }
  return n;
}

int launched() { return hipGetLastError() == hipSuccess ? MI_ATTN_OK : MI_ATTN_ELAUNCH; }

}  // namespace

MI_PAGES_EXPORT uint64_t pages_workspace(const mi_pages_args* args) {
  return check(args) == MI_ATTN_OK ? lay_out(args, nullptr, nullptr) : 0;
}

MI_PAGES_EXPORT int pages_update(const mi_pages_args* a, hipStream_t stream) {
  if (check(a) != MI_ATTN_OK) return MI_ATTN_EINVAL;
  const bool compact = a->op == MI_PAGES_COMPACT;
  const bool entries = a->rows > 0 && a->block_table_cols > 0;
  if ((a->rows > 0 && (a->lengths == nullptr || (!compact && (a->given == nullptr || a->out == nullptr)))) ||
      (entries && a->block_table == nullptr) || (a->num_pages > 0 && a->refs == nullptr) ||
      (compact && a->num_pages > 1 && a->out == nullptr))
    return MI_ATTN_EINVAL;
  const void* words[] = {a->block_table, a->lengths, a->refs, a->given, a->out};
  for (const void* x : words)
    if (!aligned(x, 4)) return MI_ATTN_EINVAL;
  if (!aligned(a->workspace, 16)) return MI_ATTN_EINVAL;
  if (compact ? a->num_pages < 2 : a->rows == 0) return MI_ATTN_OK;
  PagesArgs p = {};
  const uint64_t need = lay_out(a, static_cast<char*>(a->workspace), &p);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need)) return MI_ATTN_EWORKSPACE;
  p.table = a->block_table; p.lengths = a->lengths; p.refs = a->refs; p.in = a->given; p.out = a->out;
  p.pages = a->num_pages; p.stride = a->block_table_stride; p.chunks = chunks_of(a);
  p.rows = a->rows; p.cols = a->block_table_cols; p.lb = __builtin_ctz(static_cast<unsigned>(a->block_size));
  if (is_small(a)) {
    const dim3 one(1), all(kSmallThreads);
    if (a->op == MI_PAGES_FORK) small_kernel<MI_PAGES_FORK><<<one, all, 0, stream>>>(p);
    else if (a->op == MI_PAGES_GROW) small_kernel<MI_PAGES_GROW><<<one, all, 0, stream>>>(p);
    else small_kernel<MI_PAGES_COMPACT><<<one, all, 0, stream>>>(p);
    return launched();
  }
  const dim3 b(kThreads);
  auto blocks = [](int64_t n) { return dim3(static_cast<unsigned>(n)); };
  if (a->op == MI_PAGES_FORK) {
    const int64_t groups = (static_cast<int64_t>(p.rows) - 1) / kGroup, wide = (static_cast<int64_t>(p.rows) + kThreads - 1) / kThreads;
    if (p.chunks + p.rows + groups > kMostBlocks) return MI_ATTN_EINVAL;
    if (p.first != nullptr) {
      fork_clear_kernel<<<blocks(wide), b, 0, stream>>>(p);
      fork_first_kernel<<<blocks(wide), b, 0, stream>>>(p);
    }
    fork_rows_kernel<<<blocks(p.rows), b, 0, stream>>>(p);
    fork_write_kernel<<<blocks(p.chunks + p.rows + groups), b, 0, stream>>>(p);
    fork_last_kernel<<<blocks((static_cast<int64_t>(p.rows) + 3) / 4), b, 0, stream>>>(p);
  } else if (a->op == MI_PAGES_GROW) {
    if (p.rows > kMostBlocks) return MI_ATTN_EINVAL;
    grow_ask_kernel<<<blocks(p.chunks + (static_cast<int64_t>(p.rows) + kGroup - 1) / kGroup), b, 0, stream>>>(p);
    grow_kernel<<<blocks(p.rows), b, 0, stream>>>(p);
  } else {
    const int64_t pairs = (p.pages / 2 + kThreads - 1) / kThreads;
    if (pairs + p.rows > kMostBlocks) return MI_ATTN_EINVAL;
    free_kernel<<<blocks(p.chunks), b, 0, stream>>>(p);
    compact_list_kernel<<<blocks(p.chunks), b, 0, stream>>>(p);
    compact_rows_kernel<<<blocks(pairs + (entries ? p.rows : 0)), b, 0, stream>>>(p, pairs);
  }
  return launched();
}

MI_PAGES_EXPORT int pages_copy(const mi_pages_copy_args* a, hipStream_t stream) {
  if (a == nullptr || !block_ok(a->block_size) || (a->dim != 64 && a->dim != 128) || a->kv_heads < 1 || a->num < 0 ||
      a->num > INT32_MAX || a->num_pages < 0 || a->num_pages > INT32_MAX ||
      static_cast<int64_t>(a->kv_heads) * a->block_size * a->dim > INT32_MAX)
    return MI_ATTN_EINVAL;
  if ((a->num > 0 && a->copies == nullptr) ||
      (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr || a->k_scale == nullptr || a->v_scale == nullptr)))
    return MI_ATTN_EINVAL;
  if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4) ||
      !aligned(a->k_mean, 4) || !aligned(a->copies, 4))
    return MI_ATTN_EINVAL;
  if (a->num == 0 || a->num_pages == 0) return MI_ATTN_OK;
  CopyArgs p;
  p.k = static_cast<char*>(a->k_cache);
  p.v = static_cast<char*>(a->v_cache);
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.mean = a->k_mean;
  p.copies = a->copies;
  p.num = a->num;
  p.pages = a->num_pages;
  p.page_bytes = static_cast<int64_t>(a->kv_heads) * a->block_size * a->dim;
  p.heads = a->kv_heads;
  p.mean_floats = a->k_mean == nullptr ? 0 : a->kv_heads * a->dim;
  const int64_t pieces = (2 * p.page_bytes + 16 * kThreads - 1) / (16 * kThreads);  // a part has 4 KB at least
  int64_t parts = (2048 + p.num - 1) / p.num;
  if (parts > pieces) parts = pieces;
  p.parts = static_cast<int>(parts);
  const int64_t grid = (p.num * parts < 4096 ? p.num : (4096 + parts - 1) / parts) * parts;
  copy_kernel<<<dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream>>>(p);
  return launched();
}
