// Kernels of the embedding (zero_embedding_*).
//
// The lookup copies rows by id, one warp a row. It is bound by memory: 131072 rows
// of width 4096 in bf16, 32620 of them distinct, take 224 us (6.0 TB/s; 266 with
// one access of a lane on its way instead of four).
//
// The gradient adds the rows of dout that have the same id. The tokens are
// sorted by id, stably, so that an id's rows are a segment of the list, in the
// order of the tokens; the list is cut into runs of equal length, one warp a run
// and block of columns, whatever the segments' lengths: a segment within a run
// goes to its row of dweight, and the shares of one that spans runs are kept in
// fp32 and joined in the order of the runs. No atomics touch a value, so equal
// inputs give equal bits. Large ones are bound by memory: 131072 tokens of width
// 4096 and as many ids, bf16, 396 us, of which the sums and zeros take 345 (2.15 GB
// at 6.2 TB/s) and the sort 35; small ones by the latency of three kernels and by
// the zeros: 8192 tokens of a table of 50257 x 768 take 29 us, 21 added to a
// dweight that is there.

#include <cuda_bf16.h>

#include <atomic>

#include "embedding_internal.h"
#include "launch.cuh"

namespace ze {
namespace {

using zl::launch;
using zl::let_next_start;
using zl::wait_for_previous;

template <bool F32>
struct Type;
template <>
struct Type<true> {
  using E = float;
  static constexpr int kVec = 4;
};
template <>
struct Type<false> {
  using E = __nv_bfloat16;
  static constexpr int kVec = 8;
};

// A lane's share of a block of columns of a row: kVec elements, 16 bytes, in pieces
// of the widest accesses that all rows allow -- 16 or 4 bytes, or a bf16 value --
// which the lanes take in turn.
template <bool F32, int Width>
struct Columns {
  using E = typename Type<F32>::E;
  static constexpr int kVec = Type<F32>::kVec;
  static constexpr int kBlock = 32 * kVec;
  static constexpr int kPieces = 16 / Width, kPiece = kVec / kPieces;  // elements of one

  int64_t first;  // of the lane
  int count;      // of its elements that lie inside the row

  __device__ __forceinline__ Columns(int64_t c0, int64_t D, int lane) {
    first = c0 + lane * kPiece;
    const int64_t left = D - first;
    count = int(Width == 16 ? max(int64_t(0), min(int64_t(kVec), left))
                            : max(int64_t(0), min(int64_t(kPieces), (left + 32 * kPiece - 1) / (32 * kPiece))) * kPiece);
  }
  __device__ __forceinline__ int64_t at(int j) const { return first + j / kPiece * (32 * kPiece) + j % kPiece; }

  // The elements as they are stored, those outside the row as zeros. `Once`: they
  // are not read again, or (store) not soon.
  template <bool Once = false>
  __device__ __forceinline__ uint4 load(const void* row) const {
    const E* p = static_cast<const E*>(row);
    if (Width == 16 && count == kVec) {
      const uint4* from = reinterpret_cast<const uint4*>(p + first);
      return Once ? __ldcs(from) : *from;
    }
    uint32_t words[4] = {};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (j >= count) continue;
      if (F32) words[j % 4] = reinterpret_cast<const uint32_t*>(p)[at(j)];
      else if (Width != 4) words[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[at(j)]) << (j % 2 * 16);
      else if (j % 2 == 0) words[j / 2] = *reinterpret_cast<const uint32_t*>(p + at(j));
    }
    return make_uint4(words[0], words[1], words[2], words[3]);
  }
  template <bool Once = false>
  __device__ __forceinline__ void store(void* row, uint4 w) const {
    E* p = static_cast<E*>(row);
    if (Width == 16 && count == kVec) {
      uint4* to = reinterpret_cast<uint4*>(p + first);
      if (Once) __stcs(to, w);
      else *to = w;
      return;
    }
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (j >= count) continue;
      if (F32) reinterpret_cast<uint32_t*>(p)[at(j)] = words[j % 4];
      else if (Width != 4) reinterpret_cast<uint16_t*>(p)[at(j)] = uint16_t(words[j / 2] >> (j % 2 * 16));
      else if (j % 2 == 0) *reinterpret_cast<uint32_t*>(p + at(j)) = words[j / 2];
    }
  }
  __device__ __forceinline__ static void unpack(uint4 w, float (&x)[kVec]) {
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      x[j] = __uint_as_float(F32 ? words[j % 4] : j % 2 ? words[j / 2] & 0xffff0000u : words[j / 2] << 16);
  }
  // Each value rounded once.
  __device__ __forceinline__ static uint4 pack(const float (&x)[kVec]) {
    uint32_t words[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        words[j] = __float_as_uint(x[j]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j % kVec], x[(2 * j + 1) % kVec]);
        words[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(words[0], words[1], words[2], words[3]);
  }
};

template <bool F32>
__device__ __forceinline__ const void* row_of(const void* base, int64_t stride, int64_t row) {
  return static_cast<const typename Type<F32>::E*>(base) + row * stride;
}
template <bool F32>
__device__ __forceinline__ void* row_of(void* base, int64_t stride, int64_t row) {
  return static_cast<typename Type<F32>::E*>(base) + row * stride;
}

// ----------------------------------------------------------------- lookup --

// `Stream`: the result is larger than the L2 cache, where it would displace the
// rows that are looked up again.
template <bool F32, int Width, bool Stream>
__global__ void __launch_bounds__(256) lookup_kernel(const Args a) {
  using C = Columns<F32, Width>;
  constexpr int kAhead = 4;  // loads in flight
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * 8;
  for (int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); t < a.T; t += step) {
    const int64_t id = a.ids[t];
    const bool there = id >= 0 && id < a.V;
    const void* from = row_of<F32>(a.table, a.table_stride, there ? id : 0);
    void* to = row_of<F32>(a.out, a.out_stride, t);
    for (int64_t c0 = 0; c0 < a.D; c0 += kAhead * C::kBlock) {
      uint4 w[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const C c(c0 + q * C::kBlock, a.D, lane);
        w[q] = there && c.count > 0 ? c.load(from) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const C c(c0 + q * C::kBlock, a.D, lane);
        if (c.count == 0) break;
        if (there && a.scale != 1.0f) {
          float x[C::kVec];
          C::unpack(w[q], x);
#pragma unroll
          for (int j = 0; j < C::kVec; ++j) x[j] *= a.scale;
          w[q] = C::pack(x);
        }
        c.template store<Stream>(to, w[q]);
      }
    }
  }
}

// ------------------------------------------------------------------- sort --
//
// Few tokens: one kernel, a block for each class of ids (their low bits, so that
// the frequent ids of a vocabulary in order of frequency are spread). Each block
// reads all ids, counts those of smaller classes -- its place in the list --
// gathers its own in order and places them by the rest of their ids, counted warp
// by warp in shared memory: no exchange between blocks, and the same work however
// often an id comes. The list is in order of class, then of id. Blocks behind those
// write dweight's zeros meanwhile: 17 us for 8192 tokens beside 77 MB of zeros,
// which alone take 12. (Keys exchanged in shared memory instead of counted: 30 us for
// the whole gradient instead of 29, 76 instead of 44 where all tokens are one id.)
//
// More tokens: by digits of the id from the lowest, each pass stable: a tile's
// tokens are counted by digit, and the block of that tile adds up what comes before
// -- smaller digits of all tiles, its digit in earlier tiles -- and places its
// tokens, each warp a stretch of them in order, counting the next digit by the
// tiles that they go to. A pass takes 13 us for 131072 tokens, all of it latency:
// the columns of the counts, then the warps' two walks.

constexpr int kClassThreads = 1024;

// Rows `from` to `end` of dweight, by `warps` warps of which this is number `warp`.
// `Array`: rows off 16 bytes without a gap between them are one array of 16-byte words
// and an edge of less than one on either side (145 tokens of 100295 x 1729 in fp32: 118
// us instead of 175, 8192 of 50257 x 769 in bf16 38 instead of 43; beside the passes of
// a longer sort, 100000 of 50257 x 900 in bf16, 95 instead of 92, so not there).
template <bool F32, int Width, bool Array>
__device__ __forceinline__ void zero_rows(const Args& a, int64_t from, int64_t end, int64_t warp, int64_t warps) {
  using C = Columns<F32, Width>;
  const int lane = threadIdx.x & 31;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (Array && Width != 16 && a.out_stride == a.D) {
    using E = typename C::E;
    if (from >= end) return;
    const auto begin = reinterpret_cast<uintptr_t>(row_of<F32>(a.out, a.D, from));
    const auto stop = reinterpret_cast<uintptr_t>(row_of<F32>(a.out, a.D, end));
    const uintptr_t first = (begin + 15) / 16 * 16, last = stop / 16 * 16;  // of the words
    for (uintptr_t p = first + uintptr_t(warp * 32 + lane) * 16; p < last; p += uintptr_t(warps) * 512)
      *reinterpret_cast<uint4*>(p) = zero;
    if (warp == 0) {
      const uintptr_t head = begin + lane * sizeof(E), tail = (first > last ? first : last) + lane * sizeof(E);
      if (head < first && head < stop) *reinterpret_cast<E*>(head) = E(0.0f);
      if (tail < stop) *reinterpret_cast<E*>(tail) = E(0.0f);
    }
    return;
  }
  for (int64_t v = from + warp; v < end; v += warps) {
    void* row = row_of<F32>(a.out, a.out_stride, v);
    for (int64_t c0 = 0; c0 < a.D; c0 += C::kBlock) C(c0, a.D, lane).store(row, zero);
  }
}

// The numbers of the lane's earlier lanes and of all lanes, added up.
__device__ __forceinline__ int before_lane(int x, int lane, int* all) {
  int upto = x;
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += y;
  }
  *all = __shfl_sync(~0u, upto, 31);
  return upto - x;
}

struct ClassShared {
  uint16_t count[32][kClassIds];  // tokens of a warp's stretch by id, then their places
  uint16_t first[kClassIds];      // of an id's tokens among the class's
  // and behind it the class's tokens in order: the rest of the id, the position
};

template <bool F32, int Width>
__global__ void __launch_bounds__(kClassThreads) class_sort_kernel(const Args a) {
  constexpr int kEach = int(kFewTokens / kClassThreads);  // most tokens of a thread
  static_assert(kClassIds <= kClassThreads, "a thread for each id of a class");
  extern __shared__ ClassShared sh[];
  auto& count = sh->count;
  auto& first = sh->first;
  uint32_t* const keys = reinterpret_cast<uint32_t*>(sh + 1);
  __shared__ int32_t own_of[32], less_of[32], none_of[32];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int classes = 1 << a.class_bits, mine = blockIdx.x;
  if (mine >= classes) {
    zero_rows<F32, Width, true>(a, a.zero_from, a.V, int64_t(mine - classes) * 32 + warp,
                                int64_t(gridDim.x - classes) * 32);
    return;
  }
  // Each warp's stretch of the tokens; an id that is not the class's becomes -1.
  const int T = int(a.T), stretch = (T + 1023) / 1024 * 32, begin = warp * stretch;
  int32_t id[kEach];
  int less = 0, none = 0, own = 0;
#pragma unroll
  for (int q0 = 0; q0 < kEach; q0 += 8) {
    if (q0 * 32 >= stretch) break;
    int64_t x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int o = (q0 + q) * 32 + lane, t = begin + o;
      x[q] = o < stretch && t < T ? a.ids[t] : -2;
      if (o >= stretch || t >= T) --none;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool valid = x[q] >= 0 && x[q] < a.V && x[q] != a.padding_id;
      const int its = int(x[q]) & (classes - 1);
      none += !valid;
      less += valid && its < mine;
      id[q0 + q] = valid && its == mine ? int32_t(x[q]) : -1;
      own += __popc(__ballot_sync(~0u, id[q0 + q] >= 0));
    }
  }
  for (int n = threadIdx.x; n < 32 * kClassIds / 2; n += kClassThreads) reinterpret_cast<uint32_t*>(count)[n] = 0;
  for (int o = 16; o; o >>= 1) {
    less += __shfl_xor_sync(~0u, less, o);
    none += __shfl_xor_sync(~0u, none, o);
  }
  if (lane == 0) {
    own_of[warp] = own;
    less_of[warp] = less;
    none_of[warp] = none;
  }
  __syncthreads();
  int n, place = before_lane(own_of[lane], lane, &n);
  before_lane(less_of[lane], lane, &less);
  before_lane(none_of[lane], lane, &none);
  place = __shfl_sync(~0u, place, warp);
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    if (q * 32 >= stretch) break;
    const unsigned in = __ballot_sync(~0u, id[q] >= 0);
    if (id[q] >= 0)
      keys[place + __popc(in & ((1u << lane) - 1))] =
          uint32_t(id[q] >> a.class_bits) << kPositionBits | uint32_t(begin + q * 32 + lane);
    place += __popc(in);
  }
  __syncthreads();
  // The class's tokens, again a stretch for each warp.
  const int each = (n + 1023) / 1024 * 32, from = warp * each, to = min(n, from + each);
  for (int i0 = from; i0 < to; i0 += 32) {
    const int rest = i0 + lane < to ? int(keys[i0 + lane] >> kPositionBits) : -1;
    const unsigned same = __match_any_sync(~0u, rest);
    if (rest >= 0 && lane == __ffs(same) - 1) count[warp][rest] += uint16_t(__popc(same));
    __syncwarp();
  }
  __syncthreads();
  int mine_of_id = 0;  // a thread for each id
#pragma unroll 8
  for (int w = 0; w < 32; ++w) {
    const int x = count[w][threadIdx.x];
    count[w][threadIdx.x] = uint16_t(mine_of_id);
    mine_of_id += x;
  }
  int all;
  const int before = before_lane(mine_of_id, lane, &all);
  if (lane == 0) own_of[warp] = all;
  __syncthreads();
  const int warps_before = before_lane(own_of[lane], lane, &all);
  first[threadIdx.x] = uint16_t(before + __shfl_sync(~0u, warps_before, warp));
  __syncthreads();
  for (int i0 = from; i0 < to; i0 += 32) {
    const bool in = i0 + lane < to;
    const uint32_t key = in ? keys[i0 + lane] : 0;
    const int rest = in ? int(key >> kPositionBits) : -1;
    const unsigned same = __match_any_sync(~0u, rest);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (in)
      a.list[0][less + first[rest] + count[warp][rest] + rank] =
          Entry{uint32_t(rest) << a.class_bits | uint32_t(mine), key & uint32_t(kFewTokens - 1)};
    __syncwarp();
    if (in && rank == 0) count[warp][rest] += uint16_t(__popc(same));
    __syncwarp();
  }
  if (mine == 0)
    for (int i = threadIdx.x; i < none; i += kClassThreads) a.list[0][T - none + i] = Entry{uint32_t(a.V), 0};
}

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

// The id as the sort's key: V for one that has no row, or no gradient.
__device__ __forceinline__ Entry token(const Args& a, int pass, int64_t i) {
  if (pass > 0) return a.list[(pass - 1) & 1][i];
  const int64_t id = a.ids[i];
  return Entry{id >= 0 && id < a.V && id != a.padding_id ? uint32_t(id) : uint32_t(a.V), uint32_t(i)};
}

// The first digit's counts; the other digits' begin as zero.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const Args a) {
  __shared__ int32_t count[kMostBins];
  let_next_start();
  const int bins = 1 << a.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.tile, end = min(a.T, begin + a.tile);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&count[token(a, 0, i).id & (bins - 1)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    for (int p = 0; p < a.passes; ++p)
      a.counts[(int64_t(p) * a.tiles + blockIdx.x) * bins + b] = p == 0 ? count[b] : 0;
  }
}

template <bool F32, int Width>
__global__ void __launch_bounds__(kSortThreads) place_kernel(const Args a, int pass) {
  constexpr int kHeld = 4;  // of a lane's tokens, read once (those of a tile of 2048)
  __shared__ int32_t place[kSortWarps][kMostBins], warp_sum[kSortWarps];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (int(blockIdx.x) >= a.tiles) {  // a pass's part of the zeros
    const int64_t part = (a.V - a.zero_from + a.passes - 1) / a.passes, from = a.zero_from + pass * part;
    zero_rows<F32, Width, false>(a, from, min(a.V, from + part), int64_t(blockIdx.x - a.tiles) * kSortWarps + warp,
                                 int64_t(gridDim.x - a.tiles) * kSortWarps);
    return;
  }
  const int bins = 1 << a.bits, shift = pass * a.bits;
  for (int n = threadIdx.x; n < kSortWarps * kMostBins; n += kSortThreads) place[n / kMostBins][n % kMostBins] = 0;
  // The warps' stretches of the tile, in order.
  const int64_t stretch = a.tile / kSortWarps;
  const int64_t begin = blockIdx.x * a.tile + warp * stretch, end = min(a.T, begin + stretch);
  if (pass > 0) wait_for_previous();  // (the ids are there before)
  Entry held[kHeld];
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    held[q] = begin + q * 32 + lane < end ? token(a, pass, begin + q * 32 + lane) : Entry{};
  if (pass == 0) wait_for_previous();
  // What comes before the tile: a thread for each digit.
  static_assert(kSortThreads >= kMostBins, "a thread for each digit");
  int32_t before = 0, all = 0;
  if (int(threadIdx.x) < bins) {
    const int32_t* const counts = a.counts + int64_t(pass) * a.tiles * bins + threadIdx.x;
#pragma unroll 32
    for (int j = 0; j < a.tiles; ++j) {
      const int32_t n = counts[int64_t(j) * bins];
      all += n;
      before += j < int(blockIdx.x) ? n : 0;
    }
  }
  int32_t upto = all;
  for (int o = 1; o < 32; o *= 2) {
    const int32_t x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int32_t base = before + upto - all;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  // Each stretch's tokens by digit, then the first place of each.
  const auto each = [&](auto f) {
#pragma unroll
    for (int q = 0; q < kHeld; ++q)
      if (begin + q * 32 < end) f(begin + q * 32 + lane < end, held[q]);
    for (int64_t i0 = begin + kHeld * 32; i0 < end; i0 += 32) {
      const bool in = i0 + lane < end;
      f(in, in ? token(a, pass, i0 + lane) : Entry{});
    }
  };
  each([&](bool in, Entry e) {
    if (in) atomicAdd(&place[warp][e.id >> shift & (bins - 1)], 1);
  });
  __syncthreads();
  if (int(threadIdx.x) < bins) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t n = place[w][threadIdx.x];
      place[w][threadIdx.x] = base;
      base += n;
    }
  }
  __syncthreads();
  Entry* const to = a.list[pass & 1];
  int32_t* const next = pass + 1 < a.passes ? a.counts + int64_t(pass + 1) * a.tiles * bins : nullptr;
  each([&](bool in, Entry e) {
    const int digit = in ? int(e.id >> shift & (bins - 1)) : -1;
    const unsigned same = __match_any_sync(~0u, digit);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (in) {
      const int64_t at = place[warp][digit] + rank;
      to[at] = e;
      // the next pass's counts: whole numbers, whose order does not matter
      if (next) atomicAdd(&next[at / a.tile * bins + (e.id >> (shift + a.bits) & (bins - 1))], 1);
    }
    __syncwarp();
    if (in && rank == 0) place[warp][digit] += __popc(same);
    __syncwarp();
  });
}

// ------------------------------------------------------------------- sums --

constexpr uint32_t kNone = 0xffffffffu;  // no key: above V

// A segment's sum to its row of dweight, rounded once. `Rests`: to its slot's.
template <bool F32, int Width, bool Rests>
__device__ __forceinline__ void finish(const Args& a, const Columns<F32, Width>& c, uint32_t id,
                                       const float (&sum)[Columns<F32, Width>::kVec]) {
  using C = Columns<F32, Width>;
  if (c.count == 0) return;
  const int64_t to = Rests ? slot_of(a.slots[id / 32], id % 32) : int64_t(id);
  if (Rests && to < 0) return;
  void* row = row_of<F32>(a.out, a.out_stride, to);
  float x[C::kVec];
  if (a.accumulate) {
    C::unpack(c.load(row), x);
#pragma unroll
    for (int j = 0; j < C::kVec; ++j) x[j] = fmaf(a.scale, sum[j], x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < C::kVec; ++j) x[j] = a.scale * sum[j];
  }
  c.store(row, C::pack(x));
}

// A run's share of a segment: kVec floats of each lane side by side, whatever
// columns they are.
template <int kVec>
__device__ __forceinline__ float4* share(const Args& a, int64_t run, int which, int64_t block, int lane) {
  return reinterpret_cast<float4*>(a.part + (2 * run + which) * a.Dp + block * 32 * kVec + lane * kVec);
}
template <int kVec>
__device__ __forceinline__ void add_share(const float4* from, float (&sum)[kVec]) {
#pragma unroll
  for (int q = 0; q < kVec / 4; ++q) {
    const float4 x = from[q];
    sum[4 * q] += x.x;
    sum[4 * q + 1] += x.y;
    sum[4 * q + 2] += x.z;
    sum[4 * q + 3] += x.w;
  }
}
template <int kVec>
__device__ __forceinline__ void put_share(float4* to, const float (&sum)[kVec]) {
#pragma unroll
  for (int q = 0; q < kVec / 4; ++q) to[q] = make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
}

// Rows of dweight that no token has, below zero_from: zeros. A warp for 32 ids, each
// lane looks its own up in the list (in order of id).
template <bool F32, int Width>
__device__ __forceinline__ void zero_absent_rows(const Args& a, int64_t v0) {
  using C = Columns<F32, Width>;
  const int lane = threadIdx.x & 31;
  const int64_t v = v0 + lane;
  int64_t lo = 0, hi = a.T;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (a.sorted[mid].id < v) lo = mid + 1;
    else hi = mid;
  }
  const bool absent = v < a.zero_from && !(lo < a.T && a.sorted[lo].id == v);
  for (unsigned left = __ballot_sync(~0u, absent); left; left &= left - 1) {
    void* row = row_of<F32>(a.out, a.out_stride, v0 + __ffs(left) - 1);
    for (int64_t c0 = 0; c0 < a.D; c0 += C::kBlock) C(c0, a.D, lane).store(row, make_uint4(0, 0, 0, 0));
  }
}

// A warp for 32 ids whose rows may have to become zero -- the long pieces of work
// first -- and one for each run and block of columns, with eight rows on their way at
// a time, as they are stored: 80 registers, three blocks an SM. `Rests`: each row
// counts a number of times that is the token's own, and rows that count none are not
// read.
template <bool F32, int Width, bool Rests = false>
__global__ void __launch_bounds__(256, 3) sum_kernel(const Args a, int64_t zero_warps) {
  using C = Columns<F32, Width>;
  constexpr int kVec = C::kVec, kAhead = 8;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const Entry* const list = a.sorted;
  const int64_t step = int64_t(gridDim.x) * 8, sums = a.runs * a.blocks;
  for (int64_t g = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5) - zero_warps; g < sums; g += step) {
    if (g < 0) {
      zero_absent_rows<F32, Width>(a, (g + zero_warps) * 32);
      continue;
    }
    const int64_t run = g / a.blocks, first = run * a.run, block = g % a.blocks;
    const C c(block * C::kBlock, a.D, lane);
    const int count = int(min(int64_t(a.run), a.T - first));
    const uint32_t prev = first > 0 ? list[first - 1].id : kNone;
    float sum[kVec] = {};
    bool begun = true;  // the segment begins in this run
    for (int s0 = 0; s0 < count; s0 += 32) {  // 32 entries at a time, one a lane
      const int held = min(32, count - s0);
      const Entry e = lane < held ? list[first + s0 + lane] : Entry{kNone, 0};
      const uint32_t next = first + s0 + held < a.T ? list[first + s0 + held].id : kNone;
      const int n = __popc(__ballot_sync(~0u, e.id < a.V));  // those without a row come last
      const float rest = Rests && lane < n ? rest_of(a.scales[e.t], a.weights[e.t]) : 0.0f;
      if (s0 == 0) begun = __shfl_sync(~0u, e.id, 0) != prev;
      for (int i0 = 0; i0 < n; i0 += kAhead) {
        uint4 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t t = __shfl_sync(~0u, e.t, (i0 + i) & 31);
          const bool counts = !Rests || __shfl_sync(~0u, rest, (i0 + i) & 31) != 0.0f;  // (also a NaN)
          if (i0 + i < n && counts) w[i] = c.template load<true>(row_of<F32>(a.table, a.table_stride, t));
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint32_t id = __shfl_sync(~0u, e.id, (i0 + i) & 31);
          const uint32_t following = __shfl_sync(~0u, e.id, (i0 + i + 1) & 31);
          if (i0 + i >= n) break;
          const float times = Rests ? __shfl_sync(~0u, rest, (i0 + i) & 31) : 1.0f;
          if (times != 0.0f) {
            float x[kVec];
            C::unpack(w[i], x);
#pragma unroll
            for (int j = 0; j < kVec; ++j) sum[j] = Rests ? fmaf(times, x[j], sum[j]) : sum[j] + x[j];
          }
          const bool ends = (i0 + i + 1 == held ? next : following) != id;
          const bool last = s0 + i0 + i + 1 == count;
          if (ends && begun) finish<F32, Width, Rests>(a, c, id, sum);
          else if (ends || last) put_share(share<kVec>(a, run, begun ? 1 : 0, block, lane), sum);
          if (ends) {
            begun = true;
#pragma unroll
            for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
          }
        }
      }
      if (n < held) break;
    }
  }
}

// The segments that a run began and did not end: the runs' shares in order. A
// warp looks for one in a run and block of columns and adds up to kShort shares
// itself; longer ones are added by the block's eight warps together, each a
// stretch of the shares in order, and the stretches in order. (A block has
// neighbouring runs, of which few begin a long segment, not the columns of one:
// 131072 tokens of width 4096 15 us instead of 97.)
template <bool F32, int Width, bool Rests = false>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  using C = Columns<F32, Width>;
  constexpr int kVec = C::kVec, kShort = 8;
  __shared__ int64_t long_run[8], long_block[8], long_end[8];
  __shared__ float4 parts[8][32 * kVec / 4];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Entry* const list = a.sorted;
  const int64_t all = (a.runs - 1) * a.blocks;
  for (int64_t g0 = int64_t(blockIdx.x) * 8; g0 < all; g0 += int64_t(gridDim.x) * 8) {
    const int64_t g = g0 + warp;
    const int64_t run = g % (a.runs - 1), block = g / (a.runs - 1), next = (run + 1) * a.run;
    bool joins = false;
    uint32_t id = 0;
    if (g < all) {
      id = list[next].id;
      joins = id < a.V && list[next - 1].id == id && !(run > 0 && list[next - a.run - 1].id == id);
    }
    int64_t end = run + 1;  // behind the last run with a share
    if (joins) {
      // The runs that begin with the segment, first by 32s, then one by one.
      for (;;) {
        const int64_t r = end + lane * 32 + 31;
        const unsigned in = __ballot_sync(~0u, r < a.runs && list[r * a.run].id == id);
        const int n = in == ~0u ? 32 : __ffs(~in) - 1;
        end += 32 * n;
        if (n < 32) break;
      }
      const int64_t r = end + lane;
      const unsigned in = __ballot_sync(~0u, r < a.runs && list[r * a.run].id == id);
      end += in == ~0u ? 32 : __ffs(~in) - 1;
    }
    const bool together = joins && end - run > kShort;
    if (joins && !together) {
      float sum[kVec] = {};
      add_share<kVec>(share<kVec>(a, run, 1, block, lane), sum);
#pragma unroll 4
      for (int64_t r = run + 1; r < end; ++r) add_share<kVec>(share<kVec>(a, r, 0, block, lane), sum);
      finish<F32, Width, Rests>(a, C(block * C::kBlock, a.D, lane), id, sum);
    }
    if (lane == 0) {
      long_run[warp] = together ? run : -1;
      long_block[warp] = block;
      long_end[warp] = end;
    }
    if (!__syncthreads_or(together)) continue;
    for (int q = 0; q < 8; ++q) {
      const int64_t r0 = long_run[q], r1 = long_end[q], b = long_block[q];
      if (r0 < 0) continue;
      const int64_t each = (r1 - r0 + 7) / 8;
      float sum[kVec] = {};
      const int64_t from = r0 + warp * each, to = min(r1, from + each);
#pragma unroll 8
      for (int64_t r = from; r < to; ++r) add_share<kVec>(share<kVec>(a, r, r == r0 ? 1 : 0, b, lane), sum);
      put_share<kVec>(&parts[warp][lane * kVec / 4], sum);
      __syncthreads();
      if (warp == q) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) add_share<kVec>(&parts[w][lane * kVec / 4], sum);
        finish<F32, Width, Rests>(a, C(b * C::kBlock, a.D, lane), id, sum);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

// Blocks of eight warps for `warps` of them.
unsigned blocks_of(int64_t warps) {
  const int64_t blocks = (warps + 7) / 8;
  return unsigned(blocks < 1 ? 1 : blocks > (1 << 30) ? 1 << 30 : blocks);
}

template <bool F32, int Width>
cudaError_t sort(const Args& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.few) {
    // Zeros: a block of them for each SM at most.
    const int64_t rows = (a.V - a.zero_from + 31) / 32;
    const unsigned blocks = unsigned((1 << a.class_bits) + (rows < kSms ? rows : kSms));
    const auto shared = [](int64_t tokens) { return sizeof(ClassShared) + size_t(tokens) * sizeof(uint32_t); };
    // Once per device (a race only does it twice): the kernel's shared memory.
    static std::atomic<bool> ready[64];
    int device = 0;
    e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device >= 64 || !ready[device].load(std::memory_order_acquire))) {
      e = cudaFuncSetAttribute(class_sort_kernel<F32, Width>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(shared(kFewTokens)));
      if (e == cudaSuccess && device < 64) ready[device].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    return launch(class_sort_kernel<F32, Width>, blocks, kClassThreads, shared(a.T), s, false, a);
  }
  const int64_t part = (a.V - a.zero_from + a.passes - 1) / a.passes;
  const int64_t zero_blocks = part / kSortWarps < 2 * kSms ? (part + kSortWarps - 1) / kSortWarps : 2 * kSms;
  e = launch(count_kernel, unsigned(a.tiles), kSortThreads, 0, s, false, a);
  for (int p = 0; e == cudaSuccess && p < a.passes; ++p)
    e = launch(place_kernel<F32, Width>, unsigned(a.tiles + zero_blocks), kSortThreads, 0, s, true, a, p);
  return e;
}

template <bool F32, int Width, bool Rests = false>
cudaError_t sums(const Args& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int64_t zero_warps = a.accumulate || Rests ? 0 : (a.zero_from + 31) / 32;
  cudaError_t e = launch(sum_kernel<F32, Width, Rests>, blocks_of(a.runs * a.blocks + zero_warps), 256, 0, s, true, a,
                         zero_warps);
  if (e == cudaSuccess && a.runs > 1)
    e = launch(join_kernel<F32, Width, Rests>, blocks_of((a.runs - 1) * a.blocks), 256, 0, s, true, a);
  return e;
}

}  // namespace

cudaError_t launch_lookup(const Args& a, cudaStream_t s) {
  const bool stream = a.T * a.D * (a.f32 ? 4 : 2) > kCacheBytes;
  const auto run = [&](auto* kernel) { return launch(kernel, blocks_of(a.T), 256, 0, s, false, a); };
  if (a.f32) {
    if (a.width == 16) return stream ? run(lookup_kernel<true, 16, true>) : run(lookup_kernel<true, 16, false>);
    return run(lookup_kernel<true, 4, false>);
  }
  if (a.width == 16) return stream ? run(lookup_kernel<false, 16, true>) : run(lookup_kernel<false, 16, false>);
  return a.width == 4 ? run(lookup_kernel<false, 4, false>) : run(lookup_kernel<false, 2, false>);
}

cudaError_t launch_sort(const Args& a, cudaStream_t s) {
  if (a.f32) return a.width == 16 ? sort<true, 16>(a, s) : sort<true, 4>(a, s);
  return a.width == 16 ? sort<false, 16>(a, s) : a.width == 4 ? sort<false, 4>(a, s) : sort<false, 2>(a, s);
}

cudaError_t launch_sums(const Args& a, cudaStream_t s) {
  if (a.f32) return a.width == 16 ? sums<true, 16>(a, s) : sums<true, 4>(a, s);
  return a.width == 16 ? sums<false, 16>(a, s) : a.width == 4 ? sums<false, 4>(a, s) : sums<false, 2>(a, s);
}

// (Of bf16 rows; fp32's are never cut down to bf16.)
cudaError_t launch_rests(const Args& a, cudaStream_t s) {
  return a.width == 16 ? sums<false, 16, true>(a, s) : a.width == 4 ? sums<false, 4, true>(a, s) : sums<false, 2, true>(a, s);
}

}  // namespace ze
