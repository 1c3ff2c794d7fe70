// Kernels of the embedding (zero_embedding_*).
//
// The lookup copies rows by id, one warp a row.
//
// The gradient adds the rows of dout that have the same id. The tokens are
// sorted by id, stably, so that an id's rows are a segment of the list, in the
// order of the tokens; the list is cut into runs of equal length, one warp a run
// and block of columns, whatever the segments' lengths: a segment within a run
// goes to its row of dweight, and the shares of one that spans runs are kept in
// fp32 and joined in the order of the runs. No atomics touch a value, so equal
// inputs give equal bits.

#include <cuda_bf16.h>

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

// A lane's share of a block of columns of a row: kVec elements side by side where
// 16-byte accesses fit, else every 32nd one.
template <bool F32, bool Vector>
struct Columns {
  using E = typename Type<F32>::E;
  static constexpr int kVec = Type<F32>::kVec;
  static constexpr int kBlock = 32 * kVec;

  int64_t first;  // of the lane
  int count;      // that lie inside the row

  __device__ __forceinline__ Columns(int64_t c0, int64_t D, int lane) {
    if (Vector) {
      first = c0 + lane * kVec;
      count = int(max(int64_t(0), min(int64_t(kVec), D - first)));
    } else {
      first = c0 + lane;
      count = int(max(int64_t(0), min(int64_t(kVec), (D - first + 31) / 32)));
    }
  }
  __device__ __forceinline__ int64_t at(int j) const { return first + (Vector ? j : 32 * j); }

  __device__ __forceinline__ void load(const void* row, float (&x)[kVec]) const {
    const E* p = static_cast<const E*>(row);
    if (Vector && count == kVec) {
      const uint4 w = *reinterpret_cast<const uint4*>(p + first);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        x[j] = F32 ? __uint_as_float(words[j])
                   : __uint_as_float(j % 2 ? words[j / 2] & 0xffff0000u : words[j / 2] << 16);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) x[j] = j < count ? float(p[at(j)]) : 0.0f;
    }
  }
  __device__ __forceinline__ void store(void* row, const float (&x)[kVec]) const {
    E* p = static_cast<E*>(row);
    if (Vector && count == kVec) {
      uint4 w;
      if (F32) {
        w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      } else {
        uint32_t words[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j % kVec], x[(2 * j + 1) % kVec]);
          words[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        w = make_uint4(words[0], words[1], words[2], words[3]);
      }
      *reinterpret_cast<uint4*>(p + first) = w;
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < count) p[at(j)] = E(x[j]);
    }
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

template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) lookup_kernel(const Args a) {
  using C = Columns<F32, Vector>;
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * 8;
  for (int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); t < a.T; t += step) {
    const int64_t id = a.ids[t];
    const bool there = id >= 0 && id < a.V;
    const void* from = row_of<F32>(a.table, a.table_stride, there ? id : 0);
    void* to = row_of<F32>(a.out, a.out_stride, t);
#pragma unroll 4
    for (int64_t c0 = 0; c0 < a.D; c0 += C::kBlock) {
      const C c(c0, a.D, lane);
      float x[C::kVec] = {};
      if (there) c.load(from, x);
#pragma unroll
      for (int j = 0; j < C::kVec; ++j) x[j] = there ? x[j] * a.scale : 0.0f;
      c.store(to, x);
    }
  }
}

// ------------------------------------------------------------------- sort --
//
// By digits from the lowest, each pass stable: a tile's tokens are counted by
// digit, and the next kernel's block of that tile adds up what comes before --
// smaller digits of all tiles, its digit in earlier tiles -- and places its
// tokens, each warp a stretch of them in order.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

// The id as the sort's key: V for one that has no row, or no gradient.
__device__ __forceinline__ Entry token(const Args& a, int pass, int64_t i) {
  if (pass > 0) return a.list[(pass - 1) & 1][i];
  const int64_t id = a.ids[i];
  return Entry{id >= 0 && id < a.V && id != a.padding_id ? uint32_t(id) : uint32_t(a.V), uint32_t(i)};
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const Args a, int pass) {
  __shared__ int32_t count[kMostBins];
  let_next_start();
  wait_for_previous();
  const int bins = 1 << a.bits, shift = pass * a.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.tile, end = min(a.T, begin + a.tile);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&count[token(a, pass, i).id >> shift & (bins - 1)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) a.counts[int64_t(blockIdx.x) * bins + b] = count[b];
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const Args a, int pass) {
  __shared__ int32_t place[kSortWarps][kMostBins], warp_sum[kSortWarps];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bins = 1 << a.bits, shift = pass * a.bits;
  for (int n = threadIdx.x; n < kSortWarps * kMostBins; n += kSortThreads) place[n / kMostBins][n % kMostBins] = 0;
  wait_for_previous();
  // A thread for each digit.
  static_assert(kSortThreads >= kMostBins, "a thread for each digit");
  int32_t before = 0, all = 0;
  if (int(threadIdx.x) < bins) {
#pragma unroll 8
    for (int j = 0; j < a.tiles; ++j) {
      const int32_t n = a.counts[int64_t(j) * bins + threadIdx.x];
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
  // The warps' stretches: their tokens by digit, then the first place of each.
  const int64_t stretch = a.tile / kSortWarps;
  const int64_t begin = blockIdx.x * a.tile + warp * stretch, end = min(a.T, begin + stretch);
  for (int64_t i = begin + lane; i < end; i += 32)
    atomicAdd(&place[warp][token(a, pass, i).id >> shift & (bins - 1)], 1);
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
  for (int64_t i0 = begin; i0 < end; i0 += 32) {
    const bool in = i0 + lane < end;
    const Entry e = in ? token(a, pass, i0 + lane) : Entry{};
    const int digit = in ? int(e.id >> shift & (bins - 1)) : -1;
    const unsigned same = __match_any_sync(~0u, digit);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (in) to[place[warp][digit] + rank] = e;
    __syncwarp();
    if (in && rank == 0) place[warp][digit] += __popc(same);
    __syncwarp();
  }
}

// ------------------------------------------------------------------- sums --

constexpr uint32_t kNone = 0xffffffffu;  // no key: above V

// A segment's sum to its row of dweight, rounded once.
template <bool F32, bool Vector>
__device__ __forceinline__ void finish(const Args& a, const Columns<F32, Vector>& c, uint32_t id,
                                       const float (&sum)[Columns<F32, Vector>::kVec]) {
  constexpr int kVec = Columns<F32, Vector>::kVec;
  void* row = row_of<F32>(a.out, a.out_stride, id);
  float x[kVec];
  if (a.accumulate) {
    c.load(row, x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = fmaf(a.scale, sum[j], x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = a.scale * sum[j];
  }
  c.store(row, x);
}

template <bool F32, bool Vector>
__device__ __forceinline__ float* share(const Args& a, int64_t run, int which, const Columns<F32, Vector>& c) {
  return a.part + (2 * run + which) * a.Dp + c.first;
}

template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) sum_kernel(const Args a) {
  using C = Columns<F32, Vector>;
  constexpr int kVec = C::kVec, kAhead = 8;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const Entry* const list = a.list[(a.passes - 1) & 1];
  const int64_t step = int64_t(gridDim.x) * 8;
  for (int64_t g = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); g < a.runs * a.blocks; g += step) {
    const int64_t run = g / a.blocks, first = run * a.run;
    const C c(g % a.blocks * C::kBlock, a.D, lane);
    const int count = int(min(int64_t(a.run), a.T - first));
    const Entry e = lane < count ? list[first + lane] : Entry{kNone, 0};
    const uint32_t prev = first > 0 ? list[first - 1].id : kNone;
    const uint32_t next = first + count < a.T ? list[first + count].id : kNone;
    const int n = __popc(__ballot_sync(~0u, e.id < a.V));  // those without a row come last
    bool begun = __shfl_sync(~0u, e.id, 0) != prev;  // the segment begins in this run
    float sum[kVec] = {};
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      float x[kAhead][kVec];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t t = __shfl_sync(~0u, e.t, (i0 + i) & 31);
        if (i0 + i < n) c.load(row_of<F32>(a.table, a.table_stride, t), x[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t id = __shfl_sync(~0u, e.id, (i0 + i) & 31);
        const uint32_t following = __shfl_sync(~0u, e.id, (i0 + i + 1) & 31);
        if (i0 + i >= n) break;
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] += x[i][j];
        const bool last = i0 + i + 1 == count;
        const bool ends = (last ? next : following) != id;
        if (ends && begun) {
          finish(a, c, id, sum);
        } else if (ends || last) {
          float* to = share(a, run, begun ? 1 : 0, c);
#pragma unroll
          for (int j = 0; j < kVec; ++j) to[Vector ? j : 32 * j] = sum[j];
        }
        if (ends) {
          begun = true;
#pragma unroll
          for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
        }
      }
    }
  }
}

// The segments that a run began and did not end: the runs' shares in order.
template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  using C = Columns<F32, Vector>;
  constexpr int kVec = C::kVec;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const Entry* const list = a.list[(a.passes - 1) & 1];
  const int64_t step = int64_t(gridDim.x) * 8;
  for (int64_t g = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); g < (a.runs - 1) * a.blocks; g += step) {
    const int64_t run = g / a.blocks, next = (run + 1) * a.run;
    const uint32_t id = list[next].id;
    if (id >= a.V || list[next - 1].id != id) continue;
    if (run > 0 && list[next - a.run - 1].id == id) continue;  // an earlier run began it
    const C c(g % a.blocks * C::kBlock, a.D, lane);
    float sum[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum[j] = share(a, run, 1, c)[Vector ? j : 32 * j];
    for (int64_t r = run + 1; r < a.runs;) {
      // The runs from r on that begin with the segment, up to 32 of them.
      const unsigned in = __ballot_sync(~0u, r + lane < a.runs && list[min(r + lane, a.runs - 1) * a.run].id == id);
      const int n = __ffs(~in) ? __ffs(~in) - 1 : 32;
#pragma unroll 4
      for (int q = 0; q < n; ++q)
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] += share(a, r + q, 0, c)[Vector ? j : 32 * j];
      r += n;
      if (n < 32) break;
    }
    finish(a, c, id, sum);
  }
}

// Rows of dweight that no token has: zeros. A warp for 32 ids, each lane looks
// its own up in the list.
template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) absent_kernel(const Args a) {
  using C = Columns<F32, Vector>;
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const Entry* const list = a.list[(a.passes - 1) & 1];
  const int64_t step = int64_t(gridDim.x) * 8 * 32;
  for (int64_t v0 = (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 32; v0 < a.V; v0 += step) {
    const int64_t v = v0 + lane;
    int64_t lo = 0, hi = a.T;
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (list[mid].id < v) lo = mid + 1;
      else hi = mid;
    }
    const bool absent = v < a.V && !(lo < a.T && list[lo].id == v);
    for (unsigned left = __ballot_sync(~0u, absent); left; left &= left - 1) {
      void* row = row_of<F32>(a.out, a.out_stride, v0 + __ffs(left) - 1);
      const float zero[C::kVec] = {};
      for (int64_t c0 = 0; c0 < a.D; c0 += C::kBlock) C(c0, a.D, lane).store(row, zero);
    }
  }
}

// Blocks of eight warps for `warps` of them.
unsigned blocks_of(int64_t warps) {
  const int64_t blocks = (warps + 7) / 8;
  return unsigned(blocks < 1 ? 1 : blocks > (1 << 30) ? 1 << 30 : blocks);
}

template <bool F32, bool Vector>
cudaError_t sums(const Args& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  bool behind = a.T > 0;  // the sort
  if (!a.accumulate) {
    e = launch(absent_kernel<F32, Vector>, blocks_of((a.V + 31) / 32), 256, 0, s, behind, a);
    behind = true;
  }
  if (e == cudaSuccess && a.T > 0)
    e = launch(sum_kernel<F32, Vector>, blocks_of(a.runs * a.blocks), 256, 0, s, behind, a);
  if (e == cudaSuccess && a.runs > 1)
    e = launch(join_kernel<F32, Vector>, blocks_of((a.runs - 1) * a.blocks), 256, 0, s, true, a);
  return e;
}

}  // namespace

cudaError_t launch_lookup(const Args& a, cudaStream_t s) {
  const unsigned blocks = blocks_of(a.T);
  if (a.f32) return launch(a.vector ? lookup_kernel<true, true> : lookup_kernel<true, false>, blocks, 256, 0, s, false, a);
  return launch(a.vector ? lookup_kernel<false, true> : lookup_kernel<false, false>, blocks, 256, 0, s, false, a);
}

cudaError_t launch_sort(const Args& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  for (int p = 0; e == cudaSuccess && p < a.passes; ++p) {
    e = launch(count_kernel, unsigned(a.tiles), kSortThreads, 0, s, p > 0, a, p);
    if (e == cudaSuccess) e = launch(place_kernel, unsigned(a.tiles), kSortThreads, 0, s, true, a, p);
  }
  return e;
}

cudaError_t launch_sums(const Args& a, cudaStream_t s) {
  if (a.f32) return a.vector ? sums<true, true>(a, s) : sums<true, false>(a, s);
  return a.vector ? sums<false, true>(a, s) : sums<false, false>(a, s);
}

}  // namespace ze
