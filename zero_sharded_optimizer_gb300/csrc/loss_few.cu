// The products of a policy or a preference loss of few rows.
//
// The tensor cores' tiles are 256 rows high, whatever there is of them, their kernel
// forms the logits twice, and fp32 takes six passes over a weight split in a kernel of
// its own. Few rows' logits are small, and what is left is traffic: the weight read
// for the logits and for dhidden, dweight written. So the logits are kept here, sums
// are fp32 multiply-adds on the plain cores, and nothing is packed, split into parts
// or waited for.
//   logits     z = h W^T, eight hidden states at a time in shared memory: a warp
//              takes four rows of the weight, its lanes along them, the next four
//              on their way. Blocks go on until the vocabulary is done, each with
//              one maximum and sum of exponentials for a row in the end.
//   gradients  G from z, lse and the rows' scales where it is needed, 32 values a
//              warp, which its lanes hand round: dW = f G^T h in tiles of 64 rows,
//              dH = G W in parts of the vocabulary, which dhidden_out adds up, both
//              in one launch
// Every sum has a fixed order. Which calls come here, and what that gains:
// loss_host.cpp.

#include <math.h>

#include <atomic>
#include <type_traits>

#include "loss_device.cuh"

namespace zl {
namespace {

constexpr int kGroup = kFewGroup;  // rows of the batch that are worked on together

template <bool F32>
using Element = typename std::conditional<F32, float, __nv_bfloat16>::type;
template <bool F32>
constexpr int kWide = F32 ? 4 : 8;  // elements of 16 bytes

template <bool F32>
__device__ __forceinline__ void unpack(uint4 w, float (&x)[kWide<F32>]) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < kWide<F32>; ++j)
    x[j] = __uint_as_float(F32 ? words[j % 4] : j % 2 ? words[j / 2] & 0xffff0000u : words[j / 2] << 16);
}

// 16 bytes of a row from element k on as they are stored, zeros behind its end.
// `vector`: rows begin on 16 bytes.
template <bool F32>
__device__ __forceinline__ uint4 load(const Element<F32>* row, int64_t k, int64_t D, bool vector) {
  if (vector && k + kWide<F32> <= D) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t words[4] = {};
#pragma unroll
  for (int j = 0; j < kWide<F32>; ++j) {
    if (k + j >= D) continue;
    if (F32) words[j % 4] = reinterpret_cast<const uint32_t*>(row)[k + j];
    else words[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[k + j]) << (j % 2 * 16);
  }
  return make_uint4(words[0], words[1], words[2], words[3]);
}

// Rows of the weight on their way: each lane copies the 16 bytes of four rows that it
// will read itself into a ring in shared memory, kAhead steps before, so nothing but
// its own copies has to be waited for.
constexpr int kAhead = 3;
struct Ring {
  uint4* mine;  // of the lane: [kAhead][4], 32 apart
  int at = 0;
  __device__ __forceinline__ explicit Ring(uint4* shared, int warp, int lane) : mine(shared + warp * kAhead * 4 * 32 + lane) {}
  // Row q's 16 bytes; `from` NULL: zeros.
  template <bool F32>
  __device__ __forceinline__ void copy(int q, const Element<F32>* row, int64_t k, int64_t D, bool vector) {
    uint4* const to = mine + (at * 4 + q) * 32;
    if (vector && k + kWide<F32> <= D)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(row + k)
                   : "memory");
    else
      *to = load<F32>(row, k, D, vector);
  }
  // After a step's copies; then the ring is at the step copied longest ago.
  __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    at = at + 1 == kAhead ? 0 : at + 1;
  }
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
  __device__ __forceinline__ uint4 operator[](int q) const { return mine[(at * 4 + q) * 32]; }
};
constexpr int kRingBytes = 8 * kAhead * 4 * 32 * 16;

// Adds each of 32 values over the warp's lanes: lane l is left with the l-th sum.
// Each step adds up half of the values with the lane that keeps the other half.
template <int N, int All>
__device__ __forceinline__ void halve(float (&x)[All], int lane) {
  const bool upper = lane & N;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float sent = upper ? x[j] : x[j + N], kept = upper ? x[j + N] : x[j];
    x[j] = kept + __shfl_xor_sync(~0u, sent, N);
  }
}
__device__ __forceinline__ float add_lanes(float (&x)[32], int lane) {
  halve<16>(x, lane);
  halve<8>(x, lane);
  halve<4>(x, lane);
  halve<2>(x, lane);
  halve<1>(x, lane);
  return x[0];
}

// Logits lie as [group][v][row of the group], the order in which a warp forms them.
__device__ __forceinline__ int64_t logit_at(const Args& a, int group, int64_t v, int i) {
  return (int64_t(group) * a.V + v) * kGroup + i;
}

// e^d for d <= 0.
__device__ __forceinline__ float exp_even(float d) { return exp2_even(fmaf(d, kLog2e, d * kLog2eRest)); }

// A running maximum and sum of exponentials. (Of differences of logits: a logit times
// log2(e), taken from a rounded maximum of such, would leave its rounding in the
// exponent, which for logits beyond 1e9 goes past fp32's range.)
struct Sum {
  float m = -INFINITY, s = 0.0f;
  __device__ __forceinline__ void join(float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = top == -INFINITY ? s + s2 : s * exp_even(m - top) + s2 * exp_even(m2 - top);
    m = top;
  }
};

template <bool F32>
__global__ void __launch_bounds__(256, 2) few_logits_kernel(const Args a, int width, bool hidden_vector,
                                                            bool weight_vector) {
  using E = Element<F32>;
  constexpr int W = kWide<F32>, kStep = 32 * W;  // elements that a warp takes of a row at a time
  extern __shared__ __align__(16) uint4 shared[];  // the ring, and [kGroup][width / W]
  uint4* const hidden = shared + kRingBytes / 16;
  __shared__ float2 sums[8][kGroup];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = blockIdx.y;
  const int rows = min(kGroup, a.head->rows - group * kGroup);
  if (rows <= 0) return;
  const int64_t blocks = (a.V + 31) / 32;  // of the vocabulary: four rows a warp
  const int wide = width / W;
  Ring ring(shared, warp, lane);
  int64_t next_block = blockIdx.x;  // what is copied next
  int next_k = 0;
  const auto fetch = [&] {
    if (next_block < blocks) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t v = min(next_block * 32 + warp * 4 + q, a.V - 1);
        ring.copy<F32>(q, static_cast<const E*>(a.weight) + v * a.weight_stride, next_k + lane * W, a.D, weight_vector);
      }
    }
    next_k += kStep;
    if (next_k >= width) {
      next_k = 0;
      next_block += gridDim.x;
    }
    ring.commit();
  };
#pragma unroll
  for (int n = 0; n < kAhead; ++n) fetch();  // the first, beside the hidden states
  for (int n = threadIdx.x; n < kGroup * wide; n += 256) {
    const int i = n / wide;
    hidden[n] = i < rows ? load<F32>(static_cast<const E*>(a.hidden) + a.rowmap[group * kGroup + i] * a.hidden_stride,
                                     n % wide * W, a.D, hidden_vector)
                         : make_uint4(0, 0, 0, 0);
  }
  const int i = lane % kGroup;
  const int64_t t = i < rows ? a.rowmap[group * kGroup + i] : -1;
  const int32_t y = t >= 0 ? a.ids[t] : -1;
  __syncthreads();
  Sum sum;
  float dot[32] = {};  // [four rows of the weight][kGroup]
  int k = 0;
  for (int64_t block = blockIdx.x; block < blocks;) {
    ring.wait();
    float x[4][W];
#pragma unroll
    for (int q = 0; q < 4; ++q) unpack<F32>(ring[q], x[q]);
    fetch();
    const int at = k / W + lane;
    const int64_t v = block * 32 + warp * 4 + lane / kGroup;
    k += kStep;
    const bool done = k >= width;
    if (done) {
      k = 0;
      block += gridDim.x;
    }
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      if (r >= rows) break;  // (the same in all lanes)
      float h[W];
      unpack<F32>(hidden[r * wide + at], h);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < W; ++j) dot[q * kGroup + r] = fmaf(h[j], x[q][j], dot[q * kGroup + r]);
    }
    if (!done) continue;
    const float z = add_lanes(dot, lane);
#pragma unroll
    for (int j = 0; j < 32; ++j) dot[j] = 0.0f;
    if (v < a.V && t >= 0) {
      a.z[logit_at(a, group, v, i)] = z;
      if (y != v) sum.join(z, 1.0f);  // the statistics are those of the other columns
    }
  }
  if (!a.forward) return;
  // The lanes of a row, then the warps, in order.
  for (int o = kGroup; o < 32; o *= 2) {
    const float m = __shfl_xor_sync(~0u, sum.m, o), s = __shfl_xor_sync(~0u, sum.s, o);
    sum.join(m, s);
  }
  if (lane < kGroup) sums[warp][lane] = make_float2(sum.m, sum.s);
  __syncthreads();
  if (int(threadIdx.x) < rows) {
    Sum all;
    for (int q = 0; q < 8; ++q) all.join(sums[q][threadIdx.x].x, sums[q][threadIdx.x].y);
    a.stats[int64_t(blockIdx.x) * a.Tp + group * kGroup + threadIdx.x] =
        make_float2(isnan(all.s) ? NAN : all.m, all.s);
  }
}

constexpr int kTileV = 64;  // rows of dweight's tiles

// What a lane needs of its row (of a group of eight) for G.
struct FewRow {
  int64_t t = -1;
  float scale = 0.0f, lse = 0.0f, gap = 0.0f;  // gap: p - 1 of the label
  int32_t y = -1;
  __device__ __forceinline__ FewRow(const Args& a, int i, int rows) {
    if (i >= rows) return;
    t = a.rowmap[i];
    scale = a.scales[t];
    lse = a.lse[t];
    gap = a.weights[t];
    y = a.ids[t];
  }
  // G of the row at column v with logit z, without the common factor; a row without a
  // slope has none, whatever its logits.
  __device__ __forceinline__ float gradient(float z, int64_t v) const {
    return scale == 0.0f ? 0.0f : scale * (y == v ? gap : expf(z - lse));
  }
};

// Tiles of dweight, every `step`-th from `tile` on: eight rows a warp, 16 bytes of each
// a lane. Up to eight rows of the batch stay where they are from tile to tile.
template <bool F32, int R>
__device__ __forceinline__ void weight_tiles(const Args& a, int64_t tile, int64_t step, int64_t d0, int rows,
                                             bool hidden_vector, bool dweight_vector) {
  using E = Element<F32>;
  constexpr int W = kWide<F32>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t d = d0 + lane * W;
  const float f = a.head->factor;
  FewRow row(a, 0, 0);
  uint4 w[R];
  unsigned sloped = 0;
  int held = -1;  // the group that row and w are of
  for (; tile * kTileV < a.V; tile += step) {
    const int64_t vs = tile * kTileV + warp * 8;
    if (vs >= a.V) break;
    float sum[8][W] = {};
    for (int group = 0; group * kGroup < rows; ++group) {
      if (held != group) {
        held = group;
        row = FewRow(a, group * kGroup + lane % kGroup, rows);
        sloped = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int64_t t = __shfl_sync(~0u, row.t, i);
          const bool has = __shfl_sync(~0u, row.scale, i) != 0.0f && t >= 0;
          sloped |= unsigned(has) << i;
          w[i] = has ? load<F32>(static_cast<const E*>(a.hidden) + t * a.hidden_stride, d, a.D, hidden_vector)
                     : make_uint4(0, 0, 0, 0);
        }
      }
      float g[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int64_t v = vs + n * 4 + lane / kGroup;
        g[n] = row.t >= 0 && v < a.V ? row.gradient(a.z[logit_at(a, group, v, lane % kGroup)], v) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!(sloped >> i & 1)) continue;
        float h[W];
        unpack<F32>(w[i], h);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float x = __shfl_sync(~0u, g[q / 4], q % 4 * kGroup + i);
#pragma unroll
          for (int j = 0; j < W; ++j) sum[q][j] = fmaf(x, h[j], sum[q][j]);
        }
      }
    }
    if (d >= a.D) continue;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (vs + q >= a.V) break;
      E* const to = static_cast<E*>(a.dweight) + (vs + q) * a.dweight_stride;
      float x[W];
      if (a.accumulate) {
        unpack<F32>(load<F32>(to, d, a.D, dweight_vector), x);
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = fmaf(f, sum[q][j], x[j]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = f * sum[q][j];
      }
      if (dweight_vector && d + W <= a.D) {
        uint32_t words[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (F32) {
            words[j] = __float_as_uint(x[j % W]);
          } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j % W], x[(2 * j + 1) % W]);
            words[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        *reinterpret_cast<uint4*>(to + d) = make_uint4(words[0], words[1], words[2], words[3]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (d + j < a.D) to[d + j] = E(x[j]);
      }
    }
  }
}

// Part `part` of the vocabulary's products for a group's rows of dhidden: the warps take
// the weight's rows in turn, four at a time, and their sums are added in order.
template <bool F32, int R>
__device__ __forceinline__ void hidden_part(const Args& a, int part, int64_t d0, int group, int rows, bool vector,
                                            uint4* shared) {
  using E = Element<F32>;
  constexpr int W = kWide<F32>;
  float* const sums = reinterpret_cast<float*>(shared);  // when the ring is through
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t fours = (a.V + 3) / 4, begin = fours * part / a.splits, end = fours * (part + 1) / a.splits;
  const int64_t d = d0 + lane * W;
  const FewRow row(a, group * kGroup + lane % kGroup, rows);
  const int count = min(kGroup, rows - group * kGroup);
  float sum[R][W] = {};
  Ring ring(shared, warp, lane);
  int64_t next = begin + warp;
  float z[kAhead];  // the logits of the steps on their way
  const auto fetch = [&](int n) {
    if (next < end) {
      const int64_t v = next * 4 + lane / kGroup;
      z[n] = row.t >= 0 && v < a.V ? a.z[logit_at(a, group, v, lane % kGroup)] : 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ring.copy<F32>(q, static_cast<const E*>(a.weight) + min(next * 4 + q, a.V - 1) * a.weight_stride, d, a.D, vector);
    }
    next += 8;
    ring.commit();
  };
#pragma unroll
  for (int n = 0; n < kAhead; ++n) fetch(n);
  for (int64_t four = begin + warp; four < end;) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n, four += 8) {
      if (four >= end) break;
      const int64_t v = four * 4 + lane / kGroup;
      const float g = row.t >= 0 && v < a.V ? row.gradient(z[n], v) : 0.0f;
      ring.wait();
      float x[4][W];
#pragma unroll
      for (int q = 0; q < 4; ++q) unpack<F32>(ring[q], x[q]);
      fetch(n);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (four * 4 + q >= a.V) break;  // (the same in all lanes)
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float y = __shfl_sync(~0u, g, q * kGroup + i);
#pragma unroll
          for (int j = 0; j < W; ++j) sum[i][j] = fmaf(y, x[q][j], sum[i][j]);
        }
      }
    }
  }
  // [warp][column], a row of the group at a time.
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i >= count) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) sums[(warp * 32 + lane) * W + j] = sum[i][j];
    __syncthreads();
    for (int n = threadIdx.x; n < 32 * W; n += 256) {
      float x = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) x += sums[q * 32 * W + n];
      if (d0 + n < a.Dp) a.dh[(int64_t(part) * a.Tp + group * kGroup + i) * a.Dp + d0 + n] = x;
    }
  }
}

// R: rows of a group that there can be, 4 or 8.
template <bool F32, int R>
__global__ void __launch_bounds__(256, 2) few_gradients_kernel(const Args a, int64_t hidden_blocks, int wide,
                                                               bool hidden_vector, bool weight_vector,
                                                               bool dweight_vector) {
  constexpr int kBlock = 32 * kWide<F32>;  // columns
  extern __shared__ __align__(16) uint4 shared[];
  static_assert(8 * kBlock * int(sizeof(float)) <= kRingBytes, "the sums take the ring's place");
  let_next_start();
  wait_for_previous();
  const int rows = a.head->rows;
  if (int64_t(blockIdx.x) < hidden_blocks) {  // (the longer pieces of work first)
    const int n = blockIdx.x, group = n / (wide * a.splits), rest = n % (wide * a.splits);
    if (group * kGroup < rows)
      hidden_part<F32, R>(a, rest / wide, int64_t(rest % wide) * kBlock, group, rows, weight_vector, shared);
  } else {
    const int64_t n = int64_t(blockIdx.x) - hidden_blocks, all = int64_t(gridDim.x) - hidden_blocks;
    weight_tiles<F32, R>(a, n / wide, all / wide, n % wide * kBlock, rows, hidden_vector, dweight_vector);
  }
}

}  // namespace

cudaError_t launch_few_logits(const Args& a, int device, cudaStream_t s) {
  const bool f32 = a.planes == 3;
  const int es = f32 ? 4 : 2, step = f32 ? 128 : 256;
  const int width = int((a.D + step - 1) / step * step);
  const size_t shared = kRingBytes + size_t(kGroup) * width * es;
  auto* kernel = f32 ? few_logits_kernel<true> : few_logits_kernel<false>;
  // Once per device (a race only does it twice): the kernel's shared memory.
  static std::atomic<bool> ready[2][64];
  if (device < 0 || device >= 64 || !ready[f32][device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRingBytes + kFewHiddenBytes);
    if (e != cudaSuccess) return e;
    if (device >= 0 && device < 64) ready[f32][device].store(true, std::memory_order_release);
  }
  const dim3 grid(unsigned(a.partials), unsigned((a.T + kGroup - 1) / kGroup));
  return launch(kernel, grid, 256, shared, s, true, a, width, aligned16(a.hidden, a.hidden_stride * es),
                aligned16(a.weight, a.weight_stride * es));
}

cudaError_t launch_few_gradients(const Args& a, cudaStream_t s) {
  const bool f32 = a.planes == 3;
  const int es = f32 ? 4 : 2;
  const int64_t block = f32 ? 128 : 256, wide = (a.D + block - 1) / block;
  const int64_t tiles = (a.V + kTileV - 1) / kTileV, most = 4 * kSms / wide;
  const int64_t weight_blocks = a.dweight ? (tiles < most ? tiles : most < 1 ? 1 : most) * wide : 0;
  const int64_t hidden_blocks = a.dhidden ? (a.T + kGroup - 1) / kGroup * wide * a.splits : 0;
  auto* kernel = a.T <= 4 ? (f32 ? few_gradients_kernel<true, 4> : few_gradients_kernel<false, 4>)
                          : (f32 ? few_gradients_kernel<true, 8> : few_gradients_kernel<false, 8>);
  return launch(kernel, dim3(unsigned(weight_blocks + hidden_blocks)), 256, kRingBytes, s, true, a, hidden_blocks, int(wide),
                aligned16(a.hidden, a.hidden_stride * es), aligned16(a.weight, a.weight_stride * es),
                a.dweight && aligned16(a.dweight, a.dweight_stride * es));
}

}  // namespace zl
