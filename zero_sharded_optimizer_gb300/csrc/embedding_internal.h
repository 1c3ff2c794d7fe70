// Internal interface between the host side of the embedding (embedding_host.cpp)
// and its kernels (embedding_kernels.cu). Not part of the public C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "host_checks.h"
#include "zero_gb300.h"

namespace ze {

constexpr int kSms = 152;        // GB300's multiprocessors
constexpr int64_t kCacheBytes = int64_t(100) << 20;  // that the L2 cache keeps of a stream of stores
constexpr int kMostBits = 9;     // of a digit of the sort
constexpr int kMostBins = 1 << kMostBits;
constexpr int kMostTiles = 256;  // of the sort

// Up to so many tokens, and ids below so many, one kernel sorts (class_sort_kernel).
constexpr int kPositionBits = 15;
constexpr int64_t kFewTokens = int64_t(1) << kPositionBits;
constexpr int kClassIds = 1024;                     // most ids of a class
constexpr int kMostClassBits = 8;
constexpr int64_t kFewIds = int64_t(kClassIds) << kMostClassBits;

// A token in the sorted list: its id (V, at the list's end: none) and its position.
struct Entry {
  uint32_t id, t;
};

struct Args {
  int64_t T, V, D;
  int32_t f32;
  int32_t accumulate;
  const int64_t* ids;
  int64_t padding_id;
  float scale;
  const void* table;       // forward: weight; backward: dout
  int64_t table_stride;
  void* out;               // forward: out; backward: dweight
  int64_t out_stride;
  int32_t width;           // of the accesses that fit the rows of both: 16, 4 or an element's bytes

  // Backward: the sort's digits and tiles, and the sums' runs of sorted tokens.
  int64_t zero_from;       // rows of dweight from here on become zero while the tokens are sorted, rows
                           // below that no token has while the sums are taken (V, and none, where the
                           // sums are added to dweight)
  int32_t few;             // the tokens are sorted by one kernel
  int32_t class_bits;      // of an id, that say its class there
  int32_t bits, passes;    // of a digit; digits
  int64_t tile;            // tokens of a tile, a multiple of the block's threads
  int32_t tiles;
  int32_t run;             // sorted tokens that one warp adds up
  int64_t runs;
  int32_t blocks;          // blocks of columns
  int64_t Dp;              // their columns
  int32_t* counts;         // [passes][tiles][bins] tokens of a tile by digit
  Entry* list[2];          // [T] before and after a pass
  const Entry* sorted;     // the one that the last pass writes
  float* part;             // [runs][2][Dp] a run's share of the segment that began before it, and of
                           // the one that it began and did not end

  // The sums of the vocabulary losses' rests (loss_kernels.cu): a token's row counts
  // rest_of(scales[t], weights[t]) times, and an id's sum goes to the row of `out` that
  // its slot says.
  const float *scales, *weights;
  const uint2* slots;
};

#ifdef __CUDACC__
// Of 32 ids: which have a slot, and how many slots are before theirs. Slots are in order of id.
__device__ __forceinline__ int32_t slot_of(uint2 slots, int id) {
  return slots.x >> id & 1 ? int32_t(slots.y + __popc(slots.x & ((1u << id) - 1))) : -1;
}

// What the rounding of a label's entry of G to bf16 leaves of it (its weight may be anything
// where its row has no scale).
__device__ __forceinline__ float rest_of(float scale, float weight) {
  const float x = scale == 0.0f ? 0.0f : scale * weight;
  return x - __bfloat162float(__float2bfloat16_rn(x));
}
#endif

// The widest accesses that the rows of table and out allow, of elements of `es` bytes.
int32_t width_of(const Args& a, int es);
// Sets the sort's and the sums' plan for the problem that `a` has, and takes their arrays.
void plan_sums(Args* a, zl::Layout* w);

cudaError_t launch_lookup(const Args& a, cudaStream_t s);
cudaError_t launch_sort(const Args& a, cudaStream_t s);
cudaError_t launch_sums(const Args& a, cudaStream_t s);
cudaError_t launch_rests(const Args& a, cudaStream_t s);

}  // namespace ze
