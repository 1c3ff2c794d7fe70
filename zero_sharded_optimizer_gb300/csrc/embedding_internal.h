// Internal interface between the host side of the embedding (embedding_host.cpp)
// and its kernels (embedding_kernels.cu). Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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
};

cudaError_t launch_lookup(const Args& a, cudaStream_t s);
cudaError_t launch_sort(const Args& a, cudaStream_t s);
cudaError_t launch_sums(const Args& a, cudaStream_t s);

}  // namespace ze
