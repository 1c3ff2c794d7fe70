// Kernels of the vocabulary losses (zero_xent_*, zero_distill_*).
#include <math.h>

#include "loss_device.cuh"

namespace zl {
namespace {

__device__ __forceinline__ float warp_max(float x) {
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// ------------------------------------------------------------------- rows --

// One warp per row: its terms, and its sparse entries -- the ids whose logits
// enter the loss one by one -- with the weights c in
//   loss = ce*lse + kd*tau*lse' + konst - sum_e c_e z_e,
//   dloss/dz_v = ce*p_v + kd*p'_v - sum_{e: id_e = v} c_e
// (c = ce for the label, kd*q for a teacher entry; kd = alpha*tau). Equal ids
// are merged, in entry order, and the ids are sorted so that a tile's entries
// are found by bisection.
__device__ __forceinline__ void prepare_row(const Args& a, int64_t t, int32_t* sh) {
  const int lane = threadIdx.x & 31;
  const int K = a.K;
  int64_t y = a.has_ce ? a.labels[t] : -1;
  const bool has_y = a.has_ce && y != a.ignore_index && y >= 0 && y < a.V;
  int32_t* ids = a.ids + t * a.L;
  float* weights = a.weights + t * a.L;
  bool has_kd = false;
  if (K == 0) {
    if (lane == 0) {
      ids[0] = has_y ? int32_t(y) : kNoId;
      weights[0] = a.ce;
      a.konst[t] = 0.0f;
    }
  } else {
    int32_t* id = sh;
    float* c = reinterpret_cast<float*>(id + (K + 1));
    int32_t* id2 = id + 2 * (K + 1);
    float* c2 = reinterpret_cast<float*>(id + 3 * (K + 1));
    float top = -INFINITY;
    for (int k = lane; k < K; k += 32) {
      const int64_t v = a.teacher_ids[t * K + k];
      const float u = a.teacher_logits[t * K + k] / float(a.tau);
      const bool there = v >= 0 && v < a.V && u != -INFINITY;
      id[k] = there ? int32_t(v) : kNoId;
      c[k] = u;
      if (there) {
        has_kd = true;
        top = fmaxf(top, u);
      }
    }
    has_kd = __any_sync(~0u, has_kd);
    top = warp_max(top);
    float sum = 0.0f;
    for (int k = lane; k < K; k += 32) {
      const float e = id[k] == kNoId ? 0.0f : expf(c[k] - top);
      c[k] = e;
      sum += e;
    }
    sum = warp_sum(sum);
    float entropy = 0.0f;
    for (int k = lane; k < K; k += 32) {
      const float q = has_kd ? c[k] / sum : 0.0f;
      if (q != 0.0f) entropy += q * logf(q);
      c[k] = a.kd * q;
    }
    entropy = warp_sum(entropy);
    __syncwarp();
    bool found = false;
    for (int k = lane; k < K; k += 32) {
      const int32_t v = id[k];
      float w = 0.0f;
      bool first = v != kNoId;
      for (int j = 0; first && j < K; ++j) {
        if (id[j] != v) continue;
        if (j < k) first = false;
        w += c[j];
      }
      if (first && has_y && v == y) {
        w += a.ce;
        found = true;
      }
      id2[k] = first ? v : kNoId;
      c2[k] = w;
    }
    found = __any_sync(~0u, found);
    if (lane == 0) {
      id2[K] = has_y && !found ? int32_t(y) : kNoId;
      c2[K] = a.ce;
      a.konst[t] = has_kd ? float(double(a.kd) * a.tau * entropy) : 0.0f;
    }
    __syncwarp();
    int kept = 0;
    for (int k = lane; k <= K; k += 32) kept += id2[k] != kNoId;
    kept = __reduce_add_sync(~0u, kept);
    for (int k = lane; k <= K; k += 32) {
      const int32_t v = id2[k];
      if (v == kNoId) continue;
      int rank = 0;
      for (int j = 0; j <= K; ++j) rank += id2[j] < v;
      ids[rank] = v;
      weights[rank] = c2[k];
    }
    for (int k = kept + lane; k < a.L; k += 32) {
      ids[k] = kNoId;
      weights[k] = 0.0f;
    }
  }
  if (lane == 0) {
    a.coef[t] = make_float2(has_y ? a.ce : 0.0f, has_kd ? a.kd : 0.0f);
    a.rowpos[t] = has_y || has_kd ? 0 : -1;
    if (a.forward && !(has_y || has_kd)) {
      a.loss[t] = 0.0f;
      if (a.has_ce) a.lse[t] = 0.0f;
      if (a.has_kd) a.lse_tau[t] = 0.0f;
    }
  }
}

__global__ void rows_kernel(const Args a) {
  extern __shared__ int32_t sh[];
  const int warp = threadIdx.x >> 5;
  const int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (t < a.T) prepare_row(a, t, sh + warp * 4 * (a.K + 1));
}

// One block: numbers the rows that have a target, in order, up to 16 times
// 1024 rows at a time. With `Prepare` (few rows) it prepares them first, which
// saves a launch.
template <bool Prepare>
__global__ void __launch_bounds__(1024) number_rows_kernel(const Args a) {
  extern __shared__ int32_t sh[];
  __shared__ int32_t before[16][32], total[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (Prepare) {
    for (int64_t t = warp; t < a.T; t += 32) prepare_row(a, t, sh + warp * 4 * (a.K + 1));
    __syncthreads();
  }
  for (int64_t n = threadIdx.x; n < a.zeros; n += 1024) a.counters[n] = 0;
  int32_t base = 0;
  for (int64_t t0 = 0; t0 < a.T; t0 += 16 * 1024) {
    uint32_t mask[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t t = t0 + 1024 * q + threadIdx.x;
      mask[q] = t < a.T && a.rowpos[t] >= 0;
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      mask[q] = __ballot_sync(~0u, mask[q] != 0);
      if (lane == 0) before[q][warp] = __popc(mask[q]);
    }
    __syncthreads();
    if (warp < 16) {
      const int32_t mine = before[warp][lane];
      int32_t upto = mine;
      for (int o = 1; o < 32; o *= 2) {
        const int32_t x = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += x;
      }
      before[warp][lane] = upto - mine;
      if (lane == 31) total[warp] = upto;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      if (mask[q] >> lane & 1) {
        const int64_t t = t0 + 1024 * q + threadIdx.x;
        const int32_t i = base + before[q][warp] + __popc(mask[q] & ((1u << lane) - 1));
        a.rowpos[t] = i;
        a.rowmap[i] = int32_t(t);
      }
      base += total[q];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    // The factor of both gradients that does not depend on the row: grad_scale,
    // the mean's count, and the reduced loss's own gradient.
    double f = a.grad_scale;
    if (a.reduction == ZERO_REDUCE_MEAN) f /= double(max(1, base));
    if (a.reduction != ZERO_REDUCE_NONE && a.dloss) f *= double(*a.dloss);
    *a.head = Head{base, 0, 0, float(f)};
  }
}

// ------------------------------------------------------------------- pack --

// Eight elements of a row from `from` (16-byte aligned where `Vector`), those
// from D on as zeros, as 16-byte words of the planes.
template <bool F32, bool Vector>
__device__ __forceinline__ void pack8(const void* from, int64_t offset, int valid, __nv_bfloat16* to, int64_t plane) {
  if (F32) {
    const float* p = static_cast<const float*>(from) + offset;
    float x[8];
    if (Vector && valid >= 8) {
      *reinterpret_cast<float4*>(x) = reinterpret_cast<const float4*>(p)[0];
      *reinterpret_cast<float4*>(x + 4) = reinterpret_cast<const float4*>(p)[1];
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = q < valid ? p[q] : 0.0f;
    }
    __nv_bfloat16 part[8][3];
#pragma unroll
    for (int q = 0; q < 8; ++q) split(x[q], part[q]);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      uint4 w;
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(&w);
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] = part[q][i];
      *reinterpret_cast<uint4*>(to + i * plane) = w;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(from) + offset;
    uint4 w;
    if (Vector && valid >= 8) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(&w);
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] = q < valid ? p[q] : __nv_bfloat16(0.0f);
    }
    *reinterpret_cast<uint4*>(to) = w;
  }
}

// Rows with a target side by side; zeros after the last, up to the tile.
template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) pack_hidden_kernel(const Args a) {
  const int32_t rows = a.head->rows;
  const int32_t wide = int32_t(a.Dp / 8), all = (rows + kTileM - 1) / kTileM * kTileM;
  for (int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x; n < int64_t(all) * wide; n += int64_t(gridDim.x) * 256) {
    const int32_t i = int32_t(n / wide), k = int32_t(n % wide) * 8;
    const int64_t t = i < rows ? a.rowmap[i] : 0;
    pack8<F32, Vector>(a.hidden, t * a.hidden_stride + k, i < rows ? int(min(a.D - k, int64_t(8))) : 0,
                       a.hp + i * a.Dp + k, a.Tp * a.Dp);
  }
}

template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) pack_weight_kernel(const Args a, __nv_bfloat16* to) {
  const int32_t wide = int32_t(a.Dp / 8);
  for (int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x; n < a.V * wide; n += int64_t(gridDim.x) * 256) {
    const int64_t v = n / wide, k = n % wide * 8;
    pack8<F32, Vector>(a.weight, v * a.weight_stride + k, int(min(a.D - k, int64_t(8))), to + v * a.Dp + k,
                       a.V * a.Dp);
  }
}

// The rows' sums over all pieces, with the common factor, four elements a thread.
template <bool F32, bool Vector>
__global__ void __launch_bounds__(256) dhidden_out_kernel(const Args a) {
  const float f = a.head->fault ? NAN : a.head->factor;
  const int32_t wide = int32_t((a.D + 3) / 4);
  for (int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x; n < a.T * wide; n += int64_t(gridDim.x) * 256) {
    const int64_t t = n / wide, d = n % wide * 4;
    const int32_t i = a.rowpos[t];
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= 0) {
      for (int p = 0; p < a.splits; ++p) {
        const float4 y = *reinterpret_cast<const float4*>(a.dh + (p * a.Tp + i) * a.Dp + d);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
      x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
    }
    const int64_t at = t * a.dhidden_stride + d;
    const float v[4] = {x.x, x.y, x.z, x.w};
    if (F32) {
      float* to = static_cast<float*>(a.dhidden) + at;
      if (Vector && d + 4 <= a.D) {
        *reinterpret_cast<float4*>(to) = x;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (d + q < a.D) to[q] = v[q];
      }
    } else {
      __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.dhidden) + at;
      if (Vector && d + 4 <= a.D) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t*>(&lo);
        w.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(to) = w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (d + q < a.D) to[q] = __float2bfloat16_rn(v[q]);
      }
    }
  }
}

// ------------------------------------------------------------------- losses --

// The row's log-sum-exp from its partial maxima and sums (maxima in powers of
// two): 8 lanes of a row, each every eighth partial, eight loads in flight.
__device__ __forceinline__ double row_lse(const float2* stats, int64_t count, int64_t Tp, int64_t i,
                                          int lane, float2 (*sh)[33], int r) {
  float m = -INFINITY, s = 0.0f;
  for (int64_t j0 = lane; j0 < count; j0 += 64) {
    float2 x[8];
    float top = m;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      x[q] = j0 + 8 * q < count ? stats[(j0 + 8 * q) * Tp + i] : make_float2(-INFINITY, 0.0f);
      top = fmaxf(top, x[q].x);
    }
    if (top == -INFINITY) {
      // Nothing yet -- unless a partial is NaN (fmaxf passes it over).
#pragma unroll
      for (int q = 0; q < 8; ++q) s += x[q].y;
      continue;
    }
    s = m == -INFINITY ? s : s * exp2f(m - top);
#pragma unroll
    for (int q = 0; q < 8; ++q) s += x[q].y * exp2f(x[q].x - top);  // 0 where x is -inf
    m = top;
  }
  sh[lane][r] = make_float2(m, s);
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, sh[j][r].x);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += top == -INFINITY ? sh[j][r].y : sh[j][r].y * exp2f(sh[j][r].x - top);
  }
  __syncthreads();
  return lane == 0 ? (double(top) + log2(double(sum))) * 0.69314718055994530942 : 0.0;
}

__global__ void __launch_bounds__(256) losses_kernel(const Args a) {
  __shared__ float2 sh[8][33];
  __shared__ double part[256];
  __shared__ bool last;
  const int r = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int32_t rows = a.head->rows;
  double mine = 0.0;
  for (int64_t i0 = int64_t(blockIdx.x) * 32; i0 < rows; i0 += int64_t(gridDim.x) * 32) {
    const int64_t i = i0 + r;
    const int64_t at = min(i, int64_t(rows) - 1);
    const double lse = a.has_ce ? row_lse(a.stats, 2 * a.tiles, a.Tp, at, lane, sh, r) : 0.0;
    const double lse_tau = a.has_kd ? row_lse(a.stats_tau, 2 * a.tiles, a.Tp, at, lane, sh, r) : 0.0;
    if (lane == 0 && i < rows) {
      const int64_t t = a.rowmap[i];
      const float2 f = a.coef[t];
      double loss = double(a.konst[t]);
      if (f.x != 0.0f) loss += double(f.x) * lse;
      if (f.y != 0.0f) loss += double(f.y) * a.tau * lse_tau;
      for (int e = 0; e < a.L && a.ids[t * a.L + e] != kNoId; ++e)
        loss -= double(a.weights[t * a.L + e]) * double(a.zent[t * a.L + e]);
      if (a.head->fault) loss = NAN;
      a.loss[t] = float(loss);
      if (a.has_ce) a.lse[t] = float(lse);
      if (a.has_kd) a.lse_tau[t] = float(lse_tau);
      mine += double(float(loss));
    }
  }
  if (a.reduction == ZERO_REDUCE_NONE) return;
  // Each block's sum in lane order; the last block to finish adds the blocks'.
  if (lane == 0) {
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
    if (r == 0) {
      a.sums[blockIdx.x] = mine;
      __threadfence();
      last = atomicAdd(&a.head->ticket, 1) == int32_t(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
  for (int b = threadIdx.x; b < int(gridDim.x); b += 256) sum += __ldcg(a.sums + b);
  part[threadIdx.x] = sum;
  __syncthreads();
  for (int w = 128; w; w >>= 1) {
    if (int(threadIdx.x) < w) part[threadIdx.x] += part[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0)
    *a.reduced = float(a.reduction == ZERO_REDUCE_MEAN ? part[0] / double(max(1, rows)) : part[0]);
}

}  // namespace

namespace {

// A grid for `n` items of 256 threads, a few blocks a thread at most.
unsigned blocks_for(int64_t n) {
  const int64_t blocks = (n + 255) / 256;
  return unsigned(blocks < 1 ? 1 : blocks > 152 * 32 ? 152 * 32 : blocks);
}

bool aligned16(const void* p, int64_t stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  // Few rows: one block prepares them too (32 warps, a row each at a time).
  const size_t row = a.K ? size_t(16) * (a.K + 1) : 0;
  if (a.T <= 256 && 32 * row <= 48 * 1024) {
    number_rows_kernel<true><<<1, 1024, 32 * row, s>>>(a);
    return cudaGetLastError();
  }
  if (a.T > 0) {
    const int warps = a.K > 256 ? 1 : 4;
    rows_kernel<<<unsigned((a.T + warps - 1) / warps), warps * 32, warps * row, s>>>(a);
  }
  number_rows_kernel<false><<<1, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pack_hidden(const Args& a, cudaStream_t s) {
  const bool vector = aligned16(a.hidden, a.hidden_stride * (a.planes == 3 ? 4 : 2));
  const unsigned blocks = blocks_for(a.Tp * a.Dp / 8);
  if (a.planes == 3) {
    if (vector) pack_hidden_kernel<true, true><<<blocks, 256, 0, s>>>(a);
    else pack_hidden_kernel<true, false><<<blocks, 256, 0, s>>>(a);
  } else {
    if (vector) pack_hidden_kernel<false, true><<<blocks, 256, 0, s>>>(a);
    else pack_hidden_kernel<false, false><<<blocks, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_pack_weight(const Args& a, __nv_bfloat16* to, cudaStream_t s) {
  const unsigned blocks = blocks_for(a.V * a.Dp / 8);
  if (a.planes == 3) {
    if (aligned16(a.weight, a.weight_stride * 4)) pack_weight_kernel<true, true><<<blocks, 256, 0, s>>>(a, to);
    else pack_weight_kernel<true, false><<<blocks, 256, 0, s>>>(a, to);
  } else {  // bf16 that is aligned is read in place
    pack_weight_kernel<false, false><<<blocks, 256, 0, s>>>(a, to);
  }
  return cudaGetLastError();
}

cudaError_t launch_losses(const Args& a, cudaStream_t s) {
  const int64_t blocks = (a.T + 31) / 32;
  losses_kernel<<<unsigned(blocks < 1 ? 1 : blocks < kLossBlocks ? blocks : kLossBlocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_dhidden_out(const Args& a, cudaStream_t s) {
  const bool vector = aligned16(a.dhidden, a.dhidden_stride * (a.planes == 3 ? 4 : 2));
  const unsigned blocks = blocks_for(a.T * ((a.D + 3) / 4));
  if (a.planes == 3) {
    if (vector) dhidden_out_kernel<true, true><<<blocks, 256, 0, s>>>(a);
    else dhidden_out_kernel<true, false><<<blocks, 256, 0, s>>>(a);
  } else {
    if (vector) dhidden_out_kernel<false, true><<<blocks, 256, 0, s>>>(a);
    else dhidden_out_kernel<false, false><<<blocks, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace zl
