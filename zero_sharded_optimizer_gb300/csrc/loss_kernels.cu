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
__global__ void rows_kernel(const Args a) {
  extern __shared__ int32_t sh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = int64_t(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
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
    int32_t* id = sh + warp * 4 * (K + 1);
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

// One block: numbers the rows that have a target, in order.
__global__ void __launch_bounds__(1024) number_rows_kernel(const Args a) {
  __shared__ int32_t warps[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t base = 0;
  for (int64_t t0 = 0; t0 < a.T; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    const bool there = t < a.T && a.rowpos[t] >= 0;
    const unsigned mask = __ballot_sync(~0u, there);
    if (lane == 0) warps[warp] = __popc(mask);
    __syncthreads();
    int32_t before = base, all = base;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warps[w];
      all += warps[w];
    }
    if (there) {
      const int32_t i = before + __popc(mask & ((1u << lane) - 1));
      a.rowpos[t] = i;
      a.rowmap[i] = int32_t(t);
    }
    base = all;
    __syncthreads();
  }
  for (int64_t n = threadIdx.x; n < a.launches; n += 1024) a.counters[n] = 0;
  if (threadIdx.x == 0) {
    a.head->rows = base;
    a.head->ticket = 0;
    a.head->fault = 0;
  }
}

// ------------------------------------------------------------------- pack --

template <bool F32>
__device__ __forceinline__ void pack_row(const void* from, int64_t offset, bool there, int64_t D,
                                         int64_t Dp, __nv_bfloat16* to, int64_t plane) {
  for (int64_t k = threadIdx.x; k < Dp; k += blockDim.x) {
    const bool in = there && k < D;
    if (F32) {
      __nv_bfloat16 part[3];
      split(in ? static_cast<const float*>(from)[offset + k] : 0.0f, part);
      for (int p = 0; p < 3; ++p) to[p * plane + k] = part[p];
    } else {
      to[k] = in ? static_cast<const __nv_bfloat16*>(from)[offset + k] : __nv_bfloat16(0.0f);
    }
  }
}

// Rows with a target side by side; zeros after the last, up to the tile.
template <bool F32>
__global__ void pack_hidden_kernel(const Args a) {
  const int64_t i = blockIdx.x;
  const int32_t rows = a.head->rows;
  if (i >= (int64_t(rows) + kTileM - 1) / kTileM * kTileM) return;
  const bool there = i < rows;
  const int64_t t = there ? a.rowmap[i] : 0;
  pack_row<F32>(a.hidden, t * a.hidden_stride, there, a.D, a.Dp, a.hp + i * a.Dp, a.Tp * a.Dp);
}

template <bool F32>
__global__ void pack_weight_kernel(const Args a, __nv_bfloat16* to) {
  const int64_t v = blockIdx.x;
  pack_row<F32>(a.weight, v * a.weight_stride, true, a.D, a.Dp, to + v * a.Dp, a.V * a.Dp);
}

template <bool F32>
__global__ void dhidden_out_kernel(const Args a) {
  const int64_t t = blockIdx.x;
  const int32_t i = a.rowpos[t];
  const float f = a.head->fault ? NAN : grad_factor(a);
  for (int64_t d = threadIdx.x; d < a.D; d += blockDim.x) {
    float x = 0.0f;
    if (i >= 0) {
      for (int p = 0; p < a.splits; ++p) x += a.dh[(p * a.Tp + i) * a.Dp + d];
      x *= f;
    }
    if (F32) static_cast<float*>(a.dhidden)[t * a.dhidden_stride + d] = x;
    else static_cast<__nv_bfloat16*>(a.dhidden)[t * a.dhidden_stride + d] = __float2bfloat16_rn(x);
  }
}

// ------------------------------------------------------------------- losses --

// The row's log-sum-exp from its partial maxima and sums (maxima in powers of
// two): 8 lanes of a row, each every eighth partial.
__device__ __forceinline__ double row_lse(const float2* stats, int64_t count, int64_t Tp, int64_t i,
                                          int lane, float2 (*sh)[33], int r) {
  float m = -INFINITY, s = 0.0f;
  for (int64_t j = lane; j < count; j += 8) {
    const float2 x = stats[j * Tp + i];
    if (!(x.x <= m)) {      // a NaN maximum goes on
      s = s * (m == -INFINITY ? 0.0f : exp2f(m - x.x)) + x.y;
      m = x.x;
    } else {
      s += x.x == -INFINITY ? 0.0f : x.y * exp2f(x.x - m);
    }
  }
  sh[lane][r] = make_float2(m, s);
  __syncthreads();
  double top = -INFINITY, sum = 0.0;
  if (lane == 0) {
    for (int j = 0; j < 8; ++j)
      if (!(sh[j][r].x <= top)) top = sh[j][r].x;
    for (int j = 0; j < 8; ++j)
      if (sh[j][r].x != -INFINITY) sum += double(sh[j][r].y) * exp2(double(sh[j][r].x) - top);
  }
  __syncthreads();
  return (top + log2(sum)) * 0.69314718055994530942;
}

__global__ void __launch_bounds__(256) losses_kernel(const Args a) {
  __shared__ float2 sh[8][33];
  __shared__ double part[256];
  __shared__ bool last;
  const int r = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int32_t rows = a.head->rows;
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
    }
  }
  if (a.reduction == ZERO_REDUCE_NONE) return;
  // The last block to finish adds the losses in a fixed order.
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    last = atomicAdd(&a.head->ticket, 1) == int32_t(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
  for (int64_t t = threadIdx.x; t < a.T; t += 256) sum += double(__ldcg(a.loss + t));
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

cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  if (a.T > 0) {
    const int warps = a.K > 256 ? 1 : 4;
    const size_t sh = a.K ? size_t(warps) * 16 * (a.K + 1) : 0;
    rows_kernel<<<unsigned((a.T + warps - 1) / warps), warps * 32, sh, s>>>(a);
  }
  number_rows_kernel<<<1, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pack_hidden(const Args& a, cudaStream_t s) {
  if (a.planes == 3) pack_hidden_kernel<true><<<unsigned(a.Tp), 128, 0, s>>>(a);
  else pack_hidden_kernel<false><<<unsigned(a.Tp), 128, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pack_weight(const Args& a, __nv_bfloat16* to, cudaStream_t s) {
  if (a.planes == 3) pack_weight_kernel<true><<<unsigned(a.V), 128, 0, s>>>(a, to);
  else pack_weight_kernel<false><<<unsigned(a.V), 128, 0, s>>>(a, to);
  return cudaGetLastError();
}

cudaError_t launch_losses(const Args& a, cudaStream_t s) {
  const int64_t blocks = a.Tp / 32;
  losses_kernel<<<unsigned(blocks < 608 ? blocks : 608), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_dhidden_out(const Args& a, cudaStream_t s) {
  if (a.planes == 3) dhidden_out_kernel<true><<<unsigned(a.T), 128, 0, s>>>(a);
  else dhidden_out_kernel<false><<<unsigned(a.T), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace zl
