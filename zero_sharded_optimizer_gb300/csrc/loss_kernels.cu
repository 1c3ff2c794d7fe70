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

// First entry of the row whose id is not below v.
__device__ __forceinline__ int first_entry(const int32_t* ids, int L, int32_t v) {
  int lo = 0, hi = L;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ids[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// Rows are prepared for the products: each row's terms, and its sparse entries
// -- the ids whose logits enter the loss one by one -- with the weights c in
//   loss = ce*lse + kd*tau*lse' + konst - sum_e c_e z_e,
//   dloss/dz_v = ce*p_v + kd*p'_v - sum_{e: id_e = v} c_e
// (c = ce for the label, kd*q for a teacher entry; kd = alpha*tau).

__device__ __forceinline__ int64_t label_of(const Args& a, int64_t t) {  // -1: none
  if (!a.has_ce) return -1;
  const int64_t y = a.labels[t];
  return y != a.ignore_index && y >= 0 && y < a.V ? y : -1;
}

__device__ __forceinline__ void finish_row(const Args& a, int64_t t, bool has_y, bool has_kd, float konst) {
  a.konst[t] = konst;
  a.coef[t] = make_float2(has_y ? a.ce : 0.0f, has_kd ? a.kd : 0.0f);
  a.rowpos[t] = has_y || has_kd ? 0 : -1;
  if (a.forward && !(has_y || has_kd)) {
    a.loss[t] = 0.0f;
    if (a.has_ce) a.lse[t] = 0.0f;
    if (a.has_kd) a.lse_tau[t] = 0.0f;
  }
}

// Cross entropy: the label is the only entry. One thread per row.
__device__ __forceinline__ void prepare_label(const Args& a, int64_t t) {
  const int64_t y = label_of(a, t);
  a.ids[t] = y >= 0 ? int32_t(y) : kNoId;
  a.weights[t] = a.ce;
  finish_row(a, t, y >= 0, false, 0.0f);
}

// Distillation: one warp per row. The entries are sorted by id, equal ids
// merged (in the order given, the label last), so that a tile's entries are a
// range of them. `id` and `c` hold n4 = K + 1 rounded up to 4 values each, as
// do `sid` and `sc`, in shared memory. Leaves the merged ids in `id`, ended by
// kNoId, and returns their number.
__device__ __forceinline__ int prepare_teacher(const Args& a, int64_t t, int n4, int32_t* id, float* c, int32_t* sid,
                                               float* sc) {
  const int lane = threadIdx.x & 31, K = a.K;
  const int64_t y = label_of(a, t);
  bool has_kd = false;
  float top = -INFINITY;
  for (int k = lane; k < K; k += 32) {
    const int64_t v = a.teacher_ids[t * K + k];
    const float u = a.teacher_logits[t * K + k];
    const bool there = v >= 0 && v < a.V && u != -INFINITY;
    id[k] = there ? int32_t(v) : kNoId;  // (ids end below kNoId - 1, so that one can be added)
    c[k] = u;
    if (there) {
      has_kd = true;
      top = fmaxf(top, u);
    }
  }
  for (int k = K + lane; k < n4; k += 32) {
    id[k] = k == K && y >= 0 ? int32_t(y) : kNoId;
    c[k] = a.ce;
  }
  has_kd = __any_sync(~0u, has_kd);
  top = warp_max(top);
  float sum = 0.0f;
  for (int k = lane; k < K; k += 32) {
    // From the maximum before the division: a temperature below one takes large
    // finite logits past fp32's range.
    const float e = id[k] == kNoId ? 0.0f : expf((c[k] - top) / float(a.tau));
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
  // Each entry's place: the entries before it by id, then by position. Four
  // entries a lane at a time against all of them.
  for (int k0 = 0; k0 < n4; k0 += 128) {
    int32_t mine[4];
    int place[4] = {};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + lane + 32 * q;
      mine[q] = k < n4 ? id[k] : 0;
    }
    for (int j = 0; j < n4; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(id + j);
      const int32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (k0 + 32 * q >= n4) break;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          place[q] += w[r] < mine[q] + (j + r < k0 + lane + 32 * q);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + lane + 32 * q;
      if (k < n4) {
        sid[place[q]] = mine[q];
        sc[place[q]] = c[k];
      }
    }
  }
  __syncwarp();
  int kept = 0;
  for (int p0 = 0; p0 < n4; p0 += 32) {
    const int p = p0 + lane;
    const int32_t v = p < n4 ? sid[p] : kNoId;
    const bool first = v != kNoId && (p == 0 || sid[p - 1] != v);
    const unsigned mask = __ballot_sync(~0u, first);
    if (first) {
      float w = sc[p];
      for (int q = p + 1; q < n4 && sid[q] == v; ++q) w += sc[q];
      const int at = kept + __popc(mask & ((1u << lane) - 1));
      id[at] = v;
      a.ids[t * a.L + at] = v;
      a.weights[t * a.L + at] = w;
    }
    kept += __popc(mask);
  }
  for (int k = kept + lane; k < a.L; k += 32) a.ids[t * a.L + k] = kNoId;
  if (lane == 0) finish_row(a, t, y >= 0, has_kd, has_kd ? float(double(a.kd) * a.tau * entropy) : 0.0f);
  return kept;
}

__global__ void __launch_bounds__(256) label_rows_kernel(const Args a) {
  let_next_start();
  const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t < a.T) prepare_label(a, t);
}

constexpr int kTeacherRows = 16;                  // most rows of a block of teacher_rows_kernel
constexpr size_t kSharedWithoutAsking = 48 << 10;  // static and dynamic shared memory of a launch

// A block's rows, one a warp, and where each half tile's entries begin in
// them: starts[h][t] is the first entry with an id of 128 h at least.
__global__ void teacher_rows_kernel(const Args a) {
  extern __shared__ __align__(16) int32_t sh[];
  __shared__ int kept[kTeacherRows];
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = blockDim.x >> 5;
  const int n4 = (a.K + 4) / 4 * 4;
  const int64_t t0 = int64_t(blockIdx.x) * rows, t = t0 + warp;
  int32_t* id = sh + warp * 4 * n4;
  if (t < a.T) {
    const int n = prepare_teacher(a, t, n4, id, reinterpret_cast<float*>(id + n4), id + 2 * n4,
                                  reinterpret_cast<float*>(id + 3 * n4));
    if (lane == 0) kept[warp] = n;
  }
  __syncthreads();
  const int r = threadIdx.x & (rows - 1);  // rows: a power of two
  if (t0 + r >= a.T) return;
  const int32_t* ids = sh + r * 4 * n4;
  const int n = kept[r];
  // 32 threads a row, each a stretch of the half tiles.
  const int halves = int(2 * a.tiles + 1), stretch = (halves + 31) / 32;
  const int h0 = threadIdx.x / rows * stretch, h1 = min(halves, h0 + stretch);
  int e = h0 < h1 ? first_entry(ids, n, h0 * 128) : 0;
  for (int h = h0; h < h1; ++h) {
    while (e < n && ids[e] < h * 128) ++e;
    a.starts[h * a.T + t0 + r] = uint16_t(e);
  }
}

// ------------------------------------------------------------------- pack --

// A value as bf16 parts: x = p0 + p1 + p2 up to fp32's rounding (each part
// holds the next 8 bits; the rests are exact differences). An infinity and
// a value that would round to one keep the parts finite or zero.
__device__ __forceinline__ void split(float x, __nv_bfloat16 (&part)[3]) {
  part[0] = __float2bfloat16_rn(x);
  if (isinf(__bfloat162float(part[0])) && !isinf(x)) part[0] = __float2bfloat16_rz(x);
  if (isinf(x)) {
    part[1] = part[2] = __float2bfloat16_rn(0.0f);
    return;
  }
  const float r = x - __bfloat162float(part[0]);
  part[1] = __float2bfloat16_rn(r);
  part[2] = __float2bfloat16_rn(r - __bfloat162float(part[1]));
}

// Eight elements of a row from `from` (16-byte aligned where `vector`), those
// from D on as zeros, as 16-byte words of the planes.
template <bool F32>
__device__ __forceinline__ void pack8(const void* from, int64_t offset, int valid, bool vector, __nv_bfloat16* to,
                                      int64_t plane) {
  if (F32) {
    const float* p = static_cast<const float*>(from) + offset;
    float x[8];
    if (vector && valid >= 8) {
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
    if (vector && valid >= 8) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(&w);
#pragma unroll
      for (int q = 0; q < 8; ++q) out[q] = q < valid ? p[q] : __nv_bfloat16(0.0f);
    }
    *reinterpret_cast<uint4*>(to) = w;
  }
}

// Rows with a target side by side, and zeros after the last up to the next
// block of K, for dweight's sums. (Tiles hold further rows, of whatever is
// there: nothing uses what becomes of them.)
template <bool F32>
__device__ __forceinline__ void pack_rows(const Args& a, int32_t rows, bool vector, int64_t first, int64_t step) {
  const int32_t wide = int32_t(a.Dp / 8), all = (rows + 63) / 64 * 64;
  for (int64_t n = first; n < int64_t(all) * wide; n += step) {
    const int32_t i = int32_t(n / wide), k = int32_t(n % wide) * 8;
    const int64_t t = i < rows ? a.rowmap[i] : 0;
    pack8<F32>(a.hidden, t * a.hidden_stride + k, i < rows ? int(min(a.D - k, int64_t(8))) : 0, vector,
               a.hp + i * a.Dp + k, a.Tp * a.Dp);
  }
}

// One block: numbers the rows that have a target, in order, up to 16 times
// 1024 rows at a time. With `Prepare` (few rows, labels alone) it prepares them
// first: a launch saved.
template <bool Prepare>
__global__ void __launch_bounds__(1024) number_rows_kernel(const Args a) {
  __shared__ int32_t before[16][32], total[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  let_next_start();
  if (!Prepare) wait_for_previous();
  if (Prepare) {
    for (int64_t t = threadIdx.x; t < a.T; t += 1024) prepare_label(a, t);
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

// The weight's rows (where it is not read in place; this does not wait for the
// kernels before), and the rows with a target.
template <bool F32>
__global__ void __launch_bounds__(256) pack_kernel(const Args a, __nv_bfloat16* packed_weight, bool hidden_vector,
                                                   bool weight_vector) {
  let_next_start();
  const int32_t wide = int32_t(a.Dp / 8);
  const int64_t first = int64_t(blockIdx.x) * 256 + threadIdx.x, step = int64_t(gridDim.x) * 256;
  if (packed_weight) {
    for (int64_t n = first; n < a.V * wide; n += step) {
      const int64_t v = n / wide, k = n % wide * 8;
      pack8<F32>(a.weight, v * a.weight_stride + k, int(min(a.D - k, int64_t(8))), weight_vector,
                 packed_weight + v * a.Dp + k, a.V * a.Dp);
    }
  }
  wait_for_previous();
  pack_rows<F32>(a, a.head->rows, hidden_vector, first, step);
}

// Where a wait of the matrix kernel ran out, the call's results become NaN --
// dweight, which may be half written, and a step's losses, which were formed
// before the backward pass -- so that nothing goes on with them unnoticed.
__device__ __noinline__ void mark_fault(const Args& a, bool f32, int64_t first, int64_t step) {
  if (a.dweight) {
    for (int64_t n = first; n < a.V * a.D; n += step) {
      const int64_t at = n / a.D * a.dweight_stride + n % a.D;
      if (f32) static_cast<float*>(a.dweight)[at] = NAN;
      else static_cast<__nv_bfloat16*>(a.dweight)[at] = __float2bfloat16_rn(NAN);
    }
  }
  if (!a.forward) return;
  for (int64_t t = first; t < a.T; t += step) {
    if (a.rowpos[t] < 0) continue;
    a.loss[t] = NAN;
    if (a.has_ce) a.lse[t] = NAN;
    if (a.has_kd) a.lse_tau[t] = NAN;
  }
  if (first == 0 && a.reduction != ZERO_REDUCE_NONE) *a.reduced = NAN;
}

__global__ void __launch_bounds__(256) mark_kernel(const Args a) {
  let_next_start();
  wait_for_previous();
  if (a.head->fault) mark_fault(a, a.planes == 3, int64_t(blockIdx.x) * 256 + threadIdx.x, int64_t(gridDim.x) * 256);
}

// The rows' sums over all pieces, with the common factor: a block takes
// 256 / Lanes groups of four elements of a row at a time, each group's `Lanes`
// threads share the parts that the sums are split in.
template <bool F32, bool Vector, int Lanes>
__global__ void __launch_bounds__(256) dhidden_out_kernel(const Args a) {
  constexpr int kGroups = 256 / Lanes;
  __shared__ float4 part[Lanes][kGroups];
  let_next_start();
  wait_for_previous();
  const bool fault = a.head->fault;
  const float f = fault ? NAN : a.head->factor;
  const int group = threadIdx.x % kGroups, lane = threadIdx.x / kGroups;
  const int64_t wide = (a.D + 3) / 4;
  const int64_t stretches = (wide + kGroups - 1) / kGroups;  // of a row
  for (int64_t b = blockIdx.x; b < a.T * stretches; b += gridDim.x) {
    const int64_t t = b / stretches, d = (b % stretches * kGroups + group) * 4;
    const int32_t i = a.rowpos[t];
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= 0 && d < a.D) {
#pragma unroll 8
      for (int p = lane; p < a.splits; p += Lanes) {
        const float4 y = *reinterpret_cast<const float4*>(a.dh + (p * a.Tp + i) * a.Dp + d);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
    }
    if (Lanes > 1) {
      part[lane][group] = x;
      __syncthreads();
      if (lane == 0) {
#pragma unroll
        for (int p = 1; p < Lanes; ++p) {
          const float4 y = part[p][group];
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
      }
      __syncthreads();
    }
    if (lane > 0 || d >= a.D) continue;
    if (i >= 0) x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
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
  if (fault) mark_fault(a, F32, int64_t(blockIdx.x) * 256 + threadIdx.x, int64_t(gridDim.x) * 256);
}

// ------------------------------------------------------------------- losses --

// The row's log-sum-exp from its partial maxima and sums (maxima in powers of
// two): each of the row's lanes takes every lanes-th partial, eight loads in
// flight; the first lane joins them.
__device__ __forceinline__ double row_lse(const float2* stats, int64_t count, int64_t Tp, int64_t i, int lane,
                                          int lanes, float2* sh, int r, int rows) {
  float m = -INFINITY, s = 0.0f;
  for (int64_t j0 = lane; j0 < count; j0 += 8 * lanes) {
    float2 x[8];
    float top = m;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      x[q] = j0 + lanes * q < count ? stats[(j0 + lanes * q) * Tp + i] : make_float2(-INFINITY, 0.0f);
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
  // A tree over the lanes, in a fixed order.
  sh[lane * rows + r] = make_float2(m, s);
  __syncthreads();
  for (int w = lanes / 2; w; w >>= 1) {
    if (lane < w) {
      const float2 x = sh[lane * rows + r], y = sh[(lane + w) * rows + r];
      const float top = fmaxf(x.x, y.x);
      const float sum = top == -INFINITY ? x.y + y.y : x.y * exp2f(x.x - top) + y.y * exp2f(y.x - top);
      sh[lane * rows + r] = make_float2(top, sum);
    }
    __syncthreads();
  }
  const float2 x = sh[r];
  __syncthreads();
  return lane == 0 ? (double(x.x) + log2(double(x.y))) * 0.69314718055994530942 : 0.0;
}

// 256 threads: `block_rows` rows (a power of two, up to 32), 256 / block_rows lanes each.
__global__ void __launch_bounds__(256) losses_kernel(const Args a, int block_rows) {
  __shared__ float2 sh[256];
  __shared__ double part[256];
  __shared__ bool last;
  let_next_start();
  wait_for_previous();
  const int r = threadIdx.x % block_rows, lane = threadIdx.x / block_rows, lanes = 256 / block_rows;
  const int32_t rows = a.head->rows;
  double mine = 0.0;
  for (int64_t i0 = int64_t(blockIdx.x) * block_rows; i0 < rows; i0 += int64_t(gridDim.x) * block_rows) {
    const int64_t i = min(i0 + r, int64_t(rows) - 1);
    const int64_t t = a.rowmap[i];
    double entries = 0.0;
#pragma unroll 4
    for (int e = lane; e < a.L; e += lanes) {
      const int64_t at = t * a.L + e;
      if (a.ids[at] != kNoId) entries += double(a.weights[at]) * double(a.zent[at]);
    }
    const double lse = a.has_ce ? row_lse(a.stats, 2 * a.tiles, a.Tp, i, lane, lanes, sh, r, block_rows) : 0.0;
    const double lse_tau =
        a.has_kd ? row_lse(a.stats_tau, 2 * a.tiles, a.Tp, i, lane, lanes, sh, r, block_rows) : 0.0;
    part[threadIdx.x] = entries;
    __syncthreads();
    for (int w = lanes / 2; w; w >>= 1) {
      if (lane < w) part[threadIdx.x] += part[threadIdx.x + w * block_rows];
      __syncthreads();
    }
    if (lane == 0 && i0 + r < rows) {
      const float2 f = a.coef[t];
      double loss = double(a.konst[t]);
      if (f.x != 0.0f) loss += double(f.x) * lse;
      if (f.y != 0.0f) loss += double(f.y) * a.tau * lse_tau;
      loss -= part[r];
      const bool fault = a.head->fault;  // NaN in lse too: a backward call's gradients show it then
      if (fault) loss = NAN;
      a.loss[t] = float(loss);
      if (a.has_ce) a.lse[t] = fault ? NAN : float(lse);
      if (a.has_kd) a.lse_tau[t] = fault ? NAN : float(lse_tau);
      mine += double(float(loss));
    }
    __syncthreads();
  }
  if (a.reduction == ZERO_REDUCE_NONE) return;
  // Each block's sum in a fixed order; the last block to finish adds the blocks'.
  part[threadIdx.x] = mine;  // zero but for the rows' first lanes
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int q = 1; q < block_rows; ++q) mine += part[q];
    a.sums[blockIdx.x] = mine;
    __threadfence();
    last = atomicAdd(&a.head->ticket, 1) == int32_t(gridDim.x) - 1;
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
  return unsigned(blocks < 1 ? 1 : blocks > kSms * 32 ? kSms * 32 : blocks);
}

// `dependent`: a programmatic launch behind the kernel before it.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned blocks, int threads, size_t shared, cudaStream_t s, bool dependent,
                   const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(unsigned(threads));
  c.dynamicSmemBytes = shared;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

bool aligned16(const void* p, int64_t stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  // Up to as many rows as its block has threads, the numbering kernel prepares
  // them itself. A loss of a vocabulary of 1009 at width 96, replayed: 18.0 us
  // for one row, 18.1 with two kernels; 21.1 and 21.1 for 1024 rows; 21.3 and
  // 20.9 for 2048; 22.7 and 21.6 for 4096. A call that is waited for (one row,
  // GPT-2-small's head): 67 and 70 us. (Packing the rows there too: 33.4 us
  // instead of 31.2, replayed; 39.1 instead of 39.0 from the host.)
  if (a.K == 0 && a.T <= 1024) return launch(number_rows_kernel<true>, 1, 1024, 0, s, false, a);
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    if (a.K == 0) {
      e = launch(label_rows_kernel, unsigned((a.T + 255) / 256), 256, 0, s, false, a);
    } else {
      const size_t row = size_t(16) * ((a.K + 4) / 4 * 4);
      // Rows of a block: 16, whose places in the table fill a 32-byte sector, or
      // what shared memory holds beside `kept`, and fewer where they leave SMs idle
      // (333 rows: 197 us a step instead of 200).
      int rows = kTeacherRows * (row + sizeof(int)) <= kSharedWithoutAsking ? kTeacherRows : 2;
      while (rows > 2 && a.T / rows < kSms) rows /= 2;
      e = launch(teacher_rows_kernel, unsigned((a.T + rows - 1) / rows), rows * 32, rows * row, s, false, a);
    }
  }
  return e != cudaSuccess ? e : launch(number_rows_kernel<false>, 1, 1024, 0, s, a.T > 0, a);
}

cudaError_t launch_pack(const Args& a, __nv_bfloat16* weight, cudaStream_t s) {
  const int es = a.planes == 3 ? 4 : 2;
  const bool hv = aligned16(a.hidden, a.hidden_stride * es), wv = aligned16(a.weight, a.weight_stride * es);
  const unsigned blocks = blocks_for((weight && a.V > a.Tp ? a.V : a.Tp) * a.Dp / 8);
  if (a.planes == 3) return launch(pack_kernel<true>, blocks, 256, 0, s, true, a, weight, hv, wv);
  return launch(pack_kernel<false>, blocks, 256, 0, s, true, a, weight, hv, wv);
}

cudaError_t launch_losses(const Args& a, cudaStream_t s) {
  // As many lanes to a row as leave a block for each SM (333 rows with two
  // softmaxes and 100 entries: a step of 197 us, 227 with 32 rows a block).
  int rows = 32;
  while (rows > 1 && a.T / rows < kSms) rows /= 2;
  const int64_t blocks = (a.T + rows - 1) / rows;
  return launch(losses_kernel, unsigned(blocks < 1 ? 1 : blocks < kLossBlocks ? blocks : kLossBlocks), 256, 0, s,
                true, a, rows);
}

cudaError_t launch_mark(const Args& a, cudaStream_t s) {
  return launch(mark_kernel, kSms, 256, 0, s, true, a);
}

cudaError_t launch_dhidden_out(const Args& a, cudaStream_t s) {
  const bool vector = aligned16(a.dhidden, a.dhidden_stride * (a.planes == 3 ? 4 : 2));
  // Eight lanes where the sums come in that many parts (one row of width 768 in
  // 64 parts: 6 us instead of 18).
  const bool lanes = a.splits >= 8;
  const int64_t groups = lanes ? 32 : 256;
  const int64_t stretches = a.T * (((a.D + 3) / 4 + groups - 1) / groups);
  const unsigned blocks = unsigned(stretches < kSms * 32 ? stretches : kSms * 32);
  const auto run = [&](auto* kernel) { return launch(kernel, blocks, 256, 0, s, true, a); };
  if (a.planes == 3) {
    if (vector) return lanes ? run(dhidden_out_kernel<true, true, 8>) : run(dhidden_out_kernel<true, true, 1>);
    return lanes ? run(dhidden_out_kernel<true, false, 8>) : run(dhidden_out_kernel<true, false, 1>);
  }
  if (vector) return lanes ? run(dhidden_out_kernel<false, true, 8>) : run(dhidden_out_kernel<false, true, 1>);
  return lanes ? run(dhidden_out_kernel<false, false, 8>) : run(dhidden_out_kernel<false, false, 1>);
}

}  // namespace zl
