// Kernels of the vocabulary losses (zero_xent_*, zero_distill_*, zero_policy_*,
// zero_preference_*).
#include <math.h>

#include <type_traits>

#include "embedding_internal.h"
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
  if (a.scales) a.scales[t] = 0.0f;
  if (a.forward && !(has_y || has_kd)) {
    if (a.kind != kPreference) a.loss[t] = 0.0f;
    if (a.row_logps) a.row_logps[t] = 0.0f;
    if (a.kind == kPolicy) a.slopes[t] = 0.0f;
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

// Whether a preference call's offsets ascend within the rows (all threads of the block).
__device__ __forceinline__ bool offsets_ascend(const Args& a) {
  bool good = true;
  if (a.kind == kPreference && a.offsets) {
    for (int64_t n = threadIdx.x; n <= 2 * a.pairs; n += blockDim.x) {
      const int64_t x = a.offsets[n];
      good &= x >= 0 && x <= a.T && (n == 0 || a.offsets[n - 1] <= x);
    }
  }
  return __syncthreads_and(good);
}

// Which rows number_rows_kernel numbers: those with a target, prepared before or
// (few rows, labels alone: a launch saved) by itself, or, before a backward pass by
// slopes, those whose slope is not zero. (8192 rows: 7 us, beside which 30 % fewer
// rows in a policy step's backward products save 350.)
enum Numbering { kTargets, kPrepare, kSlopes };

// One block: numbers the rows in order, up to 16 times 1024 rows at a time.
template <Numbering N>
__global__ void __launch_bounds__(1024) number_rows_kernel(const Args a) {
  __shared__ int32_t before[16][32], total[16], total_of[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  let_next_start();
  if (N != kPrepare) wait_for_previous();
  if (N == kPrepare) {
    for (int64_t t = threadIdx.x; t < a.T; t += 1024) prepare_label(a, t);
    __syncthreads();
  }
  if (N != kSlopes)
    for (int64_t n = threadIdx.x; n < a.zeros; n += 1024) a.counters[n] = 0;
  const bool ascend = N == kSlopes || offsets_ascend(a);
  // A preference loss has the same slope in all rows of a sequence, and often
  // nearly the same in all pairs. Its scales are taken relative to the largest,
  // which the factor of both gradients gets: G's entries of labels that the model
  // finds unlikely, s (1 - p), are near powers of two then, and lose nothing to
  // bf16, where one rounding would go through the whole gradient.
  float unit = 1.0f;
  if (N == kSlopes && a.kind == kPreference) {
    unit = __uint_as_float(a.head->steepest);
    if (!(unit > 0.0f && unit < INFINITY)) unit = 1.0f;
  }
  const int32_t targets = N == kSlopes ? a.head->rows : 0;
  int32_t base = 0;
  for (int64_t t0 = 0; t0 < a.T; t0 += 16 * 1024) {
    uint32_t mask[16];
    int32_t pos[16];
    float scale[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t t = t0 + 1024 * q + threadIdx.x;
      pos[q] = t < a.T ? a.rowpos[t] : -1;
      if (N == kSlopes) scale[q] = t < a.T ? a.scales[t] : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int64_t t = t0 + 1024 * q + threadIdx.x;
      mask[q] = pos[q] >= 0;
      if (N == kSlopes && mask[q]) {
        if (unit != 1.0f) a.scales[t] = scale[q] /= unit;
        mask[q] = scale[q] != 0.0f;  // (also a NaN)
        if (!mask[q]) a.rowpos[t] = -2;
      }
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
        if (N == kSlopes && a.slots) atomicOr(&a.slots[a.ids[t] / 32].x, 1u << a.ids[t] % 32);
      }
      base += total[q];
    }
    __syncthreads();
  }
  if (N == kSlopes && a.slots) {  // the labels in order of id, before each 32 of them
    __threadfence();
    __syncthreads();
    const int64_t words = (a.V + 31) / 32;
    int32_t first = 0;
    for (int64_t w0 = 0; w0 < words; w0 += 1024) {
      const int64_t w = w0 + threadIdx.x;
      const int32_t mine = w < words ? __popc(__ldcg(&a.slots[w].x)) : 0;
      int32_t upto = mine;
      for (int o = 1; o < 32; o *= 2) {
        const int32_t x = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) total_of[warp] = upto;
      __syncthreads();
      int32_t all = 0;
      for (int q = 0; q < 32; ++q) {
        if (q < warp) upto += total_of[q];
        all += total_of[q];
      }
      if (w < words) a.slots[w].y = uint32_t(first + upto - mine);
      first += all;
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) {
    // The factor of both gradients that does not depend on the row: grad_scale,
    // the mean's count, and the reduced loss's own gradient.
    double f = a.grad_scale;
    if (a.reduction == ZERO_REDUCE_MEAN) f /= double(max(1, N != kSlopes ? base : a.kind == kPreference ? a.head->pairs : targets));
    if (a.reduction != ZERO_REDUCE_NONE && a.dloss) f *= double(*a.dloss);
    f *= double(unit);
    if (N == kSlopes) {
      a.head->repack = targets != base;
      a.head->rows = base;
      a.head->factor = float(f);
    } else {
      *a.head = Head{base, 0, !ascend, float(f), 0, 0, 0};
    }
  }
}

// The weight's rows (where it is not read in place; this does not wait for the
// kernels before), and the rows with a target.
template <bool F32>
__global__ void __launch_bounds__(256) pack_kernel(const Args a, __nv_bfloat16* packed_weight, bool hidden_vector,
                                                   bool weight_vector, bool again) {
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
  if (!again || a.head->repack) pack_rows<F32>(a, a.head->rows, hidden_vector, first, step);
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
    if (a.rowpos[t] == -1) continue;
    if (a.kind != kPreference) a.loss[t] = NAN;
    if (a.row_logps) a.row_logps[t] = NAN;
    if (a.kind == kPolicy) a.slopes[t] = NAN;
    if (a.has_ce) a.lse[t] = NAN;
    if (a.has_kd) a.lse_tau[t] = NAN;
  }
  if (a.kind == kPreference) {
    for (int64_t i = first; i < a.pairs; i += step) a.loss[i] = NAN;
    for (int64_t i = first; i < 2 * a.pairs; i += step) a.logps[i] = a.slopes[i] = NAN;
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
    int32_t i = a.rowpos[t];
    if (a.few && i >= 0 && a.scales[t] == 0.0f) i = -2;  // without a slope; few rows are not numbered again
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
    if (!F32 && a.rests && i >= 0) {
      const float rest = ze::rest_of(a.scales[t], a.weights[t]);
      const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.weight) + a.ids[t] * a.weight_stride + d;
      x.x += rest * float(w[0]);
      if (d + 1 < a.D) x.y += rest * float(w[1]);
      if (d + 2 < a.D) x.z += rest * float(w[2]);
      if (d + 3 < a.D) x.w += rest * float(w[3]);
    }
    if (i >= 0 || (fault && i < -1)) x = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
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

// A row's maximum (in powers of two) and sum of exponentials; `Slopes`: and which
// partial has the maximum.
template <bool Slopes>
struct RowSum {
  float m = -INFINITY, s = 0.0f;
  int32_t best = 0;
};

// The same from the partial ones: each of the row's lanes takes every lanes-th, eight
// loads in flight; the first lane joins them. `Slopes`: by exponentials without a mean
// error, of maxima that are logits, in powers of two (mma) or as they are (few rows).
template <bool Slopes>
__device__ __forceinline__ RowSum<Slopes> row_sum(const float2* stats, bool few, int64_t count, int64_t Tp, int64_t i,
                                                  int lane, int lanes, RowSum<Slopes>* sh, int r, int rows) {
  const float unit = few ? kLog2e : 1.0f;
  const auto exp2_of = [&](float x) { return Slopes ? exp2_even(x * unit) : exp2f(x); };
  RowSum<Slopes> x;
  for (int64_t j0 = lane; j0 < count; j0 += 8 * lanes) {
    float2 p[8];
    float top = x.m;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      p[q] = j0 + lanes * q < count ? stats[(j0 + lanes * q) * Tp + i] : make_float2(-INFINITY, 0.0f);
      if (Slopes && !few) p[q].x = __fmul_rn(p[q].x, kLog2e);
      if (Slopes && p[q].x > top) x.best = int32_t(j0 + lanes * q);
      top = fmaxf(top, p[q].x);
    }
    if (top == -INFINITY) {
      // Nothing yet -- unless a partial is NaN (fmaxf passes it over).
#pragma unroll
      for (int q = 0; q < 8; ++q) x.s += p[q].y;
      continue;
    }
    x.s = x.m == -INFINITY ? x.s : x.s * exp2_of(x.m - top);
#pragma unroll
    for (int q = 0; q < 8; ++q) x.s += p[q].y * exp2_of(p[q].x - top);  // 0 where x is -inf
    x.m = top;
  }
  // A tree over the lanes, in a fixed order: between warps through shared memory,
  // then (row r's lanes are `rows` threads apart) within the first.
  const auto join = [&](const RowSum<Slopes>& x, const RowSum<Slopes>& y) {
    RowSum<Slopes> z;
    z.m = fmaxf(x.m, y.m);
    z.s = z.m == -INFINITY ? x.s + y.s : x.s * exp2_of(x.m - z.m) + y.s * exp2_of(y.m - z.m);
    if (Slopes) z.best = y.m > x.m ? y.best : x.best;
    return z;
  };
  int w = lanes / 2;
  if (w * rows >= 32) {
    sh[lane * rows + r] = x;
    __syncthreads();
    for (; w * rows >= 32; w >>= 1) {
      if (lane < w) sh[lane * rows + r] = join(sh[lane * rows + r], sh[(lane + w) * rows + r]);
      __syncthreads();
    }
    x = sh[lane * rows + r];
    __syncthreads();
  }
  for (; w; w >>= 1) {
    RowSum<Slopes> y;
    y.m = __shfl_down_sync(~0u, x.m, w * rows);
    y.s = __shfl_down_sync(~0u, x.s, w * rows);
    if (Slopes) y.best = __shfl_down_sync(~0u, x.best, w * rows);
    if (lane < w) x = join(x, y);
  }
  return x;
}

constexpr double kLn2 = 0.69314718055994530942;

// The log-sum-exp of a row's joined statistics.
__device__ __forceinline__ double lse_of(RowSum<false> x) { return (double(x.m) + log2(double(x.s))) * kLn2; }

// The products of N rows' hidden states t and one row y each of the weight in fp32, rounded
// at every addition: a warp's lanes take every 32nd group of elements, all rows'
// loads in flight together. Rows t below zero are left out.
template <bool F32, int N>
__device__ __forceinline__ void column_logits(const Args& a, const int64_t (&t)[N], const int32_t (&y)[N], bool vector,
                                             int lane, float (&logit)[N]) {
  using E = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int kWide = F32 ? 4 : 8;
  const E *h[N], *w[N];
  float sum[N][kWide] = {};
#pragma unroll
  for (int q = 0; q < N; ++q) {
    h[q] = static_cast<const E*>(a.hidden) + (t[q] < 0 ? 0 : t[q]) * a.hidden_stride;
    w[q] = static_cast<const E*>(a.weight) + (t[q] < 0 ? 0 : y[q]) * a.weight_stride;
  }
  const int64_t whole = vector ? a.D / kWide * kWide : 0;
#pragma unroll 2
  for (int64_t k = lane * kWide; k < whole; k += 32 * kWide) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if (t[q] < 0) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(h[q] + k), z = *reinterpret_cast<const uint4*>(w[q] + k);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (F32) {
          sum[q][j] = fmaf(__uint_as_float(xs[j]), __uint_as_float(zs[j]), sum[q][j]);
        } else {
          sum[q][2 * j % kWide] =
              fmaf(__uint_as_float(xs[j] << 16), __uint_as_float(zs[j] << 16), sum[q][2 * j % kWide]);
          sum[q][(2 * j + 1) % kWide] = fmaf(__uint_as_float(xs[j] & 0xffff0000u),
                                             __uint_as_float(zs[j] & 0xffff0000u), sum[q][(2 * j + 1) % kWide]);
        }
      }
    }
  }
  for (int64_t k = whole + lane; k < a.D; k += 32) {
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (t[q] >= 0) sum[q][0] = fmaf(float(h[q][k]), float(w[q][k]), sum[q][0]);
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
#pragma unroll
    for (int n = kWide / 2; n; n /= 2)
#pragma unroll
      for (int j = 0; j < n; ++j) sum[q][j] += sum[q][j + n];
    logit[q] = warp_sum(sum[q][0]);
  }
}

// log(1 + s 2^e).
__device__ __forceinline__ double log1p_of(double s, double e) {
  return e > 512.0 ? (e + log2(s)) * kLn2 : log1p(s * exp2(e));
}

// The policy loss of a row and its slope by the log-probability l. What is not a
// number stays none (maxima by comparison, not by fmax). An advantage of zero
// has no part in the loss, whatever the ratio. (The exponentials are fp32's, off
// by 2^-22 of themselves, less than l's own error makes them.)
struct PolicyRow {
  float advantage, old_logp, ref_logp, dloss;
};
__device__ __forceinline__ void policy_loss(const Args& a, const PolicyRow& row, float l, double* loss,
                                            double* slope) {
  *loss = *slope = 0.0;
  const double adv = double(row.advantage);
  if (adv != 0.0) {
    const double ratio = expf(float(double(l) - double(row.old_logp)));
    const double bounded = ratio < a.low ? a.low : ratio > a.high ? a.high : ratio;
    const double free = -adv * ratio, held = -adv * bounded;
    *loss = free < held ? held : free;
    *slope = free < held ? 0.0 : free;
  }
  if (a.kl_weight != 0.0) {
    const double d = double(row.ref_logp) - double(l), e = expm1f(float(d));
    *loss += a.kl_weight * (e - d);
    *slope -= a.kl_weight * e;
  }
}

constexpr int kSlopeRows = 16;  // most rows of a block of losses_kernel that goes by slopes

// What the matrix kernel does to a sum of exponentials. It takes logits times log2(e)
// in fp32: a maximum in powers of two is one of the logit by this factor. And ex2.approx
// cuts its results off, that is takes half a step of 2^-23 on average, relative to a
// value of [1, 2) whose logarithm is spread evenly 2^-24 / (2 ln 2) = 4.3e-8: from every
// term once, and again where a half tile's sum is rescaled, which of its four stretches
// of 32 columns the k-th finds 1/2 + ... + 1/4 of a time behind it: (1/2 + 2/3 + 3/4) / 4
// = 0.48 times a term. (The joins of the half tiles have no mean error.)
constexpr double kOfLogit = 1.0 / double(kLog2e);
constexpr double kCutOff = 1.48 * 4.3e-8;

// 256 threads: `block_rows` rows (a power of two, up to 32), 256 / block_rows lanes each.
//
// `Slopes` (the policy and the preference loss): a row's log-probability, of
// which those losses are functions, instead of a loss that is its negative. Such
// a loss hangs on small differences of log-probabilities, and a preference loss
// on sums of many, so what the tensor cores' truncating sums take from a large
// logit of the label counts (up to 8e-6 at a logit of 9 and width 768, always of
// one sign). The label's logit z is therefore taken in rounding fp32, and the
// statistics are those of the other columns: l = -log(1 + S e^-z), whose error is in
// proportion to what the model leaves to the others. (With the label's exponential in
// S, l and the label's p - 1 were off by S's last bits, up to 2e-7, however sure the
// model was.) Of the others the one with the largest logit is taken again likewise and
// corrected in S, most of which it is where the model expects it: 6000 rows of width
// 768 with a logit of 14 beside their label were 5.6e-6 too large on average, and are
// 8e-8 too small. (8192 rows of width 768: 31 us, 21 without that, bound by latency:
// twice two rows a warp, and between them the statistics' columns.)
template <bool Slopes, bool F32>
__global__ void __launch_bounds__(256, 4) losses_kernel(const Args a, int block_rows, bool vector) {
  __shared__ RowSum<Slopes> sh[256];
  __shared__ double part[256];
  constexpr int kLogits = kSlopeRows / 8;
  __shared__ float logit[kSlopeRows], largest[kSlopeRows];
  __shared__ int32_t column[kSlopeRows];
  __shared__ bool last;
  let_next_start();
  wait_for_previous();
  const int r = threadIdx.x % block_rows, lane = threadIdx.x / block_rows, lanes = 256 / block_rows;
  const int32_t rows = a.head->rows;
  double mine = 0.0;
  for (int64_t i0 = int64_t(blockIdx.x) * block_rows; i0 < rows; i0 += int64_t(gridDim.x) * block_rows) {
    const int64_t i = min(i0 + r, int64_t(rows) - 1);
    const int64_t t = a.rowmap[i];
    PolicyRow row{0.0f, 0.0f, 0.0f, 1.0f};  // read ahead of its use
    if (Slopes && a.kind == kPolicy && lane == 0) {
      row.advantage = a.advantages[t];
      row.old_logp = a.old_logps[t];
      if (a.kl_weight != 0.0) row.ref_logp = a.ref_logps[t];
      if (a.scales && a.reduction == ZERO_REDUCE_NONE && a.dloss) row.dloss = a.dloss[t];
    }
    // One logit of each row, of its label or its column: the block's warps take the rows
    // in turn, each up to kLogits.
    const auto logits = [&](bool label, float* to) {
      int64_t u[kLogits];
      int32_t y[kLogits];
      float z[kLogits];
#pragma unroll
      for (int n = 0; n < kLogits; ++n) {
        const int q = (threadIdx.x >> 5) + 8 * n;
        u[n] = q < block_rows && i0 + q < rows ? a.rowmap[i0 + q] : -1;
      }
#pragma unroll
      for (int n = 0; n < kLogits; ++n) y[n] = u[n] < 0 ? 0 : label ? a.ids[u[n]] : column[(threadIdx.x >> 5) + 8 * n];
      if (u[0] >= 0) column_logits<F32, kLogits>(a, u, y, vector, threadIdx.x & 31, z);
#pragma unroll
      for (int n = 0; n < kLogits; ++n)
        if ((threadIdx.x & 31) == 0 && u[n] >= 0) to[(threadIdx.x >> 5) + 8 * n] = z[n];
      __syncthreads();
    };
    if (Slopes) logits(true, logit);
    double entries = 0.0;
    if (!Slopes) {
#pragma unroll 4
      for (int e = lane; e < a.L; e += lanes) {
        const int64_t at = t * a.L + e;
        if (a.ids[at] != kNoId) entries += double(a.weights[at]) * double(a.zent[at]);
      }
    }
    RowSum<Slopes> sum;
    RowSum<false> sum_tau;
    if (a.has_ce) sum = row_sum<Slopes>(a.stats, a.few, a.partials, a.Tp, i, lane, lanes, sh, r, block_rows);
    if constexpr (!Slopes)
      if (a.has_kd) sum_tau = row_sum<false>(a.stats_tau, false, a.partials, a.Tp, i, lane, lanes, sh, r, block_rows);
    float seen = 0.0f;  // the largest logit, as the matrix kernel has it
    if (Slopes && !a.few) {
      if (lane == 0) {
        const int64_t at = sum.best * a.Tp + i;
        seen = a.stats[at].x;
        column[r] = int32_t(min(int64_t(sum.best) * (kTileN / 2) + a.places[at], a.V - 1));
      }
      __syncthreads();
      logits(false, largest);
    }
    if (!Slopes && a.L > 1) {
      part[threadIdx.x] = entries;
      __syncthreads();
      for (int w = lanes / 2; w; w >>= 1) {
        if (lane < w) part[threadIdx.x] += part[threadIdx.x + w * block_rows];
        __syncthreads();
      }
      entries = part[r];
    }
    const bool fault = a.head->fault;  // NaN in lse too: a backward call's gradients show it then
    if (Slopes && lane == 0 && i0 + r < rows) {
      const double z = logit[r], top = a.few ? double(sum.m) : double(sum.m) * kOfLogit;
      double others = sum.s, added = 0.0;
      if (!a.few) {
        const double off = double(largest[r]) - double(seen);  // small: e^off - 1 by two terms
        if (fabs(off) < 0.001) added = off + 0.5 * off * off;
        others = others * (1.0 + kCutOff) + added;
      }
      double more = log1p_of(others, (top - z) / kLn2), lse = z + more;
      if (!isfinite(z)) {
        lse = z < 0.0 ? top + log(others) : z;
        more = lse - z;
      }
      const double logp = fault ? NAN : -more;
      const float l = float(logp), gap = expm1f(l);
      // The backward pass forms the matrix kernel's logits again: their lse, without what
      // was added to the largest (with it, fp32 gradients of rows that expect another token
      // are 5e-6 off, as the largest probability is then).
      if (added != 0.0) lse += double(gap) * added / others;
      a.lse[t] = fault ? NAN : float(lse);
      a.row_logps[t] = l;
      if (a.scales) a.weights[t] = gap;
      if (a.kind == kPreference) {
        a.terms[t] = logp;
      } else {
        double loss, slope;
        policy_loss(a, row, l, &loss, &slope);
        a.loss[t] = fault ? NAN : float(loss);
        const float s = fault ? NAN : float(slope);
        a.slopes[t] = s;
        if (a.scales) a.scales[t] = -s * row.dloss;
        mine += double(fault ? NAN : float(loss));
      }
    } else if (!Slopes && lane == 0 && i0 + r < rows) {
      const float2 f = a.coef[t];
      double lse = 0.0, lse_tau = 0.0;
      if constexpr (!Slopes) {
        if (a.has_ce) lse = lse_of(sum);
        if (a.has_kd) lse_tau = lse_of(sum_tau);
      }
      double loss = double(a.konst[t]);
      if (f.x != 0.0f) loss += double(f.x) * lse;
      if (f.y != 0.0f) loss += double(f.y) * a.tau * lse_tau;
      loss -= entries;
      if (fault) loss = NAN;
      a.loss[t] = float(loss);
      if (a.has_ce) a.lse[t] = fault ? NAN : float(lse);
      if (a.has_kd) a.lse_tau[t] = fault ? NAN : float(lse_tau);
      mine += double(float(loss));
    }
    __syncthreads();
  }
  if (a.reduction == ZERO_REDUCE_NONE || a.kind == kPreference) return;
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

// ------------------------------------------------------------------- pairs --

// The sums over the block's 256 threads, in a fixed order, in all of them.
template <int N>
__device__ __forceinline__ void block_sums(double (&x)[N], double (*sh)[8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    for (int o = 16; o; o >>= 1) x[q] += __shfl_xor_sync(~0u, x[q], o);
    if (lane == 0) sh[q][warp] = x[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < N; ++q) {
    x[q] = sh[q][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) x[q] += sh[q][w];
  }
  __syncthreads();
}

// The loss of a pair and its slopes by each of its rows' log-probabilities, from
// the sequences' sums over n[k] labelled rows.
__device__ __forceinline__ void pair_loss(const Args& a, const double (&sum)[2], const int (&n)[2],
                                          const float (&ref)[2], double* loss, double (&slope)[2]) {
  double x[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) x[k] = (a.average ? sum[k] / max(1, n[k]) : sum[k]) - double(ref[k]);
  const double u = a.beta * (x[0] - x[1]) - a.margin;
  double du;
  if (a.squared) {
    *loss = u * u;
    du = 2.0 * u;
  } else {
    // log(1 + e^-u) and log(1 + e^u), and sigmoid(-u), from e^-|u|, in double: with
    // smoothing the slope is a difference
    const double e = exp(-fabs(u)), l = log1p(e), down = (u < 0.0 ? 1.0 : e) / (1.0 + e);
    *loss = (1.0 - a.smoothing) * ((u < 0.0 ? -u : 0.0) + l) + a.smoothing * ((u > 0.0 ? u : 0.0) + l);
    if (u != u) *loss = u;
    du = a.smoothing - down;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) slope[k] = (k ? -du : du) * a.beta / (a.average ? max(1, n[k]) : 1);
  if (a.nll_weight != 0.0 && n[0] > 0) {
    *loss -= a.nll_weight * sum[0] / n[0];
    slope[0] -= a.nll_weight / n[0];
  }
}

// A block for each pair (in turn). `Forward`: sums, losses and slopes, else the
// slopes are given; then the rows' scales where a backward pass follows. (16 pairs
// of 8192 rows: 13 us of dependent reads and double arithmetic.)
template <bool Forward>
__global__ void __launch_bounds__(256) pairs_kernel(const Args a) {
  __shared__ double sh[4][8];
  __shared__ float slopes[2];
  __shared__ bool last;
  let_next_start();
  wait_for_previous();
  const bool fault = a.head->fault;
  if (fault) {
    // The offsets may point anywhere: nothing is read by them.
    const int64_t first = int64_t(blockIdx.x) * 256 + threadIdx.x, step = int64_t(gridDim.x) * 256;
    if (a.scales)
      for (int64_t t = first; t < a.T; t += step)
        if (a.rowpos[t] >= 0) a.scales[t] = NAN;
    if (Forward) {
      for (int64_t t = first; t < a.T; t += step)
        if (a.rowpos[t] >= 0) a.lse[t] = a.row_logps[t] = NAN;
      for (int64_t i = first; i < a.pairs; i += step) a.loss[i] = NAN;
      for (int64_t i = first; i < 2 * a.pairs; i += step) {
        a.logps[i] = a.slopes[i] = NAN;
        a.seq_counts[i] = 0;
      }
      if (first == 0 && a.reduction != ZERO_REDUCE_NONE) *a.reduced = NAN;
    }
    return;
  }
  double mine = 0.0;
  const int64_t length = a.offsets || a.pairs == 0 ? 0 : a.T / (2 * a.pairs);
  for (int64_t i = blockIdx.x; i < a.pairs; i += gridDim.x) {
    int64_t begin[2], end[2];
    double x[4] = {};  // the sequences' labelled rows and their log-probabilities
    float ref[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t s = i + k * a.pairs;
      if (Forward && a.ref_logps && threadIdx.x == 0) ref[k] = a.ref_logps[s];  // ahead of its use
      begin[k] = a.offsets ? a.offsets[s] : s * length;
      end[k] = a.offsets ? a.offsets[s + 1] : (s + 1) * length;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll 4
      for (int64_t t = begin[k] + threadIdx.x; t < end[k]; t += 256) {
        const bool labelled = a.rowpos[t] >= 0;
        const double l = Forward ? a.terms[t] : 0.0;  // (of a row without a label: anything)
        x[k] += labelled ? 1.0 : 0.0;
        if (Forward) x[2 + k] += labelled ? l : 0.0;
      }
    }
    block_sums(x, sh);
    const int n[2] = {int(x[0]), int(x[1])};
    const double sum[2] = {x[2], x[3]};
    const bool some = n[0] + n[1] > 0;
    if (threadIdx.x == 0) {
      if (some) atomicAdd(&a.head->pairs, 1);
      double loss = 0.0, slope[2] = {};
      if (Forward) {
        if (some) pair_loss(a, sum, n, ref, &loss, slope);
        a.loss[i] = float(loss);
        mine += double(float(loss));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t s = i + k * a.pairs;
        if (Forward) {
          a.logps[s] = float(sum[k]);
          a.seq_counts[s] = n[k];
          a.slopes[s] = n[k] ? float(slope[k]) : 0.0f;
        }
        slopes[k] = n[k] ? (Forward ? float(slope[k]) : a.slopes[s]) : 0.0f;
      }
    }
    __syncthreads();
    if (a.scales && some) {
      const float d = a.reduction == ZERO_REDUCE_NONE && a.dloss ? a.dloss[i] : 1.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        for (int64_t t = begin[k] + threadIdx.x; t < end[k]; t += 256)
          if (a.rowpos[t] >= 0) {
            a.scales[t] = -slopes[k] * d;
            if (!Forward) a.weights[t] = expm1f(a.row_logps[t]);
          }
      // (sizes of floats are in the order of their bits)
      if (threadIdx.x < 2) atomicMax(&a.head->steepest, __float_as_uint(fabsf(slopes[threadIdx.x] * d)));
    }
    __syncthreads();
  }
  // The blocks' sums in order, by the last block to finish; and, where no rows are
  // numbered after this, the mean's part in the factor of both gradients.
  const bool reduce = Forward && a.reduction != ZERO_REDUCE_NONE;
  const bool factor = a.few && a.scales && a.reduction == ZERO_REDUCE_MEAN;
  if (!reduce && !factor) return;
  if (threadIdx.x == 0) {
    a.sums[blockIdx.x] = mine;
    __threadfence();
    last = atomicAdd(&a.head->ticket, 1) == int32_t(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const double pairs = double(max(1, __ldcg(&a.head->pairs)));
  if (factor && threadIdx.x == 0) a.head->factor = float(a.grad_scale / pairs * (a.dloss ? double(*a.dloss) : 1.0));
  if (!reduce) return;
  double sum[1] = {};
  for (int b = threadIdx.x; b < int(gridDim.x); b += 256) sum[0] += __ldcg(a.sums + b);
  block_sums(sum, sh);
  if (threadIdx.x == 0) *a.reduced = float(a.reduction == ZERO_REDUCE_MEAN ? sum[0] / pairs : sum[0]);
}

// The rows' scales and weights of a policy's backward call.
__global__ void __launch_bounds__(256) scales_kernel(const Args a) {
  let_next_start();
  wait_for_previous();
  const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t >= a.T || a.rowpos[t] < 0) return;
  a.scales[t] = -a.slopes[t] * (a.reduction == ZERO_REDUCE_NONE && a.dloss ? a.dloss[t] : 1.0f);
  a.weights[t] = expm1f(a.row_logps[t]);
}

// What G's rounding left of the labels' entries, times their rows of the hidden states,
// added up by label: a block for each row and 256 columns, which goes on if no earlier row
// has the row's label; its warps take a stretch of the rows each, whose sums are added
// in order. More rows are sorted by their labels and added up as the embedding's gradient
// is. (A step of GPT-2-small's head, this way and by sorting: 257 rows 178 and 194 us, 512
// 194 and 206, 1024 286 and 293, 2048 457 and 453; where all rows have one label 188 and
// 191, 204 and 204, 307 and 293, 494 and 458.)
template <bool Vector>
__global__ void __launch_bounds__(256) rests_kernel(const Args a, int64_t wide) {
  constexpr int kAhead = 4;
  __shared__ uint32_t same[kRestRows / 32];
  __shared__ float part[8][256];
  let_next_start();
  wait_for_previous();
  const int t = int(blockIdx.x / wide), T = int(a.T), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t d0 = blockIdx.x % wide * 256;
  if (a.rowpos[t] < 0) return;
  const int32_t y = a.ids[t];
  bool earlier = false;
  for (int j0 = 0; j0 < T; j0 += 256) {
    const int j = j0 + threadIdx.x;
    const bool has = j < T && a.ids[j] == y && a.rowpos[j] >= 0;
    earlier |= has && j < t;
    const unsigned mask = __ballot_sync(~0u, has);
    if (lane == 0 && j < T) same[j / 32] = mask;
  }
  if (__syncthreads_or(earlier)) return;
  const int64_t d = d0 + lane * 8;
  const int words = (T + 31) / 32, each = (words + 7) / 8, end = min(words, (warp + 1) * each);
  float sum[8] = {};
  for (int w = warp * each; w < end; ++w) {
    for (uint32_t left = same[w]; left;) {
      uint4 x[kAhead];
      float times[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        times[q] = 0.0f;
        if (!left) continue;
        const int64_t u = w * 32 + __ffs(left) - 1;
        left &= left - 1;
        times[q] = ze::rest_of(a.scales[u], a.weights[u]);
        const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.hidden) + u * a.hidden_stride + d;
        if (Vector && d + 8 <= a.D) {
          x[q] = *reinterpret_cast<const uint4*>(row);
        } else {
          uint32_t words[4] = {};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (d + j < a.D) words[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[j]) << (j % 2 * 16);
          x[q] = make_uint4(words[0], words[1], words[2], words[3]);
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (times[q] == 0.0f) continue;
        const uint32_t words[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sum[j] = fmaf(times[q], __uint_as_float(j % 2 ? words[j / 2] & 0xffff0000u : words[j / 2] << 16), sum[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  const int64_t column = d0 + threadIdx.x;
  if (column >= a.D) return;
  float all = part[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < 8; ++w) all += part[w][threadIdx.x];
  a.rest_rows[ze::slot_of(a.slots[y / 32], y % 32) * a.rest_stride + column] = __float2bfloat16_rn(all);
}

}  // namespace

namespace {

// A grid for `n` items of 256 threads, a few blocks a thread at most.
unsigned blocks_for(int64_t n) {
  const int64_t blocks = (n + 255) / 256;
  return unsigned(blocks < 1 ? 1 : blocks > kSms * 32 ? kSms * 32 : blocks);
}

}  // namespace

cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  // Up to as many rows as its block has threads, the numbering kernel prepares
  // them itself. A loss of a vocabulary of 1009 at width 96, replayed: 18.0 us
  // for one row, 18.1 with two kernels; 21.1 and 21.1 for 1024 rows; 21.3 and
  // 20.9 for 2048; 22.7 and 21.6 for 4096. A call that is waited for (one row,
  // GPT-2-small's head): 67 and 70 us. (Packing the rows there too: 33.4 us
  // instead of 31.2, replayed; 39.1 instead of 39.0 from the host.)
  if (a.K == 0 && a.T <= 1024) return launch(number_rows_kernel<kPrepare>, 1, 1024, 0, s, false, a);
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
  return e != cudaSuccess ? e : launch(number_rows_kernel<kTargets>, 1, 1024, 0, s, a.T > 0, a);
}

cudaError_t launch_pack(const Args& a, __nv_bfloat16* weight, bool again, cudaStream_t s) {
  const int es = a.planes == 3 ? 4 : 2;
  const bool hv = aligned16(a.hidden, a.hidden_stride * es), wv = aligned16(a.weight, a.weight_stride * es);
  const unsigned blocks = blocks_for((weight && a.V > a.Tp ? a.V : a.Tp) * a.Dp / 8);
  if (a.planes == 3) return launch(pack_kernel<true>, blocks, 256, 0, s, true, a, weight, hv, wv, again);
  return launch(pack_kernel<false>, blocks, 256, 0, s, true, a, weight, hv, wv, again);
}

cudaError_t launch_losses(const Args& a, cudaStream_t s) {
  // As many lanes to a row as leave a block for each SM (333 rows with two
  // softmaxes and 100 entries: a step of 197 us, 227 with 32 rows a block).
  const bool slopes = a.kind == kPolicy || a.kind == kPreference;
  int rows = slopes ? kSlopeRows : 32;
  while (rows > 1 && a.T / rows < kSms) rows /= 2;
  int64_t blocks = (a.T + rows - 1) / rows;
  blocks = blocks < 1 ? 1 : blocks < kLossBlocks ? blocks : kLossBlocks;
  const bool f32 = a.planes == 3;
  const bool vector = aligned16(a.hidden, a.hidden_stride * (f32 ? 4 : 2)) &&
                      aligned16(a.weight, a.weight_stride * (f32 ? 4 : 2));
  auto* kernel = !slopes ? losses_kernel<false, false> : f32 ? losses_kernel<true, true> : losses_kernel<true, false>;
  return launch(kernel, unsigned(blocks), 256, 0, s, true, a, rows, vector);
}

cudaError_t launch_pairs(const Args& a, cudaStream_t s) {
  const int64_t blocks = a.pairs < 1 ? 1 : a.pairs < kLossBlocks ? a.pairs : kLossBlocks;
  return launch(pairs_kernel<true>, unsigned(blocks), 256, 0, s, true, a);
}

cudaError_t launch_scales(const Args& a, cudaStream_t s) {
  if (a.kind == kPreference) {
    const int64_t blocks = a.pairs < 1 ? 1 : a.pairs < kLossBlocks ? a.pairs : kLossBlocks;
    return launch(pairs_kernel<false>, unsigned(blocks), 256, 0, s, true, a);
  }
  return launch(scales_kernel, unsigned(a.T > 0 ? (a.T + 255) / 256 : 1), 256, 0, s, true, a);
}

cudaError_t launch_sloped_rows(const Args& a, cudaStream_t s) {
  return launch(number_rows_kernel<kSlopes>, 1, 1024, 0, s, true, a);
}

cudaError_t launch_mark(const Args& a, cudaStream_t s) {
  return launch(mark_kernel, kSms, 256, 0, s, true, a);
}

cudaError_t launch_rests(const Args& a, cudaStream_t s) {
  const int64_t wide = (a.D + 255) / 256;
  auto* kernel = aligned16(a.hidden, a.hidden_stride * 2) ? rests_kernel<true> : rests_kernel<false>;
  return launch(kernel, unsigned(a.T * wide), 256, 0, s, true, a, wide);
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
