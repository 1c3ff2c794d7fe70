// Host side of the vocabulary losses: argument checks, the workspace's layout
// the tensor maps and the order of the launches. Device work is in
// loss_kernels.cu and loss_mma.cu.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "loss_internal.h"

namespace {

using zl::Args;
using zl::Program;
using zl::set_error;

constexpr int64_t kMostSize = 0x7fffffff - 1024;  // T, V and D: 32-bit tile coordinates
// A piece of the logits' gradient is at most this many bytes (one tile's width
// of columns at least); kBuffers of them are held. More bytes mean fewer
// additions to dhidden's sums, fewer bytes a shorter pipeline: a step of 8192
// rows of width 768 took 1.92 ms with 16 MB, 1.57 with 32, 1.47 with 40 and 1.46
// with 128; one of 2048 rows 352, 354, 356 and 422 us.
constexpr int64_t kPieceBytes = int64_t(40) << 20;

// Up to this many rows of bf16 G is kept in two bf16 parts instead of one. With
// one, the gradients are 1.0 to 1.5 times as far from the exact ones as their own
// rounding makes them, and up to 2.6 times where a few rows hang on one value of
// G; with two it is 1.00 times. The second part costs 3 to 22 % of a step while
// a row tile's products wait for the weight anyway, but 21 to 33 % at 512 rows
// and 34 to 49 % at 1000 (widths 768 and 2048, vocabularies 50257 and 32000),
// where many rows' errors even out.
constexpr int64_t kFineRows = 256;

// A wait inside the matrix kernel gives up after this long; under normal running
// none is longer than a few tiles.
constexpr int64_t kWaitLimitNs = int64_t(10) * 1000 * 1000 * 1000;

// Failure injection for this thread's next call (zero_debug_withhold_head_loss).
struct Withheld {
  int32_t passes = 0;
  int64_t limit_ns = kWaitLimitNs;
};
thread_local Withheld g_withheld;

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

int elem_size(int32_t precision) { return precision == ZERO_FP32 ? 4 : 2; }

enum Pass { kForward = 1, kBackward = 2 };

// A buffer the call touches: `rows` rows of `bytes` bytes, `stride` bytes apart.
struct Span {
  const void* p;
  int64_t rows, bytes, stride;
  const char* what;
  bool written;
};

// Whether two buffers share a byte. Rows of equal stride are compared by their
// phase, so that column blocks of one wider buffer pass.
bool overlap(const Span& x, const Span& y) {
  if (!x.p || !y.p || !x.rows || !y.rows || !x.bytes || !y.bytes) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const uintptr_t a1 = a + uintptr_t((x.rows - 1) * x.stride + x.bytes);
  const uintptr_t b1 = b + uintptr_t((y.rows - 1) * y.stride + y.bytes);
  if (a1 <= b || b1 <= a) return false;
  if (x.stride == y.stride && x.rows > 1 && y.rows > 1) {
    const uintptr_t s = uintptr_t(x.stride);
    const uintptr_t d = b >= a ? (b - a) % s : (s - (a - b) % s) % s;
    if (d >= uintptr_t(x.bytes) && s - d >= uintptr_t(y.bytes)) return false;
  }
  return true;
}

int check_sizes(const zero_head_loss_t* p, bool distill) {
  if (!p) return set_error(ZERO_EINVAL, "the problem is NULL");
  if (p->T < 0 || p->T > kMostSize) return set_error(ZERO_EINVAL, "T=%lld is out of range", (long long)p->T);
  if (p->V < 1 || p->V > kMostSize) return set_error(ZERO_EINVAL, "V=%lld is out of range", (long long)p->V);
  if (p->D < 1 || p->D > kMostSize) return set_error(ZERO_EINVAL, "D=%lld is out of range", (long long)p->D);
  if (p->precision != ZERO_FP32 && p->precision != ZERO_BF16_MIXED)
    return set_error(ZERO_EINVAL, "precision %d is neither ZERO_FP32 nor ZERO_BF16_MIXED", p->precision);
  if (p->reduction != ZERO_REDUCE_NONE && p->reduction != ZERO_REDUCE_MEAN &&
      p->reduction != ZERO_REDUCE_SUM)
    return set_error(ZERO_EINVAL, "unknown reduction %d", p->reduction);
  const int64_t most = INT64_MAX / 8;
  struct { int64_t stride, rows; const char* what; bool used; } strides[] = {
      {p->hidden_stride, p->T, "hidden_stride", true},
      {p->weight_stride, p->V, "weight_stride", true},
      {p->dhidden_stride, p->T, "dhidden_stride", p->dhidden != nullptr},
      {p->dweight_stride, p->V, "dweight_stride", p->dweight != nullptr}};
  for (const auto& s : strides) {
    if (!s.used) continue;
    if (s.stride < p->D)
      return set_error(ZERO_EINVAL, "%s=%lld is below D=%lld", s.what, (long long)s.stride, (long long)p->D);
    if (s.rows > 1 && s.stride > most / s.rows)
      return set_error(ZERO_EINVAL, "%s=%lld is out of range", s.what, (long long)s.stride);
  }
  if (distill) {
    if (p->teacher_k < 1 || p->teacher_k > ZERO_DISTILL_MAX_K)
      return set_error(ZERO_EINVAL, "teacher_k=%lld is not in [1, %d]", (long long)p->teacher_k, ZERO_DISTILL_MAX_K);
    if (!std::isfinite(p->temperature) || !(p->temperature > 0.0) ||
        !std::isfinite(float(p->temperature)) || !(float(p->temperature) > 0.0f) ||
        !std::isfinite(float(1.0 / p->temperature)))
      return set_error(ZERO_EINVAL, "temperature must be finite and > 0");
    if (!(p->alpha >= 0.0 && p->alpha <= 1.0)) return set_error(ZERO_EINVAL, "alpha must lie in [0, 1]");
    if (!p->labels && p->alpha != 1.0 && p->T > 0)
      return set_error(ZERO_EINVAL, "without labels alpha must be 1");
  } else if (p->teacher_ids || p->teacher_logits || p->teacher_k || p->lse_tau) {
    return set_error(ZERO_EINVAL, "teacher fields are set: use the zero_distill calls");
  }
  return ZERO_OK;
}

int check_pointer(const void* ptr, int64_t count, size_t align, const char* what) {
  if (!ptr && count > 0) return set_error(ZERO_EINVAL, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(ptr) % align)
    return set_error(ZERO_EALIGN, "%s is not aligned to %zu bytes", what, align);
  return ZERO_OK;
}

int check_buffers(const zero_head_loss_t* p, bool distill, int pass) {
  const int es = elem_size(p->precision);
  const int64_t T = p->T, V = p->V, D = p->D;
  int e;
  if ((e = check_pointer(p->hidden, T, es, "hidden"))) return e;
  if ((e = check_pointer(p->weight, V, es, "weight"))) return e;
  if ((e = check_pointer(p->labels, distill ? 0 : T, 8, "labels"))) return e;
  const bool ce = !distill || p->labels;
  if (distill) {
    if ((e = check_pointer(p->teacher_ids, T, 8, "teacher_ids"))) return e;
    if ((e = check_pointer(p->teacher_logits, T, 4, "teacher_logits"))) return e;
    if ((e = check_pointer(p->lse_tau, T, 4, "lse_tau"))) return e;
  }
  if ((e = check_pointer(p->lse, ce ? T : 0, 4, "lse"))) return e;
  const bool reduce = p->reduction != ZERO_REDUCE_NONE;
  if (pass & kForward) {
    if ((e = check_pointer(p->loss, T, 4, "loss"))) return e;
    if (reduce && (e = check_pointer(p->reduced, 1, 4, "reduced"))) return e;
  }
  if (pass & kBackward) {
    if (!p->dhidden && !p->dweight && T > 0) return set_error(ZERO_EINVAL, "neither dhidden nor dweight is given");
    if ((e = check_pointer(p->dhidden, 0, es, "dhidden"))) return e;
    if ((e = check_pointer(p->dweight, 0, es, "dweight"))) return e;
    if ((e = check_pointer(p->dloss, 0, 4, "dloss"))) return e;
    if (!std::isfinite(p->grad_scale)) return set_error(ZERO_EINVAL, "grad_scale must be finite");
  }
  const bool fwd = pass & kForward, bwd = pass & kBackward;
  const Span spans[] = {
      {p->hidden, T, D * es, p->hidden_stride * es, "hidden", false},
      {p->weight, V, D * es, p->weight_stride * es, "weight", false},
      {p->labels, 1, 8 * T, 8 * T, "labels", false},
      {distill ? p->teacher_ids : nullptr, 1, 8 * T * p->teacher_k, 8 * T * p->teacher_k, "teacher_ids", false},
      {distill ? p->teacher_logits : nullptr, 1, 4 * T * p->teacher_k, 4 * T * p->teacher_k, "teacher_logits", false},
      {fwd ? p->loss : nullptr, 1, 4 * T, 4 * T, "loss", true},
      {ce ? p->lse : nullptr, 1, 4 * T, 4 * T, "lse", fwd},
      {distill ? p->lse_tau : nullptr, 1, 4 * T, 4 * T, "lse_tau", fwd},
      {fwd && reduce ? p->reduced : nullptr, 1, 4, 4, "reduced", true},
      {bwd ? p->dloss : nullptr, 1, reduce ? 4 : 4 * T, reduce ? 4 : 4 * T, "dloss", false},
      {bwd ? p->dhidden : nullptr, T, D * es, p->dhidden_stride * es, "dhidden", true},
      {bwd ? p->dweight : nullptr, V, D * es, p->dweight_stride * es, "dweight", true},
      {p->workspace, 1, p->workspace_bytes, p->workspace_bytes, "workspace", true}};
  const int n = int(sizeof(spans) / sizeof(spans[0]));
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if ((spans[i].written || spans[j].written) && overlap(spans[i], spans[j]))
        return set_error(ZERO_EINVAL, "buffers overlap (%s and %s)", spans[j].what, spans[i].what);
  return ZERO_OK;
}

// Places the call's arrays in the workspace (base NULL: only counts bytes).
// Returns false when the size overflows.
struct Layout {
  uint8_t* base;
  int64_t at = 0;
  bool fits = true;
  template <typename T>
  T* take(int64_t count, int64_t times = 1) {
    const int64_t size = int64_t(sizeof(T));
    if (!fits || (times && count > (INT64_MAX / 4) / times / size)) {
      fits = false;
      return nullptr;
    }
    T* p = reinterpret_cast<T*>(base + at);
    at = round_up(at + count * times * size, 256);
    if (at > INT64_MAX / 4) fits = false;
    return p;
  }
};

// The weight can be read in place by 16-byte copies of whole rows.
bool weight_in_place(const zero_head_loss_t* p) {
  return p->precision == ZERO_BF16_MIXED && reinterpret_cast<uintptr_t>(p->weight) % 16 == 0 &&
         p->weight_stride % 8 == 0 && p->weight_stride < (int64_t(1) << 39);
}

int plan(const zero_head_loss_t* p, bool distill, int pass, Args* a, __nv_bfloat16** packed_weight,
         int64_t* bytes) {
  *a = Args{};
  a->T = p->T;
  a->V = p->V;
  a->D = p->D;
  a->Tp = std::max<int64_t>(round_up(p->T, zl::kTileM), zl::kTileM);
  a->Dp = round_up(p->D, zl::kPadD);
  a->planes = p->precision == ZERO_FP32 ? 3 : 1;
  a->parts = a->planes == 3 ? 3 : p->T <= kFineRows ? 2 : 1;
  a->has_ce = p->labels != nullptr || !distill;
  a->has_kd = distill;
  a->K = distill ? int32_t(p->teacher_k) : 0;
  a->L = a->K + (a->has_ce ? 1 : 0);
  a->tau = distill ? p->temperature : 1.0;
  a->inv_tau = float(1.0 / a->tau);
  a->ce = distill ? float(1.0 - p->alpha) : 1.0f;
  a->kd = distill ? float(p->alpha * p->temperature) : 0.0f;
  a->reduction = p->reduction;
  a->ignore_index = p->ignore_index;
  a->grad_scale = p->grad_scale;
  a->accumulate = p->accumulate != 0;
  a->forward = (pass & kForward) != 0;
  a->hidden = p->hidden;
  a->hidden_stride = p->hidden_stride;
  a->weight = p->weight;
  a->weight_stride = p->weight_stride;
  a->labels = p->labels;
  a->teacher_ids = p->teacher_ids;
  a->teacher_logits = p->teacher_logits;
  a->loss = p->loss;
  a->lse = p->lse;
  a->lse_tau = p->lse_tau;
  a->reduced = p->reduced;
  a->dloss = p->dloss;
  a->dhidden = p->dhidden;
  a->dhidden_stride = p->dhidden_stride;
  a->dweight = p->dweight;
  a->dweight_stride = p->dweight_stride;
  a->tiles = (p->V + zl::kTileN - 1) / zl::kTileN;

  Layout w{static_cast<uint8_t*>(p->workspace)};
  a->head = w.take<zl::Head>(1);
  a->rowpos = w.take<int32_t>(a->T);
  a->rowmap = w.take<int32_t>(a->Tp);
  a->coef = w.take<float2>(a->T);
  a->konst = w.take<float>(a->T);
  a->ids = w.take<int32_t>(a->T, a->L);
  a->weights = w.take<float>(a->T, a->L);
  if (a->K) a->starts = w.take<uint16_t>(2 * a->tiles + 1, a->T);
  a->hp = w.take<__nv_bfloat16>(a->Tp * a->planes, a->Dp);
  if (weight_in_place(p)) {
    *packed_weight = nullptr;
    a->wp = static_cast<const __nv_bfloat16*>(p->weight);
    a->wp_ld = p->weight_stride;
    a->wp_plane = 0;
  } else {
    *packed_weight = w.take<__nv_bfloat16>(a->V * a->planes, a->Dp);
    a->wp = *packed_weight;
    a->wp_ld = a->Dp;
    a->wp_plane = a->V * a->Dp;
  }
  int64_t pieces = 0;
  if (pass & kBackward) {
    const int64_t widest = std::max<int64_t>(
        kPieceBytes / (2 * a->parts * a->Tp) / zl::kTileN * zl::kTileN, zl::kTileN);
    pieces = (a->V + widest - 1) / widest;
    a->piece = round_up((a->V + pieces - 1) / pieces, zl::kTileN);
    pieces = (a->V + a->piece - 1) / a->piece;
  }
  if (pass & kBackward) {
    // dhidden's sums over a piece are split where one of its tiles would be
    // more than half of what each CTA pair of the card has to do for the piece, while
    // two blocks of K are left to a part (37 rows x 1009 x 96 in fp32: a step of
    // 68 us, 87 unsplit; 333 x 10007 x 512: 197 and 419; twice the parts on 1638
    // rows x 32000 x 2048: 543 instead of 534).
    const int64_t blocks_t = (a->T + 63) / 64, blocks_v = a->piece / 64, blocks_d = a->Dp / 64;
    const int64_t wide = (a->D + zl::kTileN - 1) / zl::kTileN;
    const int64_t rows = a->Tp / zl::kTileM, cols = a->piece / zl::kTileN;
    const int64_t terms = a->planes == 1 ? a->parts : 1;  // of a product with G, to one of the logits
    const int64_t work = terms * (rows * wide * blocks_v + (p->dweight ? cols * wide * blocks_t : 0)) +
                         (pieces > 1 ? rows * cols * blocks_d : 0);
    a->splits = 1;
    while (a->splits < 64 && terms * blocks_v / a->splits > std::max<int64_t>(work / zl::kSms, 2 * terms)) a->splits *= 2;
  }
  // The words that begin as zero.
  const int64_t tiles = pass & kBackward ? a->splits * (a->Tp / zl::kTileM) * ((a->D + 255) / 256) : 0;
  a->zeros = 3 + 2 * pieces + tiles;
  a->counters = w.take<int32_t>(a->zeros);
  a->never = reinterpret_cast<uint32_t*>(a->counters + 2);
  a->formed = a->never + 1;
  a->used = a->formed + pieces;
  a->added = a->used + pieces;
  // The forward pass's arrays and the backward pass's lie over one another.
  const int64_t common = w.at;
  a->sums = w.take<double>(zl::kLossBlocks);
  a->zent = w.take<float>(a->T, a->L);
  if (a->has_ce) a->stats = w.take<float2>(2 * a->tiles, a->Tp);
  if (a->has_kd) a->stats_tau = w.take<float2>(2 * a->tiles, a->Tp);
  int64_t most = w.at;
  if (pass & kBackward) {
    w.at = common;
    for (int b = 0; b < zl::kBuffers; ++b)
      a->g[b] = b < pieces ? w.take<__nv_bfloat16>(a->Tp * a->parts, a->piece) : a->g[0];
    if (p->dhidden) a->dh = w.take<float>(a->splits * a->Tp, a->Dp);
    most = std::max(most, w.at);
  }
  // The matrix kernel numbers its tiles in 32 bits.
  const double row_tiles = double(a->Tp / zl::kTileM), wide_tiles = double((a->D + 255) / 256);
  if (row_tiles * double(a->tiles) > 1e9 ||
      (pass & kBackward && (row_tiles + wide_tiles) * double((a->V + 255) / 256) +
                                   double(pieces) * row_tiles * wide_tiles * double(a->splits) > 1e9))
    return set_error(ZERO_EINVAL, "the problem has more than 1e9 tiles");
  if (!w.fits) return set_error(ZERO_EINVAL, "the problem's workspace overflows 64 bits");
  *bytes = most;
  return ZERO_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link the driver).
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// An array [planes][rows][cols] as boxes of 128 bytes of columns by `box_rows`
// rows, in shared memory with the 128-byte swizzle; elements outside it read
// as zero and are not written.
bool tensor_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld, int64_t planes,
                int64_t plane, uint32_t box_rows, bool fp32 = false) {
  const int es = fp32 ? 4 : 2;
  const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(ld) * es, cuuint64_t(planes > 1 ? plane : ld) * es};
  const cuuint32_t box[3] = {cuuint32_t(128 / es), box_rows, 1}, unit[3] = {1, 1, 1};
  return encoder()(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_program(const Args& a, bool backward, Program* p) {
  const bool f32 = a.planes == 3;
  const int64_t wide = a.wp_plane ? a.Dp : a.D;
  bool ok = tensor_map(&p->hidden, a.hp, a.Dp, a.Tp, a.Dp, a.planes, a.Tp * a.Dp, 128) &&
            tensor_map(&p->weight, a.wp, wide, a.V, a.wp_ld, a.planes, a.wp_plane, 128);
  if (!backward) return ok;
  ok = ok && tensor_map(&p->hidden_mn, a.hp, a.Dp, a.Tp, a.Dp, a.planes, a.Tp * a.Dp, 64) &&
       tensor_map(&p->weight_mn, a.wp, wide, a.V, a.wp_ld, a.planes, a.wp_plane, 64);
  for (int b = 0; b < zl::kBuffers; ++b) {
    CUtensorMap* const to[3] = {&p->g[b], &p->g_mn[b], &p->g_out[b]};
    const uint32_t box[3] = {128, 64, 32};
    for (int i = 0; i < 3; ++i)
      ok = ok && tensor_map(to[i], a.g[b], a.piece, a.Tp, a.piece, a.parts, a.Tp * a.piece, box[i]);
  }
  if (a.dhidden) ok = ok && tensor_map(&p->dh, a.dh, a.Dp, a.Tp, a.Dp, a.splits, a.Tp * a.Dp, 32, true);
  const int es = f32 ? 4 : 2;
  // TMA writes whole 16-byte units: a row that ends inside one is left to the threads.
  p->weight_tma = a.dweight && a.D * es % 16 == 0 && reinterpret_cast<uintptr_t>(a.dweight) % 16 == 0 && a.dweight_stride * es % 16 == 0 &&
                  a.dweight_stride < (int64_t(1) << 37) && (f32 || !a.accumulate);
  if (p->weight_tma) ok = ok && tensor_map(&p->dweight, a.dweight, a.D, a.V, a.dweight_stride, 1, 0, 32, f32);
  p->pieces = int32_t((a.V + a.piece - 1) / a.piece);
  return ok;
}

int workspace_bytes(const zero_head_loss_t* p, bool distill, int64_t* bytes) {
  if (!bytes) return set_error(ZERO_EINVAL, "bytes is NULL");
  if (int e = check_sizes(p, distill)) return e;
  Args a;
  __nv_bfloat16* packed;
  zero_head_loss_t q = *p;
  q.workspace = nullptr;
  return plan(&q, distill, kForward | (p->dhidden || p->dweight ? kBackward : 0), &a, &packed, bytes);
}

int run(const zero_head_loss_t* p, bool distill, int pass, cudaStream_t s) {
  if (int e = check_sizes(p, distill)) return e;
  if (int e = check_buffers(p, distill, pass)) return e;
  if (!p->dhidden && !p->dweight) pass &= ~kBackward;  // without rows: an empty dhidden, if any
  if (!pass) return ZERO_OK;
  if (reinterpret_cast<uintptr_t>(p->workspace) % 256)
    return set_error(ZERO_EALIGN, "the workspace is not aligned to 256 bytes");
  Args a;
  __nv_bfloat16* packed;
  int64_t bytes = 0;
  if (int e = plan(p, distill, pass, &a, &packed, &bytes)) return e;
  if (!p->workspace || p->workspace_bytes < bytes)
    return set_error(ZERO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                     (long long)(p->workspace ? p->workspace_bytes : 0), (long long)bytes);
  if (!encoder()) return set_error(ZERO_ECUDA, "the CUDA driver has no cuTensorMapEncodeTiled");
  Program program{};
  if (!make_program(a, pass & kBackward, &program))
    return set_error(ZERO_EINVAL, "the problem's arrays are too large for tensor maps");
  int device = 0, sms = 0;
  cudaError_t q = cudaGetDevice(&device);
  if (q == cudaSuccess) q = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (q != cudaSuccess)
    return set_error(ZERO_ECUDA, "device: %s (%s)", cudaGetErrorString(q), cudaGetErrorName(q));
  const Withheld withheld = g_withheld;
  g_withheld = Withheld{};
  program.wait_limit_ns = uint64_t(withheld.limit_ns);
  const char* what = "rows";
  cudaError_t e = zl::launch_rows(a, s);
  auto next = [&](const char* name, auto&& launch) {
    if (e != cudaSuccess) return;
    what = name;
    e = launch();
  };
  next("packing", [&] { return zl::launch_pack(a, packed, s); });
  if (pass & kForward) {
    program.forward = 1;
    program.counter = a.counters;
    program.withheld = withheld.passes & kForward ? a.never : nullptr;
    next("logits", [&] { return zl::launch_products(a, program, device, sms, s); });
    next("losses", [&] { return zl::launch_losses(a, s); });
  }
  if (pass & kBackward) {
    program.forward = 0;
    program.counter = a.counters + 1;
    program.withheld = withheld.passes & kBackward ? a.never : nullptr;
    next("the gradients", [&] { return zl::launch_products(a, program, device, sms, s); });
    if (p->dhidden && p->T) next("dhidden", [&] { return zl::launch_dhidden_out(a, s); });
    else next("the mark", [&] { return zl::launch_mark(a, s); });
  }
  if (e != cudaSuccess)
    return set_error(ZERO_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
  return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_xent_workspace_bytes(const zero_head_loss_t* p, int64_t* bytes) {
  return workspace_bytes(p, false, bytes);
}
int zero_distill_workspace_bytes(const zero_head_loss_t* p, int64_t* bytes) {
  return workspace_bytes(p, true, bytes);
}
int zero_xent_forward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, false, kForward, stream);
}
int zero_xent_backward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, false, kBackward, stream);
}
int zero_xent_step(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, false, kForward | kBackward, stream);
}
int zero_distill_forward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, true, kForward, stream);
}
int zero_distill_backward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, true, kBackward, stream);
}
int zero_distill_step(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(p, true, kForward | kBackward, stream);
}
int zero_debug_withhold_head_loss(int32_t passes, int64_t limit_ns) {
  if (passes < 0 || passes > 3) return set_error(ZERO_EINVAL, "passes=%d is not in [0, 3]", passes);
  if (limit_ns < 1 || limit_ns > kWaitLimitNs)
    return set_error(ZERO_EINVAL, "limit_ns=%lld is not in [1, %lld]", (long long)limit_ns, (long long)kWaitLimitNs);
  g_withheld = Withheld{passes, limit_ns};
  return ZERO_OK;
}

}  // extern "C"
