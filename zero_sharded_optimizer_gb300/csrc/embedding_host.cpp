// Host side of the embedding: argument checks, the workspace's layout and the
// order of the launches. Device work is in embedding_kernels.cu.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "embedding_internal.h"
#include "host_checks.h"

namespace {

using ze::Args;
using zl::Layout;
using zl::Span;
using zl::check_pointer;
using zl::elem_size;
using zl::overlap;
using zl::round_up;
using zl::set_error;

constexpr int64_t kMostSize = 0x7fffffff - 1024;  // T, V and D: 32-bit ids and positions

constexpr int64_t kZeroBytes = int64_t(64) << 20;

int check_sizes(const zero_embedding_t* p) {
  if (!p) return set_error(ZERO_EINVAL, "the problem is NULL");
  if (p->T < 0 || p->T > kMostSize) return set_error(ZERO_EINVAL, "T=%lld is out of range", (long long)p->T);
  if (p->V < 1 || p->V > kMostSize) return set_error(ZERO_EINVAL, "V=%lld is out of range", (long long)p->V);
  if (p->D < 1 || p->D > kMostSize) return set_error(ZERO_EINVAL, "D=%lld is out of range", (long long)p->D);
  if (p->precision != ZERO_FP32 && p->precision != ZERO_BF16_MIXED)
    return set_error(ZERO_EINVAL, "precision %d is neither ZERO_FP32 nor ZERO_BF16_MIXED", p->precision);
  if (!std::isfinite(p->scale) || !std::isfinite(float(p->scale)))
    return set_error(ZERO_EINVAL, "scale must be finite");
  return ZERO_OK;
}

int check_stride(int64_t stride, int64_t rows, int64_t D, const char* what) {
  if (stride < D)
    return set_error(ZERO_EINVAL, "%s=%lld is below D=%lld", what, (long long)stride, (long long)D);
  if (rows > 1 && stride > INT64_MAX / 8 / rows)
    return set_error(ZERO_EINVAL, "%s=%lld is out of range", what, (long long)stride);
  return ZERO_OK;
}

int check_spans(const Span* spans, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if ((spans[i].written || spans[j].written) && overlap(spans[i], spans[j]))
        return set_error(ZERO_EINVAL, "buffers overlap (%s and %s)", spans[j].what, spans[i].what);
  return ZERO_OK;
}

void common(const zero_embedding_t* p, const void* table, int64_t table_stride, void* out, int64_t out_stride,
            Args* a) {
  *a = Args{};
  a->T = p->T;
  a->V = p->V;
  a->D = p->D;
  a->f32 = p->precision == ZERO_FP32;
  a->ids = p->ids;
  a->padding_id = p->padding_id;
  a->scale = float(p->scale);
  a->table = table;
  a->table_stride = table_stride;
  a->out = out;
  a->out_stride = out_stride;
  a->width = ze::width_of(*a, elem_size(p->precision));
}

// The gradient's arrays in the workspace.
int plan(const zero_embedding_t* p, Args* a, int64_t* bytes) {
  common(p, p->dout, p->dout_stride, p->dweight, p->dweight_stride, a);
  a->accumulate = p->accumulate != 0;
  Layout w{static_cast<uint8_t*>(p->workspace)};
  ze::plan_sums(a, &w);
  // Zeros that the sort, which leaves memory idle, has the time to write: all rows
  // from zero_from on, whatever tokens there are. (131072 tokens of GPT-2-small's
  // table: 86.5 us with 64 MB of them, 93 with 1 MB or 88 with 128; few tokens, where
  // most rows stay zero: 8192 tokens 29 us with all, 41 with 32 MB.)
  const int64_t rows = a->few ? p->V : kZeroBytes / (p->D * elem_size(p->precision));
  a->zero_from = a->accumulate ? p->V : std::max<int64_t>(p->V - rows, 0);
  if (!w.fits) return set_error(ZERO_EINVAL, "the problem's workspace overflows 64 bits");
  *bytes = w.at;
  return ZERO_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ZERO_OK;
  return set_error(ZERO_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

}  // namespace

int32_t ze::width_of(const Args& a, int es) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.table) | uintptr_t(a.table_stride * es) |
                        reinterpret_cast<uintptr_t>(a.out) | uintptr_t(a.out_stride * es);
  return all % 16 == 0 ? 16 : all % 4 == 0 && a.D * es % 4 == 0 ? 4 : es;
}

void ze::plan_sums(Args* a, Layout* w) {
  a->few = a->T <= kFewTokens && (a->V <= kFewIds || a->T == 0);
  // A class's ids in a block's shared memory, and no more blocks than SMs if they fit.
  a->class_bits = a->V <= int64_t(kClassIds) << 7 ? 7 : kMostClassBits;
  // The fewest digits, of equal width, that hold the ids and V itself.
  int bits = 1;
  while (a->V >> bits) ++bits;
  a->passes = (bits + kMostBits - 1) / kMostBits;
  a->bits = (bits + a->passes - 1) / a->passes;
  const int64_t least = 1024;
  a->tile = std::max(least, round_up((a->T + kMostTiles - 1) / kMostTiles, 512));
  a->tiles = int32_t((a->T + a->tile - 1) / a->tile);
  const int64_t block = a->f32 ? 128 : 256;
  a->blocks = int32_t((a->D + block - 1) / block);
  a->Dp = a->blocks * block;
  // Long runs mean few shares of segments to be written, read and joined (131072
  // tokens of width 4096: 400 us, 448 with runs of 32), short ones work for all SMs.
  a->run = 128;
  while (a->run > 8 && (a->T + a->run - 1) / a->run * a->blocks < kSms * 32) a->run /= 2;
  a->runs = (a->T + a->run - 1) / a->run;
  a->counts = w->take<int32_t>(int64_t(a->passes) * a->tiles << a->bits);
  for (auto& l : a->list) l = w->take<Entry>(a->T);
  a->sorted = a->list[a->few ? 0 : (a->passes - 1) & 1];
  a->part = w->take<float>(2 * a->runs, a->Dp);
}

extern "C" {

int zero_embedding_workspace_bytes(const zero_embedding_t* p, int64_t* bytes) {
  if (!bytes) return set_error(ZERO_EINVAL, "bytes is NULL");
  if (int e = check_sizes(p)) return e;
  zero_embedding_t q = *p;
  q.workspace = nullptr;
  Args a;
  return plan(&q, &a, bytes);
}

int zero_embedding_forward(const zero_embedding_t* p, zero_stream_t stream) {
  if (int e = check_sizes(p)) return e;
  const int64_t T = p->T, V = p->V, D = p->D;
  const int es = elem_size(p->precision);
  int e;
  if ((e = check_stride(p->weight_stride, V, D, "weight_stride"))) return e;
  if ((e = check_stride(p->out_stride, T, D, "out_stride"))) return e;
  if ((e = check_pointer(p->ids, T, 8, "ids"))) return e;
  if ((e = check_pointer(p->weight, V, es, "weight"))) return e;
  if ((e = check_pointer(p->out, T, es, "out"))) return e;
  const Span spans[] = {{p->ids, 1, 8 * T, 8 * T, "ids", false},
                        {p->weight, V, D * es, p->weight_stride * es, "weight", false},
                        {p->out, T, D * es, p->out_stride * es, "out", true}};
  if ((e = check_spans(spans, 3))) return e;
  if (T == 0) return ZERO_OK;
  Args a;
  common(p, p->weight, p->weight_stride, p->out, p->out_stride, &a);
  return launched(ze::launch_lookup(a, stream), "the lookup");
}

int zero_embedding_backward(const zero_embedding_t* p, zero_stream_t stream) {
  if (int e = check_sizes(p)) return e;
  const int64_t T = p->T, V = p->V, D = p->D;
  const int es = elem_size(p->precision);
  int e;
  if ((e = check_stride(p->dout_stride, T, D, "dout_stride"))) return e;
  if ((e = check_stride(p->dweight_stride, V, D, "dweight_stride"))) return e;
  if ((e = check_pointer(p->ids, T, 8, "ids"))) return e;
  if ((e = check_pointer(p->dout, T, es, "dout"))) return e;
  if ((e = check_pointer(p->dweight, V, es, "dweight"))) return e;
  const Span spans[] = {{p->ids, 1, 8 * T, 8 * T, "ids", false},
                        {p->dout, T, D * es, p->dout_stride * es, "dout", false},
                        {p->dweight, V, D * es, p->dweight_stride * es, "dweight", true},
                        {p->workspace, 1, p->workspace_bytes, p->workspace_bytes, "workspace", true}};
  if ((e = check_spans(spans, 4))) return e;
  if (reinterpret_cast<uintptr_t>(p->workspace) % 256)
    return set_error(ZERO_EALIGN, "the workspace is not aligned to 256 bytes");
  Args a;
  int64_t bytes = 0;
  if ((e = plan(p, &a, &bytes))) return e;
  if (bytes && (!p->workspace || p->workspace_bytes < bytes))
    return set_error(ZERO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                     (long long)(p->workspace ? p->workspace_bytes : 0), (long long)bytes);
  if (T == 0 && a.accumulate) return ZERO_OK;
  if ((e = launched(ze::launch_sort(a, stream), "the sort"))) return e;
  return launched(ze::launch_sums(a, stream), "the sums");
}

}  // extern "C"
