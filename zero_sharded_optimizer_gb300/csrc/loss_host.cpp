// Host side of the vocabulary losses: argument checks, the workspace's layout
// the tensor maps and the order of the launches. Device work is in
// loss_kernels.cu and loss_mma.cu.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "embedding_internal.h"
#include "host_checks.h"
#include "loss_internal.h"

namespace {

using zl::Args;
using zl::Layout;
using zl::Program;
using zl::Span;
using zl::check_pointer;
using zl::elem_size;
using zl::overlap;
using zl::round_up;
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
// where many rows' errors even out. (The policy and the preference loss get back what
// one part loses where it counts: see `rests` below.)
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

enum Pass { kForward = 1, kBackward = 2 };

// A call's problem: the common part, and what its loss has besides.
struct Problem {
  const zero_head_loss_t* p;
  zl::Kind kind;
  const zero_policy_t* policy = nullptr;
  const zero_preference_t* preference = nullptr;

  bool distill() const { return kind == zl::kDistill; }
  bool slopes() const { return policy || preference; }
  int64_t losses() const { return preference ? preference->pairs : p->T; }  // that `loss` and `dloss` have
};

int check_options(const zero_policy_t* q) {
  if (!std::isfinite(q->clip_low) || q->clip_low < 0.0 || !std::isfinite(q->clip_high) || q->clip_high < 0.0)
    return set_error(ZERO_EINVAL, "clip_low and clip_high must be finite and at least 0");
  if (!std::isfinite(q->kl_weight)) return set_error(ZERO_EINVAL, "kl_weight must be finite");
  return ZERO_OK;
}

int check_options(const zero_preference_t* q, int64_t T) {
  if (q->pairs < 0 || q->pairs > kMostSize / 2)
    return set_error(ZERO_EINVAL, "pairs=%lld is out of range", (long long)q->pairs);
  if (!q->offsets && (q->pairs ? T % (2 * q->pairs) : T) != 0)
    return set_error(ZERO_EINVAL, "T=%lld rows are not 2 * %lld sequences of equal length", (long long)T,
                     (long long)q->pairs);
  if (q->kind != ZERO_PREFERENCE_SIGMOID && q->kind != ZERO_PREFERENCE_SQUARED)
    return set_error(ZERO_EINVAL, "unknown kind %d of preference loss", q->kind);
  if (!std::isfinite(q->beta)) return set_error(ZERO_EINVAL, "beta must be finite");
  if (!(q->smoothing >= 0.0 && q->smoothing <= 1.0))
    return set_error(ZERO_EINVAL, "smoothing must lie in [0, 1]");
  if (q->kind != ZERO_PREFERENCE_SIGMOID && q->smoothing != 0.0)
    return set_error(ZERO_EINVAL, "smoothing is the sigmoid loss's");
  if (!std::isfinite(q->margin)) return set_error(ZERO_EINVAL, "margin must be finite");
  if (!std::isfinite(q->nll_weight)) return set_error(ZERO_EINVAL, "nll_weight must be finite");
  return ZERO_OK;
}

int check_sizes(const Problem& problem) {
  const zero_head_loss_t* p = problem.p;
  const bool distill = problem.distill();
  if (problem.kind == zl::kPolicy && !problem.policy) return set_error(ZERO_EINVAL, "the policy's part is NULL");
  if (problem.kind == zl::kPreference && !problem.preference)
    return set_error(ZERO_EINVAL, "the preference's part is NULL");
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
  if (problem.policy) return check_options(problem.policy);
  if (problem.preference) return check_options(problem.preference, p->T);
  return ZERO_OK;
}

int check_buffers(const Problem& problem, int pass) {
  const zero_head_loss_t* p = problem.p;
  const bool distill = problem.distill();
  const int es = elem_size(p->precision);
  const int64_t T = p->T, V = p->V, D = p->D, losses = problem.losses();
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
  const bool fwd = pass & kForward, bwd = pass & kBackward;
  if (fwd) {
    if ((e = check_pointer(p->loss, losses, 4, "loss"))) return e;
    if (reduce && (e = check_pointer(p->reduced, 1, 4, "reduced"))) return e;
  }
  if (bwd) {
    if (!p->dhidden && !p->dweight && T > 0) return set_error(ZERO_EINVAL, "neither dhidden nor dweight is given");
    if ((e = check_pointer(p->dhidden, 0, es, "dhidden"))) return e;
    if ((e = check_pointer(p->dweight, 0, es, "dweight"))) return e;
    if ((e = check_pointer(p->dloss, 0, 4, "dloss"))) return e;
    if (!std::isfinite(p->grad_scale)) return set_error(ZERO_EINVAL, "grad_scale must be finite");
  }
  // What the policy and the preference loss have besides: nothing, an entry for
  // each row, or for each sequence.
  const zero_policy_t* po = problem.policy;
  const zero_preference_t* pr = problem.preference;
  const int64_t each = po ? T : pr ? 2 * pr->pairs : 0;
  const float* ref = !fwd ? nullptr : po ? (po->kl_weight != 0.0 ? po->ref_logps : nullptr) : pr ? pr->ref_logps : nullptr;
  float* const slopes = po ? po->slopes : pr ? pr->slopes : nullptr;
  float* const rows = po ? po->logps : pr ? pr->row_logps : nullptr;  // [T], written and read as lse is
  float* const logps = fwd && pr ? pr->logps : nullptr;
  if ((e = check_pointer(slopes, each, 4, "slopes"))) return e;
  if ((e = check_pointer(rows, po || pr ? T : 0, 4, po ? "logps" : "row_logps"))) return e;
  if (fwd && pr && (e = check_pointer(logps, each, 4, "logps"))) return e;
  if ((e = check_pointer(ref, fwd && po && po->kl_weight != 0.0 ? T : 0, 4, "ref_logps"))) return e;
  if (fwd && po) {
    if ((e = check_pointer(po->old_logps, T, 4, "old_logps"))) return e;
    if ((e = check_pointer(po->advantages, T, 4, "advantages"))) return e;
  }
  if (pr) {
    if ((e = check_pointer(pr->offsets, 0, 8, "offsets"))) return e;
    if (fwd && (e = check_pointer(pr->counts, each, 4, "counts"))) return e;
  }
  const int64_t offsets = pr ? 8 * (each + 1) : 0;
  const Span spans[] = {
      {p->hidden, T, D * es, p->hidden_stride * es, "hidden", false},
      {p->weight, V, D * es, p->weight_stride * es, "weight", false},
      {p->labels, 1, 8 * T, 8 * T, "labels", false},
      {distill ? p->teacher_ids : nullptr, 1, 8 * T * p->teacher_k, 8 * T * p->teacher_k, "teacher_ids", false},
      {distill ? p->teacher_logits : nullptr, 1, 4 * T * p->teacher_k, 4 * T * p->teacher_k, "teacher_logits", false},
      {fwd ? p->loss : nullptr, 1, 4 * losses, 4 * losses, "loss", true},
      {ce ? p->lse : nullptr, 1, 4 * T, 4 * T, "lse", fwd},
      {distill ? p->lse_tau : nullptr, 1, 4 * T, 4 * T, "lse_tau", fwd},
      {fwd && reduce ? p->reduced : nullptr, 1, 4, 4, "reduced", true},
      {bwd ? p->dloss : nullptr, 1, reduce ? 4 : 4 * losses, reduce ? 4 : 4 * losses, "dloss", false},
      {bwd ? p->dhidden : nullptr, T, D * es, p->dhidden_stride * es, "dhidden", true},
      {bwd ? p->dweight : nullptr, V, D * es, p->dweight_stride * es, "dweight", true},
      {fwd && po ? po->old_logps : nullptr, 1, 4 * T, 4 * T, "old_logps", false},
      {fwd && po ? po->advantages : nullptr, 1, 4 * T, 4 * T, "advantages", false},
      {ref, 1, 4 * each, 4 * each, "ref_logps", false},
      {pr ? pr->offsets : nullptr, 1, offsets, offsets, "offsets", false},
      {rows, 1, 4 * T, 4 * T, po ? "logps" : "row_logps", fwd},
      {logps, 1, 4 * each, 4 * each, "logps", true},
      {slopes, 1, 4 * each, 4 * each, "slopes", fwd},
      {fwd && pr ? pr->counts : nullptr, 1, 4 * each, 4 * each, "counts", true},
      {p->workspace, 1, p->workspace_bytes, p->workspace_bytes, "workspace", true}};
  const int n = int(sizeof(spans) / sizeof(spans[0]));
  for (int i = 0; i < n; ++i) {
    if (!spans[i].p) continue;
    for (int j = 0; j < i; ++j)
      if ((spans[i].written || spans[j].written) && overlap(spans[i], spans[j]))
        return set_error(ZERO_EINVAL, "buffers overlap (%s and %s)", spans[j].what, spans[i].what);
  }
  return ZERO_OK;
}

// The weight can be read in place by 16-byte copies of whole rows.
bool weight_in_place(const zero_head_loss_t* p) {
  return p->precision == ZERO_BF16_MIXED && reinterpret_cast<uintptr_t>(p->weight) % 16 == 0 &&
         p->weight_stride % 8 == 0 && p->weight_stride < (int64_t(1) << 39);
}

// Whether a call's products are better made without the tensor cores (loss_few.cu):
// for a few rows, whose work is the weight's traffic, and some more where they are
// small with the weight and latency is all. GPU time of a policy's step in a replayed
// graph, here and on the tensor cores, us (V x D):
//   rows            1          4          8          16         32         64
//   bf16 1009 x 96       29, 55     31, 56     35, 57     39, 57     47, 57
//   bf16 8000 x 512      41, 70     43, 71     48, 71     53, 72     68, 71
//   bf16 50257 x 64      57, 83     62, 84     72, 84     109, 84    174, 83
//   bf16 50257 x 256     53, 99     58, 100    68, 100    91, 101    140, 100
//   bf16 50257 x 768     96, 144    104, 144   131, 144   198, 145   332, 142
//   bf16 32000 x 2048    134, 203   141, 202   187, 201   298, 201   533, 201
//   bf16 131072 x 64     90, 141    99, 141    122, 142   216, 142   389, 140
//   bf16 131072 x 4096   691, 986   770, 982   1069, 983
//   fp32 1009 x 96       30, 62                32, 63     33, 63     39, 63     47, 64
//   fp32 8000 x 512      41, 100               47, 100    57, 103    78, 100    117, 106
//   fp32 50257 x 64      51, 122               59, 122    80, 122    123, 121   211, 121
//   fp32 50257 x 256     78, 165               92, 166    125, 166   186, 166   313, 165
//   fp32 50257 x 768     137, 375              160, 373   251, 375   422, 374   786, 377
//   fp32 131072 x 64     76, 204               92, 206    153, 205   271, 203   505, 204
//   fp32 131072 x 4096   1204, 3789            1618, 3791
// and with the weight's rows off 16 bytes, which are read element by element here:
//   bf16 1009 x 97       31, 60     33, 61     37, 62     43, 62     55, 62
//   bf16 8000 x 513      60, 88     65, 89     72, 89     92, 89     134, 89
//   bf16 50257 x 769     261, 224   265, 222   290, 222   499, 223   810, 223
//   fp32 8000 x 513      49, 113               57, 114    76, 114    115, 115   184, 116
//   fp32 50257 x 769     256, 444              284, 444   518, 443   907, 442   1722, 444
// A warp takes 256 columns of bf16 or 128 of fp32 at a time and a block eight rows,
// whatever there is of them, so that is what the work is counted in. (A call that is issued
// by the host takes 47 us here and 63 on the tensor cores.)
bool few_rows(const zero_head_loss_t* p) {
  const bool f32 = p->precision == ZERO_FP32;
  const int es = f32 ? 4 : 2;
  const int64_t wide = round_up(p->D, f32 ? 128 : 256);
  if (p->T < 1 || wide * es > zl::kFewHiddenBytes / zl::kFewGroup) return false;  // (a group's hidden states)
  const bool aligned = reinterpret_cast<uintptr_t>(p->weight) % 16 == 0 && p->weight_stride * es % 16 == 0;
  const double weight = double(p->V) * double(wide);
  const int64_t most = f32 ? (aligned ? 16 : 8) : !aligned ? 0 : weight <= 1e8 ? 8 : 4;
  return p->T <= most ||
         (p->T <= (f32 ? 64 : 32) && double(round_up(p->T, zl::kFewGroup)) * weight <= (aligned ? 1.5e8 : 1e8));
}

// The sums of the rests: the embedding's gradient of the labels, whose rows are the hidden
// states, each as many times as its rest is.
ze::Args rests_of(const Args& a, Layout* w) {
  ze::Args r{};
  r.T = a.T;
  r.V = a.V;
  r.D = a.D;
  r.ids = a.labels;
  r.padding_id = a.ignore_index;
  r.scale = 1.0f;
  r.table = a.hidden;
  r.table_stride = a.hidden_stride;
  r.out = a.rest_rows;
  r.out_stride = a.rest_stride;
  r.width = ze::width_of(r, 2);
  r.zero_from = a.V;  // none
  r.scales = a.scales;
  r.weights = a.weights;
  r.slots = a.slots;
  ze::plan_sums(&r, w);
  return r;
}

int plan(const Problem& problem, int pass, Args* a, __nv_bfloat16** packed_weight, ze::Args* rests, int64_t* bytes) {
  const zero_head_loss_t* p = problem.p;
  const bool distill = problem.distill();
  *a = Args{};
  a->kind = problem.kind;
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
  a->row_scale = p->reduction == ZERO_REDUCE_NONE ? p->dloss : nullptr;
  if (const zero_policy_t* q = problem.policy) {
    a->old_logps = q->old_logps;
    a->advantages = q->advantages;
    a->ref_logps = q->ref_logps;
    a->low = 1.0 - q->clip_low;
    a->high = 1.0 + q->clip_high;
    a->kl_weight = q->kl_weight;
    a->logps = a->row_logps = q->logps;
    a->slopes = q->slopes;
  }
  if (const zero_preference_t* q = problem.preference) {
    a->pairs = q->pairs;
    a->offsets = q->offsets;
    a->ref_logps = q->ref_logps;
    a->squared = q->kind == ZERO_PREFERENCE_SQUARED;
    a->average = q->average != 0;
    a->beta = q->beta;
    a->smoothing = q->smoothing;
    a->margin = q->margin;
    a->nll_weight = q->nll_weight;
    a->logps = q->logps;
    a->row_logps = q->row_logps;
    a->slopes = q->slopes;
    a->seq_counts = q->counts;
  }
  a->dhidden = p->dhidden;
  a->dhidden_stride = p->dhidden_stride;
  a->dweight = p->dweight;
  a->dweight_stride = p->dweight_stride;
  a->tiles = (p->V + zl::kTileN - 1) / zl::kTileN;
  a->partials = 2 * a->tiles;
  a->few = problem.slopes() && few_rows(p);
  const int64_t groups = (p->T + zl::kFewGroup - 1) / zl::kFewGroup;
  if (a->few) {
    // Blocks that go through the vocabulary, each with its own share of the statistics.
    a->Tp = std::max<int64_t>(groups, 1) * zl::kFewGroup;
    a->partials = std::max<int64_t>(std::min<int64_t>(2 * zl::kSms / std::max<int64_t>(groups, 1), (p->V + 31) / 32), 1);
  }

  Layout w{static_cast<uint8_t*>(p->workspace)};
  a->head = w.take<zl::Head>(1);
  a->rowpos = w.take<int32_t>(a->T);
  a->rowmap = w.take<int32_t>(a->Tp);
  a->coef = w.take<float2>(a->T);
  a->konst = w.take<float>(a->T);
  a->ids = w.take<int32_t>(a->T, a->L);
  a->weights = w.take<float>(a->T, a->L);
  if (a->K) a->starts = w.take<uint16_t>(2 * a->tiles + 1, a->T);
  if (problem.slopes() && (pass & kBackward)) a->row_scale = a->scales = w.take<float>(a->T);
  // G in one bf16 part: both gradients hang on the labels' entries, whose rounding
  // they get back: dhidden at the end, dweight from sums over each label's rows, taken
  // before the products. (8192 rows of GPT-2-small's head: without, dhidden is 1.41 and
  // dweight 1.2 to 1.46 times as far from the exact ones as their own rounding makes
  // them, with them 1.00 times; the sums take 27 us of a step of 1515.)
  a->rests = a->scales && a->parts == 1 && !a->few;
  if (!a->few) a->hp = w.take<__nv_bfloat16>(a->Tp * a->planes, a->Dp);
  if (a->few) {
    *packed_weight = nullptr;
    a->z = w.take<float>(a->Tp, a->V);
  } else if (weight_in_place(p)) {
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
  if (a->few) {
    // dhidden's parts: as many as make blocks for the card.
    const int64_t block = a->planes == 3 ? 128 : 256, each = std::max<int64_t>(groups, 1) * ((p->D + block - 1) / block);
    a->splits = int32_t(std::max<int64_t>(std::min<int64_t>(2 * zl::kSms / each, (p->V + 31) / 32), 1));
  } else if (pass & kBackward) {
    const int64_t widest = std::max<int64_t>(
        kPieceBytes / (2 * a->parts * a->Tp) / zl::kTileN * zl::kTileN, zl::kTileN);
    pieces = (a->V + widest - 1) / widest;
    a->piece = round_up((a->V + pieces - 1) / pieces, zl::kTileN);
    pieces = (a->V + a->piece - 1) / a->piece;
  }
  if (pass & kBackward && !a->few) {
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
  const int64_t tiles = pass & kBackward && !a->few ? a->splits * (a->Tp / zl::kTileM) * ((a->D + 255) / 256) : 0;
  const int64_t slots = a->rests && p->dweight ? (p->V + 31) / 32 : 0, before = 3 + 2 * pieces + tiles;
  a->zeros = round_up(before, 2) + 2 * slots;
  a->counters = w.take<int32_t>(a->zeros);
  a->never = reinterpret_cast<uint32_t*>(a->counters + 2);
  a->formed = a->never + 1;
  a->used = a->formed + pieces;
  a->added = a->used + pieces;
  if (slots) a->slots = reinterpret_cast<uint2*>(a->counters + round_up(before, 2));
  // The forward pass's arrays and the backward pass's lie over one another.
  const int64_t common = w.at;
  a->sums = w.take<double>(zl::kLossBlocks);
  a->zent = w.take<float>(a->T, a->L);
  if (problem.preference) a->terms = w.take<double>(a->T);
  if (a->has_ce) a->stats = w.take<float2>(a->partials, a->Tp);
  if (problem.slopes() && !a->few) a->places = w.take<uint8_t>(a->partials, a->Tp);
  if (a->has_kd) a->stats_tau = w.take<float2>(a->partials, a->Tp);
  int64_t most = w.at;
  if (pass & kBackward) {
    w.at = common;
    for (int b = 0; b < zl::kBuffers && !a->few; ++b)
      a->g[b] = b < pieces ? w.take<__nv_bfloat16>(a->Tp * a->parts, a->piece) : a->g[0];
    if (p->dhidden) a->dh = w.take<float>(a->splits * a->Tp, a->Dp);
    if (slots) {
      a->rest_rows = p->dhidden ? static_cast<__nv_bfloat16*>(p->dhidden) : w.take<__nv_bfloat16>(p->T, a->Dp);
      a->rest_stride = p->dhidden ? p->dhidden_stride : a->Dp;
    }
    most = std::max(most, w.at);
    if (slots && p->T > zl::kRestRows) {  // over the products' arrays, before them
      w.at = common;
      *rests = rests_of(*a, &w);
      most = std::max(most, w.at);
    }
  }
  // The matrix kernel numbers its tiles in 32 bits.
  const double row_tiles = double((a->Tp + zl::kTileM - 1) / zl::kTileM), wide_tiles = double((a->D + 255) / 256);
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

int workspace_bytes(const Problem& problem, int64_t* bytes) {
  if (!bytes) return set_error(ZERO_EINVAL, "bytes is NULL");
  if (int e = check_sizes(problem)) return e;
  Args a;
  __nv_bfloat16* packed;
  ze::Args rests;
  zero_head_loss_t q = *problem.p;
  q.workspace = nullptr;
  Problem without = problem;
  without.p = &q;
  return plan(without, kForward | (q.dhidden || q.dweight ? kBackward : 0), &a, &packed, &rests, bytes);
}

int run(const Problem& problem, int pass, cudaStream_t s) {
  if (int e = check_sizes(problem)) return e;
  if (int e = check_buffers(problem, pass)) return e;
  const zero_head_loss_t* p = problem.p;
  if (!p->dhidden && !p->dweight) pass &= ~kBackward;  // without rows: an empty dhidden, if any
  if (!pass) return ZERO_OK;
  if (reinterpret_cast<uintptr_t>(p->workspace) % 256)
    return set_error(ZERO_EALIGN, "the workspace is not aligned to 256 bytes");
  Args a;
  __nv_bfloat16* packed;
  ze::Args rests;
  int64_t bytes = 0;
  if (int e = plan(problem, pass, &a, &packed, &rests, &bytes)) return e;
  if (!p->workspace || p->workspace_bytes < bytes)
    return set_error(ZERO_EINVAL, "the workspace has %lld bytes, %lld are needed",
                     (long long)(p->workspace ? p->workspace_bytes : 0), (long long)bytes);
  Program program{};
  if (!a.few) {
    if (!encoder()) return set_error(ZERO_ECUDA, "the CUDA driver has no cuTensorMapEncodeTiled");
    if (!make_program(a, pass & kBackward, &program))
      return set_error(ZERO_EINVAL, "the problem's arrays are too large for tensor maps");
  }
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
  if (problem.slopes() && !(pass & kForward)) {
    next("scales", [&] { return zl::launch_scales(a, s); });
    if (!a.few) next("rows with a slope", [&] { return zl::launch_sloped_rows(a, s); });
  }
  if (a.few)
    next("logits", [&] { return zl::launch_few_logits(a, device, s); });
  else
    next("packing", [&] { return zl::launch_pack(a, packed, false, s); });
  if (pass & kForward) {
    program.forward = 1;
    program.counter = a.counters;
    program.withheld = withheld.passes & kForward ? a.never : nullptr;
    if (!a.few) next("logits", [&] { return zl::launch_products(a, program, device, sms, s); });
    next("losses", [&] { return zl::launch_losses(a, s); });
    if (problem.preference) next("pairs", [&] { return zl::launch_pairs(a, s); });
    if (problem.slopes() && !a.few && (pass & kBackward)) {
      next("rows with a slope", [&] { return zl::launch_sloped_rows(a, s); });
      next("packing", [&] { return zl::launch_pack(a, nullptr, true, s); });
    }
  }
  if (pass & kBackward) {
    program.forward = 0;
    program.counter = a.counters + 1;
    program.withheld = withheld.passes & kBackward ? a.never : nullptr;
    if (a.slots && a.T <= zl::kRestRows) {
      next("the rests", [&] { return zl::launch_rests(a, s); });
    } else if (a.slots) {
      next("the labels", [&] { return ze::launch_sort(rests, s); });
      next("the rests", [&] { return ze::launch_rests(rests, s); });
    }
    next("the gradients", [&] {
      return a.few ? zl::launch_few_gradients(a, s) : zl::launch_products(a, program, device, sms, s);
    });
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
  return workspace_bytes(Problem{p, zl::kXent}, bytes);
}
int zero_xent_forward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kXent}, kForward, stream);
}
int zero_xent_backward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kXent}, kBackward, stream);
}
int zero_xent_step(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kXent}, kForward | kBackward, stream);
}
int zero_distill_workspace_bytes(const zero_head_loss_t* p, int64_t* bytes) {
  return workspace_bytes(Problem{p, zl::kDistill}, bytes);
}
int zero_distill_forward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kDistill}, kForward, stream);
}
int zero_distill_backward(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kDistill}, kBackward, stream);
}
int zero_distill_step(const zero_head_loss_t* p, zero_stream_t stream) {
  return run(Problem{p, zl::kDistill}, kForward | kBackward, stream);
}
int zero_policy_workspace_bytes(const zero_head_loss_t* p, const zero_policy_t* q, int64_t* bytes) {
  return workspace_bytes(Problem{p, zl::kPolicy, q}, bytes);
}
int zero_policy_forward(const zero_head_loss_t* p, const zero_policy_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPolicy, q}, kForward, stream);
}
int zero_policy_backward(const zero_head_loss_t* p, const zero_policy_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPolicy, q}, kBackward, stream);
}
int zero_policy_step(const zero_head_loss_t* p, const zero_policy_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPolicy, q}, kForward | kBackward, stream);
}
int zero_preference_workspace_bytes(const zero_head_loss_t* p, const zero_preference_t* q, int64_t* bytes) {
  return workspace_bytes(Problem{p, zl::kPreference, nullptr, q}, bytes);
}
int zero_preference_forward(const zero_head_loss_t* p, const zero_preference_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPreference, nullptr, q}, kForward, stream);
}
int zero_preference_backward(const zero_head_loss_t* p, const zero_preference_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPreference, nullptr, q}, kBackward, stream);
}
int zero_preference_step(const zero_head_loss_t* p, const zero_preference_t* q, zero_stream_t stream) {
  return run(Problem{p, zl::kPreference, nullptr, q}, kForward | kBackward, stream);
}
int zero_debug_withhold_head_loss(int32_t passes, int64_t limit_ns) {
  if (passes < 0 || passes > 3) return set_error(ZERO_EINVAL, "passes=%d is not in [0, 3]", passes);
  if (limit_ns < 1 || limit_ns > kWaitLimitNs)
    return set_error(ZERO_EINVAL, "limit_ns=%lld is not in [1, %lld]", (long long)limit_ns, (long long)kWaitLimitNs);
  g_withheld = Withheld{passes, limit_ns};
  return ZERO_OK;
}

}  // extern "C"
