// Internal interface between the host side of the vocabulary losses
// (loss_host.cpp) and their kernels (loss_kernels.cu, and the matrix products
// in loss_mma.cu). Not part of the public
// C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zero_gb300.h"

namespace zl {

// Sets the calling thread's error message and returns `code` (zero_host.cpp).
int set_error(int code, const char* fmt, ...);

// Tile of the logits: rows (tokens) by columns (vocabulary).
constexpr int kTileM = 256;
constexpr int kTileN = 256;
constexpr int kPadD = 64;       // packed operands are padded to this width
constexpr int32_t kNoId = 0x7ffffffe;  // above every id, and so is kNoId + 1
constexpr int kSms = 152;        // GB300's multiprocessors. (The layout is planned for them, not for
                                 // what a device reports: the workspace query runs without one.)
constexpr int kBuffers = 3;      // of G
constexpr int kLossBlocks = 608; // most blocks of the losses' kernel
constexpr int kFewGroup = 8;     // few rows are worked on in groups of these
constexpr int kRestRows = 512;   // most rows whose labels' sums are taken without sorting the labels
constexpr int kFewHiddenBytes = 160 << 10;  // most shared memory for a group's hidden states

// Which loss a call takes.
enum Kind : int32_t { kXent, kDistill, kPolicy, kPreference };

// Device-side scalars of a call, at the start of the workspace.
struct Head {
  int32_t rows;    // rows with a target (the compact rows); of a backward pass that goes by
                   // slopes, those whose slope is not zero
  int32_t ticket;  // blocks of the reduction that are done
  int32_t fault;   // a wait of the matrix kernel ran out, or a preference call's offsets do not
                   // ascend: what the call writes becomes NaN
  float factor;    // of both gradients, the same for every row
  int32_t pairs;   // pairs that are not empty
  int32_t repack;  // the backward pass has other rows than the forward pass
  uint32_t steepest; // the largest size of a scale of a preference call, as bits
};

// Everything the kernels read or write. Rows with a target are packed densely:
// compact row i stands for row rowmap[i], and the matrix kernels see only
// compact rows, head->rows of them. Per-row arrays of T entries are indexed
// by the row, those of Tp entries by the compact row.
struct Args {
  int64_t T, V, D;
  int64_t Tp, Dp;         // T and D padded to the tiles
  int32_t planes;         // bf16 parts of a value: 1, or 3 for fp32 storage
  int32_t parts;          // bf16 parts of G: 1 or 2, or 3 for fp32 storage
  int32_t L;              // sparse entries per row
  int32_t K;              // teacher entries per row
  int32_t has_ce, has_kd;
  float ce, kd;           // weights of the two terms' gradients: 1 - alpha, alpha * tau
  float inv_tau;
  double tau;
  int32_t reduction;
  int64_t ignore_index;
  double grad_scale;
  int32_t accumulate;
  int32_t forward;        // the call writes losses

  const void* hidden;
  int64_t hidden_stride;
  const void* weight;
  int64_t weight_stride;
  const int64_t* labels;
  const int64_t* teacher_ids;
  const float* teacher_logits;
  float* loss;
  float* lse;
  float* lse_tau;
  float* reduced;
  const float* dloss;
  const float* row_scale; // [T] factor of each row's gradient, or NULL: dloss where it has an entry a
                          // row, or (in the workspace, `scales`) less the loss's slope by the label's
                          // log-probability
  void* dhidden;
  int64_t dhidden_stride;
  void* dweight;
  int64_t dweight_stride;

  // The policy and the preference loss.
  Kind kind;
  int32_t few;            // few rows: the products are loss_few.cu's
  const float* old_logps;
  const float* advantages;
  const float* ref_logps; // [T], [2 pairs] or NULL
  double low, high;       // bounds of the ratio
  double kl_weight;
  int64_t pairs;
  const int64_t* offsets; // [2 pairs + 1], or NULL: sequences of equal length
  int32_t squared, average;
  double beta, smoothing, margin, nll_weight;
  float* logps;           // [T] or [2 pairs]
  float* row_logps;       // [T] the labels' log-probabilities: logps, or a preference loss's own
  float* slopes;
  int32_t* seq_counts;    // [2 pairs] labelled rows

  // workspace
  Head* head;
  int32_t* rowpos;        // [T] the row's compact row, -1 for an empty row, -2 for one without a slope
  int32_t* rowmap;        // [Tp] the compact row's row
  float2* coef;           // [T] (ce or 0, kd or 0)
  float* konst;           // [T] the loss's part that no logit enters
  int32_t* ids;           // [T][L] ascending, kNoId after the last
  float* weights;         // [T][L] weight of each entry's logit in loss and gradient; a loss by
                          // slopes: p - 1 of the label, from its log-probability, for the gradient
  uint16_t* starts;       // distillation: [2 tiles + 1][T] first entry of each half tile
  float* scales;          // [T] row_scale of a call that goes by slopes
  int32_t rests;          // G is one bf16 value, and what that leaves of the labels' entries (ze::rest_of of
                          // scale and weight) is put back
  uint2* slots;           // [V / 32] with `rests` and dweight: where the labels' rows of `rest_rows` are
  __nv_bfloat16* rest_rows;    // what the rests add to the rows of dweight that are labels', less the common
  int64_t rest_stride;         // factor: in dhidden, which is written last, or in the workspace
  double* terms;          // [T] a preference call's labels' log-probabilities in double
  double* sums;           // [kLossBlocks] parts of the reduced loss
  float* zent;            // [T][L] logits of the entries
  __nv_bfloat16* hp;      // [planes][Tp][Dp] packed hidden states
  const __nv_bfloat16* wp;  // [planes][V][Dp], or the caller's weight (then wp_ld)
  int64_t wp_ld, wp_plane;
  int64_t tiles;          // vocabulary tiles
  int64_t partials;       // of a row's statistics: 2 tiles, or the few rows' blocks
  float2* stats;          // [partials][Tp] some columns' (half a tile's) (m, sum of 2^(z log2(e) - m));
                          // a loss by slopes: of the columns but the label's, and the largest logit z' in m's
                          // place, which is z' log2(e), rounded; few rows: (z', sum of e^(z - z'))
  float2* stats_tau;      // [partials][Tp] of z / tau
  uint8_t* places;        // [partials][Tp] a loss by slopes: which of the half tile's columns z' is in
  float* z;               // [groups][V][kFewGroup] the logits, for few rows
  int32_t* counters;      // [2] units handed out, forward and backward
  uint32_t* never;        // stays zero
  uint32_t* formed;       // [pieces] finished units of a piece's gradient
  uint32_t* used;         // [pieces] finished units of the products with it
  uint32_t* added;        // [tiles of dh] finished units of a tile
  int64_t zeros;          // 32-bit words from `counters` on that begin as zero
  __nv_bfloat16* g[kBuffers];  // [parts][Tp][piece] gradients of pieces of the logits
  int64_t piece;          // columns of a piece, a multiple of kTileN
  int32_t splits;         // parts of a piece's columns that dhidden is summed in
  float* dh;              // [splits][Tp][Dp] running sums of dhidden over the pieces
};

// The matrix kernel's work: see loss_mma.cu.
enum Mode : int32_t { kForward, kGradient, kHidden, kWeight };

struct Program {
  // Operands read along K (boxes of 128 rows) and across it (_mn, boxes of 64
  // rows of K); G, the sums of dhidden and dweight as a warp writes them.
  CUtensorMap hidden, hidden_mn, weight, weight_mn;
  CUtensorMap g[kBuffers], g_mn[kBuffers], g_out[kBuffers];
  CUtensorMap dh, dweight;
  int32_t forward;     // the forward pass (else the backward pass)
  int32_t pieces;
  int32_t weight_tma;  // dweight can be written by TMA
  int32_t* counter;    // units handed out
  uint64_t wait_limit_ns;    // after which a wait gives up
  const uint32_t* withheld;  // NULL, or a word that the kernel waits for (failure injection)
};

// Prepares and numbers the rows.
cudaError_t launch_rows(const Args& a, cudaStream_t s);
// Rows with a target side by side, and the weight's rows to `weight` (NULL: read in place).
// `again`: the rows of the backward pass of a step, where they are others.
cudaError_t launch_pack(const Args& a, __nv_bfloat16* weight, bool again, cudaStream_t s);
cudaError_t launch_losses(const Args& a, cudaStream_t s);
// The logits, their statistics and both gradients, for few rows.
cudaError_t launch_few_logits(const Args& a, int device, cudaStream_t s);
cudaError_t launch_few_gradients(const Args& a, cudaStream_t s);
// The preference loss of the pairs from their rows' log-probabilities.
cudaError_t launch_pairs(const Args& a, cudaStream_t s);
// A backward call's scales from the slopes that it is given.
cudaError_t launch_scales(const Args& a, cudaStream_t s);
// Numbers the rows that have a slope.
cudaError_t launch_sloped_rows(const Args& a, cudaStream_t s);
// The labels' sums of the rests, for up to kRestRows rows.
cudaError_t launch_rests(const Args& a, cudaStream_t s);
// dhidden from its sums; a call whose waits ran out is marked.
cudaError_t launch_dhidden_out(const Args& a, cudaStream_t s);
// The mark alone, where there is no dhidden to write.
cudaError_t launch_mark(const Args& a, cudaStream_t s);
cudaError_t launch_products(const Args& a, const Program& prog, int device, int sms, cudaStream_t s);

}  // namespace zl
