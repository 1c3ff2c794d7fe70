// The matrix products of the vocabulary losses on the tensor cores (tcgen05).
//
// One persistent kernel works off a list of phases, each a grid of tiles:
//   kForward   z = H W^T, kept only as each row's maximum and sum of exponentials
//   kGradient  z again, as the logits' gradient G of one piece of the vocabulary
//   kWeight    dW = G^T H of that piece's rows
//   kHidden    dH += G W over that piece
// The forward pass is one phase; the backward pass is G_0 G_1 W_0 H_0 G_2 W_1
// H_1 G_3 ..., one launch: G has three buffers, so that a piece is formed while
// the two products of an earlier one run, and no launch's beginning and end
// leave the machine idle between pieces. Order between phases is kept by
// counters in global memory (see Progress).
//
// A pair of CTAs (a cluster on two neighbouring SMs) forms one 256 x 256 tile
// with one tcgen05.mma.cta_group::2 stream: each CTA holds 128 rows of A and
// half of B's columns, so an operand byte read from L2 feeds twice the
// multiplications of a single CTA's 128 x 256 tile.
//
// Warps: 0 copies operand tiles by TMA into a ring of stages, 1 (of the pair's
// first CTA) issues the products, 4..11 read finished accumulators from tensor
// memory; two accumulators of 256 columns let the next tile's products run
// under this tile's epilogue. Tiles are handed out by a counter, the long ones
// first: warp 2 of the pair's first CTA takes a number, works out what it
// stands for and passes that to the other warps of both CTAs through a small
// ring, ahead of their need (worked out by the copying thread itself, between
// two tiles, it held the copies up: 26 % on a forward pass of width 768).
//
// fp32 storage: each operand is three bf16 parts and the products of the parts
// are summed into one accumulator, smallest first, in six passes over K.
//
// What bounds it: the tensor pipes, 95 % busy in the forward pass and 82 % in
// the backward pass of 8192 rows of width 768 and a vocabulary of 50257 (312 us,
// 2.0 PFLOP/s, and 1.10 ms, 1.7 PFLOP/s), and over many calls the power limit,
// which lowers the clock: 1.72 PFLOP/s forward, where cuBLAS keeps 1.75. What
// the backward pass loses: dH's additions 4 %, waits between phases 4 %, G's
// stores 2 %, the rest to operands that come from DRAM instead of L2.
//
// The tensor cores' fp32 accumulators truncate: a chain of n additions of one
// sign loses about n 2^-24 of the sum (measured: 1.4e-5 over K = 4096, where
// fp32 additions that round lose 5e-8). Where the sum is kept in fp32 -- the
// logits of the losses, everything of fp32 storage -- it is therefore taken in
// segments of K, which the epilogue adds in registers with rounding.

#include <cuda.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "embedding_internal.h"
#include "loss_device.cuh"

namespace zl {
namespace {

constexpr int kThreads = 384;
constexpr int kEpilogueWarp = 4;   // first of eight
constexpr int kBlockK = 64;        // elements of K a stage holds: 128 bytes
constexpr int kHalf = 128;         // rows of A, and of B, that a CTA holds
constexpr int kOperandBytes = kHalf * kBlockK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kWarpBox = 32 * 64 * 2;      // 32 rows x 64 columns of G on their way out
constexpr int kRing = 3;                   // units on their way to the warps
constexpr int kRegsCopies = 88, kRegsEpilogue = 208;  // 128 x 88 + 256 x 208 = 384 x 168, the launch's

// 192 KB of stages and 32 KB of boxes fill the 227 KB of shared memory. (Five
// stages and two boxes a warp: 2 % slower on a backward pass in bf16, the same
// in fp32.)
constexpr int kStages = 6;
constexpr int kSharedBytes = kStages * kStageBytes + 8 * kWarpBox + 1024 + 512;

// 64-element blocks of K in a segment. Finer ones cost time where the tensor
// pipes are busy (16384 rows of width 768: 644 us, 685 with two segments of six
// blocks, 821 with three of four); up to a tile of rows, where the weight's way
// from memory is waited for anyway, they cost little (one token: 40 us, 42 with
// segments of four blocks) and a loss, being the difference of a sum and one
// logit, gains most (one token: 7e-7 of it, 1.8e-7 with four blocks). The policy
// and the preference loss, which hang on small differences, take segments of six
// blocks (8 us of a step of 8192 rows of width 768).
template <int PLANES>
__device__ __forceinline__ int segment_of(const Args& a, int mode) {
  return PLANES == 3 ? 8 : mode == kForward ? (a.Tp <= kTileM ? 4 : a.kind >= kPolicy ? 6 : 16) : 1 << 24;
}

// ------------------------------------------------------------------- PTX --

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return uint32_t(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void barrier_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Without an order for the thread's earlier memory accesses: for what it has
// read, which needs none. (A release waits for its stores on their way out: with
// it a forward pass of width 768 took 22 % longer.)
__device__ __forceinline__ void barrier_arrive_read(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// `Cluster`: the wait also orders memory that threads of the other CTA wrote.
template <bool Cluster>
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if (Cluster)
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.b32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.b32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// A wait gives up after the program's limit, or when another warp of the CTA has:
// the kernel then ends without its results, the fault is kept in the workspace's
// head, and the call's last kernels set what it writes to NaN.
struct Waiter {
  volatile uint32_t* given_up;  // shared
  Head* head;
  const uint64_t& limit_ns;
  template <bool Cluster = false>
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (barrier_try<Cluster>(bar, parity)) return true;
    const uint64_t begin = timer_ns();
    for (uint32_t n = 1;; ++n) {
      if (barrier_try<Cluster>(bar, parity)) return true;
      if ((n & 1023) == 0 && (*given_up || timer_ns() - begin > limit_ns)) {
        *given_up = 1;
        head->fault = 1;
        return false;
      }
    }
  }
};

// Counts of finished units, one arrival of each CTA (two a unit), made when its
// stores are complete. A unit waits only for units that were handed out before
// it and a pair works its units off in order, so the first unfinished unit never
// waits: no wait is for ever, however few of the grid's pairs run.
struct Progress {
  volatile uint32_t* given_up;
  Head* head;
  const uint64_t& limit_ns;
  __device__ __forceinline__ bool reached(const uint32_t* count, uint32_t target) const {
    uint64_t begin = 0;
    for (uint32_t n = 0;; ++n) {
      uint32_t x;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(count) : "memory");
      if (x >= target) break;
      if (n == 0) begin = timer_ns();
      __nanosleep(100);
      if ((n & 63) == 63 && (*given_up || timer_ns() - begin > limit_ns)) {
        *given_up = 1;
        head->fault = 1;
        return false;
      }
    }
    // What follows reads, or writes over, data that TMA wrote or read.
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return true;
  }
  // One thread, after its stores are complete.
  __device__ __forceinline__ void arrive(uint32_t* count) const {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
  }
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                         uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(map), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
// The same as an addition of fp32 values.
__device__ __forceinline__ void tma_add(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   map), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void store_remote(uint32_t cluster_addr, int4 x) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(x.x), "r"(x.y),
               "r"(x.z), "r"(x.w) : "memory");
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(uint32_t(add)) : "memory");
}
// The barrier at this offset in both CTAs gets one arrival when the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          bar), "h"(uint16_t(3)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const float (&v)[32]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n"
      "tcgen05.wait::st.sync.aligned;" ::
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory matrix descriptor, 128-byte swizzle, 8-row groups 1024 bytes
// apart. K-major (a row of K is 128 bytes): the leading offset is not used.
// MN-major (64 elements of M or N are 128 bytes, one row per k): the leading
// offset is the distance of the next 64 elements.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn_major) {
  const uint64_t lead = mn_major ? (64 * kBlockK * 2) >> 4 : 1;
  return uint64_t((addr & 0x3ffff) >> 4) | lead << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}

// ------------------------------------------------------------------ units --

// The six products of three-part operands, smallest first.
__device__ constexpr int kTermA[6] = {0, 1, 2, 0, 1, 0};
__device__ constexpr int kTermB[6] = {2, 1, 0, 1, 0, 0};

struct Unit {
  int mode;           // negative: no more
  int piece;
  int m0, n0;         // first row and column of the pair's tile
  int n;              // columns of the product: up to 256, a multiple of 32
  int k0, blocks;     // first K element and number of 64-element blocks
  int split;
};

// A unit without terms (no rows, or an empty split) still goes through one
// block, whose product the epilogue does not read: blocks is negative.
__device__ __forceinline__ int blocks_of(const Unit& u) { return u.blocks < 0 ? 1 : u.blocks; }

template <int PLANES>
__device__ __forceinline__ int segments_of(const Args& a, const Unit& u) {
  const int segment = segment_of<PLANES>(a, u.mode);
  return (blocks_of(u) + segment - 1) / segment;
}

__device__ __forceinline__ int piece_cols(const Args& a, int p) {
  return int(min(a.piece, a.V - p * a.piece));
}
__device__ __forceinline__ int tiles_of(int n) { return (n + 255) / 256; }

// Units of a piece's phases.
__device__ __forceinline__ int gradient_units(const Args& a, int rows, int p) {
  return tiles_of(rows) * tiles_of(piece_cols(a, p));
}
__device__ __forceinline__ int weight_units(const Args& a, int p) {
  return a.dweight ? tiles_of(piece_cols(a, p)) * tiles_of(int(a.D)) : 0;
}
__device__ __forceinline__ int hidden_units(const Args& a, int rows) {
  return a.dhidden ? tiles_of(rows) * tiles_of(int(a.D)) * a.splits : 0;
}

// The count of pieces' parts in a tile of dH's sums.
__device__ __forceinline__ uint32_t* hidden_tile(const Args& a, int rows, const Unit& u) {
  return a.added + (u.split * tiles_of(int(a.D)) + u.n0 / 256) * tiles_of(rows) + u.m0 / 256;
}

// The phases in order; the units are numbered through them.
struct Phases {
  int phase = 0, base = 0;

  __device__ __forceinline__ Unit unit(const Args& a, const Program& prog, int rows, int u) {
    const int lead = min(2, prog.pieces);
    for (;; ++phase) {
      if (prog.forward) {
        if (phase > 0) break;
        const int count = tiles_of(rows) * int(a.tiles);
        if (u < count) return tile(a, rows, kForward, 0, u);
        break;
      }
      if (phase < lead) {
        const int count = gradient_units(a, rows, phase);
        if (u < base + count) return tile(a, rows, kGradient, phase, u - base);
        base += count;
        continue;
      }
      const int p = (phase - lead) / 3, which = (phase - lead) % 3;
      if (p >= prog.pieces) break;
      const Mode mode = which == 0 ? kWeight : which == 1 ? kHidden : kGradient;
      const int q = which == 2 ? p + 2 : p;
      const int count = mode == kWeight ? weight_units(a, q) : mode == kHidden ? hidden_units(a, rows)
                        : q < prog.pieces ? gradient_units(a, rows, q) : 0;
      if (u < base + count) return tile(a, rows, mode, q, u - base);
      base += count;
    }
    Unit none{};
    none.mode = -1;
    return none;
  }

  __device__ __forceinline__ static Unit tile(const Args& a, int rows, Mode mode, int p, int u) {
    const bool logits = mode == kForward || mode == kGradient;
    const int cols = mode == kForward ? int(a.V) : piece_cols(a, p);
    const int width = logits ? cols : int(a.D);
    const int depth = mode == kWeight ? rows : mode == kHidden ? cols : int(a.D);
    const int mt = tiles_of(mode == kWeight ? cols : rows), nt = tiles_of(width);
    const int splits = mode == kHidden ? a.splits : 1;
    const int at = u % (mt * nt);
    Unit x;
    x.mode = mode;
    x.piece = p;
    x.split = u / (mt * nt);
    x.m0 = (logits ? at % mt : at / nt) * 256;
    x.n0 = (logits ? at / mt : at % nt) * 256;
    x.n = min(256, (width - x.n0 + 31) / 32 * 32);
    const int blocks = (depth + kBlockK - 1) / kBlockK;
    const int first = int(int64_t(blocks) * x.split / splits);
    x.k0 = first * kBlockK;
    x.blocks = int(int64_t(blocks) * (x.split + 1) / splits) - first;
    if (x.blocks == 0) x.blocks = -1;
    return x;
  }
};

// --------------------------------------------------------------- epilogues --

struct Thread {          // of the epilogue
  int row;               // of the CTA's 128
  int half;              // columns [128 half, 128 half + 128)
};

// A row of the logits: what the epilogues of kForward and kGradient need of
// it, read while the products are still running.
struct Row {
  int i;                   // compact row
  int64_t t;
  bool there;
  int e, end;              // its sparse entries in the thread's columns
  int32_t id, next_id;     // of entry e and the one after it
  float w, next_w;         // their weights (kGradient)
  float2 f;                // weights of the two terms (kGradient, with scale, lse and lse_kd)
  float scale, lse, lse_kd;
};

__device__ __forceinline__ void entry_ahead(const Args& a, const Unit& u, const Row& r, int e, int32_t& id, float& w) {
  id = e < r.end ? a.ids[r.t * a.L + e] : kNoId;
  w = e < r.end && u.mode == kGradient ? a.weights[r.t * a.L + e] : 0.0f;
}

template <bool CE, bool KD>
__device__ __forceinline__ Row row_of(const Args& a, int rows, const Unit& u, const Thread& th, uint32_t rank) {
  Row r{};
  r.i = u.m0 + int(rank) * kHalf + th.row;
  r.there = r.i < rows;
  r.id = r.next_id = kNoId;
  if (!r.there) return r;
  r.t = a.rowmap[r.i];
  const int64_t v = u.piece * a.piece + u.n0 + th.half * 128;
  if (u.mode == kGradient) {
    r.f = a.coef[r.t];
    if (CE) r.lse = a.lse[r.t];
    if (KD) r.lse_kd = a.lse_tau[r.t];
    r.scale = a.row_scale ? a.row_scale[r.t] : 1.0f;
  }
  if (a.K == 0) {
    r.id = a.ids[r.t];
    if (u.mode == kGradient) r.w = a.weights[r.t];
    r.end = 1;
    if (r.id < v) r.id = kNoId;
  } else {
    const uint16_t* at = a.starts + v / 128 * a.T + r.t;
    r.e = at[0];
    r.end = at[a.T];
    entry_ahead(a, u, r, r.e, r.id, r.w);
    entry_ahead(a, u, r, r.e + 1, r.next_id, r.next_w);
  }
  return r;
}

// Calls f(at) while a row of the warp has a sparse entry (r.e, of weight r.w)
// among the 32 columns from v on: `at` is the thread's own entry's column among
// them, or -1. (The columns are registers, so f picks by comparing.)
template <typename F>
__device__ __forceinline__ void each_entry(const Args& a, const Unit& u, Row& r, int64_t v, F f) {
  for (;;) {
    const int64_t c = r.id - v;
    const int at = c >= 0 && c < 32 ? int(c) : -1;
    if (!__any_sync(~0u, at >= 0)) break;
    f(at);
    if (at >= 0) {
      ++r.e;
      r.id = r.next_id;
      r.w = r.next_w;
      entry_ahead(a, u, r, r.e + 1, r.next_id, r.next_w);
    }
  }
}

// x to the power of P.
template <int P>
__device__ __forceinline__ float power(float x) {
  return P == 1 ? x : P == 2 ? x * x : (x * x) * (x * x);
}

// Sums of 2^(c z - m) with m moved to the maximum. m is the rounded product,
// the reference that the sum is stored with, so its rounding cancels. Where tau
// is 1, 2 or 4 the values of z are powers of those of z / tau, and with m_ce
// = tau m_kd so are the references: one exponential serves both sums (P). (At
// tau = 2, 4096 rows of a vocabulary of 50257: a step of 822 us, 839 with two.)
struct Sums {
  float m_ce, ce, m_kd, kd;
};

template <bool CE, bool KD, int P>
__device__ __forceinline__ void add_exponentials(const float (&z)[32], float top, float c_ce, float c_kd, Sums& s) {
  const bool begun = (CE && P == 0 ? s.m_ce : s.m_kd) != -INFINITY;
  const float next_kd = __fmul_rn(top, c_kd);
  const float next_ce = P ? float(P) * next_kd : __fmul_rn(top, c_ce);
  const float base_kd = next_kd == -INFINITY ? 0.0f : next_kd, base_ce = next_ce == -INFINITY ? 0.0f : next_ce;
  float ce[2] = {begun && CE ? s.ce * exp2_fast(s.m_ce - base_ce) : 0.0f, 0.0f};
  float kd[2] = {begun && KD ? s.kd * exp2_fast(s.m_kd - base_kd) : 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float x = 0.0f;
    if (KD) {
      x = exp2_fast(fmaf(z[j], c_kd, -base_kd));
      kd[j & 1] += x;
    }
    if (CE) ce[j & 1] += KD && P ? power<P>(x) : exp2_fast(fmaf(z[j], c_ce, -base_ce));
  }
  s = Sums{next_ce, ce[0] + ce[1], next_kd, kd[0] + kd[1]};
}

// The power of tau that add_exponentials and the gradient use, 0 for none.
__device__ __forceinline__ int shared_power(float tau) { return tau == 1.0f ? 1 : tau == 2.0f ? 2 : tau == 4.0f ? 4 : 0; }

// 32 columns of a row into its statistics, and the logits of the entries among them
// (a loss by slopes: all but the label's column, see losses_kernel).
// `at`, a loss by slopes: which of the thread's columns the maximum is in, counted from `c` for these
// (8192 rows of GPT-2-small's head: 342 us instead of 327).
template <bool CE, bool KD, bool Slopes>
__device__ __forceinline__ void forward_columns(const Args& a, const Unit& u, Row& r, int64_t v, int valid, int p,
                                                float (&z)[32], float& top, Sums& s, int c, int& at) {
  const float c_ce = kLog2e, c_kd = KD ? a.inv_tau * kLog2e : kLog2e;
  if (valid < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j >= valid) z[j] = -INFINITY;
  }
  each_entry(a, u, r, v, [&](int entry) {
    if (Slopes) {  // the statistics are those of the other columns
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == entry) z[j] = -INFINITY;
      return;
    }
    float x = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j == entry) x = z[j];
    if (entry >= 0) a.zent[r.t * a.L + r.e] = x;
  });
  float t0 = top, t1 = -INFINITY;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    t0 = fmaxf(t0, z[j]);
    t1 = fmaxf(t1, z[j + 1]);
  }
  top = fmaxf(t0, t1);
  if (Slopes) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (z[j] == top) at = c + j;
  }
  if (CE && KD) {
    if (p == 1) add_exponentials<CE, KD, 1>(z, top, c_ce, c_kd, s);
    else if (p == 2) add_exponentials<CE, KD, 2>(z, top, c_ce, c_kd, s);
    else if (p == 4) add_exponentials<CE, KD, 4>(z, top, c_ce, c_kd, s);
    else add_exponentials<CE, KD, 0>(z, top, c_ce, c_kd, s);
  } else {
    add_exponentials<CE, KD, 0>(z, top, c_ce, c_kd, s);
  }
}

// `Held`: the logits are in registers already (the segments' sum), else they
// are in the accumulator.
template <bool CE, bool KD, bool Slopes, bool Held>
__device__ __forceinline__ void forward_epilogue(const Args& a, const Unit& u, const Thread& th, Row& r, uint32_t acc,
                                                 float (&held)[4][32]) {
  if (!__any_sync(~0u, r.there)) return;
  const int64_t v0 = u.n0;
  const int begin = th.half * 128;
  const int cols = int(min(int64_t(256), a.V - v0));
  const int p = CE && KD ? shared_power(float(a.tau)) : 0;
  float top = -INFINITY;
  int place = 0;
  Sums s = {-INFINITY, 0.0f, -INFINITY, 0.0f};
  if (Held) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = begin + 32 * k;
      if (c < cols) forward_columns<CE, KD, Slopes>(a, u, r, v0 + c, cols - c, p, held[k], top, s, 32 * k, place);
    }
  } else {
#pragma unroll 1
    for (int c = begin; c < min(cols, begin + 128); c += 32) {
      float z[32];
      tmem_load32(acc + c, z);
      forward_columns<CE, KD, Slopes>(a, u, r, v0 + c, cols - c, p, z, top, s, c - begin, place);
    }
  }
  if (!r.there) return;
  const int64_t at = (v0 / 256 * 2 + th.half) * a.Tp + r.i;
  const bool nan = isnan(s.ce + s.kd);
  if (Slopes) {
    a.stats[at] = make_float2(nan ? NAN : top, s.ce);
    a.places[at] = uint8_t(place);
    return;
  }
  if (CE) a.stats[at] = make_float2(nan ? NAN : s.m_ce, s.ce);
  if (KD) a.stats_tau[at] = make_float2(nan ? NAN : s.m_kd, s.kd);
}

// Two values as a word of bf16, rounded to nearest.
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The same, with what the rounding left over in place of the values: called
// again and again it gives the parts of the values.
__device__ __forceinline__ uint32_t next_part(float& x0, float& x1) {
  const uint32_t w = pack_bf16(x0, x1);
  x0 -= __uint_as_float(w << 16);
  x1 -= __uint_as_float(w & 0xffff0000u);
  return w;
}

// The warp's staging box may be written again: its last store has read it.
__device__ __forceinline__ void box_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// 32 fp32 values of the lane's row into a box of 32 rows x 128 bytes.
__device__ __forceinline__ void stage_fp32(uint8_t* box, int lane, const float (&x)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ (lane & 7)) * 16)) =
        make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}

// The logits' gradient without the factor that all rows share, as the bf16
// operand of the two products: rounded once, or in PARTS parts (fp32 storage and
// a few rows of bf16: loss_host.cpp says when). Each warp stages boxes of its 32
// rows by 64 columns and stores them by TMA.
template <int PLANES, int PARTS, bool CE, bool KD, int P, bool Slopes>
__device__ __forceinline__ void gradient_epilogue(const Args& a, const CUtensorMap* out, const Unit& u,
                                                  const Thread& th, int rows, Row& r, uint32_t acc, uint32_t rank,
                                                  uint8_t* box) {
  const int begin = th.half * 128, lane = th.row & 31;
  if (r.i - lane >= (rows + kBlockK - 1) / kBlockK * kBlockK) {  // rows that no product's terms reach
    if (lane == 0)
      for (int n = 0; n < 2 * PARTS; ++n) store_commit();  // the groups are counted
    return;
  }
  const int64_t v0 = u.piece * a.piece + u.n0;
  const int cols = int(min(int64_t(256), a.V - v0));
  const float c_ce = kLog2e, c_kd = a.inv_tau * kLog2e;
  // Terms that the row does not have are 2^-inf = 0, whatever the accumulator holds.
  const float lse = CE && r.f.x != 0.0f ? r.lse : INFINITY, lse_kd = KD && r.f.y != 0.0f ? r.lse_kd : INFINITY;
  // P: p_v = softmax(z)_v is softmax(z / tau)_v^tau times a factor of the row.
  const float m_kd = (KD && P && lse_kd == INFINITY ? lse * a.inv_tau : lse_kd) * kLog2e, m_ce = lse * kLog2e;
  const float w_kd = r.f.y * r.scale;
  const float w_ce = r.f.x == 0.0f ? 0.0f : r.f.x * r.scale * (P ? exp2_fast(float(P) * m_kd - m_ce) : 1.0f);
  const float lse_shared = KD && P && lse_kd == INFINITY ? lse * a.inv_tau : lse_kd;
  auto value = [&](float z) {
    float g = 0.0f;
    if (KD) {
      // fp32: the difference first, whose rounding is relative to it, not to the logit
      const float x = PLANES == 1 ? exp2_fast(fmaf(z, c_kd, -m_kd))
                                  : exp2_fast(fmaf(z, a.inv_tau, -lse_shared) * kLog2e);
      g = w_kd * x;
      if (CE && P) return fmaf(w_ce, power<P>(x), g);
    }
    if (CE) {
      const float x = PLANES == 1 ? exp2_fast(fmaf(z, c_ce, -m_ce)) : exp2_fast((z - lse) * kLog2e);
      g = KD ? fmaf(w_ce, x, g) : w_ce * x;
    }
    return g;
  };
  // 32 columns of the row.
  auto columns = [&](int c0, float (&g)[32]) {
    tmem_load32(acc + c0, g);
    const int valid = cols - c0;
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] = value(g[j]);
    if (valid < 32 || !r.there) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= valid || !r.there) g[j] = 0.0f;
    }
    each_entry(a, u, r, v0 + c0, [&](int at) {
      const float d = r.scale * r.w;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == at) g[j] = Slopes ? d : g[j] - d;  // (by slopes: d is s (p - 1))
    });
  };
  // They, or their next part, into half a box.
  auto stage = [&](int half, float (&g)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float &x0 = g[8 * q + 2 * n], &x1 = g[8 * q + 2 * n + 1];
        w[n] = PARTS == 1 ? pack_bf16(x0, x1) : next_part(x0, x1);
      }
      *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * half + q) ^ (lane & 7)) * 16)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  auto store = [&](int b, int p) {
    proxy_fence();
    __syncwarp();
    if (lane == 0) {
      tma_store(out, smem_u32(box), u.n0 + begin + 64 * b, u.m0 + int(rank) * kHalf + th.row, p);
      store_commit();
    }
  };
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {  // 64 columns at a time
    if (PARTS == 1) {
      box_free(lane);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        float g[32];
        columns(begin + 64 * b + 32 * k, g);
        stage(k, g);
      }
      store(b, 0);
    } else {
      float g[2][32];
      columns(begin + 64 * b, g[0]);
      columns(begin + 64 * b + 32, g[1]);
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        box_free(lane);
        stage(0, g[0]);
        stage(1, g[1]);
        store(b, p);
      }
    }
  }
}

// 32 columns of the accumulator, or zeros for a unit without terms.
__device__ __forceinline__ void load_terms(const Unit& u, uint32_t addr, float (&x)[32]) {
  if (u.blocks > 0) {
    tmem_load32(addr, x);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
  }
}

// dH of a piece, fp32: stored by the first piece, added by the others (TMA
// reductions in L2, 2.6 TB/s where all tiles leave at once). An element gets one
// addition of each piece, and a piece's comes after the one before is complete,
// so the order is fixed. (The earlier sum read by the threads while the products
// ran, then a plain store: 30 % slower on the whole pass. H's tiles spread among
// the next piece's G: no faster.)
__device__ __forceinline__ void hidden_epilogue(const CUtensorMap* out, const Unit& u, const Thread& th, int rows,
                                                uint32_t acc, uint32_t rank, uint8_t* box) {
  const int lane = th.row & 31, begin = th.half * 128;
  const int row = u.m0 + int(rank) * kHalf + th.row;
  if (row - lane >= rows) return;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const int c = begin + 32 * k;
    if (c >= u.n) break;
    float x[32];
    load_terms(u, acc + c, x);
    box_free(lane);
    stage_fp32(box, lane, x);
    proxy_fence();
    __syncwarp();
    if (lane == 0) {
      if (u.piece == 0) tma_store(out, smem_u32(box), u.n0 + c, row, u.split);
      else tma_add(out, smem_u32(box), u.n0 + c, row, u.split);
      store_commit();
    }
  }
}

// Adds 32 columns of a row of the rests from d on.
__device__ __forceinline__ void add_rests(const Args& a, const __nv_bfloat16* row, int64_t d, float (&x)[32]) {
  if (d + 32 <= a.D && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {  // (d: a multiple of 32)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 w = reinterpret_cast<const uint4*>(row + d)[q];
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        x[8 * q + 2 * n] += __uint_as_float(words[n] << 16);
        x[8 * q + 2 * n + 1] += __uint_as_float(words[n] & 0xffff0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (d + j < a.D) x[j] += __bfloat162float(row[d + j]);
}

// dW of a piece's rows, by TMA where the caller's rows are 16-byte aligned
// (fp32: also the addition to what is there; bf16 would round it twice), else
// by the threads. `Rests`: to labels' rows what G's rounding left of their entries is
// added, from their slots. (A warp's rows share a word of `slots`.)
template <int PLANES, bool Rests>
__device__ __forceinline__ void weight_epilogue(const Args& a, const Program& prog, const Unit& u, const Thread& th,
                                                float factor, uint32_t acc, uint32_t rank, uint8_t* box) {
  using T = typename std::conditional<PLANES == 1, __nv_bfloat16, float>::type;
  const int lane = th.row & 31, begin = th.half * 128;
  const int64_t v = u.piece * a.piece + u.m0 + int(rank) * kHalf + th.row;
  const int64_t slot = Rests && v < a.V ? ze::slot_of(a.slots[v / 32], int(v % 32)) : -1;
  const __nv_bfloat16* const rests = Rests ? a.rest_rows + max(slot, int64_t(0)) * a.rest_stride : nullptr;
  if (prog.weight_tma) {
    constexpr int wide = 128 / sizeof(T);  // columns of a box
#pragma unroll 1
    for (int k = 0; k < 128 / wide; ++k) {
      const int c = begin + wide * k;
      if (c >= u.n) break;
      box_free(lane);
#pragma unroll
      for (int h = 0; h < wide / 32; ++h) {
        float x[32];
        load_terms(u, acc + c + 32 * h, x);
        if (Rests && slot >= 0) add_rests(a, rests, u.n0 + c + 32 * h, x);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] *= factor;
        if (PLANES == 3) {
          stage_fp32(box, lane, x);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t word[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) word[q] = pack_bf16(x[8 * j + 2 * q], x[8 * j + 2 * q + 1]);
            *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * h + j) ^ (lane & 7)) * 16)) =
                make_uint4(word[0], word[1], word[2], word[3]);
          }
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) {
        // Rows and columns past the matrix are not written.
        if (v < a.V) {
          if (a.accumulate) tma_add(&prog.dweight, smem_u32(box), u.n0 + c, int(v), 0);
          else tma_store(&prog.dweight, smem_u32(box), u.n0 + c, int(v), 0);
        }
        store_commit();
      }
    }
    return;
  }
  // 32 columns at a time through shared memory, so that a warp's accesses run
  // along a row.
  const int64_t v_warp = v - lane;
  box_free(lane);
  const float* values = reinterpret_cast<const float*>(box);
#pragma unroll 1
  for (int c = begin; c < min(u.n, begin + 128); c += 32) {
    float x[32];
    load_terms(u, acc + c, x);
    if (Rests && slot >= 0) add_rests(a, rests, u.n0 + c, x);
    __syncwarp();
    stage_fp32(box, lane, x);
    __syncwarp();
    const bool in = u.n0 + c + lane < a.D;
    T* to = static_cast<T*>(a.dweight) + v_warp * a.dweight_stride + u.n0 + c + lane;
#pragma unroll 4
    for (int i = 0; i < 32; ++i, to += a.dweight_stride) {
      if (!in || v_warp + i >= a.V) continue;
      const float y = factor * values[i * 32 + (((lane / 4) ^ (i & 7)) * 4) + lane % 4];
      *to = T(a.accumulate ? float(*to) + y : y);
    }
  }
}

// ----------------------------------------------------------------- kernel --

// `Slopes`: of a loss by slopes.
template <int PLANES, int PARTS, bool CE, bool KD, bool Slopes>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    products_kernel(const __grid_constant__ Args a, const __grid_constant__ Program prog) {
  static_assert(PLANES == 1 ? PARTS <= 2 : PLANES == 3 && PARTS == 3, "the products of the parts");
  // Products of parts that a block of K stands for: with two parts of G one
  // after the other, so that the block of the other operand stays in L2.
  auto terms_of = [](const Unit& x) {
    return PLANES == 3 ? 6 : PARTS == 2 && (x.mode == kWeight || x.mode == kHidden) ? 2 : 1;
  };
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = base + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 8 * kWarpBox);
  // Barriers: stage full and empty, accumulator full and empty, ring full and empty.
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, ring_full = acc_empty + 16, ring_empty = ring_full + 8 * kRing;
  int4* ring = reinterpret_cast<int4*>(bars + 2 * kStages + 4 + 2 * kRing);
  static_assert((2 * kStages + 4 + 2 * kRing) % 2 == 0, "the ring is read 16 bytes at a time");
  uint64_t* stored_bars = reinterpret_cast<uint64_t*>(ring + 2 * kRing);
  const uint32_t stored = smem_u32(stored_bars);
  uint32_t** counts = reinterpret_cast<uint32_t**>(stored_bars + 2);  // [2][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(counts + 4);
  volatile uint32_t* given_up = tmem_slot + 1;
  volatile int* counted = reinterpret_cast<volatile int*>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  let_next_start();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      barrier_init(full + 8 * s, 1);
      barrier_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      barrier_init(acc_full + 8 * b, 1);
      barrier_init(acc_empty + 8 * b, 16);  // eight warps of each CTA
    }
    for (int q = 0; q < kRing; ++q) {
      barrier_init(ring_full + 8 * q, 1);
      barrier_init(ring_empty + 8 * q, 16);
    }
    barrier_init(stored, 8);
    barrier_init(stored + 8, 8);
    *given_up = 0;
    *counted = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  const int rows = a.head->rows;
  const Waiter wait{given_up, a.head, prog.wait_limit_ns};
  const Progress progress{given_up, a.head, prog.wait_limit_ns};
  Unit u;
  // The ring's next entry. The epilogue warps give it back to the pair's first
  // CTA once the unit's first accumulator is full: by then the copies and the
  // products have read it too. (Arrivals of theirs as well, across the pair, cost
  // the forward pass of width 768 11 %.)
  int slot = 0;
  uint32_t slot_phase = 0;
  auto next_unit = [&] {
    if (!wait.operator()<true>(ring_full + 8 * slot, slot_phase)) return false;
    const int4 x = ring[2 * slot], y = ring[2 * slot + 1];
    u = Unit{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (++slot == kRing) {
      slot = 0;
      slot_phase ^= 1;
    }
    return true;
  };

  if (warp < kEpilogueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCopies));
    if (warp == 0) {
      // ---- copies
      if (elect_one()) {
        const uint32_t full0 = in_cta(full, 0);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int formed = -1;  // the last piece known to be there
        if (prog.withheld) ok = progress.reached(prog.withheld, 1);
        while (ok) {
          if (!(ok = next_unit()) || u.mode < 0) break;
          const bool a_mn = u.mode == kWeight, b_mn = u.mode == kWeight || u.mode == kHidden;
          if (b_mn && u.piece > formed) {
            if (!(ok = progress.reached(a.formed + u.piece, 2 * gradient_units(a, rows, u.piece)))) break;
            formed = u.piece;
          }
          const int c0 = int(u.piece * a.piece), buffer = u.piece % kBuffers;
          const CUtensorMap* map_a = u.mode == kWeight ? &prog.g_mn[buffer]
                                     : u.mode == kHidden ? &prog.g[buffer] : &prog.hidden;
          const CUtensorMap* map_b = u.mode == kWeight ? &prog.hidden_mn
                                     : u.mode == kHidden ? &prog.weight_mn : &prog.weight;
          const int am = u.m0 + int(rank) * kHalf;
          const int bn = u.n0 + int(rank) * (u.n / 2) + (u.mode == kGradient ? c0 : 0);
          const int b_k0 = u.mode == kHidden ? c0 : 0;
          const int b_boxes = b_mn ? (u.n / 2 + 63) / 64 : 0;
          const uint32_t bytes = 2 * (kOperandBytes + (b_mn ? b_boxes * 64 * kBlockK * 2 : kOperandBytes));
          const int segments = segments_of<PLANES>(a, u);
          const int segment = segment_of<PLANES>(a, u.mode);
          for (int s = 0; ok && s < segments; ++s) {
            const int k_begin = s * segment, k_end = min(blocks_of(u), k_begin + segment);
            for (int term = 0; ok && term < (PLANES == 3 ? 6 : 1); ++term) {
              const int pb = PLANES == 3 ? kTermB[term] : 0;
              const int each = PLANES == 3 ? 1 : terms_of(u);  // 1 or 2
              for (int i = k_begin * each; i < k_end * each; ++i) {
                const int k = i >> (each - 1);
                const int pa = PLANES == 3 ? kTermA[term] : (i + 1) & (each - 1);
                if (!(ok = wait(empty + 8 * stage, phase ^ 1))) break;
                const uint32_t sa = smem_u32(base + stage * kStageBytes), sb = sa + kOperandBytes;
                const uint32_t bar = full0 + 8 * stage;
                if (rank == 0) barrier_expect(full + 8 * stage, bytes);
                const int kk = u.k0 + k * kBlockK;
                if (a_mn) {
                  tma_load(sa, map_a, am, kk, pa, bar);
                  tma_load(sa + 64 * kBlockK * 2, map_a, am + 64, kk, pa, bar);
                } else {
                  tma_load(sa, map_a, kk, am, pa, bar);
                }
                if (b_mn) {
                  for (int c = 0; c < b_boxes; ++c)
                    tma_load(sb + c * 64 * kBlockK * 2, map_b, bn + 64 * c, kk + b_k0, pb, bar);
                } else {
                  tma_load(sb, map_b, kk, bn, pb, bar);
                }
                if (++stage == kStages) {
                  stage = 0;
                  phase ^= 1;
                }
              }
            }
          }
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ---- products
      if (elect_one()) {
        int stage = 0;
        uint32_t phase = 0, acc_phase = 0;
        int buffer = 0;
        bool ok = true;
        while (ok && next_unit() && u.mode >= 0) {
          const bool a_mn = u.mode == kWeight, b_mn = u.mode == kWeight || u.mode == kHidden;
          const int segments = segments_of<PLANES>(a, u);
          // fp32 accumulator, bf16 operands, majors, N, M = 256
          const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | uint32_t(a_mn) << 15 | uint32_t(b_mn) << 16 |
                                 uint32_t(u.n / 8) << 17 | uint32_t(256 / 16) << 24;
          const uint64_t a_step = (a_mn ? 16 * 128 : 32) >> 4, b_step = (b_mn ? 16 * 128 : 32) >> 4;
          const int segment = segment_of<PLANES>(a, u.mode);
          for (int s = 0; ok && s < segments; ++s) {
            const uint32_t d = tmem + buffer * 256;
            if (!(ok = wait(acc_empty + 8 * buffer, acc_phase ^ 1))) break;
            fence_after();
            bool add = false;
            const int count = (min(blocks_of(u), (s + 1) * segment) - s * segment) * terms_of(u);
            for (int k = 0; k < count; ++k) {
              if (!(ok = wait(full + 8 * stage, phase))) break;
              fence_after();
              const uint32_t sa = smem_u32(base + stage * kStageBytes);
              const uint64_t da = operand_desc(sa, a_mn), db = operand_desc(sa + kOperandBytes, b_mn);
#pragma unroll
              for (int q = 0; q < kBlockK / 16; ++q) {
                mma(d, da + q * a_step, db + q * b_step, idesc, add);
                add = true;
              }
              mma_commit(empty + 8 * stage);
              if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
              }
            }
            mma_commit(acc_full + 8 * buffer);
            if (++buffer == 2) {
              buffer = 0;
              acc_phase ^= 1;
            }
          }
        }
      }
    } else if (warp == 2 && rank == 0) {
      // ---- hands out the units
      if (elect_one()) {
        // In the forward pass, where no unit waits for another, a pair's first one
        // is its own number. In the backward pass that would give units to pairs
        // that do not run yet, and the others could wait for them while holding
        // the SMs that they need (beside another such launch).
        const int32_t given = prog.forward ? int32_t(gridDim.x / 2) : 0;
        Phases phases;
        for (int32_t n = prog.forward ? int32_t(blockIdx.x / 2) : atomicAdd(prog.counter, 1);;
             n = given + atomicAdd(prog.counter, 1)) {
          const Unit x = phases.unit(a, prog, rows, n);
          if (!wait(ring_empty + 8 * slot, slot_phase ^ 1)) break;
          for (uint32_t c = 0; c < 2; ++c) {
            const uint32_t to = in_cta(smem_u32(ring + 2 * slot), c);
            store_remote(to, make_int4(x.mode, x.piece, x.m0, x.n0));
            store_remote(to + 16, make_int4(x.n, x.k0, x.blocks, x.split));
            barrier_arrive_remote(in_cta(ring_full + 8 * slot, c));
          }
          if (++slot == kRing) {
            slot = 0;
            slot_phase ^= 1;
          }
          if (x.mode < 0) break;
        }
      }
    } else if (warp == 3 && !prog.forward) {
      // ---- counts the finished units, off the epilogues' path: a release waits
      // for stores still on their way (5 % of a backward pass of 8192 rows)
      if (elect_one()) {
        for (int n = 0; wait(stored + 8 * (n & 1), (n >> 1) & 1); ++n) {
          uint32_t *const unit = counts[2 * (n & 1)], *const tile = counts[2 * (n & 1) + 1];
          if (!unit) break;
          if (tile) progress.arrive(tile);
          progress.arrive(unit);
          *counted = n + 1;
        }
      }
    }
  } else {
    // ---- epilogues
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
    Thread th;
    th.row = (warp & 3) * 32 + lane;
    th.half = (warp - kEpilogueWarp) / 4;
    uint8_t* box = staging + (warp - kEpilogueWarp) * kWarpBox;
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t acc_empty0 = in_cta(acc_empty, 0);
    const float factor = a.head->factor;
    int buffer = 0, used = -1;  // used: the last piece known to be through
    uint32_t phase = 0;
    auto full_accumulator = [&] {
      if (!wait(acc_full + 8 * buffer, phase)) return false;
      fence_after();
      return true;
    };
    auto give_back = [&] {
      fence_before();
      __syncwarp();
      if (lane == 0) barrier_arrive_read(acc_empty0 + 8 * buffer);
      if (++buffer == 2) {
        buffer = 0;
        phase ^= 1;
      }
    };
    // A finished unit is counted once its stores are complete: at the end of
    // the next unit where both are kGradient, so that nothing waits for the
    // stores; else before the next unit's accumulator is waited for, since what
    // that waits for may be this. Each warp reports to warp 3; two units may be
    // on their way there.
    uint32_t *finished = nullptr, *finished_tile = nullptr;
    int reports = 0;
    auto report = [&](uint32_t* unit, uint32_t* tile) {
      for (uint32_t n = 0; *counted < reports - 1 && !*given_up; ++n) __nanosleep(20);
      if (warp == kEpilogueWarp) {
        counts[2 * (reports & 1)] = unit;
        counts[2 * (reports & 1) + 1] = tile;
      }
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(stored + 8 * (reports & 1)) : "memory");
      ++reports;
    };
    auto count_finished = [&] {
      if (lane == 0 && finished) {
        store_wait();
        report(finished, finished_tile);
      }
      finished = finished_tile = nullptr;
    };
    for (;;) {
      const uint32_t entry = in_cta(ring_empty + 8 * slot, 0);
      if (!__all_sync(~0u, next_unit()) || u.mode < 0) break;
      if (u.mode != kGradient) count_finished();
      Row r{};
      bool ok = true;
      const int segments = segments_of<PLANES>(a, u);
      if (u.mode == kForward || u.mode == kGradient) r = row_of<CE, KD>(a, rows, u, th, rank);
      if (segments == 1) {
        ok = __all_sync(~0u, full_accumulator());
        if (lane == 0) barrier_arrive_read(entry);
      } else {
        const int begin = th.half * 128;
        float sum[4][32] = {};
        for (int s = 0; ok && s < segments; ++s) {
          if (!(ok = __all_sync(~0u, full_accumulator()))) break;
          if (s == 0 && lane == 0) barrier_arrive_read(entry);
          const uint32_t acc = lanes + buffer * 256 + begin;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x[16];
            tmem_load16(acc + 16 * k, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[k / 2][k % 2 * 16 + j] += x[j];
          }
          if (s < segments - 1 || u.mode == kForward) {
            give_back();
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_store32(acc + 32 * k, sum[k]);
          }
        }
        if (ok && u.mode == kForward) {  // both accumulators are the next unit's already
          forward_epilogue<CE, KD, Slopes, true>(a, u, th, r, 0, sum);
          continue;
        }
      }
      if (!ok) break;
      // The buffer that G goes to has been read by both products of the piece
      // that was there; a tile of dH has its earlier pieces.
      const int earlier = u.mode == kGradient ? u.piece - kBuffers : -1;
      if (earlier > used) {
        count_finished();
        ok = progress.reached(a.used + earlier, 2 * (weight_units(a, earlier) + hidden_units(a, rows)));
        used = earlier;
      }
      uint32_t* const tile = u.mode == kHidden ? hidden_tile(a, rows, u) : nullptr;
      if (tile && u.piece > 0) {
        count_finished();
        ok = progress.reached(tile, 2 * u.piece);
      }
      if (!__all_sync(~0u, ok)) break;
      const uint32_t acc = lanes + buffer * 256;
      if (u.mode == kForward) {
        float none[4][32];
        forward_epilogue<CE, KD, Slopes, false>(a, u, th, r, acc, none);
      } else if (u.mode == kGradient) {
        const CUtensorMap* out = &prog.g_out[u.piece % kBuffers];
        const int p = CE && KD ? shared_power(float(a.tau)) : 0;
        if (CE && KD && p == 1) gradient_epilogue<PLANES, PARTS, CE, KD, 1, Slopes>(a, out, u, th, rows, r, acc, rank, box);
        else if (CE && KD && p == 2) gradient_epilogue<PLANES, PARTS, CE, KD, 2, Slopes>(a, out, u, th, rows, r, acc, rank, box);
        else if (CE && KD && p == 4) gradient_epilogue<PLANES, PARTS, CE, KD, 4, Slopes>(a, out, u, th, rows, r, acc, rank, box);
        else gradient_epilogue<PLANES, PARTS, CE, KD, 0, Slopes>(a, out, u, th, rows, r, acc, rank, box);
        if (lane == 0 && finished) {  // the unit before: its stores are the older ones
          asm volatile("cp.async.bulk.wait_group %0;" ::"n"(2 * PARTS) : "memory");
          report(finished, finished_tile);
        }
        finished = a.formed + u.piece;
        finished_tile = nullptr;
      } else if (u.mode == kHidden) {
        hidden_epilogue(&prog.dh, u, th, rows, acc, rank, box);
        finished = a.used + u.piece;
        finished_tile = tile;
      } else {
        // G has been read, and nothing in the launch waits for dW itself.
        if (lane == 0) report(a.used + u.piece, nullptr);
        weight_epilogue<PLANES, Slopes && PLANES == 1 && PARTS == 1>(a, prog, u, th, factor, acc, rank, box);
      }
      give_back();
    }
    count_finished();
    if (lane == 0) {
      report(nullptr, nullptr);
      store_wait();
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (*given_up) {  // let the copies and products in flight end before the CTA's memory goes
    const uint64_t begin = timer_ns();
    while (timer_ns() - begin < 2000000) __nanosleep(1000);
  }
  cluster_sync();
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int PLANES, int PARTS, bool CE, bool KD, bool Slopes = false>
cudaError_t launch(const Args& a, const Program& prog, int device, int sms, cudaStream_t s) {
  auto* kernel = products_kernel<PLANES, PARTS, CE, KD, Slopes>;
  // Once per device (a race only does it twice): the kernel's shared memory, and
  // a check that the register shares of its warps do not exceed what a launch
  // brings.
  static std::atomic<bool> ready[64];
  if (device < 0 || device >= 64 || !ready[device].load(std::memory_order_acquire)) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs * kThreads < 128 * kRegsCopies + 256 * kRegsEpilogue) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
    if (e != cudaSuccess) return e;
    if (device >= 0 && device < 64) ready[device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(unsigned(sms / 2 * 2));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSharedBytes;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a, prog);
}

}  // namespace

template <int PLANES, int PARTS>
static cudaError_t launch_terms(const Args& a, const Program& prog, int device, int sms, cudaStream_t s) {
  if (a.kind >= kPolicy) return launch<PLANES, PARTS, true, false, true>(a, prog, device, sms, s);
  if (!a.has_kd) return launch<PLANES, PARTS, true, false>(a, prog, device, sms, s);
  return a.has_ce ? launch<PLANES, PARTS, true, true>(a, prog, device, sms, s)
                  : launch<PLANES, PARTS, false, true>(a, prog, device, sms, s);
}

cudaError_t launch_products(const Args& a, const Program& prog, int device, int sms, cudaStream_t s) {
  if (a.planes == 3) return launch_terms<3, 3>(a, prog, device, sms, s);
  // The forward pass forms no G: one kernel serves it for any number of rows.
  return a.parts == 2 && !prog.forward ? launch_terms<1, 2>(a, prog, device, sms, s)
                                       : launch_terms<1, 1>(a, prog, device, sms, s);
}

}  // namespace zl
