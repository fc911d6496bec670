// Causal attention of packed prompts of different lengths, on sm_103a.
//
//   S = Q K^T,  P = 2^(S c - m),  O = P V / sum P      (c = scale log2 e)
//
// per tile of up to 128 query rows and per block of 128 keys: 4 d operations a
// (query, key) pair against 4 d / 128 bytes from L2, so the tensor cores bound
// it from a few hundred keys a query on, and the chain of one block's steps
// bounds short prompts.
//
// Tiles.  A tile's rows are `tokens` consecutive tokens of one sequence times
// `heads` query heads of one KV head (row = token * heads + head): K and V are
// loaded once for all of them, and a prompt of 40 tokens fills two tiles of 32
// tokens x 4 heads where four tiles of one head each would be a third full.
// heads is the largest divisor of the group up to 16 that leaves at most 3 of
// the 128 rows unused (7 heads: 18 tokens, 126 rows).
//
// Schedule.  One CTA per processor runs items: a tile, or a range of its key
// blocks.  A first, one-CTA launch reads the lengths (a captured call follows
// them) and either
//   lists the tiles, those with most key blocks first (a counting sort), for the
//   CTAs to take from a counter; KV head by KV head where the keys and values of
//   all heads would not stay in L2: whole prompts, whose short tiles make an even
//   end; or,
//   where sequences have more keys than queries, cuts all blocks into equal
//   shares, a CTA each; tiles at a share's end are cut, their ranges leave their
//   reference, sums and unnormalised output, and a third launch joins them in key
//   order.  Head groups go round by round, so that a round's keys and values stay
//   in L2: two chunks of 509 tokens behind 44K and 65K, 64/8 heads: 1.36 ms, against
//   1.43 from the counter (512 items of two lengths do not divide by 152) and
//   1.53 with rounds of 100 MB instead of 50 (all three before the last steps below).
//   (The choice goes by the tensors' sizes, total keys against total queries: it is
//   made on the host, where the lengths are not known.)
// Where every tile gets a CTA of its own the CTAs find their tiles themselves and
// there is no first launch.
//
// Roles of the 24 warps: 0 producer (items, Q, K; it looks items up ahead and
// loads the next one's Q while this one's K blocks are on their way), 1 issues
// Q K^T into one of two S buffers of tensor memory, 2 producer of V, 3 issues
// P V (P in columns of its own, O accumulates in tensor memory), 4-19 softmax:
// four column groups of four warps, a thread has one row and a quarter of its
// columns, which it has in registers before it works on them, so that the S buffer
// is free again; 20-23 output: a thread has a row of O.  Registers are dealt out by
// role.
//
// Shared memory bounds d = 128: a block's Q K^T would read 64 KB there (8 KB a step
// of 64 cycles, as much as there is), P V reads 32 KB and the copies write 64 KB,
// 1250 cycles at 128 bytes each where the products take 1024.  So the output warps,
// idle until an item's end, copy the Q of items of four blocks or more into tensor
// memory, where Q K^T reads it from then on (blocks before that take it from shared
// memory).  That leaves 64 columns for P: P V of a block has to be done before the
// next block's P is stored.  d = 64, bound by softmax, has two P buffers instead.
//
// Softmax.  The reference m of a row is its maximum over the item's first
// block, exchanged once between the groups; later weights may pass 1 and m
// cancels in O / l.  bf16 has fp32's exponents, so that is exact until a sum
// passes 2^126.  The exponents S c - m are single fused operations, whose product is
// not rounded as m is: a maximum's own weight is 2 to the rounding of m, which a
// score of 2^30 takes out of the range.  An item with a row whose sum is not between
// 2^-60 and 2^126 is done again behind the others: first Q K^T alone for the rows'
// true maxima, then with these as m, large ones taken from the scores before the product
// with c, so that a maximum weighs 1 whatever its size.  It costs 1.5 times an item,
// whatever the values, and nothing on the common path.  Where O overflows all the same
// (values near the end of fp32's range), it is done once more, with exponents less by
// log2 of the keys and one, so that no sum of weights passes 1.
//
// The weights are rounded to bf16 for the tensor cores.  The sum that divides O adds
// the rounded ones, in fp32: a row of one dominant key gives its value exactly,
// wherever in the row the key is (a weight of 2^(s - m) behind the first block is no
// power of two), where a sum of unrounded ones would leave the rounding, up to 2^-8,
// in the output.  The log-sum-exp, where it is asked for, adds the unrounded ones.
//
// Masked places.  Scores of keys that a row does not see become -infinity
// whatever they are.  Their values meet weights of 0 in the tensor core, which
// infinities and NaN survive: a row whose O is not finite has its item done again
// too, with such elements of V zeroed in shared memory in the blocks where the
// mask cuts (at most two a tile); the rows that do see them add them back from
// global memory at the end.
//
// Every wait is bounded; on a timeout the CTA flags SA_DEV_TIMEOUT, lets its
// copies and MMAs drain, frees its tensor memory and exits.  No CTA waits for
// another.
//
// Measured (GB300; 1937 TFLOP/s bf16, 1725 sustained under the power cap; masked
// halves of blocks not counted as work; with log-sum-exps; the lower times in runs of
// milliseconds, the others under a load of seconds): a prompt of 32768 tokens, 32/8
// heads, d = 128: 5.6 to 5.75 ms, 1530 to 1560 TFLOP/s, 79 to 81%; 16 prompts of 1 to
// 4096 (29166 tokens in all), 28/4 heads: 427 to 455 us, 1150 to 1230 TFLOP/s, 60 to
// 63%; the chunks above: 1200 to 1305 us, 1400 to 1520 TFLOP/s, 72 to 79%; 24 prompts
// of 1 to 1024, 8/2 heads, d = 64: 28 us; one of 41 tokens: 9.2 us; 16 tokens behind
// 128K keys, 64/8 heads: 125 us of 79 at the copy rate; a prompt of 32768, 32/8 heads,
// d = 64: 4.0 ms, 1090 TFLOP/s, and 3.8 without log-sum-exps.
//
// The long prompt, the 16 and the chunks, step by step: 6030, 468 and 1368 us with P
// over its S in three buffers and Q in shared memory; 5740, 456 and 1305 with the
// layout of now, and a join of few ranges in one latency.  (Two S buffers without the
// copies of Q: 6120, 456 and 1360.)  The two sums of the weights take seven
// instructions a pair of weights, one sum would take five: 5720, 448 and 1303 where two
// took 5785, 460 and 1328.  What is left: P's columns, whose P V must be done before
// the next P is stored, some 1000 cycles from P to that; and items' ends.  Measured and
// not kept (with one sum: 5570, 438 and 1265 without them): pairs of CTAs on tiles of
// 256 rows, which share K and V (6140 and 479: what one CTA signals the other takes 800
// cycles, and the loop crosses three times); P in two halves (5530, but 466); two sets
// of eight softmax warps on every other block each (3% and 1% slower); one arrival a
// warp at P's barrier (0.5% slower); the sums behind P's store (4% slower).
//
// Before that, the 16 prompts: 513 us with softmax warps that also write the output
// and scan V in every block that the mask cuts; 505 with output warps; 482 with the
// output through a buffer of its own instead of the items' Q stages, whose next
// loads then waited for it; 468 with 64 columns of a row in registers at a time
// instead of all.  Items of one block (256 prompts of 32 tokens, 32/8 heads) take as
// long as their output does: 84 us with TMA stores, whose reads of the buffer it
// waited for, 68 with whole rows in registers, 61 with a short loop (67 with two sums).

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "packed.h"
#include "paged.h"
#include "ptx.cuh"

namespace {

using namespace sa_dev;
using sa_packed::Args;

constexpr int kRows = 128;            // query rows of a tile
constexpr int kBK = 128;              // keys of a block
constexpr int kSoftmaxThreads = 512;
constexpr int kOutThreads = 128;
constexpr int kThreads = 128 + kSoftmaxThreads + kOutThreads;
constexpr int kCopyBlocks = 4;        // key blocks of an item whose Q is copied (10: the same)
constexpr int kNI = 4;                // item descriptions in flight
constexpr int kBatch = 512;           // items between two looks at what is to be done again
constexpr int kDirectBlocks = 8;      // key blocks of a tile that is not worth cutting
constexpr int kRounds = 8;            // at most, of head groups, so that a round's keys and values stay in L2
constexpr int kItemCost = 2;          // what an item costs beside its blocks, in blocks
constexpr int kBins = 1024;
constexpr int kScheduleThreads = 1024;
constexpr int kSeqShared = 1024;      // sequences that stay in shared memory
constexpr int kTileRegs = 4;          // tiles of a thread that it remembers
constexpr int kMaxWorkers = 256;      // CTAs that share the work: a tile has no more ranges
constexpr int kFew = 4;               // ranges that a thread joins by itself
constexpr int kJoinRows = 8;          // rows of a CTA's part of a join
constexpr float kWeightless = -3.402823466e38f;   // reference of a range of weights 0 alone
constexpr int64_t kL2Share = int64_t(64) << 20;   // keys and values that stay in L2: half of it

// Registers of a thread by role, together the launch's 768 x 80: the others give up
// what the output warps need.  80 is what 768 threads leave each of a processor's
// 65536 registers, in eights, and so what the compiler has for them; a kernel that
// it gave fewer is refused, as its output warps would wait for ever.
constexpr int kControlRegs = 64, kSoftmaxRegs = 72, kOutRegs = 128;
constexpr int kAllRegs =
    128 * kControlRegs + kSoftmaxThreads * kSoftmaxRegs + kOutThreads * kOutRegs;
static_assert(kAllRegs <= kThreads * (65536 / kThreads / 8 * 8),
              "more than a launch has: it would wait for ever");

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;            // 128-byte column panels
  static constexpr int kQPanel = kRows * 128;
  static constexpr int kKVPanel = kBK * 128;
  static constexpr int kQBytes = kPanels * kQPanel;
  static constexpr int kKVBytes = kPanels * kKVPanel;
  static constexpr int kNQ = 2;
  static constexpr int kNK = D == 128 ? 2 : 4;      // 32 or 16 KB each
  static constexpr int kNV = kNK;
  static constexpr int kNS = 2;
  static constexpr int kNP = D == 128 ? 1 : 2;
  static constexpr bool kCopyQ = D == 128;
  static constexpr int kCols = kBK / 4;             // S columns of a softmax group
  // columns of tensor memory: S, P, Q and O
  static constexpr uint32_t kP = kNS * kBK;
  static constexpr uint32_t kQ = kP + kNP * kBK / 2;
  static constexpr uint32_t kO = kQ + (kCopyQ ? D / 2 : 0);
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kData = kNQ * kQBytes + (kNK + kNV) * kKVBytes + kQPanel;
};

// One tile, or a range of its key blocks, in the schedule.
struct __align__(16) Entry {
  int32_t q0, ntok;       // its tokens (rows of q)
  int32_t kbeg;           // first key of the sequence (row of k)
  int32_t lim0;           // last key, from kbeg, that its first token sees (may be negative)
  int32_t b0, n;          // key blocks
  int32_t slot;           // of a range: its place among the partial states; -1: the whole tile
  int32_t hg;             // with ranges: head group within the round
};

// A tile that was cut.
struct __align__(16) Cut {
  int32_t q0, ntok, hg;
  int32_t slot, ranges;   // partial states, in key order
  int32_t pad[3];
};

struct Header {
  int32_t counter;        // items handed out beyond each CTA's first
  int32_t entries;        // tiles (without ranges)
  int32_t cuts;
  int32_t rounds;         // with ranges: of head groups
};

struct __align__(16) Item {
  Entry e;
  int32_t head0, g;       // first query head, KV head
  int32_t mt;             // blocks before the first masked one
  int32_t pos;            // place in the batch of items
  int32_t careful;        // kClean, kMaxima, kSmall
  int32_t pad[3];
};
enum { kEnd = 0, kMarker = -1 };      // values of e.n that are not items
// Done again: with V cleaned; with true maxima; with weights that add up to 1 at most.
enum { kClean = 1, kMaxima = 2, kSmall = 4 };

struct Shared {
  uint64_t q_full[2], q_empty[2];
  // (k_empty, v_empty: where there are more stages than S buffers; otherwise S done
  // frees the K stage and P V done the V stage, without a commit of its own)
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t q_copied[2];   // items in turn, of those whose Q is copied to tensor memory
  uint64_t o_last;        // a phase per item: its last P V is complete
  uint64_t o_free;        // a phase per item: O is in registers
  uint64_t xch_bar;       // exchanges between the softmax groups
  uint64_t sum_full[2], sum_empty[2];   // items in turn: the rows' sums
  uint64_t batch_done;    // a phase per marker: every output before it is through
  uint64_t drain_qk, drain_pv;
  uint64_t info_full[kNI], info_empty[kNI];
  Item info[kNI];
  Entry ahead[2];         // entries on their way
  int32_t ids[kBatch];    // items of the batch
  uint32_t again[kBatch / 32], maxima[kBatch / 32];   // to be done again; with true maxima
  float xch[2][4][kRows];
  float sum[2][4][kRows];     // per softmax group: sums of rounded weights
  float sum_x[2][4][kRows];   // and of unrounded ones, for the log-sum-exp
  float ref[2][kRows];        // the rows' references
  int64_t row_at[kRows];      // a tile's row in o, from its first
  int32_t any_again;      // one item: it is to be done again
  int32_t bad_v[kNI];     // per description: the item (by its number, from 1) that met
                          // infinities or NaN in masked blocks
  uint32_t tmem_base;
  int abort;
};

// How a CTA gets its work: its one tile, tiles from a counter (those with most
// blocks first), or an equal share of all blocks.
enum { kDirect = 0, kTiles = 1, kRanges = 2 };

struct Params {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  float* lse;
  const Header* header;
  int32_t* counter;
  const Entry* entries;
  const int32_t* first;   // with ranges: [grid + 1] first entry of each CTA's share of a round
  float4* part_o;         // [slot][D / 4][128]
  float4* part_ml;        // [slot][128]: reference, sum, what exponents were less by,
                          // sum of unrounded weights
  int64_t v_st, v_sh, o_st, o_sh;
  int32_t total_q, total_k, batch, Hq, group, tile_heads, tile_tokens;
  int32_t head_groups;    // tiles' heads: Hq / tile_heads
  int32_t mode;           // kDirect, kTiles or kRanges
  int32_t by_head;        // tiles: KV head by KV head
  int32_t round_slots;    // ranges
  float scale_log2;
  int32_t* dev_status;
  uint64_t wait_ns;
};

__device__ __forceinline__ void raise_abort(Shared* sh, const Params& p) {
  atomicOr(p.dev_status, SA_DEV_TIMEOUT);
  *(volatile int*)&sh->abort = 1;
}

__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t issued, uint32_t stages) {
  const uint32_t first = issued > stages ? issued - stages : 0;
  for (uint32_t x = first; x < issued; ++x)
    mbar_wait(&full[x % stages], (x / stages) & 1, nullptr);
}

// Key blocks that a tile's last token sees, one at least (an all-masked block
// then gives the tile's empty rows).
__device__ __forceinline__ int32_t blocks_of(int32_t lim0, int32_t ntok) {
  const int32_t seen = lim0 + ntok;
  return seen <= 0 ? 1 : (seen + kBK - 1) / kBK;
}

__device__ __forceinline__ int32_t clamp_to(int32_t x, int32_t hi) { return min(max(x, 0), hi); }

// ------------------------------------------------------------- the schedule
struct ScheduleParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  Header* header;
  int4* seqs;             // [batch]: first query, queries, first key, keys
  int32_t* tile0;         // [batch] first tile of each sequence
  int32_t* cost0;         // [tiles] cost of the tiles before (ranges)
  Entry* entries;
  int32_t* first;         // [workers + 1]
  Cut* cuts;
  int32_t total_q, total_k, batch, tile_tokens, workers, bin_shift;
  int32_t mode, head_groups;
  int64_t key_bytes;      // of a key and its value, all heads
  int32_t* dev_status;
};

// Rounds of head groups: as many as keep the keys and values of a round that are
// read again within their share of L2, but a divisor of the groups.
__host__ __device__ inline int32_t rounds_of(int64_t bytes, int32_t head_groups) {
  int32_t rounds = 1;
  for (int32_t r = 2; r <= kRounds && bytes / rounds > kL2Share; ++r)
    if (head_groups % r == 0) rounds = r;
  return rounds;
}

// Inclusive scans over a warp.
__device__ __forceinline__ int32_t warp_scan_max(int32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, y);
  }
  return x;
}
__device__ __forceinline__ int32_t warp_scan_sum(int32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The sequence that tile t belongs to: the last one whose first tile is <= t.
__device__ __forceinline__ int32_t seq_of_tile(const int32_t* tile0, int32_t batch, int32_t t) {
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (tile0[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ Entry tile_entry(const int4& s, int32_t tile, int32_t tokens) {
  Entry e;
  const int32_t at = tile * tokens;
  e.q0 = s.x + at;
  e.ntok = min(tokens, s.y - at);
  e.kbeg = s.z;
  e.lim0 = at + s.w - s.y;
  e.b0 = 0;
  e.n = blocks_of(e.lim0, e.ntok);
  e.slot = -1;
  e.hg = 0;
  return e;
}

__global__ void __launch_bounds__(kScheduleThreads)
    schedule_kernel(const __grid_constant__ ScheduleParams p) {
  __shared__ int4 seqs_s[kSeqShared];
  __shared__ int32_t tile0_s[kSeqShared];
  __shared__ int32_t bins[kBins];
  __shared__ int32_t wq[32], wk[32], wt[32];
  __shared__ int32_t slots, cuts;
  __shared__ unsigned long long shared_keys;   // of sequences of several tiles
  launch_dependents();
  wait_dependency();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // sequences: starts that never decrease, and the tiles before each
  int32_t carry_q = clamp_to(p.cu_q[0], p.total_q), carry_k = clamp_to(p.cu_k[0], p.total_k);
  int32_t carry_t = 0;
  bool bad = p.cu_q[0] != carry_q || p.cu_k[0] != carry_k;
  if (tid == 0) {
    slots = cuts = 0;
    shared_keys = 0;
  }
  bins[tid] = 0;
  const bool near = p.batch <= kSeqShared;
  int4* seqs = near ? seqs_s : p.seqs;
  int32_t* tile0 = near ? tile0_s : p.tile0;
  for (int32_t base = 0; base < p.batch; base += kScheduleThreads) {
    const int32_t s = base + tid;
    int32_t q = 0, k = 0;
    if (s < p.batch) {
      const int32_t rq = p.cu_q[s + 1], rk = p.cu_k[s + 1];
      q = clamp_to(rq, p.total_q);
      k = clamp_to(rk, p.total_k);
      bad |= q != rq || k != rk;
    }
    int32_t mq = warp_scan_max(q, lane), mk = warp_scan_max(k, lane);
    if (lane == 31) {
      wq[warp] = mq;
      wk[warp] = mk;
    }
    __syncthreads();
    const int32_t aq = max(warp_scan_max(wq[lane], lane), carry_q);
    const int32_t ak = max(warp_scan_max(wk[lane], lane), carry_k);
    int32_t before_q = __shfl_sync(0xffffffffu, aq, warp ? warp - 1 : 0);
    int32_t before_k = __shfl_sync(0xffffffffu, ak, warp ? warp - 1 : 0);
    if (warp == 0) {
      before_q = carry_q;
      before_k = carry_k;
    }
    const int32_t top_q = __shfl_sync(0xffffffffu, aq, 31);
    const int32_t top_k = __shfl_sync(0xffffffffu, ak, 31);
    mq = max(mq, before_q);
    mk = max(mk, before_k);
    int32_t q0 = __shfl_up_sync(0xffffffffu, mq, 1), k0 = __shfl_up_sync(0xffffffffu, mk, 1);
    if (lane == 0) {
      q0 = before_q;
      k0 = before_k;
    }
    bad |= s < p.batch && (q < q0 || k < k0);
    const int32_t nq = s < p.batch ? mq - q0 : 0;
    const int32_t tiles = (nq + p.tile_tokens - 1) / p.tile_tokens;
    const int32_t st = warp_scan_sum(tiles, lane);
    if (lane == 31) wt[warp] = st;
    __syncthreads();
    const int32_t at = warp_scan_sum(wt[lane], lane) + carry_t;
    int32_t before_t = __shfl_sync(0xffffffffu, at, warp ? warp - 1 : 0);
    if (warp == 0) before_t = carry_t;
    const int32_t all_t = __shfl_sync(0xffffffffu, at, 31);
    if (s < p.batch) {
      seqs[s] = make_int4(q0, nq, k0, mk - k0);
      tile0[s] = before_t + st - tiles;
      if (p.mode == kRanges && tiles > 1) atomicAdd(&shared_keys, (unsigned long long)(mk - k0));
    }
    carry_q = top_q;
    carry_k = top_k;
    carry_t = all_t;
    __syncthreads();
  }
  if (bad) atomicOr(p.dev_status, SA_DEV_BAD_COUNT);
  const int32_t tiles = carry_t;
  auto entry = [&](int32_t t) {
    const int32_t s = seq_of_tile(tile0, p.batch, t);
    return tile_entry(seqs[s], t - tile0[s], p.tile_tokens);
  };
  // exclusive scan of one value a thread, and its total
  auto scan_block = [&](int32_t x, int32_t* all) -> int32_t {
    const int32_t y = warp_scan_sum(x, lane);
    if (lane == 31) wt[warp] = y;
    __syncthreads();
    const int32_t w = warp_scan_sum(wt[lane], lane);
    const int32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    *all = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return (warp ? before : 0) + y - x;
  };

  if (p.mode == kTiles) {
    // most blocks first: a counting sort of the tiles
    auto bin_of = [&](int32_t n) { return kBins - 1 - min(n >> p.bin_shift, kBins - 1); };
    Entry mine[kTileRegs];
#pragma unroll
    for (int i = 0; i < kTileRegs; ++i) {
      const int32_t t = tid + i * kScheduleThreads;
      if (t < tiles) {
        mine[i] = entry(t);
        atomicAdd(&bins[bin_of(mine[i].n)], 1);
      }
    }
    for (int32_t t = tid + kTileRegs * kScheduleThreads; t < tiles; t += kScheduleThreads)
      atomicAdd(&bins[bin_of(entry(t).n)], 1);
    __syncthreads();
    int32_t all;
    bins[tid] = scan_block(bins[tid], &all);
    __syncthreads();
    auto put = [&](const Entry& e) { p.entries[atomicAdd(&bins[bin_of(e.n)], 1)] = e; };
#pragma unroll
    for (int i = 0; i < kTileRegs; ++i)
      if (tid + i * kScheduleThreads < tiles) put(mine[i]);
    for (int32_t t = tid + kTileRegs * kScheduleThreads; t < tiles; t += kScheduleThreads)
      put(entry(t));
    if (tid == 0) *p.header = Header{0, tiles, 0, 1};
    return;
  }

  const int32_t rounds = rounds_of(int64_t(shared_keys) * p.key_bytes, p.head_groups);
  const int32_t round_groups = p.head_groups / rounds;
  // Ranges: the blocks of a round's tiles (head groups one behind the other),
  // an item's cost before each tile's, in equal shares.  A share's end inside a
  // tile cuts it, unless one side would have few blocks.  (All below 2^31.)
  int32_t cost = 0;
  for (int32_t base = 0; base < tiles; base += kScheduleThreads) {
    const int32_t t = base + tid;
    int32_t all;
    const int32_t before = scan_block(t < tiles ? entry(t).n + kItemCost : 0, &all);
    if (t < tiles) p.cost0[t] = cost + before;
    cost += all;
  }
  __syncthreads();
  const int32_t share =
      max((cost * round_groups + p.workers - 1) / p.workers, 2 * kItemCost + 2);
  const int32_t least = min(share / 8 + 1, 4);
  // first block of tile [at, at + n + kItemCost) that belongs to share k or a later one
  auto cut_at = [&](int32_t at, int32_t n, int32_t k) -> int32_t {
    const int32_t b = k * share - at - kItemCost;
    return b < least ? 0 : n - b < least ? n : b;
  };
  int32_t placed = 0;
  for (int32_t hg = 0; hg < round_groups; ++hg) {
    for (int32_t base = 0; base < tiles; base += kScheduleThreads) {
      const int32_t t = base + tid;
      Entry e;
      int32_t n = 0, ranges = 0, at = 0, k0 = 0, k1 = -1;
      if (t < tiles) {
        e = entry(t);
        e.hg = hg;
        n = e.n;
        at = hg * cost + p.cost0[t];
        k0 = at / share;
        k1 = (at + n + kItemCost - 1) / share;
        for (int32_t k = k0; k <= k1; ++k) {
          const int32_t first = k == k0 ? 0 : cut_at(at, n, k);
          const int32_t end = k == k1 ? n : cut_at(at, n, k + 1);
          ranges += end > first;
        }
      }
      int32_t all;
      int32_t x = placed + scan_block(ranges, &all);
      placed += all;
      if (t >= tiles) continue;
      int32_t slot = -1;
      if (ranges > 1) {
        slot = atomicAdd(&slots, ranges);
        p.cuts[atomicAdd(&cuts, 1)] = Cut{e.q0, e.ntok, e.hg, slot, ranges, {0, 0, 0}};
      }
      for (int32_t k = k0; k <= k1; ++k) {
        const int32_t first = k == k0 ? 0 : cut_at(at, n, k);
        const int32_t end = k == k1 ? n : cut_at(at, n, k + 1);
        if (end <= first) continue;
        e.b0 = first;
        e.n = end - first;
        e.slot = slot < 0 ? -1 : slot++;
        atomicAdd(&bins[k], 1);              // entries of share k
        p.entries[x++] = e;
      }
    }
  }
  __syncthreads();
  int32_t all;
  const int32_t before = scan_block(tid < p.workers ? bins[tid] : 0, &all);
  if (tid <= p.workers) p.first[tid] = before;
  if (tid == 0) *p.header = Header{0, tiles, cuts, rounds};
}

// Joins the ranges of the tiles that were cut, in key order: a range's weight is
// 2^(m + log2 l), relative to the largest m first, as m may be too large for a sum's
// logarithm to change it; its output is divided by its own sum first, as that may be
// as large as fp32 goes.  A CTA takes 8 rows of a tile, a thread four columns of one:
// the weights of a row's ranges once, to shared memory, then the sums over ranges,
// eight loads under way.  Of up to kFew ranges a thread loads and weighs all of its
// row by itself, in one latency (the chunks of the header: 65 us with shared
// memory's barriers between, 40 so, before it compared references first).
struct JoinParams {
  const Header* header;
  const Cut* cuts;
  const float4* part_o;
  const float4* part_ml;
  __nv_bfloat16* o;
  float* lse;
  int64_t o_st, o_sh;
  int32_t Hq, tile_heads, head_groups, round_slots;
};

template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4)
    join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int kThreadsJ = kJoinRows * D / 4;
  constexpr int kUnits = kRows / kJoinRows;
  // a range's weight, and what its output is divided by, inverted
  __shared__ float2 weight[kMaxWorkers][kJoinRows];
  __shared__ float top_m[kThreadsJ / 32][kJoinRows], top[kThreadsJ / 32][kJoinRows];
  __shared__ float2 total[kThreadsJ / 32][kJoinRows];
  launch_dependents();
  wait_dependency();
  const int32_t rounds = __ldcg(&p.header->rounds);
  const int64_t units = int64_t(__ldcg(&p.header->cuts)) * rounds * kUnits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t c = u / kUnits;
    const int32_t round = int32_t(c % rounds);
    const int4* at = reinterpret_cast<const int4*>(&p.cuts[c / rounds]);
    const int4 a0 = __ldcg(at), a1 = __ldcg(at + 1);
    const Cut cut{a0.x, a0.y, a0.z, a0.w, a1.x, {0, 0, 0}};
    const int row0 = int(u % kUnits) * kJoinRows;
    if (row0 / p.tile_heads >= cut.ntok) continue;           // no query in these rows
    const int64_t slot0 = int64_t(round) * p.round_slots + cut.slot;
    const int r = tid % kJoinRows, row = row0 + r;
    const int c4 = tid / kJoinRows;
    const float4* ml = p.part_ml + slot0 * kRows + row;
    const float4* po = p.part_o + (slot0 * (D / 4) + c4) * kRows + row;
    // the largest reference, the largest logarithm of a range's weight beside it, and
    // the sums of rounded and of unrounded weights
    float m = -INFINITY, e = -INFINITY, l = 0.f, lx = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // a range's weight f, and what its output is divided by, inverted
    auto add = [&](const float4& z, float f, float inv) {
      if (inv == 0.f) return;
      acc.x = fmaf(f, z.x * inv, acc.x);
      acc.y = fmaf(f, z.y * inv, acc.y);
      acc.z = fmaf(f, z.z * inv, acc.z);
      acc.w = fmaf(f, z.w * inv, acc.w);
    };
    // (a sum of 0: the row sees no key of this range)
    auto log_of = [&](const float4& y) {
      return y.y == 0.f ? -INFINITY : (y.x - m) + (y.z + log2f(y.y));
    };
    auto inverse = [](float x) { return x == 0.f ? 0.f : 1.f / x; };
    // (every reference -infinity, or NaN: so is the result)
    auto weigh = [&](float x, float inv) { return inv == 0.f ? 0.f : ex2(x - e); };
    if (cut.ranges <= kFew) {
      float4 y[kFew], z[kFew];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        y[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        z[i] = acc;
        if (i >= cut.ranges) continue;
        y[i] = __ldcg(ml + int64_t(i) * kRows);
        z[i] = __ldcg(po + int64_t(i) * (D / 4) * kRows);
      }
#pragma unroll
      for (int i = 0; i < kFew; ++i) m = fmaxf(m, y[i].x);
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        y[i].x = log_of(y[i]);
        y[i].y = inverse(y[i].y);
        e = fmaxf(e, y[i].x);
      }
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        l += y[i].x = weigh(y[i].x, y[i].y);
        lx = fmaf(y[i].x, y[i].w * y[i].y, lx);
      }
      const float inv = inverse(l);                          // sees no key at all: 0
#pragma unroll
      for (int i = 0; i < kFew; ++i) add(z[i], y[i].x * inv, y[i].y);
    } else {
      // the references and sums of this row's ranges: a thread has every
      // (threads / 8)-th of them
      auto largest = [&](float x, float (&of)[kThreadsJ / 32][kJoinRows]) {
        // lanes 8 apart have the same row
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        if (lane < kJoinRows) of[warp][lane] = x;
        __syncthreads();
        x = of[0][r];
#pragma unroll
        for (int w = 1; w < kThreadsJ / 32; ++w) x = fmaxf(x, of[w][r]);
        return x;
      };
      for (int32_t i = tid / kJoinRows; i < cut.ranges; i += kThreadsJ / kJoinRows)
        m = fmaxf(m, __ldcg(ml + int64_t(i) * kRows).x);
      m = largest(m, top_m);
      for (int32_t i = tid / kJoinRows; i < cut.ranges; i += kThreadsJ / kJoinRows) {
        const float4 y = __ldcg(ml + int64_t(i) * kRows);
        weight[i][r] = make_float2(log_of(y), inverse(y.y));
        e = fmaxf(e, weight[i][r].x);
      }
      e = largest(e, top);
      for (int32_t i = tid / kJoinRows; i < cut.ranges; i += kThreadsJ / kJoinRows) {
        const float w = weigh(weight[i][r].x, weight[i][r].y);
        l += weight[i][r].x = w;
        lx = fmaf(w, __ldcg(ml + int64_t(i) * kRows).w * weight[i][r].y, lx);
      }
#pragma unroll
      for (int o = 8; o <= 16; o <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        lx += __shfl_xor_sync(0xffffffffu, lx, o);
      }
      if (lane < kJoinRows) total[warp][lane] = make_float2(l, lx);
      __syncthreads();
      l = lx = 0.f;
#pragma unroll
      for (int w = 0; w < kThreadsJ / 32; ++w) {
        l += total[w][r].x;
        lx += total[w][r].y;
      }
      const float inv = inverse(l);
#pragma unroll 8
      for (int32_t i = 0; i < cut.ranges; ++i)
        add(__ldcg(po + int64_t(i) * (D / 4) * kRows), weight[i][r].x * inv, weight[i][r].y);
      __syncthreads();                                       // before the weights change
    }
    if (l == 0.f && m == kWeightless) acc.x = acc.y = acc.z = acc.w = NAN;
    const int tok = row / p.tile_heads, head = row - tok * p.tile_heads;
    if (tok < cut.ntok) {
      const int64_t t = int64_t(cut.q0) + tok;
      const int32_t h = (round * (p.head_groups / rounds) + cut.hg) * p.tile_heads + head;
      *reinterpret_cast<uint2*>(p.o + t * p.o_st + h * p.o_sh + c4 * 4) = make_uint2(
          pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
      if (p.lse && c4 == 0)
        p.lse[t * p.Hq + h] =
            l == 0.f ? -INFINITY : (m + (e + log2f(lx))) * 0.6931471805599453f;
    }
  }
}

// A direct CTA's tile: the warp walks the sequences.  False: there is none.
__device__ __forceinline__ bool find_tile(const Params& p, int32_t tile, int lane, Entry* out) {
  int32_t carry_q = clamp_to(__ldcg(p.cu_q), p.total_q), carry_k = clamp_to(__ldcg(p.cu_k), p.total_k);
  int32_t carry_t = 0;
  bool bad = __ldcg(p.cu_q) != carry_q || __ldcg(p.cu_k) != carry_k;
  bool found = false;
  for (int32_t base = 0; base < p.batch && !found; base += 32) {
    const int32_t s = base + lane;
    int32_t q = 0, k = 0;
    if (s < p.batch) {
      const int32_t rq = __ldcg(&p.cu_q[s + 1]), rk = __ldcg(&p.cu_k[s + 1]);
      q = clamp_to(rq, p.total_q);
      k = clamp_to(rk, p.total_k);
      bad |= q != rq || k != rk;
    }
    const int32_t mq = max(warp_scan_max(q, lane), carry_q);
    const int32_t mk = max(warp_scan_max(k, lane), carry_k);
    int32_t q0 = __shfl_up_sync(0xffffffffu, mq, 1), k0 = __shfl_up_sync(0xffffffffu, mk, 1);
    if (lane == 0) {
      q0 = carry_q;
      k0 = carry_k;
    }
    bad |= s < p.batch && (q < q0 || k < k0);
    const int32_t nq = s < p.batch ? mq - q0 : 0;
    const int32_t tiles = (nq + p.tile_tokens - 1) / p.tile_tokens;
    const int32_t after = carry_t + warp_scan_sum(tiles, lane);
    const uint32_t here = __ballot_sync(0xffffffffu, tile >= after - tiles && tile < after);
    if (here) {
      const int src = __ffs(here) - 1;
      int4 seq;
      seq.x = __shfl_sync(0xffffffffu, q0, src);
      seq.y = __shfl_sync(0xffffffffu, nq, src);
      seq.z = __shfl_sync(0xffffffffu, k0, src);
      seq.w = __shfl_sync(0xffffffffu, mk - k0, src);
      *out = tile_entry(seq, tile - __shfl_sync(0xffffffffu, after - tiles, src), p.tile_tokens);
      found = true;
    }
    carry_q = __shfl_sync(0xffffffffu, mq, 31);
    carry_k = __shfl_sync(0xffffffffu, mk, 31);
    carry_t = __shfl_sync(0xffffffffu, after, 31);
  }
  if (bad) atomicOr(p.dev_status, SA_DEV_BAD_COUNT);
  return found;
}

// What an item's exponents are less by, so that no sum of weights passes 1.
__device__ __forceinline__ float less_of(int32_t blocks) {
  return float(33 - __clz(blocks * kBK));
}

// Whether any of the two bf16 values is an infinity or NaN (an exponent of all ones).
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// kLse: the log-sum-exps are written.  kOne: each CTA has its one tile.
template <int D, bool kLse, bool kOne>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ CUtensorMap tq,
                            const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv,
                            const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.dev_status, SA_DEV_BAD_LAUNCH);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sK = sQ + C::kNQ * C::kQBytes;
  uint8_t* sV = sK + C::kNK * C::kKVBytes;
  uint8_t* sO = sV + C::kNV * C::kKVBytes;       // a panel of an output tile, 4 KB a warp
  Shared* sh = reinterpret_cast<Shared*>(sO + C::kQPanel);
  volatile int* abort = &sh->abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh->q_full[s], 1);
      mbar_init(&sh->q_empty[s], 1 + kOutThreads / 32);
      mbar_init(&sh->q_copied[s], kOutThreads / 32);
      mbar_init(&sh->sum_full[s], kSoftmaxThreads);
      mbar_init(&sh->sum_empty[s], kOutThreads);
    }
    for (int s = 0; s < C::kNK; ++s) {
      mbar_init(&sh->k_full[s], 1);
      mbar_init(&sh->k_empty[s], 1);
      mbar_init(&sh->v_full[s], 1);
      mbar_init(&sh->v_empty[s], 1);
    }
    for (int s = 0; s < C::kNS; ++s) {
      mbar_init(&sh->s_full[s], 1);
      mbar_init(&sh->s_empty[s], kSoftmaxThreads / 32);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh->p_full[s], kSoftmaxThreads);
      mbar_init(&sh->pv_done[s], 1);
    }
    for (int s = 0; s < kNI; ++s) {
      mbar_init(&sh->info_full[s], 1);
      mbar_init(&sh->info_empty[s], 3 + (kSoftmaxThreads + kOutThreads) / 32);
    }
    mbar_init(&sh->o_last, 1);
    mbar_init(&sh->o_free, kOutThreads);
    mbar_init(&sh->xch_bar, kSoftmaxThreads);
    mbar_init(&sh->batch_done, kOutThreads);
    mbar_init(&sh->drain_qk, 1);
    mbar_init(&sh->drain_pv, 1);
    sh->abort = 0;
    for (int s = 0; s < kNI; ++s) sh->bad_v[s] = 0;
    sh->any_again = 0;
    fence_mbar_init();
  }
  for (int x = threadIdx.x; x < kBatch / 32; x += kThreads) sh->again[x] = sh->maxima[x] = 0;
  if (threadIdx.x < kRows) {
    const int tok = int(threadIdx.x) / p.tile_heads;
    sh->row_at[threadIdx.x] = tok * p.o_st + (int(threadIdx.x) - tok * p.tile_heads) * p.o_sh;
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  // Behind the only item of a CTA a role sees by itself whether it is to be done
  // again, 0.5 us before the producer could tell it.  (With a check like this
  // where a CTA has many items, the roles' loops came out 1 to 4% slower.)
  uint32_t marks = 0;
  auto go_on = [&](bool* ok) -> bool {
    if (!kOne) return true;
    *ok = wait_all(&sh->batch_done, marks++ & 1, abort, p.wait_ns);
    return *ok && *(volatile int32_t*)&sh->any_again;
  };

  // (the roles in this order: up to 2% faster than with the producers first)
  if (warp >= 20) {
    // ------------------------------------------------- output
    registers_inc<kOutRegs>();
    const int row = (warp & 3) * 32 + lane;       // a thread's row, whole
    const int tok = row / p.tile_heads;
    const int head = row - tok * p.tile_heads;
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16) + C::kO;
    uint32_t ii = 0, qi = 0, copies = 0;
    bool ok = true;
    for (;; ++ii) {
      const uint32_t slot = ii % kNI;
      if (!wait_all(&sh->info_full[slot], (ii / kNI) & 1, abort, p.wait_ns)) {
        ok = false;
        break;
      }
      const Item& it = sh->info[slot];            // released at the end
      const int32_t n = it.e.n;
      if (n <= 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
        if (n == kEnd) break;
        mbar_arrive(&sh->batch_done);
        if (!go_on(&ok)) break;
        continue;
      }
      // Q of a longer item into tensor memory, where Q K^T reads it faster from then
      // on (the last item's is done: its output is)
      const uint32_t w = qi & 1;
      if (C::kCopyQ && n >= kCopyBlocks) {
        if (!wait_all(&sh->q_full[w], (qi >> 1) & 1, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint8_t* from = sQ + w * C::kQBytes + row * 128;
#pragma unroll 1
        for (int s = 0; s < C::kPanels; ++s) {
          uint32_t r[32];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint4 y =
                *reinterpret_cast<const uint4*>(from + s * C::kQPanel + ((x ^ (row & 7)) << 4));
            r[4 * x] = y.x;
            r[4 * x + 1] = y.y;
            r[4 * x + 2] = y.z;
            r[4 * x + 3] = y.w;
          }
          tmem_st32(lanes - C::kO + C::kQ + 32 * s, r);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_copied[copies & 1]);
        ++copies;
      }
      if (lane == 0) mbar_arrive(&sh->q_empty[w]);
      if (!wait_all(&sh->sum_full[w], (qi >> 1) & 1, abort, p.wait_ns)) {
        ok = false;
        break;
      }
      float l = (sh->sum[w][0][row] + sh->sum[w][1][row]) +
                (sh->sum[w][2][row] + sh->sum[w][3][row]);
      float lx = kLse ? (sh->sum_x[w][0][row] + sh->sum_x[w][1][row]) +
                            (sh->sum_x[w][2][row] + sh->sum_x[w][3][row])
                      : 0.f;
      float m = sh->ref[w][row];
      mbar_arrive(&sh->sum_empty[w]);
      const int32_t lim = it.e.lim0 + tok;
      const bool live = tok < it.e.ntok;                     // a query of the tile
      const bool some = lim >= it.e.b0 * kBK;                // that sees a key of the range
      const bool whole = it.e.slot < 0;
      const float less = it.careful & kSmall ? less_of(n) : 0.f;
      // (a NaN is not in range either)
      const bool in_range = l >= 0x1p-60f && l <= 0x1p126f;
      if (!some) {
        l = whole ? 1.f : 0.f;
        lx = 0.f;
        m = -INFINITY;
      }
      const float inv = whole ? 1.f / l : 1.f;
      float4* part = p.part_o + int64_t(whole ? 0 : it.e.slot) * (D / 4) * kRows + row;
      const bool blank = __any_sync(0xffffffffu, !some);     // rarely: a branch
      // (the softmax warps may be two items ahead, but not at the next item of this
      // description's place)
      const bool dirty =
          it.careful && *(volatile int32_t*)&sh->bad_v[slot] == int32_t(qi + 1);
      float osum = 0.f, osum2 = 0.f;
      if (!wait_all(&sh->o_last, qi & 1, abort, p.wait_ns)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int rows = it.e.ntok * p.tile_heads;
      __nv_bfloat16* o = p.o + int64_t(it.e.q0) * p.o_st + int64_t(it.head0) * p.o_sh +
                         (lane & 7) * 8;
      uint8_t* mine = sO + (row - lane) * 128;
      // 32 columns at a time, in a short loop: five roles share a scheduler's
      // instruction cache
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(lanes + 32 * c, r);
        tmem_ld_wait(r);
        if (c == D / 32 - 1) {
          // O is read: the next item's first P V may overwrite it
          tc_fence_before();
          mbar_arrive(&sh->o_free);
        }
        if (blank && !some) {
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 32; x += 2)
          add2(osum, osum2, __uint_as_float(r[x]), __uint_as_float(r[x + 1]));
        if (!whole) {
          // a range's columns, as they are, to its slot
          if (live) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              part[(8 * c + x) * kRows] =
                  make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]),
                              __uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3]));
          }
          continue;
        }
        // through the warp's buffer, 64 columns at a time (16-byte chunks of a row
        // are swapped by its number, so that neither side meets bank conflicts)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t ob[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float a0, a1;
            mul2(a0, a1, __uint_as_float(r[8 * x + 2 * y]),
                 __uint_as_float(r[8 * x + 2 * y + 1]), inv, inv);
            ob[y] = pack_bf16x2(a0, a1);
          }
          *reinterpret_cast<uint4*>(mine + lane * 128 +
                                    ((((c & 1) * 4 + x) ^ (lane & 7)) << 4)) =
              make_uint4(ob[0], ob[1], ob[2], ob[3]);
        }
        if (!(c & 1)) continue;
        // out in whole 128-byte rows: 8 lanes a row
        __syncwarp();
#pragma unroll 4
        for (int x = 0; x < 8; ++x) {
          const int y = 4 * x + (lane >> 3), at = row - lane + y;
          if (at < rows)
            *reinterpret_cast<uint4*>(o + sh->row_at[at] + 32 * (c - 1)) =
                *reinterpret_cast<const uint4*>(mine + y * 128 + (((lane & 7) ^ (y & 7)) << 4));
        }
        __syncwarp();
      }
      if (dirty) {
        // what clean_v took out of the values that a row sees comes back, now that
        // the row is written
        __syncwarp();
        if (live && some) {
          const __nv_bfloat16* v = p.v + it.g * p.v_sh;
          __nv_bfloat16* mine_o = p.o + int64_t(it.e.q0) * p.o_st + int64_t(it.head0) * p.o_sh +
                                  sh->row_at[row];
          const int32_t end = min(lim + 1, (it.e.b0 + n) * kBK);
          for (int32_t u = (it.e.b0 + it.mt) * kBK; u < end; ++u)
#pragma unroll 1
            for (int x = 0; x < D; ++x) {
              const float y = __bfloat162float(v[(int64_t(it.e.kbeg) + u) * p.v_st + x]);
              if (fabsf(y) <= 3.4e38f) continue;
              if (whole) {
                mine_o[x] = __float2bfloat16_rn(__bfloat162float(mine_o[x]) + y);
              } else {
                float* at = reinterpret_cast<float*>(&part[(x / 4) * kRows]) + x % 4;
                *at += y;
              }
            }
        }
      }
      // the range that the first pass keeps: the sum from 2^-60 (no weight that counts
      // vanished) to 2^126 (none overflowed) and O finite; the second one's O may
      // overflow
      const bool finite = fabsf(osum + osum2) <= 3.0e38f;
      if (live && some && !(it.careful & kSmall) &&
          (it.careful ? in_range && !finite : !(in_range && finite))) {
        const uint32_t bit = 1u << (it.pos & 31);
        if (kOne) *(volatile int32_t*)&sh->any_again = 1;
        atomicOr(&sh->again[it.pos >> 5], bit);
        if (!in_range) atomicOr(&sh->maxima[it.pos >> 5], bit);
      }
      if (!whole) {
        // (keys of which none weighs anything are not the same as none at all: a row of
        // such ranges alone has no mean)
        if (some && l == 0.f) m = kWeightless;
        if (live) p.part_ml[int64_t(it.e.slot) * kRows + row] = make_float4(m, l, less, lx);
      } else if (kLse && live) {
        p.lse[(int64_t(it.e.q0) + tok) * p.Hq + it.head0 + head] =
            some ? (m + (less + log2f(lx))) * 0.6931471805599453f : -INFINITY;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
      ++qi;
    }
    if (!ok) raise_abort(sh, p);
    tmem_ld_wait();
    tmem_st_wait();
    tc_fence_before();
  } else if (warp >= 4 && warp < 20) {
    // ------------------------------------------------- softmax groups
    registers_dec<kSoftmaxRegs>();
    const int grp = (warp - 4) >> 2;              // column group 0..3
    const int quarter = warp & 3;                 // TMEM lane quarter of this warp
    const int row = quarter * 32 + lane;
    const int tok = row / p.tile_heads;           // token of this row's query
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + grp * C::kCols;
    const float c = p.scale_log2;
    uint32_t ii = 0, qi = 0, xn = 0;              // xn: uses of the exchange buffer
    uint32_t sb = 0, vb = 0;                      // S blocks; those with P V
    bool ok = true;

    // The largest of this thread's scores.
    auto row_max = [&](const float (&s)[C::kCols]) {
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int x = 4; x + 8 <= C::kCols; x += 8)
#pragma unroll
        for (int a = 0; a < 4; ++a) mx[a] = max3(mx[a], s[x + a], s[x + 4 + a]);
#pragma unroll
      for (int a = 0; a < 4; ++a) mx[a] = fmaxf(mx[a], s[C::kCols - 4 + a]);
      return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
    };
    // The row's maximum from the groups' ones.  Use xn writes buffer xn & 1:
    // every thread read use xn-2 before it posted use xn-1, which this thread
    // saw complete.
    auto exchange_max = [&](float mx, float* out) -> bool {
      float* xb = &sh->xch[xn & 1][0][0];
      xb[grp * 128 + row] = mx;
      mbar_arrive(&sh->xch_bar);
      if (!wait_all(&sh->xch_bar, xn & 1, abort, p.wait_ns)) return false;
      *out = max3(fmaxf(xb[row], xb[128 + row]), xb[256 + row], xb[384 + row]);
      ++xn;
      return true;
    };
    // S into registers; its buffer may be written again
    auto load_s = [&](float (&s)[C::kCols]) {
      uint32_t sr[32];
      static_assert(C::kCols == 32, "group width");
      tmem_ld32(lanes + (sb & 1) * kBK, sr);
      tmem_ld_wait(sr);
#pragma unroll
      for (int x = 0; x < 32; ++x) s[x] = __uint_as_float(sr[x]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->s_empty[sb & 1]);
    };
    static_assert(C::kNS == 2, "S buffers in turn");
    // Infinities and NaN of a V block that the mask cuts become 0 in shared
    // memory (this thread's share of the stage); the item is marked.
    auto clean_v = [&](uint32_t item, uint32_t slot) {
      uint8_t* stage = sV + (vb % C::kNV) * C::kKVBytes;
      const int x = (warp - 4) * 32 + lane;
#pragma unroll 1
      for (int i = 0; i < C::kKVBytes / 16 / kSoftmaxThreads; ++i) {
        uint4* at = reinterpret_cast<uint4*>(stage) + x + i * kSoftmaxThreads;
        uint4 w = *at;
        uint32_t b0 = not_finite(w.x), b1 = not_finite(w.y), b2 = not_finite(w.z),
                 b3 = not_finite(w.w);
        if (b0 | b1 | b2 | b3) {
          // 0x8000 in each bad half -> 0xffff
          auto wipe = [](uint32_t v, uint32_t b) { return v & ~((b >> 15) * 0xffffu); };
          *at = make_uint4(wipe(w.x, b0), wipe(w.y, b1), wipe(w.z, b2), wipe(w.w, b3));
          *(volatile int32_t*)&sh->bad_v[slot] = int32_t(item + 1);
          fence_proxy_async_smem();
        }
      }
    };

    for (;; ++ii) {
      const uint32_t slot = ii % kNI;
      if (!wait_all(&sh->info_full[slot], (ii / kNI) & 1, abort, p.wait_ns)) {
        ok = false;
        break;
      }
      const int32_t n = sh->info[slot].e.n, mt = sh->info[slot].mt;
      // last visible column of this thread's quarter of the first block
      const int32_t vis0 =
          sh->info[slot].e.lim0 + tok - sh->info[slot].e.b0 * kBK - grp * C::kCols;
      const int32_t careful = sh->info[slot].careful;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
      if (n == kEnd) break;
      if (n == kMarker) {
        if (!go_on(&ok)) break;
        continue;
      }
      // the reference; with true maxima, what scores are less by before the product with
      // c, and what exponents add after it
      float m_used = -INFINITY, top = 0.f, last = 0.f;
      if (careful & kMaxima) {
        // the rows' maxima over all blocks, without P V
        float mx = -INFINITY;
        for (int32_t t = 0; t < n; ++t) {
          if (!wait_all(&sh->s_full[sb & 1], (sb >> 1) & 1, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float s[C::kCols];
          load_s(s);
#pragma unroll
          for (int x = 0; x < C::kCols; ++x)
            if (t >= mt && x > vis0 - t * kBK) s[x] = -INFINITY;
          mx = fmaxf(mx, row_max(s));
          ++sb;
        }
        if (!ok) break;
        if (!exchange_max(mx, &top)) {
          ok = false;
          break;
        }
        m_used = top * c;
        last = careful & kSmall ? -less_of(n) : 0.f;
        // (below 2^20 the reference's rounding leaves 2^-5 of an exponent at most, and a
        // row that is done again for another's sake keeps its bits if its maximum was in
        // the first block)
        if (!(careful & kSmall) && fabsf(m_used) <= 0x1p20f) {
          last = -m_used;
          top = 0.f;
        }
        // (no score of the item is above -infinity: no weight above 0)
        if (top == -INFINITY) top = 0.f;
      }
      // the sums of rounded weights and of unrounded ones, in parts
      float sum0 = 0.f, sum1 = 0.f, x0 = 0.f, x1 = 0.f;
      // (a loop of its own for items that are done again: it keeps the others' short)
      auto weigh = [&](auto again) {
        constexpr bool kAgain = decltype(again)::value;
        for (int32_t t = 0; t < n; ++t) {
          if (!wait_all(&sh->s_full[sb & 1], (sb >> 1) & 1, abort, p.wait_ns)) {
            ok = false;
            return;
          }
          tc_fence_after();
          float s[C::kCols];
          load_s(s);
          if (t >= mt) {
            const int32_t vis = vis0 - t * kBK;
#pragma unroll
            for (int x = 0; x < C::kCols; ++x)
              if (x > vis) s[x] = -INFINITY;
            if (kAgain) {
              if (!wait_all(&sh->v_full[vb % C::kNV], (vb / C::kNV) & 1, abort, p.wait_ns)) {
                ok = false;
                return;
              }
              clean_v(qi, slot);
            }
          }
          ++vb;
          if (t == 0 && !(kAgain && (careful & kMaxima))) {
            if (!exchange_max(row_max(s), &m_used)) {
              ok = false;
              return;
            }
            m_used *= c;
          }
          if (kAgain && (careful & kMaxima)) {
#pragma unroll
            for (int x = 0; x < C::kCols; ++x) s[x] -= top;
          }
          {
            uint32_t pk[C::kCols / 2];
            const float nm = kAgain && (careful & kMaxima) ? last : -m_used;
#pragma unroll
            for (int x = 0; x < C::kCols / 2; ++x) {
              float a0, a1;
              fma2(a0, a1, s[2 * x], s[2 * x + 1], c, c, nm, nm);
              a0 = ex2(a0);
              a1 = ex2(a1);
              pk[x] = pack_bf16x2(a0, a1);
              add_bf16x2(sum0, sum1, pk[x]);
              if (kLse) add2(x0, x1, a0, a1);
            }
            // P V of kNP blocks before has read P
            const uint32_t before = vb - 1 - C::kNP;
            if (vb > uint32_t(C::kNP) &&
                !wait_all(&sh->pv_done[before & 1], (before >> 1) & 1, abort, p.wait_ns)) {
              ok = false;
              return;
            }
            tc_fence_after();
            tmem_st16(lanes + C::kP - grp * (C::kCols / 2) + (vb - 1) % C::kNP * (kBK / 2), pk);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh->p_full[(vb - 1) & 1]);
          ++sb;
        }
      };
      if (careful)
        weigh(std::true_type{});
      else
        weigh(std::false_type{});
      if (!ok) break;
      // the sums of this item, once the output warps have read those of the
      // item before the last
      const uint32_t w = qi & 1;
      if (qi >= 2 && !wait_all(&sh->sum_empty[w], ((qi >> 1) - 1) & 1, abort, p.wait_ns)) {
        ok = false;
        break;
      }
      sh->sum[w][grp][row] = sum0 + sum1;
      if (kLse) sh->sum_x[w][grp][row] = x0 + x1;
      if (grp == 0) sh->ref[w][row] = m_used;
      mbar_arrive(&sh->sum_full[w]);
      ++qi;
    }
    if (!ok) raise_abort(sh, p);
    // a role that gave up may have left a tensor-memory access in flight
    tmem_ld_wait();
    tmem_st_wait();
    tc_fence_before();
  } else {
    // (the instruction is a warpgroup's: all its warps execute the same one)
    registers_dec<kControlRegs>();
    if (warp == 0) {
      // ------------------------------------------------- producer: items, Q, K
      if (lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
      }
      wait_dependency();                   // the schedule, and what the inputs come from
      Entry tile0;
      const bool found = kOne &&
                         find_tile(p, int32_t(blockIdx.x) / p.head_groups, lane, &tile0);
      if (lane == 0) {
        const uint64_t pol_kv = l2_policy_evict_last();
        const uint64_t pol_q = l2_policy_evict_first();
        uint32_t ii = 0, qi = 0, kiss = 0;   // descriptions, items and K blocks so far
        // items: the direct CTA's tile, places in the list of tiles times head
        // groups, or the entries of this CTA's share, round by round
        int32_t entries = 0, from = 0, to = 0, round_groups = 0;
        int64_t items = found ? 1 : 0;
        if (p.mode == kTiles) {
          entries = __ldcg(&p.header->entries);
          items = int64_t(entries) * p.head_groups;
        } else if (p.mode == kRanges) {
          from = __ldcg(&p.first[blockIdx.x]);
          to = __ldcg(&p.first[blockIdx.x + 1]);
          const int32_t rounds = __ldcg(&p.header->rounds);
          round_groups = p.head_groups / rounds;
          items = int64_t(to - from) * rounds;
        }
        // An item's entry is copied to shared memory (place x & 1), without waiting;
        // landed() waits for it.
        auto head_of = [&](int32_t id) {
          return p.mode == kRanges ? id / (to - from)          // the round
                 : kOne ? int32_t(blockIdx.x) % p.head_groups
                 : p.by_head         ? id / entries
                                     : id % p.head_groups;
        };
        auto fetch = [&](int64_t id64, uint32_t x) {
          const int32_t id = int32_t(id64);
          if (kOne) {
            sh->ahead[x & 1] = tile0;
            return;
          }
          const int32_t at = p.mode == kRanges ? from + id % (to - from)
                             : p.by_head       ? id % entries
                                               : id / p.head_groups;
          async_copy_16(&sh->ahead[x & 1], &p.entries[at]);
          async_copy_16(reinterpret_cast<uint8_t*>(&sh->ahead[x & 1]) + 16,
                        reinterpret_cast<const uint8_t*>(&p.entries[at]) + 16);
        };
        auto landed = [&]() { async_wait_all(); };
        // waits, or only looks (what a look does not find is not an error)
        bool ok = true;
        auto ready = [&](uint64_t* bar, uint32_t use, uint32_t ring, bool wait) -> bool {
          if (use < ring) return true;
          const uint32_t par = ((use / ring) - 1) & 1;
          if (!wait) return mbar_test(bar, par);
          ok = mbar_wait(bar, par, abort, p.wait_ns);
          return ok;
        };
        // an item's description and its Q tile, once there is room for both
        auto publish = [&](int32_t id, uint32_t x, int32_t pos, int32_t careful,
                           bool wait) -> bool {
          const uint32_t slot = ii % kNI, qs = qi % C::kNQ;
          if (!ready(&sh->info_empty[slot], ii, kNI, wait) ||
              !ready(&sh->q_empty[qs], qi, C::kNQ, wait))
            return false;
          landed();
          Item* it = &sh->info[slot];
          Entry e = sh->ahead[x & 1];
          int32_t hg = head_of(id);
          if (p.mode == kRanges) {
            if (e.slot >= 0) e.slot += hg * p.round_slots;
            hg = hg * round_groups + e.hg;
          }
          const int32_t head0 = hg * p.tile_heads;
          it->e = e;
          it->head0 = head0;
          it->g = head0 / p.group;
          it->mt = max(0, (e.lim0 + 1) / kBK - e.b0);
          it->pos = pos;
          it->careful = careful;
          sh->ids[pos] = id;
          mbar_arrive(&sh->info_full[slot]);
          ++ii;
          // the box is tile_heads x tile_tokens rows; what it covers behind the
          // tensor counts as loaded (zeros)
          mbar_arrive_expect_tx(&sh->q_full[qs],
                                uint32_t(C::kPanels * 128 * p.tile_heads * p.tile_tokens));
#pragma unroll
          for (int s = 0; s < C::kPanels; ++s)
            tma_load_3d(sQ + qs * C::kQBytes + s * C::kQPanel, &tq, &sh->q_full[qs], s * 64,
                        head0, e.q0, pol_q);
          ++qi;
          return true;
        };
        auto special = [&](int32_t what) {
          const uint32_t slot = ii % kNI;
          if (!ready(&sh->info_empty[slot], ii, kNI, true)) return;
          sh->info[slot].e.n = what;
          mbar_arrive(&sh->info_full[slot]);
          ++ii;
        };
        auto load_k = [&](int32_t g, int32_t key) {
          const uint32_t ks = kiss % C::kNK;
          uint64_t* empty = C::kNK == C::kNS ? &sh->s_full[ks] : &sh->k_empty[ks];
          if (!ready(empty, kiss, C::kNK, true)) return;
          mbar_arrive_expect_tx(&sh->k_full[ks], C::kKVBytes);
#pragma unroll
          for (int s = 0; s < C::kPanels; ++s)
            tma_load_3d(sK + ks * C::kKVBytes + s * C::kKVPanel, &tk, &sh->k_full[ks], s * 64, g,
                        key, pol_kv);
          ++kiss;
        };
        // Items are looked up ahead, so that no load or atomic is waited for
        // between two of them, and the next one's Q is on its way while this one's
        // K blocks are.  (The first two of a CTA are dealt out forth and back.)
        const bool counted = p.mode == kTiles;
        const int32_t grid = int32_t(gridDim.x), me = int32_t(blockIdx.x);
        int64_t id0 = counted ? me : 0, id1 = counted ? 2 * grid - 1 - me : 1, id2 = 2;
        if (counted) id2 = 2 * grid + atomicAdd(p.counter, 1);
        uint32_t batches = 0, x = 0;         // x: items fetched, but for this one
        bool ended = false;                  // every role has seen the end
        if (id0 < items) {
          fetch(id0, 0);
          for (bool more = true; ok && more;) {
            // a batch of items, then those of them that are to be done again
            int32_t pos = 0;
            publish(int32_t(id0), x, 0, 0, true);
            while (ok) {
              const Entry* e = &sh->ahead[x & 1];
              const int32_t g = sh->info[(ii - 1) % kNI].g, n = e->n;
              const int32_t key0 = e->kbeg + e->b0 * kBK;
              more = id1 < items;
              if (more) fetch(id1, x + 1);
              const bool ahead = more && pos + 1 < kBatch;
              bool out = false;
              for (int32_t t = 0; ok && t < n; ++t) {
                load_k(g, key0 + t * kBK);
                if (t > 0 && ok && ahead && !out)
                  out = publish(int32_t(id1), x + 1, pos + 1, 0, false);
              }
              if (ok && ahead && !out) publish(int32_t(id1), x + 1, pos + 1, 0, true);
              if (!more) break;
              ++x;
              id0 = id1;
              id1 = id2;
              id2 = counted ? int64_t(2 * grid + atomicAdd(p.counter, 1)) : id2 + 1;
              if (!ahead) break;
              ++pos;
            }
            if (ok) special(kMarker);
            if (ok) ok = mbar_wait(&sh->batch_done, batches & 1, abort, p.wait_ns);
            ++batches;
            if (kOne && !*(volatile int32_t*)&sh->any_again) {
              ended = true;
              break;
            }
            int32_t careful = kClean;
            for (bool some = true; ok && some;) {
              some = false;
              for (int32_t w = 0; ok && w < pos / 32 + 1; ++w) {
                uint32_t bits = *(volatile uint32_t*)&sh->again[w];
                const uint32_t maxima = *(volatile uint32_t*)&sh->maxima[w];
                sh->again[w] = sh->maxima[w] = 0;
                while (ok && bits) {
                  const int at = __ffs(bits) - 1;
                  bits &= bits - 1;
                  some = true;
                  const int32_t how = careful | ((maxima >> at) & 1 ? kMaxima : 0);
                  // (the next batch's first item may be in the other place)
                  fetch(sh->ids[32 * w + at], x + 1);
                  publish(sh->ids[32 * w + at], x + 1, 32 * w + at, how, true);
                  const Entry* e = &sh->ahead[(x + 1) & 1];
                  const int32_t g = sh->info[(ii - 1) % kNI].g, n = e->n;
                  const int32_t key0 = e->kbeg + e->b0 * kBK;
                  for (int32_t t = 0; ok && t < (how & kMaxima ? 2 * n : n); ++t)
                    load_k(g, key0 + (t >= n ? t - n : t) * kBK);
                }
              }
              if (careful & kSmall) break;       // that was the last time
              careful = kClean | kMaxima | kSmall;
              if (ok && some) {
                special(kMarker);
                if (ok) ok = mbar_wait(&sh->batch_done, batches & 1, abort, p.wait_ns);
                ++batches;
              }
            }
          }
        }
        if (ok && !ended) special(kEnd);
        if (!ok) raise_abort(sh, p);
        // copies still in flight must land before this CTA's shared memory goes
        drain_ring(sh->q_full, qi, C::kNQ);
        drain_ring(sh->k_full, kiss, C::kNK);
      }
    } else if (warp == 2) {
      // ------------------------------------------------- producer: V
      const uint64_t pol_kv = l2_policy_evict_last();
      uint32_t ii = 0, viss = 0;
      bool ok = true;
      for (;; ++ii) {
        const int slot = ii % kNI;
        if (!warp_wait(&sh->info_full[slot], (ii / kNI) & 1, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        const int32_t n = sh->info[slot].e.n, g = sh->info[slot].g;
        const int32_t row0 = sh->info[slot].e.kbeg + sh->info[slot].e.b0 * kBK;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
        if (n == kEnd) break;
        if (kOne && n == kMarker && !go_on(&ok)) break;
        if (lane == 0) {
          for (int32_t t = 0; t < n; ++t) {
            const uint32_t vs = viss % C::kNV;
            if (viss >= uint32_t(C::kNV) &&
                !mbar_wait(C::kNV == 2 ? &sh->pv_done[vs] : &sh->v_empty[vs],
                           ((viss / C::kNV) - 1) & 1, abort, p.wait_ns)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sh->v_full[vs], C::kKVBytes);
#pragma unroll
            for (int s = 0; s < C::kPanels; ++s)
              tma_load_3d(sV + vs * C::kKVBytes + s * C::kKVPanel, &tv, &sh->v_full[vs], s * 64, g,
                          row0 + t * kBK, pol_kv);
            ++viss;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
      if (lane == 0) {
        if (!ok) raise_abort(sh, p);
        drain_ring(sh->v_full, viss, C::kNV);
      }
    } else if (warp == 1) {
      // ------------------------------------------------- Q K^T issuer
      constexpr uint32_t idesc_qk = idesc_bf16(kRows, kBK, 0, 0);
      uint32_t ii = 0, qi = 0, stage = 0, phase = 0, kb = 0, kst = 0, kph = 0;
      uint32_t copies = 0;                 // items whose Q is copied, so far
      bool ok = true;
      for (;; ++ii) {
        const int slot = ii % kNI;
        if (!warp_wait(&sh->info_full[slot], (ii / kNI) & 1, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        const int32_t n = sh->info[slot].e.n, careful = sh->info[slot].careful;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
        if (n == kEnd) break;
        if (n == kMarker) {
          if (!go_on(&ok)) break;
          continue;
        }
        const int32_t blocks = careful & kMaxima ? 2 * n : n;
        const uint32_t qs = qi % C::kNQ;
        if (!warp_wait(&sh->q_full[qs], (qi / C::kNQ) & 1, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        const uint64_t qdesc = smem_desc_sw128(smem_u32(sQ + qs * C::kQBytes), 16, 1024);
        const bool copy = C::kCopyQ && n >= kCopyBlocks;
        bool near = false;                 // Q is in tensor memory
        for (int32_t t = 0; t < blocks; ++t) {
          // lane 0: K of this block; lane 1: S of two blocks ago is read; lane 2: Q
          const bool reuse = kb >= 2;
          uint64_t* bar = &sh->k_full[kst];
          uint32_t par = kph;
          if (lane == 1 && reuse) {
            bar = &sh->s_empty[stage];
            par = phase ^ 1u;
          }
          if (lane == 2) {
            bar = &sh->q_copied[copies & 1];
            par = (copies >> 1) & 1;
          }
          const uint32_t have = __ballot_sync(0xffffffffu, mbar_test(bar, par));
          near = copy && (near || (have & 4u));
          if (!(have & 1u) && !warp_wait(&sh->k_full[kst], kph, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          if (reuse && !(have & 2u) &&
              !warp_wait(&sh->s_empty[stage], phase ^ 1u, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t kdesc = smem_desc_sw128(smem_u32(sK + kst * C::kKVBytes), 16, 1024);
          const uint32_t s_tmem = tmem + stage * kBK;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t qoff = (kk / 4) * C::kQPanel + (kk % 4) * 32;
              const uint32_t koff = (kk / 4) * C::kKVPanel + (kk % 4) * 32;
              const uint64_t b = kdesc + uint64_t(koff >> 4);
              if (near)
                mma_ts(s_tmem, tmem + C::kQ + kk * 8, b, idesc_qk, kk > 0 ? 1u : 0u);
              else
                mma_ss(s_tmem, qdesc + uint64_t(qoff >> 4), b, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(&sh->s_full[stage]);
            if (C::kNK != C::kNS) mma_commit(&sh->k_empty[kst]);
            if (t == blocks - 1) mma_commit(&sh->q_empty[qs]);
          }
          __syncwarp();
          ++kb;
          if (++stage == uint32_t(C::kNS)) {
            stage = 0;
            phase ^= 1u;
          }
          if (++kst == C::kNK) {
            kst = 0;
            kph ^= 1u;
          }
        }
        if (!ok) break;
        ++qi;
        copies += copy;
      }
      if (lane == 0) {
        if (!ok) raise_abort(sh, p);
        mma_commit(&sh->drain_qk);   // complete before the tensor memory is freed
        mbar_wait(&sh->drain_qk, 0, nullptr);
      }
    } else if (warp == 3) {
      // ------------------------------------------------- P V issuer
      constexpr uint32_t idesc_pv = idesc_bf16(kRows, D, 0, 1);   // P (TMEM), V MN-major
      uint32_t ii = 0, qi = 0, pb = 0, vstage = 0, vphase = 0;
      bool ok = true;
      for (;; ++ii) {
        const int slot = ii % kNI;
        if (!warp_wait(&sh->info_full[slot], (ii / kNI) & 1, abort, p.wait_ns)) {
          ok = false;
          break;
        }
        const int32_t n = sh->info[slot].e.n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
        if (n == kEnd) break;
        if (n == kMarker) {
          if (!go_on(&ok)) break;
          continue;
        }
        for (int32_t t = 0; t < n; ++t) {
          const bool need_o = t == 0 && qi > 0;  // the previous epilogue has read O
          // lane 0: P, lane 1: V, lane 2: O
          const uint32_t pp = (pb >> 1) & 1;
          uint64_t* bar = &sh->p_full[pb & 1];
          uint32_t par = pp;
          if (lane == 1) {
            bar = &sh->v_full[vstage];
            par = vphase;
          }
          if (lane == 2 && need_o) {
            bar = &sh->o_free;
            par = (qi - 1) & 1;
          }
          const uint32_t have = __ballot_sync(0xffffffffu, mbar_test(bar, par));
          if (!(have & 1u) && !warp_poll(&sh->p_full[pb & 1], pp, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          if (!(have & 2u) && !warp_wait(&sh->v_full[vstage], vphase, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          if (need_o && !(have & 4u) && !warp_wait(&sh->o_free, (qi - 1) & 1, abort, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t p_at = tmem + C::kP + pb % C::kNP * (kBK / 2);
          const uint64_t vdesc =
              smem_desc_sw128(smem_u32(sV + vstage * C::kKVBytes), C::kKVPanel, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              mma_ts(tmem + C::kO, p_at + kk * 8, vdesc + uint64_t((kk * 16 * 128) >> 4), idesc_pv,
                     (t == 0 && kk == 0) ? 0u : 1u);
            mma_commit(&sh->pv_done[pb & 1]);
            if (C::kNV != 2) mma_commit(&sh->v_empty[vstage]);
            if (t == n - 1) mma_commit(&sh->o_last);
          }
          __syncwarp();
          ++pb;
          if (++vstage == C::kNV) {
            vstage = 0;
            vphase ^= 1u;
          }
        }
        if (!ok) break;
        ++qi;
      }
      if (lane == 0) {
        if (!ok) raise_abort(sh, p);
        mma_commit(&sh->drain_pv);
        mbar_wait(&sh->drain_pv, 0, nullptr);
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (fn) return fn;
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess) {
    fn = reinterpret_cast<EncodeFn>(ptr);
    known.store(fn, std::memory_order_relaxed);
  }
  return fn;
}

// [tokens, heads, d] bf16 view, boxes of 64 columns x box_heads x box_tokens,
// 128-byte swizzle.  The stride of an extent of one is not used.
bool make_map(CUtensorMap* map, const void* base, int64_t tokens, int64_t heads, int d, int64_t st,
              int64_t shd, int box_heads, int box_tokens) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(heads > 1 ? shd : d) * 2,
                                 cuuint64_t(tokens > 1 ? st : d) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

static_assert(kMaxWorkers < kBins, "the schedule counts shares in its bins");
int workers_of(int sms) { return std::min(sms, kMaxWorkers); }

// Tiles are cut where sequences have more keys than queries, on the whole: the
// tiles of whole prompts have from one block to all, and taking the long ones
// first leaves an even end.  (The schedule adds up their blocks in 32 bits.)
bool may_cut(const sa_packed_shape& s) {
  const int64_t blocks = (int64_t(s.total_k) + kBK - 1) / kBK + kItemCost;
  const int64_t tiles =
      sa_packed::most_tiles(s) * (s.num_q_heads / sa_packed::tile_of(s).heads);
  return s.total_k > s.total_q && tiles < (int64_t(1) << 30) / blocks;
}

// Bytes of a key and its value, all heads.
int64_t key_bytes(const sa_packed_shape& s) {
  return int64_t(s.num_kv_heads) * s.head_dim * 4;
}

struct Layout {
  size_t header, seqs, tile0, entries, cost0, first, cuts, part_ml, part_o, end;
  int64_t max_entries, round_slots;
};

Layout layout_of(const sa_packed_shape& s, int sms) {
  Layout l;
  const int64_t tiles = sa_packed::most_tiles(s), workers = workers_of(sms);
  l.max_entries = tiles * (s.num_q_heads / sa_packed::tile_of(s).heads) + 2 * workers;
  l.round_slots = 2 * workers;        // a cut tile of r ranges takes r - 1 of the shares' ends
  l.header = 0;
  l.seqs = up(sizeof(Header));
  l.tile0 = l.seqs + up(size_t(s.batch) * 16);
  l.entries = l.tile0 + up(size_t(s.batch) * 4);
  l.cost0 = l.entries + up(size_t(l.max_entries) * sizeof(Entry));
  l.first = l.cost0 + up(size_t(tiles) * 4);
  l.cuts = l.first + up(size_t(workers + 1) * 4);
  l.part_ml = l.cuts + up(size_t(workers) * sizeof(Cut));
  const int64_t head_groups = s.num_q_heads / sa_packed::tile_of(s).heads;
  const size_t slots =
      size_t(rounds_of(s.total_k * key_bytes(s), int32_t(head_groups)) * l.round_slots);
  l.part_o = l.part_ml + up(slots * kRows * 16);
  l.end = l.part_o + up(slots * kRows * size_t(s.head_dim) * 4);
  return l;
}

template <class Kernel, class... Params>
cudaError_t launch_kernel(Kernel* kern, unsigned grid, int threads, int smem, cudaStream_t st,
                          const Params&... params) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, params...);
}

template <int D, bool kLse, bool kOne>
cudaError_t launch_attention(const Params& p, unsigned grid, const CUtensorMap& tq,
                             const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = Cfg<D>;
  constexpr int kSmem = C::kData + int(sizeof(Shared));
  static_assert(kSmem <= 232448, "shared memory budget");
  static std::atomic<uint64_t> done{0};
  auto kern = packed_attention_kernel<D, kLse, kOne>;
  // the roles' shares of the registers (which come in eights) need as many at launch
  static std::atomic<bool> counted{false};
  if (!counted.load(std::memory_order_relaxed)) {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    if (kThreads * ((attr.numRegs + 7) / 8 * 8) < kAllRegs) return cudaErrorInvalidKernelImage;
    counted.store(true, std::memory_order_relaxed);
  }
  cudaError_t e = sa_paged::allow_shared(kern, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, kThreads, kSmem, st, tq, tk, tv, p);
}

template <int D>
cudaError_t launch_d(const Args& a, int sms, cudaStream_t st, bool* encode_failed) {
  const sa_packed_shape& s = a.s;
  const sa_packed::Tile tile = sa_packed::tile_of(s);
  const Layout lay = layout_of(s, sms);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const int64_t head_groups = s.num_q_heads / tile.heads;
  const int64_t tiles = sa_packed::most_tiles(s);
  const int64_t key_blocks = (int64_t(s.total_k) + kBK - 1) / kBK;

  // no keys at all: the map only has to be valid, every score is masked
  const bool none = s.total_k == 0;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, a.q, s.total_q, s.num_q_heads, D, s.q_stride_t, s.q_stride_h, tile.heads,
                tile.tokens) ||
      !make_map(&tk, none ? a.q : a.k, none ? 1 : s.total_k, none ? 1 : s.num_kv_heads, D,
                s.k_stride_t, s.k_stride_h, 1, kBK) ||
      !make_map(&tv, none ? a.q : a.v, none ? 1 : s.total_k, none ? 1 : s.num_kv_heads, D,
                s.v_stride_t, s.v_stride_h, 1, kBK)) {
    *encode_failed = true;
    return cudaErrorInvalidValue;
  }
  const bool ranges = may_cut(s);
  const int workers = workers_of(sms);
  auto at = [&](size_t offset) { return static_cast<void*>(ws + offset); };
  Params p;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.header = static_cast<const Header*>(at(lay.header));
  p.counter = &static_cast<Header*>(at(lay.header))->counter;
  p.entries = static_cast<const Entry*>(at(lay.entries));
  p.first = static_cast<const int32_t*>(at(lay.first));
  p.part_ml = static_cast<float4*>(at(lay.part_ml));
  p.part_o = static_cast<float4*>(at(lay.part_o));
  p.v_st = s.v_stride_t;
  p.v_sh = s.num_kv_heads > 1 ? s.v_stride_h : 0;
  p.o_st = s.o_stride_t;
  p.o_sh = s.num_q_heads > 1 ? s.o_stride_h : 0;
  p.total_q = s.total_q;
  p.total_k = s.total_k;
  p.batch = s.batch;
  p.Hq = s.num_q_heads;
  p.group = s.num_q_heads / s.num_kv_heads;
  p.tile_heads = tile.heads;
  p.tile_tokens = tile.tokens;
  p.head_groups = int32_t(head_groups);
  p.by_head = s.total_k * key_bytes(s) > kL2Share;
  p.round_slots = int32_t(lay.round_slots);
  p.scale_log2 = sa_packed::scale_log2(s);
  p.dev_status = a.dev_status;
  p.wait_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
  // every tile its own CTA, none worth cutting
  if (tiles * head_groups <= sms && (!ranges || key_blocks <= kDirectBlocks)) {
    p.mode = kDirect;
    const unsigned grid = unsigned(tiles * head_groups);
    return a.lse ? launch_attention<D, true, true>(p, grid, tq, tk, tv, st)
                 : launch_attention<D, false, true>(p, grid, tq, tk, tv, st);
  }
  p.mode = ranges ? kRanges : kTiles;
  ScheduleParams sp;
  sp.cu_q = a.cu_q;
  sp.cu_k = a.cu_k;
  sp.header = static_cast<Header*>(at(lay.header));
  sp.seqs = static_cast<int4*>(at(lay.seqs));
  sp.tile0 = static_cast<int32_t*>(at(lay.tile0));
  sp.cost0 = static_cast<int32_t*>(at(lay.cost0));
  sp.entries = static_cast<Entry*>(at(lay.entries));
  sp.first = static_cast<int32_t*>(at(lay.first));
  sp.cuts = static_cast<Cut*>(at(lay.cuts));
  sp.total_q = s.total_q;
  sp.total_k = s.total_k;
  sp.batch = s.batch;
  sp.tile_tokens = tile.tokens;
  sp.workers = workers;
  sp.bin_shift = 0;
  while ((key_blocks >> sp.bin_shift) >= kBins) ++sp.bin_shift;
  sp.mode = p.mode;
  sp.head_groups = p.head_groups;
  sp.key_bytes = key_bytes(s);
  sp.dev_status = a.dev_status;
  cudaError_t e = launch_kernel(schedule_kernel, 1, kScheduleThreads, 0, st, sp);
  if (e != cudaSuccess) return e;
  e = a.lse ? launch_attention<D, true, false>(p, unsigned(workers), tq, tk, tv, st)
            : launch_attention<D, false, false>(p, unsigned(workers), tq, tk, tv, st);
  if (e != cudaSuccess || !ranges) return e;
  JoinParams jp;
  jp.header = p.header;
  jp.cuts = sp.cuts;
  jp.part_o = p.part_o;
  jp.part_ml = p.part_ml;
  jp.o = p.o;
  jp.lse = p.lse;
  jp.o_st = p.o_st;
  jp.o_sh = p.o_sh;
  jp.Hq = p.Hq;
  jp.tile_heads = p.tile_heads;
  jp.head_groups = p.head_groups;
  jp.round_slots = p.round_slots;
  return launch_kernel(join_kernel<D>, unsigned(8 * workers), kJoinRows * D / 4, 0, st, jp);
}

}  // namespace

namespace sa_packed {

size_t workspace(const sa_packed_shape& s, int sms) { return layout_of(s, sms).end; }

cudaError_t launch(const Args& a, int sms, cudaStream_t st, bool* encode_failed) {
  return a.s.head_dim == 128 ? launch_d<128>(a, sms, st, encode_failed)
                             : launch_d<64>(a, sms, st, encode_failed);
}

}  // namespace sa_packed
