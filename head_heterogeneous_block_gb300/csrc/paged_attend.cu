// Attention of one new token per sequence over a paged key-value cache, on
// sm_103a.
//
// The work is a read of every key and value once: 4d bytes a token against
// 4dG operations for the G query heads that share it, so HBM bounds it as long
// as the arithmetic stays out of the way.  At G of 7 or 8 that is too much for
// the CUDA cores at full bandwidth, so both products run on the tensor cores
// with the tokens (then the value dimensions) as the 128 rows of the tile and
// the query heads as its 16 columns (32 for G above 16):
//
//   S^T [128 tokens x heads] = K [128 x d] Q^T        K and Q from shared memory
//   O^T [d x heads]          = V^T [d x 128] P^T      V (transposed by its
//                                                     descriptor) and P from shared memory
//
// Split.  The tokens of all rows (sequence, KV head, and for groups above 32
// heads a chunk of 32 of them) are laid end to end in tiles of 128 (64 where
// there are few) and cut into equal ranges, one per CTA, two CTAs per processor:
// the lengths differ freely between rows and no processor waits for the longest.  A row
// that lies in one range is finished there; a row that is cut leaves one
// partial state (maximum, sum, unnormalised output) per range, which the join
// kernel combines in range order.  Each CTA finds its range by a scan of the
// lengths, so a captured launch follows the lengths of its time.
//
// Roles of a CTA's warps:
//   warp 0     producer: walks the range row by row in tiles of 128 tokens,
//              looks pages up (the next tile's while waiting for room) and
//              issues TMA loads of each page's piece of K and of V into a ring
//              of stages, three of 32 KB at d = 128, so that the processor's
//              two CTAs have about 128 KB in flight while they work.
//   warp 1     issues both products, each as soon as what it reads is there.
//   others     softmax and output, in groups of four warps: a thread owns one
//              token of S and one dimension of O, for the 4 (8 above G = 8)
//              heads of its group.  Weights are 2^(s - m) with a reference m
//              per head that is moved only when a score passes it by 8 (in
//              powers of two); m cancels in the end.  A tile has one barrier
//              a group, before which all its waits lie.
//
// The weights enter the tensor core in bf16, split in two parts (hi + lo) for
// bf16 output and in three for fp32 output, as so many groups of columns of
// one product: what is left is 2^-16 (2^-24) of a weight, and the split is
// free because the product is far from its limit.  Sums and outputs are fp32.
//
// Tokens past the end of a range in its last tile have their scores set to
// -infinity, and their value rows are zeroed in shared memory up to the next
// multiple of 16, where the product stops; so nothing a page holds behind a
// row's length is ever used.
//
// Accumulating weights: the scores (in base 2) go to the workspace, 4G bytes a
// token, and the second launch adds 2^(s - lse), summed over the heads, to each
// token's weight.
//
// Measured (GB300, copy rate 6783 GB/s, read-only traffic goes a little
// higher): 16 sequences of 64K tokens, 28/4 heads, 2.1 GB: 319 us, 99%; one of
// 128K, 64/8 heads, 537 MB: 87 us, 91%.  537 MB in 32 rows or more, by query
// heads of a KV head, bf16 and fp32 output: 4 heads 85 and 86 us, 8: 88 and 88,
// 16: 87 and 97, 32: 110 and 111 (at 32, and 16 in fp32, one CTA a processor).  The rest is a fixed 9 us or so: the
// chain lengths -> page table -> first keys with a cold instruction cache
// (3 us), the last tile's softmax and store (1 us), the join (2.8 us); it is
// all there is of one 700-token sequence (8.5 us).  One CTA per processor with
// twice the stages came 4% (d = 128) to 60% (d = 64) slower, three or four 15
// to 30% (d = 64); pieces of 64 or 128 tokens instead of 32 the same, of 16
// tokens 1 to 12% slower.

#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "give_up.h"
#include "paged.h"
#include "ptx.cuh"

namespace {

using namespace sa_dev;
using sa_paged::AttendArgs;

constexpr int kTileShift = 7;
constexpr int kTile = 1 << kTileShift; // tokens per tile
constexpr int kMaxChunk = 32;          // most query heads of a row handled together
constexpr int kInfo = 8;               // tile descriptions in flight
constexpr float kMove = 8.f;           // how far a score may pass its reference
constexpr int kJoinThreads = 256;
constexpr int kWeightSteps = 4;        // tokens of a thread
constexpr int kMaxGroup = 1024;        // query heads of a KV head

template <int D, int GP, int PARTS>
struct Cfg {
  static constexpr int kPanels = D / 64;              // 128-byte column panels
  static constexpr int kPanel = kTile * 128;          // bytes of one K/V panel
  static constexpr int kStage = kPanels * kPanel;
  // softmax: kGroups groups of four warps, kHeads heads of a token a thread
  static constexpr int kChunk = GP < 16 ? 16 : GP;    // columns of S, rows of Q
  static constexpr int kHeads = GP < 16 ? 4 : 8;
  static constexpr int kGroups = GP / kHeads;
  static constexpr int kThreads = 64 + 128 * kGroups;
  // CTAs on a processor, the stages and Q tiles that then fit.  Tile j: K in
  // stage 2j % kStages, V in the next.
  static constexpr int kPerSm = GP == 32 || (D == 128 && GP * PARTS == 48) ? 1 : 2;
  static constexpr int kStages = (D == 128 ? 6 : 12) / kPerSm;
  static constexpr int kQs = GP >= 16 ? 1 : 2;
  static constexpr int kNS = kChunk;                  // columns of S
  static constexpr int kNP = (GP * PARTS + 15) / 16 * 16;   // columns of O, rows of P
  static constexpr int kQ = kPanels * kChunk * 128;   // bytes of one Q tile
  static constexpr int kP = 2 * kNP * 128;            // bytes of P (two panels of 64 tokens)
  static constexpr uint32_t kO = 2 * kNS;             // TMEM column of O
  static constexpr uint32_t kTmemCols = GP == 32 ? 256 : 128;
  // V^T has 128 rows to the tensor core; at d = 64 the second 64 read from
  // 2 KB further on (their rows of O are not used): within shared memory, since
  // P and Q follow the ring
  static constexpr uint32_t kVNext = D == 128 ? kPanel : 2048;
  static_assert(2 * kNS + kNP <= int(kTmemCols) && kPerSm * kTmemCols <= 512, "tensor memory");
  static_assert(GP % kHeads == 0 && kP + kQs * kQ >= 2048, "");
};

struct TileInfo {
  int32_t u;          // row (with its head chunk)
  int32_t t, n;       // first token, tokens; n == 0: end of the range
  int32_t flags;
};
enum { kFirst = 1, kLast = 2, kComplete = 4, kSecond = 8 };

template <class C>
struct Shared {
  // the barriers, in the order that the kernel's first threads initialise them
  uint64_t info_empty[kInfo];   // one arrival of the issuer and of each softmax warp
  uint64_t p_full;              // one of each softmax warp
  uint64_t info_full[kInfo];    // from here on: one arrival
  uint64_t kv_full[C::kStages], kv_empty[C::kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];
  uint64_t pv_done;
  uint64_t drain;
  TileInfo info[kInfo];
  // maxima by tile parity, sums by segment parity, [group][quarter][head]: a
  // group's barrier lies between any use of a buffer and the next writing of it
  float maxima[2][C::kGroups][4][C::kHeads];
  float sums[2][C::kGroups][4][C::kHeads];
  int32_t scan[C::kThreads / 32];
  int32_t u0, p0, len0;  // first row of the range, the units before it, its length
  uint32_t tmem_base;
  int abort;
  GiveUp failed[C::kGroups];  // raised by a group's warp whose wait gave up
};

// Workspace: records, row log-sum-exps, partial states, scores.  A record is
// what the join of a row needs: u is -1 where nothing is to be joined.  There
// is one a row when there are no more rows than CTAs, else one a CTA, for the
// row that begins in its range and ends in another.
struct Record {
  int32_t u, first, segs;       // the row, its first CTA, its ranges
  int32_t slot;                 // partial state of the first CTA: its first or second
};
struct Work {
  Record* rec;         // [ctas]
  Record* row_rec;     // [U], one a row, only when accumulating
  float* row_lse2;     // [U][chunk]
  float2* part_ml;     // [ctas][2][chunk]
  float* part_o;       // [ctas][2][chunk][d]
  float* scores;       // [rows][G][slots], base-2 exponents; only when accumulating
};

// Query heads of a row handled together: all up to 32, above that 32 at a time.
int chunk_of(int G) { return G <= 16 ? 16 : kMaxChunk; }

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

size_t layout(Work* w, char* base, int64_t rows, int G, int64_t cap, int d, int ctas,
              bool accumulate) {
  const int chunk = chunk_of(G);
  const int64_t U = rows * ((G + chunk - 1) / chunk);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = base + at;
    at += round256(n);
    return p;
  };
  Work x;
  x.rec = reinterpret_cast<Record*>(take(size_t(ctas) * sizeof(Record)));
  x.row_rec = reinterpret_cast<Record*>(take(accumulate ? size_t(U) * sizeof(Record) : 0));
  x.row_lse2 = reinterpret_cast<float*>(take(accumulate ? size_t(U) * chunk * 4 : 0));
  x.part_ml = reinterpret_cast<float2*>(take(size_t(ctas) * 2 * chunk * 8));
  x.part_o = reinterpret_cast<float*>(take(size_t(ctas) * 2 * chunk * d * 4));
  x.scores = reinterpret_cast<float*>(take(accumulate ? size_t(rows) * G * cap * 4 : 0));
  if (w) *w = x;
  return at;
}

struct Params {
  const int32_t* table;
  const int32_t* lens;
  int64_t num_pages;
  int32_t page_shift, max_pages, cap;
  int32_t bx_shift;            // log2 of the tokens of a TMA box
  int32_t Hkv, Hq, G, HC, U;   // HC: head chunks of a row; U = rows * HC
  int32_t chunk;               // heads of a chunk
  int32_t q_rows;              // heads of a Q box
  int32_t most_ranges;         // CTAs that get work
  int32_t by_row;              // records: one a row
  int32_t ctas;                // CTAs of the first launch
  float scale_log2;
  void* o;
  int32_t out_f32;
  float* lse;
  const float* weights;
  float* weights_out;
  Work w;
  int32_t* dev_status;
  uint64_t wait_ns;
};

// The row, and the first head of the chunk, of u.  kOne: rows have one chunk.
template <bool kOne>
__device__ __forceinline__ int32_t row_of(const Params& p, int32_t u) {
  return kOne || p.HC == 1 ? u : u / p.HC;
}
template <bool kOne>
__device__ __forceinline__ int32_t head_of(const Params& p, int32_t u) {
  return kOne || p.HC == 1 ? 0 : (u % p.HC) * p.chunk;
}

// Units of 2^shift tokens of a row.
__device__ __forceinline__ int32_t units_of(int shift, int32_t len) {
  return (len + (1 << shift) - 1) >> shift;
}

// Ranges of `per` units: CTA c has [c * per, (c + 1) * per).
struct Ranges {
  int32_t total, per;
  __device__ __forceinline__ int32_t begin(int32_t c) const {
    return int32_t(min(uint32_t(c) * uint32_t(per), uint32_t(total)));
  }
  // the CTA whose range holds unit x
  __device__ __forceinline__ int32_t owner(int32_t x) const { return x / per; }
};

template <bool kF32>
__device__ __forceinline__ void store_out(const Params& p, size_t at, float v) {
  if (kF32)
    static_cast<float*>(p.o)[at] = v;
  else
    static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(v);
}

// A wait's first polls leave the clock alone: reading it costs more than most
// waits here last.  Short limits go by the clock from the start.  What goes by
// the clock is a call, not a copy at every wait: a launch starts with a cold
// instruction cache, and its first microseconds go by the code it has to fetch.
constexpr uint64_t kClockless = 1000000;
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort,
                                       uint64_t limit_ns) {
  if (limit_ns >= kClockless) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_test_sleep(bar, parity, 2000)) return true;
  }
  return mbar_wait(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        uint64_t limit_ns) {
  return mbar_test(bar, parity) || wait_long(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_on(bar, parity, abort, limit_ns);
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  __syncwarp();
  return ok;
}
// Every lane waits on a barrier of its choice; true when all came through.
__device__ __forceinline__ bool wait_lanes(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           uint64_t limit_ns) {
  const bool ok = __all_sync(0xffffffffu, wait_on(bar, parity, abort, limit_ns));
  __syncwarp();
  return ok;
}

// The barrier of one softmax group.
template <int kGroups>
__device__ __forceinline__ bool group_any(int grp, bool flag) {
  if (kGroups > 3 && grp == 3) return bar_any<4, 128>(flag);
  if (kGroups > 2 && grp == 2) return bar_any<3, 128>(flag);
  if (kGroups > 1 && grp == 1) return bar_any<2, 128>(flag);
  return bar_any<1, 128>(flag);
}
template <int kGroups>
__device__ __forceinline__ void group_sync(int grp) {
  if (kGroups > 3 && grp == 3)
    bar_sync<4, 128>();
  else if (kGroups > 2 && grp == 2)
    bar_sync<3, 128>();
  else if (kGroups > 1 && grp == 1)
    bar_sync<2, 128>();
  else
    bar_sync<1, 128>();
}

template <int D, int GP, int PARTS>
__global__ void __launch_bounds__(Cfg<D, GP, PARTS>::kThreads, Cfg<D, GP, PARTS>::kPerSm)
    attend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using C = Cfg<D, GP, PARTS>;
  constexpr int kThreads = C::kThreads;
  constexpr int HP = C::kHeads;
  constexpr int kChunk = C::kChunk;
  constexpr bool kOne = GP < kMaxChunk;
  constexpr bool kF32 = PARTS == 3;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  launch_dependents();
  uint8_t* sKV = smem_raw;
  uint8_t* sP = sKV + C::kStages * C::kStage;
  uint8_t* sQ = sP + C::kP;
  using Sh = Shared<C>;
  Sh* sh = reinterpret_cast<Sh*>(sQ + C::kQs * C::kQ);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t cta = blockIdx.x;
  if (smem_u32(smem_raw) & 1023u) {
    wait_dependency();
    if (tid == 0) {
      atomicOr(p.dev_status, SA_DEV_BAD_LAUNCH);
      p.w.rec[cta] = Record{-1, 0, 0, 0};
    }
    return;
  }

  // ---- what needs none of the inputs, while the launch before this one ends
  if (tid == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    sh->abort = 0;
    for (int g = 0; g < C::kGroups; ++g) sh->failed[g].clear();
    sh->u0 = sh->p0 = sh->len0 = 0;
  }
  constexpr int kBars = 2 * kInfo + 1 + 2 * C::kStages + 6 + 2;
  static_assert(offsetof(Sh, info) == kBars * sizeof(uint64_t) && kBars <= kThreads, "");
  if (tid < kBars) {
    mbar_init(&sh->info_empty[0] + tid, tid < kInfo    ? 1 + 4 * C::kGroups
                                        : tid == kInfo ? 4 * C::kGroups
                                                       : 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // keys and values are read once: their lines make way first in L2
  const uint64_t pol = l2_policy_evict_first();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  wait_dependency();

  // ---- this CTA's range: a scan of every row's units, which are tiles (a part
  // of a tile takes a CTA as long as a whole one), or 64 tokens where that
  // still leaves a CTA for each.  (8 rows of 8192 tokens: 13.3 us cut into equal
  // numbers of tokens, 11.9 into tiles; of 700 tokens: 10.0 us in tiles, 8.5 in
  // 64s.)  Up to 128 rows each warp scans for itself, four rows a lane; more
  // rows are scanned by the CTA.
  const bool few = p.U <= 128;
  const int32_t per = few ? 4 : (p.U + kThreads - 1) / kThreads;
  const int32_t ua = min(p.U, (few ? lane : tid) * per), ub = min(p.U, ua + per);
  int32_t mine = 0;
  int us = kTileShift;                         // log2 of a unit's tokens
  if (few) {
    int32_t n[4], halves = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = ua + i < ub ? p.lens[row_of<kOne>(p, ua + i)] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = max(0, min(n[i], p.cap));
      halves += units_of(kTileShift - 1, n[i]);
    }
    if (int32_t(__reduce_add_sync(0xffffffffu, halves)) <= p.most_ranges) us = kTileShift - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) mine += units_of(us, n[i]);
  } else {
#pragma unroll 1
    for (int32_t u = ua; u < ub; ++u)
      mine += units_of(us, max(0, min(p.lens[row_of<kOne>(p, u)], p.cap)));
  }
  int32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  int32_t before = incl - mine, total = __shfl_sync(0xffffffffu, incl, 31);
  if (!few) {
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    total = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh->scan[w];
      total += sh->scan[w];
    }
  }
  const Ranges rg{total, max(1, (total + p.most_ranges - 1) / p.most_ranges)};
  const int32_t a = rg.begin(cta), b = rg.begin(cta + 1);
  // the thread that has the range's first row says where that begins
  if (a < b && a >= before && a < before + mine && (!few || warp == 0)) {
    int32_t at = before;
#pragma unroll 1
    for (int32_t u = ua; u < ub; ++u) {
      const int32_t n = max(0, min(p.lens[row_of<kOne>(p, u)], p.cap));
      if (a < at + units_of(us, n)) {
        sh->u0 = u;
        sh->p0 = at;
        sh->len0 = n;
        break;
      }
      at += units_of(us, n);
    }
  }
  if (few)
    __syncwarp();
  else
    __syncthreads();
  // rows without a token, taken in turn by the CTAs
  if (warp >= 2) {
#pragma unroll 1
    for (int32_t u = cta; u < p.U; u += gridDim.x) {
      if (sa_paged::row_len(p.lens, row_of<kOne>(p, u), p.cap, p.dev_status) > 0) continue;
      const int32_t r = row_of<kOne>(p, u), h0 = head_of<kOne>(p, u);
      const size_t bh = size_t(r / p.Hkv) * p.Hq + size_t(r % p.Hkv) * p.G + h0;
      const int gc = min(kChunk, p.G - h0), x0 = tid - 64;
#pragma unroll 1
      for (int x = x0; x < gc * D; x += kThreads - 64) store_out<kF32>(p, bh * D + x, 0.f);
      if (p.lse && x0 < gc) p.lse[bh + x0] = -INFINITY;
      if (p.by_row && x0 == 0) p.w.rec[u] = Record{-1, 0, 0, 0};
    }
  }
  if (a >= b) {
    if (tid == 0 && !p.by_row) p.w.rec[cta] = Record{-1, 0, 0, 0};
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }
  const int bx = 1 << p.bx_shift;

  if (warp == 0) {
    // ------------------------------------------------- producer
    int32_t u = sh->u0, pu = sh->p0;           // current row and the units before it
    int32_t len = sh->len0;
    int32_t ubase = u, ulen = 0;               // lane l holds the length of row ubase + l
    auto load_lens = [&]() {
      ulen = ubase + lane < p.U
                 ? sa_paged::row_len(p.lens, row_of<kOne>(p, ubase + lane), p.cap, p.dev_status) : 0;
    };
    auto end_of = [&]() -> int32_t {           // of the row's part in this range
      return min(len, int32_t(min(int64_t(b - pu) << us, int64_t(1) << 30)));
    };
    int32_t seg = 0;                           // row parts before this one
    int32_t t = (a - pu) << us, t1 = end_of();
    bool first = true, begins = t == 0;
    bool more = true;
    // the next tile of the range; n == 0 when it is used up
    auto next = [&]() -> TileInfo {
      while (more && t >= t1) {
        pu += units_of(us, len);
        if (pu >= b || u + 1 >= p.U) {
          more = false;
          break;
        }
        ++u;
        if (u >= ubase + 32) {
          ubase = u;
          load_lens();
        }
        len = __shfl_sync(0xffffffffu, ulen, u - ubase);
        t = 0;
        t1 = end_of();
        if (len > 0) {
          first = begins = true;
          ++seg;
        }
      }
      if (!more) return TileInfo{0, 0, 0, 0};
      const int32_t n = min(kTile, t1 - t);
      const bool last = t + n >= t1;
      TileInfo x{u, t, n,
                 (first ? kFirst : 0) | (last ? kLast : 0) |
                     (begins && t1 == len ? kComplete : 0) | (seg > 0 ? kSecond : 0)};
      first = false;
      t += n;
      return x;
    };
    // lane i: the page of box i of the tile
    auto lookup = [&](const TileInfo& x) -> int32_t {
      if ((lane << p.bx_shift) >= x.n) return 0;
      const int32_t slot = x.t + (lane << p.bx_shift);
      return p.table[int64_t(row_of<kOne>(p, x.u)) * p.max_pages + (slot >> p.page_shift)];
    };
    uint32_t i = 0, qi = 0;                    // tiles and Q tiles issued
    uint32_t issued = 0;                       // stages filled
    bool ok = true;
    // The first tile's copies are issued at once; from then on a tile's pages
    // are looked up before the one ahead of it waits for room in the ring.
    TileInfo held{0, 0, 0, 0};
    int32_t held_pg = 0;
#pragma unroll 1
    for (uint32_t k = 0;; ++k) {
      const TileInfo x = next();
      const int32_t x_pg = lookup(x);
      const TileInfo cur = k == 0 ? x : held;
      int32_t pg = k == 0 ? x_pg : held_pg;
      held = x;
      held_pg = x_pg;
      if (k == 1) {
        if (x.n == 0) break;
        continue;
      }
      if (cur.n == 0) break;
      const int boxes = (cur.n + bx - 1) >> p.bx_shift;
      const int32_t prow = (cur.t + (lane << p.bx_shift)) & ((1 << p.page_shift) - 1);
      const int slot = i % kInfo;
      if (i >= uint32_t(kInfo))
        ok = wait_warp(&sh->info_empty[slot], ((i / kInfo) - 1) & 1, abort, p.wait_ns);
      if (!ok) break;
      if (lane == 0) {
        sh->info[slot] = cur;
        mbar_arrive(&sh->info_full[slot]);
      }
      if (cur.flags & kFirst) {
        const int qs = qi % C::kQs;
        if (qi >= uint32_t(C::kQs))
          ok = wait_warp(&sh->q_empty[qs], ((qi / C::kQs) - 1) & 1, abort, p.wait_ns);
        if (!ok) break;
        if (lane == 0) {
          const int32_t r = row_of<kOne>(p, cur.u);
          const int32_t h0 = (r % p.Hkv) * p.G + head_of<kOne>(p, cur.u);
          mbar_arrive_expect_tx(&sh->q_full[qs], C::kPanels * p.q_rows * 128);
#pragma unroll
          for (int s = 0; s < C::kPanels; ++s)
            tma_load_3d(sQ + qs * C::kQ + s * kChunk * 128, &tq, &sh->q_full[qs], s * 64, h0,
                        r / p.Hkv, pol);
        }
        ++qi;
      }
      if (lane < boxes && (pg < 0 || pg >= p.num_pages)) {
        atomicOr(p.dev_status, SA_DEV_BAD_INDEX);
        pg = 0;
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int st = issued % C::kStages;
        if (issued >= uint32_t(C::kStages))
          ok = wait_warp(&sh->kv_empty[st], ((issued / C::kStages) - 1) & 1, abort, p.wait_ns);
        if (!ok) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&sh->kv_full[st], uint32_t(boxes * bx * 128 * C::kPanels));
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int s = 0; s < C::kPanels; ++s)
            tma_load_3d(sKV + st * C::kStage + s * C::kPanel + lane * bx * 128, kv ? &tv : &tk,
                        &sh->kv_full[st], s * 64, prow, pg, pol);
        }
        ++issued;
      }
      if (!ok) break;
      if (k == 0) load_lens();
      ++i;
      if (k > 0 && x.n == 0) break;
    }
    // the record of a row that begins in this range and ends in another; the
    // rows that end here are the softmax warps' to record
    if (lane == 0) {
      const bool cut = begins && pu > b;       // pu: the end of the last row
      const Record rec{cut ? u : -1, cta, cut ? rg.owner(pu - 1) - cta + 1 : 0, seg > 0 ? 1 : 0};
      if (cut || !p.by_row) p.w.rec[p.by_row ? u : cta] = rec;
      if (cut && p.weights_out) p.w.row_rec[u] = rec;
    }
    if (ok) {
      const int slot = i % kInfo;
      if (i >= uint32_t(kInfo))
        ok = wait_warp(&sh->info_empty[slot], ((i / kInfo) - 1) & 1, abort, p.wait_ns);
      if (ok && lane == 0) {
        sh->info[slot] = TileInfo{0, 0, 0, 0};
        mbar_arrive(&sh->info_full[slot]);
      }
    }
    if (lane == 0) {
      if (!ok) {
        atomicOr(p.dev_status, SA_DEV_TIMEOUT);
        *abort = 1;
      }
      // copies still in flight land before the CTA's shared memory goes
#pragma unroll 1
      for (uint32_t x = issued > uint32_t(C::kStages) ? issued - C::kStages : 0; x < issued; ++x)
        wait_long(&sh->kv_full[x % C::kStages], (x / C::kStages) & 1, nullptr, kWaitLimitNs);
#pragma unroll 1
      for (uint32_t x = qi > uint32_t(C::kQs) ? qi - C::kQs : 0; x < qi; ++x)
        wait_long(&sh->q_full[x % C::kQs], (x / C::kQs) & 1, nullptr, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------- issuer of both products
    constexpr uint32_t idesc_s = idesc_bf16(128, C::kNS, 0, 0);    // K, Q both K-major
    constexpr uint32_t idesc_o = idesc_bf16(128, C::kNP, 1, 0);    // V^T M-major, P K-major
    bool ok = true;
    uint32_t seg = 0;                          // Q tiles used
    // waits for tile j's description and returns its length and flags
    auto tile = [&](uint32_t j, int32_t& n, int32_t& flags) -> bool {
      const int slot = j % kInfo;
      if (!wait_warp(&sh->info_full[slot], (j / kInfo) & 1, abort, p.wait_ns)) return false;
      n = sh->info[slot].n;
      flags = sh->info[slot].flags;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
      return true;
    };
    auto issue_s = [&](uint32_t j, int32_t flags) {
      const int st = (2 * j) % C::kStages;
      tc_fence_after();
      const uint64_t kd = smem_desc_sw128(smem_u32(sKV + st * C::kStage), 16, 1024);
      const uint64_t qd = smem_desc_sw128(smem_u32(sQ + (seg % C::kQs) * C::kQ), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk / 4) * C::kPanel + (kk % 4) * 32;
          const uint32_t qo = (kk / 4) * kChunk * 128 + (kk % 4) * 32;
          mma_ss(tmem + (j & 1) * C::kNS, kd + uint64_t(ko >> 4), qd + uint64_t(qo >> 4), idesc_s,
                 kk > 0 ? 1u : 0u);
        }
        mma_commit(&sh->s_full[j & 1]);
        mma_commit(&sh->kv_empty[st]);
        if (flags & kLast) mma_commit(&sh->q_empty[seg % C::kQs]);
      }
      __syncwarp();
      if (flags & kLast) ++seg;
    };
    auto issue_pv = [&](uint32_t j, int32_t n) {
      const int st = (2 * j + 1) % C::kStages;
      tc_fence_after();
      const uint64_t vd = smem_desc_sw128(smem_u32(sKV + st * C::kStage), C::kVNext, 1024);
      const uint64_t pd = smem_desc_sw128(smem_u32(sP), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
          const uint32_t po = (kk / 4) * C::kNP * 128 + (kk % 4) * 32;
          if (kk * 16 < n)
            mma_ss(tmem + C::kO, vd + uint64_t((kk * 16 * 128) >> 4), pd + uint64_t(po >> 4),
                   idesc_o, kk > 0 ? 1u : 0u);
        }
        mma_commit(&sh->pv_done);
        mma_commit(&sh->kv_empty[st]);
      }
      __syncwarp();
    };
    // Tile j's output product and tile j + 1's scores, each as soon as what it
    // reads is there: lane 0 polls P, lane 1 V, lane 2 the next K, lane 3 its Q.
    // Before j = 0 only the scores of tile 0.
    int32_t n = 0, flags = 0;
    for (uint32_t j1 = 0;; ++j1) {             // j1 = j + 1
      int32_t nn = 0, nflags = 0;
      ok = tile(j1, nn, nflags);
      if (!ok) break;
      bool pv_left = j1 > 0, s_left = nn > 0;
      const uint32_t j = j1 - 1;
      uint64_t* bar = &sh->p_full;
      uint32_t par = j & 1;
      bool used = pv_left;
      if (lane == 1) {
        bar = &sh->kv_full[(2 * j + 1) % C::kStages];
        par = ((2 * j + 1) / C::kStages) & 1;
      } else if (lane == 2) {
        bar = &sh->kv_full[(2 * j1) % C::kStages];
        par = ((2 * j1) / C::kStages) & 1;
        used = s_left;
      } else if (lane == 3) {
        bar = &sh->q_full[seg % C::kQs];
        par = (seg / C::kQs) & 1;
        used = s_left && (nflags & kFirst);
      } else if (lane > 3) {
        used = false;
      }
      uint64_t t0 = 0;
      uint32_t polls = 0;
      while (pv_left || s_left) {
        const uint32_t have = __ballot_sync(0xffffffffu, !used || mbar_test(bar, par));
        __syncwarp();
        if (pv_left && (have & 3u) == 3u) {
          issue_pv(j, n);
          pv_left = false;
          if (lane < 2) used = false;
        } else if (s_left && (have & 12u) == 12u) {
          issue_s(j1, nflags);
          s_left = false;
          if (lane == 2 || lane == 3) used = false;
        } else if (p.wait_ns < kClockless || (++polls & 1023u) == 0) {
          const uint64_t now = global_ns();
          if (t0 == 0) t0 = now;
          const bool out = *abort || now - t0 > p.wait_ns;
          if (__any_sync(0xffffffffu, out)) {
            ok = false;
            break;
          }
        }
      }
      if (!ok || nn == 0) break;
      n = nn;
      flags = nflags;
    }
    (void)flags;
    if (lane == 0) {
      if (!ok) {
        atomicOr(p.dev_status, SA_DEV_TIMEOUT);
        *abort = 1;
      }
      // every product is complete before the tensor memory is freed
      mma_commit(&sh->drain);
      wait_long(&sh->drain, 0, nullptr, kWaitLimitNs);
    }
  } else {
    // ------------------------------------------------- softmax and output
    const int grp = (warp - 2) >> 2;           // heads [grp * HP, (grp + 1) * HP) of the chunk
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;       // token of the tile, dimension of O
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + grp * HP;
    const float c = p.scale_log2;
    float m[HP], l[HP], o[HP];
    uint32_t seg_in = 0, seg = 0;              // segments summed, and stored
    TileInfo prev{0, 0, 0, 0}, it{0, 0, 0, 0};
    bool ok = true;
    // the description of tile j
    auto describe = [&](uint32_t j) -> bool {
      const int slot = j % kInfo;
      if (!wait_lanes(&sh->info_full[slot], (j / kInfo) & 1, abort, p.wait_ns)) return false;
      it = sh->info[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
      return true;
    };
    bool fail = !describe(0);
    for (uint32_t j = 0;; ++j) {
      // Every wait of a tile comes before its one barrier, where the group's
      // four warps learn together whether one gave up.
      float s[HP];
      bool need = false;
      const int gc = min(kChunk, p.G - head_of<kOne>(p, it.u)) - grp * HP;   // live heads
      const bool live = !fail && it.n > 0;
      if (!fail && (live || j > 0)) {
        // lanes split over the scores, the last output product, and (for a
        // tile whose value rows have to be cleared) the values
        const uint32_t x = 2 * j + 1;
        uint64_t* bar = &sh->s_full[j & 1];
        uint32_t par = (j >> 1) & 1;
        if (j > 0 && ((lane & 3) == 1 || !live)) {
          bar = &sh->pv_done;
          par = (j - 1) & 1;
        } else if ((lane & 3) == 2 && it.n < kTile) {
          bar = &sh->kv_full[x % C::kStages];
          par = (x / C::kStages) & 1;
        }
        fail = !wait_lanes(bar, par, abort, p.wait_ns);
        tc_fence_after();
        if (live && !fail) {
          tmem_load(lanes + (j & 1) * C::kNS, s);
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            s[h] = (row < it.n && h < gc) ? s[h] * c : -INFINITY;
            if (!(it.flags & kFirst)) need |= s[h] > m[h] + kMove;   // (NaN: no)
          }
          // a segment's first tile sets the reference: its maxima are there
          // when the barrier is passed
          if (it.flags & kFirst) {
            need = true;
#pragma unroll
            for (int h = 0; h < HP; ++h) {
              const float y = warp_max(s[h]);
              if (lane == 0) sh->maxima[j & 1][grp][quarter][h] = y;
            }
          }
          // the last product step reads value rows up to the next 16th
          if (grp == 0 && row >= it.n && row < ((it.n + 15) & ~15)) {
            uint4* v = reinterpret_cast<uint4*>(sKV + (x % C::kStages) * C::kStage + row * 128);
#pragma unroll
            for (int s2 = 0; s2 < C::kPanels; ++s2)
#pragma unroll
              for (int y = 0; y < 8; ++y) v[s2 * (C::kPanel / 16) + y] = make_uint4(0, 0, 0, 0);
          }
        }
      }
      if (fail) sh->failed[grp].raise(j);
      const bool any = group_any<C::kGroups>(grp, need || fail);
      if (any && sh->failed[grp].raised(j)) {
        ok = false;
        break;
      }
      if (j > 0) {
        // the previous tile's product joins the segment's output
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          float x[HP];
          tmem_load(lanes + C::kO + q * GP, x);
#pragma unroll
          for (int h = 0; h < HP; ++h) o[h] += x[h];
        }
        if (prev.flags & kLast) {
          // ---- the end of a segment
          const float(*sum)[HP] = sh->sums[seg & 1][grp];
          ++seg;
          const int32_t r = row_of<kOne>(p, prev.u), h0 = head_of<kOne>(p, prev.u) + grp * HP;
          const size_t bh = size_t(r / p.Hkv) * p.Hq + size_t(r % p.Hkv) * p.G + h0;
          const size_t part =
              (size_t(cta) * 2 + ((prev.flags & kSecond) ? 1 : 0)) * kChunk + grp * HP;
          const bool whole = (prev.flags & kComplete) != 0;
          float mr = 0.f;                      // thread h: head h's reference
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            if (row == h) mr = m[h];
            if (h0 + h < p.G && row < D) {
              if (whole) {
                const float L = (sum[0][h] + sum[1][h]) + (sum[2][h] + sum[3][h]);
                store_out<kF32>(p, (bh + h) * D + row, __fdividef(o[h], L));
              } else {
                p.w.part_o[(part + h) * D + row] = o[h];
              }
            }
          }
          if (row < HP && h0 + row < p.G) {
            const float L = (sum[0][row] + sum[1][row]) + (sum[2][row] + sum[3][row]);
            if (whole) {
              const float lse2 = (mr == -INFINITY ? 0.f : mr) + log2f(L);
              if (p.lse) p.lse[bh + row] = lse2 * 0.6931471805599453f;
              if (p.weights_out) p.w.row_lse2[size_t(prev.u) * kChunk + grp * HP + row] = lse2;
            } else {
              p.w.part_ml[part + row] = make_float2(mr, L);
            }
          }
          if (whole && grp == 0 && row == 0) {
            if (p.by_row) p.w.rec[prev.u] = Record{-1, 0, 0, 0};
            if (p.weights_out) p.w.row_rec[prev.u] = Record{-1, 0, 0, 0};
          }
        }
      }
      if (it.n == 0) break;
      if (any) {
        // a new reference: the larger of the old one and the tile's maximum
        float(*top)[HP] = sh->maxima[j & 1][grp];
        const bool first = (it.flags & kFirst) != 0;
        if (!first) {
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float x = warp_max(s[h]);
            if (lane == 0) top[quarter][h] = x;
          }
          group_sync<C::kGroups>(grp);
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float x = fmaxf(fmaxf(top[0][h], top[1][h]), fmaxf(top[2][h], top[3][h]));
          const float mn = first ? x : fmaxf(m[h], x);
          const float alpha = first ? 0.f : mn == m[h] ? 1.f : ex2(m[h] - mn);
          l[h] = first ? 0.f : l[h] * alpha;
          o[h] = first ? 0.f : o[h] * alpha;
          m[h] = mn;
        }
      }
      if (p.weights_out && row < it.n) {
        const int32_t r = row_of<kOne>(p, it.u), h0 = head_of<kOne>(p, it.u) + grp * HP;
        float* dst = p.w.scores + (size_t(r) * p.G + h0) * p.cap + it.t + row;
#pragma unroll
        for (int h = 0; h < HP; ++h)
          if (h < gc) dst[size_t(h) * p.cap] = s[h];
      }
      // weights, in parts of bf16: row (part, head) of P, this thread's token
      // its column, in the 128-byte swizzle that the product reads
      uint8_t* col = sP + (row >> 6) * C::kNP * 128 + (row & 7) * 2;
      const uint32_t chunk = uint32_t(row & 63) >> 3;
#pragma unroll
      for (int h = 0; h < HP; h += 2) {
        float w0 = ex2(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
        float w1 = ex2(s[h + 1] - (m[h + 1] == -INFINITY ? 0.f : m[h + 1]));
        l[h] += w0;
        l[h + 1] += w1;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          const int r0 = q * GP + grp * HP + h, r1 = r0 + 1;
          const uint32_t pk = pack_bf16x2(w0, w1);
          *reinterpret_cast<uint16_t*>(col + r0 * 128 + ((chunk ^ (r0 & 7)) << 4)) = uint16_t(pk);
          *reinterpret_cast<uint16_t*>(col + r1 * 128 + ((chunk ^ (r1 & 7)) << 4)) =
              uint16_t(pk >> 16);
          w0 -= __uint_as_float(pk << 16);
          w1 -= __uint_as_float(pk & 0xFFFF0000u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full);
      if (it.flags & kLast) {
        // the segment's sums, while its last product runs
#pragma unroll
        for (int h = 0; h < HP; ++h) {
#pragma unroll
          for (int w = 16; w; w >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
        }
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < HP; ++h) sh->sums[seg_in & 1][grp][quarter][h] = l[h];
        }
        ++seg_in;
      }
      prev = it;
      fail = !describe(j + 1);
    }
    if (!ok) {
      if (lane == 0) atomicOr(p.dev_status, SA_DEV_TIMEOUT);
      *abort = 1;
    }
    tmem_ld_wait();
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Whether a record names a row to be joined.  A launch that gave up may have
// left none: whatever is there instead must not lead out of the workspace.
__device__ __forceinline__ bool usable(const Params& p, const Record& rec) {
  return rec.u >= 0 && rec.u < p.U && rec.first >= 0 && rec.segs >= 1 && rec.segs <= p.ctas &&
         rec.first <= p.ctas - rec.segs && (rec.slot & ~1) == 0;
}

// The k-th partial state of a row: the index of its first head.
__device__ __forceinline__ uint32_t state_of(const Params& p, const Record& rec, int32_t k) {
  return (uint32_t(rec.first + k) * 2 + (k == 0 ? rec.slot : 0)) * p.chunk;
}

// Block (record, head): the join of a row's partial states.  Eight warps take
// every eighth state each and bring them to their own maximum; the eight
// results are brought to the row's and added in warp order.  A chain of three
// reads (record, state, nothing else waits): 2.8 us from the end of the first
// launch at any size, of which the launch is about 1.
template <int D, bool kF32>
__device__ __forceinline__ void join(const Params& p, int32_t record, int h) {
  constexpr int kVec = D / 32;                     // elements of a lane
  constexpr int kWays = kJoinThreads / 32;
  __shared__ float acc[kWays][D], ms[kWays], ls[kWays];
  const int lane = threadIdx.x & 31, way = threadIdx.x >> 5;
  const Record rec = p.w.rec[record];
  if (!usable(p, rec)) return;
  float m = -INFINITY, l = 0.f, v[kVec];
#pragma unroll
  for (int x = 0; x < kVec; ++x) v[x] = 0.f;
#pragma unroll 4
  for (int32_t k = way; k < rec.segs; k += kWays) {
    const uint32_t at = state_of(p, rec, k) + h;
    const float2 ml = p.w.part_ml[at];
    float o[kVec];
    if constexpr (kVec == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p.w.part_o + at * D + lane * 4);
      o[0] = y.x;
      o[1] = y.y;
      o[2] = y.z;
      o[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(p.w.part_o + at * D + lane * 2);
      o[0] = y.x;
      o[1] = y.y;
    }
    const float mn = fmaxf(m, ml.x);
    const float f0 = mn == m ? 1.f : ex2(m - mn), f1 = mn == ml.x ? 1.f : ex2(ml.x - mn);
    l = l * f0 + ml.y * f1;
#pragma unroll
    for (int x = 0; x < kVec; ++x) v[x] = v[x] * f0 + o[x] * f1;
    m = mn;
  }
#pragma unroll
  for (int x = 0; x < kVec; ++x) acc[way][lane * kVec + x] = v[x];
  if (lane == 0) {
    ms[way] = m;
    ls[way] = l;
  }
  __syncthreads();
  const int x = threadIdx.x;
  const int32_t r = row_of<false>(p, rec.u), hc = head_of<false>(p, rec.u) + h;
  if (x >= D || hc >= p.G) return;
  const int ways = min(kWays, rec.segs);
  float M = ms[0];
#pragma unroll 1
  for (int y = 1; y < ways; ++y) M = fmaxf(M, ms[y]);
  float sum = 0.f, L = 0.f;
#pragma unroll 1
  for (int y = 0; y < ways; ++y) {
    const float f = ms[y] == M ? 1.f : ex2(ms[y] - M);
    L = fmaf(ls[y], f, L);
    sum = fmaf(acc[y][x], f, sum);
  }
  const int32_t b = r / p.Hkv;
  const size_t bh = size_t(b) * p.Hq + size_t(r - b * p.Hkv) * p.G + hc;
  store_out<kF32>(p, bh * D + x, __fdividef(sum, L));
  if (x == 0 && p.lse)
    p.lse[bh] = ((M == -INFINITY ? 0.f : M) + log2f(L)) * 0.6931471805599453f;
}

// A piece of a row's slots: every token's probabilities, summed over the row's
// heads, added to its weight.  4G + 8 bytes a token.  It runs beside the joins,
// so it adds up the log-sum-exps of cut rows for itself.
__device__ __forceinline__ void add_weights(const Params& p, int32_t r, int32_t t0) {
  __shared__ float lse2s[kMaxGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t n = sa_paged::row_len(p.lens, r, p.cap, p.dev_status);
  if (t0 >= n) return;
  for (int32_t h = warp; h < p.G; h += kJoinThreads / 32) {
    const int32_t u = r * p.HC + h / p.chunk, x = h % p.chunk;
    const Record rec = p.w.row_rec[u];
    float v;
    if (rec.u < 0) {
      v = p.w.row_lse2[size_t(u) * p.chunk + x];
    } else {
      float m = -INFINITY, l = 0.f;
      if (usable(p, rec)) {
        for (int32_t k = lane; k < rec.segs; k += 32) {
          const float2 ml = p.w.part_ml[state_of(p, rec, k) + x];
          const float mn = fmaxf(m, ml.x);
          l = l * (mn == m ? 1.f : ex2(m - mn)) + ml.y * (mn == ml.x ? 1.f : ex2(ml.x - mn));
          m = mn;
        }
      }
      const float M = warp_max(m);
      l *= m == M ? 1.f : ex2(m - M);
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      v = (M == -INFINITY ? 0.f : M) + log2f(l);
    }
    if (lane == 0) lse2s[h] = v;
  }
  const int32_t t = t0 + threadIdx.x;
  const float* s = p.w.scores + size_t(r) * p.G * p.cap + t;
  const size_t at = size_t(r) * p.cap + t;
  float sum[kWeightSteps], old[kWeightSteps];
#pragma unroll
  for (int i = 0; i < kWeightSteps; ++i) {
    sum[i] = 0.f;
    if (t + i * kJoinThreads < n) old[i] = p.weights[at + i * kJoinThreads];
  }
  __syncthreads();
#pragma unroll 4
  for (int32_t h = 0; h < p.G; ++h) {
    const float l = lse2s[h];
#pragma unroll
    for (int i = 0; i < kWeightSteps; ++i)
      if (t + i * kJoinThreads < n)
        sum[i] += ex2(s[size_t(h) * p.cap + i * kJoinThreads] - l);
  }
#pragma unroll
  for (int i = 0; i < kWeightSteps; ++i)
    if (t + i * kJoinThreads < n) p.weights_out[at + i * kJoinThreads] = old[i] + sum[i];
}

// The second launch.  Blocks [0, joins): join of (record, head); the others:
// weights of (row, piece).
template <int D, bool kF32, bool kWeights>
__global__ void __launch_bounds__(kJoinThreads)
    finish_kernel(const __grid_constant__ Params p, int32_t joins, int32_t pieces) {
  launch_dependents();
  wait_dependency();
  const int32_t id = blockIdx.x;
  if (!kWeights || id < joins) {
    join<D, kF32>(p, id / p.q_rows, id % p.q_rows);
  } else {
    const int32_t r = (id - joins) / pieces;
    add_weights(p, r, (id - joins - r * pieces) * (kJoinThreads * kWeightSteps));
  }
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeFn>(ptr);
  }();
  return fn;
}

// bf16 [n2][n1][d] with the given strides in elements; boxes of 64 columns x
// box rows, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, int d, int64_t n1, int64_t n2, int64_t s1,
              int64_t s2, int box) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(n1), cuuint64_t(n2)};
  const cuuint64_t strides[2] = {cuuint64_t(s1) * 2, cuuint64_t(s2) * 2};
  const cuuint32_t boxes[3] = {64, cuuint32_t(box), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
            boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

template <int D, int GP, int PARTS>
cudaError_t launch(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed) {
  using C = Cfg<D, GP, PARTS>;
  constexpr int kRing = C::kStages * C::kStage;
  constexpr int kSmem = kRing + C::kP + C::kQs * C::kQ + int(sizeof(Shared<C>));
  static_assert(C::kPerSm * (kSmem + 1024) <= 233472, "shared memory budget");
  const sa_paged_cache& c = a.c;
  const int64_t rows = int64_t(c.batch) * c.num_kv_heads;
  Params p{};
  p.page_shift = log2i(c.page);
  p.bx_shift = c.page < 32 ? p.page_shift : 5;
  p.G = a.Hq / c.num_kv_heads;
  p.chunk = C::kChunk;
  p.HC = (p.G + p.chunk - 1) / p.chunk;
  p.q_rows = p.G < p.chunk ? p.G : p.chunk;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, a.q, D, a.Hq, c.batch, a.qsh, a.qsb, p.q_rows) ||
      !make_map(&tk, c.k_pages, D, c.page, c.num_pages, D, c.k_page_stride, 1 << p.bx_shift) ||
      !make_map(&tv, c.v_pages, D, c.page, c.num_pages, D, c.v_page_stride, 1 << p.bx_shift)) {
    *encode_failed = true;
    return cudaErrorInvalidValue;
  }
  p.table = c.table;
  p.lens = c.lens;
  p.num_pages = c.num_pages;
  p.max_pages = c.max_pages;
  p.cap = c.page * c.max_pages;
  p.Hkv = c.num_kv_heads;
  p.Hq = a.Hq;
  p.U = int32_t(rows * p.HC);
  p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(D)));
  p.o = a.o;
  p.out_f32 = a.out_f32;
  p.lse = a.lse;
  p.weights = c.weights;
  p.weights_out = a.weights_out;
  p.dev_status = a.dev_status;
  p.wait_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
  const int ctas = sms * C::kPerSm;
  // a single row takes no more ranges than there are processors: its join is
  // one long chain (65536 tokens: 18.6 us in 304 ranges, 15.3 in 128)
  p.most_ranges = p.U > 1 ? ctas : sms;
  p.by_row = p.U <= ctas;
  p.ctas = ctas;
  layout(&p.w, static_cast<char*>(a.ws), rows, p.G, p.cap, D, ctas, a.weights_out != nullptr);
  auto kern = attend_kernel<D, GP, PARTS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = sa_paged::allow_shared(kern, kSmem, done);
  if (e != cudaSuccess) return e;
  // each launch may start while the one before it in the stream ends, and
  // waits for it before it touches memory
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  e = cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  const int64_t joins = int64_t(p.by_row ? p.U : ctas) * p.q_rows;
  constexpr int kPiece = kJoinThreads * kWeightSteps;
  const int32_t pieces = (p.cap + kPiece - 1) / kPiece;
  const int64_t blocks = joins + (a.weights_out ? rows * pieces : 0);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return a.weights_out
             ? cudaLaunchKernelEx(&cfg, finish_kernel<D, PARTS == 3, true>, p, int32_t(joins), pieces)
             : cudaLaunchKernelEx(&cfg, finish_kernel<D, PARTS == 3, false>, p, int32_t(joins), pieces);
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed) {
  const int G = a.Hq / a.c.num_kv_heads;
  if (a.out_f32) {
    if (G <= 4) return launch<D, 4, 3>(a, sms, st, encode_failed);
    if (G <= 8) return launch<D, 8, 3>(a, sms, st, encode_failed);
    if (G <= 16) return launch<D, 16, 3>(a, sms, st, encode_failed);
    return launch<D, 32, 3>(a, sms, st, encode_failed);
  }
  if (G <= 4) return launch<D, 4, 2>(a, sms, st, encode_failed);
  if (G <= 8) return launch<D, 8, 2>(a, sms, st, encode_failed);
  if (G <= 16) return launch<D, 16, 2>(a, sms, st, encode_failed);
  return launch<D, 32, 2>(a, sms, st, encode_failed);
}

}  // namespace

namespace sa_paged {

size_t attend_workspace(const sa_paged_cache& c, int32_t Hq, bool accumulate, int sms) {
  return layout(nullptr, nullptr, int64_t(c.batch) * c.num_kv_heads, Hq / c.num_kv_heads,
                int64_t(c.page) * c.max_pages, c.head_dim, sms * 2, accumulate);
}

cudaError_t launch_attend(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed) {
  *encode_failed = false;
  return a.c.head_dim == 128 ? launch_d<128>(a, sms, st, encode_failed)
                             : launch_d<64>(a, sms, st, encode_failed);
}

}  // namespace sa_paged
