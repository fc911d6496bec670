// Attention of one new token per sequence over a paged key-value cache, on
// sm_103a.
//
// The work is a read of every key and value once: 4d bytes a token against
// 4dG operations for the G query heads that share it, so HBM bounds it as long
// as the arithmetic stays out of the way.  At G of 7 or 8 that is too much for
// the CUDA cores at full bandwidth, so both products run on the tensor cores
// with the tokens (then the value dimensions) as the 128 rows of the tile and
// the query heads as its 16 columns:
//
//   S^T [128 tokens x 16 heads] = K [128 x d] Q^T        K and Q from shared memory
//   O^T [d x heads]             = V^T [d x 128] P^T      V (transposed by its
//                                                        descriptor) and P from shared memory
//
// Split.  The tokens of all rows (sequence, KV head, and for groups above 16
// heads a chunk of 16 of them) are laid end to end in units of `bx` tokens and
// cut into equal ranges, one per CTA, one CTA per processor: the lengths
// differ freely between rows and no processor waits for the longest.  A row
// that lies in one range is finished there; a row that is cut leaves one
// partial state (maximum, sum, unnormalised output) per range, which the join
// kernel combines in range order.  Each CTA finds its range by a scan of the
// lengths, so a captured launch follows the lengths of its time.
//
// Roles of a CTA's six warps:
//   warp 0     producer: walks the range row by row in tiles of 128 tokens,
//              looks pages up (the next tile's while waiting for room) and
//              issues TMA loads of each page's piece of K and of V into a ring
//              of stages, 32 KB each at d = 128, so that about 128 KB are in
//              flight while one tile is worked on.
//   warp 1     issues both products.
//   warps 2-5  softmax and output: a thread owns one token of S (all heads)
//              and one dimension of O (all heads).  Weights are 2^(s - m) with
//              a reference m per head that is moved only when a score passes
//              it by 8 (in powers of two): then, and at a row's first tile,
//              the tile's maxima are exchanged.  m cancels in the end.
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

#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "paged.h"
#include "ptx.cuh"

namespace {

using namespace sa_dev;
using sa_paged::AttendArgs;

constexpr int kTile = 128;             // tokens per tile
constexpr int kChunk = 16;             // query heads of a row handled together
constexpr int kThreads = 192;
constexpr int kInfo = 8;               // tile descriptions in flight
constexpr int kPerSm = 2;              // CTAs per processor
constexpr float kMove = 8.f;           // how far a score may pass its reference
constexpr int kJoinThreads = 512;
constexpr int kJoinHeads = 4;          // heads of a join block, four warps each
constexpr int kWeightThreads = 256;
constexpr int kWeightSteps = 4;        // tokens of a thread

template <int D, int GP, int PARTS>
struct Cfg {
  static constexpr int kPanels = D / 64;              // 128-byte column panels
  static constexpr int kPanel = kTile * 128;          // bytes of one K/V panel
  static constexpr int kStage = kPanels * kPanel;
  static constexpr int kStages = D == 128 ? 3 : 6;    // tile j: K in stage 2j % kStages, V next
  static constexpr int kNS = 16;                      // columns of S
  static constexpr int kNP = (GP * PARTS + 15) / 16 * 16;   // columns of O, rows of P
  static constexpr int kQ = kPanels * kChunk * 128;   // bytes of one Q tile
  // two Q tiles, but where only one leaves room for two CTAs on a processor
  static constexpr int kQs = D == 128 && GP * PARTS > 32 ? 1 : 2;
  static constexpr int kP = 2 * kNP * 128;            // bytes of P (two panels of 64 tokens)
  static constexpr uint32_t kO = 2 * kNS;             // TMEM column of O
  static constexpr uint32_t kTmemCols = 128;
  static_assert(2 * kNS + kNP <= int(kTmemCols), "tensor memory budget");
};

struct TileInfo {
  int32_t u;          // row (with its head chunk)
  int32_t t, n;       // first token, tokens; n == 0: end of the range
  int32_t flags;
};
enum { kFirst = 1, kLast = 2, kComplete = 4, kSecond = 8 };

struct Shared {
  uint64_t kv_full[6], kv_empty[6];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];
  uint64_t p_full, pv_done;
  uint64_t info_full[kInfo], info_empty[kInfo];
  uint64_t drain;
  TileInfo info[kInfo];
  float red[4][kChunk];
  int32_t scan[kThreads / 32];
  int32_t u0, p0;      // first row of the range and the units before it
  uint32_t tmem_base;
  int abort;
  int failed;          // set by a softmax warp whose wait gave up
};

// Workspace: per-CTA records, row log-sum-exps, partial states, scores.
// What the join of the row that a CTA's range starts inside of needs: u is -1
// unless this is the second range of that row.
struct Record {
  int32_t u, first, segs;       // the row, its first CTA, its ranges
  int32_t slot;                 // partial state of the first CTA: its first or second
};
struct Work {
  Record* rec;         // [ctas]
  float* row_lse2;     // [U][16]
  float2* part_ml;     // [ctas][2][16]
  float* part_o;       // [ctas][2][16][d]
  float* scores;       // [rows][G][slots], base-2 exponents; only when accumulating
};

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

size_t layout(Work* w, char* base, int64_t rows, int G, int64_t cap, int d, int ctas,
              bool accumulate) {
  const int64_t U = rows * ((G + kChunk - 1) / kChunk);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = base + at;
    at += round256(n);
    return p;
  };
  Work x;
  x.rec = reinterpret_cast<Record*>(take(size_t(ctas) * sizeof(Record)));
  x.row_lse2 = reinterpret_cast<float*>(take(accumulate ? size_t(U) * kChunk * 4 : 0));
  x.part_ml = reinterpret_cast<float2*>(take(size_t(ctas) * 2 * kChunk * 8));
  x.part_o = reinterpret_cast<float*>(take(size_t(ctas) * 2 * kChunk * d * 4));
  x.scores = reinterpret_cast<float*>(take(accumulate ? size_t(rows) * G * cap * 4 : 0));
  if (w) *w = x;
  return at;
}

struct Params {
  const int32_t* table;
  const int32_t* lens;
  int64_t num_pages;
  int32_t page_shift, max_pages, cap;
  int32_t bx_shift;            // log2 of the tokens of a unit (and of a TMA box)
  int32_t Hkv, Hq, G, HC, U;   // HC: head chunks of a row; U = rows * HC
  int32_t q_rows;              // heads of a Q box
  int32_t min_units;           // least units of a CTA
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

__device__ __forceinline__ int32_t units_of(const Params& p, int32_t len) {
  return (len + (1 << p.bx_shift) - 1) >> p.bx_shift;
}

// First unit of CTA c's range, and the CTA whose range holds unit x.
__device__ __forceinline__ int32_t range_begin(int32_t c, int32_t total, int32_t ctas) {
  return int32_t(int64_t(c) * total / ctas);
}
__device__ __forceinline__ int32_t owner(int32_t x, int32_t total, int32_t ctas) {
  return int32_t(((int64_t(x) + 1) * ctas - 1) / total);
}

__device__ __forceinline__ void store_out(const Params& p, size_t at, float v) {
  if (p.out_f32)
    static_cast<float*>(p.o)[at] = v;
  else
    static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(v);
}

// A wait's first polls leave the clock alone: reading it costs more than most
// waits here last.  Short limits go by the clock from the start.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        uint64_t limit_ns) {
  if (limit_ns >= 1000000u) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_test_sleep(bar, parity, 2000)) return true;
  }
  return mbar_wait(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_on(bar, parity, abort, limit_ns);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}
__device__ __forceinline__ bool wait_lanes(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_on(bar, parity, abort, limit_ns));
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
  static_assert(N % 16 == 0, "");
#pragma unroll
  for (int x = 0; x < N; x += 16) {
    uint32_t r[16];
    tmem_ld16(addr + x, r);
    tmem_ld_wait(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[x + i] = __uint_as_float(r[i]);
  }
}

template <int D, int GP, int PARTS>
__global__ void __launch_bounds__(kThreads, kPerSm)
    attend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const Params p) {
  using C = Cfg<D, GP, PARTS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  launch_dependents();
  wait_dependency();
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) {
      atomicOr(p.dev_status, SA_DEV_BAD_LAUNCH);
      p.w.rec[blockIdx.x] = Record{-1, 0, 0, 0};
    }
    return;
  }
  uint8_t* sKV = smem_raw;
  uint8_t* sP = sKV + C::kStages * C::kStage;
  uint8_t* sQ = sP + C::kP;
  Shared* sh = reinterpret_cast<Shared*>(sQ + C::kQs * C::kQ);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t cta = blockIdx.x;

  // ---- this CTA's range: a scan of every row's units
  const int32_t per = (p.U + kThreads - 1) / kThreads;
  const int32_t ua = min(p.U, tid * per), ub = min(p.U, ua + per);
  int32_t mine = 0;
  for (int32_t u = ua; u < ub; ++u)
    mine += units_of(p, sa_paged::row_len(p.lens, u / p.HC, p.cap, p.dev_status));
  int32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh->scan[warp] = incl;
  if (tid == 0) {
    sh->u0 = sh->p0 = 0;
    p.w.rec[cta] = Record{-1, 0, 0, 0};
  }
  __syncthreads();
  int32_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh->scan[w];
    total += sh->scan[w];
  }
  const int32_t ctas =
      max(1, min(int32_t(gridDim.x), (total + p.min_units - 1) / p.min_units));
  const int32_t a = cta < ctas ? range_begin(cta, total, ctas) : 0;
  const int32_t b = cta < ctas ? range_begin(cta + 1, total, ctas) : 0;
  if (a < b && a >= before && a < before + mine) {
    int32_t at = before;
    for (int32_t u = ua; u < ub; ++u) {
      const int32_t k = units_of(p, sa_paged::row_len(p.lens, u / p.HC, p.cap, p.dev_status));
      if (a >= at && a < at + k) {
        sh->u0 = u;
        sh->p0 = at;
        const int32_t first = owner(at, total, ctas);
        if (a > at && first == cta - 1)
          p.w.rec[cta] = Record{u, first, owner(at + k - 1, total, ctas) - first + 1,
                                at == range_begin(first, total, ctas) ? 0 : 1};
      }
      at += k;
    }
  }
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->kv_full[s], 1);
      mbar_init(&sh->kv_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh->q_full[s], 1);
      mbar_init(&sh->q_empty[s], 1);
      mbar_init(&sh->s_full[s], 1);
    }
    mbar_init(&sh->p_full, 4);                // a warp each
    mbar_init(&sh->pv_done, 1);
    mbar_init(&sh->drain, 1);
    for (int s = 0; s < kInfo; ++s) {
      mbar_init(&sh->info_full[s], 1);
      mbar_init(&sh->info_empty[s], 1 + 4);   // the issuer and the softmax warps
    }
    sh->abort = 0;
    sh->failed = 0;
    fence_mbar_init();
  }
  // rows without a token
  for (int32_t u = cta; u < p.U; u += gridDim.x) {
    if (sa_paged::row_len(p.lens, u / p.HC, p.cap, p.dev_status) > 0) continue;
    const int32_t r = u / p.HC, h0 = (u % p.HC) * kChunk;
    const size_t bh = size_t(r / p.Hkv) * p.Hq + size_t(r % p.Hkv) * p.G + h0;
    const int gc = min(kChunk, p.G - h0);
    for (int x = tid; x < gc * D; x += kThreads) store_out(p, bh * D + x, 0.f);
    if (p.lse && tid < gc) p.lse[bh + tid] = -INFINITY;
  }
  if (a >= b) return;
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int bx = 1 << p.bx_shift;

  if (warp == 0) {
    // ------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    const uint64_t pol = l2_policy_evict_first();
    const uint64_t pol_q = l2_policy_evict_last();
    int32_t u = sh->u0, pu = sh->p0;           // current row and the units before it
    int32_t ubase = u, ulen = 0;               // lane l holds the length of row ubase + l
    auto load_lens = [&]() {
      ulen = ubase + lane < p.U
                 ? sa_paged::row_len(p.lens, (ubase + lane) / p.HC, p.cap, p.dev_status) : 0;
    };
    load_lens();
    int32_t len = __shfl_sync(0xffffffffu, ulen, 0);
    int32_t t = (a - pu) << p.bx_shift;        // next token of the segment, and its end
    int32_t t1 = min(len, int32_t(min(int64_t(b - pu), int64_t(1) << 30 >> p.bx_shift) << p.bx_shift));
    bool first = true, begins = t == 0;
    int32_t seg = 0;
    bool more = true;
    // the next tile of the range; n == 0 when it is used up
    auto next = [&]() -> TileInfo {
      while (more && t >= t1) {
        pu += units_of(p, len);
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
        t1 = min(len, int32_t(min(int64_t(b - pu), int64_t(1) << 30 >> p.bx_shift) << p.bx_shift));
        if (len > 0) {
          first = true;
          begins = true;
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
      return p.table[int64_t(x.u / p.HC) * p.max_pages + (slot >> p.page_shift)];
    };
    uint32_t i = 0, qi = 0;                    // tiles and Q tiles issued
    uint32_t issued = 0;                       // stages filled
    bool ok = true;
    TileInfo cur = next();
    int32_t pg = lookup(cur);
    while (cur.n > 0) {
      const TileInfo nxt = next();
      const int32_t npg = nxt.n > 0 ? lookup(nxt) : 0;
      const int boxes = (cur.n + bx - 1) >> p.bx_shift;
      if (lane < boxes && (pg < 0 || pg >= p.num_pages)) {
        atomicOr(p.dev_status, SA_DEV_BAD_INDEX);
        pg = 0;
      }
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
          const int32_t r = cur.u / p.HC;
          const int32_t h0 = (r % p.Hkv) * p.G + (cur.u % p.HC) * kChunk;
          mbar_arrive_expect_tx(&sh->q_full[qs], C::kPanels * p.q_rows * 128);
#pragma unroll
          for (int s = 0; s < C::kPanels; ++s)
            tma_load_3d(sQ + qs * C::kQ + s * kChunk * 128, &tq, &sh->q_full[qs], s * 64, h0,
                        r / p.Hkv, pol_q);
        }
        ++qi;
      }
#pragma unroll
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
      ++i;
      cur = nxt;
      pg = npg;
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
      for (uint32_t x = issued > uint32_t(C::kStages) ? issued - C::kStages : 0; x < issued; ++x)
        mbar_wait(&sh->kv_full[x % C::kStages], (x / C::kStages) & 1, nullptr);
      for (uint32_t x = qi > uint32_t(C::kQs) ? qi - C::kQs : 0; x < qi; ++x)
        mbar_wait(&sh->q_full[x % C::kQs], (x / C::kQs) & 1, nullptr);
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
    auto issue_s = [&](uint32_t j, int32_t flags) -> bool {
      const uint32_t x = 2 * j;
      const int st = x % C::kStages;
      if ((flags & kFirst) &&
          !wait_warp(&sh->q_full[seg % C::kQs], (seg / C::kQs) & 1, abort, p.wait_ns))
        return false;
      if (!wait_warp(&sh->kv_full[st], (x / C::kStages) & 1, abort, p.wait_ns)) return false;
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
      return true;
    };
    int32_t n = 0, flags = 0;
    ok = tile(0, n, flags) && (n == 0 || issue_s(0, flags));
    for (uint32_t j = 0; ok && n > 0; ++j) {
      int32_t nn = 0, nflags = 0;
      ok = tile(j + 1, nn, nflags);
      if (!ok) break;
      // the next tile's scores go first when its keys are there
      bool early = false;
      if (nn > 0) {
        const uint32_t x = 2 * (j + 1);
        const uint32_t ready =
            mbar_test(&sh->kv_full[x % C::kStages], (x / C::kStages) & 1) ? 1u : 0u;
        early = __shfl_sync(0xffffffffu, ready, 0) != 0;
        if (early) {
          ok = issue_s(j + 1, nflags);
          if (!ok) break;
        }
      }
      const uint32_t x = 2 * j + 1;
      const int st = x % C::kStages;
      ok = wait_warp(&sh->p_full, j & 1, abort, p.wait_ns) &&
           wait_warp(&sh->kv_full[st], (x / C::kStages) & 1, abort, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = smem_desc_sw128(smem_u32(sKV + st * C::kStage), C::kPanel, 1024);
      const uint64_t pd = smem_desc_sw128(smem_u32(sP), 16, 1024);
      const int steps = (n + 15) >> 4;
      if (elect_one()) {
        for (int kk = 0; kk < steps; ++kk) {
          const uint32_t po = (kk / 4) * C::kNP * 128 + (kk % 4) * 32;
          mma_ss(tmem + C::kO, vd + uint64_t((kk * 16 * 128) >> 4), pd + uint64_t(po >> 4), idesc_o,
                 kk > 0 ? 1u : 0u);
        }
        mma_commit(&sh->pv_done);
        mma_commit(&sh->kv_empty[st]);
      }
      __syncwarp();
      if (nn > 0 && !early) ok = issue_s(j + 1, nflags);
      n = nn;
      flags = nflags;
    }
    if (lane == 0) {
      if (!ok) {
        atomicOr(p.dev_status, SA_DEV_TIMEOUT);
        *abort = 1;
      }
      // every product is complete before the tensor memory is freed
      mma_commit(&sh->drain);
      mbar_wait(&sh->drain, 0, nullptr);
    }
  } else {
    // ------------------------------------------------- softmax and output
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;       // token of the tile, dimension of O
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const float c = p.scale_log2;
    float m[GP], l[GP], o[GP];
    TileInfo prev{0, 0, 0, 0};
    bool ok = true;
    for (uint32_t j = 0;; ++j) {
      // Every wait of this tile comes before its one barrier, where the four
      // warps learn together whether one gave up.
      const int slot = j % kInfo;
      bool fail = !wait_lanes(&sh->info_full[slot], (j / kInfo) & 1, abort, p.wait_ns);
      TileInfo it{0, 0, 0, 0};
      float s[16];
      bool need = false;
      int gc = 0;
      if (!fail) {
        it = sh->info[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->info_empty[slot]);
      }
      if (!fail && it.n > 0) {
        fail = !wait_lanes(&sh->s_full[j & 1], (j >> 1) & 1, abort, p.wait_ns);
        if (!fail) {
          tc_fence_after();
          tmem_load<16>(lanes + (j & 1) * C::kNS, s);
          gc = min(kChunk, p.G - (it.u % p.HC) * kChunk);
          need = (it.flags & kFirst) != 0;
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            s[h] = (row < it.n && h < gc) ? s[h] * c : -INFINITY;
            if (!(it.flags & kFirst)) need |= s[h] > m[h] + kMove;
          }
          if (it.n < kTile) {
            // the last product step reads value rows up to the next 16th
            const uint32_t x = 2 * j + 1;
            fail = !wait_lanes(&sh->kv_full[x % C::kStages], (x / C::kStages) & 1, abort, p.wait_ns);
            if (!fail && row >= it.n && row < ((it.n + 15) & ~15)) {
              uint4* v = reinterpret_cast<uint4*>(sKV + (x % C::kStages) * C::kStage + row * 128);
#pragma unroll
              for (int s2 = 0; s2 < C::kPanels; ++s2)
#pragma unroll
                for (int y = 0; y < 8; ++y) v[s2 * (C::kPanel / 16) + y] = make_uint4(0, 0, 0, 0);
            }
          }
        }
      }
      if (!fail && j > 0) fail = !wait_lanes(&sh->pv_done, (j - 1) & 1, abort, p.wait_ns);
      if (fail) *(volatile int*)&sh->failed = 1;
      const bool any = bar_any(1, 128, need || fail);
      if (any && *(volatile int*)&sh->failed) {
        ok = false;
        break;
      }
      if (j > 0) {
        // the previous tile's product joins the segment's output
        tc_fence_after();
        float x[C::kNP];
        tmem_load<C::kNP>(lanes + C::kO, x);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          float add = x[h];
#pragma unroll
          for (int q = 1; q < PARTS; ++q) add += x[q * GP + h];
          o[h] += add;
        }
        if (prev.flags & kLast) {
          // ---- the end of a segment
#pragma unroll
          for (int h = 0; h < GP; ++h) {
#pragma unroll
            for (int w = 16; w; w >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
            if (lane == 0) sh->red[quarter][h] = l[h];
          }
          bar_sync(1, 128);
          const int32_t r = prev.u / p.HC, h0 = (prev.u % p.HC) * kChunk;
          const size_t bh = size_t(r / p.Hkv) * p.Hq + size_t(r % p.Hkv) * p.G + h0;
          const int pc = min(kChunk, p.G - h0);
          const size_t part = (size_t(cta) * 2 + ((prev.flags & kSecond) ? 1 : 0)) * kChunk;
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            if (h < pc) {
              const float L = (sh->red[0][h] + sh->red[1][h]) + (sh->red[2][h] + sh->red[3][h]);
              if (prev.flags & kComplete) {
                if (row < D) store_out(p, (bh + h) * D + row, o[h] / L);
                if (row == h) {
                  const float lse2 = (m[h] == -INFINITY ? 0.f : m[h]) + log2f(L);
                  if (p.lse) p.lse[bh + h] = lse2 * 0.6931471805599453f;
                  if (p.weights_out) p.w.row_lse2[size_t(prev.u) * kChunk + h] = lse2;
                }
              } else {
                if (row < D) p.w.part_o[(part + h) * D + row] = o[h];
                if (row == h) p.w.part_ml[part + h] = make_float2(m[h], L);
              }
            }
          }
          bar_sync(1, 128);                    // red is read before it is written again
        }
      }
      if (it.n == 0) break;
      if (it.flags & kFirst) {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          m[h] = -INFINITY;
          l[h] = 0.f;
          o[h] = 0.f;
        }
      }
      if (any) {
        // a new reference: the larger of the old one and the tile's maximum
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          float x = s[h];
#pragma unroll
          for (int w = 16; w; w >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
          if (lane == 0) sh->red[quarter][h] = x;
        }
        bar_sync(1, 128);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          const float mn = fmaxf(m[h], fmaxf(fmaxf(sh->red[0][h], sh->red[1][h]),
                                             fmaxf(sh->red[2][h], sh->red[3][h])));
          const float alpha = mn == m[h] ? 1.f : ex2(m[h] - mn);
          l[h] *= alpha;
          o[h] *= alpha;
          m[h] = mn;
        }
        bar_sync(1, 128);
      }
      if (p.weights_out && row < it.n) {
        const int32_t r = it.u / p.HC, h0 = (it.u % p.HC) * kChunk;
        float* dst = p.w.scores + (size_t(r) * p.G + h0) * p.cap + it.t + row;
#pragma unroll
        for (int h = 0; h < GP; ++h)
          if (h < gc) dst[size_t(h) * p.cap] = s[h];
      }
      // weights, in parts of bf16: row (part, head) of P, this thread's token
      // its column, in the 128-byte swizzle that the product reads
      uint8_t* col = sP + (row >> 6) * C::kNP * 128;
      const uint32_t chunk = uint32_t(row & 63) >> 3, off = uint32_t(row & 7) * 2;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float w = ex2(s[h] - (m[h] == -INFINITY ? 0.f : m[h]));
        l[h] += w;
        float rest = w;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          const int prow = q * GP + h;
          const __nv_bfloat16 x = __float2bfloat16_rn(rest);
          *reinterpret_cast<__nv_bfloat16*>(col + prow * 128 + ((chunk ^ (prow & 7)) << 4) + off) = x;
          rest -= __bfloat162float(x);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full);
      prev = it;
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

// Block (CTA c of the first launch, kJoinHeads heads): if c's range is the
// second of a row, the join of the row's partial states.  Four warps a head
// take every fourth state each, at the states' common maximum, and their sums
// are added in warp order.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Params p) {
  constexpr int kVec = D / 32;                     // elements of a lane
  constexpr int kWays = kJoinThreads / 32 / kJoinHeads;
  __shared__ float acc[kJoinHeads][kWays][D], ls[kJoinHeads][kWays];
  launch_dependents();
  wait_dependency();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Record rec = p.w.rec[blockIdx.x];
  if (rec.u < 0) return;
  const int32_t r = rec.u / p.HC, h0 = (rec.u % p.HC) * kChunk;
  const int hl = warp / kWays, way = warp % kWays;
  const int h = blockIdx.y * kJoinHeads + hl;      // head of the chunk
  const bool live = h < min(kChunk, p.G - h0);
  auto part_of = [&](int32_t k) -> size_t {
    return (size_t(rec.first + k) * 2 + (k == 0 ? rec.slot : 0)) * kChunk + h;
  };
  float M = -INFINITY;
  if (live) {
    for (int32_t k = lane; k < rec.segs; k += 32) M = fmaxf(M, p.w.part_ml[part_of(k)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, v[kVec];
#pragma unroll
    for (int x = 0; x < kVec; ++x) v[x] = 0.f;
#pragma unroll 4
    for (int32_t k = way; k < rec.segs; k += kWays) {
      const size_t at = part_of(k);
      const float2 ml = p.w.part_ml[at];
      const float f = ex2(ml.x - ref);
      L = fmaf(f, ml.y, L);
      if constexpr (kVec == 4) {
        const float4 o4 = *reinterpret_cast<const float4*>(p.w.part_o + at * D + lane * 4);
        v[0] = fmaf(f, o4.x, v[0]);
        v[1] = fmaf(f, o4.y, v[1]);
        v[2] = fmaf(f, o4.z, v[2]);
        v[3] = fmaf(f, o4.w, v[3]);
      } else {
        const float2 o2 = *reinterpret_cast<const float2*>(p.w.part_o + at * D + lane * 2);
        v[0] = fmaf(f, o2.x, v[0]);
        v[1] = fmaf(f, o2.y, v[1]);
      }
    }
#pragma unroll
    for (int x = 0; x < kVec; ++x) acc[hl][way][lane * kVec + x] = v[x];
    if (lane == 0) ls[hl][way] = L;
    M = ref;
  }
  __syncthreads();
  if (!live) return;
  float L = 0.f;
#pragma unroll
  for (int y = 0; y < kWays; ++y) L += ls[hl][y];
  const size_t bh = size_t(r / p.Hkv) * p.Hq + size_t(r % p.Hkv) * p.G + h0 + h;
  for (int x = way * 32 + lane; x < D; x += kWays * 32) {
    float sum = 0.f;
#pragma unroll
    for (int y = 0; y < kWays; ++y) sum += acc[hl][y][x];
    store_out(p, bh * D + x, sum / L);
  }
  if (way == 0 && lane == 0) {
    const float lse2 = M + log2f(L);
    if (p.lse) p.lse[bh] = lse2 * 0.6931471805599453f;
    if (p.weights_out) p.w.row_lse2[size_t(rec.u) * kChunk + h] = lse2;
  }
}

// Block (piece of a row's slots, row): every token's probabilities, summed
// over the row's heads, added to its weight.
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const Params p, int32_t pieces) {
  launch_dependents();
  wait_dependency();
  const int32_t r = blockIdx.x / pieces;
  const int32_t t0 = (blockIdx.x % pieces) * (kWeightThreads * kWeightSteps) + threadIdx.x;
  const int32_t n = sa_paged::row_len(p.lens, r, p.cap, p.dev_status);
  float sum[kWeightSteps];
#pragma unroll
  for (int i = 0; i < kWeightSteps; ++i) sum[i] = 0.f;
  if (t0 >= n) return;
  const float* s = p.w.scores + size_t(r) * p.G * p.cap;
  const float* lse2 = p.w.row_lse2 + size_t(r) * p.HC * kChunk;
#pragma unroll 4
  for (int32_t h = 0; h < p.G; ++h) {
    const float l = lse2[h];                       // chunks of 16 heads lie end to end
#pragma unroll
    for (int i = 0; i < kWeightSteps; ++i) {
      const int32_t t = t0 + i * kWeightThreads;
      if (t < n) sum[i] += ex2(s[size_t(h) * p.cap + t] - l);
    }
  }
#pragma unroll
  for (int i = 0; i < kWeightSteps; ++i) {
    const int32_t t = t0 + i * kWeightThreads;
    const size_t at = size_t(r) * p.cap + t;
    if (t < n) p.weights_out[at] = p.weights[at] + sum[i];
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
  // d = 64: the second half of the 128-row value operand lies one panel on;
  // its rows of the product are not used, but the last stage's must exist
  constexpr int kUsed = kRing + C::kP + C::kQs * C::kQ + int(sizeof(Shared));
  constexpr int kSmem = D == 64 && kUsed < kRing + C::kPanel ? kRing + C::kPanel : kUsed;
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "shared memory budget");
  const sa_paged_cache& c = a.c;
  const int64_t rows = int64_t(c.batch) * c.num_kv_heads;
  Params p{};
  p.page_shift = log2i(c.page);
  p.bx_shift = c.page < 32 ? p.page_shift : 5;
  p.G = a.Hq / c.num_kv_heads;
  p.HC = (p.G + kChunk - 1) / kChunk;
  p.q_rows = p.G < kChunk ? p.G : kChunk;
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
  p.min_units = 64 >> p.bx_shift;
  p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(D)));
  p.o = a.o;
  p.out_f32 = a.out_f32;
  p.lse = a.lse;
  p.weights = c.weights;
  p.weights_out = a.weights_out;
  p.dev_status = a.dev_status;
  p.wait_ns = a.wait_ns ? a.wait_ns : kWaitLimitNs;
  const int ctas = sms * kPerSm;
  layout(&p.w, static_cast<char*>(a.ws), rows, p.G, p.cap, D, ctas, a.weights_out != nullptr);
  auto kern = attend_kernel<D, GP, PARTS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
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
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  e = cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned(ctas), unsigned((p.q_rows + kJoinHeads - 1) / kJoinHeads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
  if (e != cudaSuccess || !a.weights_out) return e;
  constexpr int kPiece = kWeightThreads * kWeightSteps;
  const int32_t pieces = (p.cap + kPiece - 1) / kPiece;
  if (rows * pieces > INT32_MAX) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(unsigned(rows * pieces));
  cfg.blockDim = dim3(kWeightThreads);
  return cudaLaunchKernelEx(&cfg, weights_kernel, p, pieces);
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed) {
  const int G = a.Hq / a.c.num_kv_heads;
  if (a.out_f32) {
    if (G <= 4) return launch<D, 4, 3>(a, sms, st, encode_failed);
    if (G <= 8) return launch<D, 8, 3>(a, sms, st, encode_failed);
    return launch<D, 16, 3>(a, sms, st, encode_failed);
  }
  if (G <= 4) return launch<D, 4, 2>(a, sms, st, encode_failed);
  if (G <= 8) return launch<D, 8, 2>(a, sms, st, encode_failed);
  return launch<D, 16, 2>(a, sms, st, encode_failed);
}

}  // namespace

namespace sa_paged {

size_t attend_workspace(const sa_paged_cache& c, int32_t Hq, bool accumulate, int sms) {
  return layout(nullptr, nullptr, int64_t(c.batch) * c.num_kv_heads, Hq / c.num_kv_heads,
                int64_t(c.page) * c.max_pages, c.head_dim, sms * kPerSm, accumulate);
}

cudaError_t launch_attend(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed) {
  *encode_failed = false;
  return a.c.head_dim == 128 ? launch_d<128>(a, sms, st, encode_failed)
                             : launch_d<64>(a, sms, st, encode_failed);
}

}  // namespace sa_paged
