// Evicting tokens from a paged key-value cache by accumulated weight.
//
// A token's 32-bit key orders it: all ones for the first `sinks` and last
// `recent` positions, else the weight's bits mapped so that unsigned order is
// the floats' order (NaN below every number, -0 as +0).  Per row:
//
//   select   the m-th largest key T, digit by digit from the top: a histogram
//            of the keys that agree with T so far, and the bin that holds the
//            m-th.  When a bin is kept whole its lower digits do not matter.
//            Tokens above T are kept, and of those equal to T the lowest slots
//            until m are.
//   number   with K(t) the kept slots below t, an evicted slot t < m is hole
//            t - K(t) and a kept slot t >= m is source K(t) - K(m): one prefix
//            count gives both lists, in slot order.
//   move     source i goes into hole i.  Sources lie at m or above and holes
//            below, so no move reads what another writes, and only the tokens
//            that have to move are touched.
//
// Rows of up to 8192 slots: one CTA, the keys in registers (evict_row_kernel).
// Its time is a chain of latencies, not of bytes (in a cluster of two, with
// passes of 8 bits: 30 us where it takes 8), so it has as few barriers as it
// can: digits of 11 bits, histograms cleared ahead, lists in shared memory.
// Longer rows: a cluster of 2 to 8 CTAs, each with a contiguous slice whose
// keys stay in its shared memory; histograms and counts are added up over the
// cluster through distributed shared memory (evict_cluster_kernel).
// The moves of a short row are made by its own CTA; those of long rows, or of
// few rows with much to move, by a second launch over all processors
// (move_kernel).
//
// Measured: 256 rows of 544 to 2080 slots cut by 32: 7.7 us, 1.9 of them for
// the bytes (the kernels go by the table, not by the lengths: with 4096 slots
// to a row of the table 23 us, with 16384 or more 35); 16 rows of 2048 to 4096
// cut to 512 to 1024: 8.3 us in two launches; 32 rows of 32768 cut to 1024 to 8192: 34 us, 16 for the select (a
// chain of cluster barriers, each with a histogram added up across it) and 18
// for the moves' 109 MB, 6.0 TB/s.

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "paged.h"
#include "ptx.cuh"

namespace {

namespace cg = cooperative_groups;
using sa_paged::EvictArgs;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 8;
constexpr int kMaxSlice = 32768;       // keys of a cluster's CTA: 128 KB of shared memory
constexpr int kRowKeys = 16;           // keys of a thread where a CTA has the whole row
constexpr int kRowSlots = kThreads * kRowKeys;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 128;
constexpr int kMaxRanks = 8;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ bool is_forced(const EvictArgs& a, int32_t pos, int32_t newest) {
  return pos < a.sinks || (a.recent > 0 && int64_t(pos) > int64_t(newest) - a.recent);
}

// Workspace: the numbers of moves [rows], then two lists of at most cap / 2
// slots a row.
struct Work {
  int32_t* pairs;
  int32_t* lists;      // [rows][cap]: holes, then sources
};
__host__ __device__ __forceinline__ Work work_of(const EvictArgs& a) {
  const int64_t rows = int64_t(a.c.batch) * a.c.num_kv_heads;
  int32_t* p = static_cast<int32_t*>(a.ws);
  return Work{p, p + ((rows + 63) & ~int64_t(63))};
}

// Moves [g, g + group) of a row, one warp: lane i < group has pair i's slots in
// (s, t), or s < 0.  A token of d/8 lanes a key (or value) row, 16 bytes a
// lane; all loads of the group are in flight before its first store.
template <int D>
struct Mover {
  static constexpr int kPiece = D / 8;                  // lanes of one row
  static constexpr int kPer = 32 / (2 * kPiece);        // tokens of one step
  static constexpr int kGroup = kSteps * kPer;
  static __device__ __forceinline__ void move(const EvictArgs& a, int64_t r, int32_t s,
                                              int32_t t) {
    const int lane = threadIdx.x & 31;
    const int32_t cap = a.c.page * a.c.max_pages;
    const int32_t* table = a.c.table + r * a.c.max_pages;
    const int shift = __ffs(a.c.page) - 1;              // pages are powers of two
    int32_t sp = -1, tp = -1, so = 0, to = 0;
    if (s >= 0) {
      sp = table[s >> shift];
      tp = table[t >> shift];
      so = s & (a.c.page - 1);
      to = t & (a.c.page - 1);
      // (read beside the pages: a chain of loads less)
      const float w = a.c.weights[r * cap + s];
      const int32_t pos = a.positions_out ? a.c.positions[r * cap + s] : 0;
      if (sp < 0 || sp >= a.c.num_pages || tp < 0 || tp >= a.c.num_pages) {
        // the token stays where it is, and so does what the hole holds
        atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
        sp = -1;
      } else {
        a.weights_out[r * cap + t] = w;
        if (a.positions_out) a.positions_out[r * cap + t] = pos;
      }
    }
    const bool is_v = (lane / kPiece) & 1;
    const int sub = lane / (2 * kPiece);
    const int64_t stride = is_v ? a.c.v_page_stride : a.c.k_page_stride;
    __nv_bfloat16* pool =
        static_cast<__nv_bfloat16*>(is_v ? a.c.v_pages : a.c.k_pages) + (lane % kPiece) * 8;
    uint4 val[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int32_t p = __shfl_sync(0xffffffffu, sp, i * kPer + sub);
      const int32_t x = __shfl_sync(0xffffffffu, so, i * kPer + sub);
      if (p >= 0) val[i] = *reinterpret_cast<const uint4*>(pool + p * stride + int64_t(x) * D);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const bool ok = __shfl_sync(0xffffffffu, sp, i * kPer + sub) >= 0;
      const int32_t p = __shfl_sync(0xffffffffu, tp, i * kPer + sub);
      const int32_t x = __shfl_sync(0xffffffffu, to, i * kPer + sub);
      if (ok) *reinterpret_cast<uint4*>(pool + p * stride + int64_t(x) * D) = val[i];
    }
  }
};

// What the select of a row shares.  Three histograms of the row, cleared
// ahead, one for each digit.
struct Select {
  alignas(16) int32_t hist[3][kBins];
  int32_t warp_total[kWarps];
  alignas(16) int4 found;              // bin, how many of it are kept, how many it has
};

__device__ __forceinline__ void clear(Select& sel) {
  int4* h = reinterpret_cast<int4*>(&sel.hist[0][0]);
#pragma unroll
  for (int x = 0; x < 3 * kBins / 4 / kThreads; ++x)
    h[threadIdx.x + x * kThreads] = make_int4(0, 0, 0, 0);
}

// The `need`-th largest key, by digits of 11, 11 and 10 bits.  each(f) calls
// f(key) for this thread's keys.  With kCluster the CTAs of the cluster hold
// parts of the row: each counts into `local` (cleared) and adds what is not
// zero to the first CTA's histogram, which finds the bin and tells the others.
// (Every CTA reading all the others' bins took 10000 cycles a digit, every CTA
// adding to all the others' 7700.)  Returns T, and in `need` how many
// of the keys equal to T are kept; tied = false: all of them (T's lower bits
// are then zero where a whole bin is kept, and a key is kept if it is >= T).
template <bool kCluster, class Each>
__device__ __forceinline__ uint32_t radix_select(Select& sel, int32_t* local, int rank,
                                                 int ranks, Each each, int32_t& need,
                                                 bool& tied) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kMine = kBins / kThreads;            // bins of a thread
  static_assert(kMine == 4, "an int4 of bins a thread");
  uint32_t T = 0;
  tied = true;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    int32_t* hist = kCluster ? local : sel.hist[pass];
    each([&](uint32_t k) {
      if (((k ^ T) & mask) == 0) atomicAdd(&hist[(k >> shift) & digit], 1);
    });
    __syncthreads();
    // thread x has the x-th four bins from the top
    const int at = kBins / 4 - 1 - tid;
    if (kCluster) {
      int4* part = reinterpret_cast<int4*>(local) + at;
      const int4 y = *part;
      *part = make_int4(0, 0, 0, 0);
      if (y.x | y.y | y.z | y.w) {
        int32_t* to = cg::this_cluster().map_shared_rank(&sel, 0)->hist[pass] + 4 * at;
        if (y.x) atomicAdd(to, y.x);
        if (y.y) atomicAdd(to + 1, y.y);
        if (y.z) atomicAdd(to + 2, y.z);
        if (y.w) atomicAdd(to + 3, y.w);
      }
      cg::this_cluster().sync();
    }
    if (!kCluster || rank == 0) {
      const int4 c = reinterpret_cast<const int4*>(sel.hist[pass])[at];
      const int32_t sum = (c.x + c.y) + (c.z + c.w);
      int32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
      }
      if (lane == 31) sel.warp_total[warp] = before;
      before -= sum;
      __syncthreads();
#pragma unroll
      for (int x = 0; x < kWarps; ++x)
        if (x < warp) before += sel.warp_total[x];
      if (before < need && before + sum >= need) {
        int b = 4 * at + 3, n = c.w;
        if (before + n < need) { before += n; --b; n = c.z; }
        if (before + n < need) { before += n; --b; n = c.y; }
        if (before + n < need) { before += n; --b; n = c.x; }
        const int4 f = make_int4(b, need - before, n, 0);
        if (kCluster)
          for (int x = 0; x < ranks; ++x) cg::this_cluster().map_shared_rank(&sel, x)->found = f;
        else
          sel.found = f;
      }
    }
    if (kCluster)
      cg::this_cluster().sync();
    else
      __syncthreads();
    const int4 f = sel.found;
    T |= uint32_t(f.x) << shift;
    need = f.y;
    if (f.z == need) {
      tied = false;
      break;
    }
  }
  return T;
}

// ---------------------------------------------------------------- one CTA a row
struct RowShared {
  Select sel;
  uint16_t dst[kRowSlots / 2], src[kRowSlots / 2];
  int32_t warp_count[kWarps][2];
  int32_t newest;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    evict_row_kernel(const __grid_constant__ EvictArgs a, int moves_here) {
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sa_dev::launch_dependents();
  if (tid == 0) sh.newest = INT32_MIN;
  clear(sh.sel);
  __syncthreads();
  sa_dev::wait_dependency();
  const int64_t r = blockIdx.x;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t n = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int32_t m = min(n, a.keep[r % a.c.num_kv_heads]);
  const float* w = a.c.weights + r * cap;
  const int32_t* pos = a.c.positions ? a.c.positions + r * cap : nullptr;
  float* wo = a.weights_out + r * cap;
  int32_t* po = a.positions_out ? a.positions_out + r * cap : nullptr;
  const bool copy_w = wo != w, copy_p = po && po != pos;
  const Work ws = work_of(a);
  if (m == n || m == 0) {              // nothing, or everything, goes
    for (int32_t t = tid; t < m; t += kThreads) {
      if (copy_w) wo[t] = w[t];
      if (copy_p) po[t] = pos[t];
    }
    if (tid == 0) {
      a.lens_out[r] = m;
      if (!moves_here) ws.pairs[r] = 0;
    }
    return;
  }

  // ---- keys: a warp has consecutive slots, 32 a step
  const int per = (n + kThreads - 1) / kThreads;       // steps
  const int32_t w0 = warp * per * 32 + lane;           // this lane's first slot
  uint32_t key[kRowKeys];
  uint32_t live = 0;                   // bit j: slot j of this lane is in the row
  {
    float x[kRowKeys];
    int32_t q[kRowKeys];
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      const int32_t t = w0 + j * 32;
      x[j] = 0.f;
      q[j] = INT32_MIN;
      if (t < n) {
        x[j] = w[t];
        q[j] = pos ? pos[t] : t;
        live |= 1u << j;
      }
    }
    int32_t newest = INT32_MIN;
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      newest = max(newest, q[j]);
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) atomicMax(&sh.newest, newest);
    // the new state's slots, as they are: moves overwrite the holes later
    if (copy_w || copy_p) {
#pragma unroll
      for (int j = 0; j < kRowKeys; ++j) {
        if (j >= per) break;
        const int32_t t = w0 + j * 32;
        if (t < m) {
          if (copy_w) wo[t] = x[j];
          if (copy_p) po[t] = q[j];
        }
      }
    }
    __syncthreads();
    newest = sh.newest;
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      key[j] = is_forced(a, q[j], newest) ? 0xFFFFFFFFu : weight_key(x[j]);
    }
  }

  // ---- select
  int32_t need = m;
  bool tied;
  const uint32_t T = radix_select<false>(
      sh.sel, nullptr, 0, 1,
      [&](auto f) {
#pragma unroll
        for (int j = 0; j < kRowKeys; ++j) {
          if (j >= per) break;
          if (live >> j & 1u) f(key[j]);
        }
      },
      need, tied);

  // ---- number
  const uint32_t lower = (1u << lane) - 1u;
  uint32_t kept = 0;                   // bit j
  if (!tied) {
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      if ((live >> j & 1u) && key[j] >= T) kept |= 1u << j;
    }
  } else {
    int32_t ties = 0;
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      ties += __popc(__ballot_sync(0xffffffffu, (live >> j & 1u) && key[j] == T));
    }
    if (lane == 0) sh.warp_count[warp][0] = ties;
    __syncthreads();
    int32_t t = 0;
#pragma unroll
    for (int x = 0; x < kWarps; ++x)
      if (x < warp) t += sh.warp_count[x][0];
#pragma unroll
    for (int j = 0; j < kRowKeys; ++j) {
      if (j >= per) break;
      const bool in = live >> j & 1u, eq = in && key[j] == T;
      const uint32_t b = __ballot_sync(0xffffffffu, eq);
      if (in && (key[j] > T || (eq && t + __popc(b & lower) < need))) kept |= 1u << j;
      t += __popc(b);
    }
    __syncthreads();
  }
  // kept slots of the warp, and those below m; `low` has this lane's share
  const int below = min(max((m - w0 + 31) >> 5, 0), per);      // this lane's slots below m
  int32_t low = __reduce_add_sync(0xffffffffu, __popc(kept & ((1u << below) - 1u)));
  const int32_t count = __reduce_add_sync(0xffffffffu, __popc(kept));
  if (lane == 0) {
    sh.warp_count[warp][0] = count;
    sh.warp_count[warp][1] = low;
  }
  __syncthreads();
  int32_t K = 0, Km = 0;
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
    if (x < warp) K += sh.warp_count[x][0];
    Km += sh.warp_count[x][1];
  }
  const int32_t pairs = m - Km;
  int32_t* list = ws.lists + r * cap;
#pragma unroll 1
  for (int j = 0; j < per; ++j) {
    const bool keep = kept >> j & 1u;
    const uint32_t b = __ballot_sync(0xffffffffu, keep);
    const int32_t t = w0 + j * 32, k = K + __popc(b & lower);
    if (t < m && !keep) {
      if (moves_here)
        sh.dst[t - k] = uint16_t(t);
      else
        list[t - k] = t;
    }
    if (t >= m && keep) {
      if (moves_here)
        sh.src[k - Km] = uint16_t(t);
      else
        list[cap / 2 + k - Km] = t;
    }
    K += __popc(b);
  }
  if (tid == 0) {
    a.lens_out[r] = m;
    if (!moves_here) ws.pairs[r] = pairs;
  }
  if (!moves_here) return;
  __syncthreads();
  constexpr int kGroup = Mover<D>::kGroup;
  for (int32_t g = warp * kGroup; g < pairs; g += kWarps * kGroup) {
    const bool on = lane < kGroup && g + lane < pairs;
    Mover<D>::move(a, r, on ? int32_t(sh.src[g + lane]) : -1, on ? int32_t(sh.dst[g + lane]) : 0);
  }
}

// Block (piece of a row's moves, row).
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a,
                                                            int32_t pieces) {
  constexpr int kGroup = Mover<D>::kGroup;
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const Work ws = work_of(a);
  const int64_t r = blockIdx.x / pieces;
  const int32_t pairs = ws.pairs[r];
  const int lane = threadIdx.x & 31;
  const int32_t g =
      (int32_t(blockIdx.x % pieces) * (kMoveThreads / 32) + int32_t(threadIdx.x >> 5)) * kGroup;
  if (g >= pairs) return;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t* list = ws.lists + r * cap;
  const bool on = lane < kGroup && g + lane < pairs;
  Mover<D>::move(a, r, on ? list[cap / 2 + g + lane] : -1, on ? list[g + lane] : 0);
}

// ---------------------------------------------------------------- a cluster a row
struct Shared {
  Select sel;
  alignas(16) int32_t local[kBins];
  int32_t warp_count[kWarps][2];
  // what every CTA of the cluster writes into each
  int32_t newest;
  int32_t ties[kMaxRanks], kept[kMaxRanks], low[kMaxRanks];
};

// Sum over the CTA of (x, y), by every thread; each warp passes its own counts
// (the same in all its lanes) and gets those of the warps before it.
__device__ __forceinline__ int2 before_in_block(Shared& sh, int2 mine, int2& total) {
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.warp_count[warp][0] = mine.x;
    sh.warp_count[warp][1] = mine.y;
  }
  __syncthreads();
  int2 before = make_int2(0, 0);
  total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = sh.warp_count[w][0], y = sh.warp_count[w][1];
    if (w < warp) {
      before.x += x;
      before.y += y;
    }
    total.x += x;
    total.y += y;
  }
  return before;
}

__global__ void __launch_bounds__(kThreads)
    evict_cluster_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ Shared sh;
  extern __shared__ uint32_t keys[];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sa_dev::launch_dependents();
  clear(sh.sel);
  reinterpret_cast<int4*>(sh.local)[tid] = make_int4(0, 0, 0, 0);
  if (tid == 0) sh.newest = INT32_MIN;
  auto ready = cluster.barrier_arrive();       // cleared, for the others to write
  sa_dev::wait_dependency();
  const int64_t r = blockIdx.x / ranks;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t n = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int32_t m = min(n, a.keep[r % a.c.num_kv_heads]);
  const float* w = a.c.weights + r * cap;
  const int32_t* pos = a.c.positions ? a.c.positions + r * cap : nullptr;
  float* wo = a.weights_out + r * cap;
  int32_t* po = a.positions_out ? a.positions_out + r * cap : nullptr;
  const bool copy_w = wo != w, copy_p = po && po != pos;
  const Work ws = work_of(a);

  if (m == n || m == 0) {              // nothing, or everything, goes
    for (int32_t t = rank * kThreads + tid; t < m; t += ranks * kThreads) {
      if (copy_w) wo[t] = w[t];
      if (copy_p) po[t] = pos[t];
    }
    if (rank == 0 && tid == 0) {
      a.lens_out[r] = m;
      ws.pairs[r] = 0;
    }
    cluster.barrier_wait(std::move(ready));
    return;
  }

  // this CTA's slots [lo, lo + ns), a warp's [w0, w1) of them
  const int32_t slice = ((n + ranks - 1) / ranks + 31) & ~31;
  const int32_t lo = min(n, rank * slice), ns = min(n, lo + slice) - lo;
  const int32_t part = ((slice + kWarps - 1) / kWarps + 31) & ~31;
  const int32_t w0 = min(ns, warp * part), w1 = min(ns, w0 + part);

  // ---- keys, and the new state's slots as they are: moves overwrite the
  // holes later
  int32_t newest = pos ? INT32_MIN : n - 1;
  constexpr int kBatch = 8;
  for (int32_t i0 = tid; i0 < ns; i0 += kBatch * kThreads) {
    float x[kBatch];
    int32_t q[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int32_t i = i0 + y * kThreads;
      if (i < ns) {
        x[y] = w[lo + i];
        q[y] = pos ? pos[lo + i] : lo + i;
      }
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int32_t i = i0 + y * kThreads;
      if (i < ns) {
        keys[i] = weight_key(x[y]);
        newest = max(newest, q[y]);
        if (lo + i < m) {
          if (copy_w) wo[lo + i] = x[y];
          if (copy_p) po[lo + i] = q[y];
        }
      }
    }
  }
  cluster.barrier_wait(std::move(ready));
  if (pos && a.recent > 0) {
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) sh.warp_count[warp][0] = newest;
    __syncthreads();
    if (tid < ranks) {
#pragma unroll
      for (int x = 0; x < kWarps; ++x) newest = max(newest, sh.warp_count[x][0]);
      atomicMax(&cluster.map_shared_rank(&sh, tid)->newest, newest);
    }
    cluster.sync();
    newest = sh.newest;
  }
  if (a.sinks > 0 || a.recent > 0) {
    for (int32_t i0 = tid; i0 < ns; i0 += kBatch * kThreads) {
      int32_t q[kBatch];
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        const int32_t i = i0 + y * kThreads;
        if (i < ns) q[y] = pos ? pos[lo + i] : lo + i;
      }
#pragma unroll
      for (int y = 0; y < kBatch; ++y) {
        const int32_t i = i0 + y * kThreads;
        if (i < ns && is_forced(a, q[y], newest)) keys[i] = 0xFFFFFFFFu;
      }
    }
  }
  // ---- select
  int32_t need = m;
  bool tied;
  const uint32_t T = radix_select<true>(
      sh.sel, sh.local, rank, ranks,
      [&](auto f) {
        for (int32_t i0 = tid; i0 < ns; i0 += kBatch * kThreads) {
          uint32_t k[kBatch];
#pragma unroll
          for (int y = 0; y < kBatch; ++y) {
            const int32_t i = i0 + y * kThreads;
            if (i < ns) k[y] = keys[i];
          }
#pragma unroll
          for (int y = 0; y < kBatch; ++y)
            if (i0 + y * kThreads < ns) f(k[y]);
        }
      },
      need, tied);

  // ---- number: ties in slot order where they matter, then kept slots
  const uint32_t lower = (1u << lane) - 1u;
  int2 total;
  int32_t tie = 0;
  if (tied) {
    int32_t ties = 0;
    for (int32_t i = w0; i < w1; i += 32) {
      const bool eq = i + lane < w1 && keys[i + lane] == T;
      ties += __popc(__ballot_sync(0xffffffffu, eq));
    }
    tie = before_in_block(sh, make_int2(ties, 0), total).x;
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->ties[rank] = total.x;
    cluster.sync();
    for (int x = 0; x < rank; ++x) tie += sh.ties[x];
  }
  // a warp's own slots become flags: kept or not
  int32_t count = 0, low = 0;
  int32_t t = tie;
#pragma unroll 4
  for (int32_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? keys[i + lane] : 0u;
    bool kept = in && k >= T;
    if (tied) {
      const bool eq = in && k == T;
      const uint32_t b = __ballot_sync(0xffffffffu, eq);
      kept = in && (k > T || (eq && t + __popc(b & lower) < need));
      t += __popc(b);
    }
    if (in) keys[i + lane] = kept;
    count += kept;
    low += kept && lo + i + lane < m;
  }
  count = __reduce_add_sync(0xffffffffu, count);
  low = __reduce_add_sync(0xffffffffu, low);
  int32_t K = before_in_block(sh, make_int2(count, low), total).x;
  if (tid < ranks) {
    cluster.map_shared_rank(&sh, tid)->kept[rank] = total.x;
    cluster.map_shared_rank(&sh, tid)->low[rank] = total.y;
  }
  cluster.sync();                      // the last access to another CTA's shared memory
  int32_t Km = 0;
  for (int x = 0; x < ranks; ++x) {
    if (x < rank) K += sh.kept[x];
    Km += sh.low[x];
  }
  if (rank == 0 && tid == 0) {
    a.lens_out[r] = m;
    ws.pairs[r] = m - Km;
  }
  int32_t* list = ws.lists + r * cap;
#pragma unroll 4
  for (int32_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const bool kept = in && keys[i + lane];
    const uint32_t b = __ballot_sync(0xffffffffu, kept);
    const int32_t slot = lo + i + lane, k = K + __popc(b & lower);
    if (in && slot < m && !kept) list[slot - k] = slot;
    if (in && slot >= m && kept) list[cap / 2 + k - Km] = slot;
    K += __popc(b);
  }
}

template <int D>
cudaError_t launch(const EvictArgs& a, int sms, cudaStream_t st) {
  const int64_t cap = int64_t(a.c.page) * a.c.max_pages;
  const int64_t rows = int64_t(a.c.batch) * a.c.num_kv_heads;
  // the most moves that a row can have: no more than it keeps, or loses
  int64_t most = 0;
  for (int32_t g = 0; g < a.c.num_kv_heads; ++g)
    most = std::max(most, std::min<int64_t>(a.keep[g], cap - std::min<int64_t>(a.keep[g], cap)));
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cudaError_t e;
  if (cap <= kRowSlots) {
    // One launch where a row can have little to move, or the rows fill the
    // processors and can have only a kilotoken each.  (256 rows of up to 950
    // possible and 32 actual moves: 8.5 us, and 15.5 in two launches, whose
    // blocks are one for each possible piece of a row; 512 rows of 2048 moves:
    // 109 us, and 106 in two; 16 rows of up to 1024 moves: 15.9, and 8.6.)
    const bool moves_here = most <= (rows >= sms ? 1024 : 256);
    cfg.gridDim = dim3(unsigned(rows));
    e = cudaLaunchKernelEx(&cfg, evict_row_kernel<D>, a, int(moves_here));
    if (e != cudaSuccess || moves_here) return e;
  } else {
    // the least CTAs a row that hold its keys, then more while processors are
    // left and a slice is worth a CTA's while
    int ranks = 2;
    while (ranks < kMaxRanks && ((cap + ranks - 1) / ranks > kMaxSlice ||
                                 (rows * ranks < sms && cap / ranks > 2048)))
      ranks *= 2;
    const int64_t slice = ((cap + ranks - 1) / ranks + 31) & ~int64_t(31);
    if (rows * ranks > INT32_MAX) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    e = sa_paged::allow_shared(evict_cluster_kernel, kMaxSlice * 4, done);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(unsigned(rows * ranks));
    cfg.dynamicSmemBytes = size_t(slice) * 4;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_cluster_kernel, a);
    if (e != cudaSuccess) return e;
  }
  constexpr int kPiece = kMoveThreads / 32 * Mover<D>::kGroup;
  const int64_t pieces = (most + kPiece - 1) / kPiece;
  if (pieces == 0) return cudaSuccess;
  if (rows * pieces > INT32_MAX) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(unsigned(rows * pieces));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel<D>, a, int32_t(pieces));
}

}  // namespace

namespace sa_paged {

size_t evict_workspace(const sa_paged_cache& c) {
  const int64_t rows = int64_t(c.batch) * c.num_kv_heads;
  return (size_t((rows + 63) & ~int64_t(63)) + size_t(rows) * c.page * c.max_pages) *
         sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t st) {
  return a.c.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace sa_paged
