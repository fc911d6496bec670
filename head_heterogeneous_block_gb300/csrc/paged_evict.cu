// Evicting tokens from a paged key-value cache by accumulated weight.
//
// A token's 32-bit key orders it: all ones for the first `sinks` and last
// `recent` positions, else the weight's bits mapped so that unsigned order is
// the floats' order (NaN below every number, -0 as +0).  Per row:
//
//   select   the m-th largest key T, by four passes of 8 bits from the top: a
//            histogram of the keys that agree with T so far, and the bin that
//            holds the m-th.  Tokens above T are kept, and of those equal to T
//            the lowest slots until m are.
//   number   with K(t) the kept slots below t, an evicted slot t < m is hole
//            t - K(t) and a kept slot t >= m is source K(t) - K(m): one prefix
//            count gives both lists, in slot order.
//   move     source i goes into hole i.  Sources lie at m or above and holes
//            below, so no move reads what another writes, and only the tokens
//            that have to move are touched.
//
// A row is worked on by a cluster of 1 to 8 CTAs, each with a contiguous slice
// of the slots, whose keys stay in shared memory between the passes (the
// weights and positions are read from memory once, or twice for positions);
// histograms and counts are added up over the cluster through distributed
// shared memory.  Moves are spread over the cluster's warps, 8 steps of loads
// in flight each.

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "paged.h"

namespace {

namespace cg = cooperative_groups;
using sa_paged::EvictArgs;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 8;
constexpr int kMaxSlice = 32768;       // keys of a CTA: 128 KB of shared memory

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Shared {
  int32_t hist[2][256];    // by pass parity: the other CTAs may still read the last one
  int32_t warp_count[kWarps][2];
  int32_t bins[8];
  int32_t share[3][2];     // [0] largest position; [1] ties; [2] kept, kept below m
  int32_t bin, need;
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

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ Shared sh;
  extern __shared__ uint32_t keys[];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / ranks;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t n = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int32_t m = min(n, a.keep[r % a.c.num_kv_heads]);
  const float* w = a.c.weights + r * cap;
  const int32_t* pos = a.c.positions ? a.c.positions + r * cap : nullptr;
  float* wo = a.weights_out + r * cap;
  int32_t* po = a.positions_out ? a.positions_out + r * cap : nullptr;
  const bool copy_w = wo != w, copy_p = po && po != pos;

  if (m == n || m == 0) {              // nothing, or everything, goes
    for (int32_t t = rank * kThreads + tid; t < m; t += ranks * kThreads) {
      if (copy_w) wo[t] = w[t];
      if (copy_p) po[t] = pos[t];
    }
    if (rank == 0 && tid == 0) a.lens_out[r] = m;
    return;
  }

  // this CTA's slots [lo, lo + ns), a warp's [w0, w1) of them
  const int32_t slice = ((n + ranks - 1) / ranks + 31) & ~31;
  const int32_t lo = min(n, rank * slice), ns = min(n, lo + slice) - lo;
  const int32_t part = ((slice + kWarps - 1) / kWarps + 31) & ~31;
  const int32_t w0 = min(ns, warp * part), w1 = min(ns, w0 + part);

  // ---- keys
  int32_t newest = pos ? INT32_MIN : n - 1;
#pragma unroll 4
  for (int32_t i = tid; i < ns; i += kThreads) {
    keys[i] = weight_key(w[lo + i]);
    if (pos) newest = max(newest, pos[lo + i]);
  }
  if (pos && a.recent > 0) {
#pragma unroll
    for (int o = 16; o; o >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, o));
    if (lane == 0) sh.warp_count[warp][0] = newest;
    __syncthreads();
    for (int x = 0; x < kWarps; ++x) newest = max(newest, sh.warp_count[x][0]);
    if (ranks > 1) {
      if (tid == 0) sh.share[0][0] = newest;
      cluster.sync();
      for (int x = 0; x < ranks; ++x)
        newest = max(newest, cluster.map_shared_rank(&sh, x)->share[0][0]);
    }
  }
  if (a.sinks > 0 || a.recent > 0) {
    const int64_t from = int64_t(newest) - a.recent;
#pragma unroll 4
    for (int32_t i = tid; i < ns; i += kThreads) {
      const int32_t q = pos ? pos[lo + i] : lo + i;
      if (q < a.sinks || (a.recent > 0 && int64_t(q) > from)) keys[i] = 0xFFFFFFFFu;
    }
  }

  // ---- select
  uint32_t T = 0;
  int32_t need = m;                    // of the keys that agree with T so far
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int32_t* hist = sh.hist[pass & 1];
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll 4
    for (int32_t i = tid; i < ns; i += kThreads) {
      const uint32_t k = keys[i];
      if (((k ^ T) & mask) == 0) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
    int32_t mine = 0, above = 0;
    if (tid < 256) {
      // thread x has bin 255 - x, so that a prefix sum counts from the top
      mine = 0;
      for (int x = 0; x < ranks; ++x)
        mine += (ranks > 1 ? cluster.map_shared_rank(&sh, x) : &sh)->hist[pass & 1][255 - tid];
      above = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += x;
      }
      if (lane == 31) sh.bins[warp] = above;
    }
    __syncthreads();
    if (tid < 256) {
      for (int x = 0; x < warp; ++x) above += sh.bins[x];
      if (above >= need && above - mine < need) {
        sh.bin = 255 - tid;
        sh.need = need - (above - mine);
      }
    }
    __syncthreads();
    T |= uint32_t(sh.bin) << shift;
    need = sh.need;
  }

  // ---- number: ties in slot order, then kept slots
  int32_t ties = 0;
  for (int32_t i = w0; i < w1; i += 32) {
    const bool eq = i + lane < w1 && keys[i + lane] == T;
    ties += __popc(__ballot_sync(0xffffffffu, eq));
  }
  int2 total;
  int32_t tie = before_in_block(sh, make_int2(ties, 0), total).x;
  if (ranks > 1) {
    if (tid == 0) sh.share[1][0] = total.x;
    cluster.sync();
    for (int x = 0; x < rank; ++x) tie += cluster.map_shared_rank(&sh, x)->share[1][0];
  }
  const uint32_t lower = (1u << lane) - 1u;
  // whether slot i of the slice is kept; t runs over the ties before the warp's place
  auto kept_at = [&](int32_t i, int32_t& t) -> bool {
    const uint32_t k = i + lane < w1 ? keys[i + lane] : 0u;
    const bool eq = i + lane < w1 && k == T;
    const uint32_t b = __ballot_sync(0xffffffffu, eq);
    const bool kept = i + lane < w1 && (k > T || (eq && t + __popc(b & lower) < need));
    t += __popc(b);
    return kept;
  };
  int2 count = make_int2(0, 0);
  int32_t t = tie;
  for (int32_t i = w0; i < w1; i += 32) {
    const uint32_t b = __ballot_sync(0xffffffffu, kept_at(i, t));
    count.x += __popc(b);
    const int32_t below = m - (lo + i);          // slots of this step below m
    count.y += below >= 32 ? __popc(b) : below > 0 ? __popc(b & ((1u << below) - 1u)) : 0;
  }
  int32_t K = before_in_block(sh, count, total).x;
  int32_t Km = total.y;
  if (ranks > 1) {
    if (tid == 0) {
      sh.share[2][0] = total.x;
      sh.share[2][1] = total.y;
    }
    cluster.sync();
    Km = 0;
    for (int x = 0; x < ranks; ++x) {
      const Shared* other = cluster.map_shared_rank(&sh, x);
      if (x < rank) K += other->share[2][0];
      Km += other->share[2][1];
    }
  }
  const int32_t pairs = m - Km;
  int32_t* dst_list = static_cast<int32_t*>(a.ws) + r * cap;
  int32_t* src_list = dst_list + cap / 2;
  t = tie;
  for (int32_t i = w0; i < w1; i += 32) {
    const bool kept = kept_at(i, t);
    const uint32_t b = __ballot_sync(0xffffffffu, kept);
    const int32_t slot = lo + i + lane, k = K + __popc(b & lower);
    if (i + lane < w1) {
      if (slot < m && !kept) dst_list[slot - k] = slot;
      if (slot >= m && kept) src_list[k - Km] = slot;
      if (slot < m && kept) {
        if (copy_w) wo[slot] = w[slot];
        if (copy_p) po[slot] = pos[slot];
      }
    }
    K += __popc(b);
  }
  // every list entry is written, and no CTA reads another's shared memory any more
  if (ranks > 1)
    cluster.sync();
  else
    __syncthreads();
  if (rank == 0 && tid == 0) a.lens_out[r] = m;

  // ---- move
  constexpr int kPiece = D / 8;                  // lanes of one key (or value) row
  constexpr int kPer = 32 / (2 * kPiece);        // tokens of one step
  constexpr int kGroup = kSteps * kPer;
  const int32_t* table = a.c.table + r * a.c.max_pages;
  const bool is_v = (lane / kPiece) & 1;
  const int sub = lane / (2 * kPiece);
  const int64_t stride = is_v ? a.c.v_page_stride : a.c.k_page_stride;
  __nv_bfloat16* pool =
      static_cast<__nv_bfloat16*>(is_v ? a.c.v_pages : a.c.k_pages) + (lane % kPiece) * 8;
  for (int32_t g = (rank * kWarps + warp) * kGroup; g < pairs; g += ranks * kWarps * kGroup) {
    // lane i < kGroup: pair g + i
    int32_t sp = -1, tp = -1, so = 0, to = 0;
    if (lane < kGroup && g + lane < pairs) {
      const int32_t s = src_list[g + lane], x = dst_list[g + lane];
      sp = table[s / a.c.page];
      tp = table[x / a.c.page];
      so = s % a.c.page;
      to = x % a.c.page;
      wo[x] = w[s];
      if (po) po[x] = pos[s];
      if (sp < 0 || sp >= a.c.num_pages || tp < 0 || tp >= a.c.num_pages) {
        atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
        sp = -1;
      }
    }
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
}

template <int D>
cudaError_t launch(const EvictArgs& a, int sms, cudaStream_t st) {
  const int64_t cap = int64_t(a.c.page) * a.c.max_pages;
  const int64_t rows = int64_t(a.c.batch) * a.c.num_kv_heads;
  // the least CTAs a row that hold its keys, then more while processors are
  // left and a slice is worth a CTA's while
  int ranks = 1;
  while (ranks < 8 && ((cap + ranks - 1) / ranks > kMaxSlice ||
                       (rows * ranks < 2 * sms && cap / ranks > 1024)))
    ranks *= 2;
  const int64_t slice = ((cap + ranks - 1) / ranks + 31) & ~int64_t(31);
  if (rows * ranks > INT32_MAX) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = sa_paged::allow_shared(evict_kernel<D>, kMaxSlice * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(slice) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(ranks);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<D>, a);
}

}  // namespace

namespace sa_paged {

// Two lists of at most cap / 2 slots a row.
size_t evict_workspace(const sa_paged_cache& c) {
  return size_t(c.batch) * c.num_kv_heads * c.page * c.max_pages * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t st) {
  return a.c.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace sa_paged
