// Evicting tokens from a paged key-value cache by accumulated weight.
//
// One CTA per row.  A token's 32-bit key orders it: all ones for the first
// `sinks` and last `recent` positions, else the weight's bits mapped so that
// unsigned order is the floats' order (NaN below every number, -0 as +0).
// The m-th largest key T is built bit by bit; tokens above T are kept, and of
// those equal to T the lowest slots until m are kept.  Scans in slot order
// then number the evicted slots below m and the kept ones from m on: the i-th
// of these moves into the i-th of those.  Sources lie at m or above and
// destinations below, so no move reads what another writes.

#include <cuda_bf16.h>

#include "paged.h"

namespace {

using sa_paged::EvictArgs;

constexpr int kThreads = 512;
constexpr int kWarpsOf = kThreads / 32;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Shared {
  int32_t part[kWarpsOf];
  int32_t total;
};

__device__ int32_t block_sum(Shared& sh, int32_t v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  int32_t s = 0;
  for (int w = 0; w < kWarpsOf; ++w) s += sh.part[w];
  return s;
}

// Number of threads before this one whose flag is set; total: of all.
__device__ int32_t block_rank(Shared& sh, bool flag, int32_t& total) {
  const uint32_t b = __ballot_sync(0xffffffffu, flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) sh.part[warp] = __popc(b);
  __syncthreads();
  int32_t before = __popc(b & ((1u << lane) - 1u));
  total = 0;
  for (int w = 0; w < kWarpsOf; ++w) {
    if (w < warp) before += sh.part[w];
    total += sh.part[w];
  }
  return before;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t n = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int32_t m = min(n, a.keep[r % a.c.num_kv_heads]);
  const float* w = a.c.weights + r * cap;
  const int32_t* pos = a.c.positions ? a.c.positions + r * cap : nullptr;
  int32_t* dst_list = static_cast<int32_t*>(a.ws) + r * cap;
  int32_t* src_list = dst_list + cap / 2;

  int32_t newest = INT32_MIN;
  if (pos)
    for (int32_t t = tid; t < n; t += kThreads) newest = max(newest, pos[t]);
  else
    newest = n - 1;
  for (int o = 16; o; o >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, o));
  if (lane == 0) sh.part[warp] = newest;
  __syncthreads();
  for (int x = 0; x < kWarpsOf; ++x) newest = max(newest, sh.part[x]);
  auto key = [&](int32_t t) -> uint32_t {
    const int32_t p = pos ? pos[t] : t;
    if (p < a.sinks || int64_t(p) > int64_t(newest) - a.recent) return 0xFFFFFFFFu;
    return weight_key(w[t]);
  };

  int32_t pairs = 0;
  if (m > 0 && n > m) {
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = T | (1u << bit);
      int32_t c = 0;
      for (int32_t t = tid; t < n; t += kThreads) c += key(t) >= cand;
      if (block_sum(sh, c) >= m) T = cand;
    }
    int32_t above = 0;
    for (int32_t t = tid; t < n; t += kThreads) above += key(t) > T;
    const int32_t take = m - block_sum(sh, above);
    int32_t ties = 0, holes = 0;
    for (int32_t t0 = 0; t0 < n; t0 += kThreads) {
      const int32_t t = t0 + tid;
      const uint32_t k = t < n ? key(t) : 0u;
      int32_t total;
      const int32_t tie = ties + block_rank(sh, t < n && k == T, total);
      ties += total;
      const bool kept = t < n && (k > T || (k == T && tie < take));
      const bool hole = t < m && !kept, source = t >= m && kept;
      const int32_t hr = holes + block_rank(sh, hole, total);
      holes += total;
      const int32_t sr = pairs + block_rank(sh, source, total);
      pairs += total;
      if (hole) dst_list[hr] = t;
      if (source) src_list[sr] = t;
    }
  }
  // the new state's kept slots, then the moved tokens
  float* wo = a.weights_out + r * cap;
  int32_t* po = a.positions_out ? a.positions_out + r * cap : nullptr;
  for (int32_t t = tid; t < m; t += kThreads) {
    if (wo != w) wo[t] = w[t];
    if (po && po != pos) po[t] = pos[t];
  }
  __syncthreads();
  const int32_t* table = a.c.table + r * a.c.max_pages;
  for (int32_t i = warp; i < pairs; i += kWarpsOf) {
    const int32_t s = src_list[i], t = dst_list[i];
    const int32_t sp = table[s / a.c.page], tp = table[t / a.c.page];
    if (lane == 0) {
      wo[t] = w[s];
      if (po) po[t] = pos[s];
    }
    if (sp < 0 || sp >= a.c.num_pages || tp < 0 || tp >= a.c.num_pages) {
      if (lane == 0) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
      continue;
    }
    const int piece = a.c.head_dim / 8;
    if (lane < 2 * piece) {
      const bool is_v = lane >= piece;
      const int64_t stride = is_v ? a.c.v_page_stride : a.c.k_page_stride;
      __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(is_v ? a.c.v_pages : a.c.k_pages) +
                            (lane % piece) * 8;
      *reinterpret_cast<uint4*>(pool + tp * stride + int64_t(t % a.c.page) * a.c.head_dim) =
          *reinterpret_cast<const uint4*>(pool + sp * stride +
                                          int64_t(s % a.c.page) * a.c.head_dim);
    }
  }
  if (tid == 0) a.lens_out[r] = m;
}

}  // namespace

namespace sa_paged {

// Two lists of at most cap / 2 slots a row.
size_t evict_workspace(const sa_paged_cache& c) {
  return size_t(c.batch) * c.num_kv_heads * c.page * c.max_pages * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, int, cudaStream_t st) {
  evict_kernel<<<unsigned(a.c.batch * a.c.num_kv_heads), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa_paged
