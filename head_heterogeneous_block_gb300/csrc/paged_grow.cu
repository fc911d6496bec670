// Pages and slots of new tokens of a paged key-value cache, from their numbers.
//
// Row r = b*Hkv + g holds n tokens in o pages and gets c_b more: it needs
// ceil((n + c_b) / page) pages, gives back what it owns beyond that and wants
// what is missing.  The free pages and, above them, those given back (rows and
// entries in order) are a stack from whose top the wanted ones are taken, again
// in order, so that the i-th is stack[F + R - 1 - i]: every page follows from two
// prefix sums over the rows, one of the given back, one of the wanted, and no
// page waits for another.  A sequence whose pages would pass the stack's end
// gets none, nor does any later one that wants some.
//
// One CTA does the sums over sequences and rows and leaves a 16-byte record a
// row; then each (head, token) pair looks its page up by itself.  For few pairs
// that is the same CTA, with the records in shared memory: a decode step is one
// launch, and the chain of loads (counts and lengths; pages; slots) bounds it.
// For many it is a second launch over all processors, bound by the 8-byte slots
// that it writes.  Nothing that is read there is written there: pages are taken
// from rows that give back, or below the old count of free ones, and put into
// rows that want some, or above that count.

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace {

using sa_paged::GrowArgs;

constexpr int kThreads = 1024;
constexpr int kInlinePairs = 8192;    // (head, token) pairs that the first CTA does itself
constexpr int kRecords = 2048;        // rows whose records then stay in shared memory
constexpr int kSeqRecords = 1024;
constexpr int kSpread = 256;          // threads of a block of the second launch

struct Head {
  int32_t free, back, taken;          // F, R, G
};
struct Tables {
  Head* head;
  int4* seq;              // [batch] first token of its span, tokens asked for, granted, start
  int4* row;              // [rows] tokens held, pages owned, pages wanted and given back before
};

__device__ __forceinline__ int32_t clamp_to(int32_t x, int32_t lo, int32_t hi) {
  return min(max(x, lo), hi);
}

__device__ __forceinline__ int32_t scan_warp(int32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Page number at place v of the stack.
__device__ __forceinline__ int32_t page_at(const GrowArgs& a, const Tables& w, int32_t free,
                                           int32_t v) {
  if (v < free) return a.free_pages[v];
  // the last row with at most x pages given back before it
  const int32_t x = v - free;
  int32_t lo = 0, hi = a.batch * a.Hkv;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (w.row[mid].w <= x) lo = mid; else hi = mid;
  }
  const int4 r = w.row[lo];
  const int32_t need = (r.x + w.seq[lo / a.Hkv].y + a.page - 1) >> a.page_shift;
  return a.table[int64_t(lo) * a.max_pages + need + (x - r.w)];
}

// Slot (and what goes with it) of token t for KV head g.
__device__ __forceinline__ void place(const GrowArgs& a, const Tables& w, const Head& h, int32_t g,
                                      int32_t t, bool* bad) {
  int32_t b;
  if (a.cu) {
    int32_t lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (w.seq[mid].x <= t) lo = mid; else hi = mid;
    }
    b = lo;
  } else {
    b = t / a.span;
  }
  const int4 s = w.seq[b];
  const int32_t i = t - s.x;
  int64_t slot = -1;
  if (i >= 0 && i < s.z) {
    const int64_t r = int64_t(b) * a.Hkv + g;
    const int4 row = w.row[r];
    const int32_t at = row.x + i, e = at >> a.page_shift;
    int32_t page;
    if (e < row.y) {
      page = a.table[r * a.max_pages + e];
    } else {
      page = page_at(a, w, h.free, h.free + h.back - 1 - (row.z + e - row.y));
      // (what a row holds ends within its own pages, so a new page starts with a
      // new token)
      if ((at & (a.page - 1)) == 0) a.table[r * a.max_pages + e] = page;
    }
    if (page >= 0 && page < a.num_pages)
      slot = (int64_t(page) << a.page_shift) + (at & (a.page - 1));
    else
      *bad = true;
    const int64_t cell = r * (int64_t(a.max_pages) << a.page_shift) + at;
    if (a.weights) a.weights[cell] = 0.f;
    if (a.slot_positions) a.slot_positions[cell] = s.w + i;
  }
  a.slots[int64_t(g) * a.tokens + t] = slot;
  if (g == 0 && a.positions) a.positions[t] = i >= 0 && i < s.z ? s.w + i : 0;
}

// Pages given back that nobody took become free: row r's part of them.
__device__ __forceinline__ void put_back(const GrowArgs& a, const Tables& w, const Head& h,
                                         int32_t r, int lane) {
  const int4 row = w.row[r];
  const int32_t need = (row.x + w.seq[r / a.Hkv].y + a.page - 1) >> a.page_shift;
  for (int32_t k = lane; k < row.y - need && row.w + k < h.back - h.taken &&
                         h.free + row.w + k < a.num_pages; k += 32)
    a.free_pages[h.free + row.w + k] = a.table[int64_t(r) * a.max_pages + need + k];
}

__global__ void __launch_bounds__(kThreads)
    grow_kernel(const __grid_constant__ GrowArgs a, Tables ws, int32_t inl) {
  __shared__ int4 seq_s[kSeqRecords], row_s[kRecords];
  __shared__ int32_t sum_w[32], sum_b[32];
  __shared__ int32_t taken_s;
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t rows = a.batch * a.Hkv, cap = a.max_pages << a.page_shift;
  Tables w = ws;
  if (inl) {
    w.seq = seq_s;
    w.row = row_s;
  }
  bool bad = false;
  if (tid == 0) taken_s = 0;
  int32_t free = *a.free_count;
  if (free < 0 || free > a.num_pages) {
    bad = true;
    free = clamp_to(free, 0, int32_t(a.num_pages));
  }

  // what row r holds and owns
  auto row_state = [&](int32_t r, bool ended, int32_t* held, int32_t* owned) {
    int32_t n = a.lens[r], o = a.owned[r];
    if (o < 0 || o > a.max_pages) {
      bad = true;
      o = clamp_to(o, 0, a.max_pages);
    }
    const int32_t most = o << a.page_shift;
    if (n < 0 || n > most) {
      bad = true;
      n = clamp_to(n, 0, most);
    }
    *held = ended ? 0 : n;
    *owned = o;
  };

  // spans that overlap would leave new pages unnamed: nobody gets any then
  bool bad_cu = false;
  if (a.cu)
    for (int32_t b = tid; b <= a.batch; b += kThreads) {
      const int32_t c = a.cu[b];
      bad_cu |= c < 0 || c > a.tokens || (b > 0 && c < a.cu[b - 1]);
    }
  bad_cu = __syncthreads_or(bad_cu);
  bad |= bad_cu;

  // sequences: their tokens' span and what they ask for
  for (int32_t b = tid; b < a.batch; b += kThreads) {
    int32_t first, span;
    if (a.cu) {
      first = bad_cu ? 0 : a.cu[b];
      span = bad_cu ? 0 : a.cu[b + 1] - first;
    } else {
      first = b * a.span;
      span = a.span;
    }
    int32_t c = span;
    if (a.counts) {
      c = a.counts[b];
      if (c < 0 || c > span) {
        bad = true;
        c = clamp_to(c, 0, span);
      }
    }
    const bool ended = a.ended && a.ended[b];
    int32_t most = 0;
    for (int32_t g = 0; g < a.Hkv; ++g) {
      int32_t held, owned;
      row_state(b * a.Hkv + g, ended, &held, &owned);
      most = max(most, held);
    }
    if (c > cap - most) {              // more than the row's table holds: none
      bad = true;
      c = 0;
    }
    const int32_t start = a.start ? (ended ? 0 : a.start[b]) : most;
    w.seq[b] = make_int4(first, c, 0, start);
  }
  __syncthreads();

  // rows: prefix sums of the pages wanted and given back
  int32_t carry_w = 0, carry_b = 0;
  for (int32_t base = 0; base < rows; base += kThreads) {
    const int32_t r = base + tid;
    int32_t held = 0, owned = 0, want = 0, back = 0;
    if (r < rows) {
      const int32_t b = r / a.Hkv;
      row_state(r, a.ended && a.ended[b], &held, &owned);
      const int32_t need = (held + w.seq[b].y + a.page - 1) >> a.page_shift;
      want = max(0, need - owned);
      back = max(0, owned - need);
    }
    const int32_t iw = scan_warp(want, lane), ib = scan_warp(back, lane);
    if (lane == 31) {
      sum_w[warp] = iw;
      sum_b[warp] = ib;
    }
    __syncthreads();
    const int32_t tw = scan_warp(sum_w[lane], lane), tb = scan_warp(sum_b[lane], lane);
    const int32_t before_w = __shfl_sync(0xffffffffu, tw, warp ? warp - 1 : 0);
    const int32_t before_b = __shfl_sync(0xffffffffu, tb, warp ? warp - 1 : 0);
    if (r < rows)
      w.row[r] = make_int4(held, owned, carry_w + (warp ? before_w : 0) + iw - want,
                           carry_b + (warp ? before_b : 0) + ib - back);
    carry_w += __shfl_sync(0xffffffffu, tw, 31);
    carry_b += __shfl_sync(0xffffffffu, tb, 31);
    __syncthreads();
  }
  const int32_t total = free + carry_b;        // both below 2^30 + 1 and 2^30
  bad |= total > a.num_pages;                  // pages that belong to two

  // which sequences get theirs, and the new state
  for (int32_t b = tid; b < a.batch; b += kThreads) {
    const int32_t from = w.row[b * a.Hkv].z;
    const int32_t to = b + 1 < a.batch ? w.row[(b + 1) * a.Hkv].z : carry_w;
    int4 s = w.seq[b];
    const bool ok = to == from || to <= total;
    if (!ok) atomicOr(a.dev_status, SA_DEV_NO_PAGES);
    s.z = ok ? s.y : 0;
    if (ok && to != from) atomicMax(&taken_s, to);
    w.seq[b] = s;
    if (a.granted) a.granted[b] = s.z;
    if (a.start_out) a.start_out[b] = s.w + s.z;
  }
  __syncthreads();
  for (int32_t r = tid; r < rows; r += kThreads) {
    const int4 row = w.row[r], s = w.seq[r / a.Hkv];
    a.lens_out[r] = row.x + s.z;
    const int32_t need = (row.x + s.y + a.page - 1) >> a.page_shift;
    // without a grant a row keeps what it has of the pages that it asked for
    a.owned_out[r] = s.z == s.y ? need : min(row.y, need);
  }
  const Head h{free, carry_b, taken_s};
  if (tid == 0) {
    *a.free_count_out = min(h.free + h.back - h.taken, int32_t(a.num_pages));
    if (!inl) *ws.head = h;
  }
  bool bad_page = false;
  if (inl) {
    for (int32_t x = tid; x < a.tokens * a.Hkv; x += kThreads) {
      const int32_t g = x / a.tokens;
      place(a, w, h, g, x - g * a.tokens, &bad_page);
    }
    if (h.back > h.taken)
      for (int32_t r = warp; r < rows; r += kThreads / 32) put_back(a, w, h, r, lane);
  }
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_COUNT);
  if (bad_page) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
}

__global__ void __launch_bounds__(kSpread)
    spread_kernel(const __grid_constant__ GrowArgs a, Tables w) {
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const Head h = *w.head;
  bool bad = false;
  const int32_t t = int32_t(blockIdx.x) * kSpread + int32_t(threadIdx.x);
  if (t < a.tokens)
    for (int32_t g = blockIdx.y; g < a.Hkv; g += gridDim.y) place(a, w, h, g, t, &bad);
  if (h.back > h.taken) {
    const int64_t warps = int64_t(gridDim.x) * gridDim.y * (kSpread / 32);
    int64_t r = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kSpread / 32) + (threadIdx.x >> 5);
    for (; r < int64_t(a.batch) * a.Hkv; r += warps)
      put_back(a, w, h, int32_t(r), threadIdx.x & 31);
  }
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

namespace sa_paged {

size_t grow_workspace(int32_t batch, int32_t num_kv_heads) {
  return 256 + up(size_t(batch) * 16) + size_t(batch) * num_kv_heads * 16;
}

cudaError_t launch_grow(const GrowArgs& a, cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  Tables w{reinterpret_cast<Head*>(ws), reinterpret_cast<int4*>(ws + 256),
           reinterpret_cast<int4*>(ws + 256 + up(size_t(a.batch) * 16))};
  const int64_t rows = int64_t(a.batch) * a.Hkv;
  const bool inl = int64_t(a.tokens) * a.Hkv <= kInlinePairs && rows <= kRecords &&
                   a.batch <= kSeqRecords;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, grow_kernel, a, w, int32_t(inl));
  if (e != cudaSuccess || inl) return e;
  cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, (int64_t(a.tokens) + kSpread - 1) / kSpread)),
                     unsigned(std::min(a.Hkv, 256)));
  cfg.blockDim = dim3(kSpread);
  return cudaLaunchKernelEx(&cfg, spread_kernel, a, w);
}

}  // namespace sa_paged
