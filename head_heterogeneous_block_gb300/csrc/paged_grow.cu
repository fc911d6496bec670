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
// A CTA does the sums over sequences and rows and then looks each (head, token)
// pair's page up.  For few pairs there is one CTA: a decode step is one launch,
// and its chain of loads (counts and lengths; pages; slots) and barriers bounds
// it.  For many, every CTA does the same sums for itself, which costs no time that
// one would not take, and a part of the pairs; the first one also has the new
// state, which a second, small launch puts in place where it replaces what other
// CTAs still read.  Rows and sequences beyond shared memory: one CTA leaves its
// sums in the workspace, a second launch does the pairs.  Pages are read from rows
// that give back, or below the old count of free ones, and written to rows that
// want some, or above that count.
//
// Measured (GB300, in a replayed graph): a decode step of 64 sequences, 8 heads:
// 4.1 us; 16 prompts of 62K tokens in all, 8 heads: 5.9 us, 7.3 in place; 32
// sequences, 4 heads, a quarter of them ended, chunks of up to 2048 tokens: 7.3 us,
// 8.7 in place (first one CTA's sums, then the pairs in a launch of their own: 8.7
// and 9.4 us either way).  The bytes would take 0.1, 0.7 and 0.2 us; a launch with
// one dependent load takes 2, the sums 2, a look-up and its slots 1.5.  Rows beyond
// shared memory: a decode step of 600 sequences, 8 heads: 16.5 us; of 2000: 48 (one
// CTA's sums over its rows, 512 at a time); 300 sequences of 500 tokens, 16 heads:
// 25.

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace {

using sa_paged::GrowArgs;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps <= 32, "one warp scans the warps' sums");
constexpr int kInlinePairs = 4096;    // (head, token) pairs that the first CTA does itself
constexpr int kRecords = 2048;        // rows whose records then stay in shared memory
constexpr int kSeqRecords = kThreads; // a thread's sequence each
constexpr int kSpread = 256;          // tokens of a CTA, threads of a block of the second launch
constexpr int kSpreadHeads = 4;       // heads of a thread's token that it looks up together
constexpr int kSpreadRows = 1024;     // rows and sequences whose records its blocks keep
constexpr int kSpreadSeqs = 512;

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

// Sequence of row r: r / Hkv, by its reciprocal where that is exact.
__device__ __forceinline__ int32_t seq_of_row(const GrowArgs& a, int32_t r) {
  return a.inv_heads ? int32_t(__umulhi(uint32_t(r), a.inv_heads)) : r / a.Hkv;
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
  const int32_t need = (r.x + w.seq[seq_of_row(a, lo)].y + a.page - 1) >> a.page_shift;
  return a.table[int64_t(lo) * a.max_pages + need + (x - r.w)];
}

// The sequence whose span token t is in, or the last one before it.
__device__ __forceinline__ int32_t seq_of(const GrowArgs& a, const Tables& w, int32_t t) {
  if (!a.cu) return a.span == 1 ? t : t / max(a.span, 1);
  int32_t lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (w.seq[mid].x <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// A token's place in a row: looked up first, then written, so that a thread's
// look-ups are under way together.
struct Place {
  int64_t row = 0;
  int32_t at = 0, page = 0, position = 0;
  bool live = false, fresh = false;   // gets a slot; from a page that is new to the row
};

// Token t of sequence b for KV head g.  next: what pages the rows' next slots are
// in, and top: the last of the free pages, the very last first (as far as these
// are at hand: NULL and 0 where not).
__device__ __forceinline__ Place look_up(const GrowArgs& a, const Tables& w, const Head& h,
                                         int32_t g, int32_t t, int32_t b, const int32_t* next,
                                         const int32_t* top, int32_t tops) {
  Place p;
  const int4 s = w.seq[b];
  const int32_t i = t - s.x;
  p.live = i >= 0 && i < s.z;
  if (!p.live) return p;
  const int32_t r = b * a.Hkv + g;
  const int4 row = w.row[r];
  p.row = r;
  p.at = row.x + i;
  p.position = s.w + i;
  const int32_t e = p.at >> a.page_shift;
  if (e < row.y) {
    p.page = next && e == row.x >> a.page_shift ? next[r] : a.table[p.row * a.max_pages + e];
  } else {
    p.fresh = true;
    const int32_t nth = row.z + e - row.y;         // from the stack's top
    p.page = nth >= h.back && nth - h.back < tops
                 ? top[nth - h.back]
                 : page_at(a, w, h.free, h.free + h.back - 1 - nth);
  }
  return p;
}

// Writes the slot (and what goes with it) of token t for KV head g.
__device__ __forceinline__ void put(const GrowArgs& a, const Place& p, int32_t g, int32_t t,
                                    bool* bad) {
  int64_t slot = -1;
  if (p.live) {
    const int32_t in_page = p.at & (a.page - 1);
    // (what a row holds ends within its own pages, so a new page starts with a
    // new token)
    if (p.fresh && in_page == 0) a.table[p.row * a.max_pages + (p.at >> a.page_shift)] = p.page;
    if (p.page >= 0 && p.page < a.num_pages)
      slot = (int64_t(p.page) << a.page_shift) + in_page;
    else
      *bad = true;
    const int64_t cell = p.row * (int64_t(a.max_pages) << a.page_shift) + p.at;
    if (a.weights) a.weights[cell] = 0.f;
    if (a.slot_positions) a.slot_positions[cell] = p.position;
  }
  a.slots[int64_t(g) * a.tokens + t] = slot;
  if (g == 0 && a.positions) a.positions[t] = p.live ? p.position : 0;
}

// Token t's slots for heads g0 .. g1.
__device__ __forceinline__ void place_heads(const GrowArgs& a, const Tables& w, const Head& h,
                                            int32_t t, int32_t g0, int32_t g1, bool* bad) {
  const int32_t b = seq_of(a, w, t);
  for (int32_t g = g0; g < g1; g += kSpreadHeads) {
    Place p[kSpreadHeads];
#pragma unroll
    for (int i = 0; i < kSpreadHeads; ++i)
      if (g + i < g1) p[i] = look_up(a, w, h, g + i, t, b, nullptr, nullptr, 0);
#pragma unroll
    for (int i = 0; i < kSpreadHeads; ++i)
      if (g + i < g1) put(a, p[i], g + i, t, bad);
  }
}

// Pages given back that nobody took become free: row r's part of them.
__device__ __forceinline__ void put_back(const GrowArgs& a, const Tables& w, const Head& h,
                                         int32_t r, int lane) {
  const int4 row = w.row[r];
  const int32_t need = (row.x + w.seq[seq_of_row(a, r)].y + a.page - 1) >> a.page_shift;
  for (int32_t k = lane; k < row.y - need && row.w + k < h.back - h.taken &&
                         h.free + row.w + k < a.num_pages; k += 32)
    a.free_pages[h.free + row.w + k] = a.table[int64_t(r) * a.max_pages + need + k];
}

// kInline: one CTA does it all.  kMany: each does the sums and a part of the pairs;
// the new state goes to the workspace if `late`.  kFirst: the first of two launches.
enum { kInline = 0, kMany = 1, kFirst = 2 };

template <int kMode>
__global__ void __launch_bounds__(kThreads)
    grow_kernel(const __grid_constant__ GrowArgs a, Tables ws, int32_t late) {
  constexpr bool near = kMode != kFirst;   // all sequences and rows in shared memory
  constexpr bool inl = kMode == kInline;
  __shared__ int4 seq_s[near ? kSeqRecords : 1], row_s[near ? kRecords : 1];
  __shared__ int32_t sum_w[kWarps], sum_b[kWarps], most_s[near ? kSeqRecords : 1];
  __shared__ int32_t top_s[inl ? kThreads : 1], next_s[inl ? kRecords : 1];
  __shared__ int32_t taken_s;
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t rows = a.batch * a.Hkv, cap = a.max_pages << a.page_shift;
  Tables w = ws;
  if (near) {
    w.seq = seq_s;
    w.row = row_s;
  }
  bool bad = false, bad_cu = false;

  // What row r holds and owns, emptied where its sequence ended.
  auto clean_row = [&](int32_t n, int32_t o, bool ended) -> int4 {
    if (o < 0 || o > a.max_pages) {
      bad = true;
      o = clamp_to(o, 0, a.max_pages);
    }
    const int32_t most = o << a.page_shift;
    if (n < 0 || n > most) {
      bad = true;
      n = clamp_to(n, 0, most);
    }
    return make_int4(ended ? 0 : n, o, 0, 0);
  };
  auto ended = [&](int32_t b) { return a.ended && a.ended[b]; };

  // Every load that depends on nothing first (then the rows' lengths are read).
  int32_t free = *a.free_count;
  if (tid == 0) taken_s = 0;
  // (near: a thread has one sequence)
  int32_t c0 = 0, c1 = 0, cnt = 0, start = 0;
  bool end = false;
  if (near && tid < a.batch) {
    if (a.cu) {
      c0 = a.cu[tid];
      c1 = a.cu[tid + 1];
    }
    if (a.counts) cnt = a.counts[tid];
    if (a.start) start = a.start[tid];
    end = ended(tid);
    most_s[tid] = 0;
  }
  for (int32_t r = tid; r < rows; r += kThreads)
    w.row[r] = clean_row(a.lens[r], a.owned[r], ended(seq_of_row(a, r)));
  if (free < 0 || free > a.num_pages) {
    bad = true;
    free = clamp_to(free, 0, int32_t(a.num_pages));
  }
  // the pages that rows go on with, and those that the stack hands out first
  // unless others were given back: on their way until the slots need them
  constexpr int kMine = inl ? kRecords / kThreads : 1;
  const int32_t tops = min(free, kThreads);
  int32_t top = 0, next[kMine];
  if (inl) {
    if (tid < tops) top = a.free_pages[free - 1 - tid];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int32_t r = tid + i * kThreads;
      next[i] = 0;
      if (r < rows) {
        const int32_t e = w.row[r].x >> a.page_shift;
        if (e < w.row[r].y) next[i] = a.table[int64_t(r) * a.max_pages + e];
      }
    }
  }
  // spans that overlap would leave new pages unnamed: nobody gets any then
  if (near) {
    bad_cu = a.cu && tid < a.batch && (c0 < 0 || c1 < c0 || c1 > a.tokens);
  } else if (a.cu) {
    for (int32_t b = tid; b < a.batch; b += kThreads)
      bad_cu |= a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.tokens;
  }
  bad_cu = __syncthreads_or(bad_cu);
  bad |= bad_cu;
  // the longest row of each sequence
  if (near) {
    for (int32_t r = tid; r < rows; r += kThreads) atomicMax(&most_s[seq_of_row(a, r)], w.row[r].x);
    __syncthreads();
  }
  // sequences: their tokens' span and what they ask for
  for (int32_t b = tid; b < a.batch; b += kThreads) {
    int32_t first = b * a.span, span = a.span, most = 0;
    if (near) {
      most = most_s[b];
    } else {
      if (a.cu) {
        c0 = a.cu[b];
        c1 = a.cu[b + 1];
      }
      if (a.counts) cnt = a.counts[b];
      if (a.start) start = a.start[b];
      end = ended(b);
      for (int32_t g = 0; g < a.Hkv; ++g) most = max(most, w.row[b * a.Hkv + g].x);
    }
    if (a.cu) {
      first = bad_cu ? 0 : c0;
      span = bad_cu ? 0 : c1 - c0;
    }
    int32_t c = span;
    if (a.counts) {
      c = cnt;
      if (c < 0 || c > span) {
        bad = true;
        c = clamp_to(c, 0, span);
      }
    }
    if (c > cap - most) {              // more than the row's table holds: none
      bad = true;
      c = 0;
    }
    w.seq[b] = make_int4(first, c, 0, a.start ? (end ? 0 : start) : most);
  }
  __syncthreads();

  // rows: prefix sums of the pages wanted and given back
  int32_t carry_w = 0, carry_b = 0;
  for (int32_t base = 0; base < rows; base += kThreads) {
    const int32_t r = base + tid;
    int32_t held = 0, owned = 0, want = 0, back = 0;
    if (r < rows) {
      held = w.row[r].x;
      owned = w.row[r].y;
      const int32_t need = (held + w.seq[seq_of_row(a, r)].y + a.page - 1) >> a.page_shift;
      want = max(0, need - owned);
      back = max(0, owned - need);
    }
    const int32_t iw = scan_warp(want, lane), ib = scan_warp(back, lane);
    if (lane == 31) {
      sum_w[warp] = iw;
      sum_b[warp] = ib;
    }
    __syncthreads();
    const int32_t tw = scan_warp(lane < kWarps ? sum_w[lane] : 0, lane);
    const int32_t tb = scan_warp(lane < kWarps ? sum_b[lane] : 0, lane);
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
    if (kMode == kMany && (late || blockIdx.x > 0)) {
      if (late && blockIdx.x == 0) ws.seq[b] = make_int4(s.z, s.w + s.z, 0, 0);
      continue;
    }
    if (a.granted) a.granted[b] = s.z;
    if (a.start_out) a.start_out[b] = s.w + s.z;
  }
  if (inl) {
    top_s[tid] = top;
#pragma unroll
    for (int i = 0; i < kMine; ++i) next_s[tid + i * kThreads] = next[i];
  }
  __syncthreads();
  const Head h{free, carry_b, taken_s};
  if (kMode != kMany || blockIdx.x == 0) {
    for (int32_t r = tid; r < rows; r += kThreads) {
      const int4 row = w.row[r], s = w.seq[seq_of_row(a, r)];
      const int32_t need = (row.x + s.y + a.page - 1) >> a.page_shift;
      // without a grant a row keeps what it has of the pages that it asked for
      const int32_t len = row.x + s.z, owned = s.z == s.y ? need : min(row.y, need);
      if (kMode == kMany && late) {
        ws.row[r] = make_int4(len, owned, 0, 0);
      } else {
        a.lens_out[r] = len;
        a.owned_out[r] = owned;
      }
    }
    if (tid == 0) {
      const int32_t left = min(h.free + h.back - h.taken, int32_t(a.num_pages));
      if (kMode == kMany && late)
        ws.head->free = left;
      else
        *a.free_count_out = left;
      if (kMode == kFirst) *ws.head = h;
    }
  }
  bool bad_page = false;
  if (inl) {
    // 32 tokens of a head a warp at a time
    const int32_t chunks = (a.tokens + 31) / 32;
    for (int32_t u = warp; u < a.Hkv * chunks; u += kWarps) {
      const int32_t g = u / chunks, t = (u - g * chunks) * 32 + lane;
      if (t < a.tokens)
        put(a, look_up(a, w, h, g, t, seq_of(a, w, t), next_s, top_s, tops), g, t, &bad_page);
    }
  }
  if (kMode == kMany) {
    // 256 tokens at a time, two halves of the heads
    constexpr int kParts = kThreads / kSpread;
    for (int32_t t = int32_t(blockIdx.x) * kSpread + tid % kSpread; t < a.tokens;
         t += int32_t(gridDim.x) * kSpread)
      place_heads(a, w, h, t, a.Hkv * (tid / kSpread) / kParts,
                  a.Hkv * (tid / kSpread + 1) / kParts, &bad_page);
  }
  if (kMode != kFirst && h.back > h.taken)
    for (int32_t r = int32_t(blockIdx.x) * kWarps + warp; r < rows;
         r += int32_t(gridDim.x) * kWarps)
      put_back(a, w, h, r, lane);
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_COUNT);
  if (bad_page) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
}

__global__ void __launch_bounds__(kSpread)
    spread_kernel(const __grid_constant__ GrowArgs a, Tables w) {
  __shared__ int4 seq_s[kSpreadSeqs], row_s[kSpreadRows];
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int32_t rows = a.batch * a.Hkv;
  const Head h = *w.head;
  if (a.batch <= kSpreadSeqs && rows <= kSpreadRows) {
    for (int32_t b = threadIdx.x; b < a.batch; b += kSpread) seq_s[b] = w.seq[b];
    for (int32_t r = threadIdx.x; r < rows; r += kSpread) row_s[r] = w.row[r];
    w.seq = seq_s;
    w.row = row_s;
    __syncthreads();
  }
  bool bad = false;
  const int32_t t = int32_t(blockIdx.x) * kSpread + int32_t(threadIdx.x);
  if (t < a.tokens)                    // a block's heads: an equal part of all
    place_heads(a, w, h, t, int32_t(int64_t(a.Hkv) * blockIdx.y / gridDim.y),
                int32_t(int64_t(a.Hkv) * (blockIdx.y + 1) / gridDim.y), &bad);
  if (h.back > h.taken) {
    const int64_t warps = int64_t(gridDim.x) * gridDim.y * (kSpread / 32);
    int64_t r = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kSpread / 32) + (threadIdx.x >> 5);
    for (; r < rows; r += warps) put_back(a, w, h, int32_t(r), threadIdx.x & 31);
  }
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
}

// The new state that the first CTA left, put in place.
__global__ void __launch_bounds__(kSpread)
    settle_kernel(const __grid_constant__ GrowArgs a, Tables w) {
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int32_t x = int32_t(blockIdx.x) * kSpread + int32_t(threadIdx.x);
  if (x < a.batch * a.Hkv) {
    const int4 r = w.row[x];
    a.lens_out[x] = r.x;
    a.owned_out[x] = r.y;
  }
  if (x < a.batch) {
    const int4 s = w.seq[x];
    if (a.granted) a.granted[x] = s.x;
    if (a.start_out) a.start_out[x] = s.y;
  }
  if (x == 0) *a.free_count_out = w.head->free;
}

// Whether the new state shares memory with what the other CTAs still read.
bool replaces(const GrowArgs& a) {
  const size_t seqs = size_t(a.batch) * 4, rows = seqs * a.Hkv;
  const struct {
    const void* p;
    size_t n;
  } out[] = {{a.lens_out, rows}, {a.owned_out, rows}, {a.free_count_out, 4}, {a.start_out, seqs},
             {a.granted, seqs}},
    in[] = {{a.lens, rows}, {a.owned, rows}, {a.free_count, 4}, {a.cu, seqs + 4},
            {a.counts, seqs}, {a.ended, size_t(a.batch)}, {a.start, seqs}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (sa_paged::overlap(o.p, o.n, i.p, i.n)) return true;
  return false;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

namespace sa_paged {

size_t grow_workspace(int32_t batch, int32_t num_kv_heads) {
  return 256 + up(size_t(batch) * 16) + size_t(batch) * num_kv_heads * 16;
}

cudaError_t launch_grow(const GrowArgs& a, int sms, cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  Tables w{reinterpret_cast<Head*>(ws), reinterpret_cast<int4*>(ws + 256),
           reinterpret_cast<int4*>(ws + 256 + up(size_t(a.batch) * 16))};
  const int64_t rows = int64_t(a.batch) * a.Hkv;
  const bool near = rows <= kRecords && a.batch <= kSeqRecords;
  const bool inl = near && int64_t(a.tokens) * a.Hkv <= kInlinePairs;
  const int64_t blocks = std::max<int64_t>(1, (int64_t(a.tokens) + kSpread - 1) / kSpread);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (inl) return cudaLaunchKernelEx(&cfg, grow_kernel<kInline>, a, w, 0);
  if (near) {
    const bool late = replaces(a);
    // (three CTAs fit on a processor)
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(blocks, 3 * sms)));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, grow_kernel<kMany>, a, w, int32_t(late));
    if (e != cudaSuccess || !late) return e;
    cfg.gridDim = dim3(unsigned((rows + kSpread - 1) / kSpread));
    cfg.blockDim = dim3(kSpread);
    return cudaLaunchKernelEx(&cfg, settle_kernel, a, w);
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grow_kernel<kFirst>, a, w, 0);
  if (e != cudaSuccess) return e;
  // blocks of 256 tokens; their heads are split where there are few of them
  const int64_t parts = (a.Hkv + kSpreadHeads - 1) / kSpreadHeads;
  cfg.gridDim = dim3(unsigned(blocks),
                     unsigned(std::min<int64_t>({parts, std::max<int64_t>(1, 1024 / blocks), 256})));
  cfg.blockDim = dim3(kSpread);
  return cudaLaunchKernelEx(&cfg, spread_kernel, a, w);
}

}  // namespace sa_paged
