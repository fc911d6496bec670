// C ABI entry points of the paged key-value cache and of the rotary positions:
// argument checks, then the launches of paged_*.cu and rotary.cu.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "paged.h"
#include "sparse_attn.h"
#include "wait_limit.h"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 38;   // elements; a TMA stride is below 2^40 bytes

bool page_stride_ok(int64_t s, const sa_paged_cache* c) {
  return s % 8 == 0 && s >= int64_t(c->page) * c->head_dim && s < kMaxStride;
}

sa_status check_cache(const sa_paged_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->table || !c->lens) return SA_ERR_INVALID_ARG;
  if (c->page <= 0 || c->max_pages <= 0 || c->batch <= 0 || c->num_kv_heads <= 0 ||
      c->head_dim <= 0 || c->num_pages <= 0 || c->num_pages > INT32_MAX)
    return SA_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return SA_ERR_UNSUPPORTED;
  if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return SA_ERR_UNSUPPORTED;
  if (!page_stride_ok(c->k_page_stride, c) || !page_stride_ok(c->v_page_stride, c))
    return SA_ERR_INVALID_ARG;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return SA_ERR_INVALID_ARG;
  if (!aligned(c->table, 4) || !aligned(c->lens, 4) || !aligned(c->weights, 4) ||
      !aligned(c->positions, 4))
    return SA_ERR_INVALID_ARG;
  // slots of a row, rows, and 16-slot pieces of all rows are 32-bit counts, with
  // room for sums
  const int64_t cap = int64_t(c->page) * c->max_pages;
  const int64_t rows = int64_t(c->batch) * c->num_kv_heads;
  if (cap > (int64_t(1) << 30) || rows > (int64_t(1) << 24) ||
      cap / 16 > (int64_t(1) << 30) / rows)
    return SA_ERR_SHAPE;
  return SA_OK;
}

sa_status check_heads(const sa_paged_cache* c, int32_t hq) {
  if (hq <= 0 || hq % c->num_kv_heads != 0 || hq / c->num_kv_heads > 1024) return SA_ERR_SHAPE;
  const int64_t rows = int64_t(c->batch) * c->num_kv_heads;
  const int64_t chunks = (hq / c->num_kv_heads + 31) / 32;
  const int64_t pieces = int64_t(c->page) * c->max_pages / 16;
  if (rows * chunks > (int64_t(1) << 24) || pieces > (int64_t(1) << 30) / (rows * chunks))
    return SA_ERR_SHAPE;
  return SA_OK;
}

// What eviction serves: budgets are a kernel parameter, a row's keys lie in a
// cluster's shared memory.
sa_status check_evict(const sa_paged_cache* c) {
  if (c->num_kv_heads > sa_paged::kMaxKvHeads ||
      int64_t(c->page) * c->max_pages > sa_paged::kMaxEvictSlots)
    return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

sa_status check_pool(const sa_page_pool* p) {
  if (!p || !p->table || !p->lens || !p->owned || !p->free_pages || !p->free_count)
    return SA_ERR_INVALID_ARG;
  if (p->page <= 0 || p->max_pages <= 0 || p->batch <= 0 || p->num_kv_heads <= 0 ||
      p->num_pages <= 0 || p->num_pages >= (int64_t(1) << 30))
    return SA_ERR_SHAPE;
  if (p->page < 16 || p->page > 256 || (p->page & (p->page - 1))) return SA_ERR_UNSUPPORTED;
  if (!aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->owned, 4) ||
      !aligned(p->free_pages, 4) || !aligned(p->free_count, 4) || !aligned(p->weights, 4) ||
      !aligned(p->positions, 4))
    return SA_ERR_INVALID_ARG;
  // slots of a row, and the pages of all rows, are 32-bit counts with room for sums
  const int64_t rows = int64_t(p->batch) * p->num_kv_heads;
  if (rows > (1 << 20) || int64_t(p->page) * p->max_pages > (int64_t(1) << 30) ||
      p->max_pages > (int64_t(1) << 30) / rows)
    return SA_ERR_SHAPE;
  return SA_OK;
}

// Whether two rows of d elements of a [tokens][heads] output share memory (strides at
// least d where they are used).
bool rows_share(int64_t tokens, int64_t heads, int64_t d, const int64_t* s) {
  using Wide = __int128;
  if (tokens <= 1 || heads <= 1 || s[0] >= Wide(heads - 1) * s[1] + d ||
      s[1] >= Wide(tokens - 1) * s[0] + d)
    return false;
  // tokens lie between heads: h heads further is nearly t or t + 1 tokens further
  for (int64_t h = 1; h < heads; ++h) {
    const int64_t t = h * s[1] / s[0], over = h * s[1] - t * s[0];
    if ((t < tokens && over < d) || (t + 1 < tokens && s[0] - over < d)) return true;
  }
  return false;
}

// Checks and arguments of the two rotary calls, but for the store's.
sa_status rotary_args(const sa_rotary* rot, int32_t tokens, int32_t hq, int32_t hkv,
                      const int32_t* positions, const void* q, const int64_t* qs, const void* k,
                      const int64_t* ks, void* q_out, const int64_t* qos, void* k_out,
                      const int64_t* kos, bool store, sa_paged::RotaryArgs* a) {
  if (!rot) return SA_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > (1 << 30) || hq < 1 || hkv < 1 || hq > (1 << 20) || hkv > (1 << 20))
    return SA_ERR_SHAPE;
  if (rot->head_dim != 64 && rot->head_dim != 128) return SA_ERR_UNSUPPORTED;
  if (rot->rot_dim < 16 || rot->rot_dim > rot->head_dim || rot->rot_dim % 16)
    return SA_ERR_UNSUPPORTED;
  if (rot->interleaved != 0 && rot->interleaved != 1) return SA_ERR_INVALID_ARG;
  if (!std::isfinite(rot->factor)) return SA_ERR_INVALID_ARG;
  if (!rot->turns || !qs || !ks || !qos || (!store && !kos) || (k_out && !kos))
    return SA_ERR_INVALID_ARG;
  if (tokens > 0 && (!positions || !q || !k || !q_out || (!store && !k_out)))
    return SA_ERR_INVALID_ARG;
  if (!aligned(rot->turns, 8) || !aligned(positions, 4) || !aligned(q, 16) || !aligned(k, 16) ||
      !aligned(q_out, 16) || !aligned(k_out, 16))
    return SA_ERR_INVALID_ARG;
  // the stride of an extent of one is not used
  auto strides = [&](const int64_t* s, int32_t heads, int64_t least, int64_t* to) {
    to[0] = tokens > 1 ? s[0] : 0;
    to[1] = heads > 1 ? s[1] : 0;
    for (int i = 0; i < 2; ++i)
      if ((i ? heads : tokens) > 1 && (to[i] % 8 || to[i] < least || to[i] >= kMaxStride))
        return false;
    return true;
  };
  if (!strides(qs, hq, 0, a->qs) || !strides(ks, hkv, 0, a->ks) ||
      !strides(qos, hq, rot->head_dim, a->qos))
    return SA_ERR_INVALID_ARG;
  a->kos[0] = a->kos[1] = 0;
  if (k_out && !strides(kos, hkv, rot->head_dim, a->kos)) return SA_ERR_INVALID_ARG;
  // they would be written by two warps
  if (rows_share(tokens, hq, rot->head_dim, a->qos) ||
      (k_out && rows_share(tokens, hkv, rot->head_dim, a->kos)))
    return SA_ERR_INVALID_ARG;
  auto same = [](const int64_t* x, const int64_t* y) { return x[0] == y[0] && x[1] == y[1]; };
  if (tokens > 0) {
    if ((q_out == q && !same(a->qs, a->qos)) || (k_out == k && !same(a->ks, a->kos)) ||
        q_out == k || k_out == q || q_out == k_out)
      return SA_ERR_INVALID_ARG;
  }
  a->turns = rot->turns;
  a->factor = rot->factor;
  a->d = rot->head_dim;
  a->rot = rot->rot_dim;
  a->interleaved = rot->interleaved;
  a->tokens = tokens;
  a->Hq = hq;
  a->Hkv = hkv;
  a->positions = positions;
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->k = static_cast<const __nv_bfloat16*>(k);
  a->q_out = static_cast<__nv_bfloat16*>(q_out);
  a->k_out = static_cast<__nv_bfloat16*>(k_out);
  a->v = nullptr;
  a->slots = nullptr;
  a->k_pages = a->v_pages = nullptr;
  a->vs[0] = a->vs[1] = a->k_page_stride = a->v_page_stride = a->num_slots = 0;
  a->page_shift = 0;
  a->dev_status = nullptr;
  return SA_OK;
}

sa_status run_rotary(const sa_paged::RotaryArgs& a, sa_stream_t stream) {
  if (a.tokens == 0) return SA_OK;
  int sms = 0;
  const sa_status s = sa_paged::sm_count(&sms);
  if (s != SA_OK) return s;
  return sa_k::cuda_status(
      sa_paged::launch_rotary(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

using sa_k::cuda_status;
using sa_paged::sm_count;

}  // namespace

namespace sa_paged {

sa_status sm_count(int* sms) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SA_ERR_CUDA;
  const bool kept = dev < kMaxDevices;
  *sms = kept ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*sms > 0) return SA_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  if (kept) known[dev].store(*sms, std::memory_order_relaxed);
  return SA_OK;
}

}  // namespace sa_paged

extern "C" {

sa_status sparse_attn_paged_append(const sa_paged_cache* cache, const void* k_new,
                                   const void* v_new, const int64_t* k_strides,
                                   const int64_t* v_strides, int32_t num_new,
                                   const int32_t* counts, const int32_t* start, int32_t* lens_out,
                                   int32_t* dev_status, sa_stream_t stream) {
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  if (!k_new || !v_new || !k_strides || !v_strides || !lens_out || !dev_status)
    return SA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(counts, 4) || !aligned(start, 4) ||
      !aligned(lens_out, 4) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  if (num_new < 1) return SA_ERR_SHAPE;
  sa_paged::AppendArgs a;
  a.c = *cache;
  a.k_new = k_new;
  a.v_new = v_new;
  for (int i = 0; i < 3; ++i) {
    if (k_strides[i] < 0 || k_strides[i] % 8 || v_strides[i] < 0 || v_strides[i] % 8)
      return SA_ERR_INVALID_ARG;
    a.ks[i] = k_strides[i];
    a.vs[i] = v_strides[i];
  }
  // a row's new length must not replace another row's count
  const size_t per_seq = size_t(cache->batch) * 4;
  if (sa_paged::overlap(lens_out, per_seq * cache->num_kv_heads, counts, per_seq) &&
      !(cache->num_kv_heads == 1 && lens_out == counts))
    return SA_ERR_INVALID_ARG;
  a.num_new = num_new;
  a.counts = counts;
  a.start = start;
  a.lens_out = lens_out;
  a.dev_status = dev_status;
  return cuda_status(sa_paged::launch_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_paged_attend_workspace_size(const sa_paged_cache* cache,
                                                  int32_t num_q_heads, int32_t accumulate,
                                                  size_t* bytes) {
  if (!bytes) return SA_ERR_INVALID_ARG;
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  s = check_heads(cache, num_q_heads);
  if (s != SA_OK) return s;
  if (accumulate != 0 && accumulate != 1) return SA_ERR_INVALID_ARG;
  int sms = 0;
  s = sm_count(&sms);
  if (s != SA_OK) return s;
  *bytes = sa_paged::attend_workspace(*cache, num_q_heads, accumulate != 0, sms);
  return SA_OK;
}

sa_status sparse_attn_paged_attend(const sa_paged_cache* cache, const void* q, int64_t q_stride_b,
                                   int64_t q_stride_h, int32_t num_q_heads, void* o,
                                   int32_t o_dtype, float* lse, float* weights_out, void* ws,
                                   size_t ws_bytes, int32_t* dev_status, sa_stream_t stream) {
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  s = check_heads(cache, num_q_heads);
  if (s != SA_OK) return s;
  if (!q || !o || !ws || !dev_status) return SA_ERR_INVALID_ARG;
  if (o_dtype != SA_DTYPE_BF16 && o_dtype != SA_DTYPE_F32) return SA_ERR_INVALID_ARG;
  if (weights_out && !cache->weights) return SA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(ws, 256) || !aligned(lse, 4) ||
      !aligned(weights_out, 4) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  // the stride of an extent of one is not used
  if (cache->batch == 1) q_stride_b = int64_t(num_q_heads) * cache->head_dim;
  if (num_q_heads == 1) q_stride_h = cache->head_dim;
  if (q_stride_b % 8 || q_stride_h % 8 || q_stride_b < cache->head_dim ||
      q_stride_h < cache->head_dim || q_stride_b >= kMaxStride || q_stride_h >= kMaxStride)
    return SA_ERR_INVALID_ARG;
  int sms = 0;
  s = sm_count(&sms);
  if (s != SA_OK) return s;
  if (ws_bytes < sa_paged::attend_workspace(*cache, num_q_heads, weights_out != nullptr, sms))
    return SA_ERR_INVALID_ARG;
  sa_paged::AttendArgs a;
  a.c = *cache;
  a.q = q;
  a.qsb = q_stride_b;
  a.qsh = q_stride_h;
  a.Hq = num_q_heads;
  a.o = o;
  a.out_f32 = o_dtype == SA_DTYPE_F32;
  a.lse = lse;
  a.weights_out = weights_out;
  a.ws = ws;
  a.dev_status = dev_status;
  a.wait_ns = sa_host::wait_limit();
  bool encode_failed = false;
  cudaError_t e =
      sa_paged::launch_attend(a, sms, reinterpret_cast<cudaStream_t>(stream), &encode_failed);
  return encode_failed ? SA_ERR_CUDA : cuda_status(e);
}

sa_status sparse_attn_paged_evict_workspace_size(const sa_paged_cache* cache, size_t* bytes) {
  if (!bytes) return SA_ERR_INVALID_ARG;
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  s = check_evict(cache);
  if (s != SA_OK) return s;
  *bytes = sa_paged::evict_workspace(*cache);
  return SA_OK;
}

sa_status sparse_attn_paged_evict(const sa_paged_cache* cache, const int32_t* keep, int32_t sinks,
                                  int32_t recent, int32_t* lens_out, float* weights_out,
                                  int32_t* positions_out, void* ws, size_t ws_bytes,
                                  int32_t* dev_status, sa_stream_t stream) {
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  s = check_evict(cache);
  if (s != SA_OK) return s;
  if (!keep || !cache->weights || !lens_out || !weights_out || !ws || !dev_status)
    return SA_ERR_INVALID_ARG;
  if ((cache->positions != nullptr) != (positions_out != nullptr)) return SA_ERR_INVALID_ARG;
  if (sinks < 0 || recent < 0) return SA_ERR_INVALID_ARG;
  if (!aligned(lens_out, 4) || !aligned(weights_out, 4) || !aligned(positions_out, 4) ||
      !aligned(ws, 16) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  sa_paged::EvictArgs a;
  for (int32_t g = 0; g < cache->num_kv_heads; ++g) {
    if (keep[g] < 0 || int64_t(keep[g]) < int64_t(sinks) + recent) return SA_ERR_INVALID_ARG;
    a.keep[g] = keep[g];
  }
  if (ws_bytes < sa_paged::evict_workspace(*cache)) return SA_ERR_INVALID_ARG;
  int sms = 0;
  s = sm_count(&sms);
  if (s != SA_OK) return s;
  a.c = *cache;
  a.sinks = sinks;
  a.recent = recent;
  a.lens_out = lens_out;
  a.weights_out = weights_out;
  a.positions_out = positions_out;
  a.ws = ws;
  a.dev_status = dev_status;
  return cuda_status(sa_paged::launch_evict(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_rotary(const sa_rotary* rot, int32_t tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, const int32_t* positions, const void* q,
                             const int64_t* q_strides, const void* k, const int64_t* k_strides,
                             void* q_out, const int64_t* q_out_strides, void* k_out,
                             const int64_t* k_out_strides, sa_stream_t stream) {
  sa_paged::RotaryArgs a;
  const sa_status s =
      rotary_args(rot, tokens, num_q_heads, num_kv_heads, positions, q, q_strides, k, k_strides,
                  q_out, q_out_strides, k_out, k_out_strides, false, &a);
  return s != SA_OK ? s : run_rotary(a, stream);
}

sa_status sparse_attn_rotary_store(const sa_rotary* rot, int32_t tokens, int32_t num_q_heads,
                                   const int32_t* positions, const void* q,
                                   const int64_t* q_strides, const void* k,
                                   const int64_t* k_strides, const void* v,
                                   const int64_t* v_strides, void* q_out,
                                   const int64_t* q_out_strides, void* k_out,
                                   const int64_t* k_out_strides, const sa_paged_cache* cache,
                                   const int64_t* slots, int32_t* dev_status, sa_stream_t stream) {
  sa_status s = check_cache(cache);
  if (s != SA_OK) return s;
  sa_paged::RotaryArgs a;
  s = rotary_args(rot, tokens, num_q_heads, cache->num_kv_heads, positions, q, q_strides, k,
                  k_strides, q_out, q_out_strides, k_out, k_out_strides, true, &a);
  if (s != SA_OK) return s;
  if (rot->head_dim != cache->head_dim) return SA_ERR_SHAPE;
  if (!v_strides || !dev_status || (tokens > 0 && (!v || !slots))) return SA_ERR_INVALID_ARG;
  if (!aligned(v, 16) || !aligned(slots, 8) || !aligned(dev_status, 4)) return SA_ERR_INVALID_ARG;
  // (an output may be its own input, which v is not)
  if (tokens > 0 && (q_out == v || k_out == v)) return SA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    const bool used = (i ? cache->num_kv_heads : tokens) > 1;
    if (used && (v_strides[i] < 0 || v_strides[i] % 8 || v_strides[i] >= kMaxStride))
      return SA_ERR_INVALID_ARG;
    a.vs[i] = used ? v_strides[i] : 0;
  }
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.slots = slots;
  a.k_pages = static_cast<__nv_bfloat16*>(cache->k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(cache->v_pages);
  a.k_page_stride = cache->k_page_stride;
  a.v_page_stride = cache->v_page_stride;
  a.page_shift = __builtin_ctz(unsigned(cache->page));
  a.num_slots = cache->num_pages * cache->page;
  a.dev_status = dev_status;
  return run_rotary(a, stream);
}

sa_status sparse_attn_paged_grow_workspace_size(const sa_page_pool* pool, size_t* bytes) {
  if (!bytes) return SA_ERR_INVALID_ARG;
  const sa_status s = check_pool(pool);
  if (s != SA_OK) return s;
  *bytes = sa_paged::grow_workspace(pool->batch, pool->num_kv_heads);
  return SA_OK;
}

sa_status sparse_attn_paged_grow(const sa_page_pool* pool, const sa_page_growth* g, void* ws,
                                 size_t ws_bytes, int32_t* dev_status, sa_stream_t stream) {
  const sa_status s = check_pool(pool);
  if (s != SA_OK) return s;
  if (!g || !g->lens_out || !g->owned_out || !g->free_count_out || !ws || !dev_status)
    return SA_ERR_INVALID_ARG;
  if (g->tokens < 0 || g->tokens > (1 << 30) || (!g->cu && g->tokens % pool->batch))
    return SA_ERR_SHAPE;
  if (g->tokens > 0 && !g->slots) return SA_ERR_INVALID_ARG;
  if (!aligned(g->cu, 4) || !aligned(g->counts, 4) || !aligned(g->start, 4) ||
      !aligned(g->slots, 8) || !aligned(g->token_positions, 4) || !aligned(g->granted, 4) ||
      !aligned(g->lens_out, 4) || !aligned(g->owned_out, 4) || !aligned(g->free_count_out, 4) ||
      !aligned(g->start_out, 4) || !aligned(ws, 256) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  if (ws_bytes < sa_paged::grow_workspace(pool->batch, pool->num_kv_heads))
    return SA_ERR_INVALID_ARG;
  // the slots are written while lengths and counts are read
  const size_t seqs = size_t(pool->batch) * 4, rows = seqs * pool->num_kv_heads;
  const struct {
    const void* p;
    size_t n;
  } out[] = {{g->slots, size_t(g->tokens) * pool->num_kv_heads * 8},
             {g->token_positions, size_t(g->tokens) * 4}},
    other[] = {{pool->lens, rows}, {pool->owned, rows}, {pool->free_count, 4},
               {pool->free_pages, size_t(pool->num_pages) * 4},
               {pool->table, rows * pool->max_pages}, {g->cu, seqs + 4}, {g->counts, seqs},
               {g->ended, size_t(pool->batch)}, {g->start, seqs}, {g->lens_out, rows},
               {g->owned_out, rows}, {g->free_count_out, 4}, {g->start_out, seqs},
               {g->granted, seqs}};
  for (const auto& o : out)
    for (const auto& x : other)
      if (sa_paged::overlap(o.p, o.n, x.p, x.n)) return SA_ERR_INVALID_ARG;
  if (sa_paged::overlap(out[0].p, out[0].n, out[1].p, out[1].n)) return SA_ERR_INVALID_ARG;
  sa_paged::GrowArgs a;
  a.table = pool->table;
  a.lens = pool->lens;
  a.owned = pool->owned;
  a.free_pages = pool->free_pages;
  a.free_count = pool->free_count;
  a.weights = pool->weights;
  a.slot_positions = pool->positions;
  a.cu = g->cu;
  a.counts = g->counts;
  a.ended = g->ended;
  a.start = g->start;
  a.slots = g->slots;
  a.positions = g->token_positions;
  a.granted = g->granted;
  a.lens_out = g->lens_out;
  a.owned_out = g->owned_out;
  a.free_count_out = g->free_count_out;
  a.start_out = g->start_out;
  a.num_pages = pool->num_pages;
  a.page = pool->page;
  a.page_shift = __builtin_ctz(unsigned(pool->page));
  a.max_pages = pool->max_pages;
  a.batch = pool->batch;
  a.Hkv = pool->num_kv_heads;
  a.tokens = g->tokens;
  a.span = g->tokens / pool->batch;
  // exact for rows below 2^20 (their product with the error, below Hkv, stays below
  // 2^32)
  a.inv_heads = a.Hkv > 1 && a.Hkv <= 4096
                    ? uint32_t(((uint64_t(1) << 32) + uint32_t(a.Hkv) - 1) / uint32_t(a.Hkv))
                    : 0;
  a.ws = ws;
  a.dev_status = dev_status;
  int sms = 0;
  const sa_status n = sa_paged::sm_count(&sms);
  if (n != SA_OK) return n;
  return cuda_status(sa_paged::launch_grow(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
