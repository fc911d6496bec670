// C ABI entry points of the paged key-value cache: argument checks, then the
// launches of paged_append.cu, paged_attend.cu and paged_evict.cu.

#include <cuda_runtime.h>

#include <atomic>
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

}  // extern "C"
