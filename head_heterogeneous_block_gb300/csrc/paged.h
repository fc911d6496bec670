// Internal launch interface of the paged key-value cache operators.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sparse_attn.h"

namespace sa_paged {

constexpr int kMaxDevices = 64;       // of a process, for what is set up once a device
constexpr int kMaxKvHeads = 256;      // budgets travel as a kernel parameter
constexpr int64_t kMaxEvictSlots = 262144;

struct AppendArgs {
  sa_paged_cache c;
  const void* k_new;
  const void* v_new;
  int64_t ks[3], vs[3];               // sequence, head, token strides, elements
  int32_t num_new;
  const int32_t* counts;              // [Bt] or NULL
  const int32_t* start;               // [Bt] or NULL
  int32_t* lens_out;
  int32_t* dev_status;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t st);

struct AttendArgs {
  sa_paged_cache c;
  const void* q;
  int64_t qsb, qsh;
  int32_t Hq;
  void* o;
  int32_t out_f32;
  float* lse;
  float* weights_out;                 // or NULL
  void* ws;
  int32_t* dev_status;
  uint64_t wait_ns;
};
size_t attend_workspace(const sa_paged_cache& c, int32_t Hq, bool accumulate, int sms);
cudaError_t launch_attend(const AttendArgs& a, int sms, cudaStream_t st, bool* encode_failed);

struct GrowArgs {
  int32_t* table;
  const int32_t* lens;
  const int32_t* owned;
  int32_t* free_pages;
  const int32_t* free_count;
  float* weights;                     // or NULL
  int32_t* slot_positions;            // or NULL
  const int32_t* cu;                  // [batch + 1], or NULL: spans of `span` tokens
  const int32_t* counts;              // or NULL
  const uint8_t* ended;               // or NULL
  const int32_t* start;               // or NULL
  int64_t* slots;                     // [Hkv][tokens]
  int32_t* positions;                 // [tokens] or NULL
  int32_t* granted;                   // [batch] or NULL
  int32_t* lens_out;
  int32_t* owned_out;
  int32_t* free_count_out;
  int32_t* start_out;                 // or NULL
  int64_t num_pages;
  int32_t page, page_shift, max_pages, batch, Hkv, tokens, span;
  uint32_t inv_heads;                 // 2^32 / Hkv, rounded up; 0: divide
  void* ws;
  int32_t* dev_status;
};
size_t grow_workspace(int32_t batch, int32_t num_kv_heads);
cudaError_t launch_grow(const GrowArgs& a, int sms, cudaStream_t st);

struct RotaryArgs {
  const uint64_t* turns;              // [rot / 2]
  const int32_t* positions;           // [tokens]
  const __nv_bfloat16* q;             // token, head strides beside each
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;             // with slots
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;               // or NULL
  int64_t qs[2], ks[2], vs[2], qos[2], kos[2];
  const int64_t* slots;               // [Hkv][tokens] or NULL: no store
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  int64_t k_page_stride, v_page_stride, num_slots;
  int32_t page_shift, tokens, Hq, Hkv, d, rot, interleaved;
  float factor;
  int32_t* dev_status;                // with slots
};
cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t st);

struct EvictArgs {
  sa_paged_cache c;
  int32_t keep[kMaxKvHeads];
  int32_t sinks, recent;
  int32_t* lens_out;
  float* weights_out;
  int32_t* positions_out;             // NULL with c.positions == NULL
  void* ws;
  int32_t* dev_status;
};
size_t evict_workspace(const sa_paged_cache& c);
cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t st);

// Processors of the current device, asked for once.
sa_status sm_count(int* sms);

// Lets `kern` use `bytes` of dynamic shared memory on the current device: once
// a device, which bit mask `done` (of that kernel) keeps.
template <class Kernel>
cudaError_t allow_shared(Kernel* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < kMaxDevices ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Whether n bytes at p and m bytes at q (either may be NULL) share memory.
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + m && b < a + n;
}

#ifdef __CUDACC__
// A row's length, clamped to its table and flagged when it was out of range.
__device__ __forceinline__ int32_t row_len(const int32_t* lens, int64_t r, int32_t cap,
                                           int32_t* dev_status) {
  int32_t n = lens[r];
  if (n < 0 || n > cap) {
    atomicOr(dev_status, SA_DEV_BAD_COUNT);
    n = n < 0 ? 0 : cap;
  }
  return n;
}
#endif

}  // namespace sa_paged
