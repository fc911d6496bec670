// Appending new tokens to a paged key-value cache.
//
// A copy: per token and row 2d bytes of key and of value are read and written,
// plus 8 bytes of weight and position.  A warp takes kSteps * (128 / d)
// consecutive tokens of one row; a half-warp-wide piece (d/8 lanes, 16 bytes
// each) covers one token's key, the next piece its value, and the loads of all
// kSteps steps are in flight before the first store.  With one such warp per
// row (a decode step) the warp also writes the row's new length, so the length
// array may be updated in place; with several, a row's warps all read the old
// length, and an in-place update is a second, tiny launch after them.  So it is
// where the new lengths go into what other warps still read: the start
// positions (the old lengths of one sequence, say) or the counts.
//
// Measured against the copy rate (6783 GB/s): 32767 tokens, 8 heads, d = 128:
// 42 us, 94%; 57 sequences of 1147 tokens, 16 heads, d = 64: 83 us, 97%; a
// decode step of 64 sequences, 8 heads: 2.8 us, a launch's time.  Blocks of
// eight warps: 3 to 8% slower; of sixteen 25%.  Four or sixteen steps: the same
// to 4% slower.

#include <cuda_bf16.h>

#include <algorithm>

#include "paged.h"
#include "ptx.cuh"

namespace {

using sa_paged::AppendArgs;

constexpr int kSteps = 8;
constexpr int kWarps = 4;

// The number of tokens row r appends, clamped to the free slots.
__device__ __forceinline__ int32_t new_tokens(const AppendArgs& a, int64_t r, int32_t len,
                                              int32_t cap) {
  int32_t m = a.counts ? a.counts[r / a.c.num_kv_heads] : a.num_new;
  if (m < 0 || m > a.num_new || m > cap - len) {
    atomicOr(a.dev_status, SA_DEV_BAD_COUNT);
    m = max(0, min(min(m, a.num_new), cap - len));
  }
  return m;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ AppendArgs a, int32_t chunks,
                                                             int write_lens) {
  constexpr int kPiece = D / 8;                 // lanes of one key (or value) row
  constexpr int kPer = 32 / (2 * kPiece);       // tokens of one step
  constexpr int kTokens = kSteps * kPer;        // tokens of a warp
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int lane = threadIdx.x & 31;
  const int64_t task = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t r = task / chunks;
  if (r >= int64_t(a.c.batch) * a.c.num_kv_heads) return;
  const int32_t chunk = int32_t(task - r * chunks);
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t len = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int32_t m = new_tokens(a, r, len, cap);
  __syncwarp();                                 // every lane has read the length
  if (write_lens && chunk == 0 && lane == 0) a.lens_out[r] = len + m;
  const int32_t t0 = chunk * kTokens;
  if (t0 >= m) return;
  const int64_t b = r / a.c.num_kv_heads, g = r % a.c.num_kv_heads;
  const int32_t* table = a.c.table + r * a.c.max_pages;
  const bool is_v = (lane / kPiece) & 1;
  const int x = (lane % kPiece) * 8;            // element of the row
  const int sub = lane / (2 * kPiece);          // token of the step
  const __nv_bfloat16* src =
      is_v ? static_cast<const __nv_bfloat16*>(a.v_new) + b * a.vs[0] + g * a.vs[1] + x
           : static_cast<const __nv_bfloat16*>(a.k_new) + b * a.ks[0] + g * a.ks[1] + x;
  const int64_t ts = is_v ? a.vs[2] : a.ks[2];
  const int shift = __ffs(a.c.page) - 1;        // pages are powers of two
  __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(is_v ? a.c.v_pages : a.c.k_pages) + x;
  const int64_t stride = is_v ? a.c.v_page_stride : a.c.k_page_stride;
  uint4 val[kSteps];
  int32_t page[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int32_t t = t0 + i * kPer + sub;
    if (t < m) {
      val[i] = *reinterpret_cast<const uint4*>(src + t * ts);
      page[i] = table[(len + t) >> shift];
    }
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int32_t t = t0 + i * kPer + sub;
    if (t < m) {
      if (page[i] < 0 || page[i] >= a.c.num_pages)
        bad = true;
      else
        *reinterpret_cast<uint4*>(pool + page[i] * stride +
                                  int64_t((len + t) & (a.c.page - 1)) * D) = val[i];
    }
  }
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
  const int32_t t = t0 + lane;
  if (lane < kTokens && t < m) {
    const int64_t at = r * cap + len + t;
    if (a.c.weights) a.c.weights[at] = 0.f;
    if (a.c.positions) a.c.positions[at] = (a.start ? a.start[b] : len) + t;
  }
}

// The new lengths, after the rows' warps have read what they replace.
__global__ void lens_kernel(const __grid_constant__ AppendArgs a) {
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int64_t r = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (r >= int64_t(a.c.batch) * a.c.num_kv_heads) return;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t len = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  a.lens_out[r] = len + new_tokens(a, r, len, cap);
}

template <int D>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
  constexpr int kTokens = kSteps * (32 / (2 * (D / 8)));
  const int64_t rows = int64_t(a.c.batch) * a.c.num_kv_heads;
  // a row takes no more new tokens than it has slots
  const int64_t most = std::min<int64_t>(a.num_new, int64_t(a.c.page) * a.c.max_pages);
  const int64_t chunks = (most + kTokens - 1) / kTokens;
  const int64_t blocks = (rows * chunks + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const size_t out = size_t(rows) * 4, per_seq = size_t(a.c.batch) * 4;
  const bool late = (chunks > 1 && a.lens_out == a.c.lens) ||
                    sa_paged::overlap(a.lens_out, out, a.start, per_seq) ||
                    sa_paged::overlap(a.lens_out, out, a.counts, per_seq);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<D>, a, int32_t(chunks), int(!late));
  if (e != cudaSuccess || !late) return e;
  cfg.gridDim = dim3(unsigned((rows + 255) / 256));
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, lens_kernel, a);
}

}  // namespace

namespace sa_paged {

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  return a.c.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sa_paged
