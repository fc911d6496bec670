// Attention of one new token per sequence over a paged key-value cache.
//
// One CTA per (sequence, query head): four warps take every fourth slot, a
// lane holds d/32 elements of the row, the dot product is reduced over the
// warp, each warp keeps an online softmax and the four states are merged.  A
// second kernel adds each slot's probabilities to its weight.

#include <cuda_bf16.h>

#include <cmath>

#include "paged.h"
#include "ptx.cuh"

namespace {

using sa_paged::AttendArgs;

constexpr int kWarps = 4;

// The pool row of slot t: page 0 when the table's entry is out of range.
__device__ __forceinline__ int64_t slot_offset(const AttendArgs& a, int64_t r, int32_t t,
                                               int64_t stride) {
  int32_t p = a.c.table[r * a.c.max_pages + t / a.c.page];
  if (p < 0 || p >= a.c.num_pages) {
    atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
    p = 0;
  }
  return p * stride + int64_t(t % a.c.page) * a.c.head_dim;
}

template <int D>
__device__ __forceinline__ float dot(const float (&q)[D / 32], const __nv_bfloat16* k, int lane) {
  float s = 0.f;
#pragma unroll
  for (int x = 0; x < D / 32; ++x) s = fmaf(q[x], __bfloat162float(k[lane + 32 * x]), s);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const AttendArgs a, float scale_log2) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x, b = bh / a.Hq, h = bh % a.Hq;
  const int64_t r = b * a.c.num_kv_heads + h / (a.Hq / a.c.num_kv_heads);
  const int32_t n = sa_paged::row_len(a.c.lens, r, a.c.page * a.c.max_pages, a.dev_status);
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.qsb + h * a.qsh;
  float q[D / 32], o[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    q[x] = __bfloat162float(qp[lane + 32 * x]) * scale_log2;
    o[x] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int32_t t = warp; t < n; t += kWarps) {
    const float s =
        dot<D>(q, static_cast<const __nv_bfloat16*>(a.c.k_pages) + slot_offset(a, r, t, a.c.k_page_stride), lane);
    const __nv_bfloat16* v =
        static_cast<const __nv_bfloat16*>(a.c.v_pages) + slot_offset(a, r, t, a.c.v_page_stride);
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - ref), p = exp2f(s - ref);
    l = l * alpha + p;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = fmaf(p, __bfloat162float(v[lane + 32 * x]), o[x] * alpha);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < D / 32; ++x) so[warp][lane + 32 * x] = o[x];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  const float ref = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) L += sl[w] * exp2f(sm[w] - ref);
  const float lse2 = n ? ref + log2f(L) : -INFINITY;
  for (int x = threadIdx.x; x < D; x += 32 * kWarps) {
    float acc = 0.f;
    for (int w = 0; w < kWarps; ++w) acc += so[w][x] * exp2f(sm[w] - ref);
    const float val = n ? acc / L : 0.f;
    if (a.out_f32)
      static_cast<float*>(a.o)[bh * D + x] = val;
    else
      static_cast<__nv_bfloat16*>(a.o)[bh * D + x] = __float2bfloat16_rn(val);
  }
  if (threadIdx.x == 0) {
    static_cast<float*>(a.ws)[bh] = lse2;
    if (a.lse) a.lse[bh] = lse2 * 0.6931471805599453f;
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) weights_kernel(const AttendArgs a,
                                                              float scale_log2) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t cap = a.c.page * a.c.max_pages;
  const int32_t pieces = cap / 16;
  const int64_t r = blockIdx.x / pieces;
  const int32_t t0 = int32_t(blockIdx.x % pieces) * 16;
  const int32_t n = sa_paged::row_len(a.c.lens, r, cap, a.dev_status);
  const int64_t b = r / a.c.num_kv_heads, g = r % a.c.num_kv_heads;
  const int G = a.Hq / a.c.num_kv_heads;
  for (int32_t t = t0 + warp; t < min(n, t0 + 16); t += kWarps) {
    const __nv_bfloat16* k =
        static_cast<const __nv_bfloat16*>(a.c.k_pages) + slot_offset(a, r, t, a.c.k_page_stride);
    float sum = 0.f;
    for (int x = 0; x < G; ++x) {
      const int64_t h = g * G + x;
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.qsb + h * a.qsh;
      float q[D / 32];
#pragma unroll
      for (int y = 0; y < D / 32; ++y) q[y] = __bfloat162float(qp[lane + 32 * y]) * scale_log2;
      sum += exp2f(dot<D>(q, k, lane) - static_cast<const float*>(a.ws)[b * a.Hq + h]);
    }
    if (lane == 0) a.weights_out[r * cap + t] = a.c.weights[r * cap + t] + sum;
  }
}

template <int D>
cudaError_t launch(const AttendArgs& a, cudaStream_t st) {
  const float c = float(1.4426950408889634 / std::sqrt(double(D)));
  attend_kernel<D><<<unsigned(a.c.batch * a.Hq), 32 * kWarps, 0, st>>>(a, c);
  if (a.weights_out)
    weights_kernel<D><<<unsigned(int64_t(a.c.batch) * a.c.num_kv_heads * a.c.page *
                                 a.c.max_pages / 16), 32 * kWarps, 0, st>>>(a, c);
  return cudaGetLastError();
}

}  // namespace

namespace sa_paged {

size_t attend_workspace(const sa_paged_cache& c, int32_t Hq, bool, int) {
  return size_t(c.batch) * Hq * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, int, cudaStream_t st, bool* encode_failed) {
  *encode_failed = false;
  return a.c.head_dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sa_paged
