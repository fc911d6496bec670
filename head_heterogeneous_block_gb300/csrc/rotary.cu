// Rotary positions of queries and keys, with the paged cache's store of rotated
// keys and of values in the same pass.
//
// Pair i of a head's first `rot` elements, (x, y) = elements (i, i + rot/2) or
// (2i, 2i + 1), becomes m (x cos a - y sin a, y cos a + x sin a) with the angle
// a = position * f_i.  It is a copy with some arithmetic: bytes bound it.
//
// Angles.  An fp32 product of a position of a million and a frequency of one is
// off by 0.06 radians, so frequencies come as 64-bit fractions of a turn,
// t_i = f_i / 2 pi * 2^64 mod 2^64: position * t_i in wrapping integer arithmetic
// is the exact fraction of a turn for any 32-bit position (within position *
// 2^-65), its upper half as a signed number the angle in half turns, which
// sincospif takes without a range reduction of its own.
//
// Layout.  d / 16 lanes take one head, 16 elements each: eight pairs, loaded as
// two 16-byte pieces.  The same lane takes the same pairs of every head, so a
// warp works out its token's sines once for all of its heads; each lane works
// out as many as there are lanes to share them and gets the rest from the
// others.  Lanes behind `rot` pass their 16 elements on.
//
// Measured (GB300): 32767 tokens, 32/8 heads, d = 128, with the store: 129 us, 6.8
// TB/s, the copy rate; 2049 tokens, 28/4 heads, half of each head in interleaved
// pairs: 9.7 us from HBM, 6.7 with all in L2, of 5.0 at the copy rate: the chain from
// a position to its sines stands before a warp's first load, which a call of many
// waves does not see; 4096 tokens, 8/2 heads, d = 64: 4.9 and 4.2 us of 1.6; a decode
// step of 64 tokens: 2.3 us, a launch's time.

#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace {

using sa_paged::RotaryArgs;

constexpr int kWarps = 4;

// Cosine and sine, times the factor, of one pair's angle.
__device__ __forceinline__ float2 turn_of(const RotaryArgs& a, int32_t position, int pair) {
  const uint64_t t = uint64_t(int64_t(position)) * __ldg(&a.turns[pair]);
  const float half_turns = float(int32_t(t >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * a.factor, s * a.factor);
}

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// (x, y) pairs of bf16 words: half layout, x from one word and y from another.
__device__ __forceinline__ void rotate_half(uint32_t& x, uint32_t& y, float2 t0, float2 t1) {
  const float2 xs = unpack(x), ys = unpack(y);
  x = sa_dev::pack_bf16x2(xs.x * t0.x - ys.x * t0.y, xs.y * t1.x - ys.y * t1.y);
  y = sa_dev::pack_bf16x2(ys.x * t0.x + xs.x * t0.y, ys.y * t1.x + xs.y * t1.y);
}
__device__ __forceinline__ void rotate_pair(uint32_t& w, float2 t) {
  const float2 v = unpack(w);
  w = sa_dev::pack_bf16x2(v.x * t.x - v.y * t.y, v.y * t.x + v.x * t.y);
}

// A warp takes `steps` steps of 32 / (D / 16) heads of one token, kUnroll of
// them in flight.  Heads are counted through q, k and (with a store) v.
template <int D, int kUnroll>
__global__ void __launch_bounds__(32 * kWarps)
    rotary_kernel(const __grid_constant__ RotaryArgs a, int32_t chunks, int32_t steps) {
  constexpr int kLanes = D / 16;
  constexpr int kHeads = 32 / kLanes;
  sa_dev::launch_dependents();
  sa_dev::wait_dependency();
  const int lane = threadIdx.x & 31;
  const int64_t task = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int32_t t = int32_t(task / chunks);
  if (t >= a.tokens) return;
  const int32_t heads = a.Hq + a.Hkv + (a.slots ? a.Hkv : 0);
  const int32_t first = int32_t(task - int64_t(t) * chunks) * steps * kHeads;
  const int l = lane % kLanes;
  const bool turned = l * 16 < a.rot;
  // pieces of this lane: of a rotated head, and of one that is only copied
  const int half0 = a.interleaved || !turned ? l * 16 : l * 8;
  const int half1 = a.interleaved || !turned ? l * 16 + 8 : a.rot / 2 + l * 8;
  float2 cs[8];
  if (first < a.Hq + a.Hkv) {
    const int32_t position = a.positions[t];
    // lane x of the kHeads lanes that hold the same pairs works out 8 / kHeads of
    // them
    constexpr int kMine = 8 / kHeads;
    float2 mine[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      mine[i] = turned ? turn_of(a, position, l * 8 + (lane / kLanes) * kMine + i)
                       : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int src = l + (i / kMine) * kLanes;
      cs[i].x = __shfl_sync(0xffffffffu, mine[i % kMine].x, src);
      cs[i].y = __shfl_sync(0xffffffffu, mine[i % kMine].y, src);
    }
  }
  bool bad = false;
  for (int32_t s0 = 0; s0 < steps; s0 += kUnroll) {
    uint4 x[kUnroll], y[kUnroll];
    int64_t slot[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int32_t h = first + (s0 + i) * kHeads + lane / kLanes;
      if (h >= heads || s0 + i >= steps) continue;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const __nv_bfloat16* src =
          is_q ? a.q + t * a.qs[0] + h * a.qs[1]
               : is_v ? a.v + t * a.vs[0] + (h - a.Hq - a.Hkv) * a.vs[1]
                      : a.k + t * a.ks[0] + (h - a.Hq) * a.ks[1];
      x[i] = *reinterpret_cast<const uint4*>(src + (is_v ? l * 16 : half0));
      y[i] = *reinterpret_cast<const uint4*>(src + (is_v ? l * 16 + 8 : half1));
      slot[i] = -1;
      if (a.slots && !is_q)
        slot[i] = a.slots[int64_t(h - a.Hq - (is_v ? a.Hkv : 0)) * a.tokens + t];
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int32_t h = first + (s0 + i) * kHeads + lane / kLanes;
      if (h >= heads || s0 + i >= steps) continue;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      if (turned && !is_v) {
        if (a.interleaved) {
          rotate_pair(x[i].x, cs[0]);
          rotate_pair(x[i].y, cs[1]);
          rotate_pair(x[i].z, cs[2]);
          rotate_pair(x[i].w, cs[3]);
          rotate_pair(y[i].x, cs[4]);
          rotate_pair(y[i].y, cs[5]);
          rotate_pair(y[i].z, cs[6]);
          rotate_pair(y[i].w, cs[7]);
        } else {
          rotate_half(x[i].x, y[i].x, cs[0], cs[1]);
          rotate_half(x[i].y, y[i].y, cs[2], cs[3]);
          rotate_half(x[i].z, y[i].z, cs[4], cs[5]);
          rotate_half(x[i].w, y[i].w, cs[6], cs[7]);
        }
      }
      const int o0 = is_v ? l * 16 : half0, o1 = is_v ? l * 16 + 8 : half1;
      __nv_bfloat16* dst = is_q ? a.q_out + t * a.qos[0] + h * a.qos[1]
                           : is_v || !a.k_out ? nullptr
                                              : a.k_out + t * a.kos[0] + (h - a.Hq) * a.kos[1];
      if (dst) {
        *reinterpret_cast<uint4*>(dst + o0) = x[i];
        *reinterpret_cast<uint4*>(dst + o1) = y[i];
      }
      if (slot[i] >= 0 && slot[i] < a.num_slots) {
        __nv_bfloat16* pool = is_v ? a.v_pages + (slot[i] >> a.page_shift) * a.v_page_stride
                                   : a.k_pages + (slot[i] >> a.page_shift) * a.k_page_stride;
        pool += (slot[i] & ((1 << a.page_shift) - 1)) * D;
        *reinterpret_cast<uint4*>(pool + o0) = x[i];
        *reinterpret_cast<uint4*>(pool + o1) = y[i];
      } else if (slot[i] != -1) {
        bad = true;
      }
    }
  }
  if (bad) atomicOr(a.dev_status, SA_DEV_BAD_INDEX);
}

template <int D, int kUnroll>
cudaError_t launch(const RotaryArgs& a, int32_t steps, int32_t chunks, cudaStream_t st) {
  const int64_t blocks = (int64_t(a.tokens) * chunks + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<D, kUnroll>, a, chunks, steps);
}

template <int D>
cudaError_t launch_d(const RotaryArgs& a, int sms, cudaStream_t st) {
  constexpr int kHeads = 32 / (D / 16);
  const int32_t all = (a.Hq + a.Hkv + (a.slots ? a.Hkv : 0) + kHeads - 1) / kHeads;
  // Steps of all tokens a processor: up to 16 (64 tokens of 32 + 8 heads, d =
  // 128: 2.2 us) a step a warp, for latency; up to 48 two (512 tokens: 3.5 us,
  // against 4.0 with one and 4.2 with four); up to 220 four (2049 tokens: 7.8
  // us, against 9.0 with two and 9.3 with twelve); then twelve, which share the
  // token's sines (16384 tokens: 68 us, against 74 with four)
  const int64_t load = int64_t(a.tokens) * all / sms;
  auto with = [&](int32_t steps, auto unroll) {
    const int32_t chunks = (all + steps - 1) / steps;
    return launch<D, decltype(unroll)::value>(a, (all + chunks - 1) / chunks, chunks, st);
  };
  if (load <= 16) return with(1, std::integral_constant<int, 1>{});
  if (load <= 48) return with(2, std::integral_constant<int, 2>{});
  if (load <= 220) return with(4, std::integral_constant<int, 2>{});
  return with(12, std::integral_constant<int, 4>{});
}

}  // namespace

namespace sa_paged {

cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t st) {
  return a.d == 128 ? launch_d<128>(a, sms, st) : launch_d<64>(a, sms, st);
}

}  // namespace sa_paged
