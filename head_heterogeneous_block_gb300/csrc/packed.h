// Internal launch interface of the packed prompt attention.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "sparse_attn.h"

namespace sa_packed {

struct Args {
  sa_packed_shape s;
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu_q;        // [batch + 1]
  const int32_t* cu_k;
  void* o;
  float* lse;                 // [total_q][Hq] or NULL
  void* ws;
  int32_t* dev_status;
  uint64_t wait_ns;
};

// Query heads of a KV head that share a tile, and the tokens of a tile.
struct Tile {
  int32_t heads, tokens;
};
inline Tile tile_of(const sa_packed_shape& s) {
  const int32_t group = s.num_q_heads / s.num_kv_heads;
  Tile t{1, 128};
  for (int32_t f = 2; f <= 16 && f <= group; ++f)
    if (group % f == 0 && f * (128 / f) >= 125) t = Tile{f, 128 / f};
  return t;
}

// The factor of the scores' exponents, base 2.
inline float scale_log2(const sa_packed_shape& s) {
  return float(double(s.scale) * 1.4426950408889634);
}

// Tiles that any lengths of these totals can make, at most.
inline int64_t most_tiles(const sa_packed_shape& s) {
  const int64_t seqs = s.batch < s.total_q ? s.batch : s.total_q;
  return s.total_q / tile_of(s).tokens + seqs;
}

size_t workspace(const sa_packed_shape& s, int sms);
cudaError_t launch(const Args& a, int sms, cudaStream_t st, bool* encode_failed);

}  // namespace sa_packed
