// C ABI entry points of the packed prompt attention: argument checks, then the
// launches of packed.cu.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "packed.h"
#include "paged.h"
#include "sparse_attn.h"
#include "wait_limit.h"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxStride = int64_t(1) << 38;   // elements; a TMA stride is below 2^40 bytes
constexpr int32_t kMaxTokens = 1 << 30;

sa_status check_shape(const sa_packed_shape* s) {
  if (!s) return SA_ERR_INVALID_ARG;
  if (s->total_q < 0 || s->total_q > kMaxTokens || s->total_k < 0 || s->total_k > kMaxTokens ||
      s->batch < 1 || s->batch > (1 << 20) || s->num_q_heads < 1 || s->num_kv_heads < 1 ||
      s->num_q_heads % s->num_kv_heads != 0)
    return SA_ERR_SHAPE;
  if (s->head_dim != 64 && s->head_dim != 128) return SA_ERR_UNSUPPORTED;
  // items (tiles and ranges of every head) are a 32-bit count
  const int64_t heads = s->num_q_heads / sa_packed::tile_of(*s).heads;
  if (heads > (1 << 20) || (sa_packed::most_tiles(*s) + 4096) > (int64_t(1) << 30) / heads)
    return SA_ERR_SHAPE;
  // (scores are scaled to base 2)
  if (!(s->scale > 0.f) || !std::isfinite(sa_packed::scale_log2(*s))) return SA_ERR_INVALID_ARG;
  return SA_OK;
}

// The strides of [tokens][heads][d]; those of an extent of one are not used.
bool strides_ok(int64_t tokens, int64_t heads, int32_t d, int64_t st, int64_t sh) {
  auto ok = [&](int64_t x) { return x % 8 == 0 && x >= d && x < kMaxStride; };
  return (tokens <= 1 || ok(st)) && (heads <= 1 || ok(sh));
}

}  // namespace

extern "C" {

sa_status sparse_attn_packed_workspace_size(const sa_packed_shape* shp, size_t* bytes) {
  if (!bytes) return SA_ERR_INVALID_ARG;
  sa_status s = check_shape(shp);
  if (s != SA_OK) return s;
  int sms = 0;
  s = sa_paged::sm_count(&sms);
  if (s != SA_OK) return s;
  *bytes = sa_packed::workspace(*shp, sms);
  return SA_OK;
}

sa_status sparse_attn_packed_forward(const sa_packed_shape* shp, const void* q, const void* k,
                                     const void* v, const int32_t* cu_q, const int32_t* cu_k,
                                     void* o, float* lse, void* ws, size_t ws_bytes,
                                     int32_t* dev_status, sa_stream_t stream) {
  sa_status s = check_shape(shp);
  if (s != SA_OK) return s;
  if (!cu_q || !cu_k || !ws || !dev_status) return SA_ERR_INVALID_ARG;
  // an empty tensor may have no address
  if ((shp->total_q > 0 && (!q || !o)) || (shp->total_k > 0 && (!k || !v)))
    return SA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4) || !aligned(ws, 256) ||
      !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  const int64_t tq = shp->total_q, tk = shp->total_k, hq = shp->num_q_heads,
                hkv = shp->num_kv_heads;
  const int32_t d = shp->head_dim;
  if (!strides_ok(tq, hq, d, shp->q_stride_t, shp->q_stride_h) ||
      !strides_ok(tk, hkv, d, shp->k_stride_t, shp->k_stride_h) ||
      !strides_ok(tk, hkv, d, shp->v_stride_t, shp->v_stride_h) ||
      !strides_ok(tq, hq, d, shp->o_stride_t, shp->o_stride_h))
    return SA_ERR_INVALID_ARG;
  // rows of o that share memory would be written by two CTAs
  using Wide = __int128;
  if (tq > 1 && hq > 1 && shp->o_stride_t < Wide(hq - 1) * shp->o_stride_h + d &&
      shp->o_stride_h < Wide(tq - 1) * shp->o_stride_t + d)
    return SA_ERR_INVALID_ARG;
  // (o may lie between the rows of a fused tensor that holds q, k and v: only
  // the same first address is surely wrong)
  if (tq > 0 && (o == q || (tk > 0 && (o == k || o == v)))) return SA_ERR_INVALID_ARG;
  int sms = 0;
  s = sa_paged::sm_count(&sms);
  if (s != SA_OK) return s;
  if (ws_bytes < sa_packed::workspace(*shp, sms)) return SA_ERR_INVALID_ARG;
  if (shp->total_q == 0) return SA_OK;
  sa_packed::Args a;
  a.s = *shp;
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.o = o;
  a.lse = lse;
  a.ws = ws;
  a.dev_status = dev_status;
  a.wait_ns = sa_host::wait_limit();
  bool encode_failed = false;
  cudaError_t e =
      sa_packed::launch(a, sms, reinterpret_cast<cudaStream_t>(stream), &encode_failed);
  return encode_failed ? SA_ERR_CUDA : sa_k::cuda_status(e);
}

}  // extern "C"
