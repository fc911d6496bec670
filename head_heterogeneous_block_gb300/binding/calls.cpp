// The calls of PackedAttention, Rotary and PagePool: checks of their tensors and
// the C entry point, in one native function each.
//
// Reading a tensor's type, sizes, strides, device and address from Python takes
// some 0.6 us, and such a call has up to a dozen tensors: 8 of the 12 us that a
// decode step's rotary store took on the host, whose kernel takes 2.  From here
// it is a few ns.  What is wrong raises what the Python classes raise (TypeError
// for types, ValueError for the rest); the entry point's status is returned.

#include <Python.h>

#include <c10/core/ScalarType.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "sparse_attn.h"

namespace {

struct Refused {};   // a Python exception is set

constexpr int64_t kMaxStride = int64_t(1) << 38;   // elements

[[noreturn]] void type_error(const char* name, const char* what) {
  PyErr_Format(PyExc_TypeError, "%s must be %s", name, what);
  throw Refused{};
}
template <class... Args>
[[noreturn]] void value_error(const char* format, Args... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(name, "a tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, int64_t index, const char* name) {
  if (!t.is_cuda() || t.get_device() != index)
    value_error("%s must be on cuda:%lld", name, static_cast<long long>(index));
}

// A bf16 [tokens, heads, d] view, whose rows are at least `least` elements apart.
struct Rows {
  void* at = nullptr;
  int64_t tokens = 0;
  int64_t strides[2] = {0, 0};
};
Rows rows(PyObject* o, int64_t index, int64_t heads, int64_t d, int64_t least, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16) type_error(name, "bfloat16");
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d)
    value_error("%s must be [tokens, %lld, %lld]", name, static_cast<long long>(heads),
                static_cast<long long>(d));
  if (t.stride(2) != 1) value_error("the last dimension of %s must be contiguous", name);
  // (the stride of an extent of one is not used)
  for (int i = 0; i < 2; ++i)
    if (t.size(i) > 1 && (t.stride(i) % 8 || t.stride(i) < least || t.stride(i) >= kMaxStride))
      value_error("%s has a stride of %lld elements between %s: it must be a multiple of 8, at least "
                  "%lld and below 2^38", name, static_cast<long long>(t.stride(i)),
                  i ? "heads" : "tokens", static_cast<long long>(least));
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
    value_error("%s must start on a 16-byte boundary", name);
  on_device(t, index, name);
  return Rows{t.data_ptr(), t.size(0), {t.stride(0), t.stride(1)}};
}

// A contiguous tensor of n0 (x n1, where that is >= 0) elements; None: NULL.
template <class T>
T* own(PyObject* o, int64_t index, at::ScalarType type, const char* type_name, int64_t n0,
       int64_t n1, const char* name, bool required = false) {
  if (o == Py_None && !required) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const bool shape = n1 < 0 ? t.dim() == 1 && t.size(0) == n0
                            : t.dim() == 2 && t.size(0) == n0 && t.size(1) == n1;
  if (t.scalar_type() != type || !shape || !t.is_contiguous()) {
    if (n1 < 0)
      value_error("%s must be a contiguous %s tensor of shape [%lld]", name, type_name,
                  static_cast<long long>(n0));
    value_error("%s must be a contiguous %s tensor of shape [%lld, %lld]", name, type_name,
                static_cast<long long>(n0), static_cast<long long>(n1));
  }
  on_device(t, index, name);
  return static_cast<T*>(t.data_ptr());
}
int32_t* own_i32(PyObject* o, int64_t index, int64_t n0, int64_t n1, const char* name,
                 bool required = false) {
  return own<int32_t>(o, index, at::kInt, "torch.int32", n0, n1, name, required);
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
template <class T>
T* address(PyObject* o) {
  return o == Py_None ? nullptr : reinterpret_cast<T*>(number(o));
}

int32_t count(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error("%s has too many tokens", name);
  return static_cast<int32_t>(n);
}

// A call's body, with its arguments counted; exceptions end here.
template <class Body>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, Body body) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr long kNeedsWorkspace = -1;

// device, heads, kv_heads, d, scale, most tokens, most sequences, most keys, q, k, v,
// cu_q, cu_k, out, lse, workspace, its bytes, status word, stream
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 19, [&]() -> long {
    const int64_t index = number(a[0]), heads = number(a[1]), kv = number(a[2]), d = number(a[3]);
    const double scale = PyFloat_AsDouble(a[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
    const Rows q = rows(a[8], index, heads, d, d, "q"), k = rows(a[9], index, kv, d, d, "k"),
               v = rows(a[10], index, kv, d, d, "v");
    if (v.tokens != k.tokens) value_error("k and v must have the same number of tokens");
    const int64_t ends = tensor(a[11], "cu_q").numel();
    if (ends < 2) value_error("cu_q must be [batch + 1]");
    const int32_t* cu_q = own_i32(a[11], index, ends, -1, "cu_q", true);
    const int32_t* cu_k = a[12] == Py_None ? cu_q : own_i32(a[12], index, ends, -1, "cu_k");
    const Rows o = rows(a[13], index, heads, d, d, "out");
    if (o.tokens != q.tokens) value_error("out must have q's shape");
    float* lse = own<float>(a[14], index, at::kFloat, "torch.float32", q.tokens, heads, "lse");
    if (q.tokens > number(a[5]) || ends - 1 > number(a[6]) || k.tokens > number(a[7]))
      return kNeedsWorkspace;
    sa_packed_shape s;
    s.q_stride_t = q.strides[0];
    s.q_stride_h = q.strides[1];
    s.k_stride_t = k.strides[0];
    s.k_stride_h = k.strides[1];
    s.v_stride_t = v.strides[0];
    s.v_stride_h = v.strides[1];
    s.o_stride_t = o.strides[0];
    s.o_stride_h = o.strides[1];
    s.total_q = count(q.tokens, "q");
    s.total_k = count(k.tokens, "k");
    s.batch = count(ends - 1, "cu_q");
    s.num_q_heads = int32_t(heads);
    s.num_kv_heads = int32_t(kv);
    s.head_dim = int32_t(d);
    s.scale = float(scale);
    return sparse_attn_packed_forward(&s, q.at, k.at, v.at, cu_q, cu_k, o.at, lse,
                                      address<void>(a[15]), size_t(number(a[16])),
                                      address<int32_t>(a[17]), address<CUstream_st>(a[18]));
  });
}

// Heads of a [tokens, heads, d] tensor, whose other checks follow.
int64_t heads_of(PyObject* o, int64_t d, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3)
    value_error("%s must be [tokens, heads, %lld]", name, static_cast<long long>(d));
  return t.size(1);
}

// descriptor, device, d, q, k, positions, q_out, k_out, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&]() -> long {
    const int64_t index = number(a[1]), d = number(a[2]);
    const int64_t hq = heads_of(a[3], d, "q"), hkv = heads_of(a[4], d, "k");
    const Rows q = rows(a[3], index, hq, d, 0, "q"), k = rows(a[4], index, hkv, d, 0, "k"),
               qo = rows(a[6], index, hq, d, d, "q_out"),
               ko = rows(a[7], index, hkv, d, d, "k_out");
    if (k.tokens != q.tokens) value_error("q and k must have the same number of tokens");
    if (qo.tokens != q.tokens || ko.tokens != q.tokens)
      value_error("q_out and k_out must have the shapes of q and k");
    const int32_t* positions = own_i32(a[5], index, q.tokens, -1, "positions", true);
    return sparse_attn_rotary(address<sa_rotary>(a[0]), count(q.tokens, "q"), count(hq, "q"),
                              count(hkv, "k"), positions, q.at, q.strides, k.at, k.strides, qo.at,
                              qo.strides, ko.at, ko.strides, address<CUstream_st>(a[8]));
  });
}

// descriptor, device, d, kv_heads, q, k, v, positions, cache descriptor, slots, q_out,
// k_out, status word, stream
PyObject* rotary_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 14, [&]() -> long {
    const int64_t index = number(a[1]), d = number(a[2]), hkv = number(a[3]);
    const int64_t hq = heads_of(a[4], d, "q");
    const Rows q = rows(a[4], index, hq, d, 0, "q"), k = rows(a[5], index, hkv, d, 0, "k"),
               v = rows(a[6], index, hkv, d, 0, "v"), qo = rows(a[10], index, hq, d, d, "q_out");
    if (k.tokens != q.tokens || v.tokens != q.tokens)
      value_error("q, k and v must have the same number of tokens");
    Rows ko;
    if (a[11] != Py_None) ko = rows(a[11], index, hkv, d, d, "k_out");
    if (qo.tokens != q.tokens || (a[11] != Py_None && ko.tokens != q.tokens))
      value_error("q_out and k_out must have the shapes of q and k");
    const int32_t* positions = own_i32(a[7], index, q.tokens, -1, "positions", true);
    const int64_t* slots =
        own<int64_t>(a[9], index, at::kLong, "torch.int64", hkv, q.tokens, "slots", true);
    return sparse_attn_rotary_store(
        address<sa_rotary>(a[0]), count(q.tokens, "q"), count(hq, "q"), positions, q.at,
        q.strides, k.at, k.strides, v.at, v.strides, qo.at, qo.strides, ko.at,
        a[11] == Py_None ? nullptr : ko.strides, address<sa_paged_cache>(a[8]), slots,
        address<int32_t>(a[12]), address<CUstream_st>(a[13]));
  });
}

// descriptor, device, slots, cu, counts, ended, start, positions, granted, lens_out,
// owned_out, free_count_out, start_out, workspace, its bytes, status word, stream
PyObject* grow(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 17, [&]() -> long {
    const sa_page_pool* pool = address<sa_page_pool>(a[0]);
    const int64_t index = number(a[1]), b = pool->batch, h = pool->num_kv_heads;
    const at::Tensor& slots = tensor(a[2], "slots");
    if (slots.dim() != 2) value_error("slots must be [num_kv_heads, tokens]");
    const int64_t tokens = slots.size(1);
    if (a[3] == Py_None && tokens % b)
      value_error("without cu, tokens must be a multiple of the batch");
    sa_page_growth g;
    g.slots = own<int64_t>(a[2], index, at::kLong, "torch.int64", h, tokens, "slots", true);
    g.cu = own_i32(a[3], index, b + 1, -1, "cu");
    g.counts = own_i32(a[4], index, b, -1, "counts");
    g.ended = own<uint8_t>(a[5], index, at::kBool, "torch.bool", b, -1, "ended");
    int32_t* start = own_i32(a[6], index, b, -1, "start");
    g.start = start;
    g.token_positions = own_i32(a[7], index, tokens, -1, "positions");
    g.granted = own_i32(a[8], index, b, -1, "granted");
    g.lens_out = a[9] == Py_None ? pool->lens : own_i32(a[9], index, b, h, "lens_out");
    g.owned_out = a[10] == Py_None ? pool->owned : own_i32(a[10], index, b, h, "owned_out");
    g.free_count_out =
        a[11] == Py_None ? pool->free_count : own_i32(a[11], index, 1, -1, "free_count_out");
    g.start_out = a[12] == Py_None ? start : own_i32(a[12], index, b, -1, "start_out");
    g.tokens = count(tokens, "slots");
    return sparse_attn_paged_grow(pool, &g, address<void>(a[13]), size_t(number(a[14])),
                                  address<int32_t>(a[15]), address<CUstream_st>(a[16]));
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"packed", fast<packed>(), METH_FASTCALL, nullptr},
    {"rotary", fast<rotary>(), METH_FASTCALL, nullptr},
    {"rotary_store", fast<rotary_store>(), METH_FASTCALL, nullptr},
    {"grow", fast<grow>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
