// torch_calls.cpp -- the calls of qlin.py whose kernels take less time at small
// batches than Python needs to call them, as a Python extension: it checks the
// tensors, allocates what the caller did not give and calls libqlin's entry
// points on the tensors' device and its current stream.
//
// A 1 x 5120 x 1024 product runs 3.7 us on the device; its call took 11.3 us as
// Python and ctypes and takes 3.4 from here (2.6 with y given), residual
// addition + RMSNorm + act-quant 14.8 and 6.0 (2.2 with its three outputs
// given).  The kernels stay in libqlin, which knows nothing of PyTorch; its
// functions' addresses are handed over by setup().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "qlin.h"

namespace {

decltype(&qlin_add_rmsnorm_act_quant_i8) add_rmsnorm_i8;
decltype(&qlin_add_rmsnorm_act_quant_c16) add_rmsnorm_c16;
decltype(&qlin_gemm_w8a8_ch) gemm_i8;
decltype(&qlin_gemm_w8a8_ch_c16) gemm_c16;
decltype(&qlin_gemm_w8a8_ch_workspace_bytes) gemm_workspace;
decltype(&qlin_adjust_logits_bf16) logits_bf16;
decltype(&qlin_adjust_logits_f32) logits_f32;
decltype(&qlin_kv_write_i8) write_i8;
decltype(&qlin_kv_read_bf16) read_bf16;
decltype(&qlin_paged_attn_i8) attn_i8;
decltype(&qlin_paged_attn_workspace_bytes) attn_workspace;
PyObject* raise_status;   // raises the error of a status

using at::ScalarType;
using at::Tensor;

const char* dtype_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Char: return "torch.int8";
    case ScalarType::Byte: return "torch.uint8";
    default: return "torch.int32";
  }
}

bool is_none(PyObject* o) { return o == Py_None; }

void refuse_dtype(PyObject* o, const char* name, const char* wanted) {
  PyObject* got = PyObject_GetAttrString(o, "dtype");
  if (got == nullptr) return;
  PyErr_Format(PyExc_TypeError, "%s must be %s, got %S", name, wanted, got);
  Py_DECREF(got);
}

// Raises what is wrong with a tensor that tensor() turned down.
void refuse(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, int index) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return;
  }
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) {
    refuse_dtype(o, name, dtype_name(type));
  } else if (t.sizes() != shape) {
    PyObject* got = PyObject_GetAttrString(o, "shape");
    if (got == nullptr) return;
    auto n = [&](size_t i) { return static_cast<long long>(shape[i]); };
    if (shape.size() == 1)
      PyErr_Format(PyExc_ValueError, "%s must have shape [%lld], got %S", name, n(0), got);
    else if (shape.size() == 2)
      PyErr_Format(PyExc_ValueError, "%s must have shape [%lld, %lld], got %S", name, n(0), n(1), got);
    else
      PyErr_Format(PyExc_ValueError, "%s must have shape [%lld, %lld, %lld, %lld], got %S", name, n(0), n(1), n(2), n(3), got);
    Py_DECREF(got);
  } else if (!t.is_cuda() || t.get_device() != index) {
    PyErr_Format(PyExc_ValueError, "%s must be on cuda:%d, got %s", name, index, t.device().str().c_str());
  } else {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  }
}

// The tensor if it is as the call needs it, else nullptr with an error raised.
const Tensor* tensor(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, int index) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.sizes() == shape && t.is_cuda() && t.get_device() == index && t.is_contiguous())
      return &t;
  }
  refuse(o, name, type, shape, index);
  return nullptr;
}

// The argument that the others' shapes follow from.
const Tensor* lead(PyObject* o, const char* name, std::initializer_list<ScalarType> types, int64_t dims) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return nullptr;
  }
  const Tensor& t = THPVariable_Unpack(o);
  bool known = false;
  for (const ScalarType type : types) known = known || t.scalar_type() == type;
  if (!known) {
    refuse_dtype(o, name, types.size() > 1 ? "torch.bfloat16 or torch.float32" : dtype_name(*types.begin()));
  } else if (t.dim() != dims) {
    PyErr_Format(PyExc_ValueError, "%s must have %lld dimensions, got %lld", name, static_cast<long long>(dims),
                 static_cast<long long>(t.dim()));
  } else if (!t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
  } else if (!t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  } else {
    return &t;
  }
  return nullptr;
}

Tensor fresh(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

// An output: the one given, else a new one; false with an error raised.
bool output(Tensor& to, PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape, const Tensor& like) {
  if (is_none(o)) {
    to = fresh(shape, type, like);
    return true;
  }
  const Tensor* t = tensor(o, name, type, shape, like.get_device());
  if (t == nullptr) return false;
  to = *t;
  return true;
}

template <typename T>
T* out(const Tensor& t) {
  return static_cast<T*>(t.mutable_data_ptr());
}
template <typename T>
const T* in(const Tensor& t) {
  return static_cast<const T*>(t.const_data_ptr());
}

qlin_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<qlin_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

// Other Python threads run while a launch waits for room in the queue.
struct WithoutGil {
  PyThreadState* const state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

template <typename F, typename... Args>
qlin_status_t call(F entry, Args... args) {
  const WithoutGil gil;
  return entry(args...);
}

// True if the status is good, else its error is raised.
bool done(qlin_status_t status) {
  if (status == QLIN_OK) return true;
  PyObject* r = PyObject_CallFunction(raise_status, "i", static_cast<int>(status));
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, "qlin call failed");
  return false;
}

bool count(Py_ssize_t n, Py_ssize_t wanted) {
  if (n == wanted) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, n);
  return false;
}

// (c16, x, residual, gamma, eps, residual_out, q, s_a, y) -> (q, s_a, residual_out)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 9)) return nullptr;
  const bool c16 = a[0] == Py_True;
  const Tensor* x = lead(a[1], "x", {ScalarType::BFloat16}, 2);
  if (x == nullptr) return nullptr;
  const int64_t M = x->size(0), K = x->size(1);
  const int index = x->get_device();
  const Tensor* residual = tensor(a[2], "residual", ScalarType::BFloat16, {M, K}, index);
  if (residual == nullptr) return nullptr;
  const Tensor* gamma = tensor(a[3], "gamma", ScalarType::BFloat16, {K}, index);
  if (gamma == nullptr) return nullptr;
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  Tensor h, q, s_a;
  if (!output(h, a[5], "residual_out", ScalarType::BFloat16, {M, K}, *x) ||
      !output(q, a[6], "q", c16 ? ScalarType::Half : ScalarType::Char, {M, K}, *x) ||
      !output(s_a, a[7], "s_a", ScalarType::Float, {M}, *x))
    return nullptr;
  const Tensor* y = is_none(a[8]) ? nullptr : tensor(a[8], "y", ScalarType::BFloat16, {M, K}, index);
  if (y == nullptr && !is_none(a[8])) return nullptr;
  const c10::cuda::CUDAGuard guard(x->device());
  uint16_t* const yp = y == nullptr ? nullptr : out<uint16_t>(*y);
  const float e = static_cast<float>(eps);
  const qlin_status_t status =
      c16 ? call(add_rmsnorm_c16, in<uint16_t>(*x), in<uint16_t>(*residual), in<uint16_t>(*gamma), e, M, K, out<uint16_t>(h),
                            out<uint16_t>(q), out<float>(s_a), yp, stream_of(*x))
          : call(add_rmsnorm_i8, in<uint16_t>(*x), in<uint16_t>(*residual), in<uint16_t>(*gamma), e, M, K, out<uint16_t>(h),
                           out<int8_t>(q), out<float>(s_a), yp, stream_of(*x));
  if (!done(status)) return nullptr;
  PyObject* result = PyTuple_New(3);
  if (result == nullptr) return nullptr;
  const Tensor* const parts[3] = {&q, &s_a, &h};
  for (int i = 0; i < 3; ++i) {
    PyObject* const part = THPVariable_Wrap(*parts[i]);
    if (part == nullptr) {
      Py_DECREF(result);
      return nullptr;
    }
    PyTuple_SET_ITEM(result, i, part);
  }
  return result;
  END_HANDLE_TH_ERRORS
}

// (c16, q_a, s_a, qweight, s_w, y, workspace) -> y
PyObject* gemm_ch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const bool c16 = a[0] == Py_True;
  const Tensor* q = lead(a[1], "q_a", {c16 ? ScalarType::Half : ScalarType::Char}, 2);
  if (q == nullptr) return nullptr;
  const Tensor* w = lead(a[3], "qweight", {ScalarType::Int}, 2);
  if (w == nullptr) return nullptr;
  const int64_t M = q->size(0), K = q->size(1), N = w->size(1);
  const int index = q->get_device();
  if (K % 4 != 0) {
    PyErr_SetString(PyExc_ValueError, "K must be a multiple of 128");
    return nullptr;
  }
  if (tensor(a[3], "qweight", ScalarType::Int, {K / 4, N}, index) == nullptr) return nullptr;
  const Tensor* s_a = tensor(a[2], "s_a", ScalarType::Float, {M}, index);
  if (s_a == nullptr) return nullptr;
  const Tensor* s_w = tensor(a[4], "s_w", ScalarType::Float, {N}, index);
  if (s_w == nullptr) return nullptr;
  Tensor y, workspace;
  if (!output(y, a[5], "y", ScalarType::BFloat16, {M, N}, *q)) return nullptr;
  const c10::cuda::CUDAGuard guard(q->device());
  if (!is_none(a[6])) {
    const Tensor* given = lead(a[6], "workspace", {ScalarType::Byte}, 1);
    if (given == nullptr || tensor(a[6], "workspace", ScalarType::Byte, given->sizes(), index) == nullptr)
      return nullptr;
    workspace = *given;
  } else if (M > 8) {            // up to 8 rows never need one
    // its own for every call: calls on several streams, or replayed graphs, do
    // not meet in it
    const int64_t bytes = static_cast<int64_t>(gemm_workspace(M, N, K, c16 ? 1 : 0));
    if (bytes > 0) workspace = fresh({bytes}, ScalarType::Byte, *q);
  }
  void* const ws = workspace.defined() ? out<void>(workspace) : nullptr;
  const size_t bytes = workspace.defined() ? static_cast<size_t>(workspace.size(0)) : 0;
  const qlin_status_t status =
      c16 ? call(gemm_c16, in<uint16_t>(*q), in<float>(*s_a), in<int32_t>(*w), in<float>(*s_w), M, N, K, out<uint16_t>(y), ws,
                     bytes, stream_of(*q))
          : call(gemm_i8, in<int8_t>(*q), in<float>(*s_a), in<int32_t>(*w), in<float>(*s_w), M, N, K, out<uint16_t>(y), ws,
                    bytes, stream_of(*q));
  if (!done(status)) return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (greedy, logits, tokens, prompt_len, total_len, repetition, presence, frequency, bias_ids, bias, allowed, out,
// argmax) -> argmax if greedy, else out
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 13)) return nullptr;
  const bool greedy = a[0] == Py_True;
  const Tensor* x = lead(a[1], "logits", {ScalarType::BFloat16, ScalarType::Float}, 2);
  if (x == nullptr) return nullptr;
  const int64_t M = x->size(0), V = x->size(1);
  const int index = x->get_device();
  int64_t L = 0, B = 0;
  const int32_t *tokens = nullptr, *prompt = nullptr, *total = nullptr, *ids = nullptr, *allowed = nullptr;
  const float *repetition = nullptr, *presence = nullptr, *frequency = nullptr, *bias = nullptr;
  auto ints = [&](const int32_t*& to, PyObject* o, const char* name, at::IntArrayRef shape) {
    if (is_none(o)) return true;
    const Tensor* t = tensor(o, name, ScalarType::Int, shape, index);
    if (t == nullptr) return false;
    to = in<int32_t>(*t);
    return true;
  };
  auto floats = [&](const float*& to, PyObject* o, const char* name, at::IntArrayRef shape) {
    if (is_none(o)) return true;
    const Tensor* t = tensor(o, name, ScalarType::Float, shape, index);
    if (t == nullptr) return false;
    to = in<float>(*t);
    return true;
  };
  if (!is_none(a[2])) {
    const Tensor* t = lead(a[2], "tokens", {ScalarType::Int}, 2);
    if (t == nullptr) return nullptr;
    L = t->size(1);
    if (!ints(tokens, a[2], "tokens", {M, L}) || !ints(prompt, a[3], "prompt_len", {M}) ||
        !ints(total, a[4], "total_len", {M}))
      return nullptr;
  } else if (!is_none(a[3]) || !is_none(a[4])) {
    PyErr_SetString(PyExc_ValueError, "prompt_len and total_len need tokens");
    return nullptr;
  }
  if (is_none(a[8]) != is_none(a[9])) {
    PyErr_SetString(PyExc_ValueError, "bias_ids and bias go together");
    return nullptr;
  }
  if (!is_none(a[8])) {
    const Tensor* t = lead(a[8], "bias_ids", {ScalarType::Int}, 2);
    if (t == nullptr) return nullptr;
    B = t->size(1);
    if (!ints(ids, a[8], "bias_ids", {M, B}) || !floats(bias, a[9], "bias", {M, B})) return nullptr;
  }
  if (!floats(repetition, a[5], "repetition", {M}) || !floats(presence, a[6], "presence", {M}) ||
      !floats(frequency, a[7], "frequency", {M}) || !ints(allowed, a[10], "allowed", {M, (V + 31) / 32}))
    return nullptr;
  Tensor to, best;
  if (!greedy || !is_none(a[11])) {
    if (!output(to, a[11], "out", x->scalar_type(), {M, V}, *x)) return nullptr;
  }
  if (greedy) {
    if (!output(best, a[12], "argmax", ScalarType::Int, {M}, *x)) return nullptr;
  }
  const c10::cuda::CUDAGuard guard(x->device());
  int32_t* const argmax = greedy ? out<int32_t>(best) : nullptr;
  const qlin_status_t status =
      x->scalar_type() == ScalarType::BFloat16
          ? call(logits_bf16, in<uint16_t>(*x), M, V, tokens, L, prompt, total, repetition, presence, frequency, ids, bias, B,
                        allowed, to.defined() ? out<uint16_t>(to) : nullptr, argmax, stream_of(*x))
          : call(logits_f32, in<float>(*x), M, V, tokens, L, prompt, total, repetition, presence, frequency, ids, bias, B,
                       allowed, to.defined() ? out<float>(to) : nullptr, argmax, stream_of(*x));
  if (!done(status)) return nullptr;
  return THPVariable_Wrap(greedy ? best : to);
  END_HANDLE_TH_ERRORS
}

constexpr int64_t kCacheBlock = 4224;   // bytes of 16 tokens of a head

// What the calls on a paged cache share: the cache and its sequences.
struct Cache {
  void* data;
  int64_t pages, kv_heads, page_size, B, max_pages;
  const int32_t *table, *total, *fresh;
};

// false with an error raised
bool cache_of(Cache& c, PyObject* cache, PyObject* table, PyObject* total, PyObject* fresh, int index) {
  const Tensor* t = lead(cache, "cache", {ScalarType::Byte}, 4);
  if (t == nullptr) return false;
  c.pages = t->size(0);
  c.kv_heads = t->size(1);
  c.page_size = 16 * t->size(2);
  if (tensor(cache, "cache", ScalarType::Byte, {c.pages, c.kv_heads, t->size(2), kCacheBlock}, index) == nullptr) return false;
  c.data = out<void>(*t);
  const Tensor* pages = lead(table, "block_table", {ScalarType::Int}, 2);
  if (pages == nullptr || tensor(table, "block_table", ScalarType::Int, pages->sizes(), index) == nullptr) return false;
  c.B = pages->size(0);
  c.max_pages = pages->size(1);
  c.table = in<int32_t>(*pages);
  const Tensor* n = tensor(total, "total_len", ScalarType::Int, {c.B}, index);
  if (n == nullptr) return false;
  c.total = in<int32_t>(*n);
  c.fresh = nullptr;
  if (!is_none(fresh)) {
    n = tensor(fresh, "new_len", ScalarType::Int, {c.B}, index);
    if (n == nullptr) return false;
    c.fresh = in<int32_t>(*n);
  }
  return true;
}

bool whole(PyObject* o, int64_t& to) {
  to = PyLong_AsLongLong(o);
  return to != -1 || !PyErr_Occurred();
}

bool real(PyObject* o, float& to) {
  const double d = PyFloat_AsDouble(o);
  to = static_cast<float>(d);
  return d != -1.0 || !PyErr_Occurred();
}

// Rows of each sequence: M / B.
bool rows_of(int64_t M, int64_t B, const char* name, int64_t& T) {
  T = B == 0 ? 0 : M / B;
  if (M == B * T) return true;
  PyErr_Format(PyExc_ValueError, "%s must have a multiple of %lld rows, got %lld", name, static_cast<long long>(B),
               static_cast<long long>(M));
  return false;
}

// (qkv, cache, block_table, total_len, q_heads, new_len, q_gamma, k_gamma, eps, cos_sin, positions, axes, q) -> q
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 13)) return nullptr;
  const Tensor* x = lead(a[0], "qkv", {ScalarType::BFloat16}, 2);
  if (x == nullptr) return nullptr;
  const int64_t M = x->size(0);
  const int index = x->get_device();
  Cache c;
  int64_t T, q_heads, P = 0, R = 0, A = 0;
  float eps;
  if (!cache_of(c, a[1], a[2], a[3], a[5], index) || !rows_of(M, c.B, "qkv", T) || !whole(a[4], q_heads) || !real(a[8], eps))
    return nullptr;
  if (q_heads < 0 || x->size(1) != (q_heads + 2 * c.kv_heads) * 128) {
    PyErr_Format(PyExc_ValueError, "qkv must have (q_heads + 2 * %lld) * 128 columns, got %lld", static_cast<long long>(c.kv_heads),
                 static_cast<long long>(x->size(1)));
    return nullptr;
  }
  const Tensor *q_gamma = nullptr, *k_gamma = nullptr, *table = nullptr, *positions = nullptr, *axes = nullptr;
  if (!is_none(a[6]) && (q_gamma = tensor(a[6], "q_gamma", ScalarType::BFloat16, {128}, index)) == nullptr) return nullptr;
  if (!is_none(a[7]) && (k_gamma = tensor(a[7], "k_gamma", ScalarType::BFloat16, {128}, index)) == nullptr) return nullptr;
  if (!is_none(a[9])) {
    table = lead(a[9], "cos_sin", {ScalarType::Float}, 2);
    if (table == nullptr || tensor(a[9], "cos_sin", ScalarType::Float, table->sizes(), index) == nullptr) return nullptr;
    P = table->size(0);
    R = table->size(1);
    if (P == 0 || R == 0) {
      PyErr_SetString(PyExc_ValueError, "cos_sin must not be empty");
      return nullptr;
    }
  } else if (!is_none(a[10]) || !is_none(a[11])) {
    PyErr_SetString(PyExc_ValueError, "positions and axes need cos_sin");
    return nullptr;
  }
  if (!is_none(a[10])) {
    positions = lead(a[10], "positions", {ScalarType::Int}, 2);
    if (positions == nullptr) return nullptr;
    A = positions->size(0);
    if (A == 0) {
      PyErr_SetString(PyExc_ValueError, "positions must have an axis");
      return nullptr;
    }
    if (tensor(a[10], "positions", ScalarType::Int, {A, M}, index) == nullptr) return nullptr;
  }
  if (!is_none(a[11])) {
    axes = tensor(a[11], "axes", ScalarType::Byte, {R / 2}, index);
    if (axes == nullptr) return nullptr;
  } else if (A > 1) {
    PyErr_SetString(PyExc_ValueError, "positions of several axes need axes");
    return nullptr;
  }
  Tensor q;
  if (!output(q, a[12], "q", ScalarType::BFloat16, {M, q_heads * 128}, *x)) return nullptr;
  const c10::cuda::CUDAGuard guard(x->device());
  const qlin_status_t status = call(
      write_i8, in<uint16_t>(*x), c.B, T, q_heads, c.kv_heads, q_gamma == nullptr ? nullptr : in<uint16_t>(*q_gamma),
      k_gamma == nullptr ? nullptr : in<uint16_t>(*k_gamma), eps, table == nullptr ? nullptr : in<float>(*table), P, R,
      positions == nullptr ? nullptr : in<int32_t>(*positions), A, axes == nullptr ? nullptr : in<uint8_t>(*axes), c.data,
      c.pages, c.page_size, c.table, c.max_pages, c.total, c.fresh, q_heads == 0 ? nullptr : out<uint16_t>(q), stream_of(*x));
  if (!done(status)) return nullptr;
  return THPVariable_Wrap(q);
  END_HANDLE_TH_ERRORS
}

// (cache, block_table, total_len, length, start, k, v) -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const Tensor* cache = lead(a[0], "cache", {ScalarType::Byte}, 4);
  if (cache == nullptr) return nullptr;
  const int index = cache->get_device();
  Cache c;
  int64_t L;
  if (!cache_of(c, a[0], a[1], a[2], Py_None, index) || !whole(a[3], L)) return nullptr;
  if (L < 0) {
    PyErr_SetString(PyExc_ValueError, "length must not be negative");
    return nullptr;
  }
  const Tensor* start = nullptr;
  if (!is_none(a[4]) && (start = tensor(a[4], "start", ScalarType::Int, {c.B}, index)) == nullptr) return nullptr;
  Tensor k, v;
  if (!output(k, a[5], "k", ScalarType::BFloat16, {c.B, L, c.kv_heads, 128}, *cache) ||
      !output(v, a[6], "v", ScalarType::BFloat16, {c.B, L, c.kv_heads, 128}, *cache))
    return nullptr;
  const c10::cuda::CUDAGuard guard(cache->device());
  const qlin_status_t status =
      call(read_bf16, static_cast<const void*>(c.data), c.pages, c.page_size, c.kv_heads, c.table, c.B, c.max_pages, c.total,
           start == nullptr ? nullptr : in<int32_t>(*start), L, out<uint16_t>(k), out<uint16_t>(v), stream_of(*cache));
  if (!done(status)) return nullptr;
  PyObject* result = PyTuple_New(2);
  if (result == nullptr) return nullptr;
  const Tensor* const parts[2] = {&k, &v};
  for (int i = 0; i < 2; ++i) {
    PyObject* const part = THPVariable_Wrap(*parts[i]);
    if (part == nullptr) {
      Py_DECREF(result);
      return nullptr;
    }
    PyTuple_SET_ITEM(result, i, part);
  }
  return result;
  END_HANDLE_TH_ERRORS
}

// (q, cache, block_table, total_len, new_len, scale, softcap, window, causal, out, workspace) -> out
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 11)) return nullptr;
  const Tensor* q = lead(a[0], "q", {ScalarType::BFloat16}, 2);
  if (q == nullptr) return nullptr;
  const int64_t M = q->size(0), width = q->size(1);
  const int index = q->get_device();
  Cache c;
  int64_t T, window;
  float scale = 0.08838834764831845f, softcap;   // 1 / sqrt(128)
  if (!cache_of(c, a[1], a[2], a[3], a[4], index) || !rows_of(M, c.B, "q", T) || (!is_none(a[5]) && !real(a[5], scale)) ||
      !real(a[6], softcap) || !whole(a[7], window))
    return nullptr;
  if (softcap == 0.0f && PyFloat_AsDouble(a[6]) != 0.0) {      // (0 would be no cap)
    PyErr_SetString(PyExc_ValueError, "softcap must be 0 or at least fp32's smallest number");
    return nullptr;
  }
  const int causal = PyObject_IsTrue(a[8]);
  if (causal < 0) return nullptr;
  if (width == 0 || c.kv_heads == 0 || width % (128 * c.kv_heads) != 0) {
    PyErr_Format(PyExc_ValueError, "q must have a multiple of %lld * 128 columns, got %lld", static_cast<long long>(c.kv_heads),
                 static_cast<long long>(width));
    return nullptr;
  }
  const int64_t q_heads = width / 128;
  Tensor to, workspace;
  if (!output(to, a[9], "out", ScalarType::BFloat16, {M, width}, *q)) return nullptr;
  const c10::cuda::CUDAGuard guard(q->device());
  if (!is_none(a[10])) {
    const Tensor* given = lead(a[10], "workspace", {ScalarType::Byte}, 1);
    if (given == nullptr || tensor(a[10], "workspace", ScalarType::Byte, given->sizes(), index) == nullptr) return nullptr;
    workspace = *given;
  } else {
    // its own for every call: calls on several streams, or replayed graphs, do
    // not meet in it
    const int64_t bytes = static_cast<int64_t>(attn_workspace(c.B, T, q_heads, c.kv_heads));
    if (bytes > 0) workspace = fresh({bytes}, ScalarType::Byte, *q);
  }
  const qlin_status_t status =
      call(attn_i8, in<uint16_t>(*q), c.B, T, q_heads, c.kv_heads, static_cast<const void*>(c.data), c.pages, c.page_size,
           c.table, c.max_pages, c.total, c.fresh, scale, softcap, window, causal, out<uint16_t>(to),
           workspace.defined() ? out<void>(workspace) : nullptr,
           workspace.defined() ? static_cast<size_t>(workspace.size(0)) : size_t{0}, stream_of(*q));
  if (!done(status)) return nullptr;
  return THPVariable_Wrap(to);
  END_HANDLE_TH_ERRORS
}

// (raise_status, addresses of the entry points in the order below)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  void* at[11];
  for (int i = 0; i < 11; ++i) {
    at[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  add_rmsnorm_i8 = reinterpret_cast<decltype(add_rmsnorm_i8)>(at[0]);
  add_rmsnorm_c16 = reinterpret_cast<decltype(add_rmsnorm_c16)>(at[1]);
  gemm_i8 = reinterpret_cast<decltype(gemm_i8)>(at[2]);
  gemm_c16 = reinterpret_cast<decltype(gemm_c16)>(at[3]);
  gemm_workspace = reinterpret_cast<decltype(gemm_workspace)>(at[4]);
  logits_bf16 = reinterpret_cast<decltype(logits_bf16)>(at[5]);
  logits_f32 = reinterpret_cast<decltype(logits_f32)>(at[6]);
  write_i8 = reinterpret_cast<decltype(write_i8)>(at[7]);
  read_bf16 = reinterpret_cast<decltype(read_bf16)>(at[8]);
  attn_i8 = reinterpret_cast<decltype(attn_i8)>(at[9]);
  attn_workspace = reinterpret_cast<decltype(attn_workspace)>(at[10]);
  Py_INCREF(a[0]);
  raise_status = a[0];
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"setup", fast(setup), METH_FASTCALL, nullptr},
                         {"add_rmsnorm", fast(add_rmsnorm), METH_FASTCALL, nullptr},
                         {"gemm_ch", fast(gemm_ch), METH_FASTCALL, nullptr},
                         {"adjust_logits", fast(adjust_logits), METH_FASTCALL, nullptr},
                         {"kv_write", fast(kv_write), METH_FASTCALL, nullptr},
                         {"kv_read", fast(kv_read), METH_FASTCALL, nullptr},
                         {"paged_attn", fast(paged_attn), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "qlin_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qlin_torch() { return PyModule_Create(&module); }
