// torch_calls.cpp -- the tensor calls of binding.py for the operators of a
// decode step: checks of the arguments and the C call, for loops whose time is
// the host's (a 4 x 4096 rmsnorm takes the host 4.0 us, in Python over ctypes
// 6.7).  torch is used for what a tensor is -- device, format, shape,
// strides and address -- and for nothing else.
//
// Every function takes the current device's index and the stream, then the
// tensors (None where one is left out), raises ValueError for a tensor that
// does not fit, and returns the library's status, or minus the bytes of the
// workspace that the call needs and that is None.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "../include/gemm_epi_decode.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* name, const std::string& what) {
  PyErr_SetString(PyExc_ValueError, (std::string(name) + ": " + what).c_str());
  throw Refused{};
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  return THPVariable_Unpack(o);
}

// A CUDA tensor of this format and shape on device `index`.
const at::Tensor& fitting(const char* name, PyObject* o, at::ScalarType format, at::IntArrayRef shape, int index) {
  const at::Tensor& t = tensor(name, o);
  if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
  if (t.get_device() != index)
    refuse(name, "on device " + std::to_string(t.get_device()) + ", the current device is " + std::to_string(index));
  if (t.scalar_type() != format)
    refuse(name, std::string("format ") + c10::toString(t.scalar_type()) + ", expected " + c10::toString(format));
  if (t.sizes() != shape) refuse(name, "shape " + text(t.sizes()) + ", expected " + text(shape));
  return t;
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;  // elements between the rows
};

// Rows that may lie apart, packed in themselves; None: no tensor, if allowed.
Rows rows(const char* name, PyObject* o, at::ScalarType format, at::IntArrayRef shape, int index, bool optional = false) {
  if (optional && o == Py_None) return {};
  const at::Tensor& t = fitting(name, o, format, shape, index);
  int64_t row = 1;
  for (size_t d = shape.size() - 1; d > 0; --d) {
    if (shape[d] != 1 && t.stride(d) != row) refuse(name, "only the first axis may be strided");
    row *= shape[d];
  }
  return {t.data_ptr(), shape[0] != 1 ? t.stride(0) : row};  // (one row has no distance to a next one)
}

void* packed(const char* name, PyObject* o, at::ScalarType format, at::IntArrayRef shape, int index, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = fitting(name, o, format, shape, index);
  if (!t.is_contiguous()) refuse(name, "expected a contiguous tensor");
  return t.data_ptr();
}

// A tensor of `dims` axes in a 16-bit format, and the library's name of that.
const at::Tensor& half(const char* name, PyObject* o, int dims, const char* axes, gemm_epi_dtype& format) {
  const at::Tensor& t = tensor(name, o);
  if (t.dim() != dims) refuse(name, std::string("expected axes ") + axes);
  if (t.scalar_type() == at::kHalf) format = GEMM_EPI_F16;
  else if (t.scalar_type() == at::kBFloat16) format = GEMM_EPI_BF16;
  else refuse(name, std::string("format ") + c10::toString(t.scalar_type()) + "; expected float16 or bfloat16");
  return t;
}

struct Space {
  void* p;
  size_t bytes;
};
Space workspace(PyObject* o, int index) {
  const at::Tensor& t = tensor("workspace", o);
  if (!t.is_cuda() || t.get_device() != index || !t.is_contiguous())
    refuse("workspace", "expected a contiguous CUDA tensor on device " + std::to_string(index));
  return {t.data_ptr(), t.nbytes()};
}

gemm_epi_page_table page_table(PyObject* pages, PyObject* lens, int index, int cache_index) {
  if (index != cache_index)
    refuse("cache", "on device " + std::to_string(cache_index) + ", the current device is " + std::to_string(index));
  const at::Tensor& t = tensor("pages", pages);
  if (t.dim() != 2) refuse("pages", "expected axes [batch, width]");
  gemm_epi_page_table table;
  const int64_t shape[2] = {t.size(0), t.size(1)};
  const Rows r = rows("pages", pages, at::kInt, shape, index);
  table.pages = (const int32_t*)r.p;
  table.ld = r.ld;
  table.width = shape[1];
  table.lens = (const int32_t*)packed("lens", lens, at::kInt, {shape[0]}, index);
  table.batch = shape[0];
  return table;
}

template <typename F>
gemm_epi_status unlocked(F&& call) {
  gemm_epi_status s;
  Py_BEGIN_ALLOW_THREADS;
  s = call();
  Py_END_ALLOW_THREADS;
  return s;
}

// The arguments' count, the device index and the stream; then the call.
template <int N, typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, F&& f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  const int index = (int)PyLong_AsLong(a[0]);
  void* stream = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return nullptr;
  try {
    return PyLong_FromLongLong(f(index, stream));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// index, stream, x, weight, y, residual, residual_out, y_scale, eps
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(a, n, [&](int index, void* stream) -> long long {
    gemm_epi_dtype format, out;
    const at::Tensor& x = half("x", a[2], 2, "[rows, cols]", format);
    const at::ScalarType st = x.scalar_type();
    const int64_t shape[2] = {x.size(0), x.size(1)};
    const Rows rx = rows("x", a[2], st, shape, index);
    const void* w = packed("weight", a[3], st, {shape[1]}, index);
    const Rows rr = rows("residual", a[5], st, shape, index, true);
    const Rows rh = rows("residual_out", a[6], st, shape, index, true);
    const bool fp8 = a[7] != Py_None;
    float* scale = (float*)packed("y_scale", a[7], at::kFloat, {shape[0]}, index, true);
    const Rows ry = rows("y", a[4], fp8 ? at::kFloat8_e4m3fn : st, shape, index);
    out = fp8 ? GEMM_EPI_FP8_E4M3 : format;
    const double eps = PyFloat_AsDouble(a[8]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{};
    if (shape[0] == 0) return GEMM_EPI_OK;
    return unlocked([&] {
      return gemm_epi_rmsnorm(rx.p, rx.ld, rr.p, rr.ld, w, rh.p, rh.ld, ry.p, ry.ld, scale, shape[0], shape[1],
                              (float)eps, format, out, stream);
    });
  });
}

// index, stream, x, a, b, ids, c, scale, residual, workspace
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>(a, n, [&](int index, void* stream) -> long long {
    gemm_epi_dtype format, other;
    const at::Tensor& x = half("x", a[2], 2, "[M, K]", format);
    const at::ScalarType st = x.scalar_type();
    const at::Tensor& A = half("a", a[3], 3, "[adapters, rank, K]", other);
    const at::Tensor& B = half("b", a[4], 3, "[adapters, N, rank]", other);
    const int64_t M = x.size(0), K = x.size(1), adapters = A.size(0), rank = A.size(1), N = B.size(1);
    const Rows rx = rows("x", a[2], st, {M, K}, index);
    const void* pa = packed("a", a[3], st, {adapters, rank, K}, index);
    const void* pb = packed("b", a[4], st, {adapters, N, rank}, index);
    const int32_t* ids = (const int32_t*)packed("ids", a[5], at::kInt, {M}, index);
    const Rows rc = rows("c", a[6], st, {M, N}, index);
    const float* scale = (const float*)packed("scale", a[7], at::kFloat, {adapters}, index, true);
    const Rows rr = rows("residual", a[8], st, {M, N}, index, true);
    if (M == 0) return GEMM_EPI_OK;
    Space ws{nullptr, 0};
    if (a[9] != Py_None) ws = workspace(a[9], index);
    else if (const size_t need = gemm_epi_lora_workspace_size(M, N, K, rank, adapters)) return -(long long)need;
    return unlocked([&] {
      return gemm_epi_lora(rx.p, rx.ld, pa, pb, scale, ids, rr.p, rr.ld, rc.p, rc.ld, M, N, K, rank, adapters, format,
                           ws.p, ws.bytes, stream);
    });
  });
}

const gemm_epi_paged_cache* cache_at(PyObject* address) {
  const void* p = PyLong_AsVoidPtr(address);
  if (!p) throw Refused{};
  return (const gemm_epi_paged_cache*)p;
}

// index, stream, the cache's struct, its device, k, v, pages, lens, starts
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(a, n, [&](int index, void* stream) -> long long {
    const gemm_epi_paged_cache* cache = cache_at(a[2]);
    const gemm_epi_page_table table = page_table(a[6], a[7], index, (int)PyLong_AsLong(a[3]));
    gemm_epi_dtype format;
    const at::Tensor& k = half("k", a[4], 3, "[tokens, heads, head_dim]", format);
    const int64_t shape[3] = {k.size(0), cache->heads, cache->head_dim};
    const Rows rk = rows("k", a[4], k.scalar_type(), shape, index), rv = rows("v", a[5], k.scalar_type(), shape, index);
    const int32_t* starts = (const int32_t*)packed("starts", a[8], at::kInt, {table.batch + 1}, index, true);
    return unlocked([&] {
      return gemm_epi_cache_append(cache, &table, rk.p, rk.ld, rv.p, rv.ld, starts, shape[0], format, stream);
    });
  });
}

// index, stream, the cache's struct, its device, q, o, pages, lens, workspace
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<9>(a, n, [&](int index, void* stream) -> long long {
    const gemm_epi_paged_cache* cache = cache_at(a[2]);
    const gemm_epi_page_table table = page_table(a[6], a[7], index, (int)PyLong_AsLong(a[3]));
    gemm_epi_dtype format;
    const at::Tensor& q = half("q", a[4], 3, "[batch, q_heads, head_dim]", format);
    const int64_t shape[3] = {table.batch, q.size(1), cache->head_dim};
    const Rows rq = rows("q", a[4], q.scalar_type(), shape, index), ro = rows("o", a[5], q.scalar_type(), shape, index);
    if (table.batch == 0) return GEMM_EPI_OK;
    Space ws{nullptr, 0};
    if (a[8] != Py_None) ws = workspace(a[8], index);
    else if (const size_t need = gemm_epi_attention_decode_workspace_size(cache, table.batch, table.width, shape[1]))
      return -(long long)need;
    return unlocked([&] {
      return gemm_epi_attention_decode(cache, &table, rq.p, rq.ld, ro.p, ro.ld, shape[1], format, ws.p, ws.bytes, stream);
    });
  });
}

PyMethodDef methods[] = {
    {"rmsnorm", (PyCFunction)(void (*)(void))rmsnorm, METH_FASTCALL, nullptr},
    {"lora", (PyCFunction)(void (*)(void))lora, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
