// attn_binding.cpp -- the softmax-attention entry points as a Python extension.
//
// A serving step makes several of these calls for each token, and checking a
// dozen tensors and allocating the outputs in Python takes longer than the small
// calls' kernels do.  Here the tensors are looked at in place.  attention.py
// documents the functions and names their arguments; everything it passes is
// checked here before libkda is called.  A function returns what the Python
// function returns, or libkda's status as an int if that is not KDA_OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <string>

#include "kda.h"

namespace {

// A Python exception: its type and message.
struct Refused {
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(PyObject* type, std::string text) { throw Refused{type, std::move(text)}; }

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

template <class Sizes>
std::string shape_text(const Sizes& s) {
  std::string r = "(";
  size_t i = 0;
  for (int64_t x : s) r += (i++ ? ", " : "") + std::to_string(x);
  return r + (i == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor& sized(PyObject* o, const char* name, int64_t dims, const char* what) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims)
    refuse(PyExc_ValueError, std::string(name) + " must be " + what + ", got " + shape_text(t.sizes()));
  return t;
}

// Checks one argument and returns its address.
void* address(const at::Tensor& t, const char* name, at::ScalarType type,
              std::initializer_list<int64_t> shape, int64_t device) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on a CUDA device");
  if (t.get_device() != device)
    refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" +
                                 std::to_string(device));
  if (!t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())))
    refuse(PyExc_ValueError,
           std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

void* address(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
              int64_t device) {
  return address(tensor(o, name), name, type, shape, device);
}

void* optional(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
               int64_t device) {
  return o == Py_None ? nullptr : address(o, name, type, shape, device);
}

double number(PyObject* o, const char* name) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a number");
  }
  return x;
}

int32_t integer(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be an integer");
  }
  if (x < INT32_MIN || x > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(x);
}

bool truth(PyObject* o, const char* name) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be a truth value");
  }
  return x != 0;
}

int32_t size32(int64_t x, const char* name) {
  if (x > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(x);
}

// cu_seqlens (or None) against a number of sequences (or None): address and number.
const int32_t* sequences(PyObject* cu, PyObject* count, int64_t device, int32_t& N) {
  if (cu == Py_None) {
    N = count == Py_None ? 1 : integer(count, "N");
    return nullptr;
  }
  const at::Tensor& t = sized(cu, "cu_seqlens", 1, "[N + 1]");
  const int64_t n = t.size(0) - 1;
  if (count != Py_None && integer(count, "N") != n)
    refuse(PyExc_ValueError, "N is " + std::to_string(integer(count, "N")) + ", cu_seqlens has " + std::to_string(n) +
                                 " sequences");
  N = size32(n, "cu_seqlens");
  return static_cast<const int32_t*>(address(t, "cu_seqlens", at::kInt, {n + 1}, device));
}

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type, int64_t device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
}

// The caller's output tensor, or a new one.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
                  int64_t device, void** at) {
  if (o == Py_None) {
    at::Tensor t = empty(c10::IntArrayRef(shape.begin(), shape.size()), type, device);
    *at = t.data_ptr();
    return t;
  }
  const at::Tensor& t = tensor(o, name);
  *at = address(t, name, type, shape, device);
  return t;
}

// The caller's workspace, or one of `need` bytes (none for 0).
struct Workspace {
  at::Tensor keep;
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, int64_t device) {
    if (o != Py_None) {
      keep = tensor(o, "workspace");
      bytes = static_cast<size_t>(keep.numel());
      at = address(keep, "workspace", at::kByte, {keep.numel()}, device);
    } else if (need) {
      keep = empty({static_cast<int64_t>(need)}, at::kByte, device);
      bytes = need;
      at = keep.data_ptr();
    }
  }
};

// The six tensors of a cache, from a[0] on.
kda_cache cache_of(PyObject* const* a, int64_t device) {
  const at::Tensor& k = sized(a[0], "cache.k", 4, "[pages, Hk, page_size, 128]");
  const int64_t P = k.size(0), H = k.size(1), S = k.size(2), D = k.size(3);
  kda_cache c{};
  c.k = address(k, "cache.k", at::kFloat8_e4m3fn, {P, H, S, D}, device);
  c.v = address(a[1], "cache.v", at::kFloat8_e4m3fn, {P, H, S, D}, device);
  c.k_scale = static_cast<float*>(address(a[2], "cache.k_scale", at::kFloat, {P, H}, device));
  c.v_scale = static_cast<float*>(address(a[3], "cache.v_scale", at::kFloat, {P, H}, device));
  c.pos = static_cast<int32_t*>(address(a[4], "cache.pos", at::kInt, {P, H, S}, device));
  c.weight = static_cast<float*>(address(a[5], "cache.weight", at::kFloat, {P, H, S}, device));
  c.pages = size32(P, "cache.k");
  c.Hk = size32(H, "cache.k");
  c.page_size = size32(S, "cache.k");
  c.D = size32(D, "cache.k");
  return c;
}

void* stream_of(int64_t device) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}

PyObject* result(kda_status st, const at::Tensor& t) {
  return st == KDA_OK ? THPVariable_Wrap(t) : PyLong_FromLong(st);
}

// q, k, v, scale, mask, cap, slopes, prefix_lens, cu_seqlens, N, out
PyObject* attn_fwd(PyObject* const* a) {
  const at::Tensor& q = sized(a[0], "q", 3, "[T_total, heads, 128]");
  const at::Tensor& k = sized(a[1], "k", 3, "[T_total, heads, 128]");
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hk = k.size(1), dev = q.get_device();
  void* qp = address(q, "q", at::kBFloat16, {T, H, D}, dev);
  void* kp = address(k, "k", at::kBFloat16, {T, Hk, D}, dev);
  void* vp = address(a[2], "v", at::kBFloat16, {T, Hk, D}, dev);
  int32_t N = 0;
  const int32_t* cu = sequences(a[8], a[9], dev, N);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* op = nullptr;
  at::Tensor out = output(a[10], "out", at::kBFloat16, {T, H, D}, dev, &op);
  kda_attn_options o{};
  o.mask = integer(a[4], "mask");
  o.cap = static_cast<float>(number(a[5], "cap"));
  o.slopes = static_cast<const float*>(optional(a[6], "slopes", at::kFloat, {H}, dev));
  o.prefix_lens = static_cast<const int32_t*>(optional(a[7], "prefix_lens", at::kInt, {N}, dev));
  return result(kda_attn_fwd(&o, qp, kp, vp, static_cast<float>(number(a[3], "scale")), cu, T, size32(H, "q"),
                             size32(Hk, "k"), N, size32(D, "q"), op, stream_of(dev)),
                out);
}

// cache (6), k, v, block_table, lens, cu_seqlens, positions
PyObject* cache_append(PyObject* const* a) {
  const at::Tensor& k = sized(a[6], "k", 3, "[T_total, heads, 128]");
  const at::Tensor& table = sized(a[8], "block_table", 2, "[N, width]");
  const int64_t T = k.size(0), Hk = k.size(1), D = k.size(2), dev = k.get_device();
  const int64_t rows = table.size(0), width = table.size(1);
  const kda_cache c = cache_of(a, dev);
  if (Hk != c.Hk || D != c.D)
    refuse(PyExc_ValueError, "k has " + std::to_string(Hk) + " heads of " + std::to_string(D) + " channels, the cache " +
                                 std::to_string(c.Hk) + " of " + std::to_string(c.D));
  void* kp = address(k, "k", at::kBFloat16, {T, Hk, D}, dev);
  void* vp = address(a[7], "v", at::kBFloat16, {T, Hk, D}, dev);
  void* tp = address(table, "block_table", at::kInt, {rows, width}, dev);
  void* lp = address(a[9], "lens", at::kInt, {rows}, dev);
  void* pp = optional(a[11], "positions", at::kInt, {T}, dev);
  int32_t N = size32(rows, "block_table"), M = 0;
  const int32_t* cu = sequences(a[10], Py_None, dev, M);
  if (cu && M != N)
    refuse(PyExc_ValueError, "N is " + std::to_string(N) + ", cu_seqlens has " + std::to_string(M) + " sequences");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  return PyLong_FromLong(kda_cache_append(&c, kp, vp, static_cast<const int32_t*>(tp), size32(width, "block_table"),
                                          static_cast<const int32_t*>(lp), static_cast<const int32_t*>(pp), cu, T, N,
                                          stream_of(dev)));
}

// cache (6), q, block_table, lens, scale, cap, slopes, cu_seqlens, positions, accumulate, out, workspace
PyObject* cache_attn(PyObject* const* a) {
  const at::Tensor& q = sized(a[6], "q", 3, "[T_total, heads, 128]");
  const at::Tensor& table = sized(a[7], "block_table", 2, "[N, width]");
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), dev = q.get_device();
  const int64_t rows = table.size(0), width = table.size(1);
  const kda_cache c = cache_of(a, dev);
  if (D != c.D)
    refuse(PyExc_ValueError, "q has " + std::to_string(D) + " channels, the cache " + std::to_string(c.D));
  void* qp = address(q, "q", at::kBFloat16, {T, H, D}, dev);
  void* tp = address(table, "block_table", at::kInt, {rows, width}, dev);
  void* lp = address(a[8], "lens", at::kInt, {rows}, dev);
  int32_t N = size32(rows, "block_table"), M = 0;
  const int32_t* cu = sequences(a[12], Py_None, dev, M);
  if (cu && M != N)
    refuse(PyExc_ValueError, "N is " + std::to_string(N) + ", cu_seqlens has " + std::to_string(M) + " sequences");
  kda_cache_attn_options o{};
  o.cap = static_cast<float>(number(a[10], "cap"));
  o.slopes = static_cast<const float*>(optional(a[11], "slopes", at::kFloat, {H}, dev));
  o.positions = static_cast<const int32_t*>(optional(a[13], "positions", at::kInt, {T}, dev));
  o.accumulate = truth(a[14], "accumulate");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* op = nullptr;
  at::Tensor out = output(a[15], "out", at::kBFloat16, {T, H, D}, dev, &op);
  const int32_t w = size32(width, "block_table"), h = size32(H, "q");
  const Workspace ws(a[16], kda_cache_attn_workspace_size(&c, T, h, N, w, o.accumulate), dev);
  return result(kda_cache_attn(&o, &c, qp, static_cast<float>(number(a[9], "scale")), static_cast<const int32_t*>(tp), w,
                               static_cast<const int32_t*>(lp), cu, T, h, N, op, ws.at, ws.bytes, stream_of(dev)),
                out);
}

// cache (6), block_table, lens, dst_table, budget, recent, new_lens, workspace
PyObject* cache_evict(PyObject* const* a) {
  const at::Tensor& table = sized(a[6], "block_table", 2, "[N, width]");
  const at::Tensor& dst = sized(a[8], "dst_table", 2, "[N, width]");
  const int64_t rows = table.size(0), width = table.size(1), dst_width = dst.size(1), dev = table.get_device();
  const kda_cache c = cache_of(a, dev);
  void* tp = address(table, "block_table", at::kInt, {rows, width}, dev);
  void* dp = address(dst, "dst_table", at::kInt, {rows, dst_width}, dev);
  void* lp = address(a[7], "lens", at::kInt, {rows}, dev);
  const int32_t budget = integer(a[9], "budget"), recent = integer(a[10], "recent");
  const int32_t N = size32(rows, "block_table");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* np = nullptr;
  at::Tensor lens = output(a[11], "new_lens", at::kInt, {rows}, dev, &np);
  const int64_t slots = width * c.page_size;  // a budget beyond the table needs no more than one of its slots
  const Workspace ws(a[12], kda_cache_evict_workspace_size(&c, N, static_cast<int32_t>(std::min<int64_t>(budget, slots))), dev);
  return result(kda_cache_evict(&c, static_cast<const int32_t*>(tp), size32(width, "block_table"),
                                static_cast<const int32_t*>(lp), static_cast<const int32_t*>(dp),
                                size32(dst_width, "dst_table"), budget, recent, N, static_cast<int32_t*>(np), ws.at,
                                ws.bytes, stream_of(dev)),
                lens);
}

// torch's own error for device memory that is not to be had, as its allocations in Python give.
void out_of_memory(const char* text) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, text);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// No C++ exception leaves an entry.
template <PyObject* (*FN)(PyObject* const*), Py_ssize_t ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%zd arguments given, %zd needed", n, ARGS);
    return nullptr;
  }
  try {
    return FN(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    out_of_memory(e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*FN)(PyObject* const*), Py_ssize_t ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<FN, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<attn_fwd, 11>("attn_fwd"), method<cache_append, 12>("cache_append"),
                         method<cache_attn, 17>("cache_attn"), method<cache_evict, 13>("cache_evict"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "attn_binding", "Softmax attention of libkda on torch tensors.", -1,
                          methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() { return PyModule_Create(&module_def); }
