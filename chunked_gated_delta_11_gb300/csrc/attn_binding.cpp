// attn_binding.cpp -- the softmax-attention, short-convolution and state-space entry
// points as a Python extension.
//
// A serving step makes several of these calls for each token, and checking a
// dozen tensors and allocating the outputs in Python takes longer than the small
// calls' kernels do.  Here the tensors are looked at in place.  attention.py and
// recurrent.py document the functions and name their arguments; everything they pass
// is checked here before libkda is called.  A function returns what the Python
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

// A tuple of tensors (None for one that is not there).
PyObject* result(kda_status st, std::initializer_list<at::Tensor> all) {
  if (st != KDA_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(all.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : all) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Checks rows that may be cut out of wider ones (dimensions but the first contiguous, rows
// a multiple of `unit` elements apart); returns their address and the elements between
// two of them (0: one after the other).
void* strided(PyObject* o, const char* name, std::initializer_list<int64_t> shape, int64_t unit, int64_t device,
              int64_t& stride) {
  const at::Tensor& t = tensor(o, name);
  stride = 0;
  if (t.dim() < 2 || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != device ||
      !t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size())) || t.is_contiguous())
    return address(t, name, at::kBFloat16, shape, device);
  int64_t row = 1;
  for (int64_t d = t.dim() - 1; d > 0; --d) {
    if (t.size(d) != 1 && t.stride(d) != row)
      refuse(PyExc_ValueError, std::string(name) + " must be contiguous but for its first dimension");
    row *= t.size(d);
  }
  if (t.stride(0) < row || t.stride(0) % unit != 0)
    refuse(PyExc_ValueError, std::string(name) + " has rows " + std::to_string(t.stride(0)) + " elements apart: at least " +
                                 std::to_string(row) + " and a multiple of " + std::to_string(unit) + " are needed");
  stride = t.stride(0);
  return t.data_ptr();
}

// The initial state (or None) and the final one: the caller's, a new one of the same type (fp32
// without any), or none.
struct States {
  const void* init = nullptr;
  void* fin = nullptr;
  at::Tensor keep;
  at::ScalarType type = at::kFloat;
  // `only`: the one type that states have, or Undefined for fp32 or bf16
  States(PyObject* i, PyObject* f, PyObject* want, at::ScalarType only, std::initializer_list<int64_t> shape, int64_t device) {
    if (only != at::ScalarType::Undefined) {
      type = only;
    } else if (i != Py_None || f != Py_None) {
      const char* name = i != Py_None ? "initial_state" : "final_state";
      type = tensor(i != Py_None ? i : f, name).scalar_type();
      if (type != at::kFloat && type != at::kBFloat16)
        refuse(PyExc_TypeError, std::string(name) + " must be torch.float32 or torch.bfloat16, got " + name_of(type));
    }
    init = optional(i, "initial_state", type, shape, device);
    if (f != Py_None || truth(want, "output_final_state")) keep = output(f, "final_state", type, shape, device, &fin);
  }
};

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

// x, weight, bias, initial_state, cu_seqlens, N, silu, out, final_state, output_final_state
PyObject* conv_fwd(PyObject* const* a) {
  const at::Tensor& x = sized(a[0], "x", 2, "[T_total, C]");
  const at::Tensor& w = sized(a[1], "weight", 2, "[C, W]");
  const int64_t T = x.size(0), C = x.size(1), W = w.size(1), dev = x.get_device();
  kda_conv_options o{};
  void* xp = strided(a[0], "x", {T, C}, 8, dev, o.x_stride);
  void* wp = address(w, "weight", at::kBFloat16, {C, W}, dev);
  void* bp = optional(a[2], "bias", at::kBFloat16, {C}, dev);
  int32_t N = 0;
  const int32_t* cu = sequences(a[4], a[5], dev, N);
  o.silu = truth(a[6], "silu");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* op = nullptr;
  at::Tensor out = output(a[7], "out", at::kBFloat16, {T, C}, dev, &op);
  const States s(a[3], a[8], a[9], at::kBFloat16, {N, W - 1, C}, dev);
  return result(kda_conv_fwd(&o, xp, wp, bp, s.init, cu, T, size32(C, "x"), size32(W, "weight"), N, op, s.fin,
                             stream_of(dev)),
                {out, s.keep});
}

// x, dt, A, B, C, skip, dt_bias, initial_state, cu_seqlens, N, out, final_state, output_final_state, workspace
template <bool STEP>
PyObject* ssm(PyObject* const* a) {
  const at::Tensor& x = sized(a[0], "x", 3, "[T_total, heads, channels]");
  const at::Tensor& b = sized(a[3], "B", 3, "[T_total, groups, state]");
  const int64_t T = x.size(0), H = x.size(1), P = x.size(2), G = b.size(1), S = b.size(2), dev = x.get_device();
  kda_ssm_options o{};
  void* xp = strided(a[0], "x", {T, H, P}, 8, dev, o.x_stride);
  void* dp = strided(a[1], "dt", {T, H}, 1, dev, o.dt_stride);
  const float* ap = static_cast<const float*>(address(a[2], "A", at::kFloat, {H}, dev));
  void* bp = strided(a[3], "B", {T, G, S}, 8, dev, o.b_stride);
  void* cp = strided(a[4], "C", {T, G, S}, 8, dev, o.c_stride);
  o.skip = static_cast<const float*>(optional(a[5], "skip", at::kFloat, {H}, dev));
  o.dt_bias = static_cast<const float*>(optional(a[6], "dt_bias", at::kFloat, {H}, dev));
  int32_t N = 0;
  const int32_t* cu = sequences(a[8], a[9], dev, N);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* op = nullptr;
  at::Tensor out = output(a[10], "out", at::kBFloat16, {T, H, P}, dev, &op);
  const States s(a[7], a[11], a[12], at::ScalarType::Undefined, {N, H, P, S}, dev);
  o.state_dtype = s.type == at::kBFloat16 ? KDA_STATE_BF16 : KDA_STATE_F32;
  const int32_t h = size32(H, "x"), g = size32(G, "B"), p = size32(P, "x"), n = size32(S, "B");
  if constexpr (STEP)
    return result(kda_ssm_step(&o, xp, dp, ap, bp, cp, s.init, cu, T, h, g, N, p, n, op, s.fin, stream_of(dev)),
                  {out, s.keep});
  const Workspace ws(a[13], kda_ssm_workspace_size(T, h, g, N, p, n), dev);
  return result(kda_ssm_fwd(&o, xp, dp, ap, bp, cp, s.init, cu, T, h, g, N, p, n, op, s.fin, ws.at, ws.bytes,
                            stream_of(dev)),
                {out, s.keep});
}

// block_table, lens, new_rows, free_pages, free_count, page_size, rows, new_lens, cu_seqlens, slots, new_free_count
PyObject* cache_reserve(PyObject* const* a) {
  const at::Tensor& table = sized(a[0], "block_table", 2, "[N, width]");
  const at::Tensor& list = sized(a[3], "free_pages", 1, "[pages]");
  const int64_t N = table.size(0), width = table.size(1), pages = list.size(0), dev = table.get_device();
  void* tp = address(table, "block_table", at::kInt, {N, width}, dev);
  void* lp = address(a[1], "lens", at::kInt, {N}, dev);
  void* np = address(a[2], "new_rows", at::kInt, {N}, dev);
  void* fp = address(list, "free_pages", at::kInt, {pages}, dev);
  void* cp = address(a[4], "free_count", at::kInt, {1}, dev);
  const int32_t page = integer(a[5], "page_size");
  const bool known = a[6] != Py_None;
  const int64_t T = known ? integer(a[6], "rows") : INT32_MAX;
  if (T < 0) refuse(PyExc_ValueError, "rows is out of range");
  if (!known && a[9] != Py_None) refuse(PyExc_ValueError, "slots needs rows");
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void *lens = nullptr, *cu = nullptr, *slots = nullptr, *left = nullptr;
  const at::Tensor new_lens = output(a[7], "new_lens", at::kInt, {N}, dev, &lens);
  const at::Tensor sums = output(a[8], "cu_seqlens", at::kInt, {N + 1}, dev, &cu);
  const at::Tensor places = known ? output(a[9], "slots", at::kLong, {T}, dev, &slots) : at::Tensor();
  const at::Tensor count = output(a[10], "new_free_count", at::kInt, {1}, dev, &left);
  return result(kda_cache_reserve(static_cast<int32_t*>(tp), size32(width, "block_table"), static_cast<const int32_t*>(lp),
                                  static_cast<const int32_t*>(np), static_cast<const int32_t*>(fp),
                                  static_cast<const int32_t*>(cp), size32(pages, "free_pages"), page, T,
                                  size32(N, "block_table"), static_cast<int32_t*>(lens), static_cast<int32_t*>(cu),
                                  static_cast<int64_t*>(slots), static_cast<int32_t*>(left), stream_of(dev)),
                {new_lens, sums, places, count});
}

// block_table, lens, free_pages, free_count, page_size, keep, new_free_count
PyObject* cache_release(PyObject* const* a) {
  const at::Tensor& table = sized(a[0], "block_table", 2, "[N, width]");
  const at::Tensor& list = sized(a[2], "free_pages", 1, "[pages]");
  const int64_t N = table.size(0), width = table.size(1), pages = list.size(0), dev = table.get_device();
  void* tp = address(table, "block_table", at::kInt, {N, width}, dev);
  void* lp = address(a[1], "lens", at::kInt, {N}, dev);
  void* fp = address(list, "free_pages", at::kInt, {pages}, dev);
  void* cp = address(a[3], "free_count", at::kInt, {1}, dev);
  const int32_t page = integer(a[4], "page_size");
  void* kp = optional(a[5], "keep", at::kInt, {N}, dev);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* left = nullptr;
  const at::Tensor count = output(a[6], "new_free_count", at::kInt, {1}, dev, &left);
  return result(kda_cache_release(static_cast<const int32_t*>(tp), size32(width, "block_table"),
                                  static_cast<const int32_t*>(lp), static_cast<const int32_t*>(kp),
                                  static_cast<int32_t*>(fp), static_cast<const int32_t*>(cp), size32(pages, "free_pages"),
                                  page, size32(N, "block_table"), static_cast<int32_t*>(left), stream_of(dev)),
                count);
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
                         method<conv_fwd, 10>("conv_fwd"), method<ssm<false>, 14>("ssm_fwd"),
                         method<ssm<true>, 14>("ssm_step"), method<cache_reserve, 11>("cache_reserve"),
                         method<cache_release, 7>("cache_release"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "attn_binding", "Softmax attention of libkda on torch tensors.", -1,
                          methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() { return PyModule_Create(&module_def); }
