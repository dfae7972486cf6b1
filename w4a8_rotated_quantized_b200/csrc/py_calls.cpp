// py_calls.cpp -- the Python side of the adapter, checkpoint and input-gradient calls: checks of the tensors, the
// outputs and scratch from torch's allocator, the current stream, and the call into the C ABI.
//
// These calls run a few microseconds on the GPU for single tokens; marshalled through ctypes they took 11 of the
// 13 us of such a call.  Everything here is what binding.py does for the other calls: the library sees only raw
// addresses and sizes, so a tensor of the wrong shape, dtype or device is refused before its address is taken.
// All arithmetic stays in the library.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "../../include/convrot.h"

namespace {

PyObject* g_error = nullptr;  // binding.ConvRotError

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; None is refused unless `optional`, and gives an undefined tensor then.
at::Tensor tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return {};
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int as_int(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " has more than 2^31 - 1 rows or columns");
  return static_cast<int>(n);
}

struct Matrix {
  const void* p = nullptr;
  int64_t ld = 0;
};
struct Rows {  // of an output
  void* p = nullptr;
  int64_t ld = 0;
};

// A bf16 [M, C] matrix with dense columns.
Matrix matrix(const at::Tensor& t, const char* name, at::Device dev, int64_t M, int64_t C) {
  if (t.scalar_type() != at::kBFloat16 || t.device() != dev)
    refuse(PyExc_TypeError, std::string(name) + " must be a bfloat16 tensor on " + dev.str());
  const int64_t want[2] = {M, C};
  if (t.sizes() != at::IntArrayRef(want, 2))
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text({want, 2}) + ", got " + shape_text(t.sizes()));
  if (C > 1 && M > 0 && t.stride(1) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have unit stride along the last dimension");
  // the stride of a single row or of an empty tensor says nothing
  return {t.const_data_ptr(), M <= 1 || C == 0 ? C : t.stride(0)};
}

// The call's first operand, bf16 [M, C] on a CUDA device.
Matrix input(const at::Tensor& t, const char* name, int* M, int* C) {
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda())
    refuse(PyExc_TypeError, std::string(name) + " must be a CUDA bfloat16 tensor");
  if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be 2-D");
  *M = as_int(t.size(0), name);
  *C = as_int(t.size(1), name);
  return matrix(t, name, t.device(), t.size(0), t.size(1));
}

// A contiguous tensor of exactly this shape, dtype and device.
template <size_t n>
void* exact(const at::Tensor& t, const char* name, at::ScalarType dtype, at::Device dev, const int64_t (&want)[n]) {
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
  if (t.device() != dev)
    refuse(PyExc_TypeError, std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
  if (t.sizes() != at::IntArrayRef(want, n))
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text({want, n}) + ", got " + shape_text(t.sizes()));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return const_cast<void*>(t.const_data_ptr());
}

at::Tensor make(at::IntArrayRef size, at::ScalarType dtype, at::Device dev) {
  return at::empty(size, at::TensorOptions().dtype(dtype).device(dev));
}

// The caller's output or a new one, bf16 [M, C].  Taken for writing, which gives a copy-on-write tensor memory of its
// own: so before the address of any operand that may be the same tensor.
Rows output(at::Tensor& out, at::Device dev, int64_t M, int64_t C) {
  int64_t ld = C;
  if (out.defined())
    ld = matrix(out, "out", dev, M, C).ld;
  else
    out = make({M, C}, at::kBFloat16, dev);
  return {out.mutable_data_ptr(), ld};
}

// Scratch: the caller's, or a buffer of this call's own from torch's allocator on the current stream (inside a
// graph capture: from the graph's pool), so that calls on several streams and captured graphs share nothing.
struct Scratch {
  at::Tensor t;
  void* p = nullptr;
  size_t n = 0;
};
Scratch scratch(PyObject* given, size_t bytes, at::Device dev) {
  Scratch s;
  if (given != Py_None) {
    s.t = tensor(given, "workspace");
    if (s.t.scalar_type() != at::kByte || s.t.device() != dev)
      refuse(PyExc_TypeError, "workspace must be a uint8 tensor on " + dev.str());
    if (s.t.dim() != 1 || !s.t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be a contiguous 1-D uint8 tensor");
    s.p = s.t.mutable_data_ptr();
    s.n = static_cast<size_t>(s.t.numel());
  } else if (bytes > 0) {
    s.t = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    s.p = s.t.mutable_data_ptr();
    s.n = bytes;
  }
  return s;
}

// Makes a device current for the library's call.
struct On {
  c10::DeviceIndex back = -1;
  explicit On(at::Device dev) {
    const c10::DeviceIndex now = c10::cuda::current_device();
    if (now != dev.index()) {
      c10::cuda::set_device(dev.index());
      back = now;
    }
  }
  ~On() {
    if (back >= 0) c10::cuda::set_device(back);
  }
};

void* stream(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

void check(const char* call, cr_status st) {
  if (st == CR_OK) return;
  PyObject* args = Py_BuildValue("(si)", call, static_cast<int>(st));
  if (args) {
    PyErr_SetObject(g_error, args);
    Py_DECREF(args);
  }
  throw python_error();
}

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw python_error();
  return t != 0;
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

struct Pool {
  int L, r, K, N;
  void *down, *up, *scale, *adapter;
};
// The pool's factors down [L, r, K] and up [L, r, N], its scales [L] and the rows' adapters [M] or None; K or N is
// given by the call's first operand, the other (negative) by the factor.
Pool pool(const at::Tensor& down, const at::Tensor& up, const at::Tensor& scale, const at::Tensor& adapter, at::Device dev,
          int64_t M, int64_t K, int64_t N) {
  if (down.dim() != 3) refuse(PyExc_ValueError, "down must be 3-D [adapters, rank, columns]");
  if (up.dim() != 3) refuse(PyExc_ValueError, "up must be 3-D [adapters, rank, columns]");
  const int64_t L = down.size(0), r = down.size(1);
  if (K < 0) K = down.size(2);
  if (N < 0) N = up.size(2);
  Pool p;
  p.down = exact(down, "down", at::kBFloat16, dev, {L, r, K});
  p.up = exact(up, "up", at::kBFloat16, dev, {L, r, N});
  p.scale = exact(scale, "scale", at::kFloat, dev, {L});
  p.adapter = adapter.defined() ? exact(adapter, "adapter", at::kInt, dev, {M}) : nullptr;
  p.L = as_int(L, "down");
  p.r = as_int(r, "down");
  p.K = as_int(K, "down");
  p.N = as_int(N, "up");
  return p;
}

// (X, down, up, scale, adapter, base, out, save_v, workspace) -> Y or (Y, V)
PyObject* lora_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const at::Tensor X = tensor(a[0], "X");
  int M, K;
  const Matrix x = input(X, "X", &M, &K);
  const at::Device dev = X.device();
  const at::Tensor down = tensor(a[1], "down"), up = tensor(a[2], "up"), scale = tensor(a[3], "scale");
  const at::Tensor adapter = tensor(a[4], "adapter", true), base = tensor(a[5], "base", true);
  const Pool p = pool(down, up, scale, adapter, dev, M, K, -1);
  at::Tensor Y = tensor(a[6], "out", true), V;
  const Rows y = output(Y, dev, M, p.N);
  const Matrix b = base.defined() ? matrix(base, "base", dev, M, p.N) : Matrix{};
  if (truth(a[7])) V = make({M, p.r}, at::kBFloat16, dev);
  const Scratch ws = scratch(a[8], cr_lora_forward_workspace_size(M, p.N, K, p.r, p.L), dev);
  {
    On on(dev);
    check("cr_lora_forward",
          cr_lora_forward(x.p, x.ld, static_cast<const int32_t*>(p.adapter), p.down, p.up, static_cast<const float*>(p.scale),
                          b.p, b.ld, y.p, y.ld, V.defined() ? V.mutable_data_ptr() : nullptr, M, p.N, K,
                          p.r, p.L, ws.p, ws.n, stream(dev)));
  }
  PyObject* out = a[6] != Py_None ? Py_NewRef(a[6]) : wrap(Y);
  if (!V.defined() || !out) return out;
  PyObject* v = wrap(V);
  PyObject* both = v ? PyTuple_Pack(2, out, v) : nullptr;
  Py_DECREF(out);
  Py_XDECREF(v);
  return both;
  END_HANDLE_TH_ERRORS
}

// (dY, X, V, down, up, scale, adapter, base, out, need_dx, need_down, need_up, workspace) -> (dX, d_down, d_up)
PyObject* lora_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 13);
  const at::Tensor dY = tensor(a[0], "dY");
  int M, N;
  const Matrix dy = input(dY, "dY", &M, &N);
  const at::Device dev = dY.device();
  const at::Tensor down = tensor(a[3], "down"), up = tensor(a[4], "up"), scale = tensor(a[5], "scale");
  const at::Tensor adapter = tensor(a[6], "adapter", true), base = tensor(a[7], "base", true);
  const Pool p = pool(down, up, scale, adapter, dev, M, -1, N);
  const bool need_dx = truth(a[9]), need_down = truth(a[10]), need_up = truth(a[11]);
  if (need_down && a[1] == Py_None) refuse(PyExc_ValueError, "X (or its checkpoint) is needed for d_down");
  if (need_up && a[2] == Py_None) refuse(PyExc_ValueError, "V is needed for d_up");
  if (!need_dx && a[8] != Py_None) refuse(PyExc_ValueError, "out takes dX, which is not needed");
  Matrix x;
  void *codes = nullptr, *code_scales = nullptr, *v = nullptr;
  at::Tensor kept0, kept1;
  if (PyTuple_Check(a[1]) || PyList_Check(a[1])) {
    if (PySequence_Fast_GET_SIZE(a[1]) != 2) refuse(PyExc_ValueError, "a checkpoint is (codes, scales)");
    kept0 = tensor(PySequence_Fast_GET_ITEM(a[1], 0), "codes");
    kept1 = tensor(PySequence_Fast_GET_ITEM(a[1], 1), "scales");
    codes = exact(kept0, "codes", at::kChar, dev, {M, p.K});
    code_scales = exact(kept1, "scales", at::kFloat, dev, {M, p.K / 256});
  } else if (a[1] != Py_None) {
    kept0 = tensor(a[1], "X");
    x = matrix(kept0, "X", dev, M, p.K);
  }
  const at::Tensor V = tensor(a[2], "V", true);
  if (V.defined()) v = exact(V, "V", at::kBFloat16, dev, {M, p.r});
  at::Tensor dX = tensor(a[8], "out", true), dd, du;
  Rows dx;
  if (need_dx) dx = output(dX, dev, M, p.K);
  const Matrix b = base.defined() ? matrix(base, "base", dev, M, p.K) : Matrix{};
  if (need_down) dd = make({p.L, p.r, p.K}, at::kBFloat16, dev);
  if (need_up) du = make({p.L, p.r, N}, at::kBFloat16, dev);
  const Scratch ws = scratch(a[12], cr_lora_backward_workspace_size(M, N, p.K, p.r, p.L), dev);
  {
    On on(dev);
    check("cr_lora_backward",
          cr_lora_backward(dy.p, dy.ld, x.p, x.ld, codes, static_cast<const float*>(code_scales), v,
                           static_cast<const int32_t*>(p.adapter), p.down, p.up, static_cast<const float*>(p.scale), b.p,
                           b.ld, dx.p, dx.ld, dd.defined() ? dd.mutable_data_ptr() : nullptr,
                           du.defined() ? du.mutable_data_ptr() : nullptr, M, N, p.K, p.r, p.L, ws.p, ws.n, stream(dev)));
  }
  PyObject* out[3] = {a[8] != Py_None ? Py_NewRef(a[8]) : wrap(dX), wrap(dd), wrap(du)};
  PyObject* all = out[0] && out[1] && out[2] ? PyTuple_Pack(3, out[0], out[1], out[2]) : nullptr;
  for (PyObject* o : out) Py_XDECREF(o);
  return all;
  END_HANDLE_TH_ERRORS
}

// (X) -> (codes, scales)
PyObject* ckpt_save(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 1);
  const at::Tensor X = tensor(a[0], "X");
  int M, K;
  const Matrix x = input(X, "X", &M, &K);
  const at::Device dev = X.device();
  const at::Tensor codes = make({M, K}, at::kChar, dev), scales = make({M, K / 256}, at::kFloat, dev);
  {
    On on(dev);
    check("cr_ckpt_save",
          cr_ckpt_save(x.p, M, K, x.ld, codes.mutable_data_ptr(), static_cast<float*>(scales.mutable_data_ptr()), stream(dev)));
  }
  PyObject *c = wrap(codes), *s = wrap(scales);
  PyObject* both = c && s ? PyTuple_Pack(2, c, s) : nullptr;
  Py_XDECREF(c);
  Py_XDECREF(s);
  return both;
  END_HANDLE_TH_ERRORS
}

// (codes, scales, out) -> X
PyObject* ckpt_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 3);
  const at::Tensor codes = tensor(a[0], "codes");
  if (codes.scalar_type() != at::kChar || codes.dim() != 2 || !codes.is_contiguous())
    refuse(PyExc_TypeError, "codes must be a contiguous 2-D torch.int8 tensor");
  if (!codes.is_cuda()) refuse(PyExc_TypeError, "codes must be on a CUDA device, got " + codes.device().str());
  const int M = as_int(codes.size(0), "codes"), K = as_int(codes.size(1), "codes");
  const at::Device dev = codes.device();
  const at::Tensor scales = tensor(a[1], "scales");
  const void* s = exact(scales, "scales", at::kFloat, dev, {M, K / 256});
  at::Tensor X = tensor(a[2], "out", true);
  const Rows x = output(X, dev, M, K);
  {
    On on(dev);
    check("cr_ckpt_load", cr_ckpt_load(codes.const_data_ptr(), static_cast<const float*>(s), M, K, x.p, x.ld, stream(dev)));
  }
  return a[2] != Py_None ? Py_NewRef(a[2]) : wrap(X);
  END_HANDLE_TH_ERRORS
}

// (dY, Wq, w_scale, group, out, workspace) -> dX
PyObject* grad_input(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  const at::Tensor dY = tensor(a[0], "dY");
  int M, N;
  const Matrix dy = input(dY, "dY", &M, &N);
  const at::Device dev = dY.device();
  const at::Tensor Wq = tensor(a[1], "Wq"), w_scale = tensor(a[2], "w_scale");
  if (Wq.dim() != 2) refuse(PyExc_ValueError, "Wq must be 2-D [N, K/2]");
  const int K = as_int(2 * Wq.size(1), "Wq");
  const void* w = exact(Wq, "Wq", at::kByte, dev, {N, K / 2});
  const void* s = exact(w_scale, "w_scale", at::kFloat, dev, {N});
  const long group = PyLong_AsLong(a[3]);
  if (group == -1 && PyErr_Occurred()) throw python_error();
  if (group != static_cast<int>(group)) refuse(PyExc_ValueError, "group must be 16, 64, 256 or 1024");
  at::Tensor dX = tensor(a[4], "out", true);
  const Rows dx = output(dX, dev, M, K);
  const Scratch ws = scratch(a[5], cr_w4a4_grad_input_workspace_size(M, N, K, static_cast<int>(group)), dev);
  {
    On on(dev);
    check("cr_w4a4_grad_input",
          cr_w4a4_grad_input(dy.p, dy.ld, w, static_cast<const float*>(s), dx.p, dx.ld, M, N, K,
                             static_cast<int>(group), ws.p, ws.n, stream(dev)));
  }
  return a[4] != Py_None ? Py_NewRef(a[4]) : wrap(dX);
  END_HANDLE_TH_ERRORS
}

// (ConvRotError): the exception that a status other than CR_OK raises
PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"lora_forward", fast<lora_forward>(), METH_FASTCALL, nullptr},
    {"lora_backward", fast<lora_backward>(), METH_FASTCALL, nullptr},
    {"ckpt_save", fast<ckpt_save>(), METH_FASTCALL, nullptr},
    {"ckpt_load", fast<ckpt_load>(), METH_FASTCALL, nullptr},
    {"grad_input", fast<grad_input>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
