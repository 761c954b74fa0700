// _calls: the short way from Python to the gated block, the 8-bit checkpoints and the 4-bit linears, whose
// calls may take a few microseconds on the device and 9 to 11 through ctypes. Each function checks what the binding (rglru.py) checks, allocates the
// output, and calls the same C ABI on the current stream. Where anything is not as it should be, or the
// library returns an error, it returns None and has launched nothing that counts: the binding then goes
// its long way, which finds the same fault and raises for it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "rglru.h"

namespace {

constexpr int64_t kWidest = 65536;

// The tensor behind a plain torch.Tensor (or Parameter), null for anything else.
const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of that type on that device.
bool plain(const at::Tensor* t, at::ScalarType type, int device) {
  return t != nullptr && t->scalar_type() == type && t->layout() == at::kStrided && t->is_cuda() &&
         t->get_device() == device && t->is_contiguous();
}

bool same_lead(at::IntArrayRef a, at::IntArrayRef b) {
  return a.size() == b.size() && a.slice(0, a.size() - 1).equals(b.slice(0, b.size() - 1));
}

// Uninitialised memory from the caching allocator, for the current stream. (Asked for directly: the way through the
// dispatcher takes 0.3 µs more, of calls that take 3.5 with one allocation.)
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt));
}
at::Tensor with_last(const at::Tensor& x, int64_t last, at::ScalarType type) {
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = last;
  return fresh(shape, type, x.get_device());
}

// `out` as given (None: a new tensor) for a result of x's leading shape and `last` columns; undefined if it does
// not fit.
at::Tensor result(PyObject* out, const at::Tensor& x, int64_t last, at::ScalarType type, int device) {
  if (out == Py_None) return with_last(x, last, type);
  const at::Tensor* t = tensor(out);
  if (!plain(t, type, device) || !same_lead(t->sizes(), x.sizes()) || t->sizes().back() != last) return at::Tensor();
  return *t;
}

rglru_stream_t stream_of(int device) {
  return reinterpret_cast<rglru_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
}

// x's device if it is the current one, else −1.
int device_of(const at::Tensor* x) {
  if (x == nullptr || !x->is_cuda() || x->dim() < 1) return -1;
  const int d = x->get_device();
  return d == c10::cuda::current_device() ? d : -1;
}

PyObject* wrap(PyObject* out, at::Tensor t) {
  if (out != Py_None) return Py_NewRef(out);
  return THPVariable_Wrap(std::move(t));
}

// The library's call with the interpreter free for other threads, as ctypes leaves it. Addresses and the stream are
// asked for before it: that may throw (a tensor inside torch.func's transforms has no storage).
template <class F> int call(F f) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
}

// Runs f, which returns a new reference or null for "not this way"; C++ exceptions (out of memory among
// them) go the long way too.
template <class F> PyObject* guarded(F f) {
  try {
    if (PyObject* r = f()) return r;
  } catch (const std::exception&) {  // (none passes while the interpreter is released)
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (W_gate, W_up, x, activation, h | None)
PyObject* glu_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return nullptr;
    const at::Tensor *wg = tensor(a[0]), *wu = tensor(a[1]), *x = tensor(a[2]);
    const int d = device_of(x);
    if (d < 0 || !plain(x, at::kBFloat16, d) || !plain(wg, at::kBFloat16, d) || !plain(wu, at::kBFloat16, d))
      return nullptr;
    if (wg->dim() != 2 || !wu->sizes().equals(wg->sizes())) return nullptr;
    const int64_t H = wg->size(0), D = wg->size(1);
    if (H < 1 || D < 1 || H > kWidest || D > kWidest || x->sizes().back() != D) return nullptr;
    const long act = PyLong_AsLong(a[3]);
    at::Tensor h = result(a[4], *x, H, at::kBFloat16, d);
    if (!h.defined()) return nullptr;
    const void *wgp = wg->const_data_ptr(), *wup = wu->const_data_ptr(), *xp = x->const_data_ptr();
    void* hp = h.mutable_data_ptr();
    const int64_t N = x->numel() / D;
    rglru_stream_t s = stream_of(d);
    if (call([&] { return rglru_glu_forward(wgp, wup, xp, hp, N, (int)D, (int)H, (int)act, s); }) != RGLRU_OK) return nullptr;
    return wrap(a[4], std::move(h));
  });
}

// (W_gate, W_up, x | None, codes | None, scales | None, dh, activation, want_h) → (dx, dW_gate, dW_up, h | None)
PyObject* glu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return nullptr;
    const at::Tensor *wg = tensor(a[0]), *wu = tensor(a[1]), *dh = tensor(a[5]);
    const bool packed = a[2] == Py_None;
    const at::Tensor *x = tensor(packed ? a[3] : a[2]), *scales = packed ? tensor(a[4]) : nullptr;
    const int d = device_of(x);
    if (d < 0 || !plain(x, packed ? at::kChar : at::kBFloat16, d) || !plain(wg, at::kBFloat16, d) ||
        !plain(wu, at::kBFloat16, d) || !plain(dh, at::kBFloat16, d) || (packed && !plain(scales, at::kByte, d)))
      return nullptr;
    if (wg->dim() != 2 || !wu->sizes().equals(wg->sizes())) return nullptr;
    const int64_t H = wg->size(0), D = wg->size(1);
    if (H < 1 || D < 1 || H > kWidest || D > kWidest || x->sizes().back() != D || dh->dim() < 1 ||
        !same_lead(x->sizes(), dh->sizes()) || dh->sizes().back() != H)
      return nullptr;
    if (packed && (scales->dim() < 1 || !same_lead(x->sizes(), scales->sizes()) || scales->sizes().back() != (D + 31) / 32))
      return nullptr;
    const int act = (int)PyLong_AsLong(a[6]);
    const bool want_h = a[7] == Py_True;
    const int64_t N = x->numel() / D;
    const size_t bytes = rglru_glu_backward_workspace_bytes(N, (int)D, (int)H, packed);
    if (bytes == 0) return nullptr;
    at::Tensor dx = with_last(*x, D, at::kBFloat16), dwg = fresh({H, D}, at::kBFloat16, d),
               dwu = fresh({H, D}, at::kBFloat16, d), h, ws = fresh({(int64_t)bytes}, at::kByte, d);
    if (want_h) h = with_last(*x, H, at::kBFloat16);
    const void *wgp = wg->const_data_ptr(), *wup = wu->const_data_ptr(), *xp = x->const_data_ptr(),
               *dhp = dh->const_data_ptr(), *scp = packed ? scales->const_data_ptr() : nullptr;
    void *dxp = dx.mutable_data_ptr(), *dwgp = dwg.mutable_data_ptr(), *dwup = dwu.mutable_data_ptr(),
         *wsp = ws.mutable_data_ptr(), *hp = want_h ? h.mutable_data_ptr() : nullptr;
    rglru_stream_t s = stream_of(d);
    const int r = call([&] {
      return packed ? rglru_glu_backward_act8(wgp, wup, xp, scp, dhp, dxp, dwgp, dwup, hp, N, (int)D, (int)H, act, wsp, bytes, s)
                    : rglru_glu_backward(wgp, wup, xp, dhp, dxp, dwgp, dwup, hp, N, (int)D, (int)H, act, wsp, bytes, s);
    });
    if (r != RGLRU_OK) return nullptr;
    PyObject* o[4] = {THPVariable_Wrap(std::move(dx)), THPVariable_Wrap(std::move(dwg)), THPVariable_Wrap(std::move(dwu)),
                      want_h ? THPVariable_Wrap(std::move(h)) : Py_NewRef(Py_None)};
    PyObject* t = o[0] && o[1] && o[2] && o[3] ? PyTuple_Pack(4, o[0], o[1], o[2], o[3]) : nullptr;
    for (PyObject* v : o) Py_XDECREF(v);
    return t;
  });
}

// (x) → (codes, scales)
PyObject* act8_pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 1) return nullptr;
    const at::Tensor* x = tensor(a[0]);
    const int d = device_of(x);
    if (d < 0) return nullptr;
    const bool bf16 = x->scalar_type() == at::kBFloat16;
    if (!plain(x, bf16 ? at::kBFloat16 : at::kFloat, d)) return nullptr;
    const int64_t C = x->sizes().back();
    if (C < 1 || C > kWidest) return nullptr;
    at::Tensor codes = with_last(*x, C, at::kChar), scales = with_last(*x, (C + 31) / 32, at::kByte);
    const void* xp = x->const_data_ptr();
    void *cp = codes.mutable_data_ptr(), *sp = scales.mutable_data_ptr();
    const int64_t N = x->numel() / C;
    rglru_stream_t st = stream_of(d);
    if (call([&] { return rglru_act8_pack(xp, cp, sp, N, (int)C, bf16 ? RGLRU_BF16 : RGLRU_F32, st); }) != RGLRU_OK)
      return nullptr;
    PyObject* c = THPVariable_Wrap(std::move(codes));
    PyObject* s = THPVariable_Wrap(std::move(scales));
    PyObject* r = c != nullptr && s != nullptr ? PyTuple_Pack(2, c, s) : nullptr;
    Py_XDECREF(c);
    Py_XDECREF(s);
    return r;
  });
}

// (codes, scales, is_bf16, x | None)
PyObject* act8_unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return nullptr;
    const at::Tensor *codes = tensor(a[0]), *scales = tensor(a[1]);
    const int d = device_of(codes);
    if (d < 0 || !plain(codes, at::kChar, d) || !plain(scales, at::kByte, d)) return nullptr;
    const int64_t C = codes->sizes().back();
    if (C < 1 || C > kWidest || !same_lead(codes->sizes(), scales->sizes()) || scales->sizes().back() != (C + 31) / 32)
      return nullptr;
    const bool bf16 = a[2] == Py_True;
    at::Tensor x = result(a[3], *codes, C, bf16 ? at::kBFloat16 : at::kFloat, d);
    if (!x.defined()) return nullptr;
    const void *cp = codes->const_data_ptr(), *sp = scales->const_data_ptr();
    void* xp = x.mutable_data_ptr();
    const int64_t N = x.numel() / C;
    rglru_stream_t s = stream_of(d);
    if (call([&] { return rglru_act8_unpack(cp, sp, xp, N, (int)C, bf16 ? RGLRU_BF16 : RGLRU_F32, s); }) != RGLRU_OK)
      return nullptr;
    return wrap(a[3], std::move(x));
  });
}

struct W4 {
  const at::Tensor *codes, *scales;
  int64_t N, K;
};
bool w4_of(PyObject* codes, PyObject* scales, int64_t group, int device, W4& w) {
  w.codes = tensor(codes);
  w.scales = tensor(scales);
  if (group != 32 && group != 64 && group != 128) return false;
  if (!plain(w.codes, at::kByte, device) || !plain(w.scales, at::kBFloat16, device)) return false;
  if (w.codes->dim() != 2 || w.scales->dim() != 2) return false;
  w.N = w.codes->size(0);
  w.K = 2 * w.codes->size(1);
  return w.N >= 1 && w.K >= 1 && w.N <= kWidest && w.K <= kWidest && w.scales->size(0) == w.N &&
         w.scales->size(1) == w.K / group;
}

// (codes, scales, group, x, y | None)
PyObject* w4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return nullptr;
    const at::Tensor* x = tensor(a[3]);
    const int d = device_of(x);
    const long group = PyLong_AsLong(a[2]);
    W4 w;
    if (d < 0 || !plain(x, at::kBFloat16, d) || !w4_of(a[0], a[1], group, d, w) || x->sizes().back() != w.K ||
        x->numel() / w.K > 64)
      return nullptr;
    at::Tensor y = result(a[4], *x, w.N, at::kBFloat16, d);
    if (!y.defined()) return nullptr;
    const void *cp = w.codes->const_data_ptr(), *sp = w.scales->const_data_ptr(), *xp = x->const_data_ptr();
    void* yp = y.mutable_data_ptr();
    const int M = (int)(x->numel() / w.K);
    rglru_stream_t s = stream_of(d);
    if (call([&] { return rglru_w4_linear(cp, sp, xp, yp, M, (int)w.N, (int)w.K, (int)group, s); }) != RGLRU_OK) return nullptr;
    return wrap(a[4], std::move(y));
  });
}

// (gate codes, gate scales, up codes, up scales, group, x, activation, h | None)
PyObject* w4_glu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return nullptr;
    const at::Tensor* x = tensor(a[5]);
    const int d = device_of(x);
    const long group = PyLong_AsLong(a[4]);
    W4 g, u;
    if (d < 0 || !plain(x, at::kBFloat16, d) || !w4_of(a[0], a[1], group, d, g) || !w4_of(a[2], a[3], group, d, u) ||
        g.N != u.N || g.K != u.K || x->sizes().back() != g.K || x->numel() / g.K > 64)
      return nullptr;
    const long act = PyLong_AsLong(a[6]);
    at::Tensor h = result(a[7], *x, g.N, at::kBFloat16, d);
    if (!h.defined()) return nullptr;
    const void *gc = g.codes->const_data_ptr(), *gs = g.scales->const_data_ptr(), *uc = u.codes->const_data_ptr(),
               *us = u.scales->const_data_ptr(), *xp = x->const_data_ptr();
    void* hp = h.mutable_data_ptr();
    const int M = (int)(x->numel() / g.K);
    rglru_stream_t s = stream_of(d);
    if (call([&] { return rglru_w4_glu(gc, gs, uc, us, xp, hp, M, (int)g.N, (int)g.K, (int)group, (int)act, s); }) != RGLRU_OK)
      return nullptr;
    return wrap(a[7], std::move(h));
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)> PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef kMethods[] = {method<glu_forward>("glu_forward"), method<glu_backward>("glu_backward"),
                          method<act8_pack>("act8_pack"),     method<act8_unpack>("act8_unpack"),
                          method<w4_linear>("w4_linear"),     method<w4_glu>("w4_glu"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
