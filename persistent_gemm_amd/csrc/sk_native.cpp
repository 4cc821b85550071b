// The short way into the library for the block-scaled and norm calls: a CPython module that checks the
// tensors, allocates the outputs and calls the C ABI, where the same steps in Python take longer than a
// small kernel runs (a quantised norm of 16 rows: 10 us in Python, 3.6 us on the device).
//
// It only takes calls whose arguments are all as they should be.  For any other it returns None and has done
// nothing: the binding's own checks then say what is wrong.  A status of the C ABI other than SK_OK
// comes back as an int.  The library's entry points are handed in by bind(), so that both ways run the same one.

#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/sk_gemm.h"

namespace {

using at::Tensor;

struct Library {
  decltype(&sk_quantize_fp8_block) quantize = nullptr;
  decltype(&sk_gemm_fp8_block) gemm = nullptr;
  decltype(&sk_gemm_fp8_block_backward) gemm_backward = nullptr;
  decltype(&sk_norm_forward) norm_forward = nullptr;
  decltype(&sk_norm_backward) norm_backward = nullptr;
} lib;

constexpr int64_t up16(int64_t n) { return (n + 15) & ~(int64_t)15; }
constexpr int64_t blocks(int64_t n) { return (n + 127) >> 7; }

// An argument: a tensor, None, or neither.
struct Arg {
  const Tensor* t = nullptr;
  bool bad = false;
  explicit Arg(PyObject* o) {
    if (THPVariable_Check(o)) t = &THPVariable_Unpack(o);
    else bad = o != Py_None;
  }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

bool is(const Tensor& t, c10::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  return t.layout() == at::kStrided && t.device() == dev && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}
bool is_codes(const Tensor& t, c10::Device dev, at::IntArrayRef shape) {
  return is(t, dev, t.scalar_type() == at::kByte ? at::kByte : at::kFloat8_e4m3fn, shape);
}
// NULL, or as described.
bool none_or(const Arg& a, c10::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  return !a.bad && (!a.t || is(*a.t, dev, type, shape));
}

// An output, from the allocator that torch's own tensors of the device come from (the first one says which).  at::empty
// finds it through two dispatches: 0.75 us a tensor against 0.32.  The allocator serves the current device, which
// stream_of() has made sure of.
Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  static c10::Allocator* allocator = nullptr;
  if (allocator) return at::detail::empty_generic(shape, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
  const Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  allocator = t.storage().allocator();
  return t;
}

// The stream to use: the caller's handle, or torch's current one of the device (by the function bind() was given).
// False where the handle is none, or the device not the current one, which the library launches on.
PyObject* current_stream = nullptr;
bool stream_of(PyObject* o, c10::Device dev, void** s) {
  if (c10::impl::getDeviceGuardImpl(dev.type())->getDevice() != dev) return false;
  if (o == Py_None) {
    PyObject* index = PyLong_FromLong(dev.index());
    PyObject* handle = index ? PyObject_CallFunctionObjArgs(current_stream, index, nullptr) : nullptr;
    *s = handle ? PyLong_AsVoidPtr(handle) : nullptr;
    Py_XDECREF(index);
    Py_XDECREF(handle);
  } else {
    *s = PyLong_AsVoidPtr(o);
  }
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

PyObject* put(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  if (r)
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, put(t));
  return r;
}
PyObject* refuse() { Py_RETURN_NONE; }

// Whatever torch throws (out of memory, say) leaves as a Python error.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The interpreter lock given up for a call that uses the library's scratch: it may wait for another thread's call on the
// stream, or for the stream itself when the scratch has to grow.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

int elem_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? SK_ELEM_BF16 : t.scalar_type() == at::kFloat ? SK_ELEM_F32 : -1;
}

// quantize(x, tile, forms, stream): forms bit 0 the codes, bit 1 the transposed ones
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return refuse();
    const Arg x(v[0]);
    if (!x.t || !x.t->is_cuda() || x.t->dim() != 2 || !lib.quantize) return refuse();
    const int e = elem_of(*x.t);
    const int64_t R = x.t->size(0), C = x.t->size(1);
    const c10::Device dev = x.t->device();
    if (e < 0 || !is(*x.t, dev, x.t->scalar_type(), {R, C})) return refuse();
    const bool tile = PyLong_AsLong(v[1]) != 0;
    const long forms = PyLong_AsLong(v[2]);
    void* s;
    if (!stream_of(v[3], dev, &s)) return refuse();
    Tensor q, sc, qt, st;
    if (forms & 1) {
      q = make({R, up16(C)}, at::kFloat8_e4m3fn, dev);
      sc = make({tile ? blocks(R) : blocks(C), tile ? blocks(C) : R}, at::kFloat, dev);
    }
    if (forms & 2) {
      qt = make({C, up16(R)}, at::kFloat8_e4m3fn, dev);
      st = make({tile ? blocks(C) : blocks(R), tile ? blocks(R) : C}, at::kFloat, dev);
    }
    auto p = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const sk_status r = lib.quantize(x.ptr(), (sk_elem)e, tile ? SK_BLOCK_TILE : SK_BLOCK_ROW, p(q), (float*)p(sc), p(qt),
                                     (float*)p(st), R, C, s);
    if (r != SK_OK) return PyLong_FromLong(r);
    if (forms == 3) return pack({q, sc, qt, st});
    return forms == 2 ? pack({qt, st}) : pack({q, sc});
  });
}

// gemm(A, B, A_scale, B_scale, bias, C, grid_cap, stream)
PyObject* gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return refuse();
    const Arg a(v[0]), b(v[1]), sa(v[2]), sb(v[3]), bias(v[4]), out(v[5]);
    if (!a.t || !b.t || !sa.t || !sb.t || !a.t->is_cuda() || a.t->dim() != 2 || b.t->dim() != 2 || !lib.gemm) return refuse();
    const int64_t M = a.t->size(0), K = a.t->size(1), N = b.t->size(0), kb = blocks(K);
    const c10::Device dev = a.t->device();
    if (!is_codes(*a.t, dev, {M, K}) || !is_codes(*b.t, dev, {N, K}) || !is(*sa.t, dev, at::kFloat, {kb, M})) return refuse();
    const bool tile = is(*sb.t, dev, at::kFloat, {blocks(N), kb});
    if (!tile && !is(*sb.t, dev, at::kFloat, {kb, N})) return refuse();
    if (!none_or(bias, dev, at::kBFloat16, {N}) || !none_or(out, dev, at::kBFloat16, {M, N})) return refuse();
    const long cap = PyLong_AsLong(v[6]);
    void* s;
    if (PyErr_Occurred() || !stream_of(v[7], dev, &s)) {
      PyErr_Clear();
      return refuse();
    }
    const Tensor c = out.t ? *out.t : make({M, N}, at::kBFloat16, dev);
    const sk_status r = lib.gemm(a.ptr(), b.ptr(), (const float*)sa.ptr(), (const float*)sb.ptr(),
                                 tile ? SK_BLOCK_TILE : SK_BLOCK_ROW, bias.ptr(), c.data_ptr(), M, N, K, (int)cap, s);
    return r == SK_OK ? put(c) : PyLong_FromLong(r);
  });
}

// gemm_backward(dC, At, At_scale, Bt, Bt_scale, dbias, grid_cap, stream): dB with At, dA with Bt
PyObject* gemm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return refuse();
    const Arg d(v[0]), at(v[1]), ats(v[2]), bt(v[3]), bts(v[4]);
    if (!d.t || !d.t->is_cuda() || d.t->dim() != 2 || !lib.gemm_backward) return refuse();
    const int64_t M = d.t->size(0), N = d.t->size(1);
    const c10::Device dev = d.t->device();
    if (!is(*d.t, dev, at::kBFloat16, {M, N})) return refuse();
    if (at.bad || bt.bad || !at.t != !ats.t || !bt.t != !bts.t) return refuse();
    const Tensor* ref = bt.t ? bt.t : at.t;
    if (ref && ref->dim() != 2) return refuse();
    const int64_t K = ref ? ref->size(0) : 1;
    if (bt.t && (!is_codes(*bt.t, dev, {K, up16(N)}) || !is(*bts.t, dev, at::kFloat, {blocks(K), blocks(N)}))) return refuse();
    if (at.t && (!is_codes(*at.t, dev, {K, up16(M)}) || !is(*ats.t, dev, at::kFloat, {blocks(M), K}))) return refuse();
    const int want_bias = PyObject_IsTrue(v[5]);
    const long cap = PyLong_AsLong(v[6]);
    void* s;
    if (PyErr_Occurred() || !stream_of(v[7], dev, &s)) {
      PyErr_Clear();
      return refuse();
    }
    Tensor da, db, dbias;
    if (bt.t) da = make({M, K}, at::kBFloat16, dev);
    if (at.t) db = make({N, K}, at::kBFloat16, dev);
    if (want_bias) dbias = make({N}, at::kBFloat16, dev);
    auto p = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const sk_status r = [&] {
      const Unlocked u;
      return lib.gemm_backward(d.ptr(), at.ptr(), (const float*)ats.ptr(), bt.ptr(), (const float*)bts.ptr(), p(da), p(db),
                               p(dbias), M, N, K, (int)cap, s);
    }();
    return r == SK_OK ? pack({da, db, dbias}) : PyLong_FromLong(r);
  });
}

// Rows of a gate [G, D] or [D]; 0 without one, -1 where it is none.
int64_t gates_of(const Arg& g, c10::Device dev, at::ScalarType type, int64_t T, int64_t D) {
  if (g.bad) return -1;
  if (!g.t) return 0;
  const int64_t G = g.t->dim() == 1 ? 1 : g.t->dim() == 2 ? g.t->size(0) : -1;
  if (G < 1 || T % G) return -1;
  return (g.t->dim() == 1 ? is(*g.t, dev, type, {D}) : is(*g.t, dev, type, {G, D})) ? G : -1;
}

// norm_forward(h, residual, weight, gate, residual_scale, next_weight, eps, quantize, stream)
PyObject* norm_forward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) return refuse();
    const Arg h(v[0]), res(v[1]), w(v[2]), g(v[3]), rs(v[4]), nw(v[5]);
    if (!res.t || !res.t->is_cuda() || res.t->dim() != 2 || !lib.norm_forward) return refuse();
    const int e = elem_of(*res.t);
    const at::ScalarType ty = res.t->scalar_type();
    const int64_t T = res.t->size(0), D = res.t->size(1);
    const c10::Device dev = res.t->device();
    if (e < 0 || T < 1 || !is(*res.t, dev, ty, {T, D})) return refuse();
    if (!none_or(h, dev, ty, {T, D}) || !none_or(w, dev, ty, {D}) || !none_or(rs, dev, ty, {D}) || !none_or(nw, dev, ty, {D}))
      return refuse();
    if (!h.t != !w.t || (!h.t && !nw.t)) return refuse();
    const int64_t G = gates_of(g, dev, ty, T, D);
    const int quant = PyObject_IsTrue(v[7]);
    if (G < 0 || (quant && !nw.t)) return refuse();
    sk_norm_args a;
    std::memset(&a, 0, sizeof(a));
    a.eps = (float)PyFloat_AsDouble(v[6]);
    if (PyErr_Occurred() || !stream_of(v[8], dev, &a.stream)) {
      PyErr_Clear();
      return refuse();
    }
    a.elem = e;
    a.h = h.ptr();
    a.residual = res.ptr();
    a.weight = w.ptr();
    a.gate = g.ptr();
    a.residual_scale = rs.ptr();
    a.next_weight = nw.ptr();
    a.T = T;
    a.D = D;
    a.gates = G;
    Tensor out, rstd, y, q, sc, rn;
    if (h.t) {
      out = make({T, D}, ty, dev);
      rstd = make({T}, at::kFloat, dev);
      a.out = out.data_ptr();
      a.rstd = (float*)rstd.data_ptr();
    }
    if (nw.t) {
      rn = make({T}, at::kFloat, dev);
      a.rstd_next = (float*)rn.data_ptr();
      if (quant) {
        q = make({T, up16(D)}, at::kFloat8_e4m3fn, dev);
        sc = make({blocks(D), T}, at::kFloat, dev);
        a.q = q.data_ptr();
        a.scale = (float*)sc.data_ptr();
      } else {
        y = make({T, D}, ty, dev);
        a.y = y.data_ptr();
      }
    }
    const sk_status r = lib.norm_forward(&a);
    if (r != SK_OK) return PyLong_FromLong(r);
    if (!h.t) return quant ? pack({q, sc, rn}) : pack({y, rn});
    if (!nw.t) return pack({out, rstd});
    return quant ? pack({out, rstd, q, sc, rn}) : pack({out, rstd, y, rn});
  });
}

// norm_backward(dout, h, weight, rstd, gate, residual, residual_scale, dy, out, next_weight, rstd_next, stream):
// (dh, dresidual, dweight, dgate, dresidual_scale, dnext_weight), or (dx, dnext_weight) without h
PyObject* norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) return refuse();
    const Arg dout(v[0]), h(v[1]), w(v[2]), rstd(v[3]), g(v[4]), res(v[5]), rs(v[6]), dy(v[7]), out(v[8]), nw(v[9]), rn(v[10]);
    const Tensor* x = h.t ? h.t : out.t;
    if (!x || !x->is_cuda() || x->dim() != 2 || !lib.norm_backward) return refuse();
    const int e = elem_of(*x);
    const at::ScalarType ty = x->scalar_type();
    const int64_t T = x->size(0), D = x->size(1);
    const c10::Device dev = x->device();
    if (e < 0 || T < 1) return refuse();
    for (const Arg* t : {&dout, &h, &dy, &out})
      if (!none_or(*t, dev, ty, {T, D})) return refuse();
    for (const Arg* t : {&w, &rs, &nw})
      if (!none_or(*t, dev, ty, {D})) return refuse();
    if (!none_or(rstd, dev, at::kFloat, {T}) || !none_or(rn, dev, at::kFloat, {T}) || res.bad) return refuse();
    if (h.t ? !dout.t || !w.t || !rstd.t : !dy.t || w.t || rstd.t || rs.t || g.t) return refuse();
    if (dy.t ? !out.t || !nw.t || !rn.t : out.t || nw.t || rn.t) return refuse();
    if (rs.t && (!res.t || !is(*res.t, dev, ty, {T, D}))) return refuse();
    const int64_t G = gates_of(g, dev, ty, T, D);
    sk_norm_grad_args a;
    std::memset(&a, 0, sizeof(a));
    if (G < 0 || !stream_of(v[11], dev, &a.stream)) return refuse();
    a.elem = e;
    a.dout = dout.ptr();
    a.dy = dy.ptr();
    a.out = out.ptr();
    a.next_weight = nw.ptr();
    a.rstd_next = (const float*)rn.ptr();
    a.h = h.ptr();
    a.residual = rs.t ? res.ptr() : nullptr;
    a.weight = w.ptr();
    a.gate = g.ptr();
    a.residual_scale = rs.ptr();
    a.rstd = (const float*)rstd.ptr();
    a.T = T;
    a.D = D;
    a.gates = G;
    const Tensor dx = make({T, D}, ty, dev);
    Tensor dres, dw, dgate, drs, dnw;
    a.dx = dx.data_ptr();
    if (h.t) {
      dres = make({T, D}, ty, dev);
      dw = make({D}, ty, dev);
      a.dresidual = dres.data_ptr();
      a.dweight = dw.data_ptr();
      if (g.t) {
        dgate = at::empty_like(*g.t);
        a.dgate = dgate.data_ptr();
      }
      if (rs.t) {
        drs = make({D}, ty, dev);
        a.dresidual_scale = drs.data_ptr();
      }
    }
    if (dy.t) {
      dnw = make({D}, ty, dev);
      a.dnext_weight = dnw.data_ptr();
    }
    const sk_status r = [&] {
      const Unlocked u;
      return lib.norm_backward(&a);
    }();
    if (r != SK_OK) return PyLong_FromLong(r);
    return h.t ? pack({dx, dres, dw, dgate, drs, dnw}) : pack({dx, dnw});
  });
}

// bind(quantize, gemm, gemm_backward, norm_forward, norm_backward, current_stream): the library's entry points, as
// addresses, and the function that gives a device's current stream handle
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses and a function");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) p[i] = PyLong_AsVoidPtr(v[i]);
  if (PyErr_Occurred()) return nullptr;
  Py_INCREF(v[5]);
  Py_XDECREF(current_stream);
  current_stream = v[5];
  lib.quantize = (decltype(lib.quantize))p[0];
  lib.gemm = (decltype(lib.gemm))p[1];
  lib.gemm_backward = (decltype(lib.gemm_backward))p[2];
  lib.norm_forward = (decltype(lib.norm_forward))p[3];
  lib.norm_backward = (decltype(lib.norm_backward))p[4];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void*)F, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<quantize>("quantize"),         method<gemm>("gemm"),
                         method<gemm_backward>("gemm_backward"), method<norm_forward>("norm_forward"),
                         method<norm_backward>("norm_backward"), method<bind>("bind"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sknative", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sknative() { return PyModule_Create(&module); }
