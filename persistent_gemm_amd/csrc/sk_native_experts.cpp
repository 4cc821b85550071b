// The native binding's calls of a layer of experts, under the same rules as the others (sk_native.cpp): arguments that are all as
// they should be, on the current device and its current stream; for any other call None, and the binding's own checks say why.

#include "sk_native.h"

namespace {

using namespace sk_native;

struct Library {
  decltype(&sk_moe_route_work_bytes) route_work_bytes = nullptr;
  decltype(&sk_moe_route) route = nullptr;
  decltype(&sk_moe_route_backward) route_backward = nullptr;
  decltype(&sk_moe_combine) combine = nullptr;
  decltype(&sk_moe_combine_backward) combine_backward = nullptr;
  decltype(&sk_gemm_grouped) grouped = nullptr;
  decltype(&sk_gemm_grouped_backward) grouped_backward = nullptr;
  decltype(&sk_quantize_w4) quantize = nullptr;
  decltype(&sk_dequantize_w4) dequantize = nullptr;
  decltype(&sk_gemm_w4) w4 = nullptr;
} lib;

constexpr at::ScalarType kInt = at::kInt, kFloat = at::kFloat, kByte = at::kByte;

int elem_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SK_ELEM_BF16;
    case at::kHalf: return SK_ELEM_F16;
    case at::kFloat: return SK_ELEM_F32;
    default: return -1;
  }
}
int half_of(const Tensor& t) {
  const int e = elem_of(t);
  return e == SK_ELEM_F32 ? -1 : e;
}
bool on_gpu(const Arg& a, int64_t dims) { return a.t && a.t->is_cuda() && a.t->dim() == dims; }
// A truth value; false where it has none (a tensor of several elements, say), which the binding's own call then reports.
bool truth(PyObject* o, bool* b) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) PyErr_Clear();
  *b = t > 0;
  return t >= 0;
}
// The current stream, or false.
bool here(c10::Device dev, void** s) { return stream_of(Py_None, dev, s); }
void* p(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* status(sk_status r) { return PyLong_FromLong(r); }

// moe_route(logits, k, normalize)
PyObject* route(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3 || !lib.route) return refuse();
    const Arg x(v[0]);
    if (!on_gpu(x, 2) || !PyLong_CheckExact(v[1])) return refuse();
    bool normalize;
    if (!truth(v[2], &normalize)) return refuse();
    const int e = elem_of(*x.t);
    const int64_t T = x.t->size(0), E = x.t->size(1), k = PyLong_AsLong(v[1]);
    const c10::Device dev = x.t->device();
    void* s;
    if (PyErr_Occurred() || e < 0 || T < 1 || k < 1 || k > 32 || k > E || !x.t->is_contiguous() || !here(dev, &s)) {
      PyErr_Clear();
      return refuse();
    }
    const Tensor experts = make({T, k}, kInt, dev), weights = make({T, k}, kFloat, dev), offsets = make({E + 1}, kInt, dev),
                 slots = make({T, k}, kInt, dev), rows = make({T * k}, kInt, dev);
    const int64_t bytes = lib.route_work_bytes(T, E);
    const Tensor work = bytes ? make({bytes / 4}, kInt, dev) : Tensor();
    const sk_status r = lib.route(x.ptr(), (sk_elem)e, normalize, (int32_t*)p(experts), (float*)p(weights), (int32_t*)p(offsets),
                                  (int32_t*)p(slots), (int32_t*)p(rows), p(work), T, E, k, s);
    return r == SK_OK ? pack({experts, weights, offsets, slots, rows}) : status(r);
  });
}

// moe_route_backward(dweights, logits, experts, weights, normalize)
PyObject* route_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5 || !lib.route_backward) return refuse();
    const Arg d(v[0]), x(v[1]), ids(v[2]), w(v[3]);
    if (!on_gpu(x, 2) || !on_gpu(d, 2) || !ids.t || !w.t) return refuse();
    bool normalize;
    if (!truth(v[4], &normalize)) return refuse();
    const int e = elem_of(*x.t);
    const int64_t T = x.t->size(0), E = x.t->size(1), k = d.t->size(1);
    const c10::Device dev = x.t->device();
    void* s;
    if (e < 0 || !x.t->is_contiguous() || !is(*d.t, dev, kFloat, {T, k}) || !is(*w.t, dev, kFloat, {T, k}) ||
        !is(*ids.t, dev, kInt, {T, k}) || !here(dev, &s))
      return refuse();
    const Tensor out = make({T, E}, x.t->scalar_type(), dev);
    const sk_status r = lib.route_backward((const float*)d.ptr(), x.ptr(), (sk_elem)e, normalize, (const int32_t*)ids.ptr(),
                                           (const float*)w.ptr(), p(out), T, E, k, s);
    return r == SK_OK ? put(out) : status(r);
  });
}

// moe_combine(y, slots, weights)
PyObject* combine(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3 || !lib.combine) return refuse();
    const Arg y(v[0]), slots(v[1]), w(v[2]);
    if (!on_gpu(y, 2) || !on_gpu(slots, 2)) return refuse();
    const int e = elem_of(*y.t);
    const int64_t R = y.t->size(0), D = y.t->size(1), T = slots.t->size(0), k = slots.t->size(1);
    const c10::Device dev = y.t->device();
    void* s;
    if (e < 0 || !y.t->is_contiguous() || !is(*slots.t, dev, kInt, {T, k}) || !none_or(w, dev, kFloat, {T, k}) || !here(dev, &s))
      return refuse();
    const Tensor out = make({T, D}, y.t->scalar_type(), dev);
    const sk_status r = lib.combine(y.ptr(), (sk_elem)e, (const int32_t*)slots.ptr(), (const float*)w.ptr(), p(out), T, k, R, D, s);
    return r == SK_OK ? put(out) : status(r);
  });
}

// moe_combine_backward(dout, y, slots, weights, offsets)
PyObject* combine_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5 || !lib.combine_backward) return refuse();
    const Arg d(v[0]), y(v[1]), slots(v[2]), w(v[3]), o(v[4]);
    if (!on_gpu(y, 2) || !on_gpu(slots, 2) || !d.t || o.bad || (o.t && o.t->dim() != 1)) return refuse();
    const int e = elem_of(*y.t);
    const int64_t R = y.t->size(0), D = y.t->size(1), T = slots.t->size(0), k = slots.t->size(1);
    const int64_t E = o.t ? o.t->size(0) - 1 : 0;
    const c10::Device dev = y.t->device();
    void* s;
    if (e < 0 || !y.t->is_contiguous() || !is(*d.t, dev, y.t->scalar_type(), {T, D}) || !is(*slots.t, dev, kInt, {T, k}) ||
        !none_or(w, dev, kFloat, {T, k}) || !none_or(o, dev, kInt, {E + 1}) || !here(dev, &s))
      return refuse();
    const Tensor dy = make({R, D}, y.t->scalar_type(), dev);
    const Tensor dw = w.t ? make({T, k}, kFloat, dev) : Tensor();
    const sk_status r = lib.combine_backward(d.ptr(), y.ptr(), (sk_elem)e, (const int32_t*)slots.ptr(), (const float*)w.ptr(),
                                             (const int32_t*)o.ptr(), p(dy), (float*)p(dw), T, k, R, D, E, s);
    return r == SK_OK ? pack({dy, dw}) : status(r);
  });
}

// Rows of a product by expert, or -1: those of `rows`, or A's T.
int64_t rows_of(const Arg& offsets, const Arg& rows, int64_t T, int64_t E, c10::Device dev) {
  if (!offsets.t || !is(*offsets.t, dev, kInt, {E + 1}) || rows.bad) return -1;
  if (!rows.t) return T;
  return rows.t->dim() == 1 && is(*rows.t, dev, kInt, {rows.t->size(0)}) ? rows.t->size(0) : -1;
}

// gemm_grouped(A, B, offsets, bias, rows, out)
PyObject* grouped(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6 || !lib.grouped) return refuse();
    const Arg a(v[0]), b(v[1]), o(v[2]), bias(v[3]), rows(v[4]), out(v[5]);
    if (!on_gpu(a, 2) || !on_gpu(b, 3)) return refuse();
    const int e = half_of(*a.t);
    const at::ScalarType ty = a.t->scalar_type();
    const int64_t T = a.t->size(0), K = a.t->size(1), E = b.t->size(0), N = b.t->size(1);
    const c10::Device dev = a.t->device();
    const int64_t R = rows_of(o, rows, T, E, dev);
    void* s;
    if (e < 0 || R < 0 || !a.t->is_contiguous() || !is(*b.t, dev, ty, {E, N, K}) || !none_or(bias, dev, ty, {E, N}) ||
        !none_or(out, dev, ty, {R, N}) || !here(dev, &s))
      return refuse();
    const Tensor c = out.t ? *out.t : make({R, N}, ty, dev);
    const sk_status r = lib.grouped(a.ptr(), b.ptr(), (sk_elem)e, (const int32_t*)o.ptr(), (const int32_t*)rows.ptr(), bias.ptr(),
                                    c.data_ptr(), R, T, E, N, K, out.t ? 0 : 1, s);
    return r == SK_OK ? put(c) : status(r);
  });
}

// gemm_grouped_backward(dC, A, B, offsets, rows, need_dA, need_dB, need_dbias)
PyObject* grouped_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8 || !lib.grouped_backward) return refuse();
    const Arg d(v[0]), a(v[1]), b(v[2]), o(v[3]), rows(v[4]);
    if (!on_gpu(a, 2) || !on_gpu(b, 3) || !d.t) return refuse();
    const int e = half_of(*a.t);
    const at::ScalarType ty = a.t->scalar_type();
    const int64_t T = a.t->size(0), K = a.t->size(1), E = b.t->size(0), N = b.t->size(1);
    const c10::Device dev = a.t->device();
    const int64_t R = rows_of(o, rows, T, E, dev);
    bool wa, wb, ws;
    void* s;
    if (!truth(v[5], &wa) || !truth(v[6], &wb) || !truth(v[7], &ws) || e < 0 || R < 0 || !(wa || wb || ws) || !a.t->is_contiguous() || !is(*b.t, dev, ty, {E, N, K}) ||
        !is(*d.t, dev, ty, {R, N}) || !here(dev, &s))
      return refuse();
    const Tensor da = wa ? make({R, K}, ty, dev) : Tensor(), db = wb ? make({E, N, K}, ty, dev) : Tensor(),
                 dbias = ws ? make({E, N}, ty, dev) : Tensor();
    const sk_status r = lib.grouped_backward(d.ptr(), a.ptr(), b.ptr(), (sk_elem)e, (const int32_t*)o.ptr(),
                                             (const int32_t*)rows.ptr(), p(da), p(db), p(dbias), R, T, E, N, K, s);
    return r == SK_OK ? pack({da, db, dbias}) : status(r);
  });
}

// 4-bit codes [N, K / 2] or [E, N, K / 2] with scales and zero points: their sizes, or false.
struct Codes {
  int64_t E = 1, N = 0, K = 0, group = 0;
  bool by_expert = false;
  bool read(const Arg& q, const Arg& scale, const Arg& zero) {
    if (!q.t || !q.t->is_cuda() || (q.t->dim() != 2 && q.t->dim() != 3) || !scale.t || scale.t->dim() != q.t->dim()) return false;
    const c10::Device dev = q.t->device();
    by_expert = q.t->dim() == 3;
    if (by_expert) E = q.t->size(0);
    N = q.t->size(-2);
    K = 2 * q.t->size(-1);
    const int64_t groups = scale.t->size(-2);
    if (groups < 1 || K % groups) return false;
    group = K / groups;
    if (group != 32 && group != 64 && group != 128) return false;
    const at::ScalarType ty = scale.t->scalar_type();
    return q.t->scalar_type() == kByte && q.t->is_contiguous() &&
           (by_expert ? is(*scale.t, dev, ty, {E, groups, N}) && none_or(zero, dev, kByte, {E, groups, N})
                      : is(*scale.t, dev, ty, {groups, N}) && none_or(zero, dev, kByte, {groups, N}));
  }
};

// gemm_w4(x, q, scale, zero, bias, offsets, rows, out)
PyObject* w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8 || !lib.w4) return refuse();
    const Arg x(v[0]), q(v[1]), scale(v[2]), zero(v[3]), bias(v[4]), o(v[5]), rows(v[6]), out(v[7]);
    Codes c;
    if (!on_gpu(x, 2) || !c.read(q, scale, zero) || o.bad || rows.bad || c.by_expert != (o.t != nullptr) || (rows.t && !o.t)) return refuse();
    const int e = half_of(*x.t);
    const at::ScalarType ty = x.t->scalar_type();
    const int64_t T = x.t->size(0), K = x.t->size(1);
    const c10::Device dev = x.t->device();
    const int64_t R = o.t ? rows_of(o, rows, T, c.E, dev) : T;
    void* s;
    if (e < 0 || R < 0 || c.K != K || q.t->device() != dev || scale.t->scalar_type() != ty || !x.t->is_contiguous() ||
        !(c.by_expert ? none_or(bias, dev, ty, {c.E, c.N}) : none_or(bias, dev, ty, {c.N})) ||
        !none_or(out, dev, ty, {R, c.N}) || !here(dev, &s))
      return refuse();
    const Tensor y = out.t ? *out.t : make({R, c.N}, ty, dev);
    const sk_status r = lib.w4(x.ptr(), q.ptr(), scale.ptr(), (const uint8_t*)zero.ptr(), (sk_elem)e, (const int32_t*)o.ptr(),
                               (const int32_t*)rows.ptr(), bias.ptr(), y.data_ptr(), R, T, c.E, c.N, K, c.group, out.t ? 0 : 1, s);
    return r == SK_OK ? put(y) : status(r);
  });
}

// quantize_w4(w, group, zero, scales of fp16): w [N, K] or [E, N, K]
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4 || !lib.quantize) return refuse();
    const Arg w(v[0]);
    if (!w.t || !w.t->is_cuda() || (w.t->dim() != 2 && w.t->dim() != 3) || !PyLong_CheckExact(v[1])) return refuse();
    const int e = elem_of(*w.t);
    bool half, zeros;
    if (!truth(v[2], &zeros) || !truth(v[3], &half)) return refuse();
    const bool lead = w.t->dim() == 3;
    const int64_t E = lead ? w.t->size(0) : 1, N = w.t->size(-2), K = w.t->size(-1), group = PyLong_AsLong(v[1]);
    const c10::Device dev = w.t->device();
    void* s;
    if (PyErr_Occurred() || e < 0 || (group != 32 && group != 64 && group != 128) || K % group || !w.t->is_contiguous() || !here(dev, &s)) {
      PyErr_Clear();
      return refuse();
    }
    const at::ScalarType ty = half ? at::kHalf : at::kBFloat16;
    const int64_t groups = K / group;
    const Tensor q = lead ? make({E, N, K / 2}, kByte, dev) : make({N, K / 2}, kByte, dev);
    const Tensor scale = lead ? make({E, groups, N}, ty, dev) : make({groups, N}, ty, dev);
    Tensor zero;
    if (zeros) zero = lead ? make({E, groups, N}, kByte, dev) : make({groups, N}, kByte, dev);
    const sk_status r = lib.quantize(w.ptr(), (sk_elem)e, p(q), p(scale), half ? SK_ELEM_F16 : SK_ELEM_BF16, (uint8_t*)p(zero), E, N, K,
                                     group, s);
    return r == SK_OK ? pack({q, scale, zero}) : status(r);
  });
}

// dequantize_w4(q, scale, zero)
PyObject* dequantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3 || !lib.dequantize) return refuse();
    const Arg q(v[0]), scale(v[1]), zero(v[2]);
    Codes c;
    if (!c.read(q, scale, zero)) return refuse();
    const int e = half_of(*scale.t);
    const c10::Device dev = q.t->device();
    void* s;
    if (e < 0 || !here(dev, &s)) return refuse();
    const at::ScalarType ty = scale.t->scalar_type();
    const Tensor out = c.by_expert ? make({c.E, c.N, c.K}, ty, dev) : make({c.N, c.K}, ty, dev);
    const sk_status r = lib.dequantize(q.ptr(), scale.ptr(), (sk_elem)e, (const uint8_t*)zero.ptr(), p(out), c.E, c.N, c.K, c.group, s);
    return r == SK_OK ? put(out) : status(r);
  });
}

// bind_experts(address of each entry point, in Library's order)
PyObject* bind_experts(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "bind_experts takes ten addresses");
    return nullptr;
  }
  void* a[10];
  for (int i = 0; i < 10; ++i) a[i] = PyLong_AsVoidPtr(v[i]);
  if (PyErr_Occurred()) return nullptr;
  lib.route_work_bytes = (decltype(lib.route_work_bytes))a[0];
  lib.route = (decltype(lib.route))a[1];
  lib.route_backward = (decltype(lib.route_backward))a[2];
  lib.combine = (decltype(lib.combine))a[3];
  lib.combine_backward = (decltype(lib.combine_backward))a[4];
  lib.grouped = (decltype(lib.grouped))a[5];
  lib.grouped_backward = (decltype(lib.grouped_backward))a[6];
  lib.quantize = (decltype(lib.quantize))a[7];
  lib.dequantize = (decltype(lib.dequantize))a[8];
  lib.w4 = (decltype(lib.w4))a[9];
  Py_RETURN_NONE;
}

}  // namespace

namespace sk_native {
PyMethodDef experts_methods[] = {method<route>("moe_route"),
                                 method<route_backward>("moe_route_backward"),
                                 method<combine>("moe_combine"),
                                 method<combine_backward>("moe_combine_backward"),
                                 method<grouped>("gemm_grouped"),
                                 method<grouped_backward>("gemm_grouped_backward"),
                                 method<w4>("gemm_w4"),
                                 method<quantize>("quantize_w4"),
                                 method<dequantize>("dequantize_w4"),
                                 method<bind_experts>("bind_experts"),
                                 {nullptr, nullptr, 0, nullptr}};
}
