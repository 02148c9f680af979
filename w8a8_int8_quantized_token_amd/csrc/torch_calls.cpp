// The plain calls of block_ops.py and adapter_ops.py in one native step.  Through Python checks
// and ctypes a call of these entry points costs 9 to 25 us of host time, more
// than many of them run for; here it costs a third of that.
//
// Each function takes the call's arguments as Python objects, and does the
// call if it is an ordinary one: contiguous tensors of the right types and
// sizes on the current device.  Anything else (a wrong argument, another
// device, an error status, an exception) gives None with nothing launched, and
// the caller goes through the Python checks, which name what is wrong or
// make the call.  Work is enqueued on torch's current stream; outputs and
// workspaces come from torch's allocator.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include "../../include/w8a8.h"

namespace {

struct Refused {};   // not a plain call

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{};
  return THPVariable_Unpack(o);
}

// A call's device, stream and workspace.
struct Call {
  int device;
  hipStream_t stream;
  at::Tensor space;

  explicit Call(const at::Tensor& first) {
    if (!first.is_cuda()) throw Refused{};
    device = first.get_device();
    if (device != c10::hip::current_device()) throw Refused{};
    stream = c10::hip::getCurrentHIPStream(device).stream();
  }
  void check(const at::Tensor& t, at::ScalarType type) const {
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.layout() != at::kStrided) throw Refused{};
  }
  // The address of a contiguous tensor of that type and shape.
  template <class T>
  T* at(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(o);
    check(t, type);
    if (t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) throw Refused{};
    return static_cast<T*>(t.data_ptr());
  }
  template <class T>
  T* at_or_null(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : at<T>(o, type, shape);
  }
  at::Tensor empty(std::initializer_list<int64_t> shape, at::ScalarType type) const {
    return at::empty(at::IntArrayRef(shape), at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
  }
  void* workspace(size_t bytes) {
    if (bytes == 0) return nullptr;
    space = empty({(int64_t)bytes}, at::kByte);
    return space.data_ptr();
  }
};

uint16_t* bits(const at::Tensor& t) { return t.defined() ? static_cast<uint16_t*>(t.data_ptr()) : nullptr; }
PyObject* wrap(at::Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
bool flag(PyObject* o) {
  if (o == Py_True) return true;
  if (o == Py_False) return false;
  throw Refused{};
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if ((v == -1 && PyErr_Occurred()) || v < INT_MIN || v > INT_MAX) throw Refused{};
  return (int)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}
void two_dims(const at::Tensor& t) {
  if (t.dim() != 2) throw Refused{};
}
void launched(w8a8_status s) {
  if (s != W8A8_OK) throw Refused{};
}

// None in the place of everything that is not a plain call.
template <class F>
PyObject* plain(Py_ssize_t have, Py_ssize_t want, F f) {
  if (have == want) {
    try {
      return f();
    } catch (...) {
      PyErr_Clear();
    }
  }
  Py_RETURN_NONE;
}

// x, wq, w_scale, bias, gelu or act, rows of wq per channel
PyObject* dynamic(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 6, [&] {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]);
    two_dims(x);
    two_dims(w);
    Call c(x);
    const int act = integer(a[4]), per = integer(a[5]);
    const int64_t M = x.size(0), K = x.size(1), rows = w.size(0), N = rows / per;
    if (rows % per) throw Refused{};
    const auto* px = c.at<uint16_t>(a[0], at::kBFloat16, {M, K});
    const auto* pw = c.at<int8_t>(a[1], at::kChar, {rows, K});
    const auto* ps = c.at<float>(a[2], at::kFloat, {rows});
    const auto* pb = c.at_or_null<uint16_t>(a[3], at::kBFloat16, {rows});
    at::Tensor y = c.empty({M, N}, at::kBFloat16);
    const size_t need = per == 1 ? w8a8_linear_dynamic_workspace(M, N, K) : w8a8_gated_linear_dynamic_workspace(M, N, K);
    void* ws = c.workspace(need);
    launched(per == 1 ? w8a8_linear_dynamic(px, pw, ps, pb, bits(y), M, N, K, act, ws, need, c.stream)
                      : w8a8_gated_linear_dynamic(px, pw, ps, pb, bits(y), M, N, K, act, ws, need, c.stream));
    return wrap(std::move(y));
  });
}

// dy, xq, x_scale, wq, w_scale, bias, act (-1: the linear), dx, dw, dbias
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 10, [&] {
    const at::Tensor &dy = tensor(a[0]), &w = tensor(a[3]);
    two_dims(dy);
    two_dims(w);
    Call c(dy);
    const int act = integer(a[6]), per = act < 0 ? 1 : 2;
    const bool dx = flag(a[7]), dw = flag(a[8]), db = flag(a[9]);
    const int64_t M = dy.size(0), N = dy.size(1), K = w.size(1), rows = per * N;
    const auto* pdy = c.at<uint16_t>(a[0], at::kBFloat16, {M, N});
    const bool no_x = per == 1 && !dw && a[1] == Py_None && a[2] == Py_None;
    const auto* pxq = no_x ? nullptr : c.at<int8_t>(a[1], at::kChar, {M, K});
    const auto* pxs = no_x ? nullptr : c.at<float>(a[2], at::kFloat, {M});
    const auto* pw = c.at<int8_t>(a[3], at::kChar, {rows, K});
    const auto* ps = c.at<float>(a[4], at::kFloat, {rows});
    const auto* pb = c.at_or_null<uint16_t>(a[5], at::kBFloat16, {rows});
    at::Tensor gx, gw, gb;
    if (dx) gx = c.empty({M, K}, at::kBFloat16);
    if (dw) gw = c.empty({rows, K}, at::kBFloat16);
    if (db) gb = c.empty({rows}, at::kBFloat16);
    const size_t need = per == 1 ? w8a8_linear_backward_workspace(M, N, K, dx, dw, db)
                                 : w8a8_gated_linear_backward_workspace(M, N, K, dx, dw, db);
    void* ws = c.workspace(need);
    launched(per == 1 ? w8a8_linear_backward(pdy, pxq, pxs, pw, ps, bits(gx), bits(gw), bits(gb), M, N, K, ws, need, c.stream)
                      : w8a8_gated_linear_backward(pdy, pxq, pxs, pw, ps, pb, bits(gx), bits(gw), bits(gb), M, N, K, act,
                                                   ws, need, c.stream));
    return tuple({std::move(gx), std::move(gw), std::move(gb)});
  });
}

// bf16 [M, heads, D], dense along D
struct Heads {
  const uint16_t* p;
  int64_t row, head;
  Heads(const Call& c, const at::Tensor& t, int64_t M, int64_t H, int64_t D) {
    c.check(t, at::kBFloat16);
    if (t.dim() != 3 || t.size(0) != M || t.size(1) != H || t.size(2) != D || t.stride(2) != 1) throw Refused{};
    p = static_cast<const uint16_t*>(t.data_ptr());
    row = M > 1 ? t.stride(0) : 0;
    head = H > 1 ? t.stride(1) : 0;
  }
};
struct Rope {
  int64_t M, Hq, Hk, D, P, half;
  const uint16_t *qw, *kw;
  const float *cos, *sin;
  const int32_t* positions;
  float eps;
  int interleaved;
  // q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved
  Rope(const Call& c, PyObject* const* a) {
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &t = tensor(a[4]);
    if (q.dim() != 3 || k.dim() != 3) throw Refused{};
    two_dims(t);
    M = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1), P = t.size(0), half = t.size(1);
    qw = c.at_or_null<uint16_t>(a[2], at::kBFloat16, {D});
    kw = c.at_or_null<uint16_t>(a[3], at::kBFloat16, {D});
    cos = c.at<float>(a[4], at::kFloat, {P, half});
    sin = c.at<float>(a[5], at::kFloat, {P, half});
    positions = c.at_or_null<int32_t>(a[6], at::kInt, {M});
    eps = real(a[7]);
    interleaved = flag(a[8]);
  }
};

// q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 9, [&] {
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]);
    Call c(q);
    const Rope r(c, a);
    const Heads vq(c, q, r.M, r.Hq, r.D), vk(c, k, r.M, r.Hk, r.D);
    at::Tensor oq = c.empty({r.M, r.Hq, r.D}, at::kBFloat16), ok = c.empty({r.M, r.Hk, r.D}, at::kBFloat16);
    launched(w8a8_qk_norm_rope(vq.p, vq.row, vq.head, vk.p, vk.row, vk.head, r.qw, r.kw, r.cos, r.sin, r.positions,
                               bits(oq), r.Hq * r.D, r.D, bits(ok), r.Hk * r.D, r.D, r.M, r.P, r.Hq, r.Hk, r.D,
                               2 * r.half, r.eps, r.interleaved, c.stream));
    return tuple({std::move(oq), std::move(ok)});
  });
}

// q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, dq, dk, weights
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 12, [&] {
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]);
    Call c(q);
    const Rope r(c, a);
    const Heads vq(c, q, r.M, r.Hq, r.D), vk(c, k, r.M, r.Hk, r.D);
    const Heads dq(c, tensor(a[9]), r.M, r.Hq, r.D), dk(c, tensor(a[10]), r.M, r.Hk, r.D);
    const bool weights = flag(a[11]);
    at::Tensor gq = c.empty({r.M, r.Hq, r.D}, at::kBFloat16), gk = c.empty({r.M, r.Hk, r.D}, at::kBFloat16);
    at::Tensor gqw, gkw;
    size_t need = 0;
    if (weights) {
      gqw = c.empty({r.D}, at::kFloat);
      gkw = c.empty({r.D}, at::kFloat);
      need = w8a8_qk_norm_rope_backward_workspace(r.M, r.Hq, r.Hk, r.D);
    }
    void* ws = c.workspace(need);
    launched(w8a8_qk_norm_rope_backward(
        dq.p, dq.row, dq.head, dk.p, dk.row, dk.head, vq.p, vq.row, vq.head, vk.p, vk.row, vk.head, r.qw, r.kw, r.cos,
        r.sin, r.positions, bits(gq), r.Hq * r.D, r.D, bits(gk), r.Hk * r.D, r.D,
        weights ? static_cast<float*>(gqw.data_ptr()) : nullptr, weights ? static_cast<float*>(gkw.data_ptr()) : nullptr,
        r.M, r.P, r.Hq, r.Hk, r.D, 2 * r.half, r.eps, r.interleaved, ws, need, c.stream));
    return tuple({std::move(gq), std::move(gk), std::move(gqw), std::move(gkw)});
  });
}

// x, residual, weight, eps, fp8
PyObject* add_rms_norm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 5, [&] {
    const at::Tensor& x = tensor(a[0]);
    two_dims(x);
    Call c(x);
    const int64_t M = x.size(0), K = x.size(1);
    const auto* px = c.at<uint16_t>(a[0], at::kBFloat16, {M, K});
    const auto* pr = c.at_or_null<uint16_t>(a[1], at::kBFloat16, {M, K});
    const auto* pw = c.at_or_null<uint16_t>(a[2], at::kBFloat16, {K});
    const float eps = real(a[3]);
    const bool fp8 = flag(a[4]);
    at::Tensor q = c.empty({M, K}, fp8 ? at::kByte : at::kChar), s = c.empty({M}, at::kFloat), h;
    if (pr != nullptr) h = c.empty({M, K}, at::kBFloat16);
    launched(w8a8_add_rms_norm_quantize(px, pr, pw, bits(h), q.data_ptr(), static_cast<float*>(s.data_ptr()), M, K, eps,
                                        fp8, c.stream));
    return tuple({std::move(q), std::move(s), pr != nullptr ? std::move(h) : x});
  });
}

// dn, h, weight, eps, dh, whether dweight
PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 6, [&] {
    const at::Tensor& h = tensor(a[1]);
    two_dims(h);
    Call c(h);
    const int64_t M = h.size(0), K = h.size(1);
    const auto* pdn = c.at<uint16_t>(a[0], at::kBFloat16, {M, K});
    const auto* ph = c.at<uint16_t>(a[1], at::kBFloat16, {M, K});
    const auto* pw = c.at_or_null<uint16_t>(a[2], at::kBFloat16, {K});
    const float eps = real(a[3]);
    const auto* pdh = c.at_or_null<uint16_t>(a[4], at::kBFloat16, {M, K});
    at::Tensor dx = c.empty({M, K}, at::kBFloat16), dw;
    size_t need = 0;
    if (flag(a[5])) {
      dw = c.empty({K}, at::kFloat);
      need = w8a8_add_rms_norm_backward_workspace(M, K);
    }
    void* ws = c.workspace(need);
    launched(w8a8_add_rms_norm_backward(pdn, pdh, ph, pw, bits(dx), dw.defined() ? static_cast<float*>(dw.data_ptr()) : nullptr,
                                        M, K, eps, ws, need, c.stream));
    return tuple({std::move(dx), std::move(dw)});
  });
}

// The adapters of a call: a, b, ids, scaling
struct Adapters {
  int64_t R, L;
  const uint16_t *a, *b;
  const int32_t* ids;
  const float* scaling;
  Adapters(const Call& c, PyObject* const* o, int64_t M, int64_t N, int64_t K) {
    const at::Tensor& t = tensor(o[0]);
    if (t.dim() != 3) throw Refused{};
    L = t.size(0), R = t.size(1);
    a = c.at<uint16_t>(o[0], at::kBFloat16, {L, R, K});
    b = c.at<uint16_t>(o[1], at::kBFloat16, {L, N, R});
    ids = c.at<int32_t>(o[2], at::kInt, {M});
    scaling = c.at<float>(o[3], at::kFloat, {L});
  }
};

// x or xq, x_scale or None (x is bf16), wq, w_scale, bias, a, b, ids, scaling
PyObject* linear_adapters(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 9, [&] {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[2]);
    two_dims(x);
    two_dims(w);
    Call c(x);
    const bool dynamic = a[1] == Py_None;
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const uint16_t* px = dynamic ? c.at<uint16_t>(a[0], at::kBFloat16, {M, K}) : nullptr;
    const int8_t* pq = dynamic ? nullptr : c.at<int8_t>(a[0], at::kChar, {M, K});
    const float* pxs = c.at_or_null<float>(a[1], at::kFloat, {M});
    const auto* pw = c.at<int8_t>(a[2], at::kChar, {N, K});
    const auto* ps = c.at<float>(a[3], at::kFloat, {N});
    const auto* pb = c.at_or_null<uint16_t>(a[4], at::kBFloat16, {N});
    const Adapters ad(c, a + 5, M, N, K);
    at::Tensor y = c.empty({M, N}, at::kBFloat16);
    const size_t need = w8a8_linear_adapters_workspace(M, N, K, ad.R, dynamic);
    void* ws = c.workspace(need);
    launched(dynamic ? w8a8_linear_adapters_dynamic(px, pw, ps, pb, ad.a, ad.b, ad.scaling, ad.ids, bits(y), M, N, K, ad.R,
                                                    ad.L, ws, need, c.stream)
                     : w8a8_linear_adapters(pq, pxs, pw, ps, pb, ad.a, ad.b, ad.scaling, ad.ids, bits(y), M, N, K, ad.R,
                                            ad.L, -1, ws, need, c.stream));
    return wrap(std::move(y));
  });
}

// dy, xq, x_scale, wq, w_scale, a, b, ids, scaling, dx, da, db
PyObject* linear_adapters_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 12, [&] {
    const at::Tensor &dy = tensor(a[0]), &w = tensor(a[3]);
    two_dims(dy);
    two_dims(w);
    Call c(dy);
    const bool dx = flag(a[9]), da = flag(a[10]), db = flag(a[11]);
    const int64_t M = dy.size(0), N = dy.size(1), K = w.size(1);
    const auto* pdy = c.at<uint16_t>(a[0], at::kBFloat16, {M, N});
    const bool no_x = !da && !db && a[1] == Py_None && a[2] == Py_None;
    const auto* pxq = no_x ? nullptr : c.at<int8_t>(a[1], at::kChar, {M, K});
    const auto* pxs = no_x ? nullptr : c.at<float>(a[2], at::kFloat, {M});
    const auto* pw = c.at<int8_t>(a[3], at::kChar, {N, K});
    const auto* ps = c.at<float>(a[4], at::kFloat, {N});
    const Adapters ad(c, a + 5, M, N, K);
    at::Tensor gx, ga, gb;
    if (dx) gx = c.empty({M, K}, at::kBFloat16);
    if (da) ga = c.empty({ad.L, ad.R, K}, at::kBFloat16);
    if (db) gb = c.empty({ad.L, N, ad.R}, at::kBFloat16);
    const size_t need = w8a8_linear_adapters_backward_workspace(M, N, K, ad.R, ad.L, dx, da, db);
    void* ws = c.workspace(need);
    launched(w8a8_linear_adapters_backward(pdy, pxq, pxs, pw, ps, ad.a, ad.b, ad.scaling, ad.ids, bits(gx), bits(ga),
                                           bits(gb), M, N, K, ad.R, ad.L, ws, need, c.stream));
    return tuple({std::move(gx), std::move(ga), std::move(gb)});
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(dynamic), METHOD(backward), METHOD(qk_norm_rope), METHOD(qk_norm_rope_backward),
                         METHOD(add_rms_norm_quantize), METHOD(add_rms_norm_backward), METHOD(linear_adapters),
                         METHOD(linear_adapters_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
