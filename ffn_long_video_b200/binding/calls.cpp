// The generation calls from Python: argument checks, allocation and the C call in
// one step. These calls run once per layer and generated token, where the host
// time of a call counts: through ctypes a decode call took 20 us on the host, 14
// of them for checks, allocation and argument conversion; this way an append takes
// 4.1 us on the host (2.8 with its output given), a decode call as long as the GPU.
//
// Positional arguments only (the package's functions name and document them);
// None stands for an output or a workspace to be allocated. Checks raise
// ValueError or TypeError; a status other than ADASPARK_OK raises AdasparkError.
// No arithmetic happens here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "adaspark.h"

namespace {

PyObject* g_error = nullptr;  // AdasparkError

struct Raised : std::exception {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

std::string sizes(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// Arguments of a call, taken in order.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;

  PyObject* next() {
    if (left <= 0) raise(PyExc_TypeError, "too few arguments");
    --left;
    return *at++;
  }
  const at::Tensor& tensor(const char* name) {
    PyObject* o = next();
    if (o == Py_None) raise(PyExc_ValueError, std::string(name) + " is required");
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  const at::Tensor* maybe(const char* name) {
    if (left > 0 && *at == Py_None) {
      next();
      return nullptr;
    }
    return &tensor(name);
  }
  double number(const char* name) {
    PyObject* o = next();
    const double v = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) raise(PyExc_TypeError, std::string(name) + " must be a number");
    return v;
  }
  int integer(const char* name) {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) raise(PyExc_TypeError, std::string(name) + " must be an integer");
    if (v != (int)v) raise(PyExc_ValueError, std::string(name) + " is out of range");
    return (int)v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw Raised();
    return v != 0;
  }
};

// Type and device that a call's tensors share.
struct Of {
  at::ScalarType type;
  c10::Device device;
  int code;

  explicit Of(const at::Tensor& t, const char* name) : type(t.scalar_type()), device(t.device()) {
    if (!device.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (type == at::kBFloat16)
      code = ADASPARK_BF16;
    else if (type == at::kFloat)
      code = ADASPARK_FP32;
    else
      raise(PyExc_TypeError, std::string(name) + ": unsupported dtype " + c10::toString(type));
  }
};

[[noreturn]] void refuse(const at::Tensor& t, const char* name, at::ScalarType type,
                         c10::Device device, at::IntArrayRef shape) {
  raise(PyExc_ValueError, std::string(name) + " must be " + c10::toString(type) + " " +
                              sizes(shape) + " on " + device.str() + "; got " +
                              c10::toString(t.scalar_type()) + " " + sizes(t.sizes()) + " on " +
                              t.device().str() + ", strides " + sizes(t.strides()));
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device,
           at::IntArrayRef shape) {
  if (t.scalar_type() != type || t.device() != device || t.sizes() != shape ||
      t.layout() != at::kStrided)
    refuse(t, name, type, device, shape);
}

void* dense(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device,
            at::IntArrayRef shape) {
  check(t, name, type, device, shape);
  if (!t.is_contiguous()) refuse(t, name, type, device, shape);
  return t.data_ptr();
}

// A [tokens, heads, d] tensor with any token and head strides.
struct Rows {
  void* p = nullptr;
  int64_t ts = 0, hs = 0;

  Rows() = default;
  Rows(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device,
       at::IntArrayRef shape) {
    check(t, name, type, device, shape);
    if (t.stride(2) != 1)
      raise(PyExc_ValueError, std::string(name) + ": the elements of a head must be contiguous");
    p = t.data_ptr();
    ts = t.stride(0);
    hs = t.stride(1);
  }
};

struct Heads {
  int n, h, d;
  explicit Heads(const at::Tensor& t, const char* name) {
    if (t.dim() != 3)
      raise(PyExc_ValueError, std::string(name) + " must be [tokens, heads, d], got " +
                                  sizes(t.sizes()));
    for (int64_t s : t.sizes())
      if (s > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
    n = (int)t.size(0);
    h = (int)t.size(1);
    d = (int)t.size(2);
  }
};

struct Cache {
  void *k, *v;
  int64_t ps, ts, hs;
  int pages, page;

  Cache(const at::Tensor& kc, const at::Tensor& vc, const Of& of, int hkv, int d) {
    if (kc.dim() != 4)
      raise(PyExc_ValueError, "k_cache must be [pages, page_size, hkv, d], got " +
                                  sizes(kc.sizes()));
    const int64_t shape[4] = {kc.size(0), kc.size(1), hkv, d};
    check(kc, "k_cache", of.type, of.device, shape);
    check(vc, "v_cache", of.type, of.device, shape);
    if (kc.stride(3) != 1 || vc.strides() != kc.strides())
      raise(PyExc_ValueError, "k_cache and v_cache must have the same strides, with the elements "
                              "of a head contiguous");
    if (shape[0] > INT32_MAX || shape[1] > INT32_MAX)
      raise(PyExc_ValueError, "k_cache is too large");
    k = kc.data_ptr();
    v = vc.data_ptr();
    ps = kc.stride(0);
    ts = kc.stride(1);
    hs = kc.stride(2);
    pages = (int)shape[0];
    page = (int)shape[1];
  }
};

struct Table {
  int32_t* p;
  int64_t stride;
  int cols;
  Table(const at::Tensor& t, c10::Device device, int64_t n) {
    if (t.scalar_type() != at::kInt || t.device() != device || t.dim() != 2 || t.size(0) != n ||
        (t.stride(1) != 1 && t.size(1) > 1) || t.size(1) > INT32_MAX)
      raise(PyExc_ValueError, "block_table must be int32 [" + std::to_string(n) +
                                  ", max_pages] on " + device.str() + ", rows contiguous; got " +
                                  c10::toString(t.scalar_type()) + " " + sizes(t.sizes()) +
                                  " on " + t.device().str());
    p = t.data_ptr<int32_t>();
    stride = t.stride(0);
    cols = (int)t.size(1);
  }
};

struct Workspace {
  void* p;
  size_t bytes;
  Workspace(const at::Tensor& t, c10::Device device) {
    if (t.scalar_type() != at::kByte || t.device() != device || !t.is_contiguous())
      raise(PyExc_ValueError, "workspace must be a contiguous uint8 tensor on " + device.str());
    p = t.data_ptr();
    bytes = (size_t)t.numel();
  }
};

// Positions, sections, frequencies, layout, magnitude, weights, eps.
struct Rope {
  const int32_t* pos = nullptr;
  int axes = 1;
  int32_t sec[3] = {0, 0, 0};
  const double* freq = nullptr;
  int rot = 0, interleaved;
  float magnitude, eps;
  const void *wq = nullptr, *wk = nullptr;

  // positions, freq, w_q, w_k, eps, interleaved, sections, magnitude; the weights'
  // tensors are taken before (their type may be the call's)
  Rope(const at::Tensor* positions, const at::Tensor* f, const at::Tensor* w_q,
       const at::Tensor* w_k, double e, bool il, PyObject* sections, double mag,
       at::ScalarType type, c10::Device device, int n, int d)
      : interleaved(il), magnitude((float)mag), eps((float)e) {
    if (w_q) wq = dense(*w_q, "w_q", type, device, {d});
    if (w_k) wk = dense(*w_k, "w_k", type, device, {d});
    if (!f) return;
    if (!positions) raise(PyExc_ValueError, "positions is required");
    const int64_t half = f->numel();
    if (half > INT32_MAX / 2) raise(PyExc_ValueError, "freq is too large");
    freq = static_cast<const double*>(dense(*f, "freq", at::kDouble, device, {half}));
    rot = (int)(2 * half);
    if (sections == Py_None) {
      pos = static_cast<const int32_t*>(dense(*positions, "positions", at::kInt, device, {n}));
      return;
    }
    axes = 3;
    PyObject* seq = PySequence_Fast(sections, "sections must be three numbers of pairs");
    if (!seq) throw Raised();
    const bool three = PySequence_Fast_GET_SIZE(seq) == 3;
    for (int i = 0; three && i < 3; ++i) {
      const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
      sec[i] = v == (int32_t)v ? (int32_t)v : -1;  // the call refuses what is not a count
    }
    Py_DECREF(seq);
    if (PyErr_Occurred()) throw Raised();
    if (!three) raise(PyExc_ValueError, "sections must be three numbers of pairs");
    pos = static_cast<const int32_t*>(dense(*positions, "positions", at::kInt, device, {3, n}));
  }
};

// Without the dispatcher, which would add 0.4 us to a call of 4.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
  return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// Several dense tensors to be written. Small ones share one allocation, each on a
// 256-byte boundary (an allocation costs a call 0.9 us); large ones have their
// own, so that keeping one of them does not keep the others' memory.
struct Piece {
  at::SmallVector<int64_t, 3> shape;
  at::ScalarType type;
};
template <size_t N>
std::array<at::Tensor, N> make_all(const std::array<Piece, N>& pieces, c10::Device device) {
  constexpr int64_t kShared = 1 << 20;
  int64_t first[N], bytes = 0;
  for (size_t i = 0; i < N; ++i) {
    int64_t n = (int64_t)c10::elementSize(pieces[i].type);
    for (int64_t d : pieces[i].shape) n *= d;
    first[i] = bytes;
    bytes += (n + 255) / 256 * 256;
  }
  std::array<at::Tensor, N> r;
  if (bytes > kShared) {
    for (size_t i = 0; i < N; ++i) r[i] = make(pieces[i].shape, pieces[i].type, device);
    return r;
  }
  const at::Tensor all = make({bytes}, at::kByte, device);
  for (size_t i = 0; i < N; ++i) {
    r[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                    c10::scalarTypeToTypeMeta(pieces[i].type));
    r[i].unsafeGetTensorImpl()->set_sizes_contiguous(pieces[i].shape);
    r[i].unsafeGetTensorImpl()->set_storage_offset(
        first[i] / (int64_t)c10::elementSize(pieces[i].type));
  }
  return r;
}
// Two of them, where neither is given.
void make_two(at::Tensor& x, const at::Tensor* given_x, const Piece& px, at::Tensor& y,
              const at::Tensor* given_y, const Piece& py, c10::Device device) {
  if (!given_x && !given_y) {
    auto r = make_all<2>({{px, py}}, device);
    x = std::move(r[0]);
    y = std::move(r[1]);
  } else {
    x = given_x ? *given_x : make(px.shape, px.type, device);
    y = given_y ? *given_y : make(py.shape, py.type, device);
  }
}

void done(int rc, const char* what) {
  if (rc == ADASPARK_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", rc, what) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s: status %d", what, rc);
  }
  throw Raised();
}

PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o;
    if (t) {
      o = THPVariable_Wrap(*t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs a call's body on the tensors' device; no C++ exception leaves it.
template <typename F>
PyObject* guarded(F body) {
  try {
    at::AutoDispatchBelowADInplaceOrView below_autograd;
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

void* stream_on(c10::Device device) {
  return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}

// Q, K, positions, freq, w_q, w_k, eps, interleaved, sections, magnitude, out_q, out_k
PyObject* py_qk_rope(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &Q = a.tensor("Q"), &K = a.tensor("K");
    const at::Tensor *pos = a.maybe("positions"), *freq = a.maybe("freq");
    const at::Tensor *wq = a.maybe("w_q"), *wk = a.maybe("w_k");
    const double eps = a.number("eps");
    const bool il = a.truth();
    PyObject* sections = a.next();
    const double mag = a.number("magnitude");
    const at::Tensor *oq = a.maybe("out_q"), *ok = a.maybe("out_k");
    const Of of(Q, "Q");
    const c10::cuda::CUDAGuard guard(of.device);
    const Heads q(Q, "Q"), k(K, "K");
    const int64_t qs[3] = {q.n, q.h, q.d}, ks[3] = {q.n, k.h, q.d};
    const Rows rq(Q, "Q", of.type, of.device, qs), rk(K, "K", of.type, of.device, ks);
    const Rope r(pos, freq, wq, wk, eps, il, sections, mag, of.type, of.device, q.n, q.d);
    at::Tensor Qo, Ko;
    make_two(Qo, oq, {{q.n, q.h, q.d}, of.type}, Ko, ok, {{q.n, k.h, q.d}, of.type}, of.device);
    const Rows wo(Qo, "out_q", of.type, of.device, qs), wko(Ko, "out_k", of.type, of.device, ks);
    done(adaspark_qk_rope(rq.p, rq.ts, rq.hs, rk.p, rk.ts, rk.hs, of.code, r.pos, r.axes, r.sec,
                          r.freq, r.rot, r.interleaved, r.magnitude, r.wq, r.wk, r.eps, q.n, q.h,
                          k.h, q.d, wo.p, wo.ts, wo.hs, wko.p, wko.ts, wko.hs,
                          stream_on(of.device)),
         "adaspark_qk_rope");
    return tuple({&Qo, &Ko});
  });
}

// Q, K, V, positions, freq, slots, k_cache, v_cache, w_q, w_k, eps, interleaved, sections,
// magnitude, out_q
PyObject* py_qk_rope_append(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &Q = a.tensor("Q"), &K = a.tensor("K"), &V = a.tensor("V");
    const at::Tensor *pos = a.maybe("positions"), *freq = a.maybe("freq");
    const at::Tensor &slots = a.tensor("slots"), &kc = a.tensor("k_cache"),
                     &vc = a.tensor("v_cache");
    const at::Tensor *wq = a.maybe("w_q"), *wk = a.maybe("w_k");
    const double eps = a.number("eps");
    const bool il = a.truth();
    PyObject* sections = a.next();
    const double mag = a.number("magnitude");
    const at::Tensor* oq = a.maybe("out_q");
    const Of of(Q, "Q");
    const c10::cuda::CUDAGuard guard(of.device);
    const Heads q(Q, "Q"), k(K, "K");
    const int64_t qs[3] = {q.n, q.h, q.d}, ks[3] = {q.n, k.h, q.d};
    const Rows rq(Q, "Q", of.type, of.device, qs), rk(K, "K", of.type, of.device, ks),
        rv(V, "V", of.type, of.device, ks);
    const auto* sl =
        static_cast<const int32_t*>(dense(slots, "slots", at::kInt, of.device, {q.n}));
    const Cache c(kc, vc, of, k.h, q.d);
    const Rope r(pos, freq, wq, wk, eps, il, sections, mag, of.type, of.device, q.n, q.d);
    const at::Tensor Qo = oq ? *oq : make(qs, of.type, of.device);
    const Rows wo(Qo, "out_q", of.type, of.device, qs);
    done(adaspark_qk_rope_append(rq.p, rq.ts, rq.hs, rk.p, rk.ts, rk.hs, rv.p, rv.ts, rv.hs,
                                 of.code, r.pos, r.axes, r.sec, r.freq, r.rot, r.interleaved,
                                 r.magnitude, r.wq, r.wk, r.eps, q.n, q.h, k.h, q.d, sl, c.k, c.v,
                                 c.ps, c.ts, c.hs, c.pages, c.page, wo.p, wo.ts, wo.hs,
                                 stream_on(of.device)),
         "adaspark_qk_rope_append");
    return THPVariable_Wrap(Qo);
  });
}

// K, V, slots, k_cache, v_cache
PyObject* py_kv_append(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &K = a.tensor("K"), &V = a.tensor("V"), &slots = a.tensor("slots"),
                     &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
    const Of of(K, "K");
    const c10::cuda::CUDAGuard guard(of.device);
    const Heads k(K, "K");
    const int64_t ks[3] = {k.n, k.h, k.d};
    const Rows rk(K, "K", of.type, of.device, ks), rv(V, "V", of.type, of.device, ks);
    const auto* sl =
        static_cast<const int32_t*>(dense(slots, "slots", at::kInt, of.device, {k.n}));
    const Cache c(kc, vc, of, k.h, k.d);
    done(adaspark_kv_append(rk.p, rk.ts, rk.hs, rv.p, rv.ts, rv.hs, of.code, k.n, k.h, k.d, sl,
                            c.k, c.v, c.ps, c.ts, c.hs, c.pages, c.page, stream_on(of.device)),
         "adaspark_kv_append");
    Py_RETURN_NONE;
  });
}

// dQ_out, dK_out, positions, freq, Q, K, w_q, w_k, eps, interleaved, sections, magnitude, dQ, dK,
// dw_q, dw_k, workspace
PyObject* py_qk_rope_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &gQ = a.tensor("dQ_out"), &gK = a.tensor("dK_out");
    const at::Tensor *pos = a.maybe("positions"), *freq = a.maybe("freq");
    const at::Tensor *Q = a.maybe("Q"), *K = a.maybe("K");
    const at::Tensor *wq = a.maybe("w_q"), *wk = a.maybe("w_k");
    const double eps = a.number("eps");
    const bool il = a.truth();
    PyObject* sections = a.next();
    const double mag = a.number("magnitude");
    const at::Tensor *tq = a.maybe("dQ"), *tk = a.maybe("dK"), *twq = a.maybe("dw_q"),
                     *twk = a.maybe("dw_k"), *tws = a.maybe("workspace");
    const Of dy(gQ, "dQ_out");
    const c10::cuda::CUDAGuard guard(dy.device);
    const Heads q(gQ, "dQ_out"), k(gK, "dK_out");
    const int64_t qs[3] = {q.n, q.h, q.d}, ks[3] = {q.n, k.h, q.d};
    const Rows rgq(gQ, "dQ_out", dy.type, dy.device, qs),
        rgk(gK, "dK_out", dy.type, dy.device, ks);
    const at::Tensor* w = wq ? wq : wk;
    const Of of = w ? Of(*w, wq ? "w_q" : "w_k") : dy;
    if (wq && !Q) raise(PyExc_ValueError, "Q is required with w_q");
    if (wk && !K) raise(PyExc_ValueError, "K is required with w_k");
    const Rows rq = wq ? Rows(*Q, "Q", of.type, dy.device, qs) : Rows();
    const Rows rk = wk ? Rows(*K, "K", of.type, dy.device, ks) : Rows();
    const Rope r(pos, freq, wq, wk, eps, il, sections, mag, of.type, dy.device, q.n, q.d);
    at::Tensor dQ, dK, dwq, dwk, ws;
    make_two(dQ, tq, {{q.n, q.h, q.d}, at::kFloat}, dK, tk, {{q.n, k.h, q.d}, at::kFloat},
             dy.device);
    if (wq && wk) {
      make_two(dwq, twq, {{q.d}, at::kFloat}, dwk, twk, {{q.d}, at::kFloat}, dy.device);
    } else {
      if (wq) dwq = twq ? *twq : make({q.d}, at::kFloat, dy.device);
      if (wk) dwk = twk ? *twk : make({q.d}, at::kFloat, dy.device);
    }
    if (tws) {
      ws = *tws;
    } else if (w) {
      const size_t nb = adaspark_qk_rope_backward_workspace(q.n, q.h, k.h, q.d, of.code);
      if (nb == 0) done(ADASPARK_EINVAL, "adaspark_qk_rope_backward_workspace");
      ws = make({(int64_t)nb}, at::kByte, dy.device);
    }
    auto* pq = static_cast<float*>(dense(dQ, "dQ", at::kFloat, dy.device, qs));
    auto* pk = static_cast<float*>(dense(dK, "dK", at::kFloat, dy.device, ks));
    auto* pwq = wq ? static_cast<float*>(dense(dwq, "dw_q", at::kFloat, dy.device, {q.d})) : nullptr;
    auto* pwk = wk ? static_cast<float*>(dense(dwk, "dw_k", at::kFloat, dy.device, {q.d})) : nullptr;
    void* pws = nullptr;
    size_t bytes = 0;
    if (ws.defined()) {
      const Workspace x(ws, dy.device);
      pws = x.p;
      bytes = x.bytes;
    }
    done(adaspark_qk_rope_backward(rgq.p, rgq.ts, rgq.hs, rgk.p, rgk.ts, rgk.hs, dy.code, rq.p,
                                   rq.ts, rq.hs, rk.p, rk.ts, rk.hs, of.code, r.pos, r.axes, r.sec,
                                   r.freq, r.rot, r.interleaved, r.magnitude, r.wq, r.wk, r.eps,
                                   q.n, q.h, k.h, q.d, pq, pk, pwq, pwk, pws, bytes,
                                   stream_on(dy.device)),
         "adaspark_qk_rope_backward");
    return tuple({&dQ, &dK, wq ? &dwq : nullptr, wk ? &dwk : nullptr, ws.defined() ? &ws : nullptr});
  });
}

// old_lens, new_lens, block_table, free_pages, n_free, page_size, n_rows, slots, positions,
// token_starts, workspace
PyObject* py_kv_plan(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &old_lens = a.tensor("old_lens"), &new_lens = a.tensor("new_lens"),
                     &table = a.tensor("block_table"), &free_pages = a.tensor("free_pages"),
                     &n_free = a.tensor("n_free");
    const int page = a.integer("page_size"), rows = a.integer("n_rows");
    const at::Tensor *ts = a.maybe("slots"), *tp = a.maybe("positions"),
                     *tt = a.maybe("token_starts"), *tw = a.maybe("workspace");
    const c10::Device dev = old_lens.device();
    if (!dev.is_cuda()) raise(PyExc_ValueError, "old_lens must be a CUDA tensor");
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t ns = old_lens.numel(), pages = free_pages.numel();
    if (ns >= INT32_MAX || pages > INT32_MAX) raise(PyExc_ValueError, "too many sequences or pages");
    auto ints = [&](const at::Tensor& t, const char* name, int64_t n) {
      return static_cast<int32_t*>(dense(t, name, at::kInt, dev, {n}));
    };
    const int32_t* po = ints(old_lens, "old_lens", ns);
    const int32_t* pn = ints(new_lens, "new_lens", ns);
    const Table tb(table, dev, ns);
    int32_t* pf = ints(free_pages, "free_pages", pages);
    int32_t* pnf = ints(n_free, "n_free", 1);
    const size_t nb = adaspark_kv_plan_workspace((int)ns);
    if (nb == 0 || rows < 1) done(ADASPARK_EINVAL, "adaspark_kv_plan");
    at::Tensor slots, positions, starts, ws;
    if (!ts && !tp && !tt && !tw) {
      auto r = make_all<4>({{{{rows}, at::kInt}, {{rows}, at::kInt}, {{ns + 1}, at::kInt},
                             {{(int64_t)nb}, at::kByte}}}, dev);
      slots = std::move(r[0]);
      positions = std::move(r[1]);
      starts = std::move(r[2]);
      ws = std::move(r[3]);
    } else {
      slots = ts ? *ts : make({rows}, at::kInt, dev);
      positions = tp ? *tp : make({rows}, at::kInt, dev);
      starts = tt ? *tt : make({ns + 1}, at::kInt, dev);
      ws = tw ? *tw : make({(int64_t)nb}, at::kByte, dev);
    }
    const Workspace w(ws, dev);
    done(adaspark_kv_plan(po, pn, (int)ns, page, tb.p, tb.stride, tb.cols, pf, (int)pages, pnf,
                          ints(starts, "token_starts", ns + 1), ints(slots, "slots", rows),
                          ints(positions, "positions", rows), rows, w.p, w.bytes, stream_on(dev)),
         "adaspark_kv_plan");
    return tuple({&slots, &positions, &starts, &ws});
  });
}

// Q, k_cache, v_cache, block_table, seq_lens, scale, out, lse, workspace
PyObject* py_decode_attn(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return guarded([&]() -> PyObject* {
    Args a{argv, argc};
    const at::Tensor &Q = a.tensor("Q"), &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache"),
                     &table = a.tensor("block_table"), &lens = a.tensor("seq_lens");
    PyObject* sc = a.next();
    const at::Tensor *to = a.maybe("out"), *tl = a.maybe("lse"), *tw = a.maybe("workspace");
    const Of of(Q, "Q");
    const c10::cuda::CUDAGuard guard(of.device);
    const Heads q(Q, "Q");
    const int64_t qs[3] = {q.n, q.h, q.d};
    const Rows rq(Q, "Q", of.type, of.device, qs);
    if (kc.dim() != 4) raise(PyExc_ValueError, "k_cache must be [pages, page_size, hkv, d]");
    if (kc.size(2) > INT32_MAX) raise(PyExc_ValueError, "k_cache is too large");
    const int hkv = (int)kc.size(2);
    const Cache c(kc, vc, of, hkv, q.d);
    const Table tb(table, of.device, q.n);
    const auto* pl =
        static_cast<const int32_t*>(dense(lens, "seq_lens", at::kInt, of.device, {q.n}));
    float scale = 0.f;
    if (sc == Py_None) {
      scale = q.d > 0 ? (float)(1.0 / std::sqrt((double)q.d)) : 0.f;
    } else {
      const double v = PyFloat_AsDouble(sc);
      if (v == -1.0 && PyErr_Occurred()) throw Raised();
      scale = (float)v;
    }
    const size_t nb = adaspark_decode_attn_workspace(q.n, q.h, hkv, q.d, of.code);
    if (nb == 0) done(ADASPARK_EINVAL, "adaspark_decode_attn_workspace");
    at::Tensor out, lse;
    make_two(out, to, {{q.n, q.h, q.d}, of.type}, lse, tl, {{q.n, q.h}, at::kFloat}, of.device);
    const at::Tensor ws = tw ? *tw : make({(int64_t)nb}, at::kByte, of.device);
    const Workspace w(ws, of.device);
    done(adaspark_decode_attn(rq.p, rq.ts, rq.hs, c.k, c.v, c.ps, c.ts, c.hs, c.pages, c.page,
                              of.code, tb.p, tb.stride, tb.cols, pl, q.n, q.h, hkv, q.d, scale,
                              dense(out, "out", of.type, of.device, qs),
                              static_cast<float*>(
                                  dense(lse, "lse", at::kFloat, of.device, {q.n, q.h})),
                              w.p, w.bytes, stream_on(of.device)),
         "adaspark_decode_attn");
    return tuple({&out, &lse, &ws});
  });
}

PyObject* py_set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_rope),          FAST(qk_rope_append), FAST(kv_append),
                         FAST(qk_rope_backward), FAST(kv_plan),        FAST(decode_attn),
                         {"set_error", py_set_error, METH_O, nullptr},  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
