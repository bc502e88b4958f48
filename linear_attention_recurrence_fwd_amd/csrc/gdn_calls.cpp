// The short way from Python to the entries that are called for single tokens, where a
// call's time on the host counts: arguments are looked at, outputs allocated and the
// entry called here, in 3 to 5 us where the same checks in Python take 12 to 18.
//
// Each function takes the arguments of its namesake in binding.py, by position, and
// answers with its result, or with NotImplemented where anything is out of the ordinary
// (a type, shape, stride or device that does not fit, another current device, a gradient
// that would be asked for where there is none, a status other than 0): nothing was enqueued
// then (but where a launch failed, of those before it what is made again), and binding.py
// goes the long way, which says what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn.h"

namespace {

using at::Tensor;

// The arguments of a call, read one after the other; ok is false once one does not fit.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  bool ok = true;
  bool no_graph = false;  // tensors that a graph would have to lead to do not fit
  int dev = -1;           // the first tensor's device, and the current one

  PyObject* next() {
    if (at < n) return a[at++];
    ok = false;
    return Py_None;
  }
  // A tensor (null for None) on the call's device.
  const Tensor* tensor() {
    PyObject* o = next();
    if (o == Py_None || !ok) return nullptr;
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || (no_graph && t.requires_grad() && at::GradMode::is_enabled())) {
      ok = false;
      return nullptr;
    }
    const int d = t.device().index();
    if (dev < 0) {
      dev = d;
      if (c10::hip::current_device() != d) ok = false;
    } else if (d != dev) {
      ok = false;
    }
    return &t;
  }
  const Tensor& given() {
    static const Tensor none;
    const Tensor* t = tensor();
    if (!t) ok = false;
    return t ? *t : none;
  }
  int64_t integer() {
    PyObject* o = next();
    if (!ok || !PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  double number() {
    PyObject* o = next();
    if (ok && PyFloat_CheckExact(o)) return PyFloat_AS_DOUBLE(o);
    ok = false;
    return 0.0;
  }
  bool truth() {
    PyObject* o = next();
    if (o != Py_True && o != Py_False) ok = false;
    return o == Py_True;
  }
};

template <size_t N> bool shaped(const Tensor& t, const int64_t (&s)[N]) {
  if (t.dim() != static_cast<int64_t>(N)) return false;
  for (size_t i = 0; i < N; ++i)
    if (t.size(i) != s[i]) return false;
  return true;
}
// Dense, of this type and shape; an absent tensor fits.
template <size_t N> bool fits(const Tensor* t, at::ScalarType type, const int64_t (&s)[N]) {
  return !t || (t->scalar_type() == type && shaped(*t, s) && t->is_contiguous());
}
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* ptr(const Tensor& t) { return t.data_ptr(); }

bool type_of(const Tensor& t, int32_t* type) {
  *type = t.scalar_type() == at::kBFloat16 ? GDN_BF16 : GDN_F32;
  return *type == GDN_BF16 || t.scalar_type() == at::kFloat;
}

// Elements between the rows of consecutive tokens of [..., H, D], heads dense (0: dense
// altogether); the tokens evenly spaced over all dimensions before them.
bool token_stride(const Tensor& t, int64_t* out) {
  *out = 0;
  if (t.is_contiguous()) return true;
  const int64_t n = t.dim(), D = t.size(n - 1), H = t.size(n - 2);
  if ((D > 1 && t.stride(n - 1) != 1) || (H > 1 && t.stride(n - 2) != D)) return false;
  int64_t step = 0, count = 1;  // tokens of the dimensions behind
  for (int64_t i = n - 3; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (step == 0) step = t.stride(i);
    else if (t.stride(i) != count * step) return false;
    count *= t.size(i);
  }
  if (step == 0) return true;
  *out = step;
  return step >= H * D;
}

Tensor make(at::IntArrayRef s, const Tensor& like) { return at::empty(s, like.options()); }
void* stream(int dev) { return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
PyObject* declined() { Py_RETURN_NOTIMPLEMENTED; }
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// The rotation's part of the arguments: rope, axis, pos over `tokens` places.
struct Rotation {
  const Tensor *rope, *axis, *pos;
  int64_t P = 0, R = 0;
  int32_t A = 4;  // (without positions, as many axes as there can be)
  template <size_t N> bool read(Args& a, const int64_t (&tokens)[N]) {
    rope = a.tensor();
    axis = a.tensor();
    pos = a.tensor();
    if (!a.ok) return false;
    if (rope) {
      if (rope->dim() != 2 || rope->scalar_type() != at::kFloat || !rope->is_contiguous()) return false;
      P = rope->size(0);
      R = rope->size(1);
    }
    if (!fits(axis, at::kByte, {R / 2})) return false;
    if (pos) {
      if (pos->dim() != static_cast<int64_t>(N) + 1 || pos->scalar_type() != at::kInt || !pos->is_contiguous()) return false;
      A = static_cast<int32_t>(pos->size(0));
      if (A < 1 || A > 4) return false;
      for (size_t i = 0; i < N; ++i)
        if (pos->size(i + 1) != tokens[i]) return false;
    }
    return true;
  }
};

// ---- norm_rope_axes(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved)
//      norm_rope_axes_bwd(..., dyq, dyk)

struct Normed {
  gdn_norm_dims d{};
  const Tensor *q, *k, *wq, *wk;
  Rotation r;
  bool read(Args& a) {
    q = &a.given();
    k = &a.given();
    wq = a.tensor();
    wk = a.tensor();
    if (!a.ok || q->dim() != 4 || k->dim() != 4 || q->scalar_type() != k->scalar_type() || (wq == nullptr) != (wk == nullptr))
      return false;
    d.B = q->size(0);
    d.T = q->size(1);
    d.Hq = q->size(2);
    d.Hk = k->size(2);
    d.D = q->size(3);
    if (!shaped(*k, {d.B, d.T, d.Hk, d.D}) || !type_of(*q, &d.dtype)) return false;
    if (!fits(wq, at::kFloat, {d.D}) || !fits(wk, at::kFloat, {d.D}) || !r.read(a, {d.B, d.T})) return false;
    d.P = r.P;
    d.R = r.R;
    d.eps = static_cast<float>(a.number());
    d.w_offset = static_cast<float>(a.number());
    d.interleaved = a.truth();
    return a.ok && token_stride(*q, &d.q_stride) && token_stride(*k, &d.k_stride);
  }
};

PyObject* norm_rope_axes(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  Normed x;
  if (!x.read(a)) return declined();
  Tensor oq = make({x.d.B, x.d.T, x.d.Hq, x.d.D}, *x.q), ok = make({x.d.B, x.d.T, x.d.Hk, x.d.D}, *x.q);
  if (gdn_norm_rope_axes_fwd(&x.d, x.r.A, ptr(x.q), ptr(x.k), static_cast<float*>(ptr(x.wq)), static_cast<float*>(ptr(x.wk)),
                             static_cast<float*>(ptr(x.r.rope)), static_cast<uint8_t*>(ptr(x.r.axis)),
                             static_cast<int32_t*>(ptr(x.r.pos)), ptr(oq), ptr(ok), stream(a.dev)))
    return declined();
  return pair(THPVariable_Wrap(std::move(oq)), THPVariable_Wrap(std::move(ok)));
}

PyObject* norm_rope_axes_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  Normed x;
  if (!x.read(a)) return declined();
  const Tensor &dyq = a.given(), &dyk = a.given();
  if (!a.ok || !fits(&dyq, x.q->scalar_type(), {x.d.B, x.d.T, x.d.Hq, x.d.D}) ||
      !fits(&dyk, x.q->scalar_type(), {x.d.B, x.d.T, x.d.Hk, x.d.D}))
    return declined();
  size_t need = 0;
  Tensor ws, dwq, dwk;
  if (x.wq) {
    if (gdn_norm_rope_bwd_workspace_bytes(&x.d, &need)) return declined();
    if (need) ws = at::empty({static_cast<int64_t>(need)}, x.q->options().dtype(at::kByte));
    dwq = make({x.d.D}, *x.wq);
    dwk = make({x.d.D}, *x.wk);
  }
  Tensor dq = make(dyq.sizes(), dyq), dk = make(dyk.sizes(), dyk);
  if (gdn_norm_rope_axes_bwd(&x.d, x.r.A, ptr(x.q), ptr(x.k), static_cast<float*>(ptr(x.wq)), static_cast<float*>(ptr(x.wk)),
                             static_cast<float*>(ptr(x.r.rope)), static_cast<uint8_t*>(ptr(x.r.axis)),
                             static_cast<int32_t*>(ptr(x.r.pos)), ptr(dyq), ptr(dyk), ptr(dq), ptr(dk),
                             x.wq ? static_cast<float*>(ptr(dwq)) : nullptr, x.wq ? static_cast<float*>(ptr(dwk)) : nullptr,
                             need ? ptr(ws) : nullptr, need, stream(a.dev)))
    return declined();
  PyObject* out = PyDict_New();
  auto set = [&](const char* name, Tensor&& t) {
    PyObject* o = THPVariable_Wrap(std::move(t));  // (None for an undefined one)
    PyDict_SetItemString(out, name, o);
    Py_DECREF(o);
  };
  set("dq", std::move(dq));
  set("dk", std::move(dk));
  set("dwq", std::move(dwq));
  set("dwk", std::move(dwk));
  return out;
}

// ---- the pool and the sequences of a call

bool pool_of(gdn_paged_dims* d, const Tensor& kp, const Tensor& vp, const Tensor& table, const Tensor* cu, at::ScalarType type) {
  if (kp.dim() != 4 || kp.scalar_type() != type || vp.scalar_type() != type || kp.sizes() != vp.sizes() ||
      kp.strides() != vp.strides() || (kp.size(3) > 1 && kp.stride(3) != 1))
    return false;
  d->pages = kp.size(0);
  d->Hk = kp.size(1);
  d->page = kp.size(2);
  d->D = kp.size(3);
  d->page_stride = kp.stride(0);
  d->head_stride = kp.stride(1);
  d->token_stride = kp.stride(2);
  if (table.dim() != 2 || table.scalar_type() != at::kInt || !table.is_contiguous()) return false;
  d->S = table.size(0);
  d->width = table.size(1);
  return fits(cu, at::kInt, {d->S + 1});
}

// ---- paged_append(q, k, v, k_pages, v_pages, table, past, cu, wq, wk, rope, axis, pos,
//                   first, eps, w_offset, interleaved, out)

PyObject* paged_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  a.no_graph = true;
  const Tensor* q = a.tensor();
  const Tensor &k = a.given(), &v = a.given(), &kp = a.given(), &vp = a.given(), &table = a.given(), &past = a.given();
  const Tensor *cu = a.tensor(), *wq = a.tensor(), *wk = a.tensor();
  gdn_paged_dims d{};
  if (!a.ok || k.dim() != 3 || !type_of(k, &d.dtype) || !pool_of(&d, kp, vp, table, cu, k.scalar_type())) return declined();
  d.N = k.size(0);
  d.Hq = q ? q->size(1) : 0;
  if (!shaped(k, {d.N, d.Hk, d.D}) || !shaped(v, {d.N, d.Hk, d.D}) || v.scalar_type() != k.scalar_type() ||
      !fits(&past, at::kInt, {d.S}) || !fits(wq, at::kFloat, {d.D}) || !fits(wk, at::kFloat, {d.D}))
    return declined();
  if (q && (!shaped(*q, {d.N, d.Hq, d.D}) || q->scalar_type() != k.scalar_type())) return declined();
  Rotation r;
  gdn_turn t{};
  if (!r.read(a, {d.N})) return declined();
  t.first = a.integer();
  t.eps = static_cast<float>(a.number());
  t.w_offset = static_cast<float>(a.number());
  t.interleaved = a.truth();
  const Tensor* given = a.tensor();
  if (!a.ok || !token_stride(k, &t.k_stride) || !token_stride(v, &t.v_stride) || (q && !token_stride(*q, &t.q_stride)))
    return declined();
  t.P = r.P;
  t.R = r.R;
  t.A = r.A;
  if (given && (!q || !fits(given, k.scalar_type(), {d.N, d.Hq, d.D}))) return declined();
  Tensor out = given ? *given : q ? make({d.N, d.Hq, d.D}, k) : Tensor();
  if (gdn_paged_append(&d, &t, ptr(q), ptr(k), ptr(v), static_cast<float*>(ptr(wq)), static_cast<float*>(ptr(wk)),
                       static_cast<float*>(ptr(r.rope)), static_cast<uint8_t*>(ptr(r.axis)),
                       static_cast<int32_t*>(ptr(r.pos)), static_cast<int32_t*>(ptr(table)), static_cast<int32_t*>(ptr(past)),
                       static_cast<int32_t*>(ptr(cu)), q ? ptr(out) : nullptr, ptr(kp), ptr(vp), stream(a.dev)))
    return declined();
  return THPVariable_Wrap(std::move(out));
}

// ---- prefix_attention(q, k_pages, v_pages, table, lens, prefix_pages, prefix, cu, max_q,
//                       max_len, scale, out, lse)

PyObject* prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a{args, n};
  a.no_graph = true;
  const Tensor &q = a.given(), &kp = a.given(), &vp = a.given(), &table = a.given(), &lens = a.given();
  const Tensor* pages = a.tensor();
  const int64_t prefix = a.integer();
  const Tensor* cu = a.tensor();
  PyObject *max_q_ = a.next(), *max_len_ = a.next(), *scale_ = a.next();
  const Tensor* given = a.tensor();
  const bool lse = a.truth();
  gdn_paged_dims d{};
  if (!a.ok || q.dim() != 3 || !type_of(q, &d.dtype) || !pool_of(&d, kp, vp, table, cu, q.scalar_type())) return declined();
  d.N = q.size(0);
  d.Hq = q.size(1);
  if (!fits(&q, q.scalar_type(), {d.N, d.Hq, d.D}) || !fits(&lens, at::kInt, {d.S}) || prefix < 0) return declined();
  if (pages && (pages->dim() != 1 || pages->scalar_type() != at::kInt || !pages->is_contiguous())) return declined();
  if (d.page < 1 || d.S < 1 || (prefix && (!pages || pages->size(0) * d.page < prefix))) return declined();
  auto whole = [&](PyObject* o, int64_t none) {
    if (o == Py_None) return none;
    Args one{&o, 1};
    const int64_t v = one.integer();
    if (!one.ok) a.ok = false;
    return v;
  };
  int64_t max_len = whole(max_len_, std::min<int64_t>(d.width * d.page, int64_t{1} << 30)), max_q = whole(max_q_, d.N);
  if (!cu) {
    if (d.N % d.S) return declined();
    max_q = d.N / d.S;
  } else if (max_q > d.N) {
    max_q = d.N;
  }
  double scale = 1.0 / std::sqrt(static_cast<double>(d.D));
  if (scale_ != Py_None) {
    Args one{&scale_, 1};
    scale = one.number();
    if (!one.ok) a.ok = false;
  }
  size_t need = 0;
  if (!a.ok || !fits(given, q.scalar_type(), {d.N, d.Hq, d.D}) ||
      gdn_prefix_attention_workspace_bytes(&d, prefix, max_q, max_len, &need))
    return declined();
  Tensor out = given ? *given : make(q.sizes(), q), sums, ws;
  if (lse) sums = at::empty({d.N, d.Hq}, q.options().dtype(at::kFloat));
  if (need) ws = at::empty({static_cast<int64_t>(need)}, q.options().dtype(at::kByte));
  if (gdn_prefix_attention(&d, ptr(q), ptr(kp), ptr(vp), static_cast<int32_t*>(ptr(table)), static_cast<int32_t*>(ptr(lens)),
                           prefix ? static_cast<int32_t*>(ptr(pages)) : nullptr, prefix, static_cast<int32_t*>(ptr(cu)),
                           max_q, max_len, static_cast<float>(scale), ptr(out), lse ? static_cast<float*>(ptr(sums)) : nullptr,
                           need ? ptr(ws) : nullptr, need, stream(a.dev)))
    return declined();
  if (lse) return pair(THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(sums)));
  return THPVariable_Wrap(std::move(out));
}

// (no C++ exception leaves a function: an allocation that fails goes the long way too,
// and fails there)
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (...) {
    PyErr_Clear();
    return declined();
  }
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)> PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<norm_rope_axes>("norm_rope_axes"), method<norm_rope_axes_bwd>("norm_rope_axes_bwd"),
                         method<paged_append>("paged_append"), method<prefix_attention>("prefix_attention"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
