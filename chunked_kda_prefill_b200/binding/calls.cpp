// calls.cpp -- the operators' calls in their common form (tensors that fit the call, results to be
// allocated, the current stream) without the interpreter's share of their cost: about 5 us a call
// instead of 15 to 30.  Everything else, and every refusal, is the Python functions': a call that does
// not fit returns None and they take it, and say what is wrong.  A status of the library other than
// KDA_OK is returned as a number.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <vector>

#include "../../include/kda.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Shape = std::vector<int64_t>;

// The library's entry points, by address: it is loaded (or another build of it) by the interpreter.
struct {
  decltype(&kda_recurrence_forward) rec_forward;
  decltype(&kda_recurrence_backward) rec_backward;
  decltype(&kda_recurrence_step) rec_step;
  decltype(&kda_qk_norm_rope) qk_forward;
  decltype(&kda_qk_norm_rope_workspace_size) qk_workspace;
  decltype(&kda_qk_norm_rope_backward) qk_backward;
} lib;

constexpr size_t kStatusBytes = 256;  // a workspace that holds the device status alone
const char* const kLayouts[] = {"BNSD", "BSND", "TND"};

struct Plan {
  kda_recurrence_shape_t shape;
  const int32_t* host;
  size_t words, workspace, backward_workspace;
  Tensor dev;
  PyObject* owner;  // of `host`
  Shape x, rows, state, params, heads, states;
};

void drop_plan(PyObject* capsule) {
  Plan* p = static_cast<Plan*>(PyCapsule_GetPointer(capsule, "kda.plan"));
  if (!p) return;
  Py_XDECREF(p->owner);
  delete p;
}

// A plain CUDA tensor on device `dev`; null for anything else (a tensor that is another class's view
// of its own kind, has no memory, or is negated by a mark alone, included).
const Tensor* plain(PyObject* o, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.get_device() != dev || t.layout() != at::kStrided ||
      t.unsafeGetTensorImpl()->is_python_dispatch() || t.is_neg() || !t.has_storage() ||
      !t.const_data_ptr())
    return nullptr;
  return &t;
}

bool fits(const Tensor* t, ScalarType type, at::IntArrayRef shape) {
  return t && t->scalar_type() == type && t->sizes() == shape;
}
bool dense(const Tensor* t, ScalarType type, at::IntArrayRef shape) {
  return fits(t, type, shape) && t->is_contiguous();
}

// An argument that may be None: sets *t (null for None); false when it is something else that does
// not fit.
bool maybe(PyObject* o, int dev, ScalarType type, at::IntArrayRef shape, const Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  *t = plain(o, dev);
  return dense(*t, type, shape);
}

// Whether a recording of torch's operations, or another mode that sees them, is on.
bool watched() {
  using c10::DispatchKey;
  return c10::impl::TorchDispatchModeTLS::any_modes_set() ||
         c10::impl::tls_is_dispatch_key_included(DispatchKey::Tracer) ||
         c10::impl::tls_is_dispatch_key_included(DispatchKey::PreDispatch);
}

int type_code(ScalarType t) {
  return t == ScalarType::BFloat16 ? 0 : t == ScalarType::Half ? 1 : t == ScalarType::Float ? 2 : -1;
}

int layout_of(PyObject* o) {
  if (!PyUnicode_Check(o)) return -1;
  for (int i = 0; i < 3; ++i)
    if (PyUnicode_CompareWithASCIIString(o, kLayouts[i]) == 0) return i;
  return -1;
}

bool number(PyObject* o, float* v) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *v = (float)d;
  return true;
}

// kda_view_t of a tensor in a layout; false when its channels do not lie side by side.
bool view(const Tensor& t, int layout, bool channels, kda_view_t* v) {
  const auto st = t.strides();
  if (channels && st[st.size() - 1] != 1) return false;
  v->data = t.const_data_ptr();
  v->stride_b = layout == 2 ? 0 : st[0];
  v->stride_n = layout == 1 ? st[2] : st[1];
  v->stride_s = layout == 0 ? st[2] : layout == 1 ? st[1] : st[0];
  return true;
}

template <class T = float>
T* data(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

Tensor like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }
Tensor fresh(const Shape& s, const Tensor& on, ScalarType type) {
  return at::empty(s, on.options().dtype(type));
}
kda_stream_t stream_of(int dev) {
  return reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}
// Whether one carries a forward-mode derivative.
bool has_tangent(std::initializer_list<const Tensor*> ts) {
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return false;
  for (const Tensor* t : ts)
    if (t && t->_fw_grad(0).defined()) return true;  // there is one level
  return false;
}
bool wants_grad(std::initializer_list<const Tensor*> ts) {
  if (has_tangent(ts)) return true;
  if (!c10::GradMode::is_enabled()) return false;
  for (const Tensor* t : ts)
    if (t && t->requires_grad()) return true;
  return false;
}
PyObject* tuple_of(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
// Lets other threads of the interpreter run, until the end of its scope however that is left.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
#define CALL(expr)        \
  kda_status_t status;    \
  {                       \
    const Unlocked here;  \
    status = (expr);      \
  }                       \
  if (status != KDA_OK) return PyLong_FromLong(status)

// bind(addresses of the entry points, in the order of `lib`)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  void* a[6];
  for (int i = 0; i < 6; ++i) {
    a[i] = PyLong_AsVoidPtr(args[i]);
    if (!a[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  lib.rec_forward = reinterpret_cast<decltype(lib.rec_forward)>(a[0]);
  lib.rec_backward = reinterpret_cast<decltype(lib.rec_backward)>(a[1]);
  lib.rec_step = reinterpret_cast<decltype(lib.rec_step)>(a[2]);
  lib.qk_forward = reinterpret_cast<decltype(lib.qk_forward)>(a[3]);
  lib.qk_workspace = reinterpret_cast<decltype(lib.qk_workspace)>(a[4]);
  lib.qk_backward = reinterpret_cast<decltype(lib.qk_backward)>(a[5]);
  Py_RETURN_NONE;
}

// plan(layout, B, N, S, D, host address, words, owner, device copy, workspace bytes, the backward
// pass's, rows of states): what the calls need of a recurrence plan
PyObject* make_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || !THPVariable_Check(args[8])) {
    PyErr_SetString(PyExc_TypeError, "plan takes twelve values");
    return nullptr;
  }
  long long v[12] = {};
  for (int i = 0; i < 12; ++i) {
    if (i == 7 || i == 8) continue;
    v[i] = PyLong_AsLongLong(args[i]);
    if (v[i] == -1 && PyErr_Occurred()) return nullptr;
  }
  Plan* p = new Plan;
  const int64_t B = v[1], N = v[2], S = v[3], D = v[4];
  p->shape = {(int32_t)v[0], (int32_t)B, (int32_t)N, (int32_t)S, (int32_t)D, 0};
  p->host = reinterpret_cast<const int32_t*>(v[5]);
  p->words = (size_t)v[6];
  p->owner = Py_NewRef(args[7]);
  p->dev = THPVariable_Unpack(args[8]);
  p->workspace = (size_t)v[9];
  p->backward_workspace = (size_t)v[10];
  p->rows = v[0] == 0 ? Shape{B, N, S} : v[0] == 1 ? Shape{B, S, N} : Shape{S, N};
  p->x = p->rows;
  p->x.push_back(D);
  p->state = {B, N, D};
  p->params = {N, D};
  p->heads = {N};
  p->states = {v[11], N, D};
  PyObject* c = PyCapsule_New(p, "kda.plan", drop_plan);
  if (!c) {
    Py_DECREF(p->owner);
    delete p;
  }
  return c;
  END_HANDLE_TH_ERRORS
}

// The inputs that both passes of the recurrence share.
struct Inputs {
  const Plan* p;
  int dev;
  const Tensor *x, *g, *beta, *h0, *A, *bias;
  float lb;
  kda_recurrence_shape_t shape;
  kda_view_t vx, vg, vb;

  // plan, layout, x, g, beta, initial_state, A_log, dt_bias, lower_bound
  bool read(PyObject* plan, PyObject* layout, PyObject* const* a) {
    p = static_cast<const Plan*>(PyCapsule_GetPointer(plan, "kda.plan"));
    if (!p) {
      PyErr_Clear();
      return false;
    }
    if (!p->dev.is_cuda() || layout_of(layout) != p->shape.layout) return false;
    dev = p->dev.get_device();
    if (c10::cuda::current_device() != dev) return false;
    x = plain(a[0], dev);
    g = plain(a[1], dev);
    beta = plain(a[2], dev);
    A = plain(a[4], dev);
    bias = plain(a[5], dev);
    if (!x) return false;
    const ScalarType type = x->scalar_type();
    const int code = type_code(type);
    if (code < 0 || !fits(x, type, p->x) || !fits(g, type, p->x) || !fits(beta, type, p->rows) ||
        !dense(A, ScalarType::Float, p->heads) || !dense(bias, ScalarType::Float, p->params) ||
        !maybe(a[3], dev, ScalarType::Float, p->state, &h0) || !number(a[6], &lb))
      return false;
    shape = p->shape;
    shape.dtype = code;
    const int l = shape.layout;
    return view(*x, l, true, &vx) && view(*g, l, true, &vg) && view(*beta, l, false, &vb);
  }
};

// recurrence_forward(plan, layout, x, g, beta, initial_state, A_log, dt_bias, lower_bound, states?)
PyObject* recurrence_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Inputs in;
  if (n != 10 || watched() || !in.read(a[0], a[1], a + 2) ||
      wants_grad({in.x, in.g, in.beta, in.h0, in.A, in.bias}))
    Py_RETURN_NONE;
  const Plan& p = *in.p;
  const int keep = PyObject_IsTrue(a[9]);
  if (keep < 0) return nullptr;
  const Tensor out = like(*in.x), final = fresh(p.state, *in.x, ScalarType::Float);
  Tensor states, work;
  if (keep) states = fresh(p.states, *in.x, ScalarType::Float);
  if (p.workspace > kStatusBytes)
    work = fresh({(int64_t)p.workspace}, *in.x, ScalarType::Byte);
  CALL(lib.rec_forward(&in.shape, p.host, data<int32_t>(&p.dev), p.words, &in.vx, &in.vg, &in.vb,
                       data(in.h0), data(in.A), data(in.bias), in.lb, keep ? data(&states) : nullptr,
                       work.defined() ? work.data_ptr() : nullptr,
                       work.defined() ? p.workspace : 0, out.data_ptr(), data(&final),
                       stream_of(in.dev)));
  return keep ? tuple_of({&out, &final, &states}) : tuple_of({&out, &final});
  END_HANDLE_TH_ERRORS
}

// recurrence_backward(plan, layout, x, g, beta, initial_state, A_log, dt_bias, lower_bound, states,
//                     dout, dfinal_state)
PyObject* recurrence_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Inputs in;
  if (n != 12 || watched() || !in.read(a[0], a[1], a + 2)) Py_RETURN_NONE;
  const Plan& p = *in.p;
  const Tensor *dout = nullptr, *dfinal, *states = plain(a[9], in.dev);
  kda_view_t vd;
  if (!dense(states, ScalarType::Float, p.states) ||
      !maybe(a[11], in.dev, ScalarType::Float, p.state, &dfinal))
    Py_RETURN_NONE;
  if (a[10] != Py_None) {
    dout = plain(a[10], in.dev);
    if (!fits(dout, in.x->scalar_type(), p.x) || !view(*dout, p.shape.layout, true, &vd))
      Py_RETURN_NONE;
  }
  if (has_tangent({in.x, in.g, in.beta, in.h0, in.A, in.bias, states, dout, dfinal})) Py_RETURN_NONE;
  const Tensor dx = like(*in.x), dg = like(*in.x), dbeta = like(*in.beta), dA = like(*in.A),
               dbias = like(*in.bias),
               work = fresh({(int64_t)p.backward_workspace}, *in.x, ScalarType::Byte);
  Tensor dh0;
  if (in.h0) dh0 = like(*in.h0);
  CALL(lib.rec_backward(&in.shape, p.host, data<int32_t>(&p.dev), p.words, dout ? &vd : nullptr,
                        data(dfinal), &in.vx, &in.vg, &in.vb, data(in.A), data(in.bias), in.lb,
                        data(states), work.data_ptr(), p.backward_workspace, dx.data_ptr(),
                        dg.data_ptr(), dbeta.data_ptr(), in.h0 ? data(&dh0) : nullptr, data(&dA),
                        data(&dbias), stream_of(in.dev)));
  return tuple_of({&dx, &dg, &dbeta, in.h0 ? &dh0 : nullptr, &dA, &dbias});
  END_HANDLE_TH_ERRORS
}

int device_of(PyObject* o) {  // of a CUDA tensor on the current device, else -1
  if (!THPVariable_Check(o)) return -1;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda()) return -1;
  const int dev = t.get_device();
  return c10::cuda::current_device() == dev ? dev : -1;
}

// recurrence_step(x, g, beta, state, A_log, dt_bias, lower_bound, out, state_out)
PyObject* recurrence_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int dev = n == 9 && !watched() ? device_of(a[0]) : -1;
  if (dev < 0) Py_RETURN_NONE;
  const Tensor *x = plain(a[0], dev), *g = plain(a[1], dev), *beta = plain(a[2], dev),
               *A = plain(a[4], dev), *bias = plain(a[5], dev), *state, *out_arg, *state_arg;
  float lb;
  if (!x || x->dim() != 3) Py_RETURN_NONE;
  const ScalarType type = x->scalar_type();
  const int code = type_code(type);
  const auto s = x->sizes();
  if (code < 0 || s[0] > INT_MAX || s[1] > INT_MAX || s[2] > INT_MAX || !dense(x, type, s) ||
      !dense(g, type, s) || !dense(beta, type, s.slice(0, 2)) ||
      !dense(A, ScalarType::Float, s.slice(1, 1)) || !dense(bias, ScalarType::Float, s.slice(1, 2)) ||
      !maybe(a[3], dev, ScalarType::Float, s, &state) || !number(a[6], &lb) ||
      !maybe(a[7], dev, type, s, &out_arg) || !maybe(a[8], dev, ScalarType::Float, s, &state_arg) ||
      wants_grad({x, g, beta, state, A, bias, out_arg, state_arg}))
    Py_RETURN_NONE;
  const Tensor out = out_arg ? *out_arg : like(*x);
  const Tensor next = state_arg ? *state_arg : at::empty(s, x->options().dtype(ScalarType::Float));
  CALL(lib.rec_step((int32_t)s[0], (int32_t)s[1], (int32_t)s[2], code, x->data_ptr(), g->data_ptr(),
                    beta->data_ptr(), data(state), data(A), data(bias), lb, out.data_ptr(),
                    data(&next), stream_of(dev)));
  // graphs that saved a supplied result's old values are to notice
  for (const Tensor* t : {out_arg, state_arg})
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  return tuple_of({&out, &next});
  END_HANDLE_TH_ERRORS
}

// The inputs that both passes of the norm and rotation share.
struct Heads {
  int dev;
  const Tensor *q, *k, *pos, *inv, *qw, *kw;
  kda_qk_shape_t shape;
  kda_view_t vq, vk;

  // q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved
  bool read(PyObject* const* a) {
    dev = device_of(a[0]);
    const int layout = layout_of(a[7]), inter = PyObject_IsTrue(a[8]);
    if (inter < 0) PyErr_Clear();
    if (dev < 0 || layout < 0 || inter < 0) return false;
    q = plain(a[0], dev);
    k = plain(a[1], dev);
    const int dims = layout == 2 ? 3 : 4;
    if (!q || !k || q->dim() != dims || k->dim() != dims) return false;
    const ScalarType type = q->scalar_type();
    const int code = type_code(type);
    if (code < 0) return false;
    const auto s = q->sizes();
    const int hd = layout == 0 ? 1 : dims - 2;  // the heads' dimension
    Shape ks = s.vec(), tokens;
    ks[hd] = k->size(hd);
    const int64_t B = layout == 2 ? 1 : s[0], S = layout == 2 ? s[0] : layout == 0 ? s[2] : s[1];
    const int64_t D = s[dims - 1];
    if (B > INT_MAX || S > INT_MAX || s[hd] > INT_MAX || ks[hd] > INT_MAX || D > INT_MAX ||
        !fits(k, type, ks))
      return false;
    tokens = layout == 2 ? Shape{S} : Shape{B, S};
    const Shape channels{D};
    int64_t half = 0;
    inv = nullptr;
    if (a[3] != Py_None) {
      inv = plain(a[3], dev);
      if (!inv || inv->dim() != 1 || inv->size(0) > INT_MAX / 2 ||
          !dense(inv, ScalarType::Float, inv->sizes()))
        return false;
      half = inv->size(0);
    }
    if (!maybe(a[2], dev, ScalarType::Int, tokens, &pos) ||
        !maybe(a[4], dev, ScalarType::Float, channels, &qw) ||
        !maybe(a[5], dev, ScalarType::Float, channels, &kw))
      return false;
    float eps;
    if (!number(a[6], &eps)) return false;
    shape = {layout, (int32_t)B,      (int32_t)s[hd], (int32_t)ks[hd], (int32_t)S, (int32_t)D,
             code,   (int32_t)(2 * half), inter,          eps};
    return view(*q, layout, true, &vq) && view(*k, layout, true, &vk);
  }
};

// qk_forward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved)
PyObject* qk_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads in;
  if (n != 9 || watched() || !in.read(a) || wants_grad({in.q, in.k, in.inv, in.qw, in.kw})) Py_RETURN_NONE;
  const Tensor q = like(*in.q), k = like(*in.k);
  CALL(lib.qk_forward(&in.shape, &in.vq, &in.vk, data<int32_t>(in.pos), data(in.inv), data(in.qw),
                      data(in.kw), q.data_ptr(), k.data_ptr(), stream_of(in.dev)));
  return tuple_of({&q, &k});
  END_HANDLE_TH_ERRORS
}

// qk_backward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved, dq_out, dk_out)
PyObject* qk_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads in;
  if (n != 11 || watched() || !in.read(a)) Py_RETURN_NONE;
  const Tensor *dqo = plain(a[9], in.dev), *dko = plain(a[10], in.dev);
  kda_view_t vdq, vdk;
  const ScalarType type = in.q->scalar_type();
  if (!fits(dqo, type, in.q->sizes()) || !fits(dko, type, in.k->sizes()) ||
      !view(*dqo, in.shape.layout, true, &vdq) || !view(*dko, in.shape.layout, true, &vdk) ||
      has_tangent({in.q, in.k, in.inv, in.qw, in.kw, dqo, dko}))
    Py_RETURN_NONE;
  size_t bytes = 0;
  const kda_status_t st = lib.qk_workspace(&in.shape, &bytes);
  if (st != KDA_OK) return PyLong_FromLong(st);
  const Tensor dq = like(*in.q), dk = like(*in.k),
               work = fresh({(int64_t)bytes}, *in.q, ScalarType::Byte);
  Tensor dqw, dkw;
  if (in.qw) dqw = like(*in.qw);
  if (in.kw) dkw = like(*in.kw);
  CALL(lib.qk_backward(&in.shape, &vdq, &vdk, &in.vq, &in.vk, data<int32_t>(in.pos), data(in.inv),
                       data(in.qw), data(in.kw), work.data_ptr(), bytes, dq.data_ptr(),
                       dk.data_ptr(), in.qw ? data(&dqw) : nullptr, in.kw ? data(&dkw) : nullptr,
                       stream_of(in.dev)));
  return tuple_of({&dq, &dk, in.qw ? &dqw : nullptr, in.kw ? &dkw : nullptr});
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, function) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(function)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("bind", bind),
                         ENTRY("plan", make_plan),
                         ENTRY("recurrence_forward", recurrence_forward),
                         ENTRY("recurrence_backward", recurrence_backward),
                         ENTRY("recurrence_step", recurrence_step),
                         ENTRY("qk_forward", qk_forward),
                         ENTRY("qk_backward", qk_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  // the torch that it was compiled against: it fits no other
  if (m && PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
