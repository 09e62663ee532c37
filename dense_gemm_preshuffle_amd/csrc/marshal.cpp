// Argument marshalling of the small operators' calls (a module of the Python binding):
// checks of the tensors, outputs, the call of the C ABI. A call of gemm_norm that takes 3
// us on the GPU took 8.4 us on the host through ctypes, of which the launch is 3.
//
// Each function returns its outputs, or None where anything is not as it should be (a
// type, a shape, a device, a status): the binding then goes through the same call step by
// step in Python, which names what is wrong. Nothing is decided here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gemm_preshuffle.h"

namespace {

// entry points of the loaded library (its path may be another than this module's)
decltype(&gemm_norm) p_norm;
decltype(&gemm_norm_backward) p_norm_backward;
decltype(&gemm_norm_backward_workspace_size) p_norm_backward_size;
decltype(&gemm_linear) p_linear;
decltype(&gemm_linear_workspace_size) p_linear_size;
decltype(&gemm_linear_backward) p_linear_backward;
decltype(&gemm_linear_backward_workspace_size) p_linear_backward_size;

PyObject* none() { Py_RETURN_NONE; }

// A tensor argument of one call: absent, or checked against what the call expects.
struct Args {
  PyObject* const* a;
  at::ScalarType half = at::kBFloat16;
  at::Device device = at::kCPU;
  bool ok = true;

  int64_t num(int i) {
    const int64_t v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) fail();
    return v;
  }
  double real(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) fail();
    return v;
  }
  void fail() {
    PyErr_Clear();
    ok = false;
  }
  const at::Tensor* tensor(int i) {
    if (a[i] == Py_None) return nullptr;
    if (!THPVariable_Check(a[i])) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(a[i]);
  }
  // the data of tensor i, which has this type and these sizes, or null where it is absent
  void* data(int i, at::ScalarType type, at::IntArrayRef sizes) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->device() != device || t->sizes() != sizes || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
};

bool is_true(PyObject* o) { return o == Py_True; }

void* data_of(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The interpreter's lock, given up for a scope: allocation and launch may wait (for memory,
// for queue space, for the library's code to be loaded), and other Python threads, or a
// host callback that the queue itself waits for, need the lock meanwhile. No Python object,
// and no tensor that has one, is touched in the scope; what it yields is wrapped after it.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// the tensor that was given, else none yet
at::Tensor given(Args& p, int i) {
  const at::Tensor* t = p.tensor(i);
  return t ? *t : at::Tensor();
}
void make(at::Tensor& t, bool wanted, at::IntArrayRef sizes, const at::TensorOptions& options) {
  if (wanted && !t.defined()) t = at::empty(sizes, options);
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

bool lead(Args& p, int dtype, const at::Tensor* t, int64_t index) {
  if (!t || !t->is_cuda() || t->device().index() != index || t->dim() != 2) return false;
  p.half = dtype == GP_BF16 ? at::kBFloat16 : at::kHalf;
  p.device = t->device();
  return true;
}

// dt, x, residual, scale, kin, w_in, b_in, gate, kout, w_out, b_out, eps, want_r, r, y, device, stream
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 17) return none();
  try {
    Args p{a};
    const int dt = (int)p.num(0), kin = (int)p.num(4), kout = (int)p.num(8);
    const at::Tensor* x = p.tensor(1);
    if (!lead(p, dt, x, p.num(15))) return none();
    const int64_t M = x->size(0), H = x->size(1);
    const at::IntArrayRef rows = x->sizes(), vec = rows.slice(1);
    const at::Tensor* gate = p.tensor(7);
    const int64_t gates = gate && gate->dim() == 2 ? gate->size(0) : 0;
    if (gate && !gates) return none();
    const int64_t gate_rows[2] = {gates, H};
    const bool want_r = is_true(a[12]);
    void *xd = p.data(1, p.half, rows), *res = p.data(2, p.half, rows);
    auto vector = [&](int i) { return (const float*)p.data(i, at::kFloat, vec); };
    const float *w_in = vector(5), *b_in = vector(6), *w_out = vector(9), *b_out = vector(10);
    const float* g = (const float*)p.data(7, at::kFloat, at::IntArrayRef(gate_rows, 2));
    p.data(13, p.half, rows);
    p.data(14, p.half, rows);
    const float scale = (float)p.real(3), eps = (float)p.real(11);
    void* stream = (void*)p.num(16);
    if (!p.ok || (a[13] != Py_None && !want_r) || (a[14] != Py_None && !kout)) return none();
    const at::TensorOptions half = x->options();
    at::Tensor r = given(p, 13), y = given(p, 14);
    int status;
    {
      Unlocked scope;
      make(r, want_r, rows, half);
      make(y, kout != 0, rows, half);
      status = p_norm(dt, xd, res, scale, kin, w_in, b_in, g, gates, kout, w_out, b_out, eps, data_of(r), data_of(y), M, H, stream);
    }
    if (status) return none();
    return Py_BuildValue("NN", wrap(r), wrap(y));
  } catch (...) {
    return none();
  }
}

// dt, dy, dr, x, r, scale, kin, w_in, b_in, gate, kout, w_out, b_out, eps, want_dx, want_dresidual, want_params, dx,
// dresidual, workspace, device, stream
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 22) return none();
  try {
    Args p{a};
    const int dt = (int)p.num(0), kin = (int)p.num(6), kout = (int)p.num(10);
    const at::Tensor *dy = p.tensor(1), *first = dy ? dy : p.tensor(2);
    if (!lead(p, dt, first, p.num(20))) return none();
    const int64_t M = first->size(0), H = first->size(1);
    const at::IntArrayRef rows = first->sizes(), vec = rows.slice(1);
    const at::Tensor* gate = p.tensor(9);
    const int64_t gates = gate && gate->dim() == 2 ? gate->size(0) : 0;
    if (gate && !gates) return none();
    const int64_t gate_rows[2] = {gates, H};
    const at::IntArrayRef gate_sizes(gate_rows, 2);
    void *dyd = p.data(1, p.half, rows), *drd = p.data(2, p.half, rows), *xd = p.data(3, p.half, rows), *rd = p.data(4, p.half, rows);
    auto vector = [&](int i) { return (const float*)p.data(i, at::kFloat, vec); };
    const float *w_in = vector(7), *b_in = vector(8), *w_out = vector(11), *b_out = vector(12);
    const float* g = (const float*)p.data(9, at::kFloat, gate_sizes);
    p.data(17, p.half, rows);
    p.data(18, p.half, rows);
    const bool want_dx = is_true(a[14]), want_dres = is_true(a[15]), params = is_true(a[16]);
    const float scale = (float)p.real(5), eps = (float)p.real(13);
    void* stream = (void*)p.num(21);
    if (!p.ok || (a[17] != Py_None && !want_dx) || (a[18] != Py_None && !want_dres)) return none();
    const at::TensorOptions half = first->options(), f32 = half.dtype(at::kFloat);
    at::Tensor dx = given(p, 17), dres = given(p, 18), ws = given(p, 19), dw_in, db_in, dgate, dw_out, db_out;
    if (!p.ok || (ws.defined() && (ws.device() != p.device || !ws.is_contiguous()))) return none();
    int status = GP_OK;
    {
      Unlocked scope;
      make(dx, want_dx, rows, half);
      make(dres, want_dres, rows, half);
      make(dw_in, params && w_in, vec, f32);
      make(db_in, params && b_in, vec, f32);
      make(dgate, params && g, gate_sizes, f32);
      make(dw_out, params && w_out, vec, f32);
      make(db_out, params && b_out, vec, f32);
      if (!ws.defined() && params && (w_in || b_in || g || w_out || b_out)) {
        size_t bytes = 0;
        status = p_norm_backward_size(dt, M, H, gates, &bytes);
        if (!status) ws = at::empty({(int64_t)bytes}, half.dtype(at::kByte));
      }
      if (!status)
        status = p_norm_backward(dt, dyd, drd, xd, rd, scale, kin, w_in, b_in, g, gates, kout, w_out, eps, data_of(dx),
                                 data_of(dres), (float*)data_of(dw_in), (float*)data_of(db_in), (float*)data_of(dgate),
                                 (float*)data_of(dw_out), (float*)data_of(db_out), M, H, data_of(ws),
                                 ws.defined() ? ws.nbytes() : 0, stream);
    }
    if (status) return none();
    return Py_BuildValue("NNNNNNN", wrap(dx), wrap(dres), wrap(dw_in), wrap(db_in), wrap(dgate), wrap(dw_out), wrap(db_out));
  } catch (...) {
    return none();
  }
}

// dt, x, w_shuf, bias, act, residual, save, y, z, workspace, device, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return none();
  try {
    Args p{a};
    const int dt = (int)p.num(0), act = (int)p.num(4);
    const at::Tensor *x = p.tensor(1), *w = p.tensor(2);
    if (!lead(p, dt, x, p.num(10)) || !w) return none();
    const int64_t M = x->size(0), K = x->size(1), Kp = (K + 63) / 64 * 64, N = K ? w->numel() / (2 * Kp) : 0;
    const int64_t out[2] = {M, N}, bytes[1] = {2 * N * Kp}, vec[1] = {N};
    const at::IntArrayRef rows(out, 2);
    void *xd = p.data(1, p.half, x->sizes()), *wd = p.data(2, at::kByte, at::IntArrayRef(bytes, 1));
    const float* bias = (const float*)p.data(3, at::kFloat, at::IntArrayRef(vec, 1));
    void* res = p.data(5, p.half, rows);
    p.data(7, p.half, rows);
    p.data(8, p.half, rows);
    const bool save = is_true(a[6]);
    void* stream = (void*)p.num(11);
    if (!p.ok || (a[8] != Py_None && !save)) return none();
    const at::Tensor ws = given(p, 9);
    if (!p.ok || (ws.defined() && (ws.device() != p.device || !ws.is_contiguous()))) return none();
    const at::TensorOptions half = x->options();
    at::Tensor y = given(p, 7), z = given(p, 8);
    int status = GP_OK;
    {
      Unlocked scope;
      size_t need = 0;   // (without a workspace a call that needs one makes it in Python)
      if (!ws.defined()) status = p_linear_size(dt, M, N, K, &need);
      if (!status && !need) {
        make(y, true, rows, half);
        make(z, save, rows, half);
        status = p_linear(dt, xd, wd, bias, act, res, data_of(y), data_of(z), M, N, K, data_of(ws),
                          ws.defined() ? ws.nbytes() : 0, stream);
      } else {
        status = GP_EWORKSPACE;
      }
    }
    if (status) return none();
    return save ? Py_BuildValue("NN", wrap(y), wrap(z)) : wrap(y);
  } catch (...) {
    return none();
  }
}

// dt, dy, z, x, w, act, want_dx, want_dw, want_dbias, dx, dw, dbias, workspace, device, stream
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) return none();
  try {
    Args p{a};
    const int dt = (int)p.num(0), act = (int)p.num(5);
    const at::Tensor *dy = p.tensor(1), *x = p.tensor(3), *w = p.tensor(4), *wide = w ? w : x;
    if (!lead(p, dt, dy, p.num(13)) || (wide && wide->dim() != 2)) return none();
    const int64_t M = dy->size(0), N = dy->size(1), K = wide ? wide->size(1) : 32;   // (dbias alone: of no consequence)
    const int64_t mk[2] = {M, K}, nk[2] = {N, K}, vec[1] = {N};
    const at::IntArrayRef rows = dy->sizes(), xs(mk, 2), ws_(nk, 2), bs(vec, 1);
    void *dyd = p.data(1, p.half, rows), *zd = p.data(2, p.half, rows), *xd = p.data(3, p.half, xs), *wd = p.data(4, p.half, ws_);
    p.data(9, p.half, xs);
    p.data(10, p.half, ws_);
    p.data(11, at::kFloat, bs);
    const bool want_dx = is_true(a[6]), want_dw = is_true(a[7]), want_db = is_true(a[8]);
    void* stream = (void*)p.num(14);
    if (!p.ok || (a[9] != Py_None && !want_dx) || (a[10] != Py_None && !want_dw) || (a[11] != Py_None && !want_db)) return none();
    if ((want_dx && !wd) || (want_dw && !xd) || (act && !zd)) return none();
    const at::TensorOptions half = dy->options();
    at::Tensor dx = given(p, 9), dw = given(p, 10), db = given(p, 11), ws = given(p, 12);
    if (!p.ok || (ws.defined() && (ws.device() != p.device || !ws.is_contiguous()))) return none();
    int status = GP_OK;
    {
      Unlocked scope;
      if (!ws.defined()) {
        size_t bytes = 0;
        status = p_linear_backward_size(dt, M, N, K, act, want_dx, want_dw, want_db, &bytes);
        if (!status) ws = at::empty({(int64_t)bytes}, half.dtype(at::kByte));
      }
      if (!status) {
        make(dx, want_dx, xs, half);
        make(dw, want_dw, ws_, half);
        make(db, want_db, bs, half.dtype(at::kFloat));
        status = p_linear_backward(dt, dyd, zd, xd, wd, act, data_of(dx), data_of(dw), (float*)data_of(db), M, N, K,
                                   data_of(ws), ws.nbytes(), stream);
      }
    }
    if (status) return none();
    return Py_BuildValue("NNN", wrap(dx), wrap(dw), wrap(db));
  } catch (...) {
    return none();
  }
}

// The addresses of the entry points, in the order of the declarations above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind: seven addresses");
    return nullptr;
  }
  void* at[7];
  for (int i = 0; i < 7; ++i)
    if (!(at[i] = PyLong_AsVoidPtr(a[i])) && PyErr_Occurred()) return nullptr;
  p_norm = (decltype(p_norm))at[0];
  p_norm_backward = (decltype(p_norm_backward))at[1];
  p_norm_backward_size = (decltype(p_norm_backward_size))at[2];
  p_linear = (decltype(p_linear))at[3];
  p_linear_size = (decltype(p_linear_size))at[4];
  p_linear_backward = (decltype(p_linear_backward))at[5];
  p_linear_backward_size = (decltype(p_linear_backward_size))at[6];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {"norm", (PyCFunction)(void*)norm, METH_FASTCALL, nullptr},
                         {"norm_backward", (PyCFunction)(void*)norm_backward, METH_FASTCALL, nullptr},
                         {"linear", (PyCFunction)(void*)linear, METH_FASTCALL, nullptr},
                         {"linear_backward", (PyCFunction)(void*)linear_backward, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// sources: the hash of what it was built from, which the binding compares before it binds
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "sources", GP_MARSHAL_SOURCES)) Py_CLEAR(m);
  return m;
}
