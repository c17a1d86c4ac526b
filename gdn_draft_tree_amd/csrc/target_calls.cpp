// The torch binding of libgdntree_target.so: argument checks, pointer extraction and scratch
// allocation for its calls, in C++ because they are made once per layer and step.  A call's kernel
// takes about 3 us where it is small, and checking ten tensors in Python took 10 us; here the whole
// call, launch included, takes about as long as the kernel.
//
// Each function takes the positional arguments that _target.py documents, raises ValueError for a
// tensor that does not fit, and GdnTreeError for a status other than GDNTREE_OK.  With `prepare` it
// returns a Call, which enqueues the same launch again with no checks and holds references to what
// the launch points at.

#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <functional>
#include <initializer_list>
#include <string>

#include "../../include/gdntree_target.h"

namespace {

PyObject *g_error = nullptr;   // GdnTreeError(status, message)
PyObject *g_string = nullptr;  // gdntree_status_str(status)

struct Refuse {};  // a Python exception is set

[[noreturn]] void refuse(const std::string &message) {
  PyErr_SetString(PyExc_ValueError, message.c_str());
  throw Refuse{};
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(std::string(name) + " must be a device tensor");
  return THPVariable_Unpack(o);
}

// The call's device: that of its first tensor, which must be the current one.
int device_of(const at::Tensor &t, const char *name) {
  const int current = c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index();
  if (t.get_device() != current)
    refuse(std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" + std::to_string(current));
  return current;
}

void *check(const at::Tensor &t, const char *name, at::ScalarType dtype, at::IntArrayRef shape, int device) {
  if (t.get_device() != device) refuse(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(device));
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dtype));
  if (t.sizes() != shape) refuse(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

void *check(PyObject *o, const char *name, at::ScalarType dtype, std::initializer_list<int64_t> shape, int device) {
  return check(tensor(o, name), name, dtype, at::IntArrayRef(shape.begin(), shape.size()), device);
}

void *optional(PyObject *o, const char *name, at::ScalarType dtype, std::initializer_list<int64_t> shape, int device) {
  return o == Py_None ? nullptr : check(o, name, dtype, shape, device);
}

int integer(PyObject *o, const char *name) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refuse{};
  if (x != (int)x) refuse(std::string(name) + " is out of range");
  return (int)x;
}

gdntree_dtype rows_dtype(const at::Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return GDNTREE_BF16;
  if (t.scalar_type() == at::kFloat) return GDNTREE_F32;
  refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " of " + name);
}

gdntree_cache cache_of(PyObject *k, PyObject *v, PyObject *ks, PyObject *vs, int device) {
  const at::Tensor &t = tensor(k, "cache.k");
  const bool fp8 = t.scalar_type() == at::kFloat8_e4m3fn;
  if ((!fp8 && t.scalar_type() != at::kBFloat16) || t.dim() != 5)
    refuse("cache.k must be bf16 or float8_e4m3fn [L][pages][H_kv][page_size][d]");
  const auto s = t.sizes();
  for (const int64_t x : s)
    if (x > INT32_MAX) refuse("cache.k is too large");
  gdntree_cache c;
  c.k = check(t, "cache.k", t.scalar_type(), s, device);
  c.v = check(tensor(v, "cache.v"), "cache.v", t.scalar_type(), s, device);
  c.k_scale = c.v_scale = nullptr;
  if (fp8) {
    if (ks == Py_None || vs == Py_None) refuse("an e4m3 cache needs k_scale and v_scale");
    c.k_scale = static_cast<uint8_t *>(check(tensor(ks, "cache.k_scale"), "cache.k_scale", at::kByte, s.slice(0, 4), device));
    c.v_scale = static_cast<uint8_t *>(check(tensor(vs, "cache.v_scale"), "cache.v_scale", at::kByte, s.slice(0, 4), device));
  }
  c.L = (int)s[0];
  c.pages = (int)s[1];
  c.H_kv = (int)s[2];
  c.page_size = (int)s[3];
  c.d = (int)s[4];
  c.dtype = fp8 ? GDNTREE_CACHE_E4M3 : GDNTREE_CACHE_BF16;
  return c;
}

const int32_t *table_of(PyObject *o, int64_t B, int device, int *width) {
  const at::Tensor &t = tensor(o, "table");
  if (t.dim() != 2 || t.size(1) > INT32_MAX) refuse("table must be [B][max_pages]");
  *width = (int)t.size(1);
  return static_cast<const int32_t *>(check(t, "table", at::kInt, {B, t.size(1)}, device));
}

void limit(int64_t x, const char *name) {
  if (x > INT32_MAX) refuse(std::string(name) + " is too large");
}

// The scratch tensor of a call: the given one, or a new one (kept alive by `own`).
void *scratch(PyObject *o, size_t size, int device, at::Tensor &own, size_t *given) {
  if (o == Py_None) {
    *given = size;
    if (size == 0) return nullptr;
    own = at::empty({(int64_t)size}, at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
    return own.data_ptr();
  }
  const at::Tensor &t = tensor(o, "workspace");
  if (t.get_device() != device || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on the call's device");
  *given = t.nbytes();
  return t.data_ptr();
}

// ---- prepared calls --------------------------------------------------------------------------------

struct Call {
  PyObject_HEAD
  std::function<gdntree_status()> *launch;
  PyObject *keep;    // what the launch points at
  PyObject *result;
};

void raise(gdntree_status st) {
  PyObject *message = PyObject_CallFunction(g_string, "i", (int)st);
  if (!message) return;
  PyObject *e = PyObject_CallFunction(g_error, "iO", (int)st, message);
  Py_DECREF(message);
  if (!e) return;
  PyErr_SetObject(g_error, e);
  Py_DECREF(e);
}

template <class F>
gdntree_status enqueue(const F &launch) {
  gdntree_status st;
  Py_BEGIN_ALLOW_THREADS
  st = launch();
  Py_END_ALLOW_THREADS
  return st;
}

PyObject *call_again(PyObject *self, PyObject *, PyObject *) {
  Call *c = reinterpret_cast<Call *>(self);
  const gdntree_status st = enqueue(*c->launch);
  if (st != GDNTREE_OK) {
    raise(st);
    return nullptr;
  }
  Py_INCREF(c->result);
  return c->result;
}

void call_free(PyObject *self) {
  Call *c = reinterpret_cast<Call *>(self);
  delete c->launch;
  Py_XDECREF(c->keep);
  Py_XDECREF(c->result);
  Py_TYPE(self)->tp_free(self);
}

PyObject *call_result(PyObject *self, void *) {
  PyObject *r = reinterpret_cast<Call *>(self)->result;
  Py_INCREF(r);
  return r;
}

PyGetSetDef call_get[] = {{"result", call_result, nullptr, "what the call returns", nullptr}, {nullptr}};
PyTypeObject CallType = {PyVarObject_HEAD_INIT(nullptr, 0)};

// Enqueues the launch, or (prepare) makes a Call of it.  Takes the reference to result.
template <class F>
PyObject *finish(F launch, PyObject *const *args, Py_ssize_t n, const at::Tensor &own, PyObject *result, bool prepare) {
  if (!prepare) {
    const gdntree_status st = enqueue(launch);
    if (st == GDNTREE_OK) return result;
    Py_DECREF(result);
    raise(st);
    return nullptr;
  }
  PyObject *keep = PyTuple_New(n + 1);
  Call *c = keep ? PyObject_New(Call, &CallType) : nullptr;
  if (!c) {
    Py_XDECREF(keep);
    Py_DECREF(result);
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    Py_INCREF(args[i]);
    PyTuple_SET_ITEM(keep, i, args[i]);
  }
  PyObject *ws = Py_None;
  if (own.defined()) ws = THPVariable_Wrap(own);
  else Py_INCREF(ws);
  PyTuple_SET_ITEM(keep, n, ws);
  c->launch = new std::function<gdntree_status()>(launch);
  c->keep = keep;
  c->result = result;
  return reinterpret_cast<PyObject *>(c);
}

PyObject *none() {
  Py_INCREF(Py_None);
  return Py_None;
}

PyObject *owned(PyObject *o) {
  Py_INCREF(o);
  return o;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, int device) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}

hipStream_t stream_of(PyObject *o) { return static_cast<hipStream_t>(PyLong_AsVoidPtr(o)); }

#define ARGS(N)                                                              \
  if (n != N) {                                                              \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");           \
    return nullptr;                                                          \
  }                                                                          \
  HANDLE_TH_ERRORS                                                           \
  try {
#define DONE                                                                 \
  } catch (const Refuse &) {                                                 \
    return nullptr;                                                          \
  }                                                                          \
  END_HANDLE_TH_ERRORS

// ---- the calls -------------------------------------------------------------------------------------

// cache k, v, k_scale, v_scale, layer, table, start, k, v, count, stream, prepare
PyObject *cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  ARGS(12)
  const at::Tensor &k = tensor(a[7], "k");
  const int dev = device_of(k, "k");
  if (k.dim() != 4) refuse("k must be [B][R][H_kv][d]");
  const auto s = k.sizes();
  const gdntree_cache c = cache_of(a[0], a[1], a[2], a[3], dev);
  if (s[2] != c.H_kv || s[3] != c.d) refuse("the rows do not match the cache's heads");
  limit(s[0], "B"), limit(s[1], "R");
  int width;
  const int layer = integer(a[4], "layer");
  const int32_t *table = table_of(a[5], s[0], dev, &width);
  const auto *start = static_cast<const int32_t *>(check(a[6], "start", at::kInt, {s[0]}, dev));
  const auto *count = static_cast<const int32_t *>(optional(a[9], "count", at::kInt, {s[0]}, dev));
  const gdntree_dtype dt = rows_dtype(k, "k");
  const void *kp = check(k, "k", k.scalar_type(), s, dev), *vp = check(tensor(a[8], "v"), "v", k.scalar_type(), s, dev);
  const hipStream_t st = stream_of(a[10]);
  const int B = (int)s[0], R = (int)s[1];
  return finish([=] { return gdntree_cache_write(c, layer, table, width, start, count, B, R, dt, kp, vp, st); }, a, n,
                at::Tensor(), none(), PyObject_IsTrue(a[11]) == 1);
  DONE
}

// cache k, v, k_scale, v_scale, layer, table, start, R, count, out k, out v, stream, prepare
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  ARGS(13)
  const at::Tensor &start_t = tensor(a[6], "start");
  const int dev = device_of(start_t, "start");
  if (start_t.dim() != 1) refuse("start must be [B]");
  const gdntree_cache c = cache_of(a[0], a[1], a[2], a[3], dev);
  const int64_t B = start_t.size(0);
  limit(B, "B");
  const int R = integer(a[7], "R"), layer = integer(a[4], "layer");
  int width;
  const int32_t *table = table_of(a[5], B, dev, &width);
  const auto *start = static_cast<const int32_t *>(check(start_t, "start", at::kInt, {B}, dev));
  const auto *count = static_cast<const int32_t *>(optional(a[8], "count", at::kInt, {B}, dev));
  const at::Tensor &k = tensor(a[9], "k");
  const gdntree_dtype dt = rows_dtype(k, "k");
  void *kp = check(k, "k", k.scalar_type(), {B, R, c.H_kv, c.d}, dev);
  void *vp = check(a[10], "v", k.scalar_type(), {B, R, c.H_kv, c.d}, dev);
  const hipStream_t st = stream_of(a[11]);
  PyObject *result = PyTuple_Pack(2, a[9], a[10]);
  if (!result) return nullptr;
  return finish([=] { return gdntree_cache_read(c, layer, table, width, start, count, (int)B, R, dt, kp, vp, st); }, a, n,
                at::Tensor(), result, PyObject_IsTrue(a[12]) == 1);
  DONE
}

// cache k, v, k_scale, v_scale, table, ctx_len, acc_len, acc_node, N, stream, prepare
PyObject *cache_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
  ARGS(11)
  const at::Tensor &node_t = tensor(a[7], "acc_node");
  const int dev = device_of(node_t, "acc_node");
  if (node_t.dim() != 2) refuse("acc_node must be [B][P+1]");
  const gdntree_cache c = cache_of(a[0], a[1], a[2], a[3], dev);
  const int64_t B = node_t.size(0), P1 = node_t.size(1);
  limit(B, "B"), limit(P1, "P");
  int width;
  const int32_t *table = table_of(a[4], B, dev, &width);
  const auto *ctx = static_cast<const int32_t *>(check(a[5], "ctx_len", at::kInt, {B}, dev));
  const auto *len = static_cast<const int32_t *>(check(a[6], "acc_len", at::kInt, {B}, dev));
  const auto *node = static_cast<const int32_t *>(check(node_t, "acc_node", at::kInt, {B, P1}, dev));
  const int N = integer(a[8], "N");
  const hipStream_t st = stream_of(a[9]);
  return finish([=] { return gdntree_cache_commit(c, table, width, ctx, (int)B, N, (int)P1 - 1, len, node, st); }, a, n,
                at::Tensor(), none(), PyObject_IsTrue(a[10]) == 1);
  DONE
}

// q, cache k, v, k_scale, v_scale, layer, table, ctx_len, anc, n_rows, scale, o, workspace, stream, prepare
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  ARGS(15)
  const at::Tensor &q = tensor(a[0], "q");
  const int dev = device_of(q, "q");
  if (q.dim() != 4) refuse("q must be [B][R][H_q][d]");
  const auto s = q.sizes();
  for (int i = 0; i < 4; ++i) limit(s[i], "q");
  const gdntree_cache c = cache_of(a[1], a[2], a[3], a[4], dev);
  if (s[3] != c.d) refuse("q does not match the cache's head size");
  const int layer = integer(a[5], "layer"), B = (int)s[0], R = (int)s[1], Hq = (int)s[2];
  int width;
  const int32_t *table = table_of(a[6], B, dev, &width);
  const auto *ctx = static_cast<const int32_t *>(check(a[7], "ctx_len", at::kInt, {B}, dev));
  const auto *anc = static_cast<const uint64_t *>(optional(a[8], "tree.anc", at::kLong, {B, R}, dev));
  const auto *rows = static_cast<const int32_t *>(optional(a[9], "n_rows", at::kInt, {B}, dev));
  double scale = 1.0 / std::sqrt((double)c.d);
  if (a[10] != Py_None) {
    scale = PyFloat_AsDouble(a[10]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const gdntree_dtype dt = rows_dtype(q, "q");
  const void *qp = check(q, "q", q.scalar_type(), s, dev);
  PyObject *result = a[11] == Py_None ? THPVariable_Wrap(fresh(s, q.scalar_type(), dev)) : owned(a[11]);
  if (!result) return nullptr;
  void *op;
  at::Tensor own;
  size_t size = 0;
  void *ws;
  try {
    op = check(tensor(result, "o"), "o", q.scalar_type(), s, dev);
    ws = scratch(a[12], gdntree_attend_workspace(R, Hq, c.H_kv, c.d, width, c.page_size), dev, own, &size);
  } catch (...) {
    Py_DECREF(result);
    throw;
  }
  const hipStream_t st = stream_of(a[13]);
  const float sc = (float)scale;
  return finish([=] { return gdntree_attend(c, layer, table, width, ctx, anc, rows, B, R, Hq, dt, qp, sc, op, ws, size, st); },
                a, n, own, result, PyObject_IsTrue(a[14]) == 1);
  DONE
}

// parent, token, n_nodes, logits, temperature, uniform, P, acc_len, acc_tok, acc_node, workspace, stream, prepare
PyObject *accept_sample(PyObject *, PyObject *const *a, Py_ssize_t n) {
  ARGS(13)
  const at::Tensor &logits = tensor(a[3], "logits");
  const int dev = device_of(logits, "logits");
  if (logits.dim() != 3) refuse("logits must be [B][N+1][V]");
  const auto s = logits.sizes();
  for (int i = 0; i < 3; ++i) limit(s[i], "logits");
  const int B = (int)s[0], R = (int)s[1], V = (int)s[2], P = integer(a[6], "P");
  gdntree_tree tree{};
  tree.parent = static_cast<int32_t *>(check(a[0], "tree.parent", at::kInt, {B, R}, dev));
  tree.token = static_cast<int32_t *>(check(a[1], "tree.token", at::kInt, {B, R}, dev));
  tree.n_nodes = static_cast<int32_t *>(check(a[2], "tree.n_nodes", at::kInt, {B}, dev));
  const gdntree_dtype dt = rows_dtype(logits, "logits");
  const void *lp = check(logits, "logits", logits.scalar_type(), s, dev);
  const auto *temp = static_cast<const float *>(check(a[4], "temperature", at::kFloat, {B}, dev));
  const auto *uni = static_cast<const double *>(check(a[5], "uniform", at::kDouble, {B, R}, dev));
  PyObject *acc[3];
  for (int i = 0; i < 3; ++i) acc[i] = a[7 + i];
  PyObject *result;
  if (acc[0] == Py_None) {
    if (P < 0 || P > 1 << 20) refuse("P is out of range");
    // one allocation: the lengths, then the tokens, then the slots
    const at::Tensor all = fresh({(int64_t)B * (2 * P + 3)}, at::kInt, dev);
    const int64_t wide = (int64_t)B * (P + 1);
    PyObject *x = THPVariable_Wrap(all.narrow(0, 0, B)), *y = THPVariable_Wrap(all.narrow(0, B, wide).view({B, P + 1})),
             *z = THPVariable_Wrap(all.narrow(0, B + wide, wide).view({B, P + 1}));
    result = PyTuple_Pack(3, x, y, z);
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    if (!result) return nullptr;
    for (int i = 0; i < 3; ++i) acc[i] = PyTuple_GET_ITEM(result, i);
  } else {
    result = PyTuple_Pack(3, acc[0], acc[1], acc[2]);
    if (!result) return nullptr;
  }
  int32_t *out[3];
  at::Tensor own;
  size_t size = 0;
  void *ws;
  try {
    out[0] = static_cast<int32_t *>(check(acc[0], "acc_len", at::kInt, {B}, dev));
    out[1] = static_cast<int32_t *>(check(acc[1], "acc_tok", at::kInt, {B, P + 1}, dev));
    out[2] = static_cast<int32_t *>(check(acc[2], "acc_node", at::kInt, {B, P + 1}, dev));
    ws = scratch(a[10], gdntree_accept_sample_workspace(B, R - 1, V), dev, own, &size);
  } catch (...) {
    Py_DECREF(result);
    throw;
  }
  const hipStream_t st = stream_of(a[11]);
  int32_t *o0 = out[0], *o1 = out[1], *o2 = out[2];
  return finish([=] { return gdntree_accept_sample(tree, B, R - 1, P, V, dt, lp, temp, uni, o0, o1, o2, ws, size, st); }, a,
                n, own, result, PyObject_IsTrue(a[12]) == 1);
  DONE
}

PyObject *set_errors(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "set_errors(error class, status text)");
    return nullptr;
  }
  g_error = owned(a[0]);
  g_string = owned(a[1]);
  return none();
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(cache_write), METHOD(cache_read), METHOD(cache_commit), METHOD(attend),
                         METHOD(accept_sample), METHOD(set_errors), {nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Checked calls of libgdntree_target.so on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  CallType.tp_name = "gdn_draft_tree_amd.Call";
  CallType.tp_basicsize = sizeof(Call);
  CallType.tp_flags = Py_TPFLAGS_DEFAULT;
  CallType.tp_doc = "A prepared call: enqueues the same launch again, with no checks.";
  CallType.tp_call = call_again;
  CallType.tp_dealloc = call_free;
  CallType.tp_getset = call_get;
  if (PyType_Ready(&CallType) < 0) return nullptr;
  return PyModule_Create(&module);
}
