// Calls of the operators in ttt_ops.h on torch tensors: the Python module _token_ops.
//
// Argument checks, outputs that are not given, workspaces and the call itself, for calls
// of a few microseconds (a new token of a stream), of which the same steps through ctypes
// took as long again (one-token rotary call 8.9 us, 4.1 here; one-token recurrence 12.3 and 5.6).  Everything else of
// the binding is in token_ops.py.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ttt_ops.h"

namespace {

using at::Tensor;

// A configured operator: its C handle, its device and the sizes that its tensors must have
struct Context {
  void* handle;
  c10::DeviceIndex index;
  at::ScalarType type;
  int64_t a, b;  // rope: d, axes; scan: D; norm: C, groups
  unsigned* status;
};
constexpr const char* kContext = "ttt_context";

// ------------------------------------------------------------------- arguments
Context& context_of(PyObject* o) {
  TORCH_CHECK_VALUE(o != Py_None, "the operator is closed");
  Context* c = static_cast<Context*>(PyCapsule_GetPointer(o, kContext));
  if (!c) throw python_error();
  return *c;
}

Tensor tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
Tensor optional(PyObject* o, const char* name) { return o == Py_None ? Tensor() : tensor(o, name); }

// on this device, of this shape and type, and its rows contiguous
void check_rows(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType type, const Context& c) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.layout() == at::kStrided, name,
                    ": expected shape ", shape, " of ", type, ", got ", t.sizes(), " of ", t.scalar_type());
  TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == c.index, name, ": expected a tensor on cuda:", int(c.index),
                    ", got one on ", t.device());
  TORCH_CHECK_VALUE(shape.empty() || t.stride(-1) == 1 || shape.back() <= 1, name,
                    ": the channels of a row must be contiguous, got strides ", t.strides());
}
void check_whole(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType type, const Context& c) {
  check_rows(name, t, shape, type, c);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, ": must be contiguous, got strides ", t.strides());
}
void check_bytes(const char* name, const Tensor& t, size_t n, const Context& c) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kByte && t.is_cuda() && t.get_device() == c.index && t.is_contiguous() &&
                        size_t(t.numel()) >= n,
                    name, ": expected at least ", n, " contiguous bytes on cuda:", int(c.index), ", got ", t.numel(), " of ",
                    t.scalar_type(), " on ", t.device());
}

Tensor make(const Context& c, at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, c.index), std::nullopt);
}
Tensor bytes(const Context& c, size_t n) { return n ? make(c, {int64_t(n)}, at::kByte) : Tensor(); }

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(ptr(t));
}
ttt_strides heads(const Tensor& t) { return {t.stride(0), t.stride(1), t.stride(2)}; }
ttt_strides rows(const Tensor& t) { return {t.stride(0), 0, t.stride(1)}; }
// channels last, or a group's tokens together
ttt_strides groups(const Tensor& t, const Context& c) {
  return t.dim() == 3 ? ttt_strides{t.stride(0), c.a / c.b, t.stride(1)} : heads(t);
}

// ----------------------------------------------------------------------- calls
// Runs a library call without the interpreter's lock; raises TTTError where it fails.
template <class F>
void call(const char* where, F&& f) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f();
  Py_END_ALLOW_THREADS;
  if (status == TTT_OK) return;
  PyObject* module = PyImport_ImportModule("weight_sequence_mixing_b200.binding");
  PyObject* error = module ? PyObject_GetAttrString(module, "TTTError") : nullptr;
  PyObject* value = error ? PyObject_CallFunction(error, "is", status, where) : nullptr;
  if (value) PyErr_SetObject(error, value);
  Py_XDECREF(value);
  Py_XDECREF(error);
  Py_XDECREF(module);
  throw python_error();
}
void* stream_of(const Context& c) { return c10::cuda::getCurrentCUDAStream(c.index).stream(); }

PyObject* pack(const Tensor& a, const Tensor& b, const Tensor& c = Tensor()) {
  PyObject* t = PyTuple_New(c.defined() ? 3 : 2);
  if (!t) throw python_error();
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  if (c.defined()) PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(c));
  return t;
}

void check_batch(int64_t n) { TORCH_CHECK_VALUE(n <= INT32_MAX, "expected at most 2^31 - 1 batch entries and heads, got ", n); }

void count(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// context(handle, device index, bf16, a, b, status pointer)
PyObject* new_context(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  int64_t v[6];
  for (int i = 0; i < 6; ++i) v[i] = PyLong_AsLongLong(arg[i]);
  if (PyErr_Occurred()) throw python_error();
  Context* c = new Context{reinterpret_cast<void*>(v[0]), c10::DeviceIndex(v[1]), v[2] ? at::kBFloat16 : at::kFloat,
                           v[3], v[4], reinterpret_cast<unsigned*>(v[5])};
  PyObject* o = PyCapsule_New(c, kContext, [](PyObject* p) { delete static_cast<Context*>(PyCapsule_GetPointer(p, kContext)); });
  if (!o) delete c;
  return o;
  END_HANDLE_TH_ERRORS
}

// rope(context, x, pos, out, inverse)
PyObject* rope(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  const Context& c = context_of(arg[0]);
  const Tensor x = tensor(arg[1], "x"), pos = tensor(arg[2], "pos");
  Tensor out = optional(arg[3], "out");
  const int inverse = PyObject_IsTrue(arg[4]);
  TORCH_CHECK_VALUE(x.dim() == 4, "x: expected [B, H, N, ", c.a, "], got ", x.sizes());
  const int64_t B = x.size(0), H = x.size(1), N = x.size(2);
  check_batch(std::max(B, H));
  check_rows("x", x, {B, H, N, c.a}, c.type, c);
  const bool each = pos.dim() == 3;
  TORCH_CHECK_VALUE(pos.scalar_type() == at::kInt || pos.scalar_type() == at::kFloat, "pos: expected int32 or float32, got ",
                    pos.scalar_type());
  if (each)
    check_whole("pos", pos, {B, N, c.b}, pos.scalar_type(), c);
  else
    check_whole("pos", pos, {N, c.b}, pos.scalar_type(), c);
  if (out.defined()) check_rows("out", out, x.sizes(), c.type, c);
  const c10::cuda::CUDAGuard guard(c.index);
  if (!out.defined()) out = make(c, x.sizes(), c.type);
  if (x.numel()) {
    const ttt_strides xs = heads(x), ys = heads(out);
    call("ttt_rope_apply", [&] {
      return ttt_rope_apply(static_cast<ttt_rope*>(c.handle), int32_t(B), int32_t(H), N, ptr(x), &xs, ptr(pos),
                            pos.scalar_type() == at::kInt ? TTT_POS_I32 : TTT_POS_F32, each ? N * c.b : 0, ptr(out), &ys,
                            inverse, stream_of(c));
    });
  }
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// the sizes of a scan call, after its checks of x and lengths
struct ScanCall {
  const Context& c;
  ttt_scan* handle;
  int64_t B, L;
  std::array<int64_t, 3> shape;
  std::array<int64_t, 2> state;
  ScanCall(const Context& c, const Tensor& x, const Tensor& lengths) : c(c), handle(static_cast<ttt_scan*>(c.handle)) {
    TORCH_CHECK_VALUE(x.dim() == 3 && x.size(0) >= 1, "x: expected [B, L, ", c.a, "], got ", x.sizes());
    B = x.size(0), L = x.size(1);
    check_batch(B);
    shape = {B, L, c.a};
    state = {B, c.a};
    if (lengths.defined()) check_whole("lengths", lengths, {B}, at::kInt, c);
  }
  void rows_of(const char* name, const Tensor& t) const {
    if (t.defined()) check_rows(name, t, shape, c.type, c);
  }
  void state_of(const char* name, const Tensor& t) const {
    if (t.defined()) check_whole(name, t, state, at::kFloat, c);
  }
  void saved_of(const Tensor& t) const { check_bytes("saved (new_saved)", t, ttt_scan_saved_size(handle, int32_t(B), L), c); }
  // rows behind a sequence's end are left as they are: zeros, in a tensor made here
  Tensor output(const Tensor& lengths) const {
    Tensor t = make(c, shape, c.type);
    if (lengths.defined()) {
      const ttt_strides s = rows(t);
      call("ttt_scan_clear",
           [&] { return ttt_scan_clear(handle, int32_t(B), L, ptr<int32_t>(lengths), ptr(t), &s, stream_of(c)); });
    }
    return t;
  }
};

// scan_forward(context, g, x, h0, lengths, saved, out, h_last)
PyObject* scan_forward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Context& c = context_of(arg[0]);
  const Tensor g = tensor(arg[1], "g"), x = tensor(arg[2], "x"), h0 = optional(arg[3], "h0"),
               lengths = optional(arg[4], "lengths"), saved = optional(arg[5], "saved");
  Tensor out = optional(arg[6], "out"), h_last = optional(arg[7], "h_last");
  const ScanCall s(c, x, lengths);
  s.rows_of("x", x), s.rows_of("g", g), s.rows_of("out", out);
  s.state_of("h0", h0), s.state_of("h_last", h_last);
  if (saved.defined()) s.saved_of(saved);
  const c10::cuda::CUDAGuard guard(c.index);
  if (!out.defined()) out = s.output(lengths);
  if (!h_last.defined()) h_last = make(c, s.state, at::kFloat);
  const size_t need = ttt_scan_workspace_size(s.handle, int32_t(s.B), s.L);
  const Tensor ws = bytes(c, need);
  const ttt_strides gs = rows(g), xs = rows(x), hs = rows(out);
  call("ttt_scan_forward", [&] {
    return ttt_scan_forward(s.handle, int32_t(s.B), s.L, ptr(g), &gs, ptr(x), &xs, ptr<float>(h0), ptr<int32_t>(lengths),
                            ptr(out), &hs, ptr<float>(h_last), ptr(saved), ptr(ws), need, c.status, stream_of(c));
  });
  return pack(out, h_last);
  END_HANDLE_TH_ERRORS
}

// scan_backward(context, dh, g, x, saved, dh_last, lengths, dg, dx, dh0)
PyObject* scan_backward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Context& c = context_of(arg[0]);
  const Tensor dh = tensor(arg[1], "dh"), g = tensor(arg[2], "g"), x = tensor(arg[3], "x"), saved = tensor(arg[4], "saved"),
               dh_last = optional(arg[5], "dh_last"), lengths = optional(arg[6], "lengths");
  Tensor dg = optional(arg[7], "dg"), dx = optional(arg[8], "dx"), dh0 = optional(arg[9], "dh0");
  const ScanCall s(c, x, lengths);
  s.rows_of("x", x), s.rows_of("g", g), s.rows_of("dh", dh), s.rows_of("dg", dg), s.rows_of("dx", dx);
  s.state_of("dh_last", dh_last), s.state_of("dh0", dh0);
  s.saved_of(saved);
  const c10::cuda::CUDAGuard guard(c.index);
  if (!dg.defined()) dg = s.output(lengths);
  if (!dx.defined()) dx = s.output(lengths);
  if (!dh0.defined()) dh0 = make(c, s.state, at::kFloat);
  const size_t need = ttt_scan_workspace_size(s.handle, int32_t(s.B), s.L);
  const Tensor ws = bytes(c, need);
  const ttt_strides dhs = rows(dh), gs = rows(g), xs = rows(x), dgs = rows(dg), dxs = rows(dx);
  call("ttt_scan_backward", [&] {
    return ttt_scan_backward(s.handle, int32_t(s.B), s.L, ptr(dh), &dhs, ptr<float>(dh_last), ptr(g), &gs, ptr(x), &xs,
                             ptr<int32_t>(lengths), ptr(saved), ptr(dg), &dgs, ptr(dx), &dxs, ptr<float>(dh0), ptr(ws), need,
                             c.status, stream_of(c));
  });
  return pack(dg, dx, dh0);
  END_HANDLE_TH_ERRORS
}

// scan_saved(context, B, L)
PyObject* scan_saved(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 3);
  const Context& c = context_of(arg[0]);
  const int64_t B = PyLong_AsLongLong(arg[1]), L = PyLong_AsLongLong(arg[2]);
  if (PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(B >= 1 && B <= INT32_MAX && L >= 0, "expected B >= 1 and L >= 0, got ", B, " and ", L);
  const size_t need = ttt_scan_saved_size(static_cast<ttt_scan*>(c.handle), int32_t(B), L);
  return THPVariable_Wrap(bytes(c, std::max<size_t>(need, 16)));
  END_HANDLE_TH_ERRORS
}

// the sizes of a norm call, after its checks of x
struct NormCall {
  const Context& c;
  ttt_norm* handle;
  int64_t B, N;
  std::array<int64_t, 3> shape;
  NormCall(const Context& c, const Tensor& x) : c(c), handle(static_cast<ttt_norm*>(c.handle)) {
    const int64_t each = c.a / c.b;
    TORCH_CHECK_VALUE(x.dim() == 3 || x.dim() == 4, "x: expected [B, N, ", c.a, "] or [B, ", c.b, ", N, ", each, "], got ",
                      x.sizes());
    B = x.size(0), N = x.size(x.dim() - 2);
    check_batch(B);
    TORCH_CHECK_VALUE(B >= 1 && N >= 1, "x: no statistics of an empty tensor, got ", x.sizes());
    shape = {B, N, c.a};
    like_x("x", x, x.dim());
  }
  void like_x(const char* name, const Tensor& t, int64_t dim) const {
    if (dim == 3)
      check_rows(name, t, shape, c.type, c);
    else
      check_rows(name, t, {B, c.b, N, c.a / c.b}, c.type, c);
  }
  void channels(const char* name, const Tensor& t) const {
    if (t.defined()) check_whole(name, t, {c.a}, at::kFloat, c);
  }
  void stats_of(const Tensor& t) const { check_whole("stats", t, {B, c.b, 2}, at::kFloat, c); }
  Tensor workspace(int backward, size_t* need) const {
    *need = ttt_norm_workspace_size(handle, int32_t(B), N, backward);
    return bytes(c, *need);
  }
};

// norm_forward(context, x, weight, bias, stats, out)
PyObject* norm_forward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  const Context& c = context_of(arg[0]);
  const Tensor x = tensor(arg[1], "x"), weight = optional(arg[2], "weight"), bias = optional(arg[3], "bias"),
               stats = optional(arg[4], "stats");
  Tensor out = optional(arg[5], "out");
  const NormCall s(c, x);
  s.channels("weight", weight), s.channels("bias", bias);
  if (stats.defined()) s.stats_of(stats);
  if (out.defined()) check_rows("out", out, s.shape, c.type, c);
  const c10::cuda::CUDAGuard guard(c.index);
  if (!out.defined()) out = make(c, s.shape, c.type);
  size_t need;
  const Tensor ws = s.workspace(0, &need);
  const ttt_strides xs = groups(x, c), ys = groups(out, c);
  call("ttt_norm_forward", [&] {
    return ttt_norm_forward(s.handle, int32_t(s.B), s.N, ptr(x), &xs, ptr<float>(weight), ptr<float>(bias), ptr(out), &ys,
                            ptr<float>(stats), ptr(ws), need, c.status, stream_of(c));
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// norm_backward(context, dy, x, weight, bias, stats, dx, dweight, dbias)
PyObject* norm_backward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Context& c = context_of(arg[0]);
  const Tensor dy = tensor(arg[1], "dy"), x = tensor(arg[2], "x"), weight = optional(arg[3], "weight"),
               bias = optional(arg[4], "bias"), stats = tensor(arg[5], "stats");
  Tensor dx = optional(arg[6], "dx"), dweight = optional(arg[7], "dweight"), dbias = optional(arg[8], "dbias");
  const NormCall s(c, x);
  check_rows("dy", dy, s.shape, c.type, c);
  s.channels("weight", weight), s.channels("bias", bias), s.channels("dweight", dweight), s.channels("dbias", dbias);
  s.stats_of(stats);
  if (dx.defined()) s.like_x("dx", dx, x.dim());
  const c10::cuda::CUDAGuard guard(c.index);
  if (!dx.defined()) dx = make(c, x.sizes(), c.type);
  if (!dweight.defined()) dweight = make(c, {c.a}, at::kFloat);
  if (!dbias.defined()) dbias = make(c, {c.a}, at::kFloat);
  size_t need;
  const Tensor ws = s.workspace(1, &need);
  const ttt_strides dys = groups(dy, c), xs = groups(x, c), dxs = groups(dx, c);
  call("ttt_norm_backward", [&] {
    return ttt_norm_backward(s.handle, int32_t(s.B), s.N, ptr(dy), &dys, ptr(x), &xs, ptr<float>(weight), ptr<float>(bias),
                             ptr<float>(stats), ptr(dx), &dxs, ptr<float>(dweight), ptr<float>(dbias), ptr(ws), need,
                             c.status, stream_of(c));
  });
  return pack(dx, dweight, dbias);
  END_HANDLE_TH_ERRORS
}

// norm_stats(context, B)
PyObject* norm_stats(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 2);
  const Context& c = context_of(arg[0]);
  const int64_t B = PyLong_AsLongLong(arg[1]);
  if (PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(B >= 1, "expected B >= 1, got ", B);
  return THPVariable_Wrap(make(c, {B, c.b, 2}, at::kFloat));
  END_HANDLE_TH_ERRORS
}

#define TTT_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"context", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(new_context)), METH_FASTCALL, nullptr},
    TTT_METHOD(rope),
    TTT_METHOD(scan_forward),
    TTT_METHOD(scan_backward),
    TTT_METHOD(scan_saved),
    TTT_METHOD(norm_forward),
    TTT_METHOD(norm_backward),
    TTT_METHOD(norm_stats),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_token_ops", "Calls of ttt_ops.h on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__token_ops() { return PyModule_Create(&module); }
