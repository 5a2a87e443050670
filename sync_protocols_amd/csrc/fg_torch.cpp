// The decoding operators on torch tensors: argument checks, outputs, stream and
// the call of the C entry (include/fg.h). ops.py holds the documented functions;
// what they do per call lives here because it is most of the time of a small
// call: 12 us for the router of one token in Python, of which the launch is 3 us.
//
// Refusals raise fg.FgError with FG_EINVAL, set up by setup(); torch's own errors
// (out of memory) pass through as they are.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fg.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;       // fg.FgError

struct Refused {};

[[noreturn]] void raise(int code, const char* what) {
  PyObject* e = PyObject_CallFunction(g_error, "is", code, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}
[[noreturn]] void refuse(const char* what) { raise(FG_EINVAL, what); }

// A tensor argument; None is an empty one where that is allowed.
const Tensor* maybe(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o) {
  const Tensor* t = maybe(o);
  if (!t) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor, got None");
    throw Refused();
  }
  return *t;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int32_t int32_of(PyObject* o, const char* what) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(what);
  return (int32_t)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}
const char* text(PyObject* o) {
  const char* v = PyUnicode_AsUTF8(o);
  if (!v) throw Refused();
  return v;
}

bool is_type(const Tensor& t, ScalarType s) { return t.scalar_type() == s; }
bool is_shape(const Tensor& t, at::IntArrayRef s) { return t.sizes() == s; }

void rows2d(const Tensor& t, const char* what) {
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1))) refuse(what);
}
#define ROWS2D(t, name) rows2d(t, name " must be [rows, columns] with consecutive columns and rows that do not overlap")

// Row distance in elements; that of a single row does not matter.
int64_t ld(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : (t.size(1) + 7) / 8 * 8; }

bool vector_of(const Tensor& t, int64_t n) { return t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1); }

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// One call: its stream, and its tensors, all on one GPU.
//
// On another stream than the current one, what the call allocates comes from that
// stream's memory: a block that the current stream has freed may still be read there
// by kernels that have not run, and nothing orders the other stream after them. The
// allocator is told that the caller's tensors are used on the other stream, and that
// new outputs, which the caller goes on with, may be used on the current one.
struct Call {
  const Tensor* used[16];
  int n = 0;
  c10::Device device;
  std::optional<c10::Stream> other;
  hipStream_t handle = nullptr;
  explicit Call(const Tensor& t) : device(t.device()) {}
  // The stream of the launch: the device's current one, or `s`.
  void on(PyObject* s) {
    if (!device.is_cuda()) refuse("tensors must be on the GPU");
    if (s == Py_None) {
      handle = c10::hip::getCurrentHIPStream(device.index()).stream();
      return;
    }
    int64_t part[3];
    const char* name[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* v = PyObject_GetAttrString(s, name[i]);
      if (!v) throw Refused();
      part[i] = PyLong_AsLongLong(v);
      Py_DECREF(v);
      if (part[i] == -1 && PyErr_Occurred()) throw Refused();
    }
    if (part[1] != device.index()) refuse("stream and tensors are on different devices");
    PyObject* v = PyObject_GetAttrString(s, "cuda_stream");
    if (!v) throw Refused();
    handle = (hipStream_t)PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Refused();
    const c10::Stream st = c10::Stream::unpack3(part[0], (c10::DeviceIndex)part[1], (c10::DeviceType)part[2]);
    if (st != current()) other = st;
  }
  c10::Stream current() const { return c10::impl::VirtualGuardImpl(device.type()).getStream(device); }
  void use(const Tensor* t) {
    if (!t) return;
    if (t->device() != device) refuse("tensors are on different devices");
    no_gradient(*t);
    used[n++] = t;
  }
  // The results have no gradient function, so a tensor that needs one is no input (nor an output buffer).
  static void no_gradient(const Tensor& t) {
    if (t.requires_grad() && at::GradMode::is_enabled())
      refuse("the decoding operators have no backward pass: call them under torch.no_grad() or detach their inputs");
  }
  // Memory of the launching stream.
  Tensor memory(at::IntArrayRef shape, ScalarType type) const {
    const c10::OptionalStreamGuard guard(other);
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }
  void check(const Tensor* given, at::IntArrayRef shape, ScalarType type, const char* what) const {
    if (!given) return;
    if (!is_type(*given, type) || !is_shape(*given, shape) || given->device() != device) refuse(what);
    no_gradient(*given);
  }
  // The output `given`, which has been checked, or a new one. Autograd, which may have
  // saved a given one, is told that it is written.
  Tensor out(const Tensor* given, at::IntArrayRef shape, ScalarType type) {
    if (given) {
      use(given);
      if (!given->is_inference()) given->unsafeGetTensorImpl()->bump_version();
      return *given;
    }
    const Tensor t = memory(shape, type);
    if (other) t.record_stream(current());
    return t;
  }
  void record() const {
    if (!other) return;
    for (int i = 0; i < n; ++i) used[i]->record_stream(*other);
  }
};

struct WithoutGil {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

template <class F>
void launch(const Call& c, const char* name, F f) {
  c.record();
  fg_status code;
  {
    const WithoutGil released;
    const c10::DeviceGuard guard(c.device);
    code = f();
  }
  if (code != FG_OK) raise(code, name);
}

template <class F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const Tensor& t, bool there = true) { return there ? THPVariable_Wrap(t) : none(); }

// A tuple of new references; nullptr if one of them is.
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  bool ok = t != nullptr;
  for (PyObject* o : items) {
    if (!o) ok = false;
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  if (ok) return t;
  Py_XDECREF(t);
  return nullptr;
}

bool counted(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
  return false;
}

// x, gamma, residual, eps, out, group, keep_bf16, sum, y, q, scale, stream -> (sum, y, q, scale)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &x = tensor(a[0]), &gamma = tensor(a[1]);
    const Tensor *res = maybe(a[2]), *sum_in = maybe(a[7]), *y_in = maybe(a[8]), *q_in = maybe(a[9]), *scale_in = maybe(a[10]);
    ROWS2D(x, "x");
    const int64_t rows = x.size(0), n = x.size(1);
    if (!is_type(x, at::kBFloat16) || !is_type(gamma, at::kBFloat16) || !vector_of(gamma, n))
      refuse("x must be bf16 [rows, n] and gamma bf16 [n]");
    if (res) {
      ROWS2D(*res, "residual");
      if (!is_type(*res, at::kBFloat16) || res->sizes() != x.sizes()) refuse("residual must be bf16 like x");
    }
    const std::string_view kind = text(a[4]);
    const bool i8 = kind == "i8", e4m3 = kind == "e4m3", bits8 = i8 || e4m3;
    if (!bits8 && kind != "bf16") refuse("out must be 'bf16', 'i8' or 'e4m3'");
    const int64_t group = integer(a[5]);
    if ((group != 0 && group != 128) || (group && (n % 128 || !bits8)))
      refuse("group must be 0, or 128 for 8-bit outputs of a multiple of 128 columns");
    if (!bits8 && (q_in || scale_in)) refuse("q and scale need an 8-bit out");
    if (n > FG_NORM_MAX_N || n < 1) refuse("fg_add_rmsnorm takes 1 to 65536 columns");
    Call c(x);
    const bool has_sum = res || sum_in, has_y = !bits8 || truth(a[6]) || y_in;
    const ScalarType qt = i8 ? at::kChar : at::kFloat8_e4m3fn;
    // what is given is checked before anything is allocated
    if (sum_in) { c.check(sum_in, x.sizes(), at::kBFloat16, "sum must be bf16 like x"); ROWS2D(*sum_in, "sum"); }
    if (y_in) { c.check(y_in, x.sizes(), at::kBFloat16, "y must be bf16 like x"); ROWS2D(*y_in, "y"); }
    if (q_in) { c.check(q_in, x.sizes(), qt, "q must be of the type that out names and like x"); ROWS2D(*q_in, "q"); }
    const int64_t sshape[2] = {rows, group ? n / group : 1};
    if (scale_in) {
      c.check(scale_in, sshape, at::kFloat, "scale must be float32 [rows, 1 or n / 128]");
      if (!scale_in->is_contiguous()) refuse("scale must be contiguous");
    }
    const float eps = (float)number(a[3]);
    c.use(&x); c.use(&gamma); c.use(res);
    c.on(a[11]);
    Tensor sum, y, q, scale;
    if (has_sum) sum = c.out(sum_in, x.sizes(), at::kBFloat16);
    if (has_y) y = c.out(y_in, x.sizes(), at::kBFloat16);
    if (bits8) {
      q = c.out(q_in, x.sizes(), qt);
      scale = c.out(scale_in, sshape, at::kFloat);
    }
    launch(c, "fg_add_rmsnorm", [&] {
      return fg_add_rmsnorm(x.data_ptr(), ld(x), ptr(res), res ? ld(*res) : 0, gamma.data_ptr(), eps, has_sum ? sum.data_ptr() : nullptr,
                            has_sum ? ld(sum) : 0, has_y ? y.data_ptr() : nullptr, has_y ? ld(y) : 0, bits8 ? q.data_ptr() : nullptr,
                            bits8 ? ld(q) : 0, i8 ? FG_I8 : FG_E4M3, (int32_t)group, bits8 ? (float*)scale.data_ptr() : nullptr, rows,
                            (int32_t)n, c.handle);
    });
    return tuple({wrap(sum, has_sum), wrap(y, has_y), wrap(q, bits8), wrap(scale, bits8)});
  });
}

// logits, k, score, renorm, scale, topk, weights, stream -> (topk, weights)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& l = tensor(a[0]);
    const Tensor *topk_in = maybe(a[5]), *w_in = maybe(a[6]);
    ROWS2D(l, "logits");
    const std::string_view score = text(a[2]);
    const bool softmax = score == "softmax";
    if ((!is_type(l, at::kFloat) && !is_type(l, at::kBFloat16)) || (!softmax && score != "sigmoid"))
      refuse("logits must be float32 or bf16, score 'softmax' or 'sigmoid'");
    const int64_t rows = l.size(0), experts = l.size(1), k = integer(a[1]);
    if (k < 1 || k > experts || k > 64) refuse("k must be in 1..min(experts, 64)");
    if (experts > FG_MOE_FEW_EXPERTS) refuse("moe_route takes up to 1024 experts");
    Call c(l);
    const int64_t shape[2] = {rows, k};
    c.check(topk_in, shape, at::kInt, "topk must be int32 [rows, k]");
    c.check(w_in, shape, at::kFloat, "weights must be float32 [rows, k]");
    if ((topk_in && !topk_in->is_contiguous()) || (w_in && !w_in->is_contiguous())) refuse("topk and weights must be contiguous");
    const bool renorm = truth(a[3]);
    const float scale = (float)number(a[4]);
    c.use(&l);
    c.on(a[7]);
    const Tensor topk = c.out(topk_in, shape, at::kInt), w = c.out(w_in, shape, at::kFloat);
    launch(c, "fg_moe_route", [&] {
      return fg_moe_route(l.data_ptr(), ld(l), is_type(l, at::kFloat) ? FG_F32 : FG_BF16, rows, (int32_t)experts, (int32_t)k,
                          softmax ? FG_SCORE_SOFTMAX : FG_SCORE_SIGMOID, renorm ? 1 : 0, scale, (int32_t*)topk.data_ptr(),
                          (float*)w.data_ptr(), c.handle);
    });
    return tuple({wrap(topk), wrap(w)});
  });
}

// Activation rows [rows, k] of the products: element type and scale group.
struct Activations {
  int32_t type, group;
};
Activations activations(const Tensor& x, const Tensor* scale, int64_t k) {
  ROWS2D(x, "x");
  const int32_t type = is_type(x, at::kBFloat16) ? FG_BF16 : is_type(x, at::kChar) ? FG_I8 : is_type(x, at::kFloat8_e4m3fn) ? FG_E4M3 : -1;
  if (type < 0 || x.size(1) != k) refuse("x must be bf16, int8 or float8_e4m3fn with as many columns as the weights");
  if (type == FG_BF16) {
    if (scale) refuse("bf16 activations take no x_scale");
    return {type, 0};
  }
  if (!scale || !is_type(*scale, at::kFloat) || !scale->is_contiguous()) refuse("8-bit activations need a contiguous float32 x_scale");
  const int64_t rows = x.size(0);
  if (scale->dim() == 1 ? scale->size(0) == rows : scale->dim() == 2 && scale->size(0) == rows && scale->size(1) == 1) return {type, 0};
  if (k % 128 == 0 && scale->dim() == 2 && scale->size(0) == rows && scale->size(1) == k / 128) return {type, 128};
  refuse("x_scale must be [rows], [rows, 1] or [rows, k / 128]");
}

// 4-bit weights of `dims` leading sizes and k columns: their group.
struct Weight4 {
  const Tensor *q, *scale, *zero;
};
int32_t group_of(const Weight4& w, int dim, int64_t k) {
  if (!is_type(*w.q, at::kByte) || w.q->dim() != dim || !w.q->is_contiguous()) refuse("w.q must be contiguous uint8 [.., n, k // 2]");
  const Tensor& s = *w.scale;
  const int64_t groups = s.dim() ? s.size(-1) : 0;
  if (!is_type(s, at::kBFloat16) || s.dim() != dim || groups < 1 || k % groups || !s.is_contiguous())
    refuse("w.scale must be contiguous bf16 [.., n, k // group]");
  for (int i = 0; i < dim - 1; ++i)
    if (s.size(i) != w.q->size(i)) refuse("w.scale must have w.q's rows");
  if (w.zero && (!is_type(*w.zero, at::kByte) || w.zero->sizes() != s.sizes() || !w.zero->is_contiguous()))
    refuse("w.zero must be contiguous uint8 like w.scale");
  const int64_t g = k / groups;
  if (g != 32 && g != 64 && g != 128) refuse("groups must be of 32, 64 or 128 weights");
  return (int32_t)g;
}

void fits_int32(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(what);
}

// x, x_scale, q, scale, zero, bias, out, stream -> out
PyObject* w4_linear(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& x = tensor(a[0]);
    const Tensor *xs = maybe(a[1]), *bias = maybe(a[5]), *out_in = maybe(a[6]);
    const Weight4 w{&tensor(a[2]), &tensor(a[3]), maybe(a[4])};
    if (w.q->dim() != 2) refuse("w.q must be [n, k // 2]");
    const int64_t n = w.q->size(0), k = 2 * w.q->size(1);
    const Activations act = activations(x, xs, k);
    const int32_t group = group_of(w, 2, k);
    fits_int32(n, "w has too many rows");
    fits_int32(k, "w has too many columns");
    if (bias && (!is_type(*bias, at::kBFloat16) || !vector_of(*bias, n))) refuse("bias must be bf16 [n]");
    Call c(x);
    const int64_t rows = x.size(0), shape[2] = {rows, n};
    if (out_in) { c.check(out_in, shape, at::kBFloat16, "out must be bf16 [rows, n]"); ROWS2D(*out_in, "out"); }
    c.use(&x); c.use(xs); c.use(w.q); c.use(w.scale); c.use(w.zero); c.use(bias);
    c.on(a[7]);
    const Tensor out = c.out(out_in, shape, at::kBFloat16);
    launch(c, "fg_w4_linear", [&] {
      return fg_w4_linear(x.data_ptr(), ld(x), act.type, (const float*)ptr(xs), act.group, w.q->data_ptr(), w.scale->data_ptr(),
                          ptr(w.zero), group, ptr(bias), out.data_ptr(), ld(out), rows, (int32_t)n, (int32_t)k, c.handle);
    });
    return wrap(out);
  });
}

// x, x_scale, w1, w1 scale, w1 zero, w2, w2 scale, w2 zero, topk, weights, expert_base, out, workspace, stream -> out
// (scales None: 16-bit weights)
PyObject* moe_few(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &x = tensor(a[0]), &topk = tensor(a[8]), &weights = tensor(a[9]);
    const Tensor *xs = maybe(a[1]), *out_in = maybe(a[11]), *ws_in = maybe(a[12]);
    const Weight4 w1{&tensor(a[2]), maybe(a[3]), maybe(a[4])}, w2{&tensor(a[5]), maybe(a[6]), maybe(a[7])};
    const bool quant = w1.scale != nullptr;
    if (quant != (w2.scale != nullptr)) refuse("w1 and w2 must be of the same kind");
    if (w1.q->dim() != 3 || w2.q->dim() != 3 || x.dim() != 2) refuse("x must be [tokens, K], w1 and w2 [experts, rows, columns]");
    const int64_t tokens = x.size(0), K = x.size(1), n_local = w1.q->size(0), F = w1.q->size(1) / 2;
    const int64_t per = quant ? 2 : 1;          // elements a stored column
    if (w1.q->size(1) % 2 || w1.q->size(2) * per != K || w2.q->size(0) != n_local || w2.q->size(1) != K || w2.q->size(2) * per != F)
      refuse("w1 must be [n_local, 2F, K] and w2 [n_local, K, F]");
    int32_t group = 0;
    if (quant) {
      group = group_of(w1, 3, K);
      if (group_of(w2, 3, F) != group) refuse("w1 and w2 must have the same group size");
    } else if (!is_type(*w1.q, at::kBFloat16) || !is_type(*w2.q, at::kBFloat16) || !w1.q->is_contiguous() || !w2.q->is_contiguous()) {
      refuse("w1 and w2 must be contiguous bf16");
    }
    const Activations act = activations(x, xs, K);
    if (!is_type(topk, at::kInt) || !is_type(weights, at::kFloat) || topk.dim() != 2 || topk.size(0) != tokens ||
        weights.sizes() != topk.sizes())
      refuse("topk must be int32 [tokens, k] and weights float32 like it");
    if (!topk.is_contiguous() || !weights.is_contiguous()) refuse("topk and weights must be contiguous");
    const int64_t k = topk.size(1);
    if (tokens > FG_MOE_FEW_TOKENS || k < 1 || k > FG_MOE_FEW_TOPK) refuse("moe_few takes up to 64 tokens with 1..16 picks each");
    if (n_local < 1 || n_local > FG_MOE_FEW_EXPERTS) refuse("moe_few takes 1 to 1024 experts");
    fits_int32(K, "too many columns");
    fits_int32(2 * F, "too many rows");
    const int32_t base = int32_of(a[10], "expert_base must be an int32");
    Call c(x);
    const int64_t shape[2] = {tokens, K};
    if (out_in) { c.check(out_in, shape, at::kBFloat16, "out must be bf16 [tokens, K]"); ROWS2D(*out_in, "out"); }
    if (ws_in && !ws_in->is_contiguous()) refuse("workspace must be contiguous");
    c.use(&x); c.use(xs); c.use(w1.q); c.use(w1.scale); c.use(w1.zero); c.use(w2.q); c.use(w2.scale); c.use(w2.zero);
    c.use(&topk); c.use(&weights); c.use(ws_in);
    c.on(a[13]);
    const Tensor out = c.out(out_in, shape, at::kBFloat16);
    const int64_t need[1] = {4 * tokens * k * F};
    const Tensor ws = ws_in ? *ws_in : c.memory(need, at::kByte);
    launch(c, "fg_moe_few", [&] {
      return fg_moe_few(x.data_ptr(), ld(x), act.type, (const float*)ptr(xs), act.group, w1.q->data_ptr(), ptr(w1.scale), ptr(w1.zero),
                        w2.q->data_ptr(), ptr(w2.scale), ptr(w2.zero), group, (const int32_t*)topk.data_ptr(),
                        (const float*)weights.data_ptr(), (int32_t)tokens, (int32_t)k, base, (int32_t)n_local, (int32_t)K, (int32_t)F,
                        ws.data_ptr(), (int64_t)ws.nbytes(), out.data_ptr(), ld(out), c.handle);
    });
    return wrap(out);
  });
}

PyObject* setup(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", setup, METH_O, "The class of refusals: (code, what)."},
    {"add_rmsnorm", (PyCFunction)(void*)add_rmsnorm, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void*)moe_route, METH_FASTCALL, nullptr},
    {"w4_linear", (PyCFunction)(void*)w4_linear, METH_FASTCALL, nullptr},
    {"moe_few", (PyCFunction)(void*)moe_few, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fg_torch() { return PyModule_Create(&module); }
