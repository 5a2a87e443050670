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

#include <cmath>

#include "fg_attention.h"

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
  const Tensor* used[20];
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
  // A tensor of the caller's that the launch writes into; all are checked before the first is marked.
  void check_write(const Tensor* t) const {
    if (!t) return;
    if (t->device() != device) refuse("tensors are on different devices");
    no_gradient(*t);
  }
  void write(const Tensor* t) {
    if (!t) return;
    use(t);
    if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  }
  // The output `given`, which has been checked, or a new one. Autograd, which may have
  // saved a given one, is told that it is written.
  Tensor out(const Tensor* given, at::IntArrayRef shape, ScalarType type) {
    if (given) {
      write(given);
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

// ------------------------------------------------------------ paged caches
// lens, add, table, ring, ends, page, tokens, lens_out, ends_out, starts, slots, positions, stream
//   -> (lens_out, ends_out, starts, slots, positions)
PyObject* page_step(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &lens = tensor(a[0]), &add = tensor(a[1]), &table = tensor(a[2]), &ring = tensor(a[3]), &ends = tensor(a[4]);
    const Tensor *lens_in = maybe(a[7]), *ends_in = maybe(a[8]), *starts_in = maybe(a[9]), *slots_in = maybe(a[10]), *pos_in = maybe(a[11]);
    const int32_t page = int32_of(a[5], "page must be an int32"), tokens = int32_of(a[6], "tokens must be an int32");
    if (page < 1 || tokens < 0) refuse("page must be positive, tokens not negative");
    ROWS2D(table, "table");
    const int64_t batch = table.size(0), width = table.size(1);
    if (!is_type(lens, at::kInt) || !vector_of(lens, batch) || !is_type(add, at::kInt) || !vector_of(add, batch) || !is_type(table, at::kInt))
      refuse("lens and add must be int32 [batch], table int32 [batch, pages]");
    if (!is_type(ring, at::kInt) || ring.dim() != 1 || !ring.is_contiguous() || ring.size(0) < 1) refuse("ring must be contiguous int32 [n_pages]");
    if (!is_type(ends, at::kLong) || !vector_of(ends, 2)) refuse("ends must be int64 [2]");
    fits_int32(batch, "too many requests");
    fits_int32(width, "the table is too wide");
    fits_int32(ring.size(0), "too many pages");
    Call c(table);
    const int64_t nb[1] = {batch}, two[1] = {2}, ns[1] = {batch + 1}, nt[1] = {tokens};
    c.check(lens_in, nb, at::kInt, "lens_out must be int32 [batch]");
    c.check(ends_in, two, at::kLong, "ends_out must be int64 [2]");
    c.check(starts_in, ns, at::kInt, "starts must be int32 [batch + 1]");
    c.check(slots_in, nt, at::kLong, "slots must be int64 [tokens]");
    c.check(pos_in, nt, at::kInt, "positions must be int32 [tokens]");
    for (const Tensor* t : {lens_in, ends_in, starts_in, slots_in, pos_in})
      if (t && !t->is_contiguous()) refuse("given outputs must be contiguous");
    c.check_write(&table); c.check_write(&ring);
    c.use(&lens); c.use(&add); c.use(&ends);
    c.on(a[12]);
    c.write(&table);
    c.write(&ring);
    const Tensor lo = c.out(lens_in, nb, at::kInt), eo = c.out(ends_in, two, at::kLong), st = c.out(starts_in, ns, at::kInt);
    const Tensor sl = c.out(slots_in, nt, at::kLong), po = c.out(pos_in, nt, at::kInt);
    launch(c, "fg_page_step", [&] {
      return fg_page_step((const int32_t*)lens.data_ptr(), (const int32_t*)add.data_ptr(), (int32_t)batch, (int32_t*)table.data_ptr(),
                          batch > 1 ? table.stride(0) : width, (int32_t)width, (int32_t*)ring.data_ptr(), (const int64_t*)ends.data_ptr(),
                          (int32_t)ring.size(0), page, (int32_t*)lo.data_ptr(), (int64_t*)eo.data_ptr(), (int32_t*)st.data_ptr(),
                          (int64_t*)sl.data_ptr(), (int32_t*)po.data_ptr(), tokens, c.handle);
    });
    return tuple({wrap(lo), wrap(eo), wrap(st), wrap(sl), wrap(po)});
  });
}

// Strides of a dimension of size 1 do not matter: as if it were dense.
int64_t stride_of(const Tensor& t, int64_t dim, int64_t dense) { return t.size(dim) > 1 ? t.stride(dim) : dense; }
bool columns_consecutive(const Tensor& t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }
int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// k, k_cache, slots, v, v_cache, k_scale, v_scale, stream -> None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &k = tensor(a[0]), &kc = tensor(a[1]), &slots = tensor(a[2]);
    const Tensor *v = maybe(a[3]), *vc = maybe(a[4]), *ks = maybe(a[5]), *vs = maybe(a[6]);
    if (!v != !vc) refuse("v and v_cache come together");
    const bool heads_there = k.dim() == 3;
    if ((k.dim() != 2 && k.dim() != 3) || kc.dim() != k.dim() + 1) refuse("rows must be [n, heads, dim] with a cache [n_pages, page, heads, dim], or [n, dim] with [n_pages, page, dim]");
    const bool e4m3 = is_type(kc, at::kFloat8_e4m3fn);
    if (!e4m3 && !is_type(kc, at::kBFloat16)) refuse("caches must be bf16 or float8_e4m3fn");
    const int64_t n = k.size(0), heads = heads_there ? k.size(1) : 1, dim = k.size(-1), pages = kc.size(0), page = kc.size(1);
    if (!is_type(slots, at::kLong) || !vector_of(slots, n)) refuse("slots must be int64 [n]");
    if (heads < 1 || dim < 1 || pages < 1 || page < 1) refuse("rows and caches must not be empty");
    fits_int32(heads, "too many heads");
    fits_int32(dim, "rows are too long");
    fits_int32(pages, "too many pages");
    fits_int32(page, "pages are too long");
    Call c(k);
    fg_append_t part[2];
    const Tensor* xs[2] = {&k, v};
    const Tensor* cs[2] = {&kc, vc};
    const Tensor* ss[2] = {ks, vs};
    if (!v && vs) refuse("v_scale needs v");
    for (int i = 0; i < (v ? 2 : 1); ++i) {
      const Tensor &x = *xs[i], &cache = *cs[i];
      if (!is_type(x, at::kBFloat16) || x.sizes() != k.sizes() || !columns_consecutive(x)) refuse("new rows must be bf16 with consecutive columns, v like k");
      if (cache.scalar_type() != kc.scalar_type() || cache.dim() != kc.dim() || cache.size(0) != pages || cache.size(1) != page ||
          cache.size(-1) != dim || (heads_there && cache.size(2) != heads) || !columns_consecutive(cache))
        refuse("caches must have consecutive columns, the rows' heads and columns, and be alike");
      if (e4m3 != (ss[i] != nullptr)) refuse("float8_e4m3fn caches need scales, bf16 caches take none");
      const int64_t sshape[3] = {pages, heads, page};
      if (ss[i]) {
        c.check(ss[i], sshape, at::kFloat, "scales must be float32 [n_pages, heads, page]");
        if (!ss[i]->is_contiguous()) refuse("scales must be contiguous");
      }
      const int64_t width = up8(dim);
      part[i].x = x.data_ptr();
      part[i].x_head = heads_there ? stride_of(x, 1, width) : width;
      part[i].x_row = stride_of(x, 0, width * heads);
      part[i].cache = cache.data_ptr();
      part[i].head_stride = heads_there ? stride_of(cache, 2, width) : width;
      part[i].row_stride = stride_of(cache, 1, width * heads);
      part[i].page_stride = stride_of(cache, 0, width * heads * page);
      part[i].scale = (float*)ptr(ss[i]);
    }
    c.check_write(&kc); c.check_write(vc); c.check_write(ks); c.check_write(vs);
    c.use(&k); c.use(v); c.use(&slots);
    c.on(a[7]);
    c.write(&kc); c.write(vc); c.write(ks); c.write(vs);
    launch(c, "fg_kv_append", [&] {
      return fg_kv_append(&part[0], v ? &part[1] : nullptr, e4m3 ? FG_E4M3 : FG_BF16, (const int64_t*)slots.data_ptr(), n, (int32_t)heads,
                          (int32_t)dim, (int32_t)pages, (int32_t)page, c.handle);
    });
    return none();
  });
}

// Tables and lengths of the requests in a cache of `pages` pages.
fg_pages_t requests(Call& c, const Tensor& table, const Tensor& lens, int64_t batch, int64_t pages, int64_t page) {
  ROWS2D(table, "table");
  if (!is_type(table, at::kInt) || table.size(0) != batch || table.size(1) < 1 || !is_type(lens, at::kInt) || !vector_of(lens, batch))
    refuse("table must be int32 [batch, pages], lens int32 [batch]");
  if (page < 16 || page % 16) refuse("pages must have a multiple of 16 rows");
  if (pages < 1) refuse("the cache must have pages");
  fits_int32(batch, "too many requests");
  fits_int32(table.size(1), "the table is too wide");
  fits_int32(pages, "too many pages");
  fits_int32(page, "pages are too long");
  c.use(&table);
  c.use(&lens);
  return {(const int32_t*)table.data_ptr(), batch > 1 ? table.stride(0) : table.size(1), (int32_t)table.size(1), (const int32_t*)lens.data_ptr(),
          (int32_t)batch, (int32_t)pages, (int32_t)page};
}

// The scale of the scores; None: one over the root of n.
float score_scale(PyObject* o, int64_t n) {
  const float s = o == Py_None ? (float)(1.0 / std::sqrt((double)n)) : (float)number(o);
  if (!(s > 0.0f) || !(s < INFINITY)) refuse("scale must be positive and finite");
  return s;
}

// Output [n][heads][dim], and lse [n][heads] if it is asked for (True) or given.
struct AttentionOut {
  Tensor out, lse;
  bool has_lse = false;
  const Tensor *out_in, *lse_in = nullptr;
  int64_t shape[3];
  AttentionOut(const Call& c, PyObject* o, PyObject* l, int64_t n, int64_t heads, int64_t dim) : out_in(maybe(o)), shape{n, heads, dim} {
    c.check(out_in, shape, at::kBFloat16, "out must be bf16 [rows, heads, dim]");
    if (out_in && !columns_consecutive(*out_in)) refuse("out must have consecutive columns");
    if (PyBool_Check(l) || l == Py_None) {
      has_lse = l == Py_True;
    } else {
      lse_in = &tensor(l);
      has_lse = true;
      c.check(lse_in, at::IntArrayRef(shape, 2), at::kFloat, "lse must be float32 [rows, heads]");
      if (!lse_in->is_contiguous()) refuse("lse must be contiguous");
    }
  }
  void make(Call& c) {
    out = c.out(out_in, shape, at::kBFloat16);
    if (has_lse) lse = c.out(lse_in, at::IntArrayRef(shape, 2), at::kFloat);
  }
  int64_t row() const { return stride_of(out, 0, shape[1] * shape[2]); }
  int64_t head() const { return stride_of(out, 1, shape[2]); }
  float* lse_ptr() const { return has_lse ? (float*)lse.data_ptr() : nullptr; }
  PyObject* result() const { return has_lse ? tuple({wrap(out), wrap(lse)}) : wrap(out); }
};

Tensor workspace_of(const Call& c, const Tensor* given, int64_t bytes) {
  const int64_t shape[1] = {bytes};
  return given ? *given : c.memory(shape, at::kByte);
}

void check_queries(const Tensor& q) {
  if (!is_type(q, at::kBFloat16) || q.dim() != 3 || !columns_consecutive(q)) refuse("q must be bf16 [rows, heads, dim] with consecutive columns");
  if (q.size(1) < 1 || q.size(1) > FG_ATTN_MAX_HEADS) refuse("1 to 65535 heads");
}

// q, k_cache, v_cache, table, lens, scale, window, k_scale, v_scale, out, lse, workspace, stream -> out or (out, lse)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &table = tensor(a[3]), &lens = tensor(a[4]);
    const Tensor *ks = maybe(a[7]), *vs = maybe(a[8]), *ws_in = maybe(a[11]);
    check_queries(q);
    const bool e4m3 = is_type(k, at::kFloat8_e4m3fn);
    if ((!e4m3 && !is_type(k, at::kBFloat16)) || k.scalar_type() != v.scalar_type() || k.dim() != 4 || v.sizes() != k.sizes() ||
        !columns_consecutive(k) || !columns_consecutive(v))
      refuse("caches must be bf16 or float8_e4m3fn [n_pages, page, heads, dim] with consecutive columns");
    const int64_t batch = q.size(0), heads = q.size(1), dim = q.size(2), kv = k.size(2);
    if (k.size(3) != dim || (dim != 64 && dim != 128 && dim != 256)) refuse("queries and caches must have 64, 128 or 256 columns");
    if (kv < 1 || heads % kv) refuse("the queries' heads must be a multiple of the cache's");
    if (batch > FG_ATTN_MAX_BATCH) refuse("up to 65535 requests");
    const float scale = score_scale(a[5], dim);
    const int32_t window = int32_of(a[6], "window must be an int32");
    if (window < 0) refuse("window must not be negative");
    if (e4m3 != (ks != nullptr) || e4m3 != (vs != nullptr)) refuse("float8_e4m3fn caches need k_scale and v_scale, bf16 caches take none");
    Call c(q);
    const int64_t sshape[3] = {k.size(0), kv, k.size(1)};
    c.check(ks, sshape, at::kFloat, "scales must be float32 [n_pages, heads, page]");
    c.check(vs, sshape, at::kFloat, "scales must be float32 [n_pages, heads, page]");
    if ((ks && !ks->is_contiguous()) || (vs && !vs->is_contiguous())) refuse("scales must be contiguous");
    AttentionOut o(c, a[9], a[10], batch, heads, dim);
    if (ws_in && !ws_in->is_contiguous()) refuse("workspace must be contiguous");
    const fg_pages_t pages = requests(c, table, lens, batch, k.size(0), k.size(1));
    c.use(&q); c.use(&k); c.use(&v); c.use(ks); c.use(vs); c.use(ws_in);
    c.on(a[12]);
    o.make(c);
    int64_t need = 0;
    if (fg_paged_attention_bytes((int32_t)batch, (int32_t)kv, (int32_t)(heads / kv), (int32_t)dim, &need) != FG_OK) refuse("too large");
    const Tensor ws = workspace_of(c, ws_in, need);
    const fg_cache_t kp{k.data_ptr(), stride_of(k, 0, k.size(1) * kv * dim), stride_of(k, 1, kv * dim), stride_of(k, 2, dim), (const float*)ptr(ks)};
    const fg_cache_t vp{v.data_ptr(), stride_of(v, 0, v.size(1) * kv * dim), stride_of(v, 1, kv * dim), stride_of(v, 2, dim), (const float*)ptr(vs)};
    launch(c, "fg_paged_attention", [&] {
      return fg_paged_attention(q.data_ptr(), stride_of(q, 0, heads * dim), stride_of(q, 1, dim), &kp, &vp, e4m3 ? FG_E4M3 : FG_BF16, &pages,
                                (int32_t)kv, (int32_t)(heads / kv), (int32_t)dim, window, scale, ws.data_ptr(), (int64_t)ws.nbytes(),
                                o.out.data_ptr(), o.row(), o.head(), o.lse_ptr(), heads, c.handle);
    });
    return o.result();
  });
}

// Sizes of latent attention, from the queries, the weights and the rows' columns.
struct LatentSizes {
  int64_t rows, heads, rank, rope, nope;
  LatentSizes(const Tensor& q, const Tensor& w, int64_t columns, int64_t nope_) : rows(q.size(0)), heads(q.size(1)), nope(nope_) {
    if (!is_type(w, at::kBFloat16) || w.dim() != 3 || !w.is_contiguous() || w.size(0) != heads || w.size(1) != 2 * nope)
      refuse("w must be contiguous bf16 [heads, 2 nope, rank]");
    rank = w.size(2);
    rope = columns - rank;
    if ((rank != 256 && rank != 512) || (rope != 32 && rope != 64) || (nope != 64 && nope != 128)) refuse("rank 256 or 512, rope 32 or 64, nope 64 or 128");
    if (q.size(2) != nope + rope) refuse("q must have nope + rope columns, the latent rows rank + rope");
  }
};

// q, w, cache, table, lens, nope, scale, out, lse, workspace, stream -> out or (out, lse)
PyObject* latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &q = tensor(a[0]), &w = tensor(a[1]), &cache = tensor(a[2]), &table = tensor(a[3]), &lens = tensor(a[4]);
    const Tensor* ws_in = maybe(a[9]);
    check_queries(q);
    if (!is_type(cache, at::kBFloat16) || cache.dim() != 3 || !columns_consecutive(cache)) refuse("cache must be bf16 [n_pages, page, rank + rope] with consecutive columns");
    const LatentSizes z(q, w, cache.size(2), int32_of(a[5], "nope must be an int32"));
    if (z.rows > FG_ATTN_MAX_BATCH) refuse("up to 65535 requests");
    const float scale = score_scale(a[6], z.nope + z.rope);
    Call c(q);
    AttentionOut o(c, a[7], a[8], z.rows, z.heads, z.nope);
    if (ws_in && !ws_in->is_contiguous()) refuse("workspace must be contiguous");
    const fg_pages_t pages = requests(c, table, lens, z.rows, cache.size(0), cache.size(1));
    c.use(&q); c.use(&w); c.use(&cache); c.use(ws_in);
    c.on(a[10]);
    o.make(c);
    int64_t need = 0;
    if (fg_latent_attention_bytes((int32_t)z.rows, (int32_t)z.heads, (int32_t)z.rank, &need) != FG_OK) refuse("too large");
    const Tensor ws = workspace_of(c, ws_in, need);
    launch(c, "fg_latent_attention", [&] {
      return fg_latent_attention(q.data_ptr(), stride_of(q, 0, z.heads * q.size(2)), stride_of(q, 1, q.size(2)), w.data_ptr(), cache.data_ptr(),
                                 stride_of(cache, 0, cache.size(1) * cache.size(2)), stride_of(cache, 1, cache.size(2)), &pages, (int32_t)z.heads,
                                 (int32_t)z.rank, (int32_t)z.rope, (int32_t)z.nope, scale, ws.data_ptr(), (int64_t)ws.nbytes(), o.out.data_ptr(), o.row(),
                                 o.head(), o.lse_ptr(), z.heads, c.handle);
    });
    return o.result();
  });
}

// q, latent, w, q_starts, k_starts, nope, scale, out, lse, workspace, stream -> out or (out, lse)
PyObject* latent_prompt(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!counted(n_args, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor &q = tensor(a[0]), &lat = tensor(a[1]), &w = tensor(a[2]), &qs = tensor(a[3]), &ks = tensor(a[4]);
    const Tensor* ws_in = maybe(a[9]);
    check_queries(q);
    ROWS2D(lat, "latent");
    if (!is_type(lat, at::kBFloat16)) refuse("latent must be bf16 [rows, rank + rope]");
    const LatentSizes z(q, w, lat.size(1), int32_of(a[5], "nope must be an int32"));
    const float scale = score_scale(a[6], z.nope + z.rope);
    if (!is_type(qs, at::kInt) || qs.dim() != 1 || qs.size(0) < 1 || !vector_of(qs, qs.size(0)) || !is_type(ks, at::kInt) || !vector_of(ks, qs.size(0)))
      refuse("q_starts and k_starts must be int32 [batch + 1]");
    const int64_t batch = qs.size(0) - 1;
    if (batch > FG_ATTN_MAX_BATCH) refuse("up to 65535 requests");
    Call c(q);
    AttentionOut o(c, a[7], a[8], z.rows, z.heads, z.nope);
    if (ws_in && !ws_in->is_contiguous()) refuse("workspace must be contiguous");
    c.use(&q); c.use(&lat); c.use(&w); c.use(&qs); c.use(&ks); c.use(ws_in);
    c.on(a[10]);
    int64_t need = 0;
    if (fg_latent_prompt_bytes(lat.size(0), (int32_t)z.heads, (int32_t)z.nope, &need) != FG_OK) refuse("too large");
    o.make(c);
    const Tensor ws = workspace_of(c, ws_in, need);
    launch(c, "fg_latent_prompt", [&] {
      return fg_latent_prompt(q.data_ptr(), stride_of(q, 0, z.heads * q.size(2)), stride_of(q, 1, q.size(2)), (const int32_t*)qs.data_ptr(), z.rows,
                              lat.data_ptr(), ld(lat), (const int32_t*)ks.data_ptr(), lat.size(0), (int32_t)batch, w.data_ptr(), (int32_t)z.heads,
                              (int32_t)z.rank, (int32_t)z.rope, (int32_t)z.nope, scale, ws.data_ptr(), (int64_t)ws.nbytes(), o.out.data_ptr(), o.row(),
                              o.head(), o.lse_ptr(), z.heads, c.handle);
    });
    return o.result();
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
    {"page_step", (PyCFunction)(void*)page_step, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void*)kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void*)paged_attention, METH_FASTCALL, nullptr},
    {"latent_attention", (PyCFunction)(void*)latent_attention, METH_FASTCALL, nullptr},
    {"latent_prompt", (PyCFunction)(void*)latent_prompt, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "fg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fg_torch() { return PyModule_Create(&module); }
