// The MXFP4 operators and the routing on torch tensors: checks of what the C
// entry points (include/fp8bq.h) cannot see, allocation of the outputs, and
// the call, on the tensors' device and its current stream. A Python extension
// module (_tensors.so) because these calls are short: an operator's kernels
// take a few microseconds for a token, and the same steps in Python took nine
// per call, of which the launch is three. tensors.py documents the functions
// and gives them their keyword arguments.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/fp8bq.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {       // becomes a ValueError
  using std::runtime_error::runtime_error;
};
struct Failed {                             // becomes an Fp8bqError
  const char* fn;
  int status;
};

template <class... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused(s.str());
}

void check(const char* fn, int status) {
  if (status != FP8BQ_OK) throw Failed{fn, status};
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
  return THPVariable_Unpack(o);
}
std::optional<Tensor> maybe(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, name);
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be an integer");
  }
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse("a flag must be a truth value");
  }
  return v;
}

int dtype_code(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kBFloat16: return FP8BQ_BF16;
    case at::kHalf: return FP8BQ_FP16;
    case at::kFloat: return FP8BQ_FP32;
    default: refuse(name, " must be bfloat16, float16 or float32 (got ", t, ")");
  }
}
std::optional<at::ScalarType> dtype_arg(PyObject* o) {
  if (o == Py_None) return std::nullopt;
  if (!THPDtype_Check(o)) refuse("dtype must be a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// All tensors on one GPU, which is made current for the call.
struct On {
  c10::OptionalDeviceGuard guard;
  void* stream;
  at::Device device{at::kCUDA};

  template <class... T>
  explicit On(const Tensor& first, const T&... more) {
    const at::Device d = first.device();
    (same(d, more), ...);
    if (!d.is_cuda()) refuse("tensors must be on the GPU, got ", d);
    guard.reset_device(d);
    stream = c10::hip::getCurrentHIPStream(d.index()).stream();
    device = d;
  }
  static void same(const at::Device& d, const Tensor& t) {
    if (t.device() != d) refuse("tensors on different devices: ", d, " and ", t.device());
  }
  static void same(const at::Device& d, const std::optional<Tensor>& t) {
    if (t) same(d, *t);
  }
  // What at::empty comes to for a GPU tensor, without the dispatcher's half microsecond.
  Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::Tensor(at::detail::empty_cuda(shape, t, device, std::nullopt));
  }
};

const Tensor& matrix(const Tensor& t, const char* name) {
  if (t.dim() != 2 || t.size(0) < 1 || t.size(1) < 1 || (t.stride(1) != 1 && t.size(1) > 1))
    refuse(name, " must be a non-empty 2-D row-major tensor (got ", t.sizes(), ", strides ", t.strides(), ")");
  return t;
}
// Leading dimension; of a single row, whose stride torch leaves open, its length.
int64_t ld(const Tensor& t) {
  const int64_t n = t.size(-1), s = t.stride(-2);
  return t.size(-2) > 1 ? s : (n > s ? n : s);
}

const Tensor& int32(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kInt) refuse(name, " must be int32 (got ", t.scalar_type(), ")");
  return t;
}
const Tensor& int32_shaped(const Tensor& t, const char* name, at::IntArrayRef shape) {
  if (int32(t, name).sizes() != shape || !t.is_contiguous())
    refuse(name, " must be contiguous, of shape ", shape, " (got ", t.sizes(), ", strides ", t.strides(), ")");
  return t;
}
const Tensor& int32_list(const Tensor& t, const char* name, int64_t least) {
  if (int32(t, name).dim() != 1 || t.numel() < least || !t.is_contiguous())
    refuse(name, " must be contiguous, 1-D, with at least ", least, " entries (got ", t.sizes(), ")");
  return t;
}

// MXFP4 codes q [rows, 128 chunks] with scales s [chunks, rows, 8], or with
// `groups` both with that leading dimension, one group's after the other's.
struct Mx {
  int64_t rows, k, ldq, lds;
  void *q, *s;

  Mx(const Tensor& qt, const Tensor& st, const char* name, int64_t groups = 0) {
    const int64_t d = groups ? 1 : 0;
    if (qt.scalar_type() != at::kByte || st.scalar_type() != at::kByte || qt.dim() != d + 2 || st.dim() != d + 3)
      refuse(name, " must be uint8 codes [rows, bytes] and uint8 scales [chunks, rows, 8]", d ? " of every group" : "");
    const int64_t width = qt.size(-1), chunks = width / 128;
    rows = qt.size(-2);
    if (rows < 1 || chunks < 1 || width % 128 || st.size(-3) != chunks || st.size(-2) != rows || st.size(-1) != 8 ||
        (d && (qt.size(0) != groups || st.size(0) != groups)))
      refuse(name, ": codes ", qt.sizes(), " do not go with scales ", st.sizes());
    k = width * 2;
    // torch leaves the stride of a single row open: where every group is one row, the distance between groups counts
    ldq = rows > 1 ? qt.stride(-2) : d && groups > 1 ? qt.stride(0) : width;
    lds = rows;
    if (d && groups > 1 && (qt.stride(0) != rows * ldq || ldq < width))
      refuse(name, ": the groups' codes must follow one another");
    if (!qt.is_contiguous() || !st.is_contiguous()) {
      if (qt.stride(-1) != 1 || st.stride(-1) != 1 || (rows > 1 && st.stride(-2) != 8) ||
          (chunks > 1 && st.stride(-3) % 8))
        refuse(name, ": codes must be row-major and scales [chunks, rows, 8] with rows contiguous");
      if (d && !st.is_contiguous()) refuse(name, ": the groups' scales must follow one another");
      if (chunks > 1) lds = st.stride(-3) / 8;
    }
    q = qt.data_ptr();
    s = st.data_ptr();
  }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const std::optional<Tensor>& t) {
  if (!t) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}
template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
  return r;
}

// ---- the functions (positional arguments; tensors.py gives the keywords) ------

// (x, src or None, rowwise, colwise, nosat)
PyObject* quant(PyObject* const* arg) {
  const Tensor& x = matrix(tensor(arg[0], "x"), "x");
  const int xtype = dtype_code(x.scalar_type(), "x");
  const std::optional<Tensor> src = maybe(arg[1], "src");
  if (src) int32_list(*src, "src", 1);
  const bool rowwise = truth(arg[2]), colwise = truth(arg[3]);
  const int flags = truth(arg[4]) ? FP8BQ_MX_NOSAT : 0;
  if (!rowwise && !colwise) refuse("neither the row form nor the column form is asked for");
  const On on(x, src);
  const int64_t xrows = x.size(0), cols = x.size(1), rows = src ? src->numel() : xrows;
  std::optional<Tensor> q, s, qt, st;
  if (rowwise) {
    const int64_t chunks = (cols + 255) / 256;
    q = on.empty({rows, chunks * 128}, at::kByte);
    s = on.empty({chunks, rows, 8}, at::kByte);
  }
  if (colwise) {
    const int64_t chunks = (rows + 255) / 256;
    qt = on.empty({cols, chunks * 128}, at::kByte);
    st = on.empty({chunks, cols, 8}, at::kByte);
  }
  auto p = [](const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; };
  auto l = [](const std::optional<Tensor>& t) { return t ? t->size(1) : 0; };
  if (src) {
    // Rows that several experts get are read once where that is worth two more launches, which only the sizes tell here.
    // Gathered / by slots, us, top-8 of 8 experts here, of 20 and of 256: 4096 x 1024 9.6 / 13.3, 5.5 / 9.9, 3.4 / 7.9; 4096 x
    // 2048 15.7 / 17.9, 9.2 / 12.1, 4.3 / 8.5; 2048 x 7168 31.4 / 22.5, 17.2 / 16.0, 5.8 / 9.1; 16384 x 1024 35.7 / 27.0,
    // 20.0 / 17.6, 6.4 / 9.4; 16384 x 7168 246 / 163, 131 / 91, 39 / 23.
    std::optional<Tensor> ws;
    if (!colwise && rows >= 2 * xrows && xrows * cols >= (12 << 20))
      ws = on.empty({xrows * (FP8BQ_DISPATCH_WORKSPACE_ROW_BYTES / 4)}, at::kInt);
    check("fp8bq_dispatch_mxfp4_1x32",
          fp8bq_dispatch_mxfp4_1x32(x.data_ptr(), xtype, xrows, cols, ld(x), src->data_ptr<int32_t>(), rows, p(q), l(q),
                                    p(s), rows, p(qt), l(qt), p(st), cols, flags, p(ws), on.stream));
  } else {
    check("fp8bq_quant_mxfp4_1x32",
          fp8bq_quant_mxfp4_1x32(x.data_ptr(), xtype, rows, cols, ld(x), p(q), l(q), p(s), rows, p(qt), l(qt), p(st),
                                 cols, flags, on.stream));
  }
  return tuple(q, s, qt, st);
}

// (q, s, cols, dtype or None)
PyObject* dequant(PyObject* const* arg) {
  const Tensor &q = tensor(arg[0], "q"), &s = tensor(arg[1], "s");
  const Mx m(q, s, "q");
  const int64_t cols = integer(arg[2], "cols");
  const at::ScalarType t = dtype_arg(arg[3]).value_or(at::kBFloat16);
  const int ytype = dtype_code(t, "dtype");
  if (cols < 1 || cols > m.k || cols <= m.k - 256)
    refuse("cols must be in (", m.k - 256, ", ", m.k, "] for codes of ", m.k / 2, " bytes, got ", cols);
  const On on(q, s);
  Tensor y = on.empty({m.rows, cols}, t);
  check("fp8bq_dequant_mxfp4_1x32",
        fp8bq_dequant_mxfp4_1x32(m.q, m.rows, cols, m.ldq, m.s, m.lds, y.data_ptr(), ytype, cols, on.stream));
  return wrap(y);
}

// The output to write to (`out` if given, else a new one of `type`) and its type.
Tensor output(const std::optional<Tensor>& out, at::IntArrayRef shape, std::optional<at::ScalarType> type,
              at::ScalarType usual, const On& on, int& otype) {
  const at::ScalarType t = out ? out->scalar_type() : type.value_or(usual);
  if (out && type && *type != t) refuse("out is ", t, ", dtype says ", *type);
  if (t != at::kBFloat16 && t != at::kFloat) refuse("the output must be bfloat16 or float32, got ", t);
  otype = t == at::kFloat ? FP8BQ_FP32 : FP8BQ_BF16;
  if (!out) return on.empty(shape, t);
  if (out->sizes() != shape || (out->size(-1) > 1 && out->stride(-1) != 1))
    refuse("out must be a row-major ", shape, " tensor (got ", out->sizes(), ", strides ", out->strides(), ")");
  return *out;
}

// (a, sa, b, sb, out or None, dtype or None)
PyObject* gemm(PyObject* const* arg) {
  const Tensor &a = tensor(arg[0], "a"), &sa = tensor(arg[1], "sa"), &b = tensor(arg[2], "b"), &sb = tensor(arg[3], "sb");
  const Mx x(a, sa, "a"), y(b, sb, "b");
  if (x.k != y.k) refuse("a has ", x.k, " elements along the inner dimension, b ", y.k);
  const std::optional<Tensor> given = maybe(arg[4], "out");
  const On on(a, sa, b, sb, given);
  int otype;
  const Tensor out = output(given, {x.rows, y.rows}, dtype_arg(arg[5]), at::kBFloat16, on, otype);
  check("fp8bq_gemm_mxfp4", fp8bq_gemm_mxfp4(x.rows, y.rows, x.k, x.q, x.ldq, x.s, x.lds, y.q, y.ldq, y.s, y.lds,
                                             out.data_ptr(), otype, ld(out), on.stream));
  return wrap(out);
}

// (row_off, a, sa, b, sb, out or None, dtype or None)
PyObject* grouped_gemm(PyObject* const* arg) {
  const Tensor& off = tensor(arg[0], "row_off");
  const Tensor &a = tensor(arg[1], "a"), &sa = tensor(arg[2], "sa"), &b = tensor(arg[3], "b"), &sb = tensor(arg[4], "sb");
  if (b.dim() != 3 || b.size(0) < 1) refuse("b must be codes [groups, n, bytes], got ", b.sizes());
  const int64_t groups = b.size(0);
  const Mx x(a, sa, "a"), y(b, sb, "b", groups);
  if (x.k != y.k) refuse("a has ", x.k, " elements along the inner dimension, b ", y.k);
  int32_shaped(off, "row_off", {groups + 1});
  const std::optional<Tensor> given = maybe(arg[5], "out");
  const On on(a, sa, b, sb, off, given);
  int otype;
  const Tensor out = output(given, {x.rows, y.rows}, dtype_arg(arg[6]), at::kBFloat16, on, otype);
  if (groups > 256) refuse("at most 256 groups, got ", groups);
  check("fp8bq_grouped_gemm_mxfp4",
        fp8bq_grouped_gemm_mxfp4((int32_t)groups, off.data_ptr<int32_t>(), x.rows, y.rows, x.k, x.q, x.ldq, x.s, x.lds,
                                 y.q, y.ldq, y.s, y.lds, out.data_ptr(), otype, ld(out), on.stream));
  return wrap(out);
}

// (row_off, a, sa, b, sb, out or None, dtype or None)
PyObject* grouped_wgrad(PyObject* const* arg) {
  const Tensor& off = int32_list(tensor(arg[0], "row_off"), "row_off", 2);
  const Tensor &a = tensor(arg[1], "a"), &sa = tensor(arg[2], "sa"), &b = tensor(arg[3], "b"), &sb = tensor(arg[4], "sb");
  const Mx x(a, sa, "a"), y(b, sb, "b");
  if (x.k != y.k) refuse("a has ", x.k, " rows, b ", y.k);
  const int64_t groups = off.numel() - 1;
  const std::optional<Tensor> given = maybe(arg[5], "out");
  const On on(a, sa, b, sb, off, given);
  int otype;
  const Tensor out = output(given, {groups, x.rows, y.rows}, dtype_arg(arg[6]), at::kFloat, on, otype);
  if (groups > 256) refuse("at most 256 groups, got ", groups);
  const int64_t ldo = groups > 1 && x.rows == 1 ? out.stride(0) : ld(out);    // a single row's stride is open
  if (groups > 1 && (out.stride(0) != x.rows * ldo || ldo < y.rows))
    refuse("the experts' gradients must follow one another in out");
  check("fp8bq_grouped_wgrad_mxfp4",
        fp8bq_grouped_wgrad_mxfp4((int32_t)groups, off.data_ptr<int32_t>(), x.rows, y.rows, x.k, x.q, x.ldq, x.s, x.lds,
                                  y.q, y.ldq, y.s, y.lds, out.data_ptr(), otype, ldo, on.stream));
  return wrap(out);
}

// (idx, groups, pad)
PyObject* moe_plan(PyObject* const* arg) {
  const Tensor& idx = int32(matrix(tensor(arg[0], "idx"), "idx"), "idx");
  const int64_t groups = integer(arg[1], "groups"), pad = integer(arg[2], "pad");
  if (groups < 1 || groups > 256) refuse("groups must be 1 .. 256, got ", groups);
  if (pad < 1 || pad > 1024) refuse("pad must be 1 .. 1024, got ", pad);
  const int64_t tokens = idx.size(0), topk = idx.size(1);
  const On on(idx);
  const int64_t cap = (tokens * topk + groups * (pad - 1) + pad - 1) / pad * pad;
  Tensor counts = on.empty({groups}, at::kInt), off = on.empty({groups + 1}, at::kInt);
  Tensor src = on.empty({cap}, at::kInt), pos = on.empty({tokens, topk}, at::kInt);
  Tensor ws = on.empty({FP8BQ_MOE_PLAN_WORKSPACE_BYTES / 4}, at::kInt);
  check("fp8bq_moe_plan",
        fp8bq_moe_plan(idx.data_ptr<int32_t>(), tokens, topk, ld(idx), (int32_t)groups, pad, counts.data_ptr<int32_t>(),
                       off.data_ptr<int32_t>(), src.data_ptr<int32_t>(), cap, pos.data_ptr<int32_t>(), ws.data_ptr(),
                       on.stream));
  return tuple(counts, off, src, pos);
}

// What both directions of the balance loss are called with.
struct Routing {
  const Tensor &logits, &idx;
  int ltype, score;
  float coef;
  std::optional<Tensor> seq_off;
  int64_t sequences = 1;

  Routing(PyObject* l, PyObject* i, PyObject* c, PyObject* sc, PyObject* so)
      : logits(matrix(tensor(l, "logits"), "logits")), idx(int32(matrix(tensor(i, "idx"), "idx"), "idx")),
        ltype(dtype_code(logits.scalar_type(), "logits")), seq_off(maybe(so, "seq_off")) {
    if (idx.size(0) != logits.size(0)) refuse("idx has ", idx.size(0), " tokens, logits ", logits.size(0));
    const char* name = PyUnicode_Check(sc) ? PyUnicode_AsUTF8(sc) : nullptr;
    if (!name) PyErr_Clear();
    const std::string s = name ? name : "";
    if (s != "softmax" && s != "sigmoid") refuse("score must be 'softmax' or 'sigmoid', got '", s, "'");
    score = s == "sigmoid" ? FP8BQ_SIGMOID : FP8BQ_SOFTMAX;
    const double v = PyFloat_AsDouble(c);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("coef must be a number");
    }
    coef = (float)v;
    if (seq_off) sequences = int32_list(*seq_off, "seq_off", 2).numel() - 1;
  }
  int64_t tokens() const { return logits.size(0); }
  int64_t experts() const { return logits.size(1); }
  const int32_t* off() const { return seq_off ? seq_off->data_ptr<int32_t>() : nullptr; }
};

// (logits, idx, coef, score, seq_off or None)
PyObject* moe_balance(PyObject* const* arg) {
  const Routing r(arg[0], arg[1], arg[2], arg[3], arg[4]);
  const On on(r.logits, r.idx, r.seq_off);
  int64_t bytes = 0;
  check("fp8bq_moe_balance_workspace_size",
        fp8bq_moe_balance_workspace_size(r.tokens(), r.experts(), r.sequences, &bytes));
  Tensor loss = on.empty({}, at::kFloat), counts = on.empty({r.sequences, r.experts()}, at::kInt);
  Tensor real = on.empty({r.sequences}, at::kInt), ws = on.empty({bytes / 4}, at::kInt);
  check("fp8bq_moe_balance",
        fp8bq_moe_balance(r.logits.data_ptr(), r.ltype, r.tokens(), r.experts(), ld(r.logits), r.idx.data_ptr<int32_t>(),
                          r.idx.size(1), ld(r.idx), r.off(), r.sequences, r.score, r.coef, loss.data_ptr<float>(),
                          counts.data_ptr<int32_t>(), real.data_ptr<int32_t>(), ws.data_ptr(), on.stream));
  return tuple(loss, counts, real);
}

// (dloss, logits, idx, counts, real, coef, score, seq_off or None)
PyObject* moe_balance_grad(PyObject* const* arg) {
  const Tensor& dloss = tensor(arg[0], "dloss");
  const Routing r(arg[1], arg[2], arg[5], arg[6], arg[7]);
  const Tensor& counts = int32_shaped(tensor(arg[3], "counts"), "counts", {r.sequences, r.experts()});
  const Tensor& real = int32_shaped(tensor(arg[4], "real"), "real", {r.sequences});
  if (dloss.scalar_type() != at::kFloat || dloss.numel() != 1) refuse("dloss must be one float32 value");
  const On on(r.logits, r.idx, r.seq_off, counts, real, dloss);
  Tensor grad = on.empty({r.tokens(), r.experts()}, r.logits.scalar_type());
  check("fp8bq_moe_balance_grad",
        fp8bq_moe_balance_grad(dloss.data_ptr<float>(), r.logits.data_ptr(), r.ltype, r.tokens(), r.experts(),
                               ld(r.logits), r.idx.data_ptr<int32_t>(), r.idx.size(1), ld(r.idx), r.off(), r.sequences,
                               r.score, r.coef, counts.data_ptr<int32_t>(), real.data_ptr<int32_t>(), grad.data_ptr(),
                               r.experts(), on.stream));
  return wrap(grad);
}

// ---- the module ----------------------------------------------------------------

// No C++ exception leaves a function: refusals become ValueError, statuses the
// package's Fp8bqError, no memory left torch's OutOfMemoryError, anything else
// RuntimeError.
PyObject* attribute(const char* module, const char* name) {
  PyObject* m = PyImport_ImportModule(module);
  PyObject* a = m ? PyObject_GetAttrString(m, name) : nullptr;
  Py_XDECREF(m);
  return a;
}
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& f) {
    PyObject* cls = attribute("fp8_fine_grained_fp8bq_amd", "Fp8bqError");
    PyObject* err = cls ? PyObject_CallFunction(cls, "sis", f.fn, f.status, fp8bq_last_error()) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* cls = attribute("torch", "OutOfMemoryError");
    if (cls) PyErr_SetString(cls, e.what());
    Py_XDECREF(cls);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<quant, 5>("quant"), method<dequant, 4>("dequant"), method<gemm, 6>("gemm"),
    method<grouped_gemm, 7>("grouped_gemm"), method<grouped_wgrad, 7>("grouped_wgrad"), method<moe_plan, 3>("moe_plan"),
    method<moe_balance, 5>("moe_balance"), method<moe_balance_grad, 8>("moe_balance_grad"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&g_module); }
