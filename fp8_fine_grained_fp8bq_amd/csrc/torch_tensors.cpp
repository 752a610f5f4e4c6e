// The MXFP4 operators, the routing and the operators around a layer's Linears
// on torch tensors: checks of what the C entry points (include/fp8bq.h) cannot
// see, allocation of the outputs, and the call, on the tensors' device and its
// current stream. A Python extension module (_tensors.so) because these calls are short: an operator's kernels
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

// ---- around a layer's Linears --------------------------------------------------

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be a number");
  }
  return v;
}
// A matrix of given shape and type, row-major.
const Tensor& like(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  if (t.scalar_type() != type) refuse(name, " must be ", type, " (got ", t.scalar_type(), ")");
  if (t.sizes() != shape || (shape.size() > 1 && t.size(-1) > 1 && t.stride(-1) != 1) || (shape.size() == 1 && !t.is_contiguous()))
    refuse(name, " must be row-major, of shape ", shape, " (got ", t.sizes(), ", strides ", t.strides(), ")");
  return t;
}
std::optional<Tensor> maybe_like(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) {
  std::optional<Tensor> t = maybe(o, name);
  if (t) like(*t, name, shape, type);
  return t;
}
void* pointer(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }
int64_t ld(const std::optional<Tensor>& t) { return t ? ld(*t) : 0; }

const Tensor& norm_weight(PyObject* o, int64_t cols, int& wtype) {
  const Tensor& w = tensor(o, "weight");
  wtype = dtype_code(w.scalar_type(), "weight");
  return like(w, "weight", {cols}, w.scalar_type());
}

// (x, weight, eps, residual or None, quant, norm, pow2)
PyObject* rmsnorm(PyObject* const* arg) {
  const Tensor& x = matrix(tensor(arg[0], "x"), "x");
  const at::ScalarType type = x.scalar_type();
  const int xtype = dtype_code(type, "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  int wtype;
  const Tensor& w = norm_weight(arg[1], cols, wtype);
  const float eps = (float)number(arg[2], "eps");
  const std::optional<Tensor> r = maybe_like(arg[3], "residual", {rows, cols}, type);
  const bool quant = truth(arg[4]), norm = truth(arg[5]);
  const int flags = truth(arg[6]) ? FP8BQ_SCALE_POW2 : 0;
  if (!quant && !norm) refuse("neither the codes nor the normalised rows are asked for");
  if (quant && cols % 128) refuse("cols must be a multiple of 128 for the codes, got ", cols);
  const On on(x, w, r);
  std::optional<Tensor> q, s, y, h;
  if (quant) {
    q = on.empty({rows, cols}, at::kByte);
    s = on.empty({cols / 128, rows}, at::kFloat);
  }
  if (norm) y = on.empty({rows, cols}, type);
  if (r) h = on.empty({rows, cols}, type);
  Tensor rstd = on.empty({rows}, at::kFloat);
  check("fp8bq_rmsnorm",
        fp8bq_rmsnorm(x.data_ptr(), xtype, rows, cols, ld(x), pointer(r), ld(r), w.data_ptr(), wtype, eps, pointer(h), cols,
                      pointer(y), cols, pointer(q), cols, static_cast<float*>(pointer(s)), rows, rstd.data_ptr<float>(), flags,
                      on.stream));
  return tuple(q, s, y, h, rstd);
}

// (dy, h, weight, rstd, dh or None)
PyObject* rmsnorm_grad(PyObject* const* arg) {
  const Tensor& h = matrix(tensor(arg[1], "h"), "h");
  const at::ScalarType type = h.scalar_type();
  const int xtype = dtype_code(type, "h");
  const int64_t rows = h.size(0), cols = h.size(1);
  const Tensor& dy = like(tensor(arg[0], "dy"), "dy", {rows, cols}, type);
  int wtype;
  const Tensor& w = norm_weight(arg[2], cols, wtype);
  const Tensor& rstd = like(tensor(arg[3], "rstd"), "rstd", {rows}, at::kFloat);
  const std::optional<Tensor> dh = maybe_like(arg[4], "dh", {rows, cols}, type);
  const On on(h, dy, w, rstd, dh);
  int64_t bytes = 0;
  check("fp8bq_rmsnorm_grad_workspace_size", fp8bq_rmsnorm_grad_workspace_size(rows, cols, &bytes));
  Tensor dx = on.empty({rows, cols}, type), dw = on.empty({cols}, at::kFloat), ws = on.empty({bytes / 4}, at::kFloat);
  check("fp8bq_rmsnorm_grad",
        fp8bq_rmsnorm_grad(dy.data_ptr(), xtype, rows, cols, ld(dy), h.data_ptr(), ld(h), w.data_ptr(), wtype,
                           rstd.data_ptr<float>(), pointer(dh), ld(dh), dx.data_ptr(), cols, dw.data_ptr<float>(),
                           ws.data_ptr(), on.stream));
  return tuple(dx, dw);
}

// The choices' rows of one plan.
const Tensor& choices(PyObject* o) {
  const Tensor& pos = int32(matrix(tensor(o, "pos"), "pos"), "pos");
  if (!pos.is_contiguous()) refuse("pos must be contiguous (got strides ", pos.strides(), ")");
  return pos;
}

// (x, src, pos, s or None, out or None, s_out or None)
PyObject* moe_dispatch(PyObject* const* arg) {
  const Tensor& x = matrix(tensor(arg[0], "x"), "x");
  const at::ScalarType type = x.scalar_type();
  if (type != at::kByte) dtype_code(type, "x that does not hold 8-bit codes (uint8)");
  const Tensor& src = int32_list(tensor(arg[1], "src"), "src", 1);
  const Tensor& pos = choices(arg[2]);
  const int64_t tokens = x.size(0), cols = x.size(1), rows = src.numel();
  if (pos.size(0) != tokens) refuse("pos has ", pos.size(0), " tokens, x ", tokens);
  std::optional<Tensor> s = maybe(arg[3], "s"), out = maybe_like(arg[4], "out", {rows, cols}, type), so;
  if (s) {
    if (type != at::kByte || cols % 128) refuse("scales go with uint8 codes of a multiple of 128 columns (got ", type, ", ", cols, " columns)");
    like(*s, "s", {cols / 128, tokens}, at::kFloat);
    so = maybe_like(arg[5], "s_out", {cols / 128, rows}, at::kFloat);
  } else if (arg[5] != Py_None) {
    refuse("s_out without s");
  }
  const On on(x, src, pos, s, out, so);
  if (!out) out = on.empty({rows, cols}, type);
  if (s && !so) so = on.empty({cols / 128, rows}, at::kFloat);
  check("fp8bq_moe_dispatch",
        fp8bq_moe_dispatch(x.data_ptr(), (int)x.element_size(), tokens, cols, ld(x), static_cast<const float*>(pointer(s)), ld(s),
                           pos.data_ptr<int32_t>(), pos.size(1), src.data_ptr<int32_t>(), rows, out->data_ptr(), ld(out),
                           static_cast<float*>(pointer(so)), ld(so), on.stream));
  return tuple(out, so);
}

// The experts' rows, which may be none.
const Tensor& rows_of_experts(PyObject* o) {
  const Tensor& y = tensor(o, "y");
  if (y.dim() == 2 && y.size(0) == 0 && y.size(1) > 0) return y;
  return matrix(y, "y");
}

// (y, pos, weight or None, base or None, out or None)
PyObject* moe_combine(PyObject* const* arg) {
  const Tensor& y = rows_of_experts(arg[0]);
  const at::ScalarType type = y.scalar_type();
  const int code = dtype_code(type, "y");
  const Tensor& pos = choices(arg[1]);
  const int64_t tokens = pos.size(0), topk = pos.size(1), rows = y.size(0), cols = y.size(1);
  const std::optional<Tensor> w = maybe_like(arg[2], "weight", {tokens, topk}, at::kFloat);
  const std::optional<Tensor> base = maybe_like(arg[3], "base", {tokens, cols}, type);
  std::optional<Tensor> out = maybe_like(arg[4], "out", {tokens, cols}, type);
  const On on(y, pos, w, base, out);
  if (!out) out = on.empty({tokens, cols}, type);
  check("fp8bq_moe_combine",
        fp8bq_moe_combine(rows ? y.data_ptr() : nullptr, code, rows, cols, ld(y), pos.data_ptr<int32_t>(), tokens, topk,
                          static_cast<const float*>(pointer(w)), ld(w), pointer(base), ld(base), out->data_ptr(), ld(out),
                          on.stream));
  return wrap(out);
}

// (dout, y, pos, weight, src, out or None)
PyObject* moe_combine_grad(PyObject* const* arg) {
  const Tensor& y = rows_of_experts(arg[1]);
  const at::ScalarType type = y.scalar_type();
  const int code = dtype_code(type, "y");
  const Tensor& pos = choices(arg[2]);
  const int64_t tokens = pos.size(0), topk = pos.size(1), rows = y.size(0), cols = y.size(1);
  const Tensor& dout = like(tensor(arg[0], "dout"), "dout", {tokens, cols}, type);
  const Tensor& w = like(tensor(arg[3], "weight"), "weight", {tokens, topk}, at::kFloat);
  const Tensor& src = int32_shaped(tensor(arg[4], "src"), "src", {rows});
  std::optional<Tensor> dy = maybe_like(arg[5], "out", {rows, cols}, type);
  const On on(y, dout, pos, w, src, dy);
  if (!dy) dy = on.empty({rows, cols}, type);
  Tensor dw = on.empty({tokens, topk}, at::kFloat);
  check("fp8bq_moe_combine_grad",
        fp8bq_moe_combine_grad(dout.data_ptr(), code, tokens, cols, ld(dout), rows ? y.data_ptr() : nullptr, rows, ld(y), pos.data_ptr<int32_t>(),
                               topk, w.data_ptr<float>(), ld(w), src.data_ptr<int32_t>(), dy->data_ptr(), ld(dy),
                               dw.data_ptr<float>(), on.stream));
  return tuple(dy, dw);
}

// x [rows, k] against codes of k elements, padded to a multiple of 256.
int64_t inner(const Tensor& x, const Mx& w) {
  const int64_t k = x.size(1);
  if (k > w.k || k <= w.k - 256) refuse("x has ", k, " columns, the codes of w stand for ", w.k - 255, " to ", w.k);
  return k;
}
// The type of a product's output, and `out` checked against it.
at::ScalarType gemv_type(const std::optional<Tensor>& out, int64_t rows, int64_t n, std::optional<at::ScalarType> dtype,
                         at::ScalarType usual, int& otype) {
  const at::ScalarType t = out ? out->scalar_type() : dtype.value_or(usual);
  if (out && dtype && *dtype != t) refuse("out is ", t, ", dtype says ", *dtype);
  otype = dtype_code(t, "the output");
  if (out) like(*out, "out", {rows, n}, t);
  return t;
}

// (x, w, ws, out or None, dtype or None)
PyObject* gemv(PyObject* const* arg) {
  const Tensor& x = matrix(tensor(arg[0], "x"), "x");
  const Tensor &w = tensor(arg[1], "w"), &ws = tensor(arg[2], "ws");
  const int xtype = dtype_code(x.scalar_type(), "x");
  const Mx b(w, ws, "w");
  const int64_t m = x.size(0), k = inner(x, b);
  const std::optional<Tensor> given = maybe(arg[3], "out");
  int otype;
  const at::ScalarType t = gemv_type(given, m, b.rows, dtype_arg(arg[4]), x.scalar_type(), otype);
  const On on(x, w, ws, given);
  const Tensor out = given ? *given : on.empty({m, b.rows}, t);
  check("fp8bq_gemv_mxfp4", fp8bq_gemv_mxfp4(m, b.rows, k, x.data_ptr(), xtype, ld(x), b.q, b.ldq, b.s, b.lds, out.data_ptr(),
                                             otype, ld(out), on.stream));
  return wrap(out);
}

// (row_off, x, w, ws, src or None, out or None, dtype or None)
PyObject* grouped_gemv(PyObject* const* arg) {
  const Tensor& off = tensor(arg[0], "row_off");
  const Tensor& x = matrix(tensor(arg[1], "x"), "x");
  const Tensor &w = tensor(arg[2], "w"), &ws = tensor(arg[3], "ws");
  const int xtype = dtype_code(x.scalar_type(), "x");
  if (w.dim() != 3 || w.size(0) < 1) refuse("w must be codes [groups, n, bytes], got ", w.sizes());
  const int64_t groups = w.size(0);
  const Mx b(w, ws, "w", groups);
  const int64_t k = inner(x, b);
  int32_shaped(off, "row_off", {groups + 1});
  const std::optional<Tensor> src = maybe(arg[4], "src"), given = maybe(arg[5], "out");
  if (src) int32_list(*src, "src", 1);
  const int64_t rows = src ? src->numel() : x.size(0);
  if (groups > 256) refuse("at most 256 groups, got ", groups);
  int otype;
  const at::ScalarType t = gemv_type(given, rows, b.rows, dtype_arg(arg[6]), x.scalar_type(), otype);
  const On on(x, w, ws, off, src, given);
  const Tensor out = given ? *given : on.empty({rows, b.rows}, t);
  check("fp8bq_grouped_gemv_mxfp4",
        fp8bq_grouped_gemv_mxfp4((int32_t)groups, off.data_ptr<int32_t>(), rows, b.rows, k, x.data_ptr(), xtype, x.size(0), ld(x),
                                 static_cast<const int32_t*>(pointer(src)), b.q, b.ldq, b.s, b.lds, out.data_ptr(), otype, ld(out),
                                 on.stream));
  return wrap(out);
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
    method<moe_balance, 5>("moe_balance"), method<moe_balance_grad, 8>("moe_balance_grad"),
    method<rmsnorm, 7>("rmsnorm"), method<rmsnorm_grad, 5>("rmsnorm_grad"), method<moe_dispatch, 6>("moe_dispatch"),
    method<moe_combine, 5>("moe_combine"), method<moe_combine_grad, 6>("moe_combine_grad"), method<gemv, 5>("gemv"),
    method<grouped_gemv, 7>("grouped_gemv"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&g_module); }
