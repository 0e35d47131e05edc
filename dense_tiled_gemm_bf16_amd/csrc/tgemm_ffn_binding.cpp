// The compiled part of the Python binding of libtgemm_ffn.so (module
// _ffn_binding): checks of types, devices, shapes and strides, allocation of
// outputs and workspaces, and the call of the C entry point on the tensors'
// device and its current stream.  It is compiled because at a few tokens the
// checks cost more than the kernels: gemm_epilogue of one token took 8.0 us of
// host time when they were Python (3.5 us of them the launch).
//
// ffn.py documents each function; the arguments here are positional, in the
// order of its signatures without the stream (ffn.py makes that current).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/tgemm_ffn.h"

namespace {

PyObject *g_error = nullptr;  // TgemmError

struct Raise {
  PyObject *type;
  std::string what;
};
[[noreturn]] void type_error(std::string s) { throw Raise{PyExc_TypeError, std::move(s)}; }
[[noreturn]] void value_error(std::string s) { throw Raise{PyExc_ValueError, std::move(s)}; }
struct Failed {
  int code;
};

using at::ScalarType;
using at::Tensor;

std::string shape_str(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
std::string name_of(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    default: return std::string("torch.") + c10::toString(t);
  }
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

bool truth(PyObject *o, const char *name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {  // (an array of several values, say)
    PyErr_Clear();
    type_error(std::string(name) + " must be true or false");
  }
  return v == 1;
}

int dtype16(const Tensor &t, const char *name) {
  if (t.scalar_type() == ScalarType::BFloat16) return TGEMM_DT_BF16;
  if (t.scalar_type() == ScalarType::Half) return TGEMM_DT_F16;
  type_error(std::string(name) + " must be bfloat16 or float16, got " + name_of(t.scalar_type()));
}
int dtype_logits(const Tensor &t) {
  return t.scalar_type() == ScalarType::Float ? TGEMM_DT_F32 : dtype16(t, "logits");
}

// Device pointer of a tensor's first element.  (Checked to be on the GPU.)
template <class T = void>
T *ptr(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

// The device a call's tensors share; makes it current while it lives.
struct On {
  at::Device device;
  int before = -1;

  On(const Tensor &first, const char *name) : device(first.device()) {
    if (!first.is_cuda()) value_error(std::string(name) + " must be on a GPU");
    const int now = c10::hip::current_device();
    if (now != device.index()) {
      before = now;
      c10::hip::set_device(device.index());
    }
  }
  ~On() {
    if (before < 0) return;
    try {
      c10::hip::set_device((c10::DeviceIndex)before);
    } catch (...) {  // (a destructor lets nothing out; the device was current before)
    }
  }
  On(const On &) = delete;

  hipStream_t stream() const { return c10::hip::getCurrentHIPStream(device.index()).stream(); }
  Tensor empty(at::IntArrayRef shape, ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(device));
  }
  const Tensor &same(const Tensor &t, const char *name) const {
    if (t.device() != device)
      value_error(std::string(name) + " is on " + t.device().str() + ", not on " + device.str() + " with the other operands");
    return t;
  }
  void typed(const Tensor &t, const char *name, ScalarType want) const {
    same(t, name);
    if (t.scalar_type() != want)
      type_error(std::string(name) + " must be " + name_of(want) + ", got " + name_of(t.scalar_type()));
  }
  void shaped(const Tensor &t, const char *name, at::IntArrayRef want) const {
    if (t.sizes() != want)
      value_error(std::string(name) + " must have shape " + shape_str(want) + ", got " + shape_str(t.sizes()));
  }
  // Row stride of a rows x cols matrix with contiguous rows.
  int64_t mat(const Tensor &t, const char *name, ScalarType want, int64_t rows, int64_t cols) const {
    typed(t, name, want);
    shaped(t, name, {rows, cols});
    const int64_t s0 = t.stride(0), s1 = t.stride(1);
    if ((s1 != 1 && cols > 1) || (rows > 1 && s0 < cols))
      value_error(std::string(name) + " must be row-major (strides " + shape_str(t.strides()) + ")");
    return std::max(s0, cols);
  }
  template <class T = void>
  T *packed(const Tensor &t, const char *name, ScalarType want, at::IntArrayRef shape) const {
    typed(t, name, want);
    shaped(t, name, shape);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return ptr<T>(t);
  }
  // A given output or a new one.
  Tensor out(PyObject *o, const char *name, ScalarType t, at::IntArrayRef shape) const {
    return o == Py_None ? empty(shape, t) : tensor(o, name);
  }
  // A given workspace or a new one of `need` bytes.
  Tensor workspace(PyObject *o, uint64_t need) const {
    if (o == Py_None) return empty({(int64_t)std::max<uint64_t>(need, 16)}, ScalarType::Byte);
    const Tensor &t = tensor(o, "workspace");
    same(t, "workspace");
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    return t;
  }
};

void matrix(const Tensor &t, const char *name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be a matrix");
}

struct Layout {
  int trans;
  int64_t ld;
};
// Storage of the r x c matrix with strides s0, s1: row-major (0) or the
// transpose of a row-major array (1).
Layout layout(int64_t r, int64_t c, int64_t s0, int64_t s1, const char *name) {
  if (s1 == 1 && (s0 >= c || r == 1)) return {0, std::max(s0, c)};
  if (s0 == 1 && (s1 >= r || c == 1)) return {1, std::max(s1, r)};
  value_error(std::string(name) + " must be row-major or a transposed row-major view (strides (" + std::to_string(s0) +
              ", " + std::to_string(s1) + "))");
}

bool gated(int64_t act) { return act == TGEMM_ACT_SWIGLU || act == TGEMM_ACT_GEGLU; }
int64_t halved(int64_t n, int64_t act) {
  if (!gated(act)) return n;
  if (n % 2) value_error("a gated activation takes an even number of columns, got " + std::to_string(n));
  return n / 2;
}

void check(int rc) {
  if (rc != TGEMM_OK) throw Failed{rc};
}
PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *tuple2(PyObject *a, PyObject *b) {
  PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}
PyObject *none() {
  Py_INCREF(Py_None);
  return Py_None;
}

typedef PyObject *const *Args;

// a, b, bias, act, residual, preact, out, workspace
PyObject *epilogue(Args o) {
  const Tensor &a = tensor(o[0], "a"), &b = tensor(o[1], "b");
  On on(a, "a");
  matrix(a, "a");
  matrix(b, "b");
  if (a.size(1) != b.size(0))
    value_error("shapes " + shape_str(a.sizes()) + " and " + shape_str(b.sizes()) + " do not multiply");
  tgemm_epilogue_args p{};
  p.dtype = dtype16(a, "a");
  if (b.scalar_type() != a.scalar_type()) type_error("a and b must both be bfloat16 or both float16");
  on.same(b, "b");
  const ScalarType t = a.scalar_type();
  p.M = a.size(0);
  p.K = a.size(1);
  p.N = b.size(1);
  p.act = integer(o[3], "act");
  const int64_t F = halved(p.N, p.act);
  const Layout la = layout(p.M, p.K, a.stride(0), a.stride(1), "a"), lb = layout(p.K, p.N, b.stride(0), b.stride(1), "b");
  p.trans_a = la.trans;
  p.lda = la.ld;
  p.trans_b = lb.trans;
  p.ldb = lb.ld;
  p.A = ptr(a);
  p.B = ptr(b);
  if (o[2] != Py_None) p.bias = on.packed(tensor(o[2], "bias"), "bias", t, {p.N});
  if (o[4] != Py_None) {
    const Tensor &r = tensor(o[4], "residual");
    p.ldr = on.mat(r, "residual", t, p.M, F);
    p.residual = ptr(r);
  }
  if (o[5] != Py_None) {
    const Tensor &z = tensor(o[5], "preact");
    p.ldp = on.mat(z, "preact", t, p.M, p.N);
    p.preact = ptr(z);
  }
  const Tensor out = on.out(o[6], "out", t, {p.M, F});
  p.ldc = on.mat(out, "out", t, p.M, F);
  p.C = ptr(out);
  const uint64_t need = tgemm_epilogue_workspace_bytes(p.trans_a, p.trans_b, p.M, p.N, p.K);
  Tensor ws;
  if (need) {
    ws = on.workspace(o[7], need);
    p.workspace = ptr(ws);
    p.workspace_bytes = (uint64_t)ws.nbytes();
  }
  check(gemm_epilogue(&p, on.stream()));
  return wrap(out);
}

// dout, preact, act, offsets, want_dbias, dz, dbias, workspace
PyObject *epilogue_backward(Args o) {
  const Tensor &dout = tensor(o[0], "dout");
  On on(dout, "dout");
  tgemm_epilogue_backward_args p{};
  p.dtype = dtype16(dout, "dout");
  matrix(dout, "dout");
  const ScalarType t = dout.scalar_type();
  p.M = dout.size(0);
  const int64_t F = dout.size(1);
  p.act = integer(o[2], "act");
  p.N = gated(p.act) ? 2 * F : F;
  p.ldd = on.mat(dout, "dout", t, p.M, F);
  p.dout = ptr(dout);
  if (p.act != TGEMM_ACT_NONE) {
    if (o[1] == Py_None) value_error("this act needs preact");
    const Tensor &z = tensor(o[1], "preact");
    p.ldp = on.mat(z, "preact", t, p.M, p.N);
    p.preact = ptr(z);
  }
  Tensor dz = dout;
  if (o[5] != Py_None || p.act != TGEMM_ACT_NONE) {
    dz = on.out(o[5], "dz", t, {p.M, p.N});
    p.ldz = on.mat(dz, "dz", t, p.M, p.N);
    p.dz = ptr(dz);
  }
  if (o[3] != Py_None) {
    const Tensor &off = tensor(o[3], "offsets");
    p.groups = off.numel() - 1;
    if (p.groups < 1) value_error("offsets must hold groups + 1 entries");
    p.offsets = on.packed<int32_t>(off, "offsets", ScalarType::Int, {p.groups + 1});
  }
  Tensor dbias, ws;
  const bool want = truth(o[4], "want_dbias");
  if (want) {
    if (p.groups) {
      dbias = on.out(o[6], "dbias", t, {p.groups, p.N});
      p.dbias = on.packed(dbias, "dbias", t, {p.groups, p.N});
    } else {
      dbias = on.out(o[6], "dbias", t, {p.N});
      p.dbias = on.packed(dbias, "dbias", t, {p.N});
    }
    ws = on.workspace(o[7], tgemm_epilogue_backward_workspace_bytes(p.M, p.N, p.groups));
    p.workspace = ptr(ws);
    p.workspace_bytes = (uint64_t)ws.nbytes();
  }
  check(gemm_epilogue_backward(&p, on.stream()));
  return tuple2(wrap(dz), want ? wrap(dbias) : none());
}

// a, b, offsets, rows, bias, act, preact, out
PyObject *grouped(Args o) {
  const Tensor &a = tensor(o[0], "a"), &b = tensor(o[1], "b"), &off = tensor(o[2], "offsets");
  On on(a, "a");
  tgemm_grouped_args p{};
  p.dtype = dtype16(a, "a");
  matrix(a, "a");
  const ScalarType t = a.scalar_type();
  const int64_t S = a.size(0);
  p.K = a.size(1);
  p.lda = on.mat(a, "a", t, S, p.K);
  p.A = ptr(a);
  if (b.dim() != 3) value_error("b must be (groups, K, N)");
  on.typed(b, "b", t);
  p.groups = b.size(0);
  p.N = b.size(2);
  if (b.size(1) != p.K)
    value_error("a has " + std::to_string(p.K) + " columns, b " + std::to_string(b.size(1)) + " rows");
  const Layout lb = layout(p.K, p.N, b.stride(1), b.stride(2), "b");
  p.trans_b = lb.trans;
  p.ldb = lb.ld;
  p.stride_b = b.stride(0);
  p.B = ptr(b);
  p.act = integer(o[5], "act");
  const int64_t F = halved(p.N, p.act);
  p.offsets = on.packed<int32_t>(off, "offsets", ScalarType::Int, {p.groups + 1});
  p.R = p.src_rows = S;
  if (o[3] != Py_None) {
    const Tensor &rows = tensor(o[3], "rows");
    p.R = rows.numel();
    p.rows = on.packed<int32_t>(rows, "rows", ScalarType::Int, {p.R});
  }
  if (o[4] != Py_None) p.bias = on.packed(tensor(o[4], "bias"), "bias", t, {p.groups, p.N});
  if (o[6] != Py_None) {
    const Tensor &z = tensor(o[6], "preact");
    p.ldp = on.mat(z, "preact", t, p.R, p.N);
    p.preact = ptr(z);
  }
  const Tensor out = on.out(o[7], "out", t, {p.R, F});
  p.ldc = on.mat(out, "out", t, p.R, F);
  p.C = ptr(out);
  check(gemm_grouped(&p, on.stream()));
  return wrap(out);
}

// x, y, offsets, out
PyObject *grouped_tn(Args o) {
  const Tensor &x = tensor(o[0], "x"), &y = tensor(o[1], "y"), &off = tensor(o[2], "offsets");
  On on(x, "x");
  tgemm_grouped_tn_args p{};
  p.dtype = dtype16(x, "x");
  matrix(x, "x");
  matrix(y, "y");
  if (x.size(0) != y.size(0)) value_error("x and y must have as many rows");
  const ScalarType t = x.scalar_type();
  p.R = x.size(0);
  p.P = x.size(1);
  p.Q = y.size(1);
  p.ldx = on.mat(x, "x", t, p.R, p.P);
  p.ldy = on.mat(y, "y", t, p.R, p.Q);
  p.X = ptr(x);
  p.Y = ptr(y);
  p.groups = off.numel() - 1;
  if (p.groups < 1) value_error("offsets must hold groups + 1 entries");
  p.offsets = on.packed<int32_t>(off, "offsets", ScalarType::Int, {p.groups + 1});
  const Tensor out = on.out(o[3], "out", t, {p.groups, p.P, p.Q});
  p.out = on.packed(out, "out", t, {p.groups, p.P, p.Q});
  check(gemm_grouped_tn(&p, on.stream()));
  return wrap(out);
}

// logits, k, score, bias, groups, groups_used, renormalize, scale, weights, ids
PyObject *topk(Args o) {
  const Tensor &x = tensor(o[0], "logits");
  On on(x, "logits");
  tgemm_route_args p{};
  p.dtype = dtype_logits(x);
  matrix(x, "logits");
  p.T = x.size(0);
  p.E = x.size(1);
  p.ld = on.mat(x, "logits", x.scalar_type(), p.T, p.E);
  p.logits = ptr(x);
  p.k = integer(o[1], "k");
  if (p.k < 0) value_error("k must not be negative");
  p.score = integer(o[2], "score");
  if (o[3] != Py_None) p.bias = on.packed<float>(tensor(o[3], "bias"), "bias", ScalarType::Float, {p.E});
  p.groups = integer(o[4], "groups");
  p.groups_used = integer(o[5], "groups_used");
  p.renormalize = truth(o[6], "renormalize");
  p.scale = PyFloat_AsDouble(o[7]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    type_error("scale must be a number");
  }
  // (More choices than experts are refused before memory is taken for them.)
  if (p.k > p.E) check(route_topk(&p, on.stream()));
  const Tensor w = on.out(o[8], "weights", ScalarType::Float, {p.T, p.k}), ids = on.out(o[9], "ids", ScalarType::Int, {p.T, p.k});
  p.weights = on.packed<float>(w, "weights", ScalarType::Float, {p.T, p.k});
  p.ids = on.packed<int32_t>(ids, "ids", ScalarType::Int, {p.T, p.k});
  check(route_topk(&p, on.stream()));
  return tuple2(wrap(w), wrap(ids));
}

// dweights, logits, ids, score, renormalize, scale, dlogits
PyObject *topk_backward(Args o) {
  const Tensor &dw = tensor(o[0], "dweights"), &x = tensor(o[1], "logits"), &ids = tensor(o[2], "ids");
  On on(x, "logits");
  tgemm_route_backward_args p{};
  p.dtype = dtype_logits(x);
  matrix(x, "logits");
  matrix(ids, "ids");
  p.T = x.size(0);
  p.E = x.size(1);
  p.k = ids.size(1);
  p.ld = on.mat(x, "logits", x.scalar_type(), p.T, p.E);
  p.logits = ptr(x);
  p.ids = on.packed<int32_t>(ids, "ids", ScalarType::Int, {p.T, p.k});
  p.dweights = on.packed<float>(dw, "dweights", ScalarType::Float, {p.T, p.k});
  p.score = integer(o[3], "score");
  p.renormalize = truth(o[4], "renormalize");
  p.scale = PyFloat_AsDouble(o[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    type_error("scale must be a number");
  }
  const Tensor d = on.out(o[6], "dlogits", x.scalar_type(), {p.T, p.E});
  p.ldo = on.mat(d, "dlogits", x.scalar_type(), p.T, p.E);
  p.dlogits = ptr(d);
  check(route_topk_backward(&p, on.stream()));
  return wrap(d);
}

// ids, experts, offsets, rows, slots, workspace
PyObject *plan(Args o) {
  const Tensor &ids = tensor(o[0], "ids");
  On on(ids, "ids");
  matrix(ids, "ids");
  const ScalarType t = ScalarType::Int;
  tgemm_route_plan_args p{};
  p.T = ids.size(0);
  p.k = ids.size(1);
  p.E = integer(o[1], "experts");
  if (p.E < 0) value_error("experts must not be negative");
  if (p.E > 1024) check(route_plan(&p, on.stream()));  // (refused before offsets for them are made)
  p.ids = on.packed<int32_t>(ids, "ids", t, {p.T, p.k});
  const Tensor off = on.out(o[2], "offsets", t, {p.E + 1}), rows = on.out(o[3], "rows", t, {p.T * p.k}),
               slots = on.out(o[4], "slots", t, {p.T, p.k});
  p.offsets = on.packed<int32_t>(off, "offsets", t, {p.E + 1});
  p.rows = on.packed<int32_t>(rows, "rows", t, {p.T * p.k});
  p.slots = on.packed<int32_t>(slots, "slots", t, {p.T, p.k});
  const uint64_t need = tgemm_route_plan_workspace_bytes(p.T, p.k, p.E);
  Tensor ws;
  if (need || o[5] != Py_None) {
    ws = on.workspace(o[5], need);
    p.workspace = ptr(ws);
    p.workspace_bytes = (uint64_t)ws.nbytes();
  }
  check(route_plan(&p, on.stream()));
  PyObject *a = wrap(off), *b = wrap(rows), *c = wrap(slots);
  PyObject *r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return r;
}

// x, rows, out
PyObject *gather(Args o) {
  const Tensor &x = tensor(o[0], "x"), &rows = tensor(o[1], "rows");
  On on(x, "x");
  dtype16(x, "x");
  matrix(x, "x");
  const ScalarType t = x.scalar_type();
  tgemm_expert_gather_args p{};
  p.src_rows = x.size(0);
  p.D = x.size(1);
  p.R = rows.numel();
  p.ldx = on.mat(x, "x", t, p.src_rows, p.D);
  p.x = ptr(x);
  p.rows = on.packed<int32_t>(rows, "rows", ScalarType::Int, {p.R});
  const Tensor out = on.out(o[2], "out", t, {p.R, p.D});
  p.ldo = on.mat(out, "out", t, p.R, p.D);
  p.out = ptr(out);
  check(expert_gather(&p, on.stream()));
  return wrap(out);
}

// h, slots, weights, residual, out
PyObject *combine(Args o) {
  const Tensor &h = tensor(o[0], "h"), &slots = tensor(o[1], "slots");
  On on(h, "h");
  tgemm_expert_combine_args p{};
  p.dtype = dtype16(h, "h");
  matrix(h, "h");
  matrix(slots, "slots");
  const ScalarType t = h.scalar_type();
  p.R = h.size(0);
  p.D = h.size(1);
  p.T = slots.size(0);
  p.k = slots.size(1);
  p.ldh = on.mat(h, "h", t, p.R, p.D);
  p.h = ptr(h);
  p.slots = on.packed<int32_t>(slots, "slots", ScalarType::Int, {p.T, p.k});
  if (o[2] != Py_None) p.weights = on.packed<float>(tensor(o[2], "weights"), "weights", ScalarType::Float, {p.T, p.k});
  if (o[3] != Py_None) {
    const Tensor &r = tensor(o[3], "residual");
    p.ldr = on.mat(r, "residual", t, p.T, p.D);
    p.residual = ptr(r);
  }
  const Tensor out = on.out(o[4], "out", t, {p.T, p.D});
  p.ldo = on.mat(out, "out", t, p.T, p.D);
  p.out = ptr(out);
  check(expert_combine(&p, on.stream()));
  return wrap(out);
}

// dout, h, slots, weights, dh, dweights
PyObject *combine_backward(Args o) {
  const Tensor &dout = tensor(o[0], "dout"), &h = tensor(o[1], "h"), &slots = tensor(o[2], "slots"),
               &w = tensor(o[3], "weights");
  On on(dout, "dout");
  tgemm_expert_combine_backward_args p{};
  p.dtype = dtype16(dout, "dout");
  matrix(dout, "dout");
  matrix(h, "h");
  matrix(slots, "slots");
  const ScalarType t = dout.scalar_type();
  p.T = dout.size(0);
  p.D = dout.size(1);
  p.R = h.size(0);
  p.k = slots.size(1);
  p.ldd = on.mat(dout, "dout", t, p.T, p.D);
  p.dout = ptr(dout);
  p.ldh = on.mat(h, "h", t, p.R, p.D);
  p.h = ptr(h);
  p.slots = on.packed<int32_t>(slots, "slots", ScalarType::Int, {p.T, p.k});
  p.weights = on.packed<float>(w, "weights", ScalarType::Float, {p.T, p.k});
  const Tensor dh = on.out(o[4], "dh", t, {p.R, p.D}), dw = on.out(o[5], "dweights", ScalarType::Float, {p.T, p.k});
  p.ldg = on.mat(dh, "dh", t, p.R, p.D);
  p.dh = ptr(dh);
  p.dweights = on.packed<float>(dw, "dweights", ScalarType::Float, {p.T, p.k});
  check(expert_combine_backward(&p, on.stream()));
  return tuple2(wrap(dh), wrap(dw));
}

// Runs F with the number of arguments it takes; nothing it throws gets out.
template <PyObject *(*F)(Args), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raise &e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Failed &e) {
    PyObject *v = Py_BuildValue("(is)", e.code, tgemm_ffn_last_error());
    if (v) PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, v);
    Py_XDECREF(v);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject *set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  return none();
}

#define TGEMM_ENTRY(NAME, F, N) {NAME, (PyCFunction)(void (*)(void))&entry<F, N>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {TGEMM_ENTRY("gemm_epilogue", epilogue, 8),
                          TGEMM_ENTRY("epilogue_backward", epilogue_backward, 8),
                          TGEMM_ENTRY("gemm_grouped", grouped, 8),
                          TGEMM_ENTRY("gemm_grouped_tn", grouped_tn, 4),
                          TGEMM_ENTRY("route_topk", topk, 10),
                          TGEMM_ENTRY("route_topk_backward", topk_backward, 7),
                          TGEMM_ENTRY("route_plan", plan, 6),
                          TGEMM_ENTRY("expert_gather", gather, 3),
                          TGEMM_ENTRY("expert_combine", combine, 5),
                          TGEMM_ENTRY("expert_combine_backward", combine_backward, 6),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ffn_binding", "Compiled part of ffn.py.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__ffn_binding(void) { return PyModule_Create(&kModule); }
