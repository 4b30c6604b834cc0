// CPython binding of the MXFP4 and integer 4-bit operators, the norm, the router and the experts: the
// checks of the tensors, their allocation and the call in one step, since a decode step's kernels
// (3 to 8 us) are shorter than the same checks written in Python (rmsnorm 7.7 us a call through ctypes).
//
// The package exports these functions as they are (a Python function around each adds 0.1 to
// 0.2 us).  None stands for an absent tensor.  Errors are TypeError and ValueError for
// what a tensor is, and the package's error class (set_error) for a status of the library.
#define PY_SSIZE_T_CLEAN
#include <ATen/ops/empty.h>
#include <c10/hip/HIPException.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "sp24.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;  // the package's error class: called with (function, status)

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Failed{};
}

bool absent(PyObject* o) { return o == Py_None; }

// The tensor of an argument, after the checks that every operand gets.
const Tensor& need(PyObject* o, const char* name, std::initializer_list<ScalarType> types, int64_t ndim,
                   const at::Device* device) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be on the GPU", name);
  if (device != nullptr && t.device() != *device)
    fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), device->str().c_str());
  bool known = false;
  for (ScalarType s : types) known = known || t.scalar_type() == s;
  if (!known)
    fail(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
         c10::toString(*types.begin()));
  if (t.dim() != ndim) fail(PyExc_ValueError, "%s must be %d-D", name, (int)ndim);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

// An output: the given tensor, of this shape, or a new one.
Tensor output(PyObject* o, const char* name, std::initializer_list<ScalarType> types, at::IntArrayRef shape,
              const at::Device& device) {
  if (absent(o)) return at::empty(shape, at::TensorOptions().dtype(*types.begin()).device(device));
  const Tensor& t = need(o, name, types, (int64_t)shape.size(), &device);
  if (t.sizes() != shape) {
    if (shape.size() == 1) fail(PyExc_ValueError, "%s must hold %lld values", name, (long long)shape[0]);
    fail(PyExc_ValueError, "%s must be [%lld, %lld]", name, (long long)shape[0], (long long)shape[1]);
  }
  return t;
}

struct Operand {  // MXFP4: codes [rows, cols/2], scales rows * cols/32 bytes
  const uint8_t *codes, *scales;
  int64_t rows, cols;
};
Operand operand(PyObject* codes, PyObject* scales, const char* name, const at::Device* device) {
  const Tensor& c = need(codes, name, {at::kByte}, 2, device);
  const at::Device d = c.device();
  const Tensor& s = need(scales, name, {at::kByte}, 1, &d);
  const int64_t rows = c.size(0), half = c.size(1);
  if (half % 64 != 0 || s.numel() * 16 != rows * half)
    fail(PyExc_ValueError, "%s: codes [%lld, %lld] need a multiple of 64 columns and %lld scales, got %lld", name,
         (long long)rows, (long long)half, (long long)(rows * half / 16), (long long)s.numel());
  return Operand{c.const_data_ptr<uint8_t>(), s.const_data_ptr<uint8_t>(), rows, 2 * half};
}

void mx4_cols(int64_t cols) {
  if (cols % 128 != 0) fail(PyExc_ValueError, "MXFP4 needs a multiple of 128 columns, got %lld", (long long)cols);
}

void* stream_of(const at::Device& d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

void check(const char* fn, int status) {
  if (status == SP24_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "si", fn, status)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

// A tuple of tensors (None where undefined).
PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) throw Failed{};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      throw Failed{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return v;
}
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// A workspace of at least this many bytes: the given tensor if it is large enough, or a new one.
Tensor workspace(PyObject* o, size_t bytes, const at::Device& d) {
  Tensor ws;
  if (!absent(o)) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "ws must be a tensor");
    ws = THPVariable_Unpack(o);
    if (!ws.is_cuda() || ws.device() != d || !ws.is_contiguous())
      fail(PyExc_ValueError, "ws must be contiguous and on %s", d.str().c_str());
  }
  if (bytes > 0 && (!ws.defined() || (size_t)ws.nbytes() < bytes))
    ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(d));
  return ws;
}

PyObject* quant(PyObject* const* a) {  // x, out, scales
  const Tensor& x = need(a[0], "x", {at::kBFloat16}, 2, nullptr);
  const int64_t rows = x.size(0), cols = x.size(1);
  mx4_cols(cols);
  const at::Device d = x.device();
  const Tensor out = output(a[1], "out", {at::kByte}, {rows, cols / 2}, d);
  const Tensor scales = output(a[2], "scales", {at::kByte}, {rows * cols / 32}, d);
  check("sp24_quant_mxfp4", sp24_quant_mxfp4(x.data_ptr(), rows, cols, out.data_ptr<uint8_t>(),
                                             scales.data_ptr<uint8_t>(), stream_of(d)));
  return pack({out, scales});
}

PyObject* dequant(PyObject* const* a) {  // codes, scales, out
  const Operand q = operand(a[0], a[1], "operand", nullptr);
  const at::Device d = THPVariable_Unpack(a[0]).device();
  const Tensor out = output(a[2], "out", {at::kBFloat16}, {q.rows, q.cols}, d);
  check("sp24_dequant_mxfp4", sp24_dequant_mxfp4(q.codes, q.scales, q.rows, q.cols, out.data_ptr(), stream_of(d)));
  return THPVariable_Wrap(out);
}

PyObject* gemm(PyObject* const* a) {  // x codes, x scales, w codes, w scales, out
  const Operand x = operand(a[0], a[1], "x", nullptr);
  const at::Device d = THPVariable_Unpack(a[0]).device();
  const Operand w = operand(a[2], a[3], "w", &d);
  if (w.cols != x.cols)
    fail(PyExc_ValueError, "w has %lld columns, x has %lld", (long long)w.cols, (long long)x.cols);
  const Tensor out = output(a[4], "out", {at::kBFloat16}, {x.rows, w.rows}, d);
  check("sp24_gemm_mxfp4", sp24_gemm_mxfp4(x.rows, w.rows, x.cols, x.codes, x.scales, w.codes, w.scales,
                                           out.data_ptr(), stream_of(d)));
  return THPVariable_Wrap(out);
}

PyObject* gated(PyObject* const* a) {  // x codes, x scales, w codes, w scales, quantise, out, out scales
  const Operand x = operand(a[0], a[1], "x", nullptr);
  const at::Device d = THPVariable_Unpack(a[0]).device();
  const Operand w = operand(a[2], a[3], "w", &d);
  if (w.cols != x.cols || w.rows % 2 != 0)
    fail(PyExc_ValueError, "w must be [2 f, %lld] values, got [%lld, %lld]", (long long)x.cols, (long long)w.rows,
         (long long)w.cols);
  const int64_t f = w.rows / 2;
  const int quantise = PyObject_IsTrue(a[4]);
  if (quantise < 0) throw Failed{};
  Tensor out, scales;
  if (quantise) {
    mx4_cols(f);
    out = output(a[5], "out", {at::kByte}, {x.rows, f / 2}, d);
    scales = output(a[6], "out_scales", {at::kByte}, {x.rows * f / 32}, d);
  } else {
    if (!absent(a[6])) fail(PyExc_ValueError, "out_scales goes with quantise=True");
    out = output(a[5], "out", {at::kBFloat16}, {x.rows, f}, d);
  }
  check("sp24_gated_mxfp4",
        sp24_gated_mxfp4(x.rows, f, x.cols, x.codes, x.scales, w.codes, w.scales, quantise ? nullptr : out.data_ptr(),
                         quantise ? out.data_ptr<uint8_t>() : nullptr,
                         quantise ? scales.data_ptr<uint8_t>() : nullptr, stream_of(d)));
  return quantise ? pack({out, scales}) : THPVariable_Wrap(out);
}

struct NormInputs {
  const Tensor &x, &weight;
  Tensor residual, residual_out;
  int64_t m, k;
};
NormInputs norm_inputs(PyObject* xo, PyObject* wo, PyObject* ro, PyObject* roo) {
  const Tensor& x = need(xo, "x", {at::kBFloat16}, 2, nullptr);
  const at::Device d = x.device();
  const Tensor& w = need(wo, "weight", {at::kBFloat16}, 1, &d);
  NormInputs n{x, w, Tensor(), Tensor(), x.size(0), x.size(1)};
  if (w.numel() != n.k) fail(PyExc_ValueError, "weight must hold %lld values", (long long)n.k);
  if (!absent(ro)) {
    n.residual = need(ro, "residual", {at::kBFloat16}, 2, &d);
    if (n.residual.sizes() != x.sizes())
      fail(PyExc_ValueError, "residual must be [%lld, %lld]", (long long)n.m, (long long)n.k);
    n.residual_out = output(roo, "residual_out", {at::kBFloat16}, {n.m, n.k}, d);
  } else if (!absent(roo)) {
    fail(PyExc_ValueError, "residual_out goes with a residual");
  }
  return n;
}

PyObject* rmsnorm(PyObject* const* a) {  // x, weight, kind, residual, eps, group, out, scales, residual_out
  const NormInputs n = norm_inputs(a[0], a[1], a[3], a[8]);
  const int64_t kind = integer(a[2]), group = integer(a[5]);
  const double eps = number(a[4]);
  const at::Device d = n.x.device();
  Tensor out, scales;
  switch (kind) {
    case SP24_NORM_MXFP4:
      mx4_cols(n.k);
      out = output(a[6], "out", {at::kByte}, {n.m, n.k / 2}, d);
      scales = output(a[7], "scales", {at::kByte}, {n.m * n.k / 32}, d);
      break;
    case SP24_NORM_BF16:
      if (!absent(a[7])) fail(PyExc_ValueError, "a bf16 output has no scales");
      out = output(a[6], "out", {at::kBFloat16}, {n.m, n.k}, d);
      break;
    case SP24_NORM_INT8_ROWS:
      out = output(a[6], "out", {at::kChar}, {n.m, n.k}, d);
      scales = output(a[7], "scales", {at::kFloat}, {n.m}, d);
      break;
    case SP24_NORM_FP8_ROWS:
      out = output(a[6], "out", {at::kByte, at::kFloat8_e4m3fn}, {n.m, n.k}, d);
      scales = output(a[7], "scales", {at::kFloat}, {n.m}, d);
      break;
    case SP24_NORM_FP8_GROUPS:
      if (group < 8 || group % 8 != 0 || n.k % group != 0)
        fail(PyExc_ValueError, "group must be a multiple of 8 that divides k=%lld", (long long)n.k);
      out = output(a[6], "out", {at::kByte, at::kFloat8_e4m3fn}, {n.m, n.k}, d);
      scales = output(a[7], "scales", {at::kFloat}, {n.m, n.k / group}, d);
      break;
    default: fail(PyExc_ValueError, "unknown norm kind %lld", (long long)kind);
  }
  check("sp24_rmsnorm", sp24_rmsnorm((int)kind, n.m, n.k, group, n.x.data_ptr(), data(n.residual),
                                     data(n.residual_out), n.weight.data_ptr(), (float)eps, out.data_ptr(),
                                     data(scales), stream_of(d)));
  return pack({out, scales, n.residual_out});
}

// x, weight, gate_up codes and scales, down codes and scales, residual, eps, out, residual_out, ws
PyObject* ffn(PyObject* const* a) {
  const NormInputs n = norm_inputs(a[0], a[1], a[6], a[9]);
  const at::Device d = n.x.device();
  const Operand gu = operand(a[2], a[3], "gate_up", &d), dn = operand(a[4], a[5], "down", &d);
  const int64_t f = dn.cols;
  if (gu.cols != n.k || dn.rows != n.k || gu.rows != 2 * f)
    fail(PyExc_ValueError, "gate_up must be [%lld, %lld] values and down [%lld, %lld], got [%lld, %lld] and [%lld, %lld]",
         (long long)(2 * f), (long long)n.k, (long long)n.k, (long long)f, (long long)gu.rows, (long long)gu.cols,
         (long long)dn.rows, (long long)f);
  const double eps = number(a[7]);
  const Tensor out = output(a[8], "out", {at::kBFloat16}, {n.m, n.k}, d);
  const size_t bytes = sp24_ffn_mxfp4_workspace_size(n.m, n.k, f);
  const Tensor ws = workspace(a[10], bytes, d);
  check("sp24_ffn_mxfp4", sp24_ffn_mxfp4(n.m, n.k, f, n.x.data_ptr(), data(n.residual), data(n.residual_out),
                                         n.weight.data_ptr(), (float)eps, gu.codes, gu.scales, dn.codes, dn.scales,
                                         out.data_ptr(), data(ws), bytes, stream_of(d)));
  return pack({out, n.residual_out});
}

struct Weight4 {  // integer 4-bit: codes [rows, cols/2], scales and zeros [rows, cols/group], or with experts in front
  const uint8_t *codes, *zeros;
  const void* scales;
  int64_t experts, rows, cols, group;
};
Weight4 weight4(PyObject* codes, PyObject* scales, PyObject* zeros, const char* name, int64_t ndim,
                const at::Device* device) {
  const Tensor& c = need(codes, name, {at::kByte}, ndim, device);
  const at::Device d = c.device();
  const Tensor& s = need(scales, "scales", {at::kBFloat16}, ndim, &d);
  const int64_t experts = ndim == 3 ? c.size(0) : 1, rows = c.size(ndim - 2), cols = 2 * c.size(ndim - 1);
  const int64_t groups = s.size(ndim - 1), group = groups > 0 ? cols / groups : 0;
  if ((ndim == 3 && s.size(0) != experts) || s.size(ndim - 2) != rows || groups * group != cols ||
      (group != 32 && group != 64 && group != 128))
    fail(PyExc_ValueError, "%s: codes of [%lld, %lld] values need a scale of each row's groups of 32, 64 or 128", name,
         (long long)rows, (long long)cols);
  const uint8_t* zp = nullptr;
  if (!absent(zeros)) {
    const Tensor& z = need(zeros, "zeros", {at::kByte}, ndim, &d);
    if (z.sizes() != s.sizes()) fail(PyExc_ValueError, "%s: zeros must have the shape of the scales", name);
    zp = z.const_data_ptr<uint8_t>();
  }
  return Weight4{c.const_data_ptr<uint8_t>(), zp, s.const_data_ptr(), experts, rows, cols, group};
}

PyObject* quant_int4(PyObject* const* a) {  // w, group, zeros, out, scales_out, zeros_out
  const Tensor& w = need(a[0], "w", {at::kBFloat16}, 2, nullptr);
  const int64_t rows = w.size(0), cols = w.size(1), group = integer(a[1]);
  if ((group != 32 && group != 64 && group != 128) || cols % group != 0)
    fail(PyExc_ValueError, "group must be 32, 64 or 128 and divide the %lld columns, got %lld", (long long)cols,
         (long long)group);
  const int zeros = PyObject_IsTrue(a[2]);
  if (zeros < 0) throw Failed{};
  const at::Device d = w.device();
  const Tensor out = output(a[3], "out", {at::kByte}, {rows, cols / 2}, d);
  const Tensor scales = output(a[4], "scales_out", {at::kBFloat16}, {rows, cols / group}, d);
  Tensor zp;
  if (zeros) zp = output(a[5], "zeros_out", {at::kByte}, {rows, cols / group}, d);
  else if (!absent(a[5])) fail(PyExc_ValueError, "zeros_out goes with zeros=True");
  check("sp24_quant_int4", sp24_quant_int4(w.data_ptr(), rows, cols, group, out.data_ptr<uint8_t>(), scales.data_ptr(),
                                           static_cast<uint8_t*>(data(zp)), stream_of(d)));
  return pack({out, scales, zp});
}

PyObject* dequant_int4(PyObject* const* a) {  // codes, scales, zeros, out
  const Weight4 w = weight4(a[0], a[1], a[2], "codes", 2, nullptr);
  const at::Device d = THPVariable_Unpack(a[0]).device();
  const Tensor out = output(a[3], "out", {at::kBFloat16}, {w.rows, w.cols}, d);
  check("sp24_dequant_int4", sp24_dequant_int4(w.codes, w.scales, w.zeros, w.rows, w.cols, w.group, out.data_ptr(),
                                               stream_of(d)));
  return THPVariable_Wrap(out);
}

PyObject* gemm_int4(PyObject* const* a) {  // x, codes, scales, zeros, out, ws
  const Tensor& x = need(a[0], "x", {at::kBFloat16}, 2, nullptr);
  const at::Device d = x.device();
  const Weight4 w = weight4(a[1], a[2], a[3], "codes", 2, &d);
  if (w.cols != x.size(1))
    fail(PyExc_ValueError, "w has %lld columns, x has %lld", (long long)w.cols, (long long)x.size(1));
  const Tensor out = output(a[4], "out", {at::kBFloat16}, {x.size(0), w.rows}, d);
  const size_t bytes = sp24_gemm_int4_workspace_size(x.size(0), w.rows, w.cols);
  const Tensor ws = workspace(a[5], bytes, d);
  check("sp24_gemm_int4", sp24_gemm_int4(x.size(0), w.rows, w.cols, w.group, x.data_ptr(), w.codes, w.scales, w.zeros,
                                         out.data_ptr(), data(ws), bytes, stream_of(d)));
  return THPVariable_Wrap(out);
}

// logits, top, kind, bias, groups, top_groups, group_best, renormalise, factor, ids, weights
PyObject* route(PyObject* const* a) {
  const Tensor& l = need(a[0], "logits", {at::kFloat, at::kBFloat16}, 2, nullptr);
  const at::Device d = l.device();
  const int64_t tokens = l.size(0);
  sp24_router r{};
  r.experts = l.size(1);
  r.logits_fp32 = l.scalar_type() == at::kFloat;
  r.top = integer(a[1]);
  const int64_t kind = integer(a[2]), best = integer(a[6]);
  if (kind != SP24_ROUTE_SOFTMAX && kind != SP24_ROUTE_SIGMOID)
    fail(PyExc_ValueError, "unknown route kind %lld", (long long)kind);
  if (best != 1 && best != 2) fail(PyExc_ValueError, "group_best must be 1 or 2, got %lld", (long long)best);
  r.kind = (int)kind;
  r.groups = integer(a[4]);
  r.top_groups = integer(a[5]);
  r.group_best = (int)best;
  r.renormalise = PyObject_IsTrue(a[7]);
  if (r.renormalise < 0) throw Failed{};
  r.factor = (float)number(a[8]);
  const float* bias = nullptr;
  if (!absent(a[3])) {
    const Tensor& b = need(a[3], "bias", {at::kFloat}, 1, &d);
    if (b.numel() != r.experts) fail(PyExc_ValueError, "bias must hold %lld values", (long long)r.experts);
    bias = b.const_data_ptr<float>();
  }
  if (r.groups < 1 || r.experts % r.groups != 0 || r.top_groups < 1 || r.top_groups > r.groups || r.top < 1 ||
      r.top > r.top_groups * (r.experts / r.groups))
    fail(PyExc_ValueError, "%lld experts cannot be chosen from %lld of %lld groups of %lld experts", (long long)r.top,
         (long long)r.top_groups, (long long)r.groups, (long long)r.experts);
  const Tensor ids = output(a[9], "ids", {at::kInt}, {tokens, r.top}, d);
  const Tensor weights = output(a[10], "weights", {at::kFloat}, {tokens, r.top}, d);
  check("sp24_route", sp24_route(&r, tokens, l.const_data_ptr(), bias, ids.data_ptr<int32_t>(),
                                 weights.data_ptr<float>(), stream_of(d)));
  return pack({ids, weights});
}

// x, ids, weights, gu_codes, gu_scales, down_codes, down_scales, gu_zeros, down_zeros, out, ws
PyObject* experts_int4(PyObject* const* a) {
  const Tensor& x = need(a[0], "x", {at::kBFloat16}, 2, nullptr);
  const at::Device d = x.device();
  const Tensor& ids = need(a[1], "ids", {at::kInt}, 2, &d);
  const Tensor& weights = need(a[2], "weights", {at::kFloat}, 2, &d);
  const Weight4 gu = weight4(a[3], a[4], a[7], "gu_codes", 3, &d), dn = weight4(a[5], a[6], a[8], "down_codes", 3, &d);
  const int64_t tokens = x.size(0), top = ids.size(1), f = dn.cols;
  if (ids.size(0) != tokens || weights.sizes() != ids.sizes())
    fail(PyExc_ValueError, "ids and weights must be [%lld, top]", (long long)tokens);
  if (gu.cols != x.size(1) || dn.rows != gu.cols || gu.rows != 2 * f || dn.experts != gu.experts ||
      dn.group != gu.group)
    fail(PyExc_ValueError, "experts of [%lld, %lld] and [%lld, %lld] values (groups of %lld and %lld) do not fit "
         "tokens of %lld", (long long)gu.rows, (long long)gu.cols, (long long)dn.rows, (long long)dn.cols,
         (long long)gu.group, (long long)dn.group, (long long)x.size(1));
  const Tensor out = output(a[9], "out", {at::kBFloat16}, {tokens, gu.cols}, d);
  const size_t bytes = sp24_experts_int4_workspace_size(tokens, gu.cols, f, gu.experts, top);
  const Tensor ws = workspace(a[10], bytes, d);
  const sp24_int4_experts w{gu.experts, gu.cols, f, gu.group, gu.codes, gu.scales, gu.zeros, dn.codes, dn.scales,
                            dn.zeros};
  check("sp24_experts_int4", sp24_experts_int4(&w, tokens, top, x.data_ptr(), ids.const_data_ptr<int32_t>(),
                                               weights.const_data_ptr<float>(), out.data_ptr(), data(ws), bytes,
                                               stream_of(d)));
  return THPVariable_Wrap(out);
}

// A function's parameters by name, with the values of those that may be left out.
constexpr int kMost = 11;
struct Function {
  const char* name;
  PyObject* (*call)(PyObject* const*);
  int required, count;
  const char* names[kMost];
  PyObject* interned[kMost];  // the names as Python's own strings
  PyObject* defaults[kMost];  // nullptr: None
};

Function g_quant{"quant_mxfp4", quant, 1, 3, {"x", "out", "scales"}};
Function g_dequant{"dequant_mxfp4", dequant, 2, 3, {"codes", "scales", "out"}};
Function g_gemm{"gemm_mxfp4", gemm, 4, 5, {"x_codes", "x_scales", "w_codes", "w_scales", "out"}};
Function g_gated{"gated_mxfp4", gated, 4, 7,
                 {"x_codes", "x_scales", "w_codes", "w_scales", "quantise", "out", "out_scales"}};
Function g_rmsnorm{"rmsnorm", rmsnorm, 2, 9,
                   {"x", "weight", "kind", "residual", "eps", "group", "out", "scales", "residual_out"}};
Function g_ffn{"ffn_mxfp4", ffn, 6, 11,
               {"x", "weight", "gu_codes", "gu_scales", "down_codes", "down_scales", "residual", "eps", "out",
                "residual_out", "ws"}};
Function g_quant4{"quant_int4", quant_int4, 1, 6, {"w", "group", "zeros", "out", "scales_out", "zeros_out"}};
Function g_dequant4{"dequant_int4", dequant_int4, 2, 4, {"codes", "scales", "zeros", "out"}};
Function g_gemm4{"gemm_int4", gemm_int4, 3, 6, {"x", "codes", "scales", "zeros", "out", "ws"}};
Function g_route{"route", route, 2, 11,
                 {"logits", "top", "kind", "bias", "groups", "top_groups", "group_best", "renormalise", "factor",
                  "ids", "weights"}};
Function g_experts{"experts_int4", experts_int4, 7, 11,
                   {"x", "ids", "weights", "gu_codes", "gu_scales", "down_codes", "down_scales", "gu_zeros",
                    "down_zeros", "out", "ws"}};

// Arguments by position and by name into the function's order.
void place(const Function& f, PyObject* const* args, Py_ssize_t count, PyObject* names, PyObject** to) {
  if (count > f.count) fail(PyExc_TypeError, "%s() takes at most %d arguments, %d given", f.name, f.count, (int)count);
  for (int i = 0; i < f.count; ++i) to[i] = i < count ? args[i] : nullptr;
  const Py_ssize_t named = names == nullptr ? 0 : PyTuple_GET_SIZE(names);
  for (Py_ssize_t j = 0; j < named; ++j) {
    PyObject* const name = PyTuple_GET_ITEM(names, j);
    int i = 0;
    while (i < f.count && f.interned[i] != name) ++i;  // names in source code are interned too
    for (int k = 0; i == f.count && k < f.count; ++k)
      if (PyUnicode_Compare(f.interned[k], name) == 0) {
        i = k;
        break;
      }
    if (i == f.count) fail(PyExc_TypeError, "%s() got an unexpected keyword argument %R", f.name, name);
    if (to[i] != nullptr) fail(PyExc_TypeError, "%s() got multiple values for argument %R", f.name, name);
    to[i] = args[count + j];
  }
  for (int i = 0; i < f.count; ++i)
    if (to[i] == nullptr) {
      if (i < f.required) fail(PyExc_TypeError, "%s() missing argument '%s'", f.name, f.names[i]);
      to[i] = f.defaults[i] != nullptr ? f.defaults[i] : Py_None;
    }
}

// A GPU made the current one for a scope (-1: none); where it is that already, one query.
class Current {
 public:
  explicit Current(c10::DeviceIndex device) {
    c10::DeviceIndex now = 0;
    if (device < 0) return;
    C10_HIP_CHECK(c10::hip::GetDevice(&now));
    if (now == device) return;
    C10_HIP_CHECK(c10::hip::SetDevice(device));
    was_ = now;
  }
  ~Current() {
    if (was_ >= 0) C10_HIP_CHECK_WARN(c10::hip::SetDevice(was_));
  }
  Current(const Current&) = delete;
  Current& operator=(const Current&) = delete;

 private:
  c10::DeviceIndex was_ = -1;
};

// No C++ exception leaves a function: what torch throws becomes the Python error that torch's
// own functions raise for it (no memory left: torch.OutOfMemoryError).  The first argument's GPU
// is the current one for the call (the default stream's handle is the same on all of them, and a
// launch on it goes to the current one); its other tensors have to be there too.
template <Function& F>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count, PyObject* names) {
  try {
    PyObject* a[kMost];
    place(F, args, count, names, a);
    const bool gpu = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).is_cuda();
    const Current on(gpu ? THPVariable_Unpack(a[0]).device().index() : (c10::DeviceIndex)-1);
    return F.call(a);
  } catch (const Failed&) {
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <Function& F>
PyMethodDef method(const char* doc) {
  return PyMethodDef{F.name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)),
                     METH_FASTCALL | METH_KEYWORDS, doc};
}

PyMethodDef g_methods[] = {
    method<g_quant>(R"(quant_mxfp4(x, out=None, scales=None)
--

bf16 [rows, cols] (cols % 128 == 0) -> MXFP4 (codes uint8 [rows, cols/2], scales uint8
[rows * cols/32] in storage order, see mxfp4_scale_index).)"),
    method<g_dequant>(R"(dequant_mxfp4(codes, scales, out=None)
--

The bf16 values [rows, cols] that MXFP4 codes and scales stand for (exact).)"),
    method<g_gemm>(R"(gemm_mxfp4(x_codes, x_scales, w_codes, w_scales, out=None)
--

Y = X . W^T of MXFP4 operands X [m, k] and W [n, k] (codes and scales of each); bf16 [m, n].)"),
    method<g_gated>(R"(gated_mxfp4(x_codes, x_scales, w_codes, w_scales, quantise=False, out=None, out_scales=None)
--

silu(X Wg^T) * (X Wu^T) of MXFP4 operands, W = [f gate rows; f up rows]: bf16 [m, f], or with
quantise=True (f % 128 == 0) MXFP4 (codes, scales), the X of the next gemm_mxfp4.)"),
    method<g_rmsnorm>(R"(rmsnorm(x, weight, kind=0, residual=None, eps=1e-06, group=128, out=None, scales=None, residual_out=None)
--

RMS norm of the rows of x (+ residual) in the form the next product reads: (out, scales,
residual_out), scales None for NORM_BF16 (the default kind) and residual_out (bf16 of x +
residual; may be `residual` itself) None without a residual.

NORM_BF16 bf16 [m, k]; NORM_FP8_ROWS / NORM_INT8_ROWS codes [m, k] (uint8 or float8_e4m3fn / int8)
and scales fp32 [m]; NORM_FP8_GROUPS scales fp32 [m, k/group]; NORM_MXFP4 codes uint8 [m, k/2] and
scales uint8 [m * k/32] in storage order.)"),
    method<g_ffn>(R"(ffn_mxfp4(x, weight, gu_codes, gu_scales, down_codes, down_scales, residual=None, eps=1e-06, out=None, residual_out=None, ws=None)
--

A pre-norm feed-forward block in MXFP4: y = down(silu(gate(v)) * up(v)), v the RMS norm of
x (+ residual) under `weight`; gate_up W [2 f, d] (gate rows first) and down W [d, f] as MXFP4
codes and scales.  Returns (y bf16 [m, d], residual_out or None); bit for bit rmsnorm(NORM_MXFP4),
gated_mxfp4(quantise=True) and gemm_mxfp4 in turn.)"),
    method<g_quant4>(R"(quant_int4(w, group=128, zeros=False, out=None, scales_out=None, zeros_out=None)
--

bf16 [rows, cols] (cols % group == 0, group 32, 64 or 128) -> integer 4-bit (codes uint8 [rows,
cols/2], scales bf16 [rows, cols/group], zeros uint8 [rows, cols/group] or None): values (q - z) s,
symmetric around 8 or, with zeros=True, between a group's least and largest.  pack_int4 puts codes
from elsewhere into this order.)"),
    method<g_dequant4>(R"(dequant_int4(codes, scales, zeros=None, out=None)
--

The bf16 values [rows, cols] that integer 4-bit codes, scales and zero points stand for.)"),
    method<g_gemm4>(R"(gemm_int4(x, codes, scales, zeros=None, out=None, ws=None)
--

Y = X . W^T, X bf16 [m, k], W [n, k] in integer 4-bit with group scales; bf16 [m, n].)"),
    method<g_route>(R"(route(logits, top, kind=0, bias=None, groups=1, top_groups=1, group_best=1, renormalise=True, factor=1.0, ids=None, weights=None)
--

The experts of each token and their weights: (ids int32 [tokens, top], weights fp32 [tokens, top]),
the best first, from logits bf16 or fp32 [tokens, experts].

Scores are the softmax (ROUTE_SOFTMAX, the default kind) or the sigmoid (ROUTE_SIGMOID) of the
logits; `bias` (fp32 [experts]) is added for the choice alone.  groups > 1: only experts of the
top_groups groups whose group_best best experts sum to most.  renormalise: the chosen scores are
divided by their sum.  Weights are times factor.  Ties go to the lower index; -inf or NaN masks an expert: it comes last,
with weight 0.)"),
    method<g_experts>(R"(experts_int4(x, ids, weights, gu_codes, gu_scales, down_codes, down_scales, gu_zeros=None, down_zeros=None, out=None, ws=None)
--

The feed-forward block of experts over integer 4-bit weights: y[t] = sum over j of weights[t, j] *
down_e(silu(gate_e(x[t])) * up_e(x[t])), e = ids[t, j]; bf16 [tokens, d].  gate_up W [experts, 2 f, d]
(gate rows first) and down W [experts, d, f] as codes and scales (and zeros) of quant_int4 with the
experts stacked.  An id outside the experts adds nothing.)"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_sp24", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

// The strings and the defaults that are not None; they live as long as the process.
bool intern(Function& f) {
  for (int i = 0; i < f.count; ++i)
    if ((f.interned[i] = PyUnicode_InternFromString(f.names[i])) == nullptr) return false;
  return true;
}
bool prepare() {
  for (Function* f : {&g_quant, &g_dequant, &g_gemm, &g_gated, &g_rmsnorm, &g_ffn, &g_quant4, &g_dequant4, &g_gemm4,
                      &g_route, &g_experts})
    if (!intern(*f)) return false;
  PyObject* const eps = PyFloat_FromDouble(1e-6);
  g_gated.defaults[4] = Py_False;
  g_rmsnorm.defaults[2] = PyLong_FromLong(SP24_NORM_BF16);
  g_rmsnorm.defaults[5] = PyLong_FromLong(128);
  g_rmsnorm.defaults[4] = g_ffn.defaults[7] = eps;
  g_quant4.defaults[1] = PyLong_FromLong(128);
  g_quant4.defaults[2] = Py_False;
  PyObject* const one = PyLong_FromLong(1);
  g_route.defaults[2] = PyLong_FromLong(SP24_ROUTE_SOFTMAX);
  g_route.defaults[4] = g_route.defaults[5] = g_route.defaults[6] = one;
  g_route.defaults[7] = Py_True;
  g_route.defaults[8] = PyFloat_FromDouble(1.0);
  return eps != nullptr && g_rmsnorm.defaults[2] != nullptr && g_rmsnorm.defaults[5] != nullptr &&
         g_quant4.defaults[1] != nullptr && one != nullptr && g_route.defaults[2] != nullptr &&
         g_route.defaults[8] != nullptr;
}

}  // namespace

PyMODINIT_FUNC PyInit__sp24() {
  PyObject* const m = prepare() ? PyModule_Create(&g_module) : nullptr;
  // for the package to compare: another PyTorch's tensors may be laid out otherwise
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
