// ar_marshal.cpp -- the argument checks of the block-boundary entry points for torch tensors, as a CPython module
// (all_reduce_reduction_ring_amd._marshal). The Python binding's own checks read five attributes of every tensor
// through the interpreter, 0.5 us each: with eight ranks a call spent 14 us on the host for 3.4 us of kernel.
//
// Every function takes the arguments of the Python entry point of its name in a fixed order and returns the ar_status of
// the call, or None if anything is not plainly as it should be (another type, device, shape or order, a tensor on a
// device that is not current, ...). Nothing was called then, and the binding goes through its own checks, which name
// what is wrong. A few things that those accept (a stream object, numbers that are no int) come back as None too.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "ar.h"

namespace {

// Entry points of the loaded libar, and torch's own lookups of the current device and its stream, from bind().
decltype(&ar_allreduce_rmsnorm) g_rmsnorm;
decltype(&ar_allreduce_rmsnorm_bwd) g_rmsnorm_bwd;
decltype(&ar_expert_sort) g_sort;
decltype(&ar_expert_dispatch) g_dispatch;
decltype(&ar_expert_combine) g_combine;
decltype(&ar_expert_combine_bwd) g_combine_bwd;
decltype(&ar_expert_gated) g_gated;
decltype(&ar_expert_gated_bwd) g_gated_bwd;
decltype(&ar_expert_linear) g_linear;
decltype(&ar_expert_linear_bwd) g_linear_bwd;
decltype(&ar_grad_norm) g_grad_norm;
decltype(&ar_grad_clip) g_grad_clip;
PyObject* g_current_device;
PyObject* g_current_stream;

struct Misfit {};  // thrown where an argument does not plainly fit

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Misfit();
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || !t.is_cuda()) throw Misfit();
  return t;
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return AR_F32;
    case at::kBFloat16: return AR_BF16;
    case at::kHalf: return AR_F16;
    default: throw Misfit();
  }
}

// What the arguments of one call have in common: all tensors on the current device.
struct Call {
  int device;
  explicit Call(const at::Tensor& first) : device(static_cast<int>(first.get_device())) {}

  // The address of a contiguous tensor of a type and shape (cols < 0: one dimension).
  void* at_(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols = -1) const {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || t.get_device() != device || t.dim() != (cols < 0 ? 1 : 2) || t.size(0) != rows ||
        (cols >= 0 && t.size(1) != cols) || !t.is_contiguous())
      throw Misfit();
    return t.data_ptr();
  }
  void* opt(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols = -1) const {
    return o == Py_None ? nullptr : at_(o, type, rows, cols);
  }
  void* codes(PyObject* o, int64_t rows, int64_t cols) const {
    const at::ScalarType t = tensor(o).scalar_type();
    if (t != at::kByte && t != at::kFloat8_e4m3fn) throw Misfit();
    return at_(o, t, rows, cols);
  }
  void* workspace(PyObject* o, size_t* bytes) const {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.get_device() != device || !t.is_contiguous()) throw Misfit();
    *bytes = t.nbytes();
    return t.data_ptr();
  }
  // The stream: an int handle, or (None) the device's current one. The device has to be the current one.
  void* stream(PyObject* o) const {
    PyObject* cur = PyObject_CallNoArgs(g_current_device);
    const long now = cur ? PyLong_AsLong(cur) : -1;
    Py_XDECREF(cur);
    if (now != device || PyErr_Occurred()) throw Misfit();
    if (o != Py_None) return handle_of(o);
    PyObject* index = PyLong_FromLong(device);
    PyObject* handle = index ? PyObject_CallOneArg(g_current_stream, index) : nullptr;
    Py_XDECREF(index);
    const uint64_t s = handle ? PyLong_AsUnsignedLongLong(handle) : kNoHandle;
    Py_XDECREF(handle);
    if (s == kNoHandle) throw Misfit();
    return reinterpret_cast<void*>(s);
  }
  // An int as a handle. What the conversion refuses (negative, past 64 bits) must not become the null stream.
  static void* handle_of(PyObject* o) {
    const uint64_t s = PyLong_Check(o) ? PyLong_AsUnsignedLongLong(o) : kNoHandle;
    if (s == kNoHandle) throw Misfit();
    return reinterpret_cast<void*>(s);
  }
  static constexpr uint64_t kNoHandle = UINT64_MAX;  // what the conversion returns with an error set
};

// A list or tuple of one tensor per rank.
struct Ranks {
  PyObject* const* items;
  int n;
  explicit Ranks(PyObject* o) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) throw Misfit();
    const Py_ssize_t size = PySequence_Fast_GET_SIZE(o);
    if (size < 1 || size > AR_MAX_RANKS) throw Misfit();
    items = PySequence_Fast_ITEMS(o);
    n = static_cast<int>(size);
  }
};

const at::Tensor& matrix(PyObject* o) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 2) throw Misfit();
  return t;
}

int64_t blocks_of(int64_t hidden) { return (hidden + AR_FP8_BLOCK - 1) / AR_FP8_BLOCK; }

at::ScalarType gamma_type(PyObject* o, at::ScalarType rows) {
  const at::ScalarType t = tensor(o).scalar_type();
  if (t != rows && t != at::kFloat) throw Misfit();
  return t;
}

int rmsnorm(PyObject* const* a) {  // ins gamma outs residual residual_out rstd out_scales saved saved_scales eps stream
  const Ranks ins(a[0]), outs(a[2]);
  const at::Tensor& x = matrix(ins.items[0]);
  const at::ScalarType type = x.scalar_type();
  const int dtype = code_of(type);
  const int64_t rows = x.size(0), hidden = x.size(1), nb = blocks_of(hidden);
  const Call c(x);
  const bool out8 = a[6] != Py_None;
  if (outs.n != ins.n) throw Misfit();
  const void* in[AR_MAX_RANKS];
  void* out[AR_MAX_RANKS];
  float* scales[AR_MAX_RANKS];
  for (int r = 0; r < ins.n; ++r) {
    in[r] = c.at_(ins.items[r], type, rows, hidden);
    out[r] = out8 ? c.codes(outs.items[r], rows, hidden) : c.at_(outs.items[r], type, rows, hidden);
  }
  if (out8) {
    const Ranks sc(a[6]);
    if (sc.n != ins.n) throw Misfit();
    for (int r = 0; r < sc.n; ++r) scales[r] = static_cast<float*>(c.at_(sc.items[r], at::kFloat, rows, nb));
  }
  const at::ScalarType gt = gamma_type(a[1], type);
  void* gamma = c.at_(a[1], gt, hidden);
  void* residual = c.opt(a[3], type, rows, hidden);
  void* residual_out = c.opt(a[4], type, rows, hidden);
  float* rstd = static_cast<float*>(c.opt(a[5], at::kFloat, rows));
  uint8_t* saved = a[7] == Py_None ? nullptr : static_cast<uint8_t*>(c.codes(a[7], rows, hidden));
  float* saved_scales = static_cast<float*>(c.opt(a[8], at::kFloat, rows, nb));
  const double eps = PyFloat_AsDouble(a[9]);
  if (eps == -1.0 && PyErr_Occurred()) throw Misfit();
  void* s = c.stream(a[10]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_rmsnorm(in, ins.n, rows, hidden, dtype, residual, gamma, code_of(gt), static_cast<float>(eps), out,
                 out8 ? scales : nullptr, residual_out, rstd, saved, saved_scales, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int rmsnorm_bwd(PyObject* const* a) {  // ins saved gamma rstd outs dgamma saved_scales residual_grad workspace stream
  const Ranks ins(a[0]), outs(a[4]);
  const at::Tensor& x = matrix(ins.items[0]);
  const at::ScalarType type = x.scalar_type();
  const int dtype = code_of(type);
  const int64_t rows = x.size(0), hidden = x.size(1);
  const Call c(x);
  if (outs.n != ins.n) throw Misfit();
  const void* in[AR_MAX_RANKS];
  void* out[AR_MAX_RANKS];
  for (int r = 0; r < ins.n; ++r) {
    in[r] = c.at_(ins.items[r], type, rows, hidden);
    out[r] = c.at_(outs.items[r], type, rows, hidden);
  }
  const float* scales = static_cast<float*>(c.opt(a[6], at::kFloat, rows, blocks_of(hidden)));
  const void* saved = scales ? c.codes(a[1], rows, hidden) : c.at_(a[1], type, rows, hidden);
  const at::ScalarType gt = gamma_type(a[2], type);
  const void* gamma = c.at_(a[2], gt, hidden);
  const float* rstd = static_cast<float*>(c.at_(a[3], at::kFloat, rows));
  float* dgamma = static_cast<float*>(c.at_(a[5], at::kFloat, hidden));
  const void* grad = c.opt(a[7], type, rows, hidden);
  size_t bytes;
  void* ws = c.workspace(a[8], &bytes);
  if (a[6] != Py_None && !scales) throw Misfit();  // an empty tensor: whether it was given is all that shows
  void* s = c.stream(a[9]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_rmsnorm_bwd(in, ins.n, rows, hidden, dtype, saved, scales, gamma, code_of(gt), rstd, grad, out, dgamma, ws,
                     bytes, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int expert_sort(PyObject* const* a) {  // ids offsets counts pos src align workspace stream
  const at::Tensor& ids = matrix(a[0]);
  const int64_t tokens = ids.size(0), k = ids.size(1), experts = tensor(a[2]).numel(), rows = tensor(a[4]).numel();
  const Call c(ids);
  const int32_t* in = static_cast<int32_t*>(c.at_(a[0], at::kInt, tokens, k));
  int32_t* offsets = static_cast<int32_t*>(c.at_(a[1], at::kInt, experts + 1));
  int32_t* counts = static_cast<int32_t*>(c.at_(a[2], at::kInt, experts));
  int32_t* pos = static_cast<int32_t*>(c.at_(a[3], at::kInt, tokens, k));
  int32_t* src = static_cast<int32_t*>(c.at_(a[4], at::kInt, rows));
  const long align = PyLong_Check(a[5]) ? PyLong_AsLong(a[5]) : -1;
  if (align < 1 || align > INT32_MAX || k > INT32_MAX || experts > INT32_MAX) throw Misfit();
  size_t bytes;
  void* ws = c.workspace(a[6], &bytes);
  void* s = c.stream(a[7]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_sort(in, tokens, static_cast<int>(k), static_cast<int>(experts), static_cast<int>(align), offsets, counts, pos,
              src, rows, ws, bytes, s);
  Py_END_ALLOW_THREADS
  return rc;
}

struct Pads {
  const int32_t *offsets = nullptr, *counts = nullptr;
  int experts = 1;
  Pads(const Call& c, PyObject* off, PyObject* cnt) {
    if ((off == Py_None) != (cnt == Py_None)) throw Misfit();
    if (off == Py_None) return;
    const int64_t n = tensor(cnt).numel();
    if (n > INT32_MAX) throw Misfit();
    experts = static_cast<int>(n);
    offsets = static_cast<int32_t*>(c.at_(off, at::kInt, n + 1));
    counts = static_cast<int32_t*>(c.at_(cnt, at::kInt, n));
  }
};

int expert_dispatch(PyObject* const* a) {  // x pos offsets counts xs x_scales xs_scales stream
  const at::Tensor &x = matrix(a[0]), &xs = matrix(a[4]), &pos = matrix(a[1]);
  const int64_t tokens = x.size(0), hidden = x.size(1), rows = xs.size(0), k = pos.size(1), nb = blocks_of(hidden);
  const Call c(x);
  const at::ScalarType type = x.scalar_type();
  if ((a[5] == Py_None) != (a[6] == Py_None) || k > INT32_MAX) throw Misfit();
  const bool rows8 = a[5] != Py_None;
  if (rows8 ? type != at::kByte && type != at::kFloat8_e4m3fn : code_of(type) < 0) throw Misfit();
  const void* from = c.at_(a[0], type, tokens, hidden);
  const float* from_scales = static_cast<float*>(c.opt(a[5], at::kFloat, tokens, nb));
  const int32_t* at = static_cast<int32_t*>(c.at_(a[1], at::kInt, tokens, k));
  const Pads pads(c, a[2], a[3]);
  void* to = c.at_(a[4], type, rows, hidden);
  float* to_scales = static_cast<float*>(c.opt(a[6], at::kFloat, rows, nb));
  if (rows8 && (!from_scales || !to_scales)) throw Misfit();
  const int size = static_cast<int>(x.element_size());
  void* s = c.stream(a[7]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_dispatch(from, from_scales, at, pads.offsets, pads.counts, tokens, static_cast<int>(k), pads.experts, hidden,
                  size, to, to_scales, rows, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int expert_combine(PyObject* const* a) {  // ys pos out weights addend stream
  const at::Tensor &ys = matrix(a[0]), &pos = matrix(a[1]), &out = matrix(a[2]);
  const int64_t tokens = out.size(0), hidden = out.size(1), rows = ys.size(0), k = pos.size(1);
  const Call c(out);
  const at::ScalarType type = out.scalar_type();
  const int dtype = code_of(type);
  if (k > INT32_MAX) throw Misfit();
  const void* from = c.at_(a[0], type, rows, hidden);
  const int32_t* at = static_cast<int32_t*>(c.at_(a[1], at::kInt, tokens, k));
  void* to = c.at_(a[2], type, tokens, hidden);
  const float* weights = static_cast<float*>(c.opt(a[3], at::kFloat, tokens, k));
  const void* addend = c.opt(a[4], type, tokens, hidden);
  void* s = c.stream(a[5]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_combine(from, at, weights, addend, tokens, static_cast<int>(k), hidden, dtype, rows, to, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int expert_combine_bwd(PyObject* const* a) {  // dout ys pos weights offsets counts dys dweights stream
  const at::Tensor &dout = matrix(a[0]), &ys = matrix(a[1]), &pos = matrix(a[2]);
  const int64_t tokens = dout.size(0), hidden = dout.size(1), rows = ys.size(0), k = pos.size(1);
  const Call c(dout);
  const at::ScalarType type = dout.scalar_type();
  const int dtype = code_of(type);
  if (k > INT32_MAX) throw Misfit();
  const void* grad = c.at_(a[0], type, tokens, hidden);
  const void* from = c.at_(a[1], type, rows, hidden);
  const int32_t* at = static_cast<int32_t*>(c.at_(a[2], at::kInt, tokens, k));
  const float* weights = static_cast<float*>(c.at_(a[3], at::kFloat, tokens, k));
  const Pads pads(c, a[4], a[5]);
  void* dys = c.at_(a[6], type, rows, hidden);
  float* dweights = static_cast<float*>(c.at_(a[7], at::kFloat, tokens, k));
  void* s = c.stream(a[8]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_combine_bwd(grad, from, at, weights, pads.offsets, pads.counts, tokens, static_cast<int>(k), pads.experts,
                     hidden, dtype, rows, dys, dweights, s);
  Py_END_ALLOW_THREADS
  return rc;
}

// The tables of the experts' segments: offsets and counts, offsets alone, or neither.
struct Segments {
  const int32_t *offsets = nullptr, *counts = nullptr;
  int experts = 1;
  Segments(const Call& c, PyObject* off, PyObject* cnt) {
    if (off == Py_None) {
      if (cnt != Py_None) throw Misfit();
      return;
    }
    const int64_t n = tensor(off).numel() - 1;
    if (n < 1 || n > AR_MAX_EXPERTS) throw Misfit();
    experts = static_cast<int>(n);
    offsets = static_cast<int32_t*>(c.at_(off, at::kInt, n + 1));
    if (cnt != Py_None) counts = static_cast<int32_t*>(c.at_(cnt, at::kInt, n));
  }
};

// A weight [experts][out][in] (without segments also [out][in]) of dense matrices, and the elements from one to the next.
struct Weight {
  void* p = nullptr;
  int64_t stride;
  Weight(const Call& c, PyObject* o, at::ScalarType type, const Segments& seg, int64_t out, int64_t in) : stride(out * in) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o);
    const int64_t d = t.dim() - 2;
    if (t.scalar_type() != type || t.get_device() != c.device || d > 1 || d < (seg.offsets ? 1 : 0) ||
        (d == 1 && t.size(0) != seg.experts) || t.size(d) != out || t.size(d + 1) != in || t.stride(d + 1) != 1 || t.stride(d) != in)
      throw Misfit();
    if (seg.experts > 1) stride = t.stride(0);
    p = t.data_ptr();
    if (!p) throw Misfit();
  }
};

int number(PyObject* o) {
  const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  if (v < 0 || v > INT32_MAX) throw Misfit();
  return static_cast<int>(v);
}

int expert_gated(PyObject* const* a) {  // xs w_gate w_up out offsets counts gate up act stream
  const at::Tensor &x = matrix(a[0]), &out = matrix(a[3]);
  const at::ScalarType type = x.scalar_type();
  const int dtype = code_of(type);
  const int64_t rows = x.size(0), hidden = x.size(1), inner = out.size(1);
  const Call c(x);
  const Segments seg(c, a[4], a[5]);
  const void* xs = c.at_(a[0], type, rows, hidden);
  const Weight g(c, a[1], type, seg, inner, hidden), u(c, a[2], type, seg, inner, hidden);
  if (g.stride != u.stride) throw Misfit();
  void* to = c.at_(a[3], type, rows, inner);
  void* gate = c.opt(a[6], type, rows, inner);
  void* up = c.opt(a[7], type, rows, inner);
  const int act = number(a[8]);
  void* s = c.stream(a[9]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_gated(xs, g.p, u.p, g.stride, seg.offsets, seg.counts, seg.experts, rows, hidden, inner, dtype, act, to, gate, up, s);
  Py_END_ALLOW_THREADS
  return rc;
}

// dout gate up xs w_gate w_up dgate dup dxs dw_gate dw_up offsets counts act stream; with xs or dxs, and both weights' gradients
// or neither (what else the binding takes goes through its own checks)
int expert_gated_bwd(PyObject* const* a) {
  const at::Tensor& d = matrix(a[0]);
  const at::ScalarType type = d.scalar_type();
  const int dtype = code_of(type);
  const bool weights = a[9] != Py_None, rows_too = a[8] != Py_None;
  if (weights != (a[10] != Py_None) || (!weights && !rows_too) || (weights && a[3] == Py_None)) throw Misfit();
  const at::Tensor& x = matrix(a[3] != Py_None ? a[3] : a[8]);
  const int64_t rows = d.size(0), inner = d.size(1), hidden = x.size(1);
  const Call c(d);
  const Segments seg(c, a[11], a[12]);
  const void* dout = c.at_(a[0], type, rows, inner);
  const void* gate = c.at_(a[1], type, rows, inner);
  const void* up = c.at_(a[2], type, rows, inner);
  const void* xs = c.opt(a[3], type, rows, hidden);
  PyObject* none = Py_None;
  const Weight g(c, rows_too ? a[4] : none, type, seg, inner, hidden), u(c, rows_too ? a[5] : none, type, seg, inner, hidden);
  if (rows_too && (!g.p || !u.p || g.stride != u.stride)) throw Misfit();
  void* dgate = c.at_(a[6], type, rows, inner);
  void* dup = c.at_(a[7], type, rows, inner);
  void* dxs = c.opt(a[8], type, rows, hidden);
  const Weight dg(c, a[9], type, seg, inner, hidden), du(c, a[10], type, seg, inner, hidden);
  if (dg.stride != du.stride) throw Misfit();
  const int act = number(a[13]);
  void* s = c.stream(a[14]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_gated_bwd(dout, gate, up, xs, g.p, u.p, g.stride, seg.offsets, seg.counts, seg.experts, rows, hidden, inner, dtype, act,
                   dgate, dup, dxs, dg.p, du.p, dg.stride, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int expert_linear(PyObject* const* a) {  // xs w out offsets counts stream
  const at::Tensor &x = matrix(a[0]), &out = matrix(a[2]);
  const at::ScalarType type = x.scalar_type();
  const int dtype = code_of(type);
  const int64_t rows = x.size(0), in = x.size(1), wide = out.size(1);
  const Call c(x);
  const Segments seg(c, a[3], a[4]);
  const void* xs = c.at_(a[0], type, rows, in);
  const Weight w(c, a[1], type, seg, wide, in);
  if (!w.p) throw Misfit();
  void* to = c.at_(a[2], type, rows, wide);
  void* s = c.stream(a[5]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_linear(xs, w.p, w.stride, seg.offsets, seg.counts, seg.experts, rows, in, wide, dtype, to, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int expert_linear_bwd(PyObject* const* a) {  // dout xs w dxs dw offsets counts stream
  const at::Tensor& d = matrix(a[0]);
  const at::ScalarType type = d.scalar_type();
  const int dtype = code_of(type);
  const bool rows_too = a[3] != Py_None;
  if ((!rows_too && a[4] == Py_None) || (a[4] != Py_None && a[1] == Py_None)) throw Misfit();
  const at::Tensor& x = matrix(rows_too ? a[3] : a[1]);
  const int64_t rows = d.size(0), wide = d.size(1), in = x.size(1);
  const Call c(d);
  const Segments seg(c, a[5], a[6]);
  const void* dys = c.at_(a[0], type, rows, wide);
  const void* xs = c.opt(a[1], type, rows, in);
  PyObject* none = Py_None;
  const Weight w(c, rows_too ? a[2] : none, type, seg, wide, in);
  if (rows_too && !w.p) throw Misfit();
  void* dxs = c.opt(a[3], type, rows, in);
  const Weight dw(c, a[4], type, seg, wide, in);
  void* s = c.stream(a[7]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_linear_bwd(dys, xs, w.p, w.stride, seg.offsets, seg.counts, seg.experts, rows, in, wide, dtype, dxs, dw.p, dw.stride, s);
  Py_END_ALLOW_THREADS
  return rc;
}

// A plan's pieces and the norm that they give.
struct Plan {
  const Call c;
  const ar_grad_piece* pieces;
  int64_t n;
  float* norm;
  void* ws;
  size_t bytes;
  Plan(PyObject* plan, PyObject* to, PyObject* workspace) : c(matrix(plan)), n(tensor(plan).size(0)) {
    pieces = static_cast<ar_grad_piece*>(c.at_(plan, at::kLong, n, sizeof(ar_grad_piece) / 8));
    const at::Tensor& t = tensor(to);
    if (t.scalar_type() != at::kFloat || t.get_device() != c.device || t.numel() != 1) throw Misfit();
    norm = static_cast<float*>(t.data_ptr());
    ws = c.workspace(workspace, &bytes);
  }
};

// A number, not what could be made one: a GPU tensor's value would be waited for.
float real(PyObject* o) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) throw Misfit();
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Misfit();
  return static_cast<float>(v);
}

int grad_norm(PyObject* const* a) {  // plan norm kind workspace stream
  const Plan p(a[0], a[1], a[3]);
  const int kind = number(a[2]);
  void* s = p.c.stream(a[4]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_grad_norm(p.pieces, p.n, kind, p.norm, p.ws, p.bytes, s);
  Py_END_ALLOW_THREADS
  return rc;
}

int grad_clip(PyObject* const* a) {  // plan max_norm norm kind eps workspace stream
  const Plan p(a[0], a[2], a[5]);
  const float most = real(a[1]), eps = real(a[4]);
  const int kind = number(a[3]);
  void* s = p.c.stream(a[6]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_grad_clip(p.pieces, p.n, kind, most, eps, p.norm, p.ws, p.bytes, s);
  Py_END_ALLOW_THREADS
  return rc;
}

// F with its N arguments; whatever is thrown becomes None.
template <int (*F)(PyObject* const*), int N> PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n == N && g_current_stream) {
    try {
      return PyLong_FromLong(F(args));
    } catch (...) {
    }
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// bind(addresses of the six entry points in the order above, current device's function, current stream's function)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses and two functions");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point's address is 0");
      return nullptr;
    }
  }
  g_rmsnorm = reinterpret_cast<decltype(g_rmsnorm)>(p[0]);
  g_rmsnorm_bwd = reinterpret_cast<decltype(g_rmsnorm_bwd)>(p[1]);
  g_sort = reinterpret_cast<decltype(g_sort)>(p[2]);
  g_dispatch = reinterpret_cast<decltype(g_dispatch)>(p[3]);
  g_combine = reinterpret_cast<decltype(g_combine)>(p[4]);
  g_combine_bwd = reinterpret_cast<decltype(g_combine_bwd)>(p[5]);
  Py_INCREF(args[6]);
  Py_INCREF(args[7]);
  Py_XDECREF(g_current_device);
  Py_XDECREF(g_current_stream);
  g_current_device = args[6];
  g_current_stream = args[7];
  Py_RETURN_NONE;
}

// bind_products(addresses of the six entry points behind those of bind, in the order above), before bind
PyObject* bind_products(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind_products takes six addresses");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point's address is 0");
      return nullptr;
    }
  }
  g_gated = reinterpret_cast<decltype(g_gated)>(p[0]);
  g_gated_bwd = reinterpret_cast<decltype(g_gated_bwd)>(p[1]);
  g_linear = reinterpret_cast<decltype(g_linear)>(p[2]);
  g_linear_bwd = reinterpret_cast<decltype(g_linear_bwd)>(p[3]);
  g_grad_norm = reinterpret_cast<decltype(g_grad_norm)>(p[4]);
  g_grad_clip = reinterpret_cast<decltype(g_grad_clip)>(p[5]);
  Py_RETURN_NONE;
}

#define AR_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<f, n>)), METH_FASTCALL, nullptr}
// The same once its entry point is bound.
template <int (*F)(PyObject* const*), int N, auto* G> PyObject* product(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (!*G) Py_RETURN_NONE;
  return entry<F, N>(self, args, n);
}
#define AR_PRODUCT(f, n, g) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(product<f, n, &g>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    AR_ENTRY(rmsnorm, 11), AR_ENTRY(rmsnorm_bwd, 10), AR_ENTRY(expert_sort, 8), AR_ENTRY(expert_dispatch, 8),
    AR_ENTRY(expert_combine, 6), AR_ENTRY(expert_combine_bwd, 9),
    {"bind_products", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind_products)), METH_FASTCALL, nullptr},
    AR_PRODUCT(expert_gated, 10, g_gated), AR_PRODUCT(expert_gated_bwd, 15, g_gated_bwd), AR_PRODUCT(expert_linear, 6, g_linear),
    AR_PRODUCT(expert_linear_bwd, 8, g_linear_bwd), AR_PRODUCT(grad_norm, 5, g_grad_norm), AR_PRODUCT(grad_clip, 7, g_grad_clip),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
