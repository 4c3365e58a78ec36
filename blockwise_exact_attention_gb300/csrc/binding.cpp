// Python binding of the calls whose own run time is of the order of the
// interpreter's: the rotary embedding and the paged K/V cache.
//
// Argument marshalling only, like the ctypes binding of the other calls: torch
// tensors are described to libbea.so's C entry points by pointer, dtype, shape
// and strides, outputs that are not given are allocated, a status code becomes
// the package's error. Described from C++, a call costs the host 2.3 us
// (paged_write), 4.7 (paged_decode), 5.7 (paged_plan) and 5.9 (rope_axes), 2.7-3.7
// us where its outputs are given, instead of 12-25 us, and the rotation's gradient is a C++ node, so that a
// backward pass does not enter the interpreter.
#include <Python.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include "../../include/bea.h"

namespace {

using at::Tensor;
using torch::autograd::Node;
using torch::autograd::variable_list;

PyObject* g_check = nullptr;  // _lib.check(code, where): raises BeaError
std::atomic<long long> g_launches{0};  // kernels launched through here since the last reset

// The tensors of one call, described; all on the current device.
class Call {
 public:
  const bea_tensor* add(const Tensor& t) {
    if (!t.defined()) return nullptr;
    TORCH_CHECK_VALUE(t.is_cuda(), "tensors must live on a CUDA device");
    TORCH_CHECK_VALUE(!t.is_neg(), "a tensor whose negation is pending (torch.resolve_neg carries it out)");
    const int dev = t.get_device();
    if (n_ == 0) dev_ = dev;
    TORCH_CHECK_VALUE(dev == dev_, "tensors on cuda:", dev_, " and cuda:", dev, ": all must live on one device");
    bea_tensor& r = records_[n_++];
    switch (t.scalar_type()) {
      case at::kBFloat16: r.dtype = BEA_BF16; break;
      case at::kFloat: r.dtype = BEA_F32; break;
      case at::kInt: r.dtype = BEA_I32; break;
      default: TORCH_CHECK_TYPE(false, "unsupported dtype ", c10::toString(t.scalar_type()));
    }
    r.data = t.data_ptr();
    const auto shape = t.sizes(), stride = t.strides();
    r.ndim = static_cast<int32_t>(shape.size());
    for (size_t i = 0; i < 4; ++i) {
      r.shape[i] = i < shape.size() ? shape[i] : 0;
      r.stride[i] = i < shape.size() ? stride[i] : 0;
    }
    return &r;
  }
  // The current stream of the tensors' device, which has to be the current one.
  void* stream() const {
    const int now = c10::cuda::current_device();
    TORCH_CHECK_VALUE(dev_ == now, "tensors on cuda:", dev_, ", the current device is cuda:", now);
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_)).stream();
  }

 private:
  bea_tensor records_[12];
  int n_ = 0, dev_ = -1;
};

// A Python argument as a tensor; None is the undefined tensor where allowed.
Tensor tensor(PyObject* o, bool or_none = false) {
  if (or_none && o == Py_None) return Tensor();
  TORCH_CHECK_TYPE(THPVariable_Check(o), "a tensor is expected, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// A tensor that the caller gives to be written: autograd may not be recording it, and learns that it changed.
Tensor to_write(const Tensor& t) {
  TORCH_CHECK_VALUE(!t.defined() || !(at::GradMode::is_enabled() && t.requires_grad()),
                    "a tensor to be written requires grad: detach it, or call under torch.no_grad()");
  return t;
}
void written(std::initializer_list<Tensor> ts) {
  for (const Tensor& t : ts)
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int clamp_int(long long v) {  // out of int's range either way: refused by the library, or without effect there
  return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : static_cast<int>(v);
}

void arguments(const char* name, Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, name, ": ", got, " arguments, ", want, " expected");
}

int counted(int rc) {
  if (rc == BEA_OK) g_launches += bea_last_launch_count();
  return rc;
}

// What every call ends with, back in Python.
void finish(int rc, const char* where) {
  if (rc == BEA_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", rc, where);
  if (r == nullptr) throw python_error();
  Py_DECREF(r);
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (out == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(out, i++, wrap(t));
  return out;
}

// ---- rotary ----------------------------------------------------------------------

// A new tensor on the device of a tensor of the call, past the dispatcher (0.8 instead of 1.6 us).
Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& beside) {
  TORCH_CHECK_VALUE(beside.is_cuda(), "tensors must live on a CUDA device");
  return at::detail::empty_cuda(shape, dtype, beside.device(), std::nullopt);
}

struct Turn {
  std::vector<int32_t> axis;  // of every pair
  std::vector<double> freq;
  bool inverse = false;
};

Tensor like(const Tensor& x) { return x.defined() ? empty(x.sizes(), x.scalar_type(), x) : Tensor(); }

int rope(const Tensor& q, const Tensor& k, const Tensor& positions, const Turn& turn, const Tensor& q_out,
         const Tensor& k_out) {
  Call c;
  const bea_tensor *a = c.add(q), *b = c.add(k), *p = c.add(positions), *x = c.add(q_out), *y = c.add(k_out);
  return counted(
      bea_rope_axes(a, b, p, turn.axis.data(), turn.freq.data(), turn.inverse ? 1 : 0, x, y, c.stream()));
}

std::pair<Tensor, Tensor> rotary(const Tensor& q, const Tensor& k, const Tensor& positions, Turn turn, int* rc);

// A gradient that autograd hands over may be of another dtype, expanded, not aligned or yet to be negated.
Tensor ready(const Tensor& g, at::ScalarType dtype) {
  Tensor x = (g.scalar_type() == dtype ? g : g.to(dtype)).resolve_neg();
  bool fits = reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0 && x.stride(-1) == 1;
  for (int64_t i = 0; i + 1 < x.dim(); ++i) fits = fits && x.stride(i) * x.element_size() % 16 == 0;
  return fits ? x : x.clone(at::MemoryFormat::Contiguous);
}

// The gradient of a rotation: the gradients of (q_out, k_out) turned back.
struct RotaryBackward : public Node {
  torch::autograd::SavedVariable positions;
  Turn turn;
  at::ScalarType dtype = at::kFloat;

  std::string name() const override { return "RotaryAxesBackward"; }
  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    positions.reset_data();
  }

  variable_list apply(variable_list&& grads) override {
    variable_list out(num_outputs());  // q's, and k's where there is one
    Tensor g[2];
    for (uint32_t i = 0; i < num_outputs(); ++i)
      if (grads[i].defined() && task_should_compute_output(i)) g[i] = ready(grads[i], dtype);
    if (!g[0].defined() && !g[1].defined()) return out;
    Turn back = turn;
    back.inverse = !turn.inverse;
    Tensor at;
    {
      std::lock_guard<std::mutex> lock(mutex_);
      at = positions.unpack();
    }
    const bool first = g[0].defined();
    int rc = 0;
    const auto r = rotary(first ? g[0] : g[1], first ? g[1] : Tensor(), at, std::move(back), &rc);
    if (rc != BEA_OK) throw std::runtime_error(std::string("rotary_axes, backward: ") + bea_status_string(rc));
    out[first ? 0 : 1] = r.first;
    if (first && out.size() > 1) out[1] = r.second;
    return out;
  }
};

// A leaf's accumulation node is shared by all graphs that live on the leaf, and keeps the stream that was current
// when it was made. If that is the legacy default stream, a backward pass captured on another stream makes autograd
// wait there in the middle of the capture, which ends the process: the call is refused before that.
void check_capture(const Tensor& x, const char* name) {
  if (!x.defined() || !x.requires_grad() || !x.is_leaf()) return;
  const auto node = torch::autograd::impl::try_get_grad_accumulator(x);
  if (node == nullptr) return;
  const auto made = node->stream();
  if (made.has_value() && c10::cuda::CUDAStream(*made).stream() == nullptr)
    throw std::runtime_error(
        std::string(name) +
        ": captured into a CUDA graph while an earlier graph of the same leaf tensor, made on the default "
        "stream, is alive; delete its outputs before the capture");
}

std::pair<Tensor, Tensor> rotary(const Tensor& q, const Tensor& k, const Tensor& positions, Turn turn, int* rc) {
  for (const Tensor* t : {&q, &k})
    TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(0).defined(), "rotary_axes has no forward-mode derivative");
  const bool grad = at::GradMode::is_enabled() && (q.requires_grad() || (k.defined() && k.requires_grad()));
  if (grad) {
    if (q.is_cuda() && c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
      check_capture(q, "rotary_axes");
      check_capture(k, "rotary_axes");
    }
  }
  Tensor qo = like(q), ko = like(k);
  *rc = rope(q, k, positions, turn, qo, ko);
  if (*rc == BEA_OK && grad) {
    auto node = std::shared_ptr<RotaryBackward>(new RotaryBackward(), torch::autograd::deleteNode);
    node->set_next_edges(k.defined() ? torch::autograd::collect_next_edges(q, k) : torch::autograd::collect_next_edges(q));
    node->positions = torch::autograd::SavedVariable(positions, false);
    node->dtype = q.scalar_type();
    node->turn = std::move(turn);
    torch::autograd::set_history(qo, node);
    if (k.defined()) torch::autograd::set_history(ko, node);
  }
  return {qo, ko};
}

// The tables as Python hands them over: bytes of int32 and of double, one entry a pair; and the number of axes, which
// positions have to be of.
Turn turn_of(PyObject* table, const Tensor& q, const Tensor& positions) {
  TORCH_CHECK_TYPE(PyTuple_Check(table) && PyTuple_GET_SIZE(table) == 3, "the rotation's tables");
  PyObject *axis = PyTuple_GET_ITEM(table, 0), *freq = PyTuple_GET_ITEM(table, 1);
  const long long axes = integer(PyTuple_GET_ITEM(table, 2));
  TORCH_CHECK_VALUE(positions.dim() == 3 && positions.size(0) == axes, "positions ", positions.sizes(), ": [", axes,
                    ", n, l] for ", axes, " sections");
  TORCH_CHECK_TYPE(PyBytes_Check(axis) && PyBytes_Check(freq) && PyBytes_GET_SIZE(axis) * 2 == PyBytes_GET_SIZE(freq),
                   "the rotation's tables");
  const auto* a = reinterpret_cast<const int32_t*>(PyBytes_AS_STRING(axis));
  const auto* f = reinterpret_cast<const double*>(PyBytes_AS_STRING(freq));
  const size_t n = PyBytes_GET_SIZE(axis) / 4;
  TORCH_CHECK_VALUE(q.dim() > 0 && static_cast<size_t>(q.size(-1) / 2) == n, "the rotation's tables are not of d / 2 pairs");
  Turn t;
  t.axis.assign(a, a + n);
  t.freq.assign(f, f + n);
  return t;
}

// rope_axes(q, k, positions, table, inverse, q_out, k_out) -> (q_out, k_out)
PyObject* py_rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("rope_axes", n, 7);
  const Tensor q = tensor(a[0]), k = tensor(a[1], true), pos = tensor(a[2]);
  Tensor qo = to_write(tensor(a[5], true)), ko = to_write(tensor(a[6], true));
  Turn turn = turn_of(a[3], q, pos);
  turn.inverse = integer(a[4]) != 0;
  if (!qo.defined()) qo = like(q);
  if (!ko.defined()) ko = like(k);
  finish(rope(q, k, pos, turn, qo, ko), "rope_axes");
  written({qo, ko});
  return tuple({qo, ko});
  END_HANDLE_TH_ERRORS
}

// rotary_axes(q, k, positions, table) -> (q_out, k_out)
PyObject* py_rotary_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("rotary_axes", n, 4);
  const Tensor q = tensor(a[0]), k = tensor(a[1], true), pos = tensor(a[2]);
  int rc = 0;
  const auto out = rotary(q, k, pos, turn_of(a[3], q, pos), &rc);
  finish(rc, "rotary_axes");
  return tuple({out.first, out.second});
  END_HANDLE_TH_ERRORS
}

// ---- rotary with other layouts, and norms ------------------------------------------

struct Layout {
  Turn turn;
  bool interleaved = false, norm = false;
  float amplitude = 1.f, eps = 0.f;
  int pairs() const { return static_cast<int>(turn.axis.size()); }
};

int norm_rope(const Tensor& q, const Tensor& k, const Tensor& positions, const Layout& how, const Tensor& qw,
              const Tensor& kw, const Tensor& q_out, const Tensor& k_out) {
  Call c;
  const bea_tensor *a = c.add(q), *b = c.add(k), *p = c.add(positions), *u = c.add(qw), *v = c.add(kw), *x = c.add(q_out),
                   *y = c.add(k_out);
  return counted(bea_norm_rope_axes(a, b, p, how.turn.axis.data(), how.turn.freq.data(), how.pairs(), how.interleaved,
                                    how.amplitude, how.turn.inverse ? 1 : 0, u, v, how.norm, how.eps, x, y, c.stream()));
}

std::pair<Tensor, Tensor> norm_rotary(const Tensor& q, const Tensor& k, const Tensor& positions, Layout how,
                                      const Tensor& qw, const Tensor& kw, int* rc);

// The gradients of q, k and their weights; without the norm that of a rotation: its adjoint.
struct NormRotaryBackward : public Node {
  torch::autograd::SavedVariable positions, x[2], weight[2];  // x and weights: of the norm's gradient alone
  Layout how;
  bool has_k = false;
  at::ScalarType dtype = at::kFloat;

  std::string name() const override { return "NormRotaryAxesBackward"; }
  void release_variables() override {
    std::lock_guard<std::mutex> lock(mutex_);
    positions.reset_data();
    for (int i = 0; i < 2; ++i) x[i].reset_data(), weight[i].reset_data();
  }

  variable_list apply(variable_list&& grads) override {
    variable_list out(4);  // of q, k, q_weight, k_weight
    Tensor g[2], at, saved[2], w[2];
    bool wanted[2];
    for (uint32_t i = 0; i < 2; ++i) {
      wanted[i] = (i == 0 || has_k) && i < grads.size() && grads[i].defined() &&
                  (task_should_compute_output(i) || task_should_compute_output(2 + i));
      if (wanted[i]) g[i] = ready(grads[i], dtype);
    }
    if (!wanted[0] && !wanted[1]) return out;
    if (how.norm && at::GradMode::is_enabled())
      throw std::runtime_error("norm_rotary_axes has no second derivative (backward with create_graph)");
    {
      std::lock_guard<std::mutex> lock(mutex_);
      at = positions.unpack();
      for (int i = 0; how.norm && i < 2; ++i)
        if (wanted[i]) saved[i] = x[i].unpack(), w[i] = weight[i].unpack();
    }
    // what the library calls q is the first of the two that has a gradient
    const int first = wanted[0] ? 0 : 1, second = first == 0 && wanted[1] ? 1 : -1;
    int rc = 0;
    if (!how.norm) {
      Layout back = how;
      back.turn.inverse = !how.turn.inverse;
      const auto r = norm_rotary(g[first], second > 0 ? g[1] : Tensor(), at, std::move(back), Tensor(), Tensor(), &rc);
      out[first] = r.first;
      if (second > 0) out[1] = r.second;
    } else {
      Tensor dw[2], ws;
      for (int i = 0; i < 2; ++i) {
        if (!wanted[i]) continue;
        out[i] = like(saved[i]);
        if (w[i].defined() && task_should_compute_output(2 + i)) dw[i] = like(w[i]);
      }
      if (dw[0].defined() || dw[1].defined())
        ws = empty({static_cast<int64_t>(bea_norm_rope_axes_bwd_workspace_size(saved[first].size(-1)))}, at::kByte, at);
      Call c;
      const int f = first, z = 1;
      const bool two = second > 0;
      const bea_tensor *q = c.add(saved[f]), *k = two ? c.add(saved[z]) : nullptr, *gq = c.add(g[f]),
                       *gk = two ? c.add(g[z]) : nullptr, *p = c.add(at), *u = c.add(w[f]),
                       *v = two ? c.add(w[z]) : nullptr, *dq = c.add(out[f]), *dk = two ? c.add(out[z]) : nullptr,
                       *du = c.add(dw[f]), *dv = two ? c.add(dw[z]) : nullptr;
      rc = counted(bea_norm_rope_axes_bwd(q, k, gq, gk, p, how.turn.axis.data(), how.turn.freq.data(), how.pairs(),
                                          how.interleaved, how.amplitude, u, v, how.eps, dq, dk, du, dv,
                                          ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                                          c.stream()));
      for (int i = 0; i < 2; ++i) {
        out[2 + i] = dw[i];
        if (!task_should_compute_output(i)) out[i] = Tensor();
      }
    }
    if (rc != BEA_OK) throw std::runtime_error(std::string("norm_rotary_axes, backward: ") + bea_status_string(rc));
    return out;
  }
};

std::pair<Tensor, Tensor> norm_rotary(const Tensor& q, const Tensor& k, const Tensor& positions, Layout how,
                                      const Tensor& qw, const Tensor& kw, int* rc) {
  const char* name = how.norm ? "norm_rotary_axes" : "rotary_axes";
  bool grad = false;
  for (const Tensor* t : {&q, &k, &qw, &kw}) {
    if (!t->defined()) continue;
    TORCH_CHECK_NOT_IMPLEMENTED(!t->_fw_grad(0).defined(), name, " has no forward-mode derivative");
    grad = grad || t->requires_grad();
  }
  grad = grad && at::GradMode::is_enabled();
  if (grad && q.is_cuda() && c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    for (const Tensor* t : {&q, &k, &qw, &kw}) check_capture(*t, name);
  Tensor qo = like(q), ko = like(k);
  *rc = norm_rope(q, k, positions, how, qw, kw, qo, ko);
  if (*rc == BEA_OK && grad) {
    auto node = std::shared_ptr<NormRotaryBackward>(new NormRotaryBackward(), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(q, k, qw, kw));
    node->positions = torch::autograd::SavedVariable(positions, false);
    if (how.norm) {
      node->x[0] = torch::autograd::SavedVariable(q, false);
      node->x[1] = torch::autograd::SavedVariable(k, false);
      node->weight[0] = torch::autograd::SavedVariable(qw, false);
      node->weight[1] = torch::autograd::SavedVariable(kw, false);
    }
    node->has_k = k.defined();
    node->dtype = q.scalar_type();
    node->how = std::move(how);
    torch::autograd::set_history(qo, node);
    if (k.defined()) torch::autograd::set_history(ko, node);
  }
  return {qo, ko};
}

// (axes, frequencies, number of axes, amplitude, interleaved): the arrays' entries are the turned pairs.
Layout layout_of(PyObject* table, const Tensor& positions) {
  TORCH_CHECK_TYPE(PyTuple_Check(table) && PyTuple_GET_SIZE(table) == 5, "the rotation's tables");
  PyObject *axis = PyTuple_GET_ITEM(table, 0), *freq = PyTuple_GET_ITEM(table, 1);
  const long long axes = integer(PyTuple_GET_ITEM(table, 2));
  TORCH_CHECK_VALUE(positions.dim() == 3 && positions.size(0) == axes, "positions ", positions.sizes(), ": [", axes,
                    ", n, l] for ", axes, " sections");
  TORCH_CHECK_TYPE(PyBytes_Check(axis) && PyBytes_Check(freq) && PyBytes_GET_SIZE(axis) * 2 == PyBytes_GET_SIZE(freq),
                   "the rotation's tables");
  const auto* a = reinterpret_cast<const int32_t*>(PyBytes_AS_STRING(axis));
  const auto* f = reinterpret_cast<const double*>(PyBytes_AS_STRING(freq));
  const size_t n = PyBytes_GET_SIZE(axis) / 4;
  Layout how;
  how.turn.axis.assign(a, a + n);
  how.turn.freq.assign(f, f + n);
  how.amplitude = static_cast<float>(real(PyTuple_GET_ITEM(table, 3)));
  how.interleaved = integer(PyTuple_GET_ITEM(table, 4)) != 0;
  return how;
}

// norm_rope_axes(q, k, positions, table, inverse, q_weight, k_weight, norm, eps, q_out, k_out) -> (q_out, k_out)
PyObject* py_norm_rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("norm_rope_axes", n, 11);
  const Tensor q = tensor(a[0]), k = tensor(a[1], true), pos = tensor(a[2]);
  const Tensor qw = tensor(a[5], true), kw = tensor(a[6], true);
  Tensor qo = to_write(tensor(a[9], true)), ko = to_write(tensor(a[10], true));
  Layout how = layout_of(a[3], pos);
  how.turn.inverse = integer(a[4]) != 0;
  how.norm = integer(a[7]) != 0;
  how.eps = static_cast<float>(real(a[8]));
  if (!qo.defined()) qo = like(q);
  if (!ko.defined()) ko = like(k);
  finish(norm_rope(q, k, pos, how, qw, kw, qo, ko), how.norm ? "norm_rope_axes" : "rope_axes");
  written({qo, ko});
  return tuple({qo, ko});
  END_HANDLE_TH_ERRORS
}

// norm_rotary_axes(q, k, positions, table, q_weight, k_weight, norm, eps) -> (q_out, k_out)
PyObject* py_norm_rotary_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("norm_rotary_axes", n, 8);
  const Tensor q = tensor(a[0]), k = tensor(a[1], true), pos = tensor(a[2]);
  const Tensor qw = tensor(a[4], true), kw = tensor(a[5], true);
  Layout how = layout_of(a[3], pos);
  how.norm = integer(a[6]) != 0;
  how.eps = static_cast<float>(real(a[7]));
  const bool norm = how.norm;
  int rc = 0;
  const auto out = norm_rotary(q, k, pos, std::move(how), qw, kw, &rc);
  finish(rc, norm ? "norm_rotary_axes" : "rotary_axes");
  return tuple({out.first, out.second});
  END_HANDLE_TH_ERRORS
}

// ---- paged cache -----------------------------------------------------------------

// New int32 tensors of one call, as views of one allocation (0.3 us each instead of 1), each on a 16-byte boundary.
class Outputs {
 public:
  int count() const { return n_; }
  void want(Tensor* t, int64_t rows, int64_t cols = 0) {  // cols 0: of one dimension
    t_[n_] = t, rows_[n_] = rows, cols_[n_] = cols;
    ++n_;
  }
  void make(const Tensor& beside) {
    if (n_ == 0) return;
    int64_t total = 0, at = 0;
    for (int i = 0; i < n_; ++i) total += size(i);
    const Tensor all = empty({total}, at::kInt, beside);
    for (int i = 0; i < n_; ++i) {
      *t_[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
      const int64_t shape[2] = {rows_[i], cols_[i]}, stride[2] = {cols_[i] > 0 ? cols_[i] : 1, 1};
      const size_t dims = cols_[i] > 0 ? 2 : 1;
      t_[i]->unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(shape, dims), at::IntArrayRef(stride, dims), at);
      at += size(i);
    }
  }

 private:
  int64_t size(int i) const { return (rows_[i] * std::max<int64_t>(cols_[i], 1) + 3) / 4 * 4; }
  Tensor* t_[8];
  int64_t rows_[8], cols_[8];
  int n_ = 0;
};

// paged_plan(lens, new_lens, block_table, free_pages, n_free, page_size, capacity, out) -> out, a tuple of
// (slot_map, positions, cu_new, cu_pages, lens, n_free); out None: allocated
PyObject* py_paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_plan", n, 8);
  Tensor in[5], out[6];
  for (int i = 0; i < 5; ++i) in[i] = i == 2 || i == 3 ? to_write(tensor(a[i])) : tensor(a[i]);
  const long long page = integer(a[5]), capacity = integer(a[6]);
  if (a[7] != Py_None) {
    TORCH_CHECK_TYPE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 6, "paged_plan: out is a PagedPlan");
    for (int i = 0; i < 6; ++i) out[i] = to_write(tensor(PyTuple_GET_ITEM(a[7], i)));
    TORCH_CHECK_VALUE(out[0].dim() != 1 || out[0].size(0) == capacity, "paged_plan: out has ", out[0].size(0),
                      " places, capacity is ", capacity);
  } else {
    TORCH_CHECK_VALUE(capacity >= 0 && capacity <= INT32_MAX, "paged_plan: capacity ", capacity);
    const int64_t rows = in[0].dim() == 1 ? in[0].size(0) : 0;
    Outputs all;
    for (int64_t size : {capacity, static_cast<long long>(capacity), static_cast<long long>(rows + 1),
                         static_cast<long long>(rows + 1), static_cast<long long>(rows), 1ll})
      all.want(&out[all.count()], size);
    all.make(in[0]);
  }
  Call c;
  const bea_tensor* r[11];
  for (int i = 0; i < 5; ++i) r[i] = c.add(in[i]);
  for (int i = 0; i < 6; ++i) r[5 + i] = c.add(out[i]);
  finish(counted(bea_paged_plan(r[0], r[1], r[2], r[3], r[4], page, r[5], r[6], r[7], r[8], r[9], r[10], c.stream())),
         "paged_plan");
  written({in[2], in[3], out[0], out[1], out[2], out[3], out[4], out[5]});
  return tuple({out[0], out[1], out[2], out[3], out[4], out[5]});
  END_HANDLE_TH_ERRORS
}

// paged_write(k, v, slot_map, k_cache, v_cache) -> (k_cache, v_cache)
PyObject* py_paged_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_write", n, 5);
  Tensor t[5];
  Call c;
  const bea_tensor* r[5];
  for (int i = 0; i < 5; ++i) r[i] = c.add(t[i] = i >= 3 ? to_write(tensor(a[i])) : tensor(a[i]));
  finish(counted(bea_paged_write(r[0], r[1], r[2], r[3], r[4], c.stream())), "paged_write");
  written({t[3], t[4]});
  return PyTuple_Pack(2, a[3], a[4]);
  END_HANDLE_TH_ERRORS
}

// paged_decode(q, k_cache, v_cache, block_table, lens, scale, window_left, out, lse, f32_out, workspace) -> (out, lse)
PyObject* py_paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_decode", n, 11);
  Tensor t[5];
  for (int i = 0; i < 5; ++i) t[i] = tensor(a[i]);
  const Tensor &q = t[0], &kc = t[1], &table = t[3];
  TORCH_CHECK_VALUE(q.dim() == 4 && kc.dim() == 4 && table.dim() == 2,
                    "paged_decode: q [n, 1, h, d], caches [pages, page_size, h_kv, d], block_table [n, max_pages]");
  const float scale = static_cast<float>(real(a[5]));
  const int left = clamp_int(integer(a[6]));
  Tensor out = to_write(tensor(a[7], true)), lse = to_write(tensor(a[8], true)), ws = tensor(a[10], true);
  if (!out.defined()) out = empty(q.sizes(), integer(a[9]) != 0 ? at::kFloat : q.scalar_type(), q);
  if (!lse.defined()) lse = empty({q.size(0), q.size(2), 1}, at::kFloat, q);
  if (!ws.defined()) {
    const size_t need = bea_paged_decode_workspace_size(q.size(2), kc.size(2), q.size(3), table.size(1) * kc.size(1));
    if (need > 0) ws = empty({static_cast<int64_t>(need)}, at::kByte, q);
  }
  Call c;
  const bea_tensor* r[7];
  for (int i = 0; i < 5; ++i) r[i] = c.add(t[i]);
  r[5] = c.add(out);
  r[6] = c.add(lse);
  TORCH_CHECK_VALUE(!ws.defined() || (ws.is_cuda() && ws.get_device() == q.get_device() && ws.is_contiguous()),
                    "paged_decode: the workspace has to be contiguous and on the tensors' device");
  finish(counted(bea_paged_decode(r[0], r[1], r[2], r[3], r[4], r[5], r[6], scale, left,
                                  ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream())),
         "paged_decode");
  written({out, lse});
  return tuple({out, lse});
  END_HANDLE_TH_ERRORS
}

// paged_decode_shared(q, k_cache, v_cache, block_table, lens, group_rows, shared_lens, scale, out, lse, f32_out, workspace)
// -> (out, lse)
PyObject* py_paged_decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_decode_shared", n, 12);
  Tensor t[7];
  for (int i = 0; i < 7; ++i) t[i] = tensor(a[i]);
  const Tensor &q = t[0], &kc = t[1], &table = t[3];
  TORCH_CHECK_VALUE(q.dim() == 4 && kc.dim() == 4 && table.dim() == 2 && t[6].dim() == 1,
                    "paged_decode_shared: q [n, 1, h, d], caches [pages, page_size, h_kv, d], block_table [n, max_pages], "
                    "shared_lens [groups]");
  const float scale = static_cast<float>(real(a[7]));
  Tensor out = to_write(tensor(a[8], true)), lse = to_write(tensor(a[9], true)), ws = tensor(a[11], true);
  if (!out.defined()) out = empty(q.sizes(), integer(a[10]) != 0 ? at::kFloat : q.scalar_type(), q);
  if (!lse.defined()) lse = empty({q.size(0), q.size(2), 1}, at::kFloat, q);
  if (!ws.defined()) {
    const size_t need = bea_paged_decode_shared_workspace_size(q.size(0), q.size(2), kc.size(2), q.size(3),
                                                               table.size(1) * kc.size(1), t[6].size(0));
    if (need > 0) ws = empty({static_cast<int64_t>(need)}, at::kByte, q);
  }
  Call c;
  const bea_tensor* r[9];
  for (int i = 0; i < 7; ++i) r[i] = c.add(t[i]);
  r[7] = c.add(out);
  r[8] = c.add(lse);
  TORCH_CHECK_VALUE(!ws.defined() || (ws.is_cuda() && ws.get_device() == q.get_device() && ws.is_contiguous()),
                    "paged_decode_shared: the workspace has to be contiguous and on the tensors' device");
  finish(counted(bea_paged_decode_shared(r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], scale,
                                         ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, c.stream())),
         "paged_decode_shared");
  written({out, lse});
  return tuple({out, lse});
  END_HANDLE_TH_ERRORS
}

// ---- shared pages ------------------------------------------------------------------

// One of a call's outputs: given, or new and shaped like `x` (where that is a vector or a matrix; the library refuses it
// otherwise).
void output(PyObject* o, Tensor* t, const Tensor& x, Outputs* made) {
  *t = to_write(tensor(o, true));
  if (t->defined()) return;
  if (x.dim() == 2 && x.size(1) > 0)
    made->want(t, x.size(0), x.size(1));
  else if (x.dim() == 1)
    made->want(t, x.size(0));
  else
    *t = like(x);
}

// Records of several tensors, for the call that takes any number of them.
bea_tensor record_of(const Tensor& t) {
  Call c;
  return *c.add(t);
}

// paged_fork(src, tokens, lens, block_table, shares, free_pages, n_free, page_size, lens_out, n_free_out, shares_out,
// copies) -> (lens, n_free, shares, copies); outputs that are None are allocated
PyObject* py_paged_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_fork", n, 12);
  Tensor in[7];
  for (int i = 0; i < 7; ++i) in[i] = i == 3 ? to_write(tensor(a[i])) : tensor(a[i], i == 1);
  const long long page = integer(a[7]);
  Tensor lens, height, shares, copies = to_write(tensor(a[11], true));
  Outputs made;
  output(a[8], &lens, in[2], &made);
  output(a[9], &height, in[6], &made);
  output(a[10], &shares, in[4], &made);
  if (!copies.defined()) made.want(&copies, in[2].dim() == 1 ? in[2].size(0) : 0, 3);
  made.make(in[2]);
  Call c;
  const bea_tensor* r[11];
  for (int i = 0; i < 7; ++i) r[i] = c.add(in[i]);
  r[7] = c.add(lens), r[8] = c.add(height), r[9] = c.add(shares), r[10] = c.add(copies);
  finish(counted(bea_paged_fork(r[0], r[1], r[2], r[3], r[4], r[5], r[6], page, r[7], r[8], r[9], r[10], c.stream())),
         "paged_fork");
  written({in[3], lens, height, shares, copies});
  return tuple({lens, height, shares, copies});
  END_HANDLE_TH_ERRORS
}

// paged_free(ends, lens, block_table, shares, free_pages, n_free, page_size, lens_out, n_free_out, shares_out) -> (lens,
// n_free, shares)
PyObject* py_paged_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_free", n, 10);
  Tensor in[6];
  for (int i = 0; i < 6; ++i) in[i] = i == 4 ? to_write(tensor(a[i])) : tensor(a[i]);
  const long long page = integer(a[6]);
  Tensor lens, height, shares;
  Outputs made;
  output(a[7], &lens, in[1], &made);
  output(a[8], &height, in[5], &made);
  output(a[9], &shares, in[3], &made);
  made.make(in[1]);
  Call c;
  const bea_tensor* r[9];
  for (int i = 0; i < 6; ++i) r[i] = c.add(in[i]);
  r[6] = c.add(lens), r[7] = c.add(height), r[8] = c.add(shares);
  finish(counted(bea_paged_free(r[0], r[1], r[2], r[3], r[4], r[5], page, r[6], r[7], r[8], c.stream())), "paged_free");
  written({in[4], lens, height, shares});
  return tuple({lens, height, shares});
  END_HANDLE_TH_ERRORS
}

// paged_compact(lens, block_table, shares, free_pages, n_free, page_size, capacity, block_table_out, shares_out,
// free_pages_out, page_map, copies) -> (block_table, shares, free_pages, page_map, copies)
PyObject* py_paged_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_compact", n, 12);
  Tensor in[5];
  for (int i = 0; i < 5; ++i) in[i] = tensor(a[i]);
  const long long page = integer(a[5]), capacity = integer(a[6]);
  TORCH_CHECK_VALUE(capacity >= 0 && capacity <= INT32_MAX, "paged_compact: capacity ", capacity);
  Tensor table, shares, pool, map, copies = to_write(tensor(a[11], true));
  Outputs made;
  output(a[7], &table, in[1], &made);
  output(a[8], &shares, in[2], &made);
  output(a[9], &pool, in[3], &made);
  output(a[10], &map, in[2], &made);
  if (!copies.defined()) made.want(&copies, capacity, 3);
  made.make(in[0]);
  TORCH_CHECK_VALUE(copies.dim() != 2 || copies.size(0) == capacity, "paged_compact: copies has ", copies.size(0),
                    " places, capacity is ", capacity);
  Call c;
  const bea_tensor* r[10];
  for (int i = 0; i < 5; ++i) r[i] = c.add(in[i]);
  r[5] = c.add(table), r[6] = c.add(shares), r[7] = c.add(pool), r[8] = c.add(map), r[9] = c.add(copies);
  finish(counted(bea_paged_compact(r[0], r[1], r[2], r[3], r[4], page, r[5], r[6], r[7], r[8], r[9], c.stream())),
         "paged_compact");
  written({table, shares, pool, map, copies});
  return tuple({table, shares, pool, map, copies});
  END_HANDLE_TH_ERRORS
}

// paged_copy(copies, caches): a tuple or list of tensors, written
PyObject* py_paged_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("paged_copy", n, 2);
  const Tensor copies = tensor(a[0]);
  TORCH_CHECK_TYPE(PyTuple_Check(a[1]) || PyList_Check(a[1]), "paged_copy: caches is a tuple or list of tensors");
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[1]);
  std::vector<Tensor> caches;
  std::vector<bea_tensor> records;
  Call c;
  const bea_tensor* list = c.add(copies);
  void* stream = c.stream();
  for (Py_ssize_t i = 0; i < count; ++i) {
    caches.push_back(to_write(tensor(PySequence_Fast_GET_ITEM(a[1], i))));
    TORCH_CHECK_VALUE(!caches.back().is_cuda() || caches.back().get_device() == copies.get_device(), "tensors on cuda:",
                      copies.get_device(), " and cuda:", caches.back().get_device(), ": all must live on one device");
    records.push_back(record_of(caches.back()));
  }
  finish(counted(bea_paged_copy(list, records.data(), clamp_int(count), stream)), "paged_copy");
  for (const Tensor& t : caches) written({t});
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// setup(check): the package's function that raises a status code
PyObject* py_setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("setup", n, 1);
  Py_INCREF(a[0]);
  Py_XSETREF(g_check, a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// launches(reset) -> kernels launched since the last reset
PyObject* py_launches(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments("launches", n, 1);
  return PyLong_FromLongLong(integer(a[0]) != 0 ? g_launches.exchange(0) : g_launches.load());
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_setup>("setup"),
                           method<py_launches>("launches"),
                           method<py_rope_axes>("rope_axes"),
                           method<py_rotary_axes>("rotary_axes"),
                           method<py_norm_rope_axes>("norm_rope_axes"),
                           method<py_norm_rotary_axes>("norm_rotary_axes"),
                           method<py_paged_plan>("paged_plan"),
                           method<py_paged_write>("paged_write"),
                           method<py_paged_decode>("paged_decode"),
                           method<py_paged_decode_shared>("paged_decode_shared"),
                           method<py_paged_fork>("paged_fork"),
                           method<py_paged_free>("paged_free"),
                           method<py_paged_compact>("paged_compact"),
                           method<py_paged_copy>("paged_copy"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&g_module); }
