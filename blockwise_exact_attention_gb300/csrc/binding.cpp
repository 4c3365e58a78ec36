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

  // A gradient that autograd hands over may be of another dtype, expanded, not aligned or yet to be negated.
  Tensor ready(const Tensor& g) const {
    Tensor x = (g.scalar_type() == dtype ? g : g.to(dtype)).resolve_neg();
    bool fits = reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0 && x.stride(-1) == 1;
    for (int64_t i = 0; i + 1 < x.dim(); ++i) fits = fits && x.stride(i) * x.element_size() % 16 == 0;
    return fits ? x : x.clone(at::MemoryFormat::Contiguous);
  }

  variable_list apply(variable_list&& grads) override {
    variable_list out(num_outputs());  // q's, and k's where there is one
    Tensor g[2];
    for (uint32_t i = 0; i < num_outputs(); ++i)
      if (grads[i].defined() && task_should_compute_output(i)) g[i] = ready(grads[i]);
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
void check_capture(const Tensor& x) {
  if (!x.defined() || !x.requires_grad() || !x.is_leaf()) return;
  const auto node = torch::autograd::impl::try_get_grad_accumulator(x);
  if (node == nullptr) return;
  const auto made = node->stream();
  if (made.has_value() && c10::cuda::CUDAStream(*made).stream() == nullptr)
    throw std::runtime_error(
        "rotary_axes: captured into a CUDA graph while an earlier graph of the same leaf tensor, made on the default "
        "stream, is alive; delete its outputs before the capture");
}

std::pair<Tensor, Tensor> rotary(const Tensor& q, const Tensor& k, const Tensor& positions, Turn turn, int* rc) {
  for (const Tensor* t : {&q, &k})
    TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(0).defined(), "rotary_axes has no forward-mode derivative");
  const bool grad = at::GradMode::is_enabled() && (q.requires_grad() || (k.defined() && k.requires_grad()));
  if (grad) {
    if (q.is_cuda() && c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
      check_capture(q);
      check_capture(k);
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

// ---- paged cache -----------------------------------------------------------------

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
    const int64_t sizes[6] = {capacity, capacity, rows + 1, rows + 1, rows, 1};
    const int64_t one = 1;
    int64_t total = 0, at = 0;
    for (int64_t s : sizes) total += (s + 3) / 4 * 4;  // each on a 16-byte boundary
    const Tensor all = empty({total}, at::kInt, in[0]);
    for (int i = 0; i < 6; ++i) {  // views of one allocation
      out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
      out[i].unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(&sizes[i], 1), at::IntArrayRef(&one, 1), at);
      at += (sizes[i] + 3) / 4 * 4;
    }
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
                           method<py_paged_plan>("paged_plan"),
                           method<py_paged_write>("paged_write"),
                           method<py_paged_decode>("paged_decode"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&g_module); }
