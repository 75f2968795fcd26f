// layers.cpp -- the layers around the linear ones (layer norm, dropout,
// embedding, loss over a vocabulary) as nodes of torch's autograd graph, on
// the library's entry points.  At the sizes of a small model a layer's kernels
// take a few microseconds; a node written in Python takes about 50 a pass,
// here a tenth of that.  A Python extension module (_layers); host code only,
// nothing is kept between calls but the list of living graphs' leaves.

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/grad_mode.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>
#include <torch/csrc/jit/frontend/tracer.h>

#include <initializer_list>
#include <memory>
#include <mutex>
#include <optional>
#include <stdexcept>
#include <string>
#include <unordered_map>
#include <vector>

#include "../../include/metis.h"

namespace {

using at::Tensor;
using torch::autograd::SavedVariable;
using torch::autograd::variable_list;

// The library's entry points (the binding has loaded it) and its error class.
struct Api {
  decltype(&metis_last_error) last_error;
  decltype(&metis_layernorm_fwd) norm_fwd;
  decltype(&metis_layernorm_bwd_workspace) norm_ws;
  decltype(&metis_layernorm_bwd) norm_bwd;
  decltype(&metis_dropout) dropout;
  decltype(&metis_embedding_fwd) embed_fwd;
  decltype(&metis_embedding_bwd_workspace) embed_ws;
  decltype(&metis_embedding_bwd) embed_bwd;
  decltype(&metis_cross_entropy_workspace) loss_ws;
  decltype(&metis_cross_entropy_fwd) loss_fwd;
  decltype(&metis_cross_entropy_bwd) loss_bwd;
} api;
PyObject* error_class = nullptr;   // MetisError(status, message)
PyObject* refuse_capture = nullptr;  // called with the leaves of a pass that a capture records

// A refused argument: becomes the Python exception of that type, or, in a
// backward pass, whose threads take standard exceptions only, a RuntimeError.
struct Refused : std::runtime_error {
  PyObject* type;
  Refused(PyObject* t, const std::string& what) : std::runtime_error(what), type(t) {}
};

[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refused(type, what); }

// An entry point's error.
struct Failed : std::runtime_error {
  int status;
  std::string text;
  Failed(int s, const std::string& what) : std::runtime_error("metis status " + std::to_string(s) + ": " + what), status(s), text(what) {}
};

void check(metis_status s) {
  if (s != METIS_OK) throw Failed(s, api.last_error());
}

int32_t float_type(const Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return METIS_BF16;
  if (t.scalar_type() == at::kFloat) return METIS_F32;
  refuse(PyExc_TypeError, std::string(what) + " must be bfloat16 or float32, got " + c10::toString(t.scalar_type()));
}

at::ScalarType scalar_type(int32_t dtype) { return dtype == METIS_BF16 ? at::kBFloat16 : at::kFloat; }

// A view whose values are negated when they are read ends up in memory: the
// kernels read memory.
Tensor plain(const Tensor& t) { return t.defined() && t.is_neg() ? t.resolve_neg() : t; }

// The last dimension's rows of a tensor as the library takes them; a copy
// where they do not lie so.
struct Rows {
  Tensor at;  // holds the memory
  int32_t dtype;
  int64_t rows, cols, ld;
  bool copied = false;

  void* data() const { return at.data_ptr(); }
};

Rows rows_of(const Tensor& x, const char* what) {
  const int32_t dtype = float_type(x, what);
  if (x.dim() < 1 || x.size(-1) < 1) refuse(PyExc_ValueError, std::string(what) + " must have features");
  if (x.layout() != at::kStrided) refuse(PyExc_ValueError, std::string(what) + " must be strided");
  const int64_t cols = x.size(-1), rows = x.numel() / cols;
  if (x.is_contiguous()) return {x, dtype, rows, cols, cols};
  if (x.dim() == 2 && (cols == 1 || x.stride(1) == 1) && (rows <= 1 || x.stride(0) >= cols))
    return {x, dtype, rows, cols, rows <= 1 ? cols : x.stride(0)};
  return {x.contiguous(), dtype, rows, cols, cols, true};
}

// The layers' kernels know nothing of tangents: they would be dropped.
void no_tangent(const Tensor& t) {
  if (t.defined() && t._fw_grad(0).defined()) refuse(PyExc_NotImplementedError, "the layers have no forward-mode derivatives");
}

// A recorder of torch's operators would see the outputs' memory allocated and
// nothing that fills it: what it records returns that memory as it is.
void no_recorder() {
  using Mode = c10::impl::TorchDispatchModeKey;
  bool any = torch::jit::tracer::isTracing();
  for (Mode m : {Mode::PROXY, Mode::FAKE, Mode::FUNCTIONAL}) any = any || c10::impl::TorchDispatchModeTLS::get_mode(m);
  if (any) refuse(PyExc_NotImplementedError, "the layers cannot be traced (torch.jit.trace, make_fx, fake tensors)");
}

// The GPU that a layer's operands are on.
int device_of(std::initializer_list<const Tensor*> tensors) {
  int device = -1;
  no_recorder();
  for (const Tensor* t : tensors) no_tangent(*t);
  for (const Tensor* t : tensors) {
    if (!t->defined()) continue;
    if (!t->is_cuda() || (device >= 0 && t->get_device() != device))
      refuse(PyExc_ValueError, "the operands must be on one GPU, got one on " + t->device().str());
    device = (int)t->get_device();
  }
  return device;
}

void* current_stream(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

bool capturing(int device) {
  hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing((hipStream_t)current_stream(device), &s) != hipSuccess) {
    (void)hipGetLastError();  // not this pass's error
    return false;
  }
  return s != hipStreamCaptureStatusNone;
}

const void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor values(const Tensor& like, at::IntArrayRef sizes, at::ScalarType type) { return at::empty(sizes, like.options().dtype(type)); }

Tensor space(const Tensor& like, size_t bytes) { return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)); }

// ------------------------------------------------------- living graphs --

// How many living nodes, recorded outside a capture, have a leaf.
std::mutex leaves_lock;
std::unordered_map<const void*, int> living;

bool is_alive(const Tensor& t) {
  std::lock_guard<std::mutex> lock(leaves_lock);
  return living.count(t.unsafeGetTensorImpl()) != 0;
}

// A layer's node: its gradients are not differentiable again, and say so where
// that is asked for.
struct LayerNode : torch::autograd::Node {
  std::vector<const void*> leaves;  // (a living graph holds them, so their addresses are theirs)

  ~LayerNode() override {
    std::lock_guard<std::mutex> lock(leaves_lock);
    for (const void* t : leaves)
      if (auto it = living.find(t); it != living.end() && --it->second == 0) living.erase(it);
  }

  virtual variable_list gradients(const Tensor& dy) = 0;

  // whether the gradients depend on the inputs, not on dy alone
  virtual bool of_inputs() const { return false; }

  variable_list apply(variable_list&& dy) override {
    if (!dy[0].defined()) return variable_list(num_outputs());
    no_tangent(dy[0]);
    no_recorder();
    variable_list out;
    {
      at::AutoGradMode off(false);
      c10::DeviceGuard device(dy[0].device());
      // (autograd lets a sparse gradient of a dense output through)
      out = gradients(plain(dy[0].layout() == at::kStrided ? dy[0] : dy[0].to_dense()));
    }
    // (a pass that builds a graph; the node exists because an input requires a gradient)
    if (at::GradMode::is_enabled() && (dy[0].requires_grad() || of_inputs())) {
      auto refused = std::make_shared<torch::autograd::DelayedError>(
          "trying to differentiate twice a function whose gradient cannot be differentiated", (int64_t)out.size());
      for (Tensor& t : out)  // the error stands behind outputs that require a gradient
        if (t.defined()) t = t.detach().requires_grad_(true);
      return (*refused)(std::move(out));
    }
    return out;
  }
};

// The node of a pass over these inputs, or none where no gradient is to come.
// Outside a capture its leaves are noted while it lives; a capture is refused
// while a graph from outside it lives that has one of them: both would
// accumulate the leaf's gradient through one node, which belongs to the
// other's stream, and joining that stream from a capture ends the process.
template <typename N>
std::shared_ptr<N> record(int device, std::initializer_list<const Tensor*> inputs) {
  bool need = false;
  if (at::GradMode::is_enabled())
    for (const Tensor* t : inputs) need = need || (t->defined() && t->requires_grad());
  if (!need) return nullptr;
  std::vector<const Tensor*> leaves;
  for (const Tensor* t : inputs)
    if (t->defined() && t->requires_grad() && t->is_leaf()) leaves.push_back(t);
  std::shared_ptr<N> node(new N(), torch::autograd::deleteNode);
  if (capturing(device)) {
    PyObject* list = PyList_New(0);
    if (!list) throw python_error();
    for (const Tensor* t : leaves) {
      PyObject* o = THPVariable_Wrap(*t);
      if (!o || PyList_Append(list, o) < 0) {
        Py_XDECREF(o);
        Py_DECREF(list);
        throw python_error();
      }
      Py_DECREF(o);
    }
    PyObject* said = PyObject_CallOneArg(refuse_capture, list);
    Py_DECREF(list);
    if (!said) throw python_error();
    Py_DECREF(said);
  } else if (!leaves.empty()) {
    std::lock_guard<std::mutex> lock(leaves_lock);
    for (const Tensor* t : leaves) {
      node->leaves.push_back(t->unsafeGetTensorImpl());
      ++living[t->unsafeGetTensorImpl()];
    }
  }
  torch::autograd::edge_list edges;
  for (const Tensor* t : inputs)
    edges.push_back(t->defined() ? torch::autograd::impl::gradient_edge(*t) : torch::autograd::Edge());
  node->set_next_edges(std::move(edges));
  return node;
}

// ---------------------------------------------------------- layer norm --

struct LayerNormNode : LayerNode {
  SavedVariable x, w, stats;
  bool has_w = false;
  int32_t w_dtype = METIS_F32;

  std::string name() const override { return "MetisLayerNorm"; }
  bool of_inputs() const override { return true; }
  void release_variables() override { x.reset_data(), w.reset_data(), stats.reset_data(); }

  variable_list gradients(const Tensor& dy) override {
    const Tensor xs = x.unpack(), ss = stats.unpack(), ws = has_w ? w.unpack() : Tensor();
    const Rows xr = rows_of(xs, "x"), g = rows_of(dy, "the gradient");
    const bool want_x = task_should_compute_output(0), want_w = task_should_compute_output(1), want_b = task_should_compute_output(2);
    Tensor dx, dw, db, room;
    if (want_x) dx = values(xs, xs.sizes(), xs.scalar_type());
    if (want_w) dw = values(xs, {xr.cols}, scalar_type(w_dtype));
    if (want_b) db = values(xs, {xr.cols}, scalar_type(w_dtype));
    size_t need = 0;
    if (want_w || want_b) room = space(xs, need = api.norm_ws(xr.rows, xr.cols));
    const float* mean = (const float*)ss.data_ptr();
    check(api.norm_bwd(g.data(), g.dtype, g.ld, xr.data(), xr.dtype, xr.rows, xr.cols, xr.ld, ptr(ws), w_dtype, mean, mean + xr.rows,
                       (void*)ptr(dx), xr.cols, (void*)ptr(dw), (void*)ptr(db), (void*)ptr(room), need, current_stream((int)xs.get_device())));
    return {dx, dw, db};
  }
};

Tensor layer_norm(const Tensor& x, const Tensor& w, const Tensor& b, double eps) {
  const int device = device_of({&x, &w, &b});
  const Rows r = rows_of(x, "x");
  int32_t w_dtype = METIS_F32;
  for (const Tensor* t : {&w, &b})
    if (t->defined()) {
      w_dtype = float_type(*t, "weight and bias");
      if (t->numel() != r.cols || !t->is_contiguous())
        refuse(PyExc_ValueError, "weight and bias must be " + std::to_string(r.cols) + " contiguous values");
    }
  if (w.defined() && b.defined() && w.scalar_type() != b.scalar_type()) refuse(PyExc_ValueError, "weight and bias must have one type");
  const auto node = record<LayerNormNode>(device, {&x, &w, &b});
  c10::DeviceGuard guard(x.device());
  Tensor y, stats;
  {
    at::AutoDispatchBelowADInplaceOrView below;
    y = values(x, x.sizes(), x.scalar_type());
    if (node) stats = values(x, {2, r.rows}, at::kFloat);
    float* mean = (float*)ptr(stats);
    check(api.norm_fwd(r.data(), r.dtype, r.rows, r.cols, r.ld, ptr(w), ptr(b), w_dtype, eps, y.data_ptr(), r.dtype, r.cols, mean,
                       mean ? mean + r.rows : nullptr, current_stream(device)));
  }
  if (node) {
    node->x = SavedVariable(r.copied ? r.at : x, false);
    node->has_w = w.defined();
    if (w.defined()) node->w = SavedVariable(w, false);
    node->stats = SavedVariable(stats, false);
    node->w_dtype = w_dtype;
    torch::autograd::set_history(y, node);
  }
  return y;
}

// ------------------------------------------------------------- dropout --

struct Draws {
  double p;
  uint64_t seed;
  uint32_t tag;
  int64_t step;
  Tensor count;  // the step on the GPU, for captured passes, or undefined

  Tensor apply(const Tensor& x, const Tensor& residual) const {
    const Rows r = rows_of(x, "x");
    const Rows s = residual.defined() ? rows_of(residual, "the residual") : Rows{};
    Tensor y = values(x, x.sizes(), x.scalar_type());
    check(api.dropout(r.data(), r.dtype, r.rows, r.cols, r.ld, residual.defined() ? s.data() : nullptr, s.ld, p, seed, tag, step,
                      (const int64_t*)ptr(count), y.data_ptr(), r.cols, current_stream((int)x.get_device())));
    return y;
  }
};

struct DropoutNode : LayerNode {
  Draws draws;

  std::string name() const override { return "MetisDropout"; }

  variable_list gradients(const Tensor& dy) override {
    return {task_should_compute_output(0) ? draws.apply(dy, Tensor()) : Tensor(), dy};
  }
};

Tensor dropout(const Tensor& x, const Tensor& residual, const Draws& draws) {
  const int device = device_of({&x, &residual, &draws.count});
  if (residual.defined() && (residual.sizes() != x.sizes() || residual.scalar_type() != x.scalar_type()))
    refuse(PyExc_ValueError, "the residual must have x's shape and type");
  const auto node = record<DropoutNode>(device, {&x, &residual});
  c10::DeviceGuard guard(x.device());
  Tensor y;
  {
    at::AutoDispatchBelowADInplaceOrView below;
    y = draws.apply(x, residual);
  }
  if (node) {
    node->draws = draws;
    torch::autograd::set_history(y, node);
  }
  return y;
}

// ----------------------------------------------------------- embedding --

Tensor numbers_of(const Tensor& t, const char* what) {
  if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
    refuse(PyExc_ValueError, std::string(what) + " must be int32 or int64, got " + c10::toString(t.scalar_type()));
  return t.contiguous();
}

int32_t bits_of(const Tensor& t) { return t.scalar_type() == at::kInt ? 32 : 64; }

struct EmbeddingNode : LayerNode {
  SavedVariable ids;
  int64_t vocab = 0, padding = -1;
  double scale = 1;
  int32_t w_dtype = METIS_F32;

  std::string name() const override { return "MetisEmbedding"; }
  void release_variables() override { ids.reset_data(); }

  variable_list gradients(const Tensor& dy) override {
    const Tensor is = numbers_of(ids.unpack(), "token numbers");
    const Rows g = rows_of(dy, "the gradient");
    Tensor dw = values(dy, {vocab, g.cols}, scalar_type(w_dtype));
    const size_t need = api.embed_ws(g.rows, g.cols);
    Tensor room = space(dy, need);
    check(api.embed_bwd(g.data(), g.dtype, g.rows, g.cols, g.ld, is.data_ptr(), bits_of(is), vocab, padding, scale, dw.data_ptr(),
                        w_dtype, g.cols, room.data_ptr(), need, current_stream((int)dy.get_device())));
    return {dw};
  }
};

Tensor embedding(const Tensor& w, const Tensor& ids, double scale, int64_t padding, int32_t out_dtype) {
  const int device = device_of({&w, &ids});
  const Rows r = rows_of(w, "the weight");
  if (w.dim() != 2) refuse(PyExc_ValueError, "the weight must be a matrix");
  const auto node = record<EmbeddingNode>(device, {&w});
  c10::DeviceGuard guard(w.device());
  Tensor y;
  {
    at::AutoDispatchBelowADInplaceOrView below;
    const Tensor is = numbers_of(ids, "token numbers");
    at::DimVector sizes(ids.sizes().begin(), ids.sizes().end());
    sizes.push_back(r.cols);
    if (out_dtype < 0) out_dtype = r.dtype;
    y = values(w, sizes, scalar_type(out_dtype));
    check(api.embed_fwd(r.data(), r.dtype, r.rows, r.cols, r.ld, is.data_ptr(), bits_of(is), is.numel(), scale, y.data_ptr(), out_dtype,
                        r.cols, current_stream(device)));
  }
  if (node) {
    node->ids = SavedVariable(ids, false);
    node->vocab = r.rows, node->padding = padding, node->scale = scale, node->w_dtype = r.dtype;
    torch::autograd::set_history(y, node);
  }
  return y;
}

// ---------------------------------------------------------------- loss --

metis_loss loss_of(const Rows& x, const Rows& w, const Tensor& targets, int64_t ignore) {
  metis_loss l{};
  l.x = x.data(), l.w = w.data(), l.targets = targets.data_ptr();
  l.tokens = x.rows, l.vocab = w.rows, l.cols = x.cols;
  l.ldx = x.ld, l.ldw = w.ld;
  l.ignore_index = ignore;
  l.x_dtype = x.dtype, l.w_dtype = w.dtype;
  l.target_bits = bits_of(targets);
  return l;
}

enum Reduction { kNone, kSum, kMean };

struct LossNode : LayerNode {
  SavedVariable x, w, targets, lse, total;
  int64_t ignore = -100;
  int reduction = kMean;

  std::string name() const override { return "MetisLinearCrossEntropy"; }
  bool of_inputs() const override { return true; }
  void release_variables() override { x.reset_data(), w.reset_data(), targets.reset_data(), lse.reset_data(), total.reset_data(); }

  variable_list gradients(const Tensor& dy) override {
    const Tensor xs = x.unpack(), ws = w.unpack(), ls = lse.unpack(), ts = numbers_of(targets.unpack(), "targets");
    const Tensor count = reduction == kMean ? total.unpack() : Tensor();
    const Tensor g = dy.contiguous();
    const Rows xr = rows_of(xs, "x"), wr = rows_of(ws, "the weight");
    const metis_loss l = loss_of(xr, wr, ts, ignore);
    Tensor dx, dw;
    if (task_should_compute_output(0)) dx = values(xs, xs.sizes(), xs.scalar_type());
    if (task_should_compute_output(1)) dw = values(ws, ws.sizes(), ws.scalar_type());
    const size_t need = api.loss_ws(&l, 1);
    Tensor room = space(xs, need);
    check(api.loss_bwd(&l, (const float*)ls.data_ptr(), (const float*)g.data_ptr(), reduction == kNone,
                       count.defined() ? (const float*)count.data_ptr() + 1 : nullptr, (void*)ptr(dx), xr.cols, (void*)ptr(dw), wr.cols,
                       room.data_ptr(), need, current_stream((int)xs.get_device())));
    return {dx, dw};
  }
};

Tensor linear_cross_entropy(const Tensor& x, const Tensor& w, const Tensor& targets, int64_t ignore, int reduction) {
  const int device = device_of({&x, &w, &targets});
  const Rows xr = rows_of(x, "x"), wr = rows_of(w, "the weight");
  if (w.dim() != 2 || wr.cols != xr.cols || targets.sizes() != x.sizes().slice(0, x.dim() - 1))
    refuse(PyExc_ValueError, "x, the weight and the targets must be ... x features, vocabulary x features and ...");
  const auto node = record<LossNode>(device, {&x, &w});
  c10::DeviceGuard guard(x.device());
  Tensor out, lse, total;
  {
    at::AutoDispatchBelowADInplaceOrView below;
    const Tensor ts = numbers_of(targets, "targets");
    const metis_loss l = loss_of(xr, wr, ts, ignore);
    lse = values(x, {xr.rows}, at::kFloat);
    if (reduction == kNone) out = values(x, targets.sizes(), at::kFloat);
    else total = values(x, {2}, at::kFloat);
    const size_t need = api.loss_ws(&l, 0);
    Tensor room = space(x, need);
    check(api.loss_fwd(&l, (float*)ptr(out), (float*)lse.data_ptr(), reduction == kMean, (float*)ptr(total), room.data_ptr(), need,
                       current_stream(device)));
    if (reduction != kNone) out = total.select(0, 0);
  }
  if (node) {
    node->x = SavedVariable(xr.copied ? xr.at : x, false);
    node->w = SavedVariable(wr.copied ? wr.at : w, false);
    node->targets = SavedVariable(targets, false);
    node->lse = SavedVariable(lse, false);
    if (total.defined()) node->total = SavedVariable(total, false);
    node->ignore = ignore, node->reduction = reduction;
    torch::autograd::set_history(out, node);
  }
  return out;
}

// -------------------------------------------------------------- module --

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, std::to_string(want) + " arguments expected, got " + std::to_string(n));
}

template <typename F>
PyObject* call(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what());
    return nullptr;
  } catch (const Failed& e) {
    if (PyObject* o = PyObject_CallFunction(error_class, "is", e.status, e.text.c_str())) {
      PyErr_SetObject(error_class, o);
      Py_DECREF(o);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* py_layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    count_args(n, 4);
    return THPVariable_Wrap(layer_norm(plain(tensor(a[0], "x")), plain(maybe(a[1], "weight")), plain(maybe(a[2], "bias")), number(a[3])));
  });
}

PyObject* py_dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    count_args(n, 7);
    const Draws d{number(a[2]), PyLong_AsUnsignedLongLongMask(a[3]), (uint32_t)integer(a[4]), integer(a[5]), maybe(a[6], "the count")};
    if (PyErr_Occurred()) throw python_error();
    return THPVariable_Wrap(dropout(plain(tensor(a[0], "x")), plain(maybe(a[1], "the residual")), d));
  });
}

PyObject* py_embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    count_args(n, 5);
    return THPVariable_Wrap(
        embedding(plain(tensor(a[0], "the weight")), tensor(a[1], "token numbers"), number(a[2]), integer(a[3]), (int32_t)integer(a[4])));
  });
}

PyObject* py_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    count_args(n, 5);
    return THPVariable_Wrap(linear_cross_entropy(plain(tensor(a[0], "x")), plain(tensor(a[1], "the weight")), tensor(a[2], "targets"), integer(a[3]),
                                                 (int)integer(a[4])));
  });
}

PyObject* py_alive(PyObject*, PyObject* o) {
  return call([&] { return PyBool_FromLong(is_alive(tensor(o, "the leaf"))); });
}

// init(addresses of the entry points in Api's order, error class, refuse_capture)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&]() -> PyObject* {
    count_args(n, 3);
    constexpr Py_ssize_t count = sizeof(Api) / sizeof(void*);
    if (!PyList_Check(a[0]) || PyList_GET_SIZE(a[0]) != count) refuse(PyExc_ValueError, "entry points");
    void** to = (void**)&api;
    for (Py_ssize_t i = 0; i < count; ++i) to[i] = (void*)(uintptr_t)integer(PyList_GET_ITEM(a[0], i));
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    Py_XSETREF(error_class, a[1]);
    Py_XSETREF(refuse_capture, a[2]);
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))py_init, METH_FASTCALL, "The library's entry points."},
    {"layer_norm", (PyCFunction)(void (*)(void))py_layer_norm, METH_FASTCALL, "layer_norm(x, weight, bias, eps)"},
    {"dropout", (PyCFunction)(void (*)(void))py_dropout, METH_FASTCALL, "dropout(x, residual, p, seed, tag, step, count)"},
    {"embedding", (PyCFunction)(void (*)(void))py_embedding, METH_FASTCALL, "embedding(weight, ids, scale, padding, dtype code or -1)"},
    {"linear_cross_entropy", (PyCFunction)(void (*)(void))py_loss, METH_FASTCALL,
     "linear_cross_entropy(x, weight, targets, ignore_index, reduction)"},
    {"alive", py_alive, METH_O, "Whether a graph of these layers from outside a capture lives that has this leaf."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", "Layers as autograd nodes on the library.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layers(void) { return PyModule_Create(&module); }
