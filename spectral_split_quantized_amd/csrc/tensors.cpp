// tensors.cpp -- reads lists of torch tensors into the library's tensor tables
// (metis_adamw_tensor), with the binding's checks.  An optimizer step names
// six tensors a parameter; gathering them from Python costs about 2 us a
// parameter, here a tenth of that.  A Python extension module (_tensors); host
// code only, nothing is kept between calls.

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <string>
#include <vector>

#include "../../include/metis.h"

namespace {

constexpr int64_t kStateBlock = 256;  // elements of an 8-bit state that share a scale

// A refused argument: becomes the Python exception of that type.
struct Refused {
  PyObject* type;
  std::string what;
};

[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refused{type, what}; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(what) + " must be tensors");
  return THPVariable_Unpack(o);
}

// Layout, size and device of one tensor; its address.
void* address(const at::Tensor& t, int64_t numel, int device, const char* what) {
  if (t.layout() != at::kStrided || !t.is_contiguous() || t.numel() != numel)
    refuse(PyExc_ValueError, std::string(what) + " must be contiguous and of the parameters' sizes");
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " must be on a GPU");
  if (t.get_device() != device) refuse(PyExc_ValueError, std::string(what) + " must be on one GPU");
  return t.data_ptr();
}

int32_t float_type(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return METIS_BF16;
  if (t.scalar_type() == at::kFloat) return METIS_F32;
  refuse(PyExc_TypeError, std::string(what) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}

int device_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(what) + " must be on a GPU");
  return (int)t.get_device();
}

void put_grad(metis_adamw_tensor& row, const at::Tensor& g, int device) {
  row.grad = address(g, row.n, device, "gradients");
  row.grad_dtype = float_type(g, "gradients");
}

void put_param(metis_adamw_tensor& row, const at::Tensor& p, int device) {
  row.n = p.numel();
  row.param = address(p, row.n, device, "parameters");
  row.param_dtype = float_type(p, "parameters");
}

// both states and, for 8 bits, their scales (null pointers: 32 bits)
void put_states(metis_adamw_tensor& row, const at::Tensor& m, const at::Tensor& v, const at::Tensor* ms,
                const at::Tensor* vs, int device) {
  if (!ms != !vs) refuse(PyExc_ValueError, "a parameter's two states must have the same width");
  const auto type = ms ? at::kFloat8_e4m3fn : at::kFloat;
  for (const at::Tensor* t : {&m, &v})
    if (t->scalar_type() != type)
      refuse(PyExc_TypeError, std::string("states must be float32, or float8_e4m3fn with scales; got ") +
                                  c10::toString(t->scalar_type()));
  row.m = address(m, row.n, device, "states");
  row.v = address(v, row.n, device, "states");
  row.state_bits = ms ? 8 : 32;
  row.m_scale = row.v_scale = nullptr;
  if (!ms) return;
  const int64_t blocks = (row.n + kStateBlock - 1) / kStateBlock;
  for (const at::Tensor* t : {ms, vs})
    if (t->scalar_type() != at::kFloat) refuse(PyExc_TypeError, "scales must be float32");
  row.m_scale = (float*)address(*ms, blocks, device, "scales");
  row.v_scale = (float*)address(*vs, blocks, device, "scales");
}

// No two of the written arrays share memory, and no gradient with one of them.
void check_apart(const metis_adamw_tensor* rows, size_t n) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Span> used;
  used.reserve(6 * n);
  auto add = [&](const void* p, int64_t bytes, bool written = true) {
    if (bytes) used.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
  };
  for (size_t i = 0; i < n; ++i) {
    const metis_adamw_tensor& r = rows[i];
    const int64_t state = r.state_bits == 8 ? r.n : 4 * r.n;
    add(r.param, r.n * (r.param_dtype == METIS_F32 ? 4 : 2));
    add(r.grad, r.n * (r.grad_dtype == METIS_F32 ? 4 : 2), false);
    add(r.m, state);
    add(r.v, state);
    if (r.state_bits == 8) {
      add(r.m_scale, (r.n + kStateBlock - 1) / kStateBlock * 4);
      add(r.v_scale, (r.n + kStateBlock - 1) / kStateBlock * 4);
    }
  }
  std::sort(used.begin(), used.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t read_end = 0, written_end = 0;  // the farthest ends so far
  for (const Span& s : used) {
    if (s.begin < written_end || (s.written && s.begin < read_end))
      refuse(PyExc_ValueError, "a parameter or a state appears twice, or two of them (or one and a gradient) overlap");
    uintptr_t& end = s.written ? written_end : read_end;
    end = std::max(end, s.end);
  }
}

// Tells autograd of the write to come, so that a graph that saved the parameter
// refuses its backward pass.
void mark_written(const at::Tensor& p) {
  if (!p.is_inference()) p.unsafeGetTensorImpl()->bump_version();
}

uint32_t default_tag(int64_t i) { return (uint32_t)(i & 0xFFFF) << 16 | (uint32_t)METIS_OPERAND_W << 12; }

// A writable buffer of n rows.
struct Table {
  Py_buffer view{};
  metis_adamw_tensor* rows;

  Table(PyObject* o, Py_ssize_t n) {
    if (PyObject_GetBuffer(o, &view, PyBUF_WRITABLE | PyBUF_C_CONTIGUOUS) != 0) throw std::bad_exception();
    if (view.len != n * (Py_ssize_t)sizeof(metis_adamw_tensor)) {
      PyBuffer_Release(&view);
      refuse(PyExc_ValueError, "the table must hold one row a tensor");
    }
    rows = (metis_adamw_tensor*)view.buf;
  }
  ~Table() { PyBuffer_Release(&view); }
  Table(const Table&) = delete;
};

// Runs f; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* item(PyObject* list, Py_ssize_t i) { return PyList_GET_ITEM(list, i); }

void check_lists(std::initializer_list<PyObject*> lists, Py_ssize_t n) {
  for (PyObject* l : lists)
    if (!PyList_Check(l) || PyList_GET_SIZE(l) != n)
      refuse(PyExc_ValueError, "parameters, gradients, states, scales and tags must be lists of one length");
}

// fill(params, grads, ms, vs, m_scales, v_scales, tags or None, table) -> device
PyObject* fill(PyObject*, PyObject* args) {
  PyObject *params, *grads, *ms, *vs, *m_scales, *v_scales, *tags, *buffer;
  if (!PyArg_ParseTuple(args, "OOOOOOOO", &params, &grads, &ms, &vs, &m_scales, &v_scales, &tags, &buffer)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!PyList_Check(params)) refuse(PyExc_ValueError, "parameters must be a list");
    const Py_ssize_t n = PyList_GET_SIZE(params);
    check_lists({grads, ms, vs, m_scales, v_scales}, n);
    if (tags != Py_None) check_lists({tags}, n);
    Table t(buffer, n);
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor& p = tensor(item(params, i), "parameters");
      if (i == 0) device = device_of(p, "parameters");
      PyObject *a = item(m_scales, i), *b = item(v_scales, i);
      put_param(t.rows[i], p, device);
      put_grad(t.rows[i], tensor(item(grads, i), "gradients"), device);
      put_states(t.rows[i], tensor(item(ms, i), "states"), tensor(item(vs, i), "states"),
                 a == Py_None ? nullptr : &tensor(a, "scales"), b == Py_None ? nullptr : &tensor(b, "scales"), device);
      t.rows[i].tag = default_tag(i);
      if (tags != Py_None) {
        t.rows[i].tag = (uint32_t)PyLong_AsUnsignedLongMask(item(tags, i));
        if (PyErr_Occurred()) return nullptr;
      }
    }
    check_apart(t.rows, (size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) mark_written(tensor(item(params, i), "parameters"));
    return PyLong_FromLong(device);
  });
}

// fill_grads(grads, table) -> device
PyObject* fill_grads(PyObject*, PyObject* args) {
  PyObject *grads, *buffer;
  if (!PyArg_ParseTuple(args, "OO", &grads, &buffer)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!PyList_Check(grads)) refuse(PyExc_ValueError, "gradients must be a list");
    const Py_ssize_t n = PyList_GET_SIZE(grads);
    Table t(buffer, n);
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor& g = tensor(item(grads, i), "gradients");
      if (i == 0) device = device_of(g, "gradients");
      t.rows[i] = metis_adamw_tensor{};
      t.rows[i].n = g.numel();
      put_grad(t.rows[i], g, device);
    }
    return PyLong_FromLong(device);
  });
}

PyObject* names[5];  // "step" and the states' keys

// fill_state(params, state, first_tag, counts_on_gpu, table) -> (device, step,
// states), the optimizer's form: gradients from the parameters, states from
// the optimizer's dict of dicts.  None where a parameter has no gradient or no
// state yet, a gradient is not contiguous, or the step counts differ (those on
// the GPU: are not one tensor): the caller sorts those out and uses fill.
PyObject* fill_state(PyObject*, PyObject* args) {
  PyObject *params, *state, *buffer;
  long long first;
  int counts_on_gpu;
  if (!PyArg_ParseTuple(args, "OOLpO", &params, &state, &first, &counts_on_gpu, &buffer)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!PyList_Check(params) || !PyDict_Check(state)) refuse(PyExc_ValueError, "parameters must be a list and state a dict");
    const Py_ssize_t n = PyList_GET_SIZE(params);
    if (n == 0) Py_RETURN_NONE;
    Table t(buffer, n);
    int device = -1;
    PyObject* step = nullptr;  // borrowed
    PyObject* states = PyList_New(n);
    if (!states) return nullptr;
    struct Drop {
      PyObject* o;
      ~Drop() { Py_XDECREF(o); }
    } drop{states};
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor& p = tensor(item(params, i), "parameters");
      const at::Tensor& g = p.grad();
      if (!g.defined() || g.layout() != at::kStrided || !g.is_contiguous()) Py_RETURN_NONE;
      PyObject* s = PyDict_GetItemWithError(state, item(params, i));
      if (!s) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
      }
      if (!PyDict_Check(s)) refuse(PyExc_TypeError, "a parameter's state must be a dict");
      PyObject* v[5];
      for (int k = 0; k < 5; ++k) {
        v[k] = PyDict_GetItemWithError(s, names[k]);
        if (!v[k] && PyErr_Occurred()) return nullptr;
      }
      if (!v[0] || !v[1] || !v[2]) Py_RETURN_NONE;
      if (i == 0) {
        device = device_of(p, "parameters");
        step = v[0];
      } else if (v[0] != step) {
        if (counts_on_gpu) Py_RETURN_NONE;
        const int equal = PyObject_RichCompareBool(v[0], step, Py_EQ);
        if (equal < 0) return nullptr;
        if (!equal) Py_RETURN_NONE;
      }
      metis_adamw_tensor& row = t.rows[i];
      put_param(row, p, device);
      put_grad(row, g, device);
      put_states(row, tensor(v[1], "states"), tensor(v[2], "states"), v[3] ? &tensor(v[3], "scales") : nullptr,
                 v[4] ? &tensor(v[4], "scales") : nullptr, device);
      row.tag = default_tag(first + i);
      Py_INCREF(s);
      PyList_SET_ITEM(states, i, s);
    }
    check_apart(t.rows, (size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) mark_written(tensor(item(params, i), "parameters"));
    return Py_BuildValue("(iOO)", device, step, states);
  });
}

PyMethodDef methods[] = {{"fill", fill, METH_VARARGS, "Lists of tensors into a table; returns their device."},
                         {"fill_grads", fill_grads, METH_VARARGS, "Gradients alone into a table; returns their device."},
                         {"fill_state", fill_state, METH_VARARGS, "An optimizer group into a table, or None."},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "Tensor lists as tables of the library.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) {
  const char* keys[5] = {"step", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"};
  for (int k = 0; k < 5; ++k)
    if (!(names[k] = PyUnicode_InternFromString(keys[k]))) return nullptr;
  return PyModule_Create(&module);
}
