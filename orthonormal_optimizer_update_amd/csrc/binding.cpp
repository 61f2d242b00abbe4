// Python binding of the calls over many tensors and of the tokens by expert: torch
// tensors to ortho_mat descriptors and the call, without the interpreter in
// between.  (Described attribute by attribute in Python a tensor costs 0.4 us in a
// list and 0.6 in a call of its own, here 0.01 to 0.02; the launch of a call takes 3.)
// Argument marshalling only: each function returns the library's status, or raises
// ValueError for tensors that no descriptor can stand for.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <new>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/ortho.h"

namespace {

// What becomes a Python ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string text(const at::Tensor& t) { return c10::str(t.device()); }

// Tensors of one call are on one GPU.
struct Device {
  int64_t index = -1;
  void check(const at::Tensor& t) {
    if (!t.is_cuda()) throw Refused("expected tensors on a GPU, got " + text(t));
    const int64_t at = t.get_device();
    if (index < 0) index = at;
    else if (at != index)
      throw Refused("expected every tensor on cuda:" + std::to_string(index) + ", got " + text(t));
  }
};

int32_t dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return ORTHO_F32;
    case at::kBFloat16: return ORTHO_BF16;
    case at::kFloat8_e4m3fn: return ORTHO_E4M3;
    case at::kFloat8_e8m0fnu: return ORTHO_E8M0;
    default: throw Refused(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
  }
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused(std::string("expected ") + what + " as a tensor");
  return THPVariable_Unpack(o);
}

// A 2-D tensor with unit column stride.
ortho_mat matrix(const at::Tensor& t, Device& dev) {
  dev.check(t);
  if (t.dim() != 2) throw Refused("expected a 2-D tensor");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (t.stride(1) != 1 && cols > 1) throw Refused("expected unit stride along columns");
  int64_t ld = cols;
  if (rows > 1) {
    ld = t.stride(0);
    if (ld < cols) throw Refused("expected rows that do not overlap");
  }
  return {t.data_ptr(), rows, cols, ld, dtype_of(t)};
}

// A tensor of any shape: its first dimension by the others, which lie without gaps; a
// vector is one row.
void shape_as_matrix(const at::Tensor& t, int64_t& rows, int64_t& cols, int64_t& ld) {
  const auto sizes = t.sizes(), strides = t.strides();
  const int64_t dims = t.dim();
  rows = dims < 2 ? 1 : sizes[0];
  cols = 1;
  for (int64_t d = dims - 1; d >= (dims < 2 ? 0 : 1); --d) {
    if (sizes[d] != 1 && strides[d] != cols) throw Refused("expected unit stride along columns");
    cols *= sizes[d];
  }
  ld = cols > 1 ? cols : 1;
  if (rows > 1) {
    ld = strides[0];
    if (ld < cols) throw Refused("expected rows that do not overlap");
  }
}

// One matrix per tensor of a list; none for None.
struct List {
  std::vector<ortho_mat> m;
  PyObject* held = nullptr;
  ~List() { Py_XDECREF(held); }
  void fill(PyObject* o, Device& dev, const char* what) {
    held = PySequence_Fast(o, what);
    if (held == nullptr) {
      PyErr_Clear();
      throw Refused(std::string("expected ") + what + " as a list of tensors");
    }
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(held);
    if (n > std::numeric_limits<int32_t>::max()) throw Refused("expected fewer tensors");
    PyObject** const items = PySequence_Fast_ITEMS(held);
    m.resize(static_cast<size_t>(n));
    for (Py_ssize_t i = 0; i < n; ++i) {
      if (items[i] == Py_None) {
        m[i] = {};
        continue;
      }
      const at::Tensor& t = tensor(items[i], what);
      dev.check(t);
      ortho_mat& a = m[i];
      shape_as_matrix(t, a.rows, a.cols, a.ld);
      a.data = t.data_ptr();
      a.dtype = dtype_of(t);
    }
  }
  void like(const List& other) const {
    if (m.size() != other.m.size())
      throw Refused("expected " + std::to_string(other.m.size()) + " tensors in each list, got " +
                    std::to_string(m.size()));
  }
  int32_t count() const { return static_cast<int32_t>(m.size()); }
};

// Consecutive elements of a type.
void* elements(PyObject* o, at::ScalarType type, int64_t count, Device& dev, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || t.numel() != count || !t.is_contiguous())
    throw Refused(std::string("expected ") + what + " as " + std::to_string(count) + " consecutive " +
                  c10::toString(type));
  dev.check(t);
  return t.data_ptr();
}

int32_t* int32s(PyObject* o, int64_t count, Device& dev, const char* what) {
  return static_cast<int32_t*>(elements(o, at::kInt, count, dev, what));
}

// The bytes behind a workspace's address (an expanded tensor has fewer elements than it shows).
void* workspace(PyObject* o, Device& dev, size_t& bytes) {
  const at::Tensor& t = tensor(o, "ws");
  dev.check(t);
  int64_t count = t.numel();
  if (!t.is_contiguous()) {
    int64_t reach = 1;
    for (int64_t d = 0; d < t.dim(); ++d) reach += (t.size(d) - 1) * t.stride(d);
    count = std::min(count, reach);
  }
  bytes = static_cast<size_t>(count) * t.element_size();
  return t.data_ptr();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::bad_exception();   // (Python's error stands)
  return v;
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::bad_exception();
  return v;
}

int32_t small(PyObject* o, const char* what) {
  const int64_t v = whole(o);
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    throw Refused(std::string("expected a smaller ") + what + ", got " + std::to_string(v));
  return static_cast<int32_t>(v);
}

void* stream_of(PyObject* o) {
  void* const s = PyLong_AsVoidPtr(o);
  if (s == nullptr && PyErr_Occurred()) throw std::bad_exception();
  return s;
}

// The library's call without the interpreter's lock: a full queue may make it wait.
template <class F>
PyObject* status_of(F call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return PyLong_FromLong(status);
}

template <int kArgs, class F>
PyObject* guarded(Py_ssize_t n, F f) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const std::bad_exception&) {   // set already
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

typedef PyObject* const* Args;

bool none(PyObject* o) { return o == Py_None; }

// Optional matrix: its descriptor in m, or null.
const ortho_mat* optional(PyObject* o, ortho_mat& m, Device& dev, const char* what) {
  if (none(o)) return nullptr;
  m = matrix(tensor(o, what), dev);
  return &m;
}

PyObject* py_check(PyObject*, Args a, Py_ssize_t n) {   // (tensors) -> the number of them
  return guarded<1>(n, [&]() -> PyObject* {
    List l;
    Device dev;
    l.fill(a[0], dev, "tensors");
    return PyLong_FromLong(l.count());
  });
}

PyObject* py_matrix(PyObject*, Args a, Py_ssize_t n) {   // (tensor) -> rows, cols, ld; any device
  return guarded<1>(n, [&]() -> PyObject* {
    int64_t rows, cols, ld;
    shape_as_matrix(tensor(a[0], "a matrix"), rows, cols, ld);
    return Py_BuildValue("LLL", (long long)rows, (long long)cols, (long long)ld);
  });
}

PyObject* py_grad_norm(PyObject*, Args a, Py_ssize_t n) {   // G, max_norm, out, ws, stream
  return guarded<5>(n, [&]() -> PyObject* {
    List g;
    Device dev;
    g.fill(a[0], dev, "gradients");
    const double most = number(a[1]);
    float* const out = static_cast<float*>(elements(a[2], at::kFloat, 2, dev, "out"));
    size_t bytes;
    void* const ws = workspace(a[3], dev, bytes);
    void* const stream = stream_of(a[4]);
    return status_of([&] { return grad_norm(g.count(), g.m.data(), most, out, ws, bytes, stream); });
  });
}

// X, G, M, V, SM, SV, lr, step, beta1, beta2, eps, weight_decay, seed, factor, stream
PyObject* py_adamw_step(PyObject*, Args a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject* {
    List l[6];
    Device dev;
    const char* const names[] = {"weights", "gradients", "M", "V", "SM", "SV"};
    for (int i = 0; i < 6; ++i) {
      if (i > 3 && none(a[i])) continue;
      l[i].fill(a[i], dev, names[i]);
      l[i].like(l[0]);
    }
    ortho_adamw h{};
    if (THPVariable_Check(a[6])) h.lr_dev = static_cast<float*>(elements(a[6], at::kFloat, 1, dev, "lr"));
    else h.lr = number(a[6]);
    h.step = 1;
    if (THPVariable_Check(a[7])) h.step_dev = static_cast<int64_t*>(elements(a[7], at::kLong, 1, dev, "step"));
    else h.step = whole(a[7]);
    h.beta1 = number(a[8]);
    h.beta2 = number(a[9]);
    h.eps = number(a[10]);
    h.weight_decay = number(a[11]);
    if (!none(a[12])) {
      h.stochastic = 1;
      h.seed = PyLong_AsUnsignedLongLongMask(a[12]);
      if (PyErr_Occurred()) throw std::bad_exception();
    }
    if (!none(a[13])) h.factor = static_cast<float*>(elements(a[13], at::kFloat, 1, dev, "factor"));
    void* const stream = stream_of(a[14]);
    return status_of([&] {
      return adamw_step(l[0].count(), l[0].m.data(), l[1].m.data(), l[2].m.data(), l[3].m.data(),
                        l[4].held ? l[4].m.data() : nullptr, l[5].held ? l[5].m.data() : nullptr, &h, stream);
    });
  });
}

// chosen, experts, align, slot, source, offsets, counts, ws, stream
PyObject* py_expert_sort(PyObject*, Args a, Py_ssize_t n) {
  return guarded<9>(n, [&]() -> PyObject* {
    Device dev;
    const at::Tensor& chosen = tensor(a[0], "chosen");
    dev.check(chosen);
    if (chosen.dim() != 2 || !chosen.is_contiguous() ||
        (chosen.scalar_type() != at::kInt && chosen.scalar_type() != at::kLong))
      throw Refused("expected chosen as a contiguous tokens x choices tensor of int32 or int64");
    const int64_t tokens = chosen.size(0);
    const int32_t choices = chosen.size(1) < 1 << 30 ? static_cast<int32_t>(chosen.size(1)) : 1 << 30;
    const int32_t experts = small(a[1], "number of experts"), align = small(a[2], "align");
    int32_t* const slot = int32s(a[3], chosen.numel(), dev, "slot");
    int32_t* const source =
        none(a[4]) ? nullptr : int32s(a[4], ortho_expert_rows(tokens, choices, experts, align), dev, "source");
    int32_t* const offsets = int32s(a[5], static_cast<int64_t>(experts) + 1, dev, "offsets");
    int32_t* const counts = int32s(a[6], experts, dev, "counts");
    size_t bytes;
    void* const ws = workspace(a[7], dev, bytes);
    void* const stream = stream_of(a[8]);
    const void* const from = chosen.data_ptr();
    const int32_t wide = static_cast<int32_t>(chosen.element_size());
    return status_of([&] {
      return expert_sort(from, wide, tokens, choices, experts, align, slot, source, offsets, counts, ws, bytes,
                         stream);
    });
  });
}

// The rows of `tokens` tokens: slot's address and choices.
const int32_t* slots(PyObject* o, int64_t tokens, Device& dev, int32_t& choices) {
  const at::Tensor& t = tensor(o, "slot");
  if (t.dim() != 2 || t.size(0) != tokens) throw Refused("expected slot with " + std::to_string(tokens) + " rows");
  choices = t.size(1) < 1 << 30 ? static_cast<int32_t>(t.size(1)) : 1 << 30;
  return int32s(o, t.numel(), dev, "slot");
}

struct Experts {
  const int32_t *offsets, *counts;
  int32_t count;
  Experts(PyObject* o, PyObject* c, Device& dev) {
    const int64_t e = tensor(c, "counts").numel();
    count = e < 1 << 30 ? static_cast<int32_t>(e) : 1 << 30;
    offsets = int32s(o, e + 1, dev, "offsets");
    counts = int32s(c, e, dev, "counts");
  }
};

// X, S, slot, offsets, counts, Y, SY, stream
PyObject* py_expert_gather(PyObject*, Args a, Py_ssize_t n) {
  return guarded<8>(n, [&]() -> PyObject* {
    Device dev;
    ortho_mat s, sy;
    const ortho_mat x = matrix(tensor(a[0], "X"), dev);
    const ortho_mat* const ps = optional(a[1], s, dev, "S");
    int32_t choices;
    const int32_t* const slot = slots(a[2], x.rows, dev, choices);
    const Experts e(a[3], a[4], dev);
    const ortho_mat y = matrix(tensor(a[5], "Y"), dev);
    const ortho_mat* const psy = optional(a[6], sy, dev, "SY");
    void* const stream = stream_of(a[7]);
    return status_of([&] {
      return expert_gather(x, ps, slot, choices, e.offsets, e.counts, e.count, y, psy, stream);
    });
  });
}

// Y, slot, weights, add, out, stream
PyObject* py_expert_combine(PyObject*, Args a, Py_ssize_t n) {
  return guarded<6>(n, [&]() -> PyObject* {
    Device dev;
    ortho_mat w, add;
    const ortho_mat y = matrix(tensor(a[0], "Y"), dev), out = matrix(tensor(a[4], "out"), dev);
    int32_t choices;
    const int32_t* const slot = slots(a[1], out.rows, dev, choices);
    const ortho_mat* const pw = optional(a[2], w, dev, "weights");
    const ortho_mat* const padd = optional(a[3], add, dev, "add");
    void* const stream = stream_of(a[5]);
    return status_of([&] { return expert_combine(y, slot, choices, pw, padd, out, stream); });
  });
}

// dOut, slot, weights, offsets, counts, dY, Y, dW, stream
PyObject* py_expert_combine_backward(PyObject*, Args a, Py_ssize_t n) {
  return guarded<9>(n, [&]() -> PyObject* {
    Device dev;
    ortho_mat w, y, dw;
    const ortho_mat d = matrix(tensor(a[0], "dOut"), dev);
    int32_t choices;
    const int32_t* const slot = slots(a[1], d.rows, dev, choices);
    const ortho_mat* const pw = optional(a[2], w, dev, "weights");
    const Experts e(a[3], a[4], dev);
    const ortho_mat dy = matrix(tensor(a[5], "dY"), dev);
    const ortho_mat* const py = optional(a[6], y, dev, "Y");
    const ortho_mat* const pdw = optional(a[7], dw, dev, "dW");
    void* const stream = stream_of(a[8]);
    return status_of([&] {
      return expert_combine_backward(d, slot, choices, pw, e.offsets, e.counts, e.count, dy, py, pdw, stream);
    });
  });
}

#define ORTHO_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ORTHO_METHOD(check),         ORTHO_METHOD(matrix),
                         ORTHO_METHOD(grad_norm),     ORTHO_METHOD(adamw_step),
                         ORTHO_METHOD(expert_sort),   ORTHO_METHOD(expert_gather),
                         ORTHO_METHOD(expert_combine), ORTHO_METHOD(expert_combine_backward),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&definition); }
