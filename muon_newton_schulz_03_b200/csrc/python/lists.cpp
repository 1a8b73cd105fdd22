// Python side of the list operators: reads lists of torch tensors and makes
// the C calls of include/muon_ns.h.
//
// A whole model is hundreds of tensors and four lists of them, so reading
// each tensor's attributes through the interpreter (about 2 us a tensor)
// costs several times the kernels. Here a tensor takes tens of nanoseconds.
// A list that does not pass returns None, and the binding says what is wrong
// with it; a C error comes back as its status code. Nothing is kept between
// calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <vector>

#include "muon_ns.h"

namespace {

decltype(&muon_grad_norm) c_norm = nullptr;
decltype(&muon_clip_grads) c_clip = nullptr;
decltype(&muon_adamw_step) c_adamw = nullptr;

constexpr int kAny = 7, kF32 = 1;   // allowed types, one bit each

struct Column {
  std::vector<void*> ptr;
  std::vector<int32_t> type;
  bool writes = false;                      // the call writes its tensors
  std::vector<c10::TensorImpl*> versions;   // tensors whose version counters move then
  void resize(size_t n) {
    ptr.assign(n, nullptr);
    type.assign(n, 0);
    if (writes) versions.reserve(n);
  }
  // Moving a counter is an atomic (8 ns). Tensors cut from one buffer share
  // theirs, and it is not moved again for a tensor whose counter is among the
  // last four. Inference tensors have none.
  void note(c10::TensorImpl* impl) {
    uintptr_t id;   // which counter: the value of the one pointer that is kept of it, null without one
    static_assert(sizeof(c10::VariableVersion) == sizeof(id), "a pointer to the counter");
    std::memcpy(&id, &impl->version_counter(), sizeof(id));
    if (id == 0 || id == recent[0] || id == recent[1] || id == recent[2] || id == recent[3]) return;
    recent[at] = id;
    at = (at + 1) % kRecent;
    versions.push_back(impl);
  }
  // The call has written the tensors: a backward pass over a graph that saved
  // the old values raises from now on.
  void written() const {
    for (c10::TensorImpl* impl : versions)
      if (!impl->is_inference()) impl->bump_version();
  }

 private:
  static constexpr int kRecent = 4;
  uintptr_t recent[kRecent] = {};
  int at = 0;
};

int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MUON_DTYPE_F32;
    case at::kBFloat16: return MUON_DTYPE_BF16;
    case at::kHalf: return MUON_DTYPE_F16;
    default: return -1;
  }
}

// Whether a tensor is strided memory on a CUDA device, read as it is. That
// follows from its set of dispatch keys, so it is asked once per set: nearly
// all tensors of a program have the same one.
bool is_plain(const at::Tensor& t, uint64_t& known) {
  const uint64_t keys = t.unsafeGetTensorImpl()->key_set().raw_repr();
  if (keys == known) return true;
  if (t.layout() != at::kStrided || !t.is_cuda() || t.is_neg()) return false;
  known = keys;
  return true;
}

// What the entries of one row have in common.
struct Row {
  c10::IntArrayRef sizes, strides;
  bool contiguous;
};

// Whether elements are at the same places: a dimension of one has any stride.
bool same_places(const Row& row, c10::IntArrayRef strides) {
  for (size_t d = 0; d < strides.size(); ++d)
    if (row.sizes[d] != 1 && row.strides[d] != strides[d]) return false;
  return true;
}

// A dense strided tensor of an allowed type on the device; `first`: of its
// row, whose others are laid out like it.
bool take(PyObject* o, c10::Device device, int allowed, bool first, Row& row, Column& c, size_t i,
          uint64_t& known) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!is_plain(t, known)) return false;
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  if (impl->device() != device) return false;
  const int type = type_of(t);
  if (type < 0 || !((allowed >> type) & 1)) return false;
  const bool contiguous = impl->is_contiguous();
  if (!contiguous && !impl->is_non_overlapping_and_dense()) return false;
  if (first) {
    row = Row{impl->sizes(), impl->strides(), contiguous};
  } else {
    if (impl->sizes() != row.sizes) return false;
    if (!(contiguous && row.contiguous) && !same_places(row, impl->strides())) return false;
  }
  // data_ptr(), without looking the element size up
  const c10::Storage& storage = impl->unsafe_storage();
  char* base = storage ? static_cast<char*>(storage.unsafeGetStorageImpl()->mutable_data()) : nullptr;
  c.type[i] = type;
  if (c.writes) c.note(impl);
  if (impl->numel() == 0) return true;
  if (base == nullptr) return false;
  c.ptr[i] = base + impl->storage_offset() * (type == MUON_DTYPE_F32 ? 4 : 2);
  return true;
}

// Paired lists; where the first holds None, the entry is skipped.
struct Lists {
  static constexpr int kMost = 4;
  PyObject* seq[kMost] = {};
  Column col[kMost];
  std::vector<int64_t> numel;
  int n = 0;
  int64_t total = 0;
  bool same_ = false;
  const Column& second() const { return col[same_ ? 0 : 1]; }
  ~Lists() {
    for (PyObject* s : seq) Py_XDECREF(s);
  }
  // `allowed` has every list's types; the lists from `first_written` on are written.
  bool read(PyObject* const* lists, const int* allowed, int count, int first_written, int64_t device_index) {
    const c10::Device device(at::kCUDA, (c10::DeviceIndex)device_index);
    same_ = count == 2 && lists[0] == lists[1];   // clipped in place
    if (same_) count = 1, first_written = 0;
    for (int k = first_written; k < count; ++k) col[k].writes = true;
    for (int k = 0; k < count; ++k) {
      seq[k] = PySequence_Fast(lists[k], "a list of tensors is needed");
      if (!seq[k]) {
        PyErr_Clear();
        return false;
      }
      if (PySequence_Fast_GET_SIZE(seq[k]) != PySequence_Fast_GET_SIZE(seq[0])) return false;
    }
    uint64_t known = 0;
    const Py_ssize_t size = PySequence_Fast_GET_SIZE(seq[0]);
    if (size > INT32_MAX) return false;
    n = (int)size;
    numel.assign((size_t)n, 0);
    for (int k = 0; k < count; ++k) col[k].resize((size_t)n);
    for (int i = 0; i < n; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(seq[0], i);
      if (o == Py_None) continue;
      Row row;
      if (!take(o, device, allowed[0], true, row, col[0], (size_t)i, known)) return false;
      total += numel[i] = THPVariable_Unpack(o).numel();
      for (int k = 1; k < count; ++k)
        if (!take(PySequence_Fast_GET_ITEM(seq[k], i), device, allowed[k], false, row, col[k], (size_t)i, known))
          return false;
    }
    return true;
  }
};

// Runs `body`, with C++ exceptions as Python ones.
template <class F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

bool want_args(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", want, got);
  return false;
}

muon_handle* handle_of(PyObject* o) { return static_cast<muon_handle*>(PyLong_AsVoidPtr(o)); }

// Results and scratch, from the memory of the stream that the call runs on.
struct Buffers {
  at::AutoDispatchBelowADInplaceOrView guard;   // plain tensors: nothing to record
  at::Tensor out, per, scratch;
  size_t bytes = 0;
  Buffers(int64_t device, const Lists& l, bool per_tensor) {
    const auto on = at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)device);
    out = at::empty({2}, on.dtype(at::kFloat));
    if (per_tensor) per = at::empty({l.n}, on.dtype(at::kFloat));
    if (l.n <= MUON_GRAD_SMALL_COUNT && l.total <= MUON_GRAD_SMALL_NUMEL) return;
    bytes = MUON_GRAD_SCRATCH_BYTES(l.n);
    scratch = at::empty({(int64_t)(bytes / 8)}, on.dtype(at::kDouble));
  }
  void* scratch_ptr() { return bytes ? scratch.data_ptr() : nullptr; }
};

// bind(norm, clip, adamw): addresses of the C functions.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args(n, 3)) return nullptr;
  c_norm = reinterpret_cast<decltype(c_norm)>(PyLong_AsVoidPtr(a[0]));
  c_clip = reinterpret_cast<decltype(c_clip)>(PyLong_AsVoidPtr(a[1]));
  c_adamw = reinterpret_cast<decltype(c_adamw)>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// grad_norm(handle, device, tensors, norm_kind, max_norm, per_tensor)
//   -> (norm, scale), (norm, scale, per_tensor), a status code, or None
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!want_args(nargs, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    muon_handle* h = handle_of(a[0]);
    const int64_t device = PyLong_AsLongLong(a[1]);
    const int kind = (int)PyLong_AsLong(a[3]);
    const double max_norm = PyFloat_AsDouble(a[4]);
    const bool per = PyObject_IsTrue(a[5]) == 1;
    if (PyErr_Occurred()) return nullptr;
    Lists l;
    const int allowed[1] = {kAny};
    if (!l.read(&a[2], allowed, 1, 1, device)) Py_RETURN_NONE;
    Buffers b(device, l, per);
    const int rc = c_norm(h, l.col[0].ptr.data(), l.numel.data(), l.col[0].type.data(), l.n, kind, max_norm,
                          b.out.data_ptr<float>(), per ? b.per.data_ptr<float>() : nullptr, b.scratch_ptr(),
                          b.bytes, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    if (rc) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(per ? 3 : 2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(b.out.select(0, 0)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b.out.select(0, 1)));
    if (per) PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(b.per));
    return r;
  });
}

// clip_grads(handle, device, grads, out, norm_kind, max_norm) -> norm, a status code, or None
PyObject* py_clip(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!want_args(nargs, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    muon_handle* h = handle_of(a[0]);
    const int64_t device = PyLong_AsLongLong(a[1]);
    const int kind = (int)PyLong_AsLong(a[4]);
    const double max_norm = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return nullptr;
    Lists l;
    const int allowed[2] = {kAny, kAny};
    if (!l.read(&a[2], allowed, 2, 1, device)) Py_RETURN_NONE;
    Buffers b(device, l, false);
    const int rc = c_clip(h, l.col[0].ptr.data(), l.second().ptr.data(), l.numel.data(), l.col[0].type.data(),
                          l.second().type.data(), l.n, kind, max_norm, b.out.data_ptr<float>(), b.scratch_ptr(),
                          b.bytes, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    if (rc) return PyLong_FromLong(rc);
    l.second().written();
    return THPVariable_Wrap(b.out.select(0, 0));
  });
}

// The address of a CUDA tensor of one element of a type; false: it is not that.
bool one_element(PyObject* o, int64_t device, at::ScalarType type, void** p) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  uint64_t known = 0;
  if (!is_plain(t, known) || t.get_device() != device || t.scalar_type() != type || t.numel() != 1) return false;
  *p = t.data_ptr();
  return true;
}

// adamw_step(handle, device, grads, params, exp_avgs, exp_avg_sqs, lr, beta1, beta2, eps, wd, step, grad_scale)
//   -> a status code, or None; step is an int or a tensor, grad_scale a tensor or None
PyObject* py_adamw(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (!want_args(nargs, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    muon_handle* h = handle_of(a[0]);
    const int64_t device = PyLong_AsLongLong(a[1]);
    double x[5];
    for (int k = 0; k < 5; ++k) x[k] = PyFloat_AsDouble(a[6 + k]);
    if (PyErr_Occurred()) return nullptr;
    int64_t step = 0;
    void *step_dev = nullptr, *scale = nullptr;
    if (!one_element(a[11], device, at::kLong, &step_dev)) {
      if (THPVariable_Check(a[11])) Py_RETURN_NONE;
      step = PyLong_AsLongLong(a[11]);
      if (PyErr_Occurred()) return nullptr;
    }
    if (a[12] != Py_None && !one_element(a[12], device, at::kFloat, &scale)) Py_RETURN_NONE;
    Lists l;
    const int allowed[4] = {kAny, kF32, kF32, kF32};
    if (!l.read(&a[2], allowed, 4, 1, device)) Py_RETURN_NONE;
    const auto f = [&](int k) { return reinterpret_cast<float* const*>(l.col[k].ptr.data()); };
    const int rc = c_adamw(h, f(1), l.col[0].ptr.data(), f(2), f(3), l.numel.data(), l.col[0].type.data(), l.n, x[0],
                           x[1], x[2], x[3], x[4], step, static_cast<const int64_t*>(step_dev),
                           static_cast<const float*>(scale),
                           c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    if (!rc)
      for (int k = 1; k < 4; ++k) l.col[k].written();
    return PyLong_FromLong(rc);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(py_bind), nullptr},
                         {"grad_norm", FAST(py_norm), nullptr},
                         {"clip_grads", FAST(py_clip), nullptr},
                         {"adamw_step", FAST(py_adamw), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists(void) { return PyModule_Create(&module); }
