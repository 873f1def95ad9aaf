// Argument marshalling of the Python binding: one native call checks a tensor and returns
// its address.  The attribute reads behind such a check cost about 0.6 us in Python, and a
// call over every layer's cache makes one per layer: more than the launch that follows.
// Nothing here computes, launches or keeps anything between calls (at::empty apart, which
// allocates an output).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cstdint>
#include <exception>
#include <string>

namespace {

// dtype codes of the Python side
constexpr at::ScalarType kTypes[] = {at::kBFloat16, at::kFloat, at::kInt};
const char* const kTypeNames[] = {"torch.bfloat16", "torch.float32", "torch.int32"};

PyObject* value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  return nullptr;
}

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

bool integer(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}

// A CUDA tensor of the type and (dev >= 0) on the device, or null with a ValueError.
const at::Tensor* cuda_tensor(PyObject* o, const char* name, int64_t type, int64_t dev) {
  if (!THPVariable_Check(o)) {
    value_error(std::string(name) + " must be a CUDA tensor");
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    value_error(std::string(name) + " must be a CUDA tensor");
    return nullptr;
  }
  if (t.scalar_type() != kTypes[type]) {
    value_error(std::string(name) + " must be " + kTypeNames[type]);
    return nullptr;
  }
  if (dev >= 0 && t.get_device() != dev) {
    value_error(std::string(name) + " must be on the current device");
    return nullptr;
  }
  return &t;
}

PyObject* address_of(const at::Tensor& t) {
  return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t.data_ptr()));
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// tensor(t, name, type, dev, shape) -> address of a contiguous tensor of that shape
PyObject* py_tensor(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 5)) return nullptr;
    const char* name = PyUnicode_AsUTF8(a[1]);
    int64_t type, dev;
    if (!name || !integer(a[2], &type) || !integer(a[3], &dev)) return nullptr;
    const at::Tensor* t = cuda_tensor(a[0], name, type, dev);
    if (!t) return nullptr;
    const Py_ssize_t dims = PyTuple_Size(a[4]);
    if (dims < 0) return nullptr;
    bool same = t->dim() == dims;
    for (Py_ssize_t i = 0; same && i < dims; ++i) {
      int64_t want;
      if (!integer(PyTuple_GET_ITEM(a[4], i), &want)) return nullptr;
      same = t->size(i) == want;
    }
    if (!same) {
      PyObject* want = PyObject_Repr(a[4]);
      if (!want) return nullptr;
      const char* s = PyUnicode_AsUTF8(want);
      const std::string what = std::string(name) + " must have shape " + (s ? s : "") + ", got " + text(t->sizes());
      Py_DECREF(want);
      return value_error(what);
    }
    if (!t->is_contiguous()) return value_error(std::string(name) + " must be contiguous");
    return address_of(*t);
  });
}

// (address, pitch) of a checked [T, V] matrix whose rows must be contiguous and apart, or
// with the vocabulary and the type where `more`.
PyObject* matrix(const at::Tensor& t, const char* name, int64_t T, int64_t V, int more) {
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != V)
    return value_error(std::string(name) + " must have shape " + text({T, V}) + ", got " + text(t.sizes()));
  if ((V > 1 && t.stride(1) != 1) || (T > 1 && t.stride(0) < V))
    return value_error(std::string(name) + " must have contiguous rows");
  const unsigned long long at = reinterpret_cast<uintptr_t>(t.data_ptr());
  const long long pitch = T > 1 ? t.stride(0) : V;
  if (more >= 0) return Py_BuildValue("(KLLi)", at, pitch, static_cast<long long>(V), more);
  return Py_BuildValue("(KL)", at, pitch);
}

// rows(t, name, type, dev, tokens, vocab) -> (address, pitch)
PyObject* py_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 6)) return nullptr;
    const char* name = PyUnicode_AsUTF8(a[1]);
    int64_t type, dev, T, V;
    if (!name || !integer(a[2], &type) || !integer(a[3], &dev) || !integer(a[4], &T) || !integer(a[5], &V))
      return nullptr;
    const at::Tensor* t = cuda_tensor(a[0], name, type, dev);
    return t ? matrix(*t, name, T, V, -1) : nullptr;
  });
}

// probabilities(t, name, dev, tokens) -> (address, pitch, vocab, type) of a float32 or
// bfloat16 matrix
PyObject* py_probabilities(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 4)) return nullptr;
    const char* name = PyUnicode_AsUTF8(a[1]);
    int64_t dev, T;
    if (!name || !integer(a[2], &dev) || !integer(a[3], &T)) return nullptr;
    int type = -1;
    if (THPVariable_Check(a[0])) {
      const at::Tensor& t = THPVariable_Unpack(a[0]);
      if (t.dim() == 2 && t.size(1) > 0)
        type = t.scalar_type() == at::kBFloat16 ? 0 : t.scalar_type() == at::kFloat ? 1 : -1;
    }
    if (type < 0) return value_error(std::string(name) + " must be a [T, vocab] tensor of float32 or bfloat16");
    const at::Tensor* t = cuda_tensor(a[0], name, type, dev);
    return t ? matrix(*t, name, T, t->size(1), type) : nullptr;
  });
}

// A layer's cache: [>= pages, page, width] bf16, or (layers) with a leading dimension.
struct CacheShape {
  int64_t dev, pages, page, width;

  bool parse(PyObject* const* a) {
    return integer(a[0], &dev) && integer(a[1], &pages) && integer(a[2], &page) && integer(a[3], &width);
  }
  const at::Tensor* check(PyObject* o, int64_t dims) const {
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.dim() != dims || t.size(dims - 3) < pages || t.size(dims - 2) != page || t.size(dims - 1) != width) {
        value_error("cache must have shape (>= " + std::to_string(pages) + ", " + std::to_string(page) + ", " +
                    std::to_string(width) + ") (num_pages, page_size, 512 + rope_dim), got " + text(t.sizes()));
        return nullptr;
      }
    }
    const at::Tensor* t = cuda_tensor(o, "cache", 0, dev);
    if (t && !t->is_contiguous()) {
      value_error("cache must be contiguous");
      return nullptr;
    }
    return t;
  }
};

// cache(t, dev, pages, page, width) -> address of one layer's cache
PyObject* py_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    CacheShape want;
    if (!arity(n, 5) || !want.parse(a + 1)) return nullptr;
    const at::Tensor* t = want.check(a[0], 3);
    return t ? address_of(*t) : nullptr;
  });
}

// Addresses of the layers' caches: `o` is a sequence of caches, one cache, or one tensor
// with a leading layer dimension.
PyObject* cache_addresses(PyObject* o, const CacheShape& want) {
  if (THPVariable_Check(o)) {
    const int64_t dims = THPVariable_Unpack(o).dim() == 4 ? 4 : 3;
    const at::Tensor* t = want.check(o, dims);
    if (!t) return nullptr;
    const int64_t layers = dims == 4 ? t->size(0) : 1;
    PyObject* out = PyBytes_FromStringAndSize(nullptr, layers * 8);
    if (!out) return nullptr;
    uint64_t* p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(out));
    const uint64_t base = reinterpret_cast<uintptr_t>(t->data_ptr());
    const uint64_t step = layers > 0 ? static_cast<uint64_t>(t->numel() / layers) * 2 : 0;
    for (int64_t i = 0; i < layers; ++i) p[i] = base + i * step;
    return out;
  }
  PyObject* seq = PySequence_Fast(o, "caches must be a tensor or a sequence of tensors");
  if (!seq) return nullptr;
  const Py_ssize_t layers = PySequence_Fast_GET_SIZE(seq);
  PyObject* out = PyBytes_FromStringAndSize(nullptr, layers * 8);
  uint64_t* p = out ? reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(out)) : nullptr;
  for (Py_ssize_t i = 0; out && i < layers; ++i) {
    const at::Tensor* t = want.check(PySequence_Fast_GET_ITEM(seq, i), 3);
    if (t)
      p[i] = reinterpret_cast<uintptr_t>(t->data_ptr());
    else
      Py_CLEAR(out);
  }
  Py_DECREF(seq);
  return out;
}

// caches(c, dev, pages, page, width) -> bytes of the layers' addresses
PyObject* py_caches(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    CacheShape want;
    if (!arity(n, 5) || !want.parse(a + 1)) return nullptr;
    return cache_addresses(a[0], want);
  });
}

// pools(c, dev) -> (bytes of the layers' addresses, pages, page, width), by the first
// cache's shape; None where there is no cache
PyObject* py_pools(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    CacheShape want;
    if (!arity(n, 2) || !integer(a[1], &want.dev)) return nullptr;
    THPObjectPtr held;
    PyObject* first = a[0];
    if (!THPVariable_Check(first)) {
      const Py_ssize_t layers = PySequence_Size(a[0]);
      if (layers < 0) return nullptr;
      if (layers == 0) Py_RETURN_NONE;
      held = PySequence_GetItem(a[0], 0);
      first = held.get();
      if (!first) return nullptr;
    }
    int64_t dims = 0;
    if (THPVariable_Check(first)) {
      const at::Tensor& t = THPVariable_Unpack(first);
      dims = t.dim();
      if (dims == 3 || (dims == 4 && first == a[0])) {
        if (dims == 4 && t.size(0) == 0) Py_RETURN_NONE;
        want.pages = t.size(dims - 3);
        want.page = t.size(dims - 2);
        want.width = t.size(dims - 1);
      } else {
        dims = 0;
      }
    }
    if (dims == 0) return value_error("caches must be [num_pages, page_size, 512 + rope_dim]");
    PyObject* at = cache_addresses(a[0], want);
    if (!at) return nullptr;
    return Py_BuildValue("(NLLL)", at, static_cast<long long>(want.pages), static_cast<long long>(want.page),
                         static_cast<long long>(want.width));
  });
}

// empty(type, dev, shape) -> a new tensor
PyObject* py_empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 3)) return nullptr;
    int64_t type, dev, shape[4];
    const Py_ssize_t dims = PyTuple_Size(a[2]);
    if (!integer(a[0], &type) || !integer(a[1], &dev) || dims < 0) return nullptr;
    if (dims > 4) return value_error("at most four dimensions");
    for (Py_ssize_t i = 0; i < dims; ++i)
      if (!integer(PyTuple_GET_ITEM(a[2], i), &shape[i])) return nullptr;
    return THPVariable_Wrap(at::empty(at::IntArrayRef(shape, dims),
                                      at::TensorOptions().dtype(kTypes[type]).device(at::kCUDA, dev)));
  });
}

// empty_parts(type, dev, sizes) -> new one-dimensional tensors, parts of one allocation
PyObject* py_empty_parts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 3)) return nullptr;
    int64_t type, dev, sum = 0, size[8];
    const Py_ssize_t parts = PyTuple_Size(a[2]);
    if (!integer(a[0], &type) || !integer(a[1], &dev) || parts < 0) return nullptr;
    if (parts > 8) return value_error("at most eight parts");
    for (Py_ssize_t i = 0; i < parts; ++i) {
      if (!integer(PyTuple_GET_ITEM(a[2], i), &size[i])) return nullptr;
      sum += size[i];
    }
    const at::Tensor all = at::empty({sum}, at::TensorOptions().dtype(kTypes[type]).device(at::kCUDA, dev));
    PyObject* out = PyTuple_New(parts);
    int64_t from = 0;
    for (Py_ssize_t i = 0; out && i < parts; from += size[i++]) {
      auto impl = all.unsafeGetTensorImpl()->shallow_copy_and_detach(c10::VariableVersion(0), true);
      impl->set_storage_offset(from);
      impl->set_sizes_contiguous({size[i]});
      PyObject* t = THPVariable_Wrap(at::Tensor(std::move(impl)));
      if (t)
        PyTuple_SET_ITEM(out, i, t);
      else
        Py_CLEAR(out);
    }
    return out;
  });
}

// device() -> the current CUDA device, -1 on a machine without one
PyObject* py_device(PyObject*, PyObject*) {
  return guarded([] { return PyLong_FromLong(c10::cuda::device_count() > 0 ? c10::cuda::current_device() : -1); });
}

// stream(dev) -> handle of torch's current stream of the device
PyObject* py_stream(PyObject*, PyObject* o) {
  return guarded([&]() -> PyObject* {
    int64_t dev;
    if (!integer(o, &dev)) return nullptr;
    return PyLong_FromUnsignedLongLong(
        reinterpret_cast<uintptr_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()));
  });
}

// address(a) -> address of a C-contiguous array's data (valid while the array lives)
PyObject* py_address(PyObject*, PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_C_CONTIGUOUS) != 0) return nullptr;
  PyObject* r = PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(b.buf));
  PyBuffer_Release(&b);
  return r;
}

PyMethodDef kMethods[] = {
    {"tensor", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_tensor)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_rows)), METH_FASTCALL, nullptr},
    {"cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_cache)), METH_FASTCALL, nullptr},
    {"caches", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_caches)), METH_FASTCALL, nullptr},
    {"pools", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_pools)), METH_FASTCALL, nullptr},
    {"probabilities", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_probabilities)), METH_FASTCALL,
     nullptr},
    {"empty_parts", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_empty_parts)), METH_FASTCALL, nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_empty)), METH_FASTCALL, nullptr},
    {"device", py_device, METH_NOARGS, nullptr},
    {"stream", py_stream, METH_O, nullptr},
    {"address", py_address, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
