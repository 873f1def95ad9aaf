// Argument marshalling of the Python binding: one native call checks a tensor and returns
// its address.  The attribute reads behind such a check cost about 0.6 us in Python, and a
// call over every layer's cache makes one per layer: more than the launch that follows.
// The short calls of a speculative step are marshalled whole and made from here (a ctypes
// call of 14 arguments costs 1 us more).  Nothing here computes, or keeps anything between
// calls but the addresses of the library's functions.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <string>

#include "../../include/mla.h"

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

// A contiguous vector of n elements, as cuda_tensor.
const at::Tensor* cuda_vector(PyObject* o, const char* name, int64_t type, int64_t dev, int64_t n) {
  const at::Tensor* t = cuda_tensor(o, name, type, dev);
  if (!t) return nullptr;
  if (t->dim() != 1 || t->size(0) != n) {
    value_error(std::string(name) + " must have shape " + text({n}) + ", got " + text(t->sizes()));
    return nullptr;
  }
  if (!t->is_contiguous()) {
    value_error(std::string(name) + " must be contiguous");
    return nullptr;
  }
  return t;
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

void* current_stream(int64_t dev) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// A new tensor whose memory belongs to the stream that the call runs on: torch's allocator
// hands out what was freed on the same stream, so neither an earlier owner's work nor a later
// one's can be under way on another.
at::Tensor empty_on(at::IntArrayRef shape, int64_t type, int64_t dev, void* stream) {
  const auto options = at::TensorOptions().dtype(kTypes[type]).device(at::kCUDA, dev);
  if (stream == current_stream(dev)) return at::empty(shape, options);
  const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(
      static_cast<cudaStream_t>(stream), static_cast<c10::DeviceIndex>(dev)));
  return at::empty(shape, options);
}

// A stream argument: its handle, or None for the device's current stream.
bool stream_of(PyObject* o, int64_t dev, void** s) {
  if (o == Py_None) {
    *s = current_stream(dev);
    return true;
  }
  int64_t v;
  if (!integer(o, &v)) return false;
  *s = reinterpret_cast<void*>(v);
  return true;
}

// empty(type, dev, shape, stream) -> a new tensor for a call on the stream
PyObject* py_empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 4)) return nullptr;
    int64_t type, dev, shape[4];
    const Py_ssize_t dims = PyTuple_Size(a[2]);
    if (!integer(a[0], &type) || !integer(a[1], &dev) || dims < 0) return nullptr;
    if (dims > 4) return value_error("at most four dimensions");
    for (Py_ssize_t i = 0; i < dims; ++i)
      if (!integer(PyTuple_GET_ITEM(a[2], i), &shape[i])) return nullptr;
    void* stream;
    if (!stream_of(a[3], dev, &stream)) return nullptr;
    return THPVariable_Wrap(empty_on(at::IntArrayRef(shape, dims), type, dev, stream));
  });
}

int64_t current_device() { return c10::cuda::device_count() > 0 ? c10::cuda::current_device() : -1; }

// device() -> the current CUDA device, -1 on a machine without one
PyObject* py_device(PyObject*, PyObject*) {
  return guarded([] { return PyLong_FromLongLong(current_device()); });
}

// stream(dev) -> handle of torch's current stream of the device
PyObject* py_stream(PyObject*, PyObject* o) {
  return guarded([&]() -> PyObject* {
    int64_t dev;
    if (!integer(o, &dev)) return nullptr;
    return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(current_stream(dev)));
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

// ------------------------------------------------------------------ whole calls
// The library's functions, as the binding loaded it.
decltype(&mla_verify_tree) g_verify = nullptr;
decltype(&mla_compact_kv) g_compact = nullptr;
decltype(&mla_copy_pages) g_copy = nullptr;

// bind(verify_tree, compact_kv, copy_pages): their addresses
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t at[3];
  if (!arity(n, 3) || !integer(a[0], &at[0]) || !integer(a[1], &at[1]) || !integer(a[2], &at[2])) return nullptr;
  g_verify = reinterpret_cast<decltype(g_verify)>(at[0]);
  g_compact = reinterpret_cast<decltype(g_compact)>(at[1]);
  g_copy = reinterpret_cast<decltype(g_copy)>(at[2]);
  Py_RETURN_NONE;
}

bool bound() {
  if (g_verify && g_compact && g_copy) return true;
  PyErr_SetString(PyExc_RuntimeError, "the library's functions are not bound");
  return false;
}

mla_plan_t plan_of(int64_t handle) { return reinterpret_cast<mla_plan_t>(handle); }

// A [T, vocab] matrix of float32 or bfloat16 whose rows are contiguous and apart; `type`
// and `vocab` receive the first one's and bind the next (type < 0, vocab < 0: not known).
const at::Tensor* probabilities(PyObject* o, const char* name, int64_t dev, int64_t T, int64_t* type, int64_t* vocab,
                                int64_t* pitch) {
  if (*type < 0) {
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.dim() == 2 && t.size(1) > 0) {
        *type = t.scalar_type() == at::kBFloat16 ? 0 : t.scalar_type() == at::kFloat ? 1 : -1;
        *vocab = t.size(1);
      }
    }
    if (*type < 0) {
      value_error(std::string(name) + " must be a [T, vocab] tensor of float32 or bfloat16");
      return nullptr;
    }
  }
  const at::Tensor* t = cuda_tensor(o, name, *type, dev);
  if (!t) return nullptr;
  if (t->dim() != 2 || t->size(0) != T || t->size(1) != *vocab) {
    value_error(std::string(name) + " must have shape " + text({T, *vocab}) + ", got " + text(t->sizes()));
    return nullptr;
  }
  if ((*vocab > 1 && t->stride(1) != 1) || (T > 1 && t->stride(0) < *vocab)) {
    value_error(std::string(name) + " must have contiguous rows");
    return nullptr;
  }
  *pitch = T > 1 ? t->stride(0) : *vocab;
  return t;
}

// verify_tree(plan, T, B, draft_tokens, target, uniform, uniform_next, draft, accept_index,
// num_accepted, next_token, stream) -> (status, accept_index, num_accepted, next_token).
// Outputs that are None are made, as parts of one allocation (three took a third of the
// call).
PyObject* py_verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t plan, T, B;
    if (!bound() || !arity(n, 12) || !integer(a[0], &plan) || !integer(a[1], &T) || !integer(a[2], &B)) return nullptr;
    const int64_t dev = current_device();
    int64_t type = -1, vocab = -1, ld_target = 0, ld_draft = 0;
    const at::Tensor* target = probabilities(a[4], "target_probs", dev, T, &type, &vocab, &ld_target);
    const at::Tensor* draft = nullptr;
    if (!target) return nullptr;
    if (a[7] != Py_None && !(draft = probabilities(a[7], "draft_probs", dev, T, &type, &vocab, &ld_draft)))
      return nullptr;
    const at::Tensor* tokens = cuda_vector(a[3], "draft_tokens", 2, dev, T);
    const at::Tensor* uniform = tokens ? cuda_vector(a[5], "uniform", 1, dev, T) : nullptr;
    const at::Tensor* next = uniform ? cuda_vector(a[6], "uniform_next", 1, dev, B) : nullptr;
    if (!next) return nullptr;
    static const char* const kNames[] = {"accept_index", "num_accepted", "next_token"};
    const int64_t size[] = {T, B, B}, from[] = {0, T, T + B};
    void* stream;
    if (!stream_of(a[11], dev, &stream)) return nullptr;
    at::Tensor made, out[3];
    for (int i = 0; i < 3; ++i) {
      if (a[8 + i] != Py_None) {
        const at::Tensor* t = cuda_vector(a[8 + i], kNames[i], 2, dev, size[i]);
        if (!t) return nullptr;
        out[i] = *t;
        continue;
      }
      if (!made.defined()) made = empty_on({T + 2 * B}, 2, dev, stream);
      auto impl = made.unsafeGetTensorImpl()->shallow_copy_and_detach(c10::VariableVersion(0), true);
      impl->set_storage_offset(from[i]);
      impl->set_sizes_contiguous({size[i]});
      out[i] = at::Tensor(std::move(impl));
    }
    mla_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_verify(plan_of(plan), static_cast<const int32_t*>(tokens->data_ptr()), target->data_ptr(), ld_target,
                  draft ? draft->data_ptr() : nullptr, ld_draft, static_cast<int32_t>(std::min<int64_t>(vocab, INT32_MAX)),
                  type == 0 ? MLA_PROB_BF16 : MLA_PROB_FP32, static_cast<const float*>(uniform->data_ptr()),
                  static_cast<const float*>(next->data_ptr()), static_cast<int32_t*>(out[0].data_ptr()),
                  static_cast<int32_t*>(out[1].data_ptr()), static_cast<int32_t*>(out[2].data_ptr()), stream);
    Py_END_ALLOW_THREADS;
    THPObjectPtr items[3];
    for (int i = 0; i < 3; ++i) {
      items[i] = a[8 + i] == Py_None ? THPVariable_Wrap(out[i]) : Py_NewRef(a[8 + i]);
      if (!items[i]) return nullptr;
    }
    return Py_BuildValue("(iNNN)", static_cast<int>(st), items[0].release(), items[1].release(), items[2].release());
  });
}

// compact_kv(plan, T, B, pages, page, width, accept_index, num_accepted, caches, stream) ->
// status
PyObject* py_compact_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t plan, T, B;
    CacheShape want;
    if (!bound() || !arity(n, 10) || !integer(a[0], &plan) || !integer(a[1], &T) || !integer(a[2], &B) ||
        !integer(a[3], &want.pages) || !integer(a[4], &want.page) || !integer(a[5], &want.width))
      return nullptr;
    want.dev = current_device();
    THPObjectPtr caches(cache_addresses(a[8], want));
    if (!caches) return nullptr;
    const at::Tensor* acc = cuda_vector(a[6], "accept_index", 2, want.dev, T);
    const at::Tensor* cnt = acc ? cuda_vector(a[7], "num_accepted", 2, want.dev, B) : nullptr;
    void* stream;
    if (!cnt || !stream_of(a[9], want.dev, &stream)) return nullptr;
    mla_status st;
    void* const* list = reinterpret_cast<void* const*>(PyBytes_AS_STRING(caches.get()));
    const int32_t layers = static_cast<int32_t>(PyBytes_GET_SIZE(caches.get()) / 8);
    Py_BEGIN_ALLOW_THREADS;
    st = g_compact(plan_of(plan), static_cast<const int32_t*>(acc->data_ptr()),
                   static_cast<const int32_t*>(cnt->data_ptr()), list, layers, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

// A C-contiguous buffer of n int32, held until the object goes.
struct Table {
  Py_buffer b{};
  bool open(PyObject* o) { return PyObject_GetBuffer(o, &b, PyBUF_C_CONTIGUOUS) == 0; }
  const int32_t* data() const { return static_cast<const int32_t*>(b.buf); }
  ~Table() {
    if (b.obj) PyBuffer_Release(&b);
  }
};

// copy_pages(src, dst, tokens, caches, stream) -> status.  The tables are int32 arrays of
// one length (tokens may be None); the geometry is the first cache's.
PyObject* py_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Table src, dst, tokens;
    if (!bound() || !arity(n, 5) || !src.open(a[0]) || !dst.open(a[1]) || (a[2] != Py_None && !tokens.open(a[2])))
      return nullptr;
    const Py_ssize_t pairs = src.b.len / 4;
    if (dst.b.len != src.b.len || (tokens.b.obj && tokens.b.len != src.b.len) || pairs > INT32_MAX)
      return value_error("tables of different lengths");
    CacheShape want;
    want.dev = current_device();
    THPObjectPtr held;
    PyObject* first = a[3];
    if (!THPVariable_Check(first)) {
      const Py_ssize_t layers = PySequence_Size(a[3]);
      if (layers < 0) return nullptr;
      if (layers == 0) return PyLong_FromLong(MLA_OK);
      held = PySequence_GetItem(a[3], 0);
      first = held.get();
      if (!first) return nullptr;
    }
    int64_t dims = 0;
    if (THPVariable_Check(first)) {
      const at::Tensor& t = THPVariable_Unpack(first);
      if (t.dim() == 3 || (t.dim() == 4 && first == a[3])) {
        dims = t.dim();
        want.pages = t.size(dims - 3);
        want.page = t.size(dims - 2);
        want.width = t.size(dims - 1);
      }
    }
    if (dims == 0) return value_error("caches must be [num_pages, page_size, 512 + rope_dim]");
    THPObjectPtr caches(cache_addresses(a[3], want));
    void* stream;
    if (!caches || !stream_of(a[4], want.dev, &stream)) return nullptr;
    auto i32 = [](int64_t v) { return static_cast<int32_t>(std::min<int64_t>(v, INT32_MAX)); };
    const mla_dims d = {128, 512, i32(want.width - 512), i32(want.page), i32(want.pages), 1.f};
    mla_status st;
    void* const* list = reinterpret_cast<void* const*>(PyBytes_AS_STRING(caches.get()));
    const int32_t layers = static_cast<int32_t>(PyBytes_GET_SIZE(caches.get()) / 8);
    Py_BEGIN_ALLOW_THREADS;
    st = g_copy(&d, src.data(), dst.data(), tokens.b.obj ? tokens.data() : nullptr, static_cast<int32_t>(pairs), list,
                layers, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(st);
  });
}

PyMethodDef kMethods[] = {
    {"tensor", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_tensor)), METH_FASTCALL, nullptr},
    {"cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_cache)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_bind)), METH_FASTCALL, nullptr},
    {"verify_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_verify_tree)), METH_FASTCALL, nullptr},
    {"compact_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_compact_kv)), METH_FASTCALL, nullptr},
    {"copy_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_copy_pages)), METH_FASTCALL, nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_empty)), METH_FASTCALL, nullptr},
    {"device", py_device, METH_NOARGS, nullptr},
    {"stream", py_stream, METH_O, nullptr},
    {"address", py_address, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
