// Python binding of the 4-bit cache's calls.  A decode step is a few
// microseconds on the device; marshalled from Python it costs the host twice
// that, so these calls check their tensors and find the stream, the output and
// the workspace here.  The C ABI does the work; its status goes to `raise`, a
// Python callable that turns it into an exception.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <mutex>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/plsh.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, int dev, const char* what) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw Refused(std::string(what) + " must be on the current CUDA device");
}

plsh_tensor rows(const at::Tensor& t, int dev, const char* what) {
  on_device(t, dev, what);
  if (t.dim() != 4) throw Refused(std::string(what) + " must be [B, H, n, d]");
  if (!t.is_contiguous()) throw Refused(std::string(what) + " must be contiguous");
  const auto dt = t.scalar_type();
  if (dt != at::kFloat && dt != at::kBFloat16)
    throw Refused(std::string(what) + ": dtype must be float32 or bfloat16");
  return plsh_tensor{t.data_ptr(), dt == at::kFloat ? PLSH_F32 : PLSH_BF16,
                     t.size(0), t.size(1), t.size(2), t.size(3)};
}

const int32_t* indices(PyObject* o, const plsh_q4_cache& c, int dev, const char* what) {
  const at::Tensor& t = tensor(o, what);
  on_device(t, dev, what);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != c.B || !t.is_contiguous())
    throw Refused(std::string(what) + " must be a contiguous int32 tensor of B = " +
                  std::to_string(c.B) + " entries");
  return static_cast<const int32_t*>(t.data_ptr());
}

// The cache's descriptor (a plsh_q4_cache as bytes) and its device, which must
// be the current one.
struct Call {
  plsh_q4_cache cache;
  int dev;
  std::optional<c10::cuda::CUDAStream> given;     // the stream, if the caller named one
  Call(PyObject* packed, PyObject* device, PyObject* stream) {
    if (!PyBytes_Check(packed) || PyBytes_GET_SIZE(packed) != (Py_ssize_t)sizeof cache)
      throw Refused("not a cache");
    memcpy(&cache, PyBytes_AS_STRING(packed), sizeof cache);
    dev = (int)PyLong_AsLong(device);
    if (dev != (int)c10::cuda::current_device())
      throw Refused("the cache is not on the current CUDA device");
    if (stream != Py_None) {
      void* h = PyLong_AsVoidPtr(stream);
      if (PyErr_Occurred()) throw Refused("stream must be a handle");
      given = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(h), (c10::DeviceIndex)dev);
    }
  }
  void* stream() const {
    return given ? given->stream() : c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

PyObject* g_raise = nullptr;

// Runs f with the interpreter released; a status becomes an exception.
template <typename F>
bool ran(F f) {
  plsh_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS if (st == PLSH_OK) return true;
  PyObject* r = PyObject_CallFunction(g_raise, "i", (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "plsh call failed");
  return false;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// write(cache, device, K, V, pos, lens | None, stream | None)
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a[0], a[1], a[6]);
    const plsh_tensor K = rows(tensor(a[2], "K"), c.dev, "K"), V = rows(tensor(a[3], "V"), c.dev, "V");
    const int32_t* pos = indices(a[4], c.cache, c.dev, "pos");
    const int32_t* len = a[5] == Py_None ? nullptr : indices(a[5], c.cache, c.dev, "lens");
    void* st = c.stream();
    if (!ran([&] { return plsh_q4_cache_write(&K, &V, &c.cache, pos, len, st); })) return nullptr;
    Py_RETURN_NONE;
  });
}

// read(cache, device, K, V, pos, lens | None, stream | None)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a[0], a[1], a[6]);
    plsh_tensor K = rows(tensor(a[2], "K"), c.dev, "K"), V = rows(tensor(a[3], "V"), c.dev, "V");
    const int32_t* pos = indices(a[4], c.cache, c.dev, "pos");
    const int32_t* len = a[5] == Py_None ? nullptr : indices(a[5], c.cache, c.dev, "lens");
    void* st = c.stream();
    if (!ran([&] { return plsh_q4_cache_read(&c.cache, pos, len, &K, &V, st); })) return nullptr;
    Py_RETURN_NONE;
  });
}

// The call's workspace: `kept`, a dict of the cache, has one for each stream
// that is current when a call is made (calls on a stream run one after the
// other; g_launch keeps the launches of two threads' calls apart); a call that
// is captured, or given a stream, takes one of its own, so that graphs that
// replay at once share none.
std::mutex g_launch;
at::Tensor workspace(const Call& c, const plsh_tensor& q, const at::Tensor& like, PyObject* kept) {
  const bool own = c.given.has_value() || c10::cuda::currentStreamCaptureStatusMayInitCtx() !=
                                              c10::cuda::CaptureStatus::None;
  PyObject* key = nullptr;
  if (!own) {
    key = PyLong_FromVoidPtr(c.stream());
    if (key == nullptr) throw Refused("stream handle");
    if (PyObject* w = PyDict_GetItemWithError(kept, key)) {
      Py_DECREF(key);
      return tensor(w, "work");
    }
  }
  int64_t bytes = 0;
  if (!ran([&] { return plsh_q4_decode_work_bytes(&q, &c.cache, &bytes); })) {
    Py_XDECREF(key);
    throw Refused("work");
  }
  at::Tensor w;
  {
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (c.given) guard.reset_stream(*c.given);
    w = at::empty({bytes}, like.options().dtype(at::kByte).requires_grad(false));
  }
  if (!own) {
    PyObject* o = THPVariable_Wrap(w);
    const int bad = o == nullptr ? -1 : PyDict_SetItem(kept, key, o);
    Py_XDECREF(o);
    Py_DECREF(key);
    if (bad) throw Refused("workspace");
  }
  return w;
}

// decode(cache, device, kept, q, bins handle | scales as bytes, pos,
//        out | None, work | None, stream | None) -> o
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Call c(a[0], a[1], a[8]);
    const at::Tensor& q = tensor(a[3], "q");
    const plsh_tensor tq = rows(q, c.dev, "q");
    const int32_t* pos = indices(a[5], c.cache, c.dev, "pos");
    const bool exact = PyBytes_Check(a[4]);
    if (exact && PyBytes_GET_SIZE(a[4]) != (Py_ssize_t)(tq.H * sizeof(double)))
      throw Refused("sigma must hold a scale per query head");
    const void* bins = exact ? nullptr : PyLong_AsVoidPtr(a[4]);
    if (PyErr_Occurred()) return nullptr;
    at::Tensor w;
    if (a[7] == Py_None) {
      if (!PyDict_Check(a[2])) throw Refused("not a cache");
      w = workspace(c, tq, q, a[2]);
    } else {
      w = tensor(a[7], "work");
      on_device(w, c.dev, "work");
      if (!w.is_contiguous()) throw Refused("work must be contiguous");
    }
    PyObject* result;
    plsh_tensor to;
    if (a[6] == Py_None) {
      c10::cuda::OptionalCUDAStreamGuard guard;
      if (c.given) guard.reset_stream(*c.given);
      const at::Tensor o = at::detail::empty_cuda(q.sizes(), q.scalar_type(), q.device(), std::nullopt);
      to = tq;
      to.data = o.data_ptr();
      result = THPVariable_Wrap(o);
      if (result == nullptr) return nullptr;
    } else {
      to = rows(tensor(a[6], "out"), c.dev, "out");
      result = a[6];
      Py_INCREF(result);
    }
    void* st = c.stream();
    void* work = w.data_ptr();
    const int64_t bytes = (int64_t)w.nbytes();
    const double* sigma = exact ? reinterpret_cast<const double*>(PyBytes_AS_STRING(a[4])) : nullptr;
    const bool ok = ran([&] {
      // a call's kernels follow one another on the stream, with no other call's
      // between them that writes the same workspace
      const std::lock_guard<std::mutex> hold(g_launch);
      return exact ? plsh_alibi_exact_decode_q4(&tq, &c.cache, sigma, pos, &to, work, bytes, st)
                   : plsh_alibi_decode_q4(&tq, &c.cache, static_cast<const plsh_bins*>(bins), pos, &to,
                                          work, bytes, st);
    });
    if (ok) return result;
    Py_DECREF(result);
    return nullptr;
  });
}

PyObject* set_raise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_raise, f);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"set_raise", set_raise, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_plsh_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__plsh_binding() { return PyModule_Create(&kModule); }
