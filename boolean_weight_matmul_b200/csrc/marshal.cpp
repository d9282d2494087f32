// Argument marshalling of the calls whose launches take less time than Python
// needs to hand them over: tensors are checked and unpacked here instead of
// attribute by attribute, and the C ABI (include/mbok.h) is called directly.
//
// Measured, host time of a call (ctypes and Python checks -> this module): see
// the binding's docstring.  The library itself is not linked: the binding loads
// it and passes the calls' addresses (bind), so that one loaded library serves
// both.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "mbok.h"

namespace {

#define MBOK_CALLS(X)        \
  X(mbok_gemv_gated)         \
  X(mbok_gemm_gated)         \
  X(mbok_gemm_backward)      \
  X(mbok_gated_backward)     \
  X(mbok_distill_loss)       \
  X(mbok_distill_backward)

struct Calls {
#define X(name) decltype(&::name) name = nullptr;
  MBOK_CALLS(X)
#undef X
};
Calls calls;

struct Failed {};   // a Python exception is set

// The arguments of one call, converted in order of use.  Every tensor must be a
// contiguous CUDA tensor on the current device: the library launches there, and
// a pointer into another GPU's memory would be dereferenced by its kernels.
class Args {
 public:
  Args(const char* name, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%s: %zd arguments, got %zd", name, want, n);
      throw Failed{};
    }
  }

  // A device pointer: of a tensor, an int as it is, None as NULL.
  template <class T>
  T* ptr(int i) {
    return static_cast<T*>(pointer(args_[i]));
  }
  template <class T>
  void ptrs(int i, T** out, int n) {
    items(i, n, [&](int k, PyObject* o) { out[k] = static_cast<T*>(pointer(o)); });
  }
  int integer(int i) { return to_int(args_[i]); }
  void integers(int i, int* out, int n) {
    items(i, n, [&](int k, PyObject* o) { out[k] = to_int(o); });
  }
  size_t size(int i) {
    PyObject* o = PyNumber_Index(args_[i]);
    if (o == nullptr) throw Failed{};
    const size_t v = PyLong_AsSize_t(o);
    Py_DECREF(o);
    if (v == size_t(-1) && PyErr_Occurred()) throw Failed{};
    return v;
  }
  float real(int i) {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return float(v);
  }
  // Bytes of a workspace tensor (0 for None).
  size_t bytes(int i) {
    if (args_[i] == Py_None) return 0;
    if (!THPVariable_Check(args_[i])) {
      PyErr_SetString(PyExc_TypeError, "a workspace is a tensor or None");
      throw Failed{};
    }
    return THPVariable_Unpack(args_[i]).nbytes();
  }
  // None: the current stream; an int: a cudaStream_t.
  void* stream(int i) {
    if (args_[i] == Py_None) return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device())).stream();
    return pointer(args_[i]);
  }

 private:
  int device() {
    if (device_ < 0) device_ = c10::cuda::current_device();
    return device_;
  }
  void* pointer(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "MBOK operates on CUDA tensors only");
        throw Failed{};
      }
      if (!t.is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "MBOK needs contiguous tensors");
        throw Failed{};
      }
      if (int(t.device().index()) != device()) {
        PyErr_Format(PyExc_ValueError,
                     "tensor on cuda:%d but the current device is cuda:%d; MBOK launches on the current device",
                     int(t.device().index()), device());
        throw Failed{};
      }
      return t.data_ptr();
    }
    if (PyLong_Check(o)) {
      void* p = PyLong_AsVoidPtr(o);
      if (p == nullptr && PyErr_Occurred()) throw Failed{};
      return p;
    }
    PyErr_Format(PyExc_TypeError, "expected a tensor, a raw device pointer or None, got %s", Py_TYPE(o)->tp_name);
    throw Failed{};
  }
  int to_int(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    if (v < INT_MIN || v > INT_MAX) {
      PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
      throw Failed{};
    }
    return int(v);
  }
  template <class F>
  void items(int i, int n, F take) {
    PyObject* seq = PySequence_Fast(args_[i], "expected a sequence");
    if (seq == nullptr) throw Failed{};
    struct Drop {
      PyObject* o;
      ~Drop() { Py_DECREF(o); }
    } drop{seq};
    if (PySequence_Fast_GET_SIZE(seq) != n) {
      PyErr_SetString(PyExc_ValueError, "one entry per matrix");
      throw Failed{};
    }
    for (int k = 0; k < n; ++k) take(k, PySequence_Fast_GET_ITEM(seq, k));
  }

  PyObject* const* args_;
  int device_ = -1;   // the current device, looked up once
};

// Runs `body` (which returns the status) and hands its status, or what it threw,
// to Python.
template <class F>
PyObject* guarded(F body) {
  try {
    return PyLong_FromLong(body());
  } catch (const Failed&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <class F>
int without_gil(F call) {
  int st = 0;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return st;
}

using u16 = uint16_t;
using u32 = uint32_t;

// packed_gate, alpha_gate, K_gate, packed_up, alpha_up, K_up, M, N, group, x, x_dtype, batch, h, h_dtype, workspace, stream
PyObject* gemv_gated(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("gemv_gated", v, n, 16);
    const u32 *pg = a.ptr<u32>(0), *pu = a.ptr<u32>(3);
    const u16 *ag = a.ptr<u16>(1), *au = a.ptr<u16>(4);
    const int kg = a.integer(2), ku = a.integer(5), M = a.integer(6), N = a.integer(7), group = a.integer(8);
    const void* x = a.ptr<void>(9);
    const int xd = a.integer(10), batch = a.integer(11), hd = a.integer(13);
    void *h = a.ptr<void>(12), *ws = a.ptr<void>(14), *s = a.stream(15);
    const size_t wsb = a.bytes(14);
    return without_gil([&] {
      return calls.mbok_gemv_gated(pg, ag, kg, pu, au, ku, M, N, group, x, xd, batch, h, hd, ws, wsb, s);
    });
  });
}

// packed_gate, alpha_gate, K_gate, packed_up, alpha_up, K_up, M, N, group, X, T, H, gate, up, workspace, stream
PyObject* gemm_gated(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("gemm_gated", v, n, 16);
    const u32 *pg = a.ptr<u32>(0), *pu = a.ptr<u32>(3);
    const u16 *ag = a.ptr<u16>(1), *au = a.ptr<u16>(4), *X = a.ptr<u16>(9);
    const int kg = a.integer(2), ku = a.integer(5), M = a.integer(6), N = a.integer(7), group = a.integer(8);
    const int T = a.integer(10);
    u16 *H = a.ptr<u16>(11), *G = a.ptr<u16>(12), *U = a.ptr<u16>(13);
    void *ws = a.ptr<void>(14), *s = a.stream(15);
    const size_t wsb = a.bytes(14);
    return without_gil([&] {
      return calls.mbok_gemm_gated(pg, ag, kg, pu, au, ku, M, N, group, X, T, H, G, U, ws, wsb, s);
    });
  });
}

// nseg, packed list, alpha list, K list, M list, N, group, X, T, dY list, dX, dalpha list, workspace, stream
PyObject* gemm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("gemm_backward", v, n, 14);
    constexpr int kMost = 8;   // the library's, which refuses more
    const int nseg = a.integer(0), held = nseg < 0 ? 0 : nseg > kMost ? kMost : nseg;
    u32* packed[kMost] = {};
    u16 *alpha[kMost] = {}, *dY[kMost] = {};
    float* dalpha[kMost] = {};
    int K[kMost] = {}, M[kMost] = {};
    if (held == nseg) {
      a.ptrs(1, packed, nseg);
      a.ptrs(2, alpha, nseg);
      a.integers(3, K, nseg);
      a.integers(4, M, nseg);
      a.ptrs(9, dY, nseg);
      a.ptrs(11, dalpha, nseg);
    }
    const int N = a.integer(5), group = a.integer(6), T = a.integer(8);
    const u16* X = a.ptr<u16>(7);
    u16* dX = a.ptr<u16>(10);
    void *ws = a.ptr<void>(12), *s = a.stream(13);
    const size_t wsb = a.bytes(12);
    return without_gil([&] {
      return calls.mbok_gemm_backward(nseg, packed, alpha, K, M, N, group, X, T, dY, dX, dalpha, ws, wsb, s);
    });
  });
}

// dH, gate, up, T, M, dgate, dup, H, stream
PyObject* gated_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("gated_backward", v, n, 9);
    const u16 *dH = a.ptr<u16>(0), *gate = a.ptr<u16>(1), *up = a.ptr<u16>(2);
    const int T = a.integer(3), M = a.integer(4);
    u16 *dg = a.ptr<u16>(5), *du = a.ptr<u16>(6), *H = a.ptr<u16>(7);
    void* s = a.stream(8);
    return without_gil([&] { return calls.mbok_gated_backward(dH, gate, up, T, M, dg, du, H, s); });
  });
}

// logits, dtype, T, V, ld, teacher, index, top, temperature, weight, loss, lse, dlogits, ld_dlogits, stream
PyObject* distill_loss(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("distill_loss", v, n, 15);
    const void* z = a.ptr<void>(0);
    const int dt = a.integer(1), T = a.integer(2), V = a.integer(3), top = a.integer(7);
    const size_t ld = a.size(4), ldz = a.size(13);
    const float *teacher = a.ptr<float>(5), *weight = a.ptr<float>(9);
    const int32_t* index = a.ptr<int32_t>(6);
    const float tau = a.real(8);
    float *loss = a.ptr<float>(10), *lse = a.ptr<float>(11);
    void *dz = a.ptr<void>(12), *s = a.stream(14);
    return without_gil([&] {
      return calls.mbok_distill_loss(z, dt, T, V, ld, teacher, index, top, tau, weight, loss, lse, dz, ldz, s);
    });
  });
}

// logits, dtype, T, V, ld, teacher, index, top, temperature, weight, lse, grad, dlogits, ld_dlogits, stream
PyObject* distill_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&] {
    Args a("distill_backward", v, n, 15);
    const void* z = a.ptr<void>(0);
    const int dt = a.integer(1), T = a.integer(2), V = a.integer(3), top = a.integer(7);
    const size_t ld = a.size(4), ldz = a.size(13);
    const float *teacher = a.ptr<float>(5), *weight = a.ptr<float>(9), *lse = a.ptr<float>(10), *grad = a.ptr<float>(11);
    const int32_t* index = a.ptr<int32_t>(6);
    const float tau = a.real(8);
    void *dz = a.ptr<void>(12), *s = a.stream(14);
    return without_gil([&] {
      return calls.mbok_distill_backward(z, dt, T, V, ld, teacher, index, top, tau, weight, lse, grad, dz, ldz, s);
    });
  });
}

// bind({name: address}): the loaded library's calls.
PyObject* bind(PyObject*, PyObject* addresses) {
  Calls c;
#define X(name)                                                                                      \
  {                                                                                                  \
    PyObject* at = PyMapping_GetItemString(addresses, #name);                                        \
    if (at == nullptr) return nullptr;                                                               \
    c.name = reinterpret_cast<decltype(c.name)>(PyLong_AsVoidPtr(at));                               \
    Py_DECREF(at);                                                                                   \
    if (c.name == nullptr) {                                                                         \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address for " #name);             \
      return nullptr;                                                                                \
    }                                                                                                \
  }
  MBOK_CALLS(X)
#undef X
  calls = c;
  Py_RETURN_NONE;
}

#define MBOK_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         MBOK_METHOD(gemv_gated),
                         MBOK_METHOD(gemm_gated),
                         MBOK_METHOD(gemm_backward),
                         MBOK_METHOD(gated_backward),
                         MBOK_METHOD(distill_loss),
                         MBOK_METHOD(distill_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
