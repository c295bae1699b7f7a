// fp8_binding.cpp — the Python binding of the 8-bit floating point operators (include/fp8.h): argument
// marshalling only, for torch CUDA tensors, on the current stream of their device.
//
// These are calls of a few microseconds of which a decoding step makes many, one after the other.
// Through ctypes, with the tensors' attributes read in Python, a call spent 6 to 8 us on the host,
// more than its kernel on the GPU; here it spends about as much as the launch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdarg>
#include <cstdio>
#include <optional>

#include "../../include/fp8.h"

namespace {

PyObject* g_error = nullptr;  // the package's GPTQError

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const char* format, ...) {
  char text[320];
  va_list ap;
  va_start(ap, format);
  vsnprintf(text, sizeof text, format, ap);
  va_end(ap);
  PyErr_SetString(PyExc_ValueError, text);
  throw Raised{};
}

// The arguments of a call by position or name, in the order of `names`; null where an optional one
// is absent or None.
template <int N>
struct Args {
  PyObject* v[N] = {};

  Args(const char* fn, const char* const (&names)[N], int required, PyObject* const* args,
       Py_ssize_t nargs, PyObject* kwnames) {
    if (nargs > N) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, N, nargs);
      throw Raised{};
    }
    for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
    const Py_ssize_t named = kwnames == nullptr ? 0 : PyTuple_GET_SIZE(kwnames);
    for (Py_ssize_t i = 0; i < named; ++i) {
      PyObject* key = PyTuple_GET_ITEM(kwnames, i);
      int at = 0;
      while (at < N && PyUnicode_CompareWithASCIIString(key, names[at]) != 0) ++at;
      if (at == N || v[at] != nullptr) {
        PyErr_Format(PyExc_TypeError,
                     at == N ? "%s() got an unexpected keyword argument '%U'"
                             : "%s() got multiple values for argument '%U'",
                     fn, key);
        throw Raised{};
      }
      v[at] = args[nargs + i];
    }
    for (int i = 0; i < N; ++i) {
      if (v[i] == nullptr && i < required) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
        throw Raised{};
      }
      if (v[i] == Py_None) v[i] = nullptr;
    }
  }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (o == nullptr || !THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const at::Tensor& matrix2(PyObject* o, const char* name) {
  if (o == nullptr || !THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2)
    refuse("%s must be a tensor of 2 dims", name);
  return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  return t.get_device();
}

int float_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return GPTQ_BF16;
    case at::kHalf: return GPTQ_F16;
    case at::kFloat: return GPTQ_F32;
    default: refuse("%s must be bfloat16, float16 or float32, got %s", name, c10::toString(t.scalar_type()));
  }
}

// The leading dimension of a [rows, cols] tensor of device `dev` with unit stride along its rows. One
// row alone has no pitch: it counts as the next multiple of `pitch`.
int64_t leading(const at::Tensor& t, const char* name, int dev, int64_t rows, int64_t cols,
                int64_t pitch) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse("%s must be a CUDA tensor on device %d, is on %s", name, dev, t.device().str().c_str());
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) {
    char shape[128];
    int at = snprintf(shape, sizeof shape, "[");
    for (int64_t i = 0; i < t.dim() && at < 100; ++i)
      at += snprintf(shape + at, sizeof shape - at, i ? ", %lld" : "%lld", (long long)t.size(i));
    refuse("%s must be [%lld, %lld], got %s]", name, (long long)rows, (long long)cols, shape);
  }
  if (t.stride(1) != 1 && cols > 1) refuse("%s must have unit stride along its last dim", name);
  return rows > 1 ? t.stride(0) : (cols + pitch - 1) / pitch * pitch;
}
int64_t leading_e4m3(const at::Tensor& t, const char* name, int dev, int64_t rows, int64_t cols) {
  if (t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte)
    refuse("%s must be float8_e4m3fn or uint8, got %s", name, c10::toString(t.scalar_type()));
  return leading(t, name, dev, rows, cols, 16);
}
int64_t leading_scales(const at::Tensor& t, const char* name, int dev, int64_t rows, int64_t cols) {
  if (t.scalar_type() != at::kFloat)
    refuse("%s must be torch.float32, got %s", name, c10::toString(t.scalar_type()));
  return leading(t, name, dev, rows, cols, 1);
}

int32_t* status_of(PyObject* o, int dev) {
  if (o == nullptr) return nullptr;
  const at::Tensor& t = tensor(o, "dev_status");
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.numel() < 2 ||
      !t.is_contiguous())
    refuse("dev_status must be a contiguous int32 CUDA tensor of 2 entries on the operands' device");
  return static_cast<int32_t*>(t.data_ptr());
}

inline uint8_t* bytes(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }
inline float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }
inline int64_t blocks(int64_t v) { return (v + 127) / 128; }

// fn(stream) on the current stream of device `dev`, made current for the call.
template <typename F>
PyObject* launch(const char* name, int dev, F fn) {
  std::optional<c10::cuda::CUDAGuard> guard;
  if (c10::cuda::current_device() != dev) guard.emplace(static_cast<c10::DeviceIndex>(dev));
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev));
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(reinterpret_cast<gptq_stream_t>(stream));
  Py_END_ALLOW_THREADS;
  if (rc == GPTQ_OK) Py_RETURN_NONE;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", rc, name)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

PyObject* quantize(PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"X", "Q", "scales", "block_rows"};
  const Args<4> a("fp8_quantize", names, 3, args, nargs, kw);
  const at::Tensor& X = matrix2(a.v[0], "X");
  const long block_rows = a.v[3] == nullptr ? 1 : PyLong_AsLong(a.v[3]);
  if (block_rows == -1 && PyErr_Occurred()) throw Raised{};
  if (block_rows != 1 && block_rows != 128) refuse("block_rows must be 1 or 128");
  const int code = float_code(X, "X"), dev = device_of(X, "X");
  const at::Tensor &Q = tensor(a.v[1], "Q"), &S = tensor(a.v[2], "scales");
  const int64_t m = X.size(0), k = X.size(1);
  const int64_t ldx = leading(X, "X", dev, m, k, 8), ldq = leading_e4m3(Q, "Q", dev, m, k);
  const int64_t lds =
      leading_scales(S, "scales", dev, block_rows == 1 ? m : blocks(m), blocks(k));
  return launch("fp8_quantize", dev, [&](gptq_stream_t stream) {
    return fp8_quantize(X.data_ptr(), code, ldx, m, k, (int)block_rows, bytes(Q), ldq, floats(S),
                        lds, stream);
  });
}

PyObject* add_rmsnorm(PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"X", "R", "gamma", "eps", "H", "Q", "scales"};
  const Args<7> a("fp8_add_rmsnorm", names, 7, args, nargs, kw);
  const at::Tensor &X = matrix2(a.v[0], "X"), &gamma = tensor(a.v[2], "gamma");
  const int code = float_code(X, "X"), gcode = float_code(gamma, "gamma");
  const int dev = device_of(X, "X");
  if (a.v[3] == nullptr) refuse("eps must be a number");
  const double eps = PyFloat_AsDouble(a.v[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
  const int64_t m = X.size(0), k = X.size(1);
  const int64_t ldx = leading(X, "X", dev, m, k, 8);
  if (!gamma.is_cuda() || gamma.get_device() != dev || gamma.dim() != 1 || gamma.size(0) != k ||
      !gamma.is_contiguous())
    refuse("gamma must be a contiguous CUDA tensor of %lld entries on device %d", (long long)k, dev);
  const void* r = nullptr;
  void* h = nullptr;
  int64_t ldr = 0, ldh = 0;
  if (a.v[1] != nullptr) {
    const at::Tensor& R = tensor(a.v[1], "R");
    if (R.scalar_type() != X.scalar_type()) refuse("R must have X's dtype");
    ldr = leading(R, "R", dev, m, k, 8);
    r = R.data_ptr();
  }
  if (a.v[4] != nullptr) {
    const at::Tensor& H = tensor(a.v[4], "H");
    if (H.scalar_type() != X.scalar_type()) refuse("H must have X's dtype");
    ldh = leading(H, "H", dev, m, k, 8);
    h = H.data_ptr();
  }
  const at::Tensor &Q = tensor(a.v[5], "Q"), &S = tensor(a.v[6], "scales");
  const int64_t ldq = leading_e4m3(Q, "Q", dev, m, k);
  const int64_t lds = leading_scales(S, "scales", dev, m, blocks(k));
  return launch("fp8_add_rmsnorm", dev, [&](gptq_stream_t stream) {
    return fp8_add_rmsnorm(X.data_ptr(), ldx, r, ldr, code, gamma.data_ptr(), gcode, (float)eps, m,
                           k, h, ldh, bytes(Q), ldq, floats(S), lds, stream);
  });
}

PyObject* gemm(PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"X", "sx", "W", "sw", "Y", "dev_status"};
  const Args<6> a("fp8_gemm", names, 5, args, nargs, kw);
  const at::Tensor &X = matrix2(a.v[0], "X"), &W = matrix2(a.v[2], "W");
  const at::Tensor &sx = tensor(a.v[1], "sx"), &sw = tensor(a.v[3], "sw");
  const at::Tensor& Y = tensor(a.v[4], "Y");
  const int dev = device_of(X, "X");
  const int64_t m = X.size(0), k = X.size(1), n = W.size(0), g = blocks(k);
  const int64_t ldx = leading_e4m3(X, "X", dev, m, k), ldsx = leading_scales(sx, "sx", dev, m, g);
  const int64_t ldw = leading_e4m3(W, "W", dev, n, k);
  const int64_t ldsw = leading_scales(sw, "sw", dev, blocks(n), g);
  const int code = float_code(Y, "Y");
  const int64_t ldy = leading(Y, "Y", dev, m, n, 8);
  int32_t* status = status_of(a.v[5], dev);
  return launch("fp8_gemm", dev, [&](gptq_stream_t stream) {
    return fp8_gemm(bytes(X), ldx, floats(sx), ldsx, bytes(W), ldw, floats(sw), ldsw, m, n, k,
                    Y.data_ptr(), code, ldy, status, stream);
  });
}

PyObject* gated_gemm(PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"X", "sx", "Wg", "sg", "Wu", "su", "Q", "scales", "dev_status"};
  const Args<9> a("fp8_gated_gemm", names, 8, args, nargs, kw);
  const at::Tensor &X = matrix2(a.v[0], "X"), &Wg = matrix2(a.v[2], "Wg");
  const at::Tensor &sx = tensor(a.v[1], "sx"), &sg = tensor(a.v[3], "sg");
  const at::Tensor &Wu = tensor(a.v[4], "Wu"), &su = tensor(a.v[5], "su");
  const at::Tensor &Q = tensor(a.v[6], "Q"), &S = tensor(a.v[7], "scales");
  const int dev = device_of(X, "X");
  const int64_t m = X.size(0), k = X.size(1), n = Wg.size(0), g = blocks(k), gn = blocks(n);
  const int64_t ldx = leading_e4m3(X, "X", dev, m, k), ldsx = leading_scales(sx, "sx", dev, m, g);
  const int64_t ldg = leading_e4m3(Wg, "Wg", dev, n, k), ldsg = leading_scales(sg, "sg", dev, gn, g);
  const int64_t ldu = leading_e4m3(Wu, "Wu", dev, n, k), ldsu = leading_scales(su, "su", dev, gn, g);
  const int64_t ldq = leading_e4m3(Q, "Q", dev, m, n);
  const int64_t lds = leading_scales(S, "scales", dev, m, gn);
  int32_t* status = status_of(a.v[8], dev);
  return launch("fp8_gated_gemm", dev, [&](gptq_stream_t stream) {
    return fp8_gated_gemm(bytes(X), ldx, floats(sx), ldsx, bytes(Wg), ldg, floats(sg), ldsg,
                          bytes(Wu), ldu, floats(su), ldsu, m, n, k, bytes(Q), ldq, floats(S), lds,
                          status, stream);
  });
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t, PyObject*)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  try {
    return F(args, nargs, kw);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t, PyObject*)>
constexpr PyMethodDef method(const char* name, const char* doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)),
          METH_FASTCALL | METH_KEYWORDS, doc};
}

PyMethodDef g_methods[] = {
    method<quantize>("fp8_quantize",
                     "fp8_quantize(X, Q, scales, block_rows=1)\n--\n\n"
                     "Q, scales = X [m, k] as e4m3 with one fp32 scale per 1 x 128 (activations) or\n"
                     "128 x 128 (weights, block_rows=128) block."),
    method<add_rmsnorm>("fp8_add_rmsnorm",
                        "fp8_add_rmsnorm(X, R, gamma, eps, H, Q, scales)\n--\n\n"
                        "h = X + R; H = h (may be X or R itself); Q, scales = h / sqrt(mean(h^2) + eps)\n"
                        "* gamma as e4m3 with one scale per row and 128 columns. R and H may be None."),
    method<gemm>("fp8_gemm",
                 "fp8_gemm(X, sx, W, sw, Y, dev_status=None)\n--\n\n"
                 "Y [m, n] (bf16, fp16 or fp32) = X W^T of X [m, k] (blocks of 1 x 128, scales sx) and\n"
                 "W [n, k] (blocks of 128 x 128, scales sw)."),
    method<gated_gemm>("fp8_gated_gemm",
                       "fp8_gated_gemm(X, sx, Wg, sg, Wu, su, Q, scales, dev_status=None)\n--\n\n"
                       "Q, scales = silu(X Wg^T) * (X Wu^T) as e4m3 [m, n] with one scale per row and\n"
                       "128 columns; X as in fp8_gemm, Wg and Wu [n, k] as its W."),
    {"set_error", set_error, METH_O, "The exception raised where a call does not return GPTQ_OK."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8_binding",
                        "Binding of the 8-bit floating point operators of libgptq_b200.so.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// With the torch and the Python whose headers it was compiled against: it reads objects by their layout.
PyMODINIT_FUNC PyInit__fp8_binding() {
  PyObject* m = PyModule_Create(&g_module);
  char built_for[64];
  snprintf(built_for, sizeof built_for, "torch %s, Python %d.%d", TORCH_VERSION, PY_MAJOR_VERSION,
           PY_MINOR_VERSION);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", built_for) != 0) Py_CLEAR(m);
  return m;
}
