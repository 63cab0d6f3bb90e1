// marshal.cpp -- CPython helpers of the binding: argument checks, output allocation and the calls of the 8-bit block.
//
// A call of a few tokens is bound by the host.  Through ctypes and the Python-level checks add_rms_norm took 20-26 us for
// one token, its kernel 3: five outputs at 1.5 us each, four checks, fourteen argument conversions.  Here a check, an
// allocation and a whole call each are one C function: checks read the tensor directly, outputs come from the caching
// allocator without the dispatcher, and a call converts its arguments by the C prototype and adds the current stream.
// The entry points called are those of include/invmoe.h; nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/invmoe.h"

namespace {

// Element types by the codes the binding passes.
constexpr at::ScalarType kTypes[] = {at::kBFloat16, at::kFloat, at::kFloat8_e4m3fn, at::kInt, at::kByte};
constexpr const char* kTypeNames[] = {"torch.bfloat16", "torch.float32", "torch.float8_e4m3fn", "torch.int32",
                                      "torch.uint8"};
constexpr long kNumTypes = 5;
constexpr Py_ssize_t kMaxDims = 4;

bool parse_code(PyObject* o, long* code) {
  *code = PyLong_AsLong(o);
  if (*code == -1 && PyErr_Occurred()) return false;
  if (*code < 0 || *code >= kNumTypes) {
    PyErr_SetString(PyExc_ValueError, "unknown element type code");
    return false;
  }
  return true;
}

bool parse_dims(PyObject* const* args, Py_ssize_t n, int64_t* dims) {
  if (n > kMaxDims) {
    PyErr_SetString(PyExc_ValueError, "too many dimensions");
    return false;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    dims[i] = PyLong_AsLongLong(args[i]);
    if (dims[i] == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

std::string type_name(at::ScalarType t) {
  for (long i = 0; i < kNumTypes; ++i)
    if (kTypes[i] == t) return kTypeNames[i];
  return at::toString(t);
}

PyObject* refuse(const char* name, const std::string& what) {
  PyErr_SetString(PyExc_ValueError, (std::string(name) + " " + what).c_str());
  return nullptr;
}

// check(tensor, name, type code, dim...): a contiguous tensor of this type and shape on the current device; without dims
// any shape.
PyObject* check(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long code;
  int64_t dims[kMaxDims];
  if (n < 3 || !parse_code(args[2], &code) || !parse_dims(args + 3, n - 3, dims)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "check(tensor, name, code, *dims)");
    return nullptr;
  }
  const char* name = PyUnicode_AsUTF8(args[1]);
  if (name == nullptr) return nullptr;
  if (args[0] == Py_None) return refuse(name, "is required");
  if (!THPVariable_Check(args[0])) return refuse(name, "must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  if (!t.is_cuda()) return refuse(name, "must be a CUDA tensor");
  // the library launches on the current device: a pointer into another GPU's memory must not reach a kernel
  const int dev = c10::cuda::current_device();
  if (t.device().index() != dev)
    return refuse(name, "is on " + t.device().str() + ", but the current CUDA device is cuda:" + std::to_string(dev));
  if (t.scalar_type() != kTypes[code])
    return refuse(name, std::string("must be ") + kTypeNames[code] + ", got " + type_name(t.scalar_type()));
  if (!t.is_contiguous()) return refuse(name, "must be contiguous");
  const at::IntArrayRef want(dims, static_cast<size_t>(n - 3));
  if (n > 3 && t.sizes() != want)
    return refuse(name, "must have shape " + shape_text(want) + ", got " + shape_text(t.sizes()));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// new(like, type code, dim...): an uninitialised tensor on the device of `like`.
PyObject* new_tensor(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long code;
  int64_t dims[kMaxDims];
  if (n < 2 || !THPVariable_Check(args[0]) || !parse_code(args[1], &code) || !parse_dims(args + 2, n - 2, dims)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "new(tensor, code, *dims)");
    return nullptr;
  }
  return THPVariable_Wrap(at::Tensor(at::detail::empty_cuda(at::IntArrayRef(dims, static_cast<size_t>(n - 2)),
                                                            kTypes[code], THPVariable_Unpack(args[0]).device(),
                                                            std::nullopt)));
  END_HANDLE_TH_ERRORS
}

// One argument by its C type: a pointer from a tensor or None, the numbers from numbers.
template <class T>
bool convert(PyObject* o, T* out) {
  if constexpr (std::is_pointer_v<T>) {
    if (o == Py_None) {
      *out = nullptr;
      return true;
    }
    if (!THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "a pointer argument must be a tensor or None");
      return false;
    }
    *out = static_cast<T>(THPVariable_Unpack(o).data_ptr());
    return true;
  } else if constexpr (std::is_same_v<T, float>) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) return false;
    *out = static_cast<float>(d);
    return true;
  } else if constexpr (std::is_same_v<T, size_t>) {
    *out = PyLong_AsSize_t(o);
    return !(*out == static_cast<size_t>(-1) && PyErr_Occurred());
  } else {
    static_assert(std::is_same_v<T, int>, "argument type");
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
      PyErr_Format(PyExc_ValueError, "%lld does not fit a 32-bit argument", v);
      return false;
    }
    *out = static_cast<int>(v);
    return true;
  }
}

template <class... A, size_t... I>
PyObject* invoke(int (*f)(A...), PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
  // the last parameter is the stream
  if (n != static_cast<Py_ssize_t>(sizeof...(I))) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", static_cast<Py_ssize_t>(sizeof...(I)), n);
    return nullptr;
  }
  std::tuple<A...> a{};
  if (!(convert(args[I], &std::get<I>(a)) && ...)) return nullptr;
  std::get<sizeof...(I)>(a) = c10::cuda::getCurrentCUDAStream().stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = std::apply(f, a);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

template <class... A>
PyObject* invoke_all(int (*f)(A...), PyObject* const* args, Py_ssize_t n) {
  return invoke(f, args, n, std::make_index_sequence<sizeof...(A) - 1>{});
}

template <auto F>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return invoke_all(F, args, n);
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward_workspace_size(T, H)
PyObject* norm_backward_bytes(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int T = 0, H = 0;
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "rms_norm_backward_workspace_size(T, H)");
    return nullptr;
  }
  if (!convert(args[0], &T) || !convert(args[1], &H)) return nullptr;
  return PyLong_FromSize_t(rms_norm_backward_workspace_size(T, H));
}

#define METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
#define ENTRY(name) METHOD(#name, &call<&name>)

PyMethodDef methods[] = {
    METHOD("check", &check),
    METHOD("new", &new_tensor),
    ENTRY(moe_router_logits),
    ENTRY(moe_route_select),
    ENTRY(moe_route_select_backward),
    ENTRY(moe_router_backward),
    ENTRY(add_rms_norm),
    ENTRY(add_rms_norm_backward),
    METHOD("rms_norm_backward_workspace_size", &norm_backward_bytes),
    ENTRY(fp8_quantize),
    ENTRY(moe_permute_rows),
    ENTRY(moe_permute_fp8),
    ENTRY(fp8_gemm),
    ENTRY(moe_grouped_swiglu_fp8),
    ENTRY(moe_grouped_down_fp8),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
