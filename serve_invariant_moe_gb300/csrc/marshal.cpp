// marshal.cpp -- CPython helpers of the binding: argument checks, output allocation and the calls of the 8-bit block.
//
// A call of a few tokens is bound by the host.  Through ctypes and the Python-level checks add_rms_norm took 20-26 us for
// one token, its kernel 3: five outputs at 1.5 us each, four checks, fourteen argument conversions.  Here a check, an
// allocation and a whole call each are one C function: checks read the tensor directly, outputs come from the caching
// allocator (through the dispatcher only where torch has something to do there), and a call converts its arguments by the C
// prototype and adds the current stream.  The norm's functions, which have most outputs, are C as a whole (one token 9.5 ->
// 6.4 us, of which five allocations are 3.5 and the launch 2.1; 2.9 with the caller's outputs; routing, with two outputs,
// would gain 0.3 of 4.7).
// The entry points called are those of include/invmoe.h; nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDACachingAllocator.h>
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

bool refuse(const char* name, const std::string& what) {
  PyErr_SetString(PyExc_ValueError, (std::string(name) + " " + what).c_str());
  return false;
}

// A contiguous tensor of this type and shape on the current device (any shape where `dims` is empty); else ValueError.
bool check_tensor(PyObject* o, const char* name, long code, at::IntArrayRef dims) {
  if (o == Py_None) return refuse(name, "is required");
  if (!THPVariable_Check(o)) return refuse(name, "must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) return refuse(name, "must be a CUDA tensor");
  // the library launches on the current device: a pointer into another GPU's memory must not reach a kernel
  const int dev = c10::cuda::current_device();
  if (t.device().index() != dev)
    return refuse(name, "is on " + t.device().str() + ", but the current CUDA device is cuda:" + std::to_string(dev));
  if (t.scalar_type() != kTypes[code])
    return refuse(name, std::string("must be ") + kTypeNames[code] + ", got " + type_name(t.scalar_type()));
  if (!t.is_contiguous()) return refuse(name, "must be contiguous");
  if (!dims.empty() && t.sizes() != dims)
    return refuse(name, "must have shape " + shape_text(dims) + ", got " + shape_text(t.sizes()));
  return true;
}

// check(tensor, name, type code, dim...)
PyObject* check(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long code;
  int64_t dims[kMaxDims];
  if (n < 3 || !parse_code(args[2], &code) || !parse_dims(args + 3, n - 3, dims)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "check(tensor, name, code, *dims)");
    return nullptr;
  }
  const char* name = PyUnicode_AsUTF8(args[1]);
  if (name == nullptr || !check_tensor(args[0], name, code, at::IntArrayRef(dims, static_cast<size_t>(n - 3))))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// On the current device, which is that of every input checked before: no device guard, 0.13 us less of 0.8.  Where a
// dispatch mode is on, or uninitialised memory is to be filled, by the dispatcher, as torch.empty would.
PyObject* new_output(long code, at::IntArrayRef dims) {
  const at::Context& ctx = at::globalContext();
  if (c10::impl::dispatch_mode_enabled() || (ctx.deterministicAlgorithms() && ctx.deterministicFillUninitializedMemory()))
    return THPVariable_Wrap(at::empty(dims, at::TensorOptions().dtype(kTypes[code]).device(at::kCUDA)));
  return THPVariable_Wrap(at::Tensor(at::detail::empty_generic(dims, c10::cuda::CUDACachingAllocator::get(),
                                                               c10::DispatchKeySet(c10::DispatchKey::CUDA), kTypes[code],
                                                               std::nullopt)));
}

// new(like, type code, dim...): an uninitialised tensor on the device of `like`, a checked input (so the current one).
PyObject* new_tensor(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long code;
  int64_t dims[kMaxDims];
  if (n < 2 || !THPVariable_Check(args[0]) || !parse_code(args[1], &code) || !parse_dims(args + 2, n - 2, dims)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "new(tensor, code, *dims)");
    return nullptr;
  }
  return new_output(code, at::IntArrayRef(dims, static_cast<size_t>(n - 2)));
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

// A reference that is dropped with its scope.
struct Ref {
  PyObject* o = nullptr;
  Ref() = default;
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(o); }
  void* data() const { return o == nullptr || o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }
};

enum Given { kSkip, kNew, kTaken };   // an output argument: False, None or True, a tensor

Given given(PyObject* o) { return o == Py_False ? kSkip : o == Py_None || o == Py_True ? kNew : kTaken; }

// An output: the caller's tensor after the usual checks, or a new one.
bool output(PyObject* o, const char* name, long code, at::IntArrayRef dims, Ref* out) {
  if (given(o) != kNew) {                  // what may be skipped has been
    if (!check_tensor(o, name, code, dims)) return false;
    Py_INCREF(o);
    out->o = o;
  } else {
    out->o = new_output(code, dims);
  }
  return out->o != nullptr;
}

void none(Ref* out) {
  Py_INCREF(Py_None);
  out->o = Py_None;
}

// [T, H] of a tensor, and its type's code, which must be that of bf16 or fp32.
bool matrix(PyObject* o, const char* name, int* T, int* H, int* code) {
  if (!THPVariable_Check(o)) return refuse(name, "must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 2) return refuse(name, "must have 2 dimensions, got shape " + shape_text(t.sizes()));
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) return refuse(name, "does not fit 32-bit sizes");
  if (t.scalar_type() != kTypes[0] && t.scalar_type() != kTypes[1])
    return refuse(name, "must be torch.bfloat16 or torch.float32, got " + type_name(t.scalar_type()));
  *T = static_cast<int>(t.size(0));
  *H = static_cast<int>(t.size(1));
  *code = t.scalar_type() == kTypes[0] ? 0 : 1;
  return true;
}

template <size_t N>
PyObject* dict_of(const char* const (&names)[N], const Ref* const (&values)[N]) {
  PyObject* d = PyDict_New();
  for (size_t i = 0; d != nullptr && i < N; ++i)
    if (PyDict_SetItemString(d, names[i], values[i]->o) != 0) Py_CLEAR(d);
  return d;
}

// norm(x, weight, residual, eps, out, fp8, residual_out, q, scale, rstd): the whole call of the binding's function of that
// name: its dict, or the status where the entry point refuses.
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "norm takes 10 arguments");
    return nullptr;
  }
  int T, H, xt, rt = 0, rT, rH;
  if (!matrix(a[0], "x", &T, &H, &xt)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(a[0]);
  const int64_t rows[] = {T}, row[] = {H}, full[] = {T, H}, blocks[] = {T, (static_cast<int64_t>(H) + 127) / 128};
  const bool has_res = a[2] != Py_None;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int fp8 = PyObject_IsTrue(a[5]);
  if (fp8 < 0) return nullptr;
  if (!check_tensor(a[0], "x", xt, full) || !check_tensor(a[1], "weight", 0, row)) return nullptr;
  Ref res_out, out, q, scale, rstd;
  if (has_res) {
    if (!matrix(a[2], "residual", &rT, &rH, &rt) || !check_tensor(a[2], "residual", rt, full) ||
        !output(a[6], "residual_out", rt, full, &res_out))
      return nullptr;
  } else {
    if (a[6] != Py_None) {
      refuse("residual_out", "needs a residual");
      return nullptr;
    }
    none(&res_out);
  }
  if (given(a[4]) == kSkip) none(&out);
  else if (!output(a[4], "out", 0, full, &out)) return nullptr;
  if (!fp8) {
    none(&q);
    none(&scale);
  } else if (!output(a[7], "q", 2, full, &q) || !output(a[8], "scale", 1, blocks, &scale)) {
    return nullptr;
  }
  if (!output(a[9], "rstd", 1, rows, &rstd)) return nullptr;
  const void* res = has_res ? THPVariable_Unpack(a[2]).data_ptr() : nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  const void* weight = THPVariable_Unpack(a[1]).data_ptr();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = add_rms_norm(x.data_ptr(), xt, res, rt, weight, T, H, static_cast<float>(eps), res_out.data(), out.data(), q.data(),
                    static_cast<float*>(scale.data()), static_cast<float*>(rstd.data()), stream);
  Py_END_ALLOW_THREADS
  if (rc != 0) return PyLong_FromLong(rc);
  return dict_of({"residual", "out", "q", "scale", "rstd"}, {&res_out, &out, &q, &scale, &rstd});
  END_HANDLE_TH_ERRORS
}

// norm_backward(dy, x, weight, rstd, dres, dx, dweight, workspace): likewise.
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "norm_backward takes 8 arguments");
    return nullptr;
  }
  int T, H, xt, dT, dH, dt;
  if (!matrix(a[1], "x", &T, &H, &xt) || !matrix(a[0], "dy", &dT, &dH, &dt)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(a[1]);
  const int64_t rows[] = {T}, row[] = {H}, full[] = {T, H};
  const bool has_dres = a[4] != Py_None;
  if (!check_tensor(a[1], "x", xt, full) || !check_tensor(a[0], "dy", dt, full) ||
      !check_tensor(a[2], "weight", 0, row) || !check_tensor(a[3], "rstd", 1, rows) ||
      (has_dres && !check_tensor(a[4], "dres", xt, full)))
    return nullptr;
  Ref dx, dweight, space;
  if (!output(a[5], "dx", xt, full, &dx)) return nullptr;
  size_t bytes = 0;
  if (given(a[6]) == kSkip) {
    none(&dweight);
    none(&space);
  } else {
    if (!output(a[6], "dweight", 1, row, &dweight)) return nullptr;
    const int64_t want[] = {static_cast<int64_t>(rms_norm_backward_workspace_size(T, H))};
    if (!output(a[7], "workspace", 4, a[7] == Py_None ? at::IntArrayRef(want) : at::IntArrayRef(), &space))
      return nullptr;
    bytes = static_cast<size_t>(THPVariable_Unpack(space.o).numel());
  }
  const void* dres = has_dres ? THPVariable_Unpack(a[4]).data_ptr() : nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  const void* dy = THPVariable_Unpack(a[0]).data_ptr();
  const void* weight = THPVariable_Unpack(a[2]).data_ptr();
  const float* rstd = static_cast<const float*>(THPVariable_Unpack(a[3]).data_ptr());
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = add_rms_norm_backward(dy, dt, x.data_ptr(), xt, weight, rstd, dres, T, H, dx.data(),
                             static_cast<float*>(dweight.data()), space.data(), bytes, stream);
  Py_END_ALLOW_THREADS
  if (rc != 0) return PyLong_FromLong(rc);
  return dict_of({"dx", "dweight"}, {&dx, &dweight});
  END_HANDLE_TH_ERRORS
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
    METHOD("norm", &norm),
    METHOD("norm_backward", &norm_backward),
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
