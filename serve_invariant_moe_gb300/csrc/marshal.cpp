// marshal.cpp -- CPython helpers of the binding: argument checks, output allocation and the calls of the 8-bit block and of a
// drafted decode step.
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

const void* data_of(PyObject* o) { return o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }

// The gate's kind by its type and shape: None, [H] bf16 (a channel's), [T] fp32 (a token's).
bool gate_kind(PyObject* o, at::IntArrayRef rows, at::IntArrayRef row, int* kind) {
  *kind = INVMOE_GATE_NONE;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return refuse("gate", "must be a tensor");
  *kind = THPVariable_Unpack(o).scalar_type() == kTypes[0] ? INVMOE_GATE_CHANNEL : INVMOE_GATE_TOKEN;
  return *kind == INVMOE_GATE_CHANNEL ? check_tensor(o, "gate", 0, row) : check_tensor(o, "gate", 1, rows);
}

// sandwich(x, w_post, residual, w_next, gate, residual_scale, branch_scale, eps, out, fp8, residual_out, q, scale, rstd_post,
// rstd): likewise, of sandwich_norm.
PyObject* sandwich(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) {
    PyErr_SetString(PyExc_TypeError, "sandwich takes 15 arguments");
    return nullptr;
  }
  int T, H, xt, rT, rH, rt;
  if (!matrix(a[0], "x", &T, &H, &xt) || !matrix(a[2], "residual", &rT, &rH, &rt)) return nullptr;
  const int64_t rows[] = {T}, row[] = {H}, full[] = {T, H}, blocks[] = {T, (static_cast<int64_t>(H) + 127) / 128};
  const bool next = a[3] != Py_None;
  float number[3];                                    // residual_scale, branch_scale, eps
  for (int i = 0; i < 3; ++i)
    if (!convert(a[5 + i], &number[i])) return nullptr;
  const int fp8 = PyObject_IsTrue(a[9]);
  if (fp8 < 0) return nullptr;
  if (!check_tensor(a[0], "x", xt, full) || !check_tensor(a[1], "w_post", 0, row) ||
      !check_tensor(a[2], "residual", rt, full) || (next && !check_tensor(a[3], "w_next", 0, row)))
    return nullptr;
  int kind;
  if (!gate_kind(a[4], rows, row, &kind)) return nullptr;
  const void* gate = data_of(a[4]);
  Ref res_out, out, q, scale, rstd_post, rstd;
  if (!output(a[10], "residual_out", rt, full, &res_out) || !output(a[13], "rstd_post", 1, rows, &rstd_post)) return nullptr;
  if (!next) {
    if (given(a[8]) == kTaken || fp8 || given(a[11]) == kTaken || given(a[12]) == kTaken || given(a[14]) == kTaken) {
      refuse("w_next", "is required for out, fp8 and rstd");
      return nullptr;
    }
    for (Ref* r : {&out, &q, &scale, &rstd}) none(r);
  } else {
    if (given(a[8]) == kSkip) none(&out);
    else if (!output(a[8], "out", 0, full, &out)) return nullptr;
    if (!fp8) {
      none(&q);
      none(&scale);
    } else if (!output(a[11], "q", 2, full, &q) || !output(a[12], "scale", 1, blocks, &scale)) {
      return nullptr;
    }
    if (!output(a[14], "rstd", 1, rows, &rstd)) return nullptr;
  }
  const void* x = THPVariable_Unpack(a[0]).data_ptr();
  const void* w_post = THPVariable_Unpack(a[1]).data_ptr();
  const void* residual = THPVariable_Unpack(a[2]).data_ptr();
  const void* w_next = next ? THPVariable_Unpack(a[3]).data_ptr() : nullptr;
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = sandwich_norm(x, xt, w_post, residual, rt, gate, kind, w_next, T, H, number[0], number[1], number[2], res_out.data(),
                     out.data(), q.data(), static_cast<float*>(scale.data()), static_cast<float*>(rstd_post.data()),
                     static_cast<float*>(rstd.data()), stream);
  Py_END_ALLOW_THREADS
  if (rc != 0) return PyLong_FromLong(rc);
  return dict_of({"residual", "out", "q", "scale", "rstd_post", "rstd"}, {&res_out, &out, &q, &scale, &rstd_post, &rstd});
  END_HANDLE_TH_ERRORS
}

// sandwich_backward(dy, dres, x, w_post, rstd_post, residual, w_next, rstd, gate, residual_scale, branch_scale, dx, dresidual,
// dweights, workspace): likewise, of sandwich_norm_backward.
PyObject* sandwich_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 15) {
    PyErr_SetString(PyExc_TypeError, "sandwich_backward takes 15 arguments");
    return nullptr;
  }
  int T, H, xt, rT, rH, rt, yT, yH, yt = 0;
  if (!matrix(a[2], "x", &T, &H, &xt) || !matrix(a[5], "residual", &rT, &rH, &rt)) return nullptr;
  const int64_t rows[] = {T}, row[] = {H}, full[] = {T, H};
  const bool next = a[0] != Py_None;
  if (next != (a[6] != Py_None) || next != (a[7] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "dy, w_next and rstd go together");
    return nullptr;
  }
  float number[2];                                    // residual_scale, branch_scale
  int kind;
  if (!convert(a[9], &number[0]) || !convert(a[10], &number[1]) || !check_tensor(a[2], "x", xt, full) ||
      !check_tensor(a[5], "residual", rt, full) || !check_tensor(a[3], "w_post", 0, row) ||
      !check_tensor(a[4], "rstd_post", 1, rows) || (a[1] != Py_None && !check_tensor(a[1], "dres", rt, full)) ||
      !gate_kind(a[8], rows, row, &kind))
    return nullptr;
  if (next && (!matrix(a[0], "dy", &yT, &yH, &yt) || !check_tensor(a[0], "dy", yt, full) ||
               !check_tensor(a[6], "w_next", 0, row) || !check_tensor(a[7], "rstd", 1, rows)))
    return nullptr;
  const int weights = PyObject_IsTrue(a[13]);
  if (weights < 0) return nullptr;
  Ref dx, dresidual, dw_post, dw_next, dgate, space;
  if (!output(a[11], "dx", xt, full, &dx) || !output(a[12], "dresidual", rt, full, &dresidual)) return nullptr;
  auto made = [](Ref* r, bool wanted, at::IntArrayRef dims) {
    if (wanted) r->o = new_output(1, dims);
    else none(r);
    return r->o != nullptr;
  };
  const bool token = kind == INVMOE_GATE_TOKEN;
  if (!made(&dw_post, weights, row) || !made(&dw_next, weights && next, row) ||
      !made(&dgate, token || (kind == INVMOE_GATE_CHANNEL && weights), token ? rows : row))
    return nullptr;
  const int64_t want[] = {static_cast<int64_t>(sandwich_norm_backward_workspace_size(T, H))};
  if (!output(a[14], "workspace", 4, a[14] == Py_None ? at::IntArrayRef(want) : at::IntArrayRef(), &space)) return nullptr;
  const size_t bytes = static_cast<size_t>(THPVariable_Unpack(space.o).numel());
  const void *dy = data_of(a[0]), *dres = data_of(a[1]), *x = data_of(a[2]), *w_post = data_of(a[3]), *r = data_of(a[5]),
             *w_next = data_of(a[6]), *gate = data_of(a[8]);
  const float *rstd_post = static_cast<const float*>(data_of(a[4])), *rstd = static_cast<const float*>(data_of(a[7]));
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = sandwich_norm_backward(dy, yt, dres, x, xt, w_post, rstd_post, r, rt, w_next, rstd, gate, kind, T, H, number[0], number[1],
                              dx.data(), dresidual.data(), static_cast<float*>(dw_post.data()),
                              static_cast<float*>(dw_next.data()), static_cast<float*>(dgate.data()), space.data(), bytes,
                              stream);
  Py_END_ALLOW_THREADS
  if (rc != 0) return PyLong_FromLong(rc);
  return dict_of({"dx", "dresidual", "dw_post", "dw_next", "dgate"}, {&dx, &dresidual, &dw_post, &dw_next, &dgate});
  END_HANDLE_TH_ERRORS
}

// verify(logits, noise, workspace, draft_tokens, draft_logits, accept_u, n_draft, temperature, tokens, n_accepted, logp):
// likewise, of verify_drafts.
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) {
    PyErr_SetString(PyExc_TypeError, "verify takes 11 arguments");
    return nullptr;
  }
  if (!THPVariable_Check(a[0])) {
    refuse("logits", "must be a tensor");
    return nullptr;
  }
  const at::Tensor& z = THPVariable_Unpack(a[0]);
  if (z.dim() != 3) {
    refuse("logits", "must have 3 dimensions, got shape " + shape_text(z.sizes()));
    return nullptr;
  }
  const int64_t B = z.size(0), D = z.size(1) - 1, V = z.size(2);
  if (D < 0 || B > INT32_MAX || D > INT32_MAX || V > INT32_MAX) {
    refuse("logits", D < 0 ? "must have at least one row per request" : "does not fit 32-bit sizes");
    return nullptr;
  }
  if (z.scalar_type() != kTypes[0] && z.scalar_type() != kTypes[1]) {
    refuse("logits", "must be torch.bfloat16 or torch.float32, got " + type_name(z.scalar_type()));
    return nullptr;
  }
  const int zt = z.scalar_type() == kTypes[0] ? 0 : 1;
  const int64_t all[] = {B, D + 1, V}, draft[] = {B, D, V}, wide[] = {B, V}, pairs[] = {B, D}, out[] = {B, D + 1}, each[] = {B};
  if (!check_tensor(a[0], "logits", zt, all) || !check_tensor(a[1], "noise", 1, wide)) return nullptr;
  if (D == 0) {
    if (a[3] != Py_None || a[4] != Py_None || a[5] != Py_None || a[6] != Py_None) {
      refuse("logits", "of one row per request leave no room for drafts");
      return nullptr;
    }
  } else if (!check_tensor(a[3], "draft_tokens", 3, pairs) || !check_tensor(a[5], "accept_u", 1, pairs) ||
             (a[4] != Py_None && !check_tensor(a[4], "draft_logits", zt, draft)) ||
             (a[6] != Py_None && !check_tensor(a[6], "n_draft", 3, each))) {
    return nullptr;
  }
  float tau = 1.0f;
  const float* temperature = nullptr;
  if (THPVariable_Check(a[7])) {
    if (!check_tensor(a[7], "temperature", 1, each)) return nullptr;
    temperature = static_cast<const float*>(data_of(a[7]));
  } else if (!convert(a[7], &tau)) {
    return nullptr;
  }
  if (!check_tensor(a[2], "workspace", 4, at::IntArrayRef())) return nullptr;
  Ref tokens, accepted, logp;
  if (!output(a[8], "tokens", 3, out, &tokens) || !output(a[9], "n_accepted", 3, each, &accepted) ||
      !output(a[10], "logp", 1, out, &logp))
    return nullptr;
  void* space = THPVariable_Unpack(a[2]).data_ptr();
  const size_t bytes = static_cast<size_t>(THPVariable_Unpack(a[2]).numel());
  const void *logits = z.data_ptr(), *draft_logits = data_of(a[4]);
  const int32_t *draft_tokens = static_cast<const int32_t*>(data_of(a[3])), *n_draft = static_cast<const int32_t*>(data_of(a[6]));
  const float *u = static_cast<const float*>(data_of(a[5])), *noise = static_cast<const float*>(data_of(a[1]));
  void* stream = c10::cuda::getCurrentCUDAStream().stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = verify_drafts(logits, zt, draft_logits, draft_tokens, u, noise, n_draft, temperature, tau, static_cast<int>(B),
                     static_cast<int>(D), static_cast<int>(V), static_cast<int32_t*>(tokens.data()),
                     static_cast<int32_t*>(accepted.data()), static_cast<float*>(logp.data()), space, bytes, stream);
  Py_END_ALLOW_THREADS
  if (rc != 0) return PyLong_FromLong(rc);
  return dict_of({"tokens", "n_accepted", "logp"}, {&tokens, &accepted, &logp});
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
    ENTRY(moe_layer_decode),
    METHOD("sandwich", &sandwich),
    METHOD("sandwich_backward", &sandwich_backward),
    METHOD("verify", &verify),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
