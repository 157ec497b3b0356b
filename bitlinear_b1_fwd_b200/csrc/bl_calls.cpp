// bl_calls.cpp -- the Python side of the calls that a decode step makes many
// times: checks of shapes, types, contiguity and devices, then the C entry point
// of the same name.  Marshalling only.  In Python with ctypes it took 6 us a
// call, twice a launch and more than most of these kernels; here under 1 us.
//
// Every function takes its arguments in the order binding.py documents, all
// positional (None where one is left out), and returns the bl_status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "bitlinear.h"

namespace {

struct Refused {};  // a Python exception is set

enum : unsigned { kF32 = 1, kBF16 = 2, kI8 = 4, kU8 = 8, kFloats = kF32 | kBF16 };

unsigned type_bit(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return kF32;
    case at::kBFloat16: return kBF16;
    case at::kChar: return kI8;
    case at::kByte: return kU8;
    default: return 0;
  }
}
int type_code(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? BL_BF16 : t.scalar_type() == at::kChar ? BL_I8 : BL_F32;
}

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Refused{};
}

std::string text(c10::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// One call: the device named by its first matrix, and the first complaint about
// a device, which comes after those about types, shapes and layout.
struct Call {
  int dev = -1;
  std::string late;
};

const at::Tensor& matrix(const char* name, PyObject* o, Call& call) {
  const at::Tensor& t = tensor(name, o);
  if (t.dim() != 2)
    refuse(PyExc_ValueError, std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, expected 2");
  if (t.is_cuda())
    call.dev = t.get_device();
  else
    call.late = std::string(name) + " must be a CUDA tensor";
  return t;
}

// The address of a contiguous tensor of this shape and one of the types on the
// call's device.
void* want(const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape, unsigned types, Call& call) {
  const c10::IntArrayRef expected(shape.begin(), shape.size());
  if ((type_bit(t) & types) == 0)
    refuse(PyExc_TypeError, std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()));
  if (t.sizes() != expected)
    refuse(PyExc_ValueError, std::string(name) + ": shape " + text(t.sizes()) + ", expected " + text(expected));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  if (!t.is_cuda() || t.get_device() != call.dev) {
    if (call.late.empty())
      call.late = std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(call.dev);
    return nullptr;
  }
  return t.data_ptr();
}
template <typename T = void>
T* want(const char* name, PyObject* o, std::initializer_list<int64_t> shape, unsigned types, Call& call) {
  return static_cast<T*>(want(name, tensor(name, o), shape, types, call));
}
template <typename T = void>
T* maybe(const char* name, PyObject* o, std::initializer_list<int64_t> shape, unsigned types, Call& call) {
  return o == Py_None ? nullptr : want<T>(name, o, shape, types, call);
}

struct Workspace {
  void* p;
  size_t bytes;
};
Workspace workspace(PyObject* o, Call& call) {
  const at::Tensor& t = tensor("the workspace", o);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "the workspace must be contiguous");
  if ((!t.is_cuda() || t.get_device() != call.dev) && call.late.empty())
    call.late = "the workspace is on " + t.device().str() + ", expected cuda:" + std::to_string(call.dev);
  return {call.late.empty() ? t.data_ptr() : nullptr, t.nbytes()};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int small(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "an integer argument is out of range");
  return static_cast<int>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return static_cast<float>(v);
}

// The given stream, or the current one of the call's device.  The last check.
void* stream_of(PyObject* o, const Call& call) {
  if (!call.late.empty()) refuse(PyExc_ValueError, call.late);
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(call.dev)).stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (h == nullptr) throw Refused{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (p == nullptr && PyErr_Occurred()) throw Refused{};
  return p;
}

// The interpreter is free while one lives, and taken back when an exception
// (of a device that cannot be made current) leaves its scope too.
struct Free {
  PyThreadState* state = PyEval_SaveThread();
  ~Free() { PyEval_RestoreThread(state); }
};

// f() with the call's device current and the interpreter free; the caller's
// device comes back.
template <typename F>
PyObject* on_device(const Call& call, F f) {
  int status;
  {
    const Free interpreter;
    const auto d = static_cast<c10::DeviceIndex>(call.dev), before = c10::cuda::current_device();
    if (d != before) c10::cuda::set_device(d);
    status = f();
    if (d != before) c10::cuda::set_device(before);
  }
  return PyLong_FromLong(status);
}

// One entry point: n arguments, exceptions to Python.
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// packed, fmt, gamma, N, K, x, scale, y, ws, bias, act, residual, preact, stream
PyObject* forward_epilogue(PyObject* const* a) {
  Call call;
  const at::Tensor& x = matrix("x", a[5], call);
  const at::Tensor& y = tensor("y", a[7]);
  const int fmt = small(a[1]), act = small(a[10]);
  const int64_t M = x.size(0), N = integer(a[3]), K = integer(a[4]);
  const void* xp = want("x", x, {M, K}, kFloats | kI8, call);
  const auto* packed = want<const uint8_t>("packed", a[0], {N, bitlinear_packed_row_bytes(K, fmt)}, kU8, call);
  const auto* gamma = want<const float>("gamma", a[2], {1}, kF32, call);
  auto* scale = want<float>("scale", a[6], {M}, kF32, call);
  void* yp = want("y", y, {M, N}, kFloats, call);
  const auto* bias = maybe<const float>("bias", a[9], {N}, kF32, call);
  const void* residual = maybe("residual", a[11], {M, N}, type_bit(y), call);
  void* preact = maybe("preact", a[12], {M, N}, type_bit(y), call);
  const Workspace ws = workspace(a[8], call);
  void* st = stream_of(a[13], call);
  const int xdt = type_code(x), ydt = type_code(y);
  return on_device(call, [&] {
    return bitlinear_forward_epilogue(packed, fmt, gamma, N, K, xp, xdt, scale, M, bias, act, residual, preact, yp, ydt,
                                      ws.p, ws.bytes, st);
  });
}

// dy, z, act, dz, dbias, ws, stream
PyObject* epilogue_backward(PyObject* const* a) {
  Call call;
  const at::Tensor& dy = matrix("dy", a[0], call);
  const int64_t M = dy.size(0), N = dy.size(1);
  const void* dyp = want("dy", dy, {M, N}, kFloats, call);
  const void* z = maybe("z", a[1], {M, N}, kFloats, call);
  void* dz = maybe("dz", a[3], {M, N}, type_bit(dy), call);
  auto* dbias = maybe<float>("dbias", a[4], {N}, kF32, call);
  const Workspace ws = workspace(a[5], call);
  void* st = stream_of(a[6], call);
  const int act = small(a[2]), dydt = type_code(dy), zdt = z == nullptr ? BL_F32 : type_code(THPVariable_Unpack(a[1]));
  return on_device(call, [&] {
    return bitlinear_epilogue_backward(dyp, dydt, z, zdt, act, M, N, dz, dbias, ws.p, ws.bytes, st);
  });
}

// packed, fmt, gamma, N, K, dz, dx, ws, stream
PyObject* backward_dx_bf16(PyObject* const* a) {
  Call call;
  const at::Tensor& dz = matrix("dz", a[5], call);
  const at::Tensor& dx = tensor("dx", a[6]);
  const int fmt = small(a[1]);
  const int64_t M = dz.size(0), N = integer(a[3]), K = integer(a[4]);
  const void* dzp = want("dz", dz, {M, N}, kBF16, call);
  const auto* packed = want<const uint8_t>("packed", a[0], {N, bitlinear_packed_row_bytes(K, fmt)}, kU8, call);
  const auto* gamma = want<const float>("gamma", a[2], {1}, kF32, call);
  void* dxp = want("dx", dx, {M, K}, kFloats, call);
  const Workspace ws = workspace(a[7], call);
  void* st = stream_of(a[8], call);
  const int dxdt = type_code(dx);
  return on_device(call, [&] {
    return bitlinear_backward_dx_bf16(packed, fmt, gamma, N, K, dzp, M, dxp, dxdt, ws.p, ws.bytes, st);
  });
}

// dz, xq, scale, gamma, dw, ws, stream
PyObject* backward_dw_bf16(PyObject* const* a) {
  Call call;
  const at::Tensor& dz = matrix("dz", a[0], call);
  const at::Tensor& xq = tensor("xq", a[1]);
  if (xq.dim() != 2) refuse(PyExc_ValueError, "xq: " + std::to_string(xq.dim()) + " dimensions, expected 2");
  const int64_t M = dz.size(0), N = dz.size(1), K = xq.size(1);
  const void* dzp = want("dz", dz, {M, N}, kBF16, call);
  const auto* q = static_cast<const int8_t*>(want("xq", xq, {M, K}, kI8, call));
  const auto* scale = want<const float>("scale", a[2], {M}, kF32, call);
  const auto* gamma = want<const float>("gamma", a[3], {1}, kF32, call);
  auto* dw = want<float>("dw", a[4], {N, K}, kF32, call);
  const Workspace ws = workspace(a[5], call);
  void* st = stream_of(a[6], call);
  return on_device(call, [&] { return bitlinear_backward_dw_bf16(dzp, q, scale, gamma, M, N, K, dw, ws.p, ws.bytes, st); });
}

// The parameters of the norms, from ten arguments: post, post_w, post_b, post_eps,
// gate, gate_rows, res_scale, branch_scale, pre, pre_w, then pre_b and pre_eps.
bl_residual_norm_params norm_params(PyObject* const* a, PyObject* pre_b, PyObject* pre_eps, int64_t M, int64_t K,
                                    Call& call) {
  bl_residual_norm_params p;
  p.post = small(a[0]);
  p.post_w = maybe<const float>("post_w", a[1], {K}, kF32, call);
  p.post_b = maybe<const float>("post_b", a[2], {K}, kF32, call);
  p.post_eps = real(a[3]);
  p.gate = nullptr;
  p.gate_rows = 0;
  if (a[4] != Py_None) {
    const at::Tensor& gate = tensor("gate", a[4]);
    p.gate_rows = integer(a[5]);
    const bool shared = p.gate_rows < 1;
    if (shared) p.gate_rows = M > 1 ? M : 1;  // one row for every token
    // a batch without tokens uses no row: a shared gate has its one all the same,
    // one with a row for every gate_rows tokens may have none
    const int64_t rows = M > 0 ? (M - 1) / p.gate_rows + 1
                         : shared || gate.dim() != 2 || gate.size(0) != 0 ? 1
                                                                          : 0;
    if (gate.dim() == 1) {
      p.gate = static_cast<const float*>(want("gate", gate, {K}, kF32, call));
      if (rows > 1) refuse(PyExc_ValueError, "gate: one row, expected " + std::to_string(rows));
    } else {
      p.gate = static_cast<const float*>(want("gate", gate, {rows, K}, kF32, call));
    }
  }
  p.res_scale = real(a[6]);
  p.branch_scale = real(a[7]);
  p.pre = small(a[8]);
  p.pre_w = maybe<const float>("pre_w", a[9], {K}, kF32, call);
  p.pre_b = pre_b == nullptr ? nullptr : maybe<const float>("pre_b", pre_b, {K}, kF32, call);
  p.pre_eps = real(pre_eps);
  return p;
}

// b, r, h, then the twelve of norm_params, then y, xq, scale, stream
PyObject* residual_norm(PyObject* const* a) {
  Call call;
  const at::Tensor& b = matrix("b", a[0], call);
  const at::Tensor& r = tensor("r", a[1]);
  const int64_t M = b.size(0), K = b.size(1);
  const void* bp = want("b", b, {M, K}, kFloats, call);
  const void* rp = want("r", r, {M, K}, kFloats, call);
  void* h = maybe("h", a[2], {M, K}, type_bit(r), call);
  void* y = maybe("y", a[15], {M, K}, kFloats, call);
  auto* xq = maybe<int8_t>("xq", a[16], {M, K}, kI8, call);
  auto* scale = maybe<float>("scale", a[17], {M}, kF32, call);
  const bl_residual_norm_params p = norm_params(a + 3, a[13], a[14], M, K, call);
  void* st = stream_of(a[18], call);
  const int bdt = type_code(b), rdt = type_code(r), ydt = y == nullptr ? BL_F32 : type_code(THPVariable_Unpack(a[15]));
  return on_device(call, [&] { return bitlinear_residual_norm(&p, bp, bdt, rp, rdt, M, K, h, y, ydt, xq, scale, st); });
}

// dy, dh, b, h, dr, db, ws, then the ten of norm_params and pre_eps, then dpost_w,
// dpost_b, dgate, dpre_w, dpre_b, stream
PyObject* residual_norm_backward(PyObject* const* a) {
  Call call;
  const at::Tensor& dy = matrix("dy", a[0], call);
  const at::Tensor &b = tensor("b", a[2]), &h = tensor("h", a[3]);
  const int64_t M = dy.size(0), K = dy.size(1);
  const void* dyp = want("dy", dy, {M, K}, kFloats, call);
  const void* bp = want("b", b, {M, K}, kFloats, call);
  const void* hp = want("h", h, {M, K}, kFloats, call);
  const void* dh = maybe("dh", a[1], {M, K}, type_bit(h), call);
  void* dr = maybe("dr", a[4], {M, K}, type_bit(h), call);
  void* db = maybe("db", a[5], {M, K}, type_bit(b), call);
  bl_residual_norm_grads g;
  g.dpost_w = maybe<float>("dpost_w", a[18], {K}, kF32, call);
  g.dpost_b = maybe<float>("dpost_b", a[19], {K}, kF32, call);
  g.dpre_w = maybe<float>("dpre_w", a[21], {K}, kF32, call);
  g.dpre_b = maybe<float>("dpre_b", a[22], {K}, kF32, call);
  const bl_residual_norm_params p = norm_params(a + 7, nullptr, a[17], M, K, call);
  g.dgate = nullptr;
  if (a[20] != Py_None) {
    if (p.gate == nullptr && a[11] == Py_None) refuse(PyExc_ValueError, "dgate without a gate");
    const at::Tensor& gate = THPVariable_Unpack(a[11]);
    g.dgate = gate.dim() == 1 ? want<float>("dgate", a[20], {K}, kF32, call)
                              : want<float>("dgate", a[20], {gate.size(0), K}, kF32, call);
    if (gate.numel() == 0) g.dgate = nullptr;  // no row
  }
  const Workspace ws = workspace(a[6], call);
  void* st = stream_of(a[23], call);
  const int dydt = type_code(dy), bdt = type_code(b), hdt = type_code(h);
  return on_device(call, [&] {
    return bitlinear_residual_norm_backward(&p, dyp, dydt, dh, bp, bdt, hp, hdt, M, K, dr, db, &g, ws.p, ws.bytes, st);
  });
}

#define BL_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<n, name>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {BL_ENTRY(forward_epilogue, 14), BL_ENTRY(epilogue_backward, 7),
                          BL_ENTRY(backward_dx_bf16, 9),  BL_ENTRY(backward_dw_bf16, 7),
                          BL_ENTRY(residual_norm, 19),    BL_ENTRY(residual_norm_backward, 24),
                          {nullptr, nullptr, 0, nullptr}};
#undef BL_ENTRY

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the Python and torch this was compiled against (build.py looks for it in
// the file)
extern "C" PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BL_CALLS_STAMP) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
