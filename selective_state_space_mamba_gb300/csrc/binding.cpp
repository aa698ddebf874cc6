// Python entry points of the operators around a layer's scan (module _binding), for _layer.py.
//
// They check shapes, types and devices, allocate the outputs on the current stream and make the C
// call.  A call for one token takes 2 to 4 us on the GPU; the same steps in Python took 12 to 16 us
// on the GPU's host, here they take 3.5 to 5.5.  Each function takes its arguments by position (None for an
// absent tensor) and returns the outputs, or the ssm_status of a refused call as an int.
//
// The C entry points are handed over by address (bind), so that this module and ctypes share one
// library and its state.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAMacros.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/ssm.h"

namespace {

struct {
  decltype(&ssm_conv_fwd) conv_fwd;
  decltype(&ssm_conv_step) conv_step;
  decltype(&ssm_selscan_fwd_workspace_bytes) selscan_fwd_workspace_bytes;
  decltype(&ssm_selscan_fwd) selscan_fwd;
  decltype(&ssm_selscan_step) selscan_step;
  decltype(&ssm_rmsnorm_fwd) rmsnorm_fwd;
  decltype(&ssm_rmsnorm_fp8_fwd) rmsnorm_fp8_fwd;
} g_fn;

struct Refusal {
  PyObject* kind;
  std::string text;
};
[[noreturn]] void fail(const char* name, const std::string& want) {
  throw Refusal{PyExc_ValueError, std::string(name) + " must be " + want};
}

// A size that the C entry points take in 32 bits.  They refuse what is too many for the kernels, but not what a
// cast has made small before they see it.
struct Unsupported {};
int narrow(int64_t v) {
  if (v != (int64_t)(int)v) throw Unsupported{};
  return (int)v;
}

// An exception of Python's own is set already.
struct Raised {};
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

using Sizes = c10::IntArrayRef;
std::string text_of(Sizes s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) fail(name, "a tensor");
  return THPVariable_Unpack(o);
}

// The first tensor's type and device, which the others are held to.
struct Like {
  const char* name;
  c10::ScalarType type;
  c10::Device device;
  ssm_dtype code;
  int bytes;

  explicit Like(const char* name, const at::Tensor& t) : name(name), type(t.scalar_type()), device(t.device()) {
    if (type != at::kFloat && type != at::kBFloat16)
      throw Refusal{PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(type) + " (float32 or bfloat16)"};
    code = type == at::kFloat ? SSM_F32 : SSM_BF16;
    bytes = type == at::kFloat ? 4 : 2;
  }
  // the C call goes to the current device
  c10::cuda::CUDAGuard guard() const {
    if (!device.is_cuda()) fail(name, "a CUDA tensor");
    return c10::cuda::CUDAGuard(device);
  }
  ssm_stream_t stream() const {
    return reinterpret_cast<ssm_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  }
  at::Tensor empty(Sizes sizes, c10::ScalarType as) const {
    return at::Tensor(at::detail::empty_cuda(sizes, as, device, std::nullopt));
  }
};

void held(const char* name, const at::Tensor& t, Sizes sizes, c10::ScalarType type, const Like& like, const char* how) {
  if (t.sizes() != sizes || t.scalar_type() != type || t.device() != like.device)
    fail(name, std::string(how) + text_of(sizes) + " of " + c10::toString(type) + ", on the first one's device");
}

// A token tensor: strided in all but its last dimension.
ssm_tokens tokens(const char* name, const at::Tensor& t, Sizes sizes, const Like& like) {
  held(name, t, sizes, like.type, like, "a CUDA tensor ");
  const auto s = t.strides();
  if (s.back() != 1 && sizes.back() != 1) fail(name, "contiguous in its last dimension");
  return {t.data_ptr(), s[0], s.size() > 1 ? s[1] : 0};
}

void* dense(const char* name, const at::Tensor& t, Sizes sizes, c10::ScalarType type, const Like& like) {
  held(name, t, sizes, type, like, "a contiguous CUDA tensor ");
  if (!t.is_contiguous()) fail(name, "a contiguous CUDA tensor " + text_of(sizes));
  return t.data_ptr();
}
void* optional(const char* name, PyObject* o, Sizes sizes, c10::ScalarType type, const Like& like) {
  return o == Py_None ? nullptr : dense(name, tensor(name, o), sizes, type, like);
}
const float* floats(const char* name, PyObject* o, Sizes sizes, const Like& like) {
  return static_cast<const float*>(optional(name, o, sizes, at::kFloat, like));
}
const int32_t* ints(const char* name, PyObject* o, int64_t n, const Like& like) {
  return static_cast<const int32_t*>(optional(name, o, {n}, at::kInt, like));
}

// An output: the caller's tensor or a new one.
struct Out {
  PyObject* object = nullptr;  // an own reference
  void* ptr = nullptr;

  Out() = default;
  Out(const Out&) = delete;
  Out& operator=(const Out&) = delete;
  ~Out() { Py_XDECREF(object); }
  void set(const char* name, PyObject* given, Sizes sizes, c10::ScalarType type, const Like& like) {
    if (given == Py_None) {
      at::Tensor t = like.empty(sizes, type);
      ptr = t.data_ptr();
      object = THPVariable_Wrap(std::move(t));
    } else {
      ptr = dense(name, tensor(name, given), sizes, type, like);
      Py_INCREF(given);
      object = given;
    }
  }
  PyObject* give() {  // the reference, or None
    PyObject* o = object;
    object = nullptr;
    if (!o) Py_INCREF(o = Py_None);
    return o;
  }
};

PyObject* result(ssm_status st, Out& a, Out& b) {
  if (st != SSM_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, a.give());
  PyTuple_SET_ITEM(t, 1, b.give());
  return t;
}

// A step's new states: in place, the caller's, or new ones (a copy where slots name some of the rows
// only: the others keep what they hold).  Returns the number of rows.
int64_t step_states(Out& out, PyObject* state, PyObject* state_out, bool inplace, bool slots, int64_t batch, int64_t d1,
                    int64_t d2, c10::ScalarType type, const Like& like) {
  if (inplace && (state == Py_None || state_out != Py_None))
    throw Refusal{PyExc_ValueError, "inplace needs a state and no state_out"};
  PyObject* target = inplace ? state : state_out;
  if (target == Py_None && state == Py_None && slots)
    throw Refusal{PyExc_ValueError, "slots need a state or a state_out"};
  int64_t n = batch;
  PyObject* rows = target != Py_None ? target : state;
  if (rows != Py_None) {
    const at::Tensor& t = tensor("state", rows);
    if (t.dim() != 3) fail("state", "of three dimensions");
    n = t.size(0);
  }
  if (target == Py_None && state != Py_None && slots) {
    at::Tensor t = tensor("state", state).clone();
    out.ptr = t.data_ptr();
    out.object = THPVariable_Wrap(std::move(t));
  } else {
    out.set("state_out", target, {n, d1, d2}, type, like);
  }
  return n;
}

PyObject* conv_fwd(PyObject* const* v) {  // x, weight, bias, state, lens, silu, y, state_out, return_final_state
  const at::Tensor &x = tensor("x", v[0]), &w = tensor("weight", v[1]);
  const Like like("x", x);
  if (x.dim() != 3 || w.dim() != 2) fail("x, weight", "[b, L, d] and [d, W]");
  const int64_t b = x.size(0), L = x.size(1);
  const int d = narrow(x.size(2)), W = narrow(w.size(1));
  const auto guard = like.guard();
  const ssm_tokens xt = tokens("x", x, {b, L, d}, like);
  const float* wp = static_cast<const float*>(dense("weight", w, {d, W}, at::kFloat, like));
  const float* bias = floats("bias", v[2], {d}, like);
  const void* state = optional("state", v[3], {b, W - 1, d}, like.type, like);
  const int32_t* lens = ints("lens", v[4], b, like);
  Out y, so;
  y.set("y", v[6], {b, L, d}, like.type, like);
  if (truth(v[8])) so.set("state_out", v[7], {b, W - 1, d}, like.type, like);
  const ssm_status st = g_fn.conv_fwd(xt, wp, bias, state, lens, y.ptr, so.ptr, b, L, d, W,
                                      truth(v[5]) ? SSM_ACT_SILU : SSM_ACT_NONE, like.code, like.stream());
  return result(st, y, so);
}

PyObject* conv_step(PyObject* const* v) {  // x, weight, bias, state, slots, silu, y, state_out, inplace
  const at::Tensor &x = tensor("x", v[0]), &w = tensor("weight", v[1]);
  const Like like("x", x);
  if (x.dim() != 2 || w.dim() != 2) fail("x, weight", "[b, d] and [d, W]");
  const int64_t b = x.size(0);
  const int d = narrow(x.size(1)), W = narrow(w.size(1));
  const auto guard = like.guard();
  const ssm_tokens xt = tokens("x", x, {b, d}, like);
  const float* wp = static_cast<const float*>(dense("weight", w, {d, W}, at::kFloat, like));
  const float* bias = floats("bias", v[2], {d}, like);
  const int32_t* slots = ints("slots", v[4], b, like);
  Out y, so;
  const int64_t n = step_states(so, v[3], v[7], truth(v[8]), slots, b, W - 1, d, like.type, like);
  const void* state = optional("state", v[3], {n, W - 1, d}, like.type, like);
  y.set("y", v[6], {b, d}, like.type, like);
  const ssm_status st = g_fn.conv_step(xt, wp, bias, state, slots, y.ptr, so.ptr, b, n, d, W,
                                       truth(v[5]) ? SSM_ACT_SILU : SSM_ACT_NONE, like.code, like.stream());
  return result(st, y, so);
}

// u, dt, A, B, C, D, z, dt_bias: what selscan_fwd and selscan_step share.  `lead`: dimensions before the channels.
ssm_selscan_args selscan_args(PyObject* const* v, const Like& like, const at::Tensor& u, int lead) {
  ssm_selscan_args a{};
  const Sizes sizes = u.sizes();
  const at::Tensor &B = tensor("B", v[3]), &C = tensor("C", v[4]);
  if (B.dim() != lead + 2 || B.sizes().slice(0, lead) != sizes.slice(0, lead))
    fail("B", text_of(sizes.slice(0, lead)) + " and groups, states");
  const int d = narrow(sizes.back()), G = narrow(B.size(lead)), N = narrow(B.size(lead + 1));
  a.u = tokens("u", u, sizes, like);
  a.dt = tokens("dt", tensor("dt", v[1]), sizes, like);
  a.B = tokens("B", B, B.sizes(), like);
  a.C = tokens("C", C, B.sizes(), like);
  if (G > 1 && (B.stride(lead) != N || C.stride(lead) != N)) fail("B, C", "contiguous in their last two dimensions");
  if (v[6] != Py_None) a.z = tokens("z", tensor("z", v[6]), sizes, like);
  a.A = static_cast<const float*>(dense("A", tensor("A", v[2]), {d, N}, at::kFloat, like));
  a.D = floats("D", v[5], {d}, like);
  a.dt_bias = floats("dt_bias", v[7], {d}, like);
  a.batch = sizes[0];
  a.channels = d;
  a.dstate = N;
  a.ngroups = G;
  a.dtype = like.code;
  return a;
}

// The workspace of each device's last scan that was given none: its status can still be read (kept_workspace).
PyObject* g_kept[C10_COMPILE_TIME_MAX_GPUS] = {};

// u, dt, A, B, C, D, z, dt_bias, h0, lens, softplus, y, h_final, return_final_state, workspace buffer
PyObject* selscan_fwd(PyObject* const* v) {
  const at::Tensor& u = tensor("u", v[0]);
  const Like like("u", u);
  if (u.dim() != 3) fail("u", "[b, L, d]");
  ssm_selscan_args a = selscan_args(v, like, u, 2);
  const auto guard = like.guard();
  a.seqlen = u.size(1);
  a.softplus = truth(v[10]);
  a.h0 = floats("h0", v[8], {a.batch, a.channels, a.dstate}, like);
  a.lens = ints("lens", v[9], a.batch, like);
  Out y, h;
  y.set("y", v[11], u.sizes(), like.type, like);
  a.y = y.ptr;
  if (truth(v[13])) h.set("h_final", v[12], {a.batch, a.channels, a.dstate}, at::kFloat, like);
  a.h_final = static_cast<float*>(h.ptr);
  at::Tensor ws;
  if (v[14] != Py_None) {
    ws = tensor("workspace", v[14]);
    if (ws.device() != like.device || ws.scalar_type() != at::kByte || !ws.is_contiguous())
      fail("workspace", "contiguous bytes on u's device");
  } else {
    const size_t need = g_fn.selscan_fwd_workspace_bytes(a.batch, a.seqlen, a.channels, a.dstate, a.ngroups);
    if (need) {
      ws = like.empty({(int64_t)need}, at::kByte);
      PyObject*& kept = g_kept[like.device.index()];
      Py_XDECREF(kept);
      kept = THPVariable_Wrap(ws);
    }
  }
  return result(g_fn.selscan_fwd(&a, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0,
                                 like.stream()),
                y, h);
}

// u, dt, A, B, C, D, z, dt_bias, state, slots, softplus, y, state_out, inplace
PyObject* selscan_step(PyObject* const* v) {
  const at::Tensor& u = tensor("u", v[0]);
  const Like like("u", u);
  if (u.dim() != 2) fail("u", "[b, d]");
  ssm_selscan_args a = selscan_args(v, like, u, 1);
  const auto guard = like.guard();
  a.seqlen = 1;
  a.softplus = truth(v[10]);
  const int32_t* slots = ints("slots", v[9], a.batch, like);
  Out y, so;
  const int64_t n =
      step_states(so, v[8], v[12], truth(v[13]), slots, a.batch, a.channels, a.dstate, at::kFloat, like);
  a.h0 = floats("state", v[8], {n, a.channels, a.dstate}, like);
  a.h_final = static_cast<float*>(so.ptr);
  y.set("y", v[11], u.sizes(), like.type, like);
  a.y = y.ptr;
  return result(g_fn.selscan_step(&a, slots, n, like.stream()), y, so);
}

// Rows of x, and the residual: what the two norms share.
struct Norm {
  const at::Tensor& x;
  Like like;
  int d;
  c10::cuda::CUDAGuard guard;
  int64_t rows, stride;
  const float* w;
  const void* residual = nullptr;
  ssm_dtype res_code;
  Out residual_out;

  Norm(PyObject* xo, PyObject* wo, PyObject* ro, PyObject* oo)
      : x(tensor("x", xo)), like("x", x), d(x.dim() ? narrow(x.size(-1)) : 0), guard(like.guard()) {
    const Sizes sizes = x.sizes();
    rows = d ? x.numel() / d : 0;
    if (x.is_contiguous())
      stride = d;
    else if (x.stride(-1) != 1 && d != 1)
      fail("x", "contiguous in its last dimension");
    else
      stride = (x.dim() == 2 ? x : x.view({rows, d})).stride(0);
    w = static_cast<const float*>(dense("weight", tensor("weight", wo), {d}, at::kFloat, like));
    res_code = like.code;
    if (ro == Py_None) {
      if (oo != Py_None) throw Refusal{PyExc_ValueError, "residual_out needs a residual"};
      return;
    }
    const at::Tensor& r = tensor("residual", ro);
    if (r.scalar_type() != at::kFloat && r.scalar_type() != like.type) fail("residual", "of float32 or x's dtype");
    res_code = r.scalar_type() == at::kFloat ? SSM_F32 : SSM_BF16;
    residual = dense("residual", r, sizes, r.scalar_type(), like);
    residual_out.set("residual_out", oo, sizes, r.scalar_type(), like);
  }
};

PyObject* kept_workspace(PyObject* const* v) {  // device index
  const long i = PyLong_AsLong(v[0]);
  if (PyErr_Occurred()) return nullptr;
  PyObject* o = i >= 0 && i < C10_COMPILE_TIME_MAX_GPUS && g_kept[i] ? g_kept[i] : Py_None;
  Py_INCREF(o);
  return o;
}

PyObject* rmsnorm_fwd(PyObject* const* v) {  // x, weight, residual, eps, y, residual_out
  Norm n(v[0], v[1], v[2], v[5]);
  const double eps = PyFloat_AsDouble(v[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  Out y;
  y.set("y", v[4], n.x.sizes(), n.like.type, n.like);
  return result(g_fn.rmsnorm_fwd(n.x.data_ptr(), n.stride, n.w, n.residual, n.residual_out.ptr, y.ptr, n.rows, n.d,
                                 (float)eps, n.like.code, n.res_code, n.like.stream()),
                y, n.residual_out);
}

PyObject* rmsnorm_fp8_fwd(PyObject* const* v) {  // x, weight, residual, eps, group, q, scale, residual_out
  const double eps = PyFloat_AsDouble(v[3]);
  const long of = PyLong_AsLong(v[4]);
  if (PyErr_Occurred()) return nullptr;
  const int group = narrow(of);
  Norm n(v[0], v[1], v[2], v[7]);
  Out q, scale;
  q.set("q", v[5], n.x.sizes(), at::kFloat8_e4m3fn, n.like);
  c10::SmallVector<int64_t, 8> sizes(n.x.sizes().begin(), n.x.sizes().end());
  if (!sizes.empty()) sizes.pop_back();
  if (group != 0) sizes.push_back(((int64_t)n.d + 127) / 128);
  scale.set("scale", v[6], sizes, at::kFloat, n.like);
  const ssm_status st = g_fn.rmsnorm_fp8_fwd(n.x.data_ptr(), n.stride, n.w, n.residual, n.residual_out.ptr, q.ptr,
                                             static_cast<float*>(scale.ptr), n.rows, n.d, group, (float)eps,
                                             n.like.code, n.res_code, n.like.stream());
  if (st != SSM_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(3);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, q.give());
  PyTuple_SET_ITEM(t, 1, scale.give());
  PyTuple_SET_ITEM(t, 2, n.residual_out.give());
  return t;
}

// No C++ exception leaves a Python entry point.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != ARGS) throw Refusal{PyExc_TypeError, "wrong number of arguments"};
    if (!g_fn.conv_fwd) throw Refusal{PyExc_RuntimeError, "the library is not bound"};
    return F(args);
  } catch (const Raised&) {
  } catch (const Unsupported&) {
    return PyLong_FromLong(SSM_ERR_UNSUPPORTED);
  } catch (const Refusal& r) {
    PyErr_SetString(r.kind, r.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(kind ? kind : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(kind);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// bind(addresses of the seven C entry points, in the order of g_fn)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_fn = {reinterpret_cast<decltype(g_fn.conv_fwd)>(p[0]),
          reinterpret_cast<decltype(g_fn.conv_step)>(p[1]),
          reinterpret_cast<decltype(g_fn.selscan_fwd_workspace_bytes)>(p[2]),
          reinterpret_cast<decltype(g_fn.selscan_fwd)>(p[3]),
          reinterpret_cast<decltype(g_fn.selscan_step)>(p[4]),
          reinterpret_cast<decltype(g_fn.rmsnorm_fwd)>(p[5]),
          reinterpret_cast<decltype(g_fn.rmsnorm_fp8_fwd)>(p[6])};
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }
PyMethodDef g_methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                           {"conv_fwd", fast(entry<conv_fwd, 9>), METH_FASTCALL, nullptr},
                           {"conv_step", fast(entry<conv_step, 9>), METH_FASTCALL, nullptr},
                           {"selscan_fwd", fast(entry<selscan_fwd, 15>), METH_FASTCALL, nullptr},
                           {"selscan_step", fast(entry<selscan_step, 14>), METH_FASTCALL, nullptr},
                           {"rmsnorm_fwd", fast(entry<rmsnorm_fwd, 6>), METH_FASTCALL, nullptr},
                           {"kept_workspace", fast(entry<kept_workspace, 1>), METH_FASTCALL, nullptr},
                           {"rmsnorm_fp8_fwd", fast(entry<rmsnorm_fp8_fwd, 8>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) { return PyModule_Create(&g_module); }
