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

#include <cmath>
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
  decltype(&ssm_delta_fwd_workspace_bytes) delta_fwd_workspace_bytes;
  decltype(&ssm_delta_fwd) delta_fwd;
  decltype(&ssm_delta_step) delta_step;
  decltype(&ssm_gatednorm_fwd) gatednorm_fwd;
  decltype(&ssm_blocknorm_fwd) blocknorm_fwd;
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
int64_t step_states(Out& out, PyObject* state, PyObject* state_out, bool inplace, bool slots, int64_t batch, Sizes inner,
                    c10::ScalarType type, const Like& like) {
  if (inplace && (state == Py_None || state_out != Py_None))
    throw Refusal{PyExc_ValueError, "inplace needs a state and no state_out"};
  PyObject* target = inplace ? state : state_out;
  if (target == Py_None && state == Py_None && slots)
    throw Refusal{PyExc_ValueError, "slots need a state or a state_out"};
  int64_t n = batch;
  PyObject* rows = target != Py_None ? target : state;
  if (rows != Py_None) {
    const at::Tensor& t = tensor("state", rows);
    if (t.dim() != 1 + (int64_t)inner.size()) fail("state", inner.size() == 2 ? "of three dimensions" : "of four dimensions");
    n = t.size(0);
  }
  if (target == Py_None && state != Py_None && slots) {
    at::Tensor t = tensor("state", state).clone();
    out.ptr = t.data_ptr();
    out.object = THPVariable_Wrap(std::move(t));
  } else {
    c10::SmallVector<int64_t, 4> sizes(1, n);
    sizes.append(inner.begin(), inner.end());
    out.set("state_out", target, sizes, type, like);
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
  const int64_t n = step_states(so, v[3], v[7], truth(v[8]), slots, b, {W - 1, d}, like.type, like);
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

// The workspace of each device's last call of a kind that was given none: its status can still be read (kept_workspace).
enum Kept { kSelscan, kDelta, kKinds };
PyObject* g_kept[kKinds][C10_COMPILE_TIME_MAX_GPUS] = {};

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
      PyObject*& kept = g_kept[kSelscan][like.device.index()];
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
      step_states(so, v[8], v[12], truth(v[13]), slots, a.batch, {a.channels, a.dstate}, at::kFloat, like);
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

PyObject* kept_workspace(PyObject* const* v) {  // device index, whether delta_fwd's
  const long i = PyLong_AsLong(v[0]);
  if (PyErr_Occurred()) return nullptr;
  const Kept kind = truth(v[1]) ? kDelta : kSelscan;
  PyObject* o = i >= 0 && i < C10_COMPILE_TIME_MAX_GPUS && g_kept[kind][i] ? g_kept[kind][i] : Py_None;
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

// q, k, v, dt, beta, A, dt_bias, and scale, softplus, sigmoid, l2norm from v[9] on: what delta_fwd and delta_step share.
// `lead`: dimensions before the heads.
ssm_delta_args delta_args(PyObject* const* v, const Like& like, const at::Tensor& q, int lead) {
  ssm_delta_args a{};
  const at::Tensor &k = tensor("k", v[1]), &x = tensor("v", v[2]);
  const Sizes first = q.sizes().slice(0, lead);
  if (x.dim() != lead + 2 || x.sizes().slice(0, lead) != first) fail("v", text_of(first) + " and heads, their size");
  const int G = narrow(q.size(lead)), N = narrow(q.size(lead + 1));
  const int nh = narrow(x.size(lead)), H = narrow(x.size(lead + 1));
  a.q = tokens("q", q, q.sizes(), like);
  a.k = tokens("k", k, q.sizes(), like);
  a.v = tokens("v", x, x.sizes(), like);
  if (G > 1 && (q.stride(lead) != N || k.stride(lead) != N)) fail("q, k", "contiguous in their last two dimensions");
  if (nh > 1 && x.stride(lead) != H) fail("v", "contiguous in its last two dimensions");
  c10::SmallVector<int64_t, 4> gates(first.begin(), first.end());
  gates.push_back(nh);
  a.dt = tokens("dt", tensor("dt", v[3]), gates, like);
  a.beta = tokens("beta", tensor("beta", v[4]), gates, like);
  a.A = static_cast<const float*>(dense("A", tensor("A", v[5]), {nh}, at::kFloat, like));
  a.dt_bias = floats("dt_bias", v[6], {nh}, like);
  a.batch = first[0];
  a.nheads = nh;
  a.headdim = H;
  a.dstate = N;
  a.ngroups = G;
  a.scale = N > 0 ? 1.f / std::sqrt((float)N) : 1.f;
  if (v[9] != Py_None) {
    const double scale = PyFloat_AsDouble(v[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    a.scale = (float)scale;
  }
  a.softplus = truth(v[10]);
  a.sigmoid = truth(v[11]);
  a.l2norm = truth(v[12]);
  a.dtype = like.code;
  return a;
}

// q, k, v, dt, beta, A, dt_bias, h0, lens, scale, softplus, sigmoid, l2norm, y, h_final, return_final_state, workspace buffer
PyObject* delta_fwd(PyObject* const* v) {
  const at::Tensor& q = tensor("q", v[0]);
  const Like like("q", q);
  if (q.dim() != 4) fail("q", "[b, L, G, N]");
  ssm_delta_args a = delta_args(v, like, q, 2);
  const auto guard = like.guard();
  a.seqlen = q.size(1);
  const int64_t state[] = {a.batch, a.nheads, a.headdim, a.dstate};
  a.h0 = floats("h0", v[7], state, like);
  a.lens = ints("lens", v[8], a.batch, like);
  Out y, h;
  y.set("y", v[13], {a.batch, a.seqlen, a.nheads, a.headdim}, like.type, like);
  a.y = y.ptr;
  if (truth(v[15])) h.set("h_final", v[14], state, at::kFloat, like);
  a.h_final = static_cast<float*>(h.ptr);
  at::Tensor ws;
  PyObject** kept = nullptr;
  if (v[16] != Py_None) {
    ws = tensor("workspace", v[16]);
    if (ws.device() != like.device || ws.scalar_type() != at::kByte || !ws.is_contiguous())
      fail("workspace", "contiguous bytes on q's device");
  } else {
    const size_t need =
        g_fn.delta_fwd_workspace_bytes(a.batch, a.seqlen, a.nheads, a.headdim, a.dstate, a.ngroups, like.code);
    if (need) {
      // the one before goes first: it may be of a gigabyte, and its memory then serves this call
      kept = &g_kept[kDelta][like.device.index()];
      Py_CLEAR(*kept);
      ws = like.empty({(int64_t)need}, at::kByte);
    }
  }
  const ssm_status st = g_fn.delta_fwd(&a, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0,
                                       like.stream());
  if (kept && st == SSM_OK) *kept = THPVariable_Wrap(ws);  // (a call that was refused has written no status)
  return result(st, y, h);
}

// q, k, v, dt, beta, A, dt_bias, state, slots, scale, softplus, sigmoid, l2norm, y, state_out, inplace
PyObject* delta_step(PyObject* const* v) {
  const at::Tensor& q = tensor("q", v[0]);
  const Like like("q", q);
  if (q.dim() != 3) fail("q", "[b, G, N]");
  ssm_delta_args a = delta_args(v, like, q, 1);
  const auto guard = like.guard();
  a.seqlen = 1;
  const int32_t* slots = ints("slots", v[8], a.batch, like);
  Out y, so;
  const int64_t n =
      step_states(so, v[7], v[14], truth(v[15]), slots, a.batch, {a.nheads, a.headdim, a.dstate}, at::kFloat, like);
  a.h0 = floats("state", v[7], {n, a.nheads, a.headdim, a.dstate}, like);
  a.h_final = static_cast<float*>(so.ptr);
  y.set("y", v[13], {a.batch, a.nheads, a.headdim}, like.type, like);
  a.y = y.ptr;
  return result(g_fn.delta_step(&a, slots, n, like.stream()), y, so);
}

// Rows of a tensor [..., d]: its pointer, and the elements from row to row.
int64_t row_stride(const char* name, const at::Tensor& t, int64_t rows, int d) {
  if (t.is_contiguous()) return d;
  if (t.stride(-1) != 1 && d != 1) fail(name, "contiguous in its last dimension");
  return (t.dim() == 2 ? t : t.view({rows, d})).stride(0);
}

PyObject* gatednorm_fwd(PyObject* const* v) {  // x, z, weight, group, gate_first, eps, y
  const at::Tensor &x = tensor("x", v[0]), &z = tensor("z", v[1]), &w = tensor("weight", v[2]);
  const Like like("x", x);
  const long of = PyLong_AsLong(v[3]);
  const double eps = of == -1 && PyErr_Occurred() ? 0.0 : PyFloat_AsDouble(v[5]);
  if (PyErr_Occurred()) return nullptr;
  const int d = x.dim() ? narrow(x.size(-1)) : 0, group = narrow(of);
  const auto guard = like.guard();
  held("z", z, x.sizes(), like.type, like, "a CUDA tensor ");
  const int64_t rows = d ? x.numel() / d : 0;
  const int ww = w.dim() == 1 ? narrow(w.size(0)) : -1;
  if (ww != d && ww != group) fail("weight", "[" + std::to_string(d) + "], or of one group");
  const float* wp = static_cast<const float*>(dense("weight", w, {ww}, at::kFloat, like));
  Out y;
  y.set("y", v[6], x.sizes(), like.type, like);
  const ssm_status st =
      g_fn.gatednorm_fwd(x.data_ptr(), row_stride("x", x, rows, d), z.data_ptr(), row_stride("z", z, rows, d), wp, ww, y.ptr,
                         rows, d, group, truth(v[4]), (float)eps, like.code, like.stream());
  return st != SSM_OK ? PyLong_FromLong(st) : y.give();
}

PyObject* blocknorm_fwd(PyObject* const* v) {  // x, weight, residual, next_weight, z, alpha, eps, y, residual_out
  if (v[2] == Py_None) fail("residual", "a tensor");
  const double alpha = PyFloat_AsDouble(v[5]);
  const double eps = alpha == -1.0 && PyErr_Occurred() ? 0.0 : PyFloat_AsDouble(v[6]);
  if (PyErr_Occurred()) return nullptr;
  Norm n(v[0], v[1], v[2], v[8]);
  const float* next = static_cast<const float*>(dense("next_weight", tensor("next_weight", v[3]), {n.d}, at::kFloat, n.like));
  const void* z = nullptr;
  int64_t z_stride = 0;
  if (v[4] != Py_None) {
    const at::Tensor& t = tensor("z", v[4]);
    held("z", t, n.x.sizes(), n.like.type, n.like, "a CUDA tensor ");
    z = t.data_ptr();
    z_stride = row_stride("z", t, n.rows, n.d);
  }
  Out y;
  y.set("y", v[7], n.x.sizes(), n.like.type, n.like);
  return result(g_fn.blocknorm_fwd(n.x.data_ptr(), n.stride, n.w, z, z_stride, n.residual, n.residual_out.ptr, next, y.ptr,
                                   n.rows, n.d, (float)alpha, (float)eps, n.like.code, n.res_code, n.like.stream()),
                y, n.residual_out);
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

// bind(addresses of the C entry points, in the order of g_fn)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kFns = 12;
  void* p[kFns];
  if (n != kFns) {
    PyErr_SetString(PyExc_TypeError, "twelve addresses");
    return nullptr;
  }
  for (int i = 0; i < kFns; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_fn = {reinterpret_cast<decltype(g_fn.conv_fwd)>(p[0]),
          reinterpret_cast<decltype(g_fn.conv_step)>(p[1]),
          reinterpret_cast<decltype(g_fn.selscan_fwd_workspace_bytes)>(p[2]),
          reinterpret_cast<decltype(g_fn.selscan_fwd)>(p[3]),
          reinterpret_cast<decltype(g_fn.selscan_step)>(p[4]),
          reinterpret_cast<decltype(g_fn.rmsnorm_fwd)>(p[5]),
          reinterpret_cast<decltype(g_fn.rmsnorm_fp8_fwd)>(p[6]),
          reinterpret_cast<decltype(g_fn.delta_fwd_workspace_bytes)>(p[7]),
          reinterpret_cast<decltype(g_fn.delta_fwd)>(p[8]),
          reinterpret_cast<decltype(g_fn.delta_step)>(p[9]),
          reinterpret_cast<decltype(g_fn.gatednorm_fwd)>(p[10]),
          reinterpret_cast<decltype(g_fn.blocknorm_fwd)>(p[11])};
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
                           {"kept_workspace", fast(entry<kept_workspace, 2>), METH_FASTCALL, nullptr},
                           {"rmsnorm_fp8_fwd", fast(entry<rmsnorm_fp8_fwd, 8>), METH_FASTCALL, nullptr},
                           {"delta_fwd", fast(entry<delta_fwd, 17>), METH_FASTCALL, nullptr},
                           {"delta_step", fast(entry<delta_step, 16>), METH_FASTCALL, nullptr},
                           {"gatednorm_fwd", fast(entry<gatednorm_fwd, 7>), METH_FASTCALL, nullptr},
                           {"blocknorm_fwd", fast(entry<blocknorm_fwd, 9>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) { return PyModule_Create(&g_module); }
