// CPython module `_native`: the binding of the linear attention with a decay per head, of the
// block norm, of the gated recurrence, of the head norms with rotation and of the gated
// feed-forward block.  Argument marshalling only, like the ctypes part of the package: it checks
// tensors against each other, allocates results that the caller did not give, and calls the C
// entry points, whose addresses the package hands over (bind).  At their smallest these calls
// take 2 to 10 us on the GPU; the same steps in Python took 11 to 23 us per call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>
#include <type_traits>

#include "../../include/loglinear.h"

namespace {

struct Entry {
  decltype(&lindecay_fwd) fwd;
  decltype(&lindecay_fwd_workspace_bytes) fwd_bytes;
  decltype(&lindecay_bwd) bwd;
  decltype(&lindecay_bwd_workspace_bytes) bwd_bytes;
  decltype(&lindecay_decode_step) step;
  decltype(&blocknorm_fwd) bn_fwd;
  decltype(&blocknorm_bwd) bn_bwd;
  decltype(&blocknorm_bwd_workspace_bytes) bn_bytes;
  decltype(&gatescan_fwd) gs_fwd;
  decltype(&gatescan_bwd) gs_bwd;
  decltype(&gatescan_bwd_workspace_bytes) gs_bwd_bytes;
  decltype(&gatescan_decode_step) gs_step;
  decltype(&headrope_fwd) hr_fwd;
  decltype(&headrope_bwd) hr_bwd;
  decltype(&headrope_bwd_workspace_bytes) hr_bytes;
  decltype(&ffgate_fwd) ff_fwd;
  decltype(&ffgate_fwd_workspace_bytes) ff_fwd_bytes;
  decltype(&ffgate_bwd) ff_bwd;
  decltype(&ffgate_bwd_workspace_bytes) ff_bwd_bytes;
} entry;
PyObject* error_class = nullptr;  // LogLinearError(status, where)

// A Python exception that has been set.
struct Raised {};

[[noreturn]] void refuse(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}
std::string sizes_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}
const char* type_text(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : t == at::kInt ? "torch.int32"
                                                                                                  : c10::toString(t);
}

// An argument: a tensor, or undefined for None.
const at::Tensor& tensor(PyObject* x, const char* name, bool optional) {
  static const at::Tensor none;
  if (x == Py_None) {
    if (!optional) refuse(PyExc_ValueError, std::string(name) + " is required");
    return none;
  }
  if (!THPVariable_Check(x)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(x);
}
void check(const at::Tensor& x, const char* name, at::IntArrayRef sizes, at::ScalarType type, int device) {
  if (!x.defined()) return;
  if (x.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + type_text(type) + ", got " + type_text(x.scalar_type()));
  if (x.sizes() != sizes)
    refuse(PyExc_ValueError,
          std::string(name) + " must have shape " + sizes_text(sizes) + ", got " + sizes_text(x.sizes()));
  if (!x.is_cuda() || x.get_device() != device)
    refuse(PyExc_ValueError, std::string(name) + " is on " + x.device().str() + ", the first tensor on cuda:" +
                                std::to_string(device));
  if (!x.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
}
int cuda_device(const at::Tensor& x) {
  if (!x.is_cuda()) refuse(PyExc_ValueError, "tensors must be on a CUDA device, got " + x.device().str());
  return x.get_device();
}
ll_dtype dtype_code(const at::Tensor& x) {
  if (x.scalar_type() == at::kBFloat16) return LL_BF16;
  if (x.scalar_type() == at::kFloat) return LL_F32;
  refuse(PyExc_TypeError, std::string("unsupported dtype ") + type_text(x.scalar_type()));
}
template <typename T = void>
T* ptr(const at::Tensor& x) {
  return x.defined() ? static_cast<T*>(x.data_ptr()) : nullptr;
}
// A new contiguous tensor like x (undefined for undefined), without the dispatcher's steps.
at::Tensor new_like(const at::Tensor& x) {
  return x.defined() ? at::Tensor(at::detail::empty_cuda(x.sizes(), x.scalar_type(), x.device(), std::nullopt)) : at::Tensor();
}
at::Tensor given_or_like(const at::Tensor& x, const at::Tensor& like) { return x.defined() ? x : new_like(like); }
// The caller's tensors that a call has written: where autograd keeps one of them for a backward,
// its raised version says that it is no longer what it was.  (Inference tensors have none.)
void written(std::initializer_list<at::Tensor> xs) {
  for (const at::Tensor& x : xs)
    if (x.defined() && !x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}

// Where a call runs: the device and stream, both current while it allocates.  Memory that the
// caching allocator hands out belongs to the current stream; were it another one than the
// call's, a result could take the place of what that stream still reads, and a workspace
// could be handed on while the call still uses it.
struct Target {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard stream;
  void* handle;
  Target(PyObject* s, int index) : device(static_cast<c10::DeviceIndex>(index)) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index));
    handle = current.stream();
    if (s == Py_None) return;
    void* given = PyLong_AsVoidPtr(s);
    if (!given && PyErr_Occurred()) throw Raised{};
    if (given == handle) return;
    handle = given;
    stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(given),
                                                         static_cast<c10::DeviceIndex>(index)));
  }
};
void check_status(ll_status st, const char* where) {
  if (st == LL_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "is", static_cast<int>(st), where);
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw Raised{};
}
// The caller's workspace, or a new one of `need` bytes (none for 16, which stands for none).
at::Tensor workspace_of(PyObject* given, size_t need, int device, const char* where) {
  if (need == 0) check_status(LL_ERR_SHAPE, where);
  const at::Tensor& w = tensor(given, "workspace", true);
  if (!w.defined())
    return need <= 16 ? at::Tensor()
                      : at::Tensor(at::detail::empty_cuda({static_cast<int64_t>(need)}, at::kByte,
                                                          c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                                          std::nullopt));
  if (!w.is_cuda() || w.get_device() != device || !w.is_contiguous())
    refuse(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:" + std::to_string(device));
  return w;
}
size_t bytes_of(const at::Tensor& x) { return x.defined() ? x.nbytes() : 0; }

PyObject* wrap(const at::Tensor& x) {
  if (x.defined()) return THPVariable_Wrap(x);
  Py_RETURN_NONE;
}
PyObject* wrap_all(std::initializer_list<at::Tensor> xs) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(xs.size()));
  if (!t) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& x : xs) {
    PyObject* o = wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw Raised{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  if (!error_class) {
    PyErr_SetString(PyExc_RuntimeError, "the native binding has not been bound to the library");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// q, k (.., G, d_k), v (.., H, d_v), log_a (H) against each other; lead = 2 for sequences.
struct Lin {
  ll_shape shape;
  int device;
  int64_t states[4];
  at::IntArrayRef state_sizes() const { return {states, 4}; }
};
Lin lin_checked(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& log_a, int lead) {
  if (q.dim() != lead + 2 || v.dim() != lead + 2)
    refuse(PyExc_ValueError, "q and v must have " + std::to_string(lead + 2) + " dimensions, got " +
                                std::to_string(q.dim()) + " and " + std::to_string(v.dim()));
  Lin l{};
  l.device = cuda_device(q);
  const int64_t G = q.size(lead), dk = q.size(lead + 1), H = v.size(lead), dv = v.size(lead + 1), B = q.size(0);
  const int64_t T = lead == 2 ? q.size(1) : 1;
  if (G == 0 || H % G)
    refuse(PyExc_ValueError, std::to_string(H) + " heads do not divide into " + std::to_string(G) + " groups");
  const int64_t most = 0x7fffffff;
  if (B > most || T > most || H > most || dk > most || dv > most) check_status(LL_ERR_SHAPE, "lindecay");
  l.shape = ll_shape{static_cast<int>(B), static_cast<int>(T), static_cast<int>(H), static_cast<int>(H / G),
                     static_cast<int>(dk), static_cast<int>(dv), 0, 0, dtype_code(q)};
  const int64_t vs[4] = {B, lead == 2 ? T : H, lead == 2 ? H : dv, dv};
  check(q, "q", q.sizes(), q.scalar_type(), l.device);
  check(k, "k", q.sizes(), q.scalar_type(), l.device);
  check(v, "v", at::IntArrayRef(vs, lead + 2), q.scalar_type(), l.device);
  check(log_a, "log_a", at::IntArrayRef(&H, 1), at::kFloat, l.device);
  l.states[0] = B;
  l.states[1] = H;
  l.states[2] = dk;
  l.states[3] = dv;
  return l;
}

PyObject* py_lindecay_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q", false), &k = tensor(a[1], "k", false), &v = tensor(a[2], "v", false),
                     &log_a = tensor(a[3], "log_a", false), &lengths = tensor(a[4], "lengths", true),
                     &s_in = tensor(a[5], "state_in", true), &s_out = tensor(a[6], "state_out", true),
                     &o_given = tensor(a[7], "o", true);
    const Lin l = lin_checked(q, k, v, log_a, 2);
    check(lengths, "lengths", q.sizes().slice(0, 1), at::kInt, l.device);
    check(s_in, "state_in", l.state_sizes(), at::kFloat, l.device);
    check(s_out, "state_out", l.state_sizes(), at::kFloat, l.device);
    check(o_given, "o", v.sizes(), v.scalar_type(), l.device);
    const Target on(a[9], l.device);
    const at::Tensor ws = workspace_of(a[8], entry.fwd_bytes(&l.shape), l.device, "lindecay_fwd");
    const at::Tensor o = given_or_like(o_given, v);
    ll_status r;
    Py_BEGIN_ALLOW_THREADS
    r = entry.fwd(&l.shape, ptr(q), ptr(k), ptr(v), ptr<float>(log_a), ptr<int>(lengths), ptr<float>(s_in), ptr(o),
                  ptr<float>(s_out), ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(r, "lindecay_fwd");
    written({o_given, s_out});
    return wrap(o);
  });
}

PyObject* py_lindecay_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q", false), &k = tensor(a[1], "k", false), &v = tensor(a[2], "v", false),
                     &log_a = tensor(a[3], "log_a", false), &dO = tensor(a[4], "dO", false),
                     &lengths = tensor(a[5], "lengths", true), &s_in = tensor(a[6], "state_in", true),
                     &ds_out = tensor(a[7], "dstate_out", true), &ds_in = tensor(a[8], "dstate_in", true);
    const Lin l = lin_checked(q, k, v, log_a, 2);
    check(dO, "dO", v.sizes(), v.scalar_type(), l.device);
    check(lengths, "lengths", q.sizes().slice(0, 1), at::kInt, l.device);
    check(s_in, "state_in", l.state_sizes(), at::kFloat, l.device);
    check(ds_out, "dstate_out", l.state_sizes(), at::kFloat, l.device);
    check(ds_in, "dstate_in", l.state_sizes(), at::kFloat, l.device);
    const Target on(a[10], l.device);
    const at::Tensor ws = workspace_of(a[9], entry.bwd_bytes(&l.shape), l.device, "lindecay_bwd");
    const at::Tensor dq = new_like(q), dk = new_like(k), dv = new_like(v);
    ll_status r;
    Py_BEGIN_ALLOW_THREADS
    r = entry.bwd(&l.shape, ptr(q), ptr(k), ptr(v), ptr<float>(log_a), ptr<int>(lengths), ptr<float>(s_in), ptr(dO),
                  ptr<float>(ds_out), ptr(dq), ptr(dk), ptr(dv), ptr<float>(ds_in), ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(r, "lindecay_bwd");
    written({ds_in});
    return wrap_all({dq, dk, dv});
  });
}

PyObject* py_lindecay_decode_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q_t", false), &k = tensor(a[1], "k_t", false), &v = tensor(a[2], "v_t", false),
                     &log_a = tensor(a[3], "log_a", false), &states = tensor(a[4], "states", false),
                     &o_given = tensor(a[5], "o_t", true);
    const Lin l = lin_checked(q, k, v, log_a, 1);
    check(states, "states", l.state_sizes(), at::kFloat, l.device);
    check(o_given, "o_t", v.sizes(), v.scalar_type(), l.device);
    const Target on(a[6], l.device);
    const at::Tensor o = given_or_like(o_given, v);
    ll_status r;
    Py_BEGIN_ALLOW_THREADS
    r = entry.step(&l.shape, ptr(q), ptr(k), ptr(v), ptr<float>(log_a), ptr(o), ptr<float>(states), on.handle);
    Py_END_ALLOW_THREADS
    check_status(r, "lindecay_decode_step");
    written({o_given, states});
    return wrap(o);
  });
}

// Shape of a block norm over `first` (.., D) with group (None: D), act and eps arguments.
blocknorm_shape bn_shape(const at::Tensor& first, PyObject* group, PyObject* act, PyObject* eps) {
  if (first.dim() == 0 || first.numel() == 0)
    refuse(PyExc_ValueError, "activations must hold at least one row, got shape " + sizes_text(first.sizes()));
  const int64_t D = first.size(first.dim() - 1);
  blocknorm_shape s{};
  s.rows = first.numel() / D;
  const long long g = group == Py_None ? D : PyLong_AsLongLong(group);
  s.act = static_cast<int>(PyLong_AsLong(act));
  s.eps = static_cast<float>(PyFloat_AsDouble(eps));
  if (PyErr_Occurred()) throw Raised{};
  if (D > 0x7fffffff || g > 0x7fffffff || g < 1) check_status(LL_ERR_SHAPE, "blocknorm");
  s.dim = static_cast<int>(D);
  s.group = static_cast<int>(g);
  s.dtype = dtype_code(first);
  return s;
}

PyObject* py_blocknorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor &y = tensor(a[0], "y", true), &w_post = tensor(a[1], "w_post", true), &x = tensor(a[2], "x", true),
                     &gate = tensor(a[3], "gate", true), &scale = tensor(a[4], "scale", true),
                     &w_pre = tensor(a[5], "w_pre", true), &xn_given = tensor(a[9], "x_new", true),
                     &h_given = tensor(a[10], "h", true);
    const at::Tensor& first = y.defined() ? y : x;
    if (!first.defined()) refuse(PyExc_ValueError, "y or x is required");
    const int device = cuda_device(first);
    const blocknorm_shape s = bn_shape(first, a[6], a[7], a[8]);
    const int64_t D = s.dim;
    const at::IntArrayRef weights(&D, 1);
    const at::ScalarType t = first.scalar_type();
    check(y, "y", first.sizes(), t, device);
    check(x, "x", first.sizes(), t, device);
    check(gate, "gate", first.sizes(), t, device);
    check(xn_given, "x_new", first.sizes(), t, device);
    check(h_given, "h", first.sizes(), t, device);
    check(w_post, "w_post", weights, at::kFloat, device);
    check(scale, "scale", weights, at::kFloat, device);
    check(w_pre, "w_pre", weights, at::kFloat, device);
    if (!y.defined()) {
      if (xn_given.defined() || gate.defined() || w_post.defined() || scale.defined())
        refuse(PyExc_ValueError, "without y there is no x_new, gate, w_post or scale");
      if (!w_pre.defined() && !h_given.defined())
        refuse(PyExc_ValueError, "nothing to compute: neither y nor w_pre is given");
    }
    const Target on(a[11], device);
    const at::Tensor xn = y.defined() ? given_or_like(xn_given, first) : at::Tensor();
    const at::Tensor h = w_pre.defined() ? given_or_like(h_given, first) : h_given;
    ll_status r;
    Py_BEGIN_ALLOW_THREADS
    r = entry.bn_fwd(&s, ptr(x), ptr(y), ptr(gate), ptr<float>(w_post), ptr<float>(scale), ptr<float>(w_pre), ptr(xn),
                     ptr(h), on.handle);
    Py_END_ALLOW_THREADS
    check_status(r, "blocknorm_fwd");
    written({xn_given, h_given});
    return wrap_all({y.defined() ? xn : x, h});
  });
}

PyObject* py_blocknorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor &dx_new = tensor(a[0], "dx_new", true), &y = tensor(a[1], "y", true),
                     &w_post = tensor(a[2], "w_post", true), &dh = tensor(a[3], "dh", true),
                     &x_new = tensor(a[4], "x_new", true), &gate = tensor(a[5], "gate", true),
                     &scale = tensor(a[6], "scale", true), &w_pre = tensor(a[7], "w_pre", true);
    const at::Tensor& first = dx_new.defined() ? dx_new : dh;
    if (!first.defined()) refuse(PyExc_ValueError, "dx_new or dh is required");
    if (dh.defined() != x_new.defined()) refuse(PyExc_ValueError, "dh and x_new go together");
    const int device = cuda_device(first);
    const blocknorm_shape s = bn_shape(first, a[8], a[9], a[10]);
    const int64_t D = s.dim;
    const at::IntArrayRef weights(&D, 1);
    const at::ScalarType t = first.scalar_type();
    check(dx_new, "dx_new", first.sizes(), t, device);
    check(dh, "dh", first.sizes(), t, device);
    check(x_new, "x_new", first.sizes(), t, device);
    check(y, "y", first.sizes(), t, device);
    check(gate, "gate", first.sizes(), t, device);
    check(w_post, "w_post", weights, at::kFloat, device);
    check(scale, "scale", weights, at::kFloat, device);
    check(w_pre, "w_pre", weights, at::kFloat, device);
    const bool residual = a[11] == Py_None ? !y.defined() || scale.defined() || x_new.defined() : a[11] == Py_True;
    const Target on(a[13], device);
    const at::Tensor ws = workspace_of(a[12], entry.bn_bytes(&s), device, "blocknorm_bwd");
    const at::Tensor dx = residual ? new_like(first) : at::Tensor(), dy = new_like(y), dgate = new_like(gate),
                     dw_post = new_like(w_post), dscale = new_like(scale), dw_pre = new_like(w_pre);
    ll_status r;
    Py_BEGIN_ALLOW_THREADS
    r = entry.bn_bwd(&s, ptr(dx_new), ptr(dh), ptr(x_new), ptr(y), ptr(gate), ptr<float>(w_post), ptr<float>(scale),
                     ptr<float>(w_pre), ptr(dx), ptr(dy), ptr(dgate), ptr<float>(dw_post), ptr<float>(dscale),
                     ptr<float>(dw_pre), ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(r, "blocknorm_bwd");
    return wrap_all({dx, dy, dgate, dw_post, dscale, dw_pre});
  });
}

// ---- gated recurrence ----
// x, r, i (lead.., D) and decay (D) against each other; lead = 2 for sequences.
struct Scan {
  gatescan_shape shape;
  int device;
  int64_t states[2];
  at::IntArrayRef state_sizes() const { return {states, 2}; }
};
Scan scan_checked(const at::Tensor& x, const at::Tensor& r, const at::Tensor& i, const at::Tensor& decay, PyObject* mix,
                  int lead) {
  if (x.dim() != lead + 1)
    refuse(PyExc_ValueError, "x must have " + std::to_string(lead + 1) + " dimensions, got " + std::to_string(x.dim()));
  Scan l{};
  l.device = cuda_device(x);
  const int64_t B = x.size(0), T = lead == 2 ? x.size(1) : 1, D = x.size(lead);
  const int64_t most = 0x7fffffff;
  if (B > most || T > most || D > most) check_status(LL_ERR_SHAPE, "gatescan");
  const int m = static_cast<int>(PyLong_AsLong(mix));
  if (PyErr_Occurred()) throw Raised{};
  l.shape = gatescan_shape{static_cast<int>(B), static_cast<int>(T), static_cast<int>(D), m, dtype_code(x)};
  check(x, "x", x.sizes(), x.scalar_type(), l.device);
  check(r, "r", x.sizes(), x.scalar_type(), l.device);
  check(i, "i", x.sizes(), x.scalar_type(), l.device);
  check(decay, "decay", at::IntArrayRef(&D, 1), at::kFloat, l.device);
  l.states[0] = B;
  l.states[1] = D;
  return l;
}

PyObject* py_gatescan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x", false), &r = tensor(a[1], "r", false), &decay = tensor(a[2], "decay", false),
                     &i = tensor(a[3], "i", true), &lengths = tensor(a[5], "lengths", true),
                     &s_in = tensor(a[6], "state_in", true), &s_out = tensor(a[7], "state_out", true),
                     &h_given = tensor(a[8], "h", true);
    const Scan l = scan_checked(x, r, i, decay, a[4], 2);
    check(lengths, "lengths", x.sizes().slice(0, 1), at::kInt, l.device);
    check(s_in, "state_in", l.state_sizes(), at::kFloat, l.device);
    check(s_out, "state_out", l.state_sizes(), at::kFloat, l.device);
    check(h_given, "h", x.sizes(), x.scalar_type(), l.device);
    const Target on(a[9], l.device);
    const at::Tensor h = given_or_like(h_given, x);
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.gs_fwd(&l.shape, ptr(x), ptr(r), ptr(i), ptr<float>(decay), ptr<int>(lengths), ptr<float>(s_in), ptr(h),
                      ptr<float>(s_out), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "gatescan_fwd");
    written({h_given, s_out});
    return wrap(h);
  });
}

PyObject* py_gatescan_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor &dh = tensor(a[0], "dh", false), &x = tensor(a[1], "x", false), &r = tensor(a[2], "r", false),
                     &decay = tensor(a[3], "decay", false), &h = tensor(a[4], "h", false), &i = tensor(a[5], "i", true),
                     &lengths = tensor(a[7], "lengths", true), &s_in = tensor(a[8], "state_in", true),
                     &ds_out = tensor(a[9], "dstate_out", true), &ds_in = tensor(a[10], "dstate_in", true);
    const Scan l = scan_checked(x, r, i, decay, a[6], 2);
    check(dh, "dh", x.sizes(), x.scalar_type(), l.device);
    check(h, "h", x.sizes(), x.scalar_type(), l.device);
    check(lengths, "lengths", x.sizes().slice(0, 1), at::kInt, l.device);
    check(s_in, "state_in", l.state_sizes(), at::kFloat, l.device);
    check(ds_out, "dstate_out", l.state_sizes(), at::kFloat, l.device);
    check(ds_in, "dstate_in", l.state_sizes(), at::kFloat, l.device);
    const Target on(a[12], l.device);
    const at::Tensor ws = workspace_of(a[11], entry.gs_bwd_bytes(&l.shape), l.device, "gatescan_bwd");
    const at::Tensor dx = new_like(x), dr = new_like(r), di = new_like(i), ddecay = new_like(decay);
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.gs_bwd(&l.shape, ptr(dh), ptr(x), ptr(r), ptr(i), ptr<float>(decay), ptr(h), ptr<int>(lengths),
                      ptr<float>(s_in), ptr<float>(ds_out), ptr(dx), ptr(dr), ptr(di), ptr<float>(ddecay),
                      ptr<float>(ds_in), ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "gatescan_bwd");
    written({ds_in});
    return wrap_all({dx, dr, di, ddecay});
  });
}

PyObject* py_gatescan_decode_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x_t", false), &r = tensor(a[1], "r_t", false),
                     &decay = tensor(a[2], "decay", false), &states = tensor(a[3], "states", false),
                     &i = tensor(a[4], "i_t", true), &h_given = tensor(a[6], "h_t", true);
    const Scan l = scan_checked(x, r, i, decay, a[5], 1);
    check(states, "states", l.state_sizes(), at::kFloat, l.device);
    check(h_given, "h_t", x.sizes(), x.scalar_type(), l.device);
    const Target on(a[7], l.device);
    const at::Tensor h = given_or_like(h_given, x);
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.gs_step(&l.shape, ptr(x), ptr(r), ptr(i), ptr<float>(decay), ptr<float>(states), ptr(h), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "gatescan_decode_step");
    written({h_given, states});
    return wrap(h);
  });
}

// ---- norms and rotation of heads ----
// q (lead.., G_q, d) and k (lead.., G_k, d) against each other; a: layout, norm, eps, scale_q, scale_k.
struct Heads {
  headrope_shape shape;
  int device;
};
Heads heads_checked(const at::Tensor& q, const at::Tensor& k, const at::Tensor& w_q, const at::Tensor& w_k,
                    const at::Tensor& inv_freq, const at::Tensor& positions, PyObject* const* a) {
  if (q.dim() < 2 || q.numel() == 0)
    refuse(PyExc_ValueError, "q must be (.., heads, values) with at least one token, got " + sizes_text(q.sizes()));
  Heads l{};
  l.device = cuda_device(q);
  const int64_t lead = q.dim() - 2, G = q.size(lead), d = q.size(lead + 1);
  headrope_shape& s = l.shape;
  s.layout = static_cast<int>(PyLong_AsLong(a[0]));
  s.norm = static_cast<int>(PyLong_AsLong(a[1]));
  s.eps = static_cast<float>(PyFloat_AsDouble(a[2]));
  s.scale_q = static_cast<float>(PyFloat_AsDouble(a[3]));
  s.scale_k = static_cast<float>(PyFloat_AsDouble(a[4]));
  if (PyErr_Occurred()) throw Raised{};
  check(q, "q", q.sizes(), q.scalar_type(), l.device);
  int64_t Gk = 0;
  if (k.defined()) {
    if (k.dim() != q.dim() || k.size(lead + 1) != d || k.sizes().slice(0, lead) != q.sizes().slice(0, lead) || k.numel() == 0)
      refuse(PyExc_ValueError, "k " + sizes_text(k.sizes()) + " must be as q " + sizes_text(q.sizes()) +
                                  ", but for the number of heads");
    check(k, "k", k.sizes(), q.scalar_type(), l.device);
    Gk = k.size(lead);
  } else if (w_k.defined()) {
    refuse(PyExc_ValueError, "w_k is given without k");
  }
  check(w_q, "w_q", at::IntArrayRef(&d, 1), at::kFloat, l.device);
  check(w_k, "w_k", at::IntArrayRef(&d, 1), at::kFloat, l.device);
  int64_t rot = 0;
  if (inv_freq.defined()) {
    if (inv_freq.dim() != 1) refuse(PyExc_ValueError, "inv_freq must have one dimension");
    rot = 2 * inv_freq.size(0);
    if (rot > d)
      refuse(PyExc_ValueError, "inv_freq rotates " + std::to_string(rot) + " values, a head has " + std::to_string(d));
    check(inv_freq, "inv_freq", inv_freq.sizes(), at::kFloat, l.device);
    if (!positions.defined() && rot && lead != 2)
      refuse(PyExc_ValueError, "positions are required unless q is (B, T, heads, values)");
  }
  check(positions, "positions", q.sizes().slice(0, lead), at::kInt, l.device);
  const int64_t rows = q.numel() / (G * d), most = 0x7fffffff;
  if (rows > most || G > most || Gk > most || d > most) check_status(LL_ERR_SHAPE, "headrope");
  s.rows = rows;
  s.T = lead == 2 ? static_cast<int>(q.size(1)) : 1;
  s.q_heads = static_cast<int>(G);
  s.k_heads = static_cast<int>(Gk);
  s.dim = static_cast<int>(d);
  s.rot = static_cast<int>(rot);
  s.dtype = dtype_code(q);
  return l;
}

PyObject* py_headrope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q", false), &k = tensor(a[1], "k", true), &w_q = tensor(a[2], "w_q", true),
                     &w_k = tensor(a[3], "w_k", true), &inv_freq = tensor(a[4], "inv_freq", true),
                     &positions = tensor(a[5], "positions", true), &qo_given = tensor(a[11], "q_out", true),
                     &ko_given = tensor(a[12], "k_out", true);
    const Heads l = heads_checked(q, k, w_q, w_k, inv_freq, positions, a + 6);
    check(qo_given, "q_out", q.sizes(), q.scalar_type(), l.device);
    if (ko_given.defined() && !k.defined()) refuse(PyExc_ValueError, "k_out is given without k");
    if (k.defined()) check(ko_given, "k_out", k.sizes(), q.scalar_type(), l.device);
    const Target on(a[13], l.device);
    const at::Tensor qo = given_or_like(qo_given, q), ko = given_or_like(ko_given, k);
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.hr_fwd(&l.shape, ptr(q), ptr(k), ptr<float>(w_q), ptr<float>(w_k), ptr<float>(inv_freq),
                      ptr<int>(positions), ptr(qo), ptr(ko), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "headrope_fwd");
    written({qo_given, ko_given});
    return wrap_all({qo, ko});
  });
}

PyObject* py_headrope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor &dqo = tensor(a[0], "dq_out", false), &q = tensor(a[1], "q", false), &dko = tensor(a[2], "dk_out", true),
                     &k = tensor(a[3], "k", true), &w_q = tensor(a[4], "w_q", true), &w_k = tensor(a[5], "w_k", true),
                     &inv_freq = tensor(a[6], "inv_freq", true), &positions = tensor(a[7], "positions", true),
                     &dq_given = tensor(a[13], "dq", true), &dk_given = tensor(a[14], "dk", true);
    const Heads l = heads_checked(q, k, w_q, w_k, inv_freq, positions, a + 8);
    check(dqo, "dq_out", q.sizes(), q.scalar_type(), l.device);
    if (k.defined() != dko.defined()) refuse(PyExc_ValueError, "k and dk_out go together");
    if (k.defined()) check(dko, "dk_out", k.sizes(), q.scalar_type(), l.device);
    check(dq_given, "dq", q.sizes(), q.scalar_type(), l.device);
    if (dk_given.defined() && !k.defined()) refuse(PyExc_ValueError, "dk is given without k");
    if (k.defined()) check(dk_given, "dk", k.sizes(), q.scalar_type(), l.device);
    const Target on(a[16], l.device);
    const bool sums = w_q.defined() || w_k.defined();
    const at::Tensor ws = sums ? workspace_of(a[15], entry.hr_bytes(&l.shape), l.device, "headrope_bwd") : at::Tensor();
    const at::Tensor dq = given_or_like(dq_given, q), dk = given_or_like(dk_given, k), dw_q = new_like(w_q), dw_k = new_like(w_k);
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.hr_bwd(&l.shape, ptr(dqo), ptr(dko), ptr(q), ptr(k), ptr<float>(w_q), ptr<float>(w_k),
                      ptr<float>(inv_freq), ptr<int>(positions), ptr(dq), ptr(dk), ptr<float>(dw_q), ptr<float>(dw_k),
                      ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "headrope_bwd");
    written({dq_given, dk_given});
    return wrap_all({dq, dk, dw_q, dw_k});
  });
}

// ---- gated feed-forward block ----
// x (.., D) and both weights (F, D) against each other, and the sizes of (.., F).
struct Feed {
  ffgate_shape shape;
  int device;
  c10::SmallVector<int64_t, 5> wide;
};
Feed feed_checked(const at::Tensor& x, const at::Tensor& w_gate, const at::Tensor& w_up, PyObject* act) {
  if (x.dim() == 0 || x.numel() == 0)
    refuse(PyExc_ValueError, "x must hold at least one row, got shape " + sizes_text(x.sizes()));
  if (w_gate.dim() != 2) refuse(PyExc_ValueError, "w_gate must have 2 dimensions, got " + std::to_string(w_gate.dim()));
  Feed l{};
  l.device = cuda_device(x);
  const int64_t D = x.size(x.dim() - 1), F = w_gate.size(0), most = 0x7fffffff;
  const int64_t ws[2] = {F, D};
  check(x, "x", x.sizes(), x.scalar_type(), l.device);
  check(w_gate, "w_gate", at::IntArrayRef(ws, 2), x.scalar_type(), l.device);
  check(w_up, "w_up", at::IntArrayRef(ws, 2), x.scalar_type(), l.device);
  if (D > most || F > most) check_status(LL_ERR_SHAPE, "ffgate");
  l.shape.rows = x.numel() / D;
  l.shape.dim = static_cast<int>(D);
  l.shape.ff = static_cast<int>(F);
  l.shape.act = static_cast<int>(PyLong_AsLong(act));
  if (PyErr_Occurred()) throw Raised{};
  l.shape.dtype = dtype_code(x);
  l.wide.append(x.sizes().begin(), x.sizes().end());
  l.wide.back() = F;
  return l;
}

PyObject* py_ffgate_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x", false), &w_gate = tensor(a[1], "w_gate", false),
                     &w_up = tensor(a[2], "w_up", false), &m_given = tensor(a[4], "m", true),
                     &gate = tensor(a[5], "gate", true), &up = tensor(a[6], "up", true);
    const Feed l = feed_checked(x, w_gate, w_up, a[3]);
    check(m_given, "m", l.wide, x.scalar_type(), l.device);
    check(gate, "gate", l.wide, x.scalar_type(), l.device);
    check(up, "up", l.wide, x.scalar_type(), l.device);
    if (gate.defined() != up.defined()) refuse(PyExc_ValueError, "gate and up go together");
    const Target on(a[8], l.device);
    const at::Tensor ws = workspace_of(a[7], entry.ff_fwd_bytes(&l.shape), l.device, "ffgate_fwd");
    const at::Tensor m = m_given.defined() ? m_given
                                           : at::Tensor(at::detail::empty_cuda(l.wide, x.scalar_type(), x.device(), std::nullopt));
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.ff_fwd(&l.shape, ptr(x), ptr(w_gate), ptr(w_up), ptr(m), ptr(gate), ptr(up), ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "ffgate_fwd");
    written({m_given, gate, up});
    return wrap(m);
  });
}

// a: dm, x, w_gate, w_up, gate, up, act, which of dx, dw_gate, dw_up (bits 0, 1, 2), workspace, stream
PyObject* py_ffgate_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &dm = tensor(a[0], "dm", false), &x = tensor(a[1], "x", false), &w_gate = tensor(a[2], "w_gate", false),
                     &w_up = tensor(a[3], "w_up", false), &gate = tensor(a[4], "gate", false), &up = tensor(a[5], "up", false);
    const Feed l = feed_checked(x, w_gate, w_up, a[6]);
    check(dm, "dm", l.wide, x.scalar_type(), l.device);
    check(gate, "gate", l.wide, x.scalar_type(), l.device);
    check(up, "up", l.wide, x.scalar_type(), l.device);
    const long which = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) throw Raised{};
    const Target on(a[9], l.device);
    const at::Tensor ws = workspace_of(a[8], entry.ff_bwd_bytes(&l.shape), l.device, "ffgate_bwd");
    const at::Tensor none, dx = which & 1 ? new_like(x) : none, dwg = which & 2 ? new_like(w_gate) : none,
                           dwu = which & 4 ? new_like(w_up) : none;
    ll_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry.ff_bwd(&l.shape, ptr(dm), ptr(x), ptr(w_gate), ptr(w_up), ptr(gate), ptr(up), ptr(dx), ptr(dwg), ptr(dwu),
                      ptr(ws), bytes_of(ws), on.handle);
    Py_END_ALLOW_THREADS
    check_status(st, "ffgate_bwd");
    return wrap_all({dx, dwg, dwu});
  });
}

// bind(addresses: tuple of ints in the order of Entry, error class)
constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);

PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind(addresses, error class)");
    return nullptr;
  }
  void* p[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a NULL address");
      return nullptr;
    }
  }
  static_assert(std::is_trivially_copyable<Entry>::value, "Entry is function pointers alone");
  std::memcpy(static_cast<void*>(&entry), p, sizeof entry);
  Py_INCREF(a[1]);
  Py_XSETREF(error_class, a[1]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),          FAST(lindecay_fwd),  FAST(lindecay_bwd), FAST(lindecay_decode_step),
                         FAST(blocknorm_fwd), FAST(blocknorm_bwd),
                         FAST(gatescan_fwd),  FAST(gatescan_bwd),  FAST(gatescan_decode_step),
                         FAST(headrope_fwd),  FAST(headrope_bwd),  FAST(ffgate_fwd),   FAST(ffgate_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
