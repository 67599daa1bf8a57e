// CPython module `_native`: the binding of the linear attention with a decay per head and of
// the block norm.  Argument marshalling only, like the ctypes part of the package: it checks
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

#include <initializer_list>
#include <string>

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

// bind(addresses: tuple of eight ints in the order of Entry, error class)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 8) {
    PyErr_SetString(PyExc_TypeError, "bind(addresses, error class)");
    return nullptr;
  }
  void* p[8];
  for (Py_ssize_t i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a NULL address");
      return nullptr;
    }
  }
  entry.fwd = reinterpret_cast<decltype(entry.fwd)>(p[0]);
  entry.fwd_bytes = reinterpret_cast<decltype(entry.fwd_bytes)>(p[1]);
  entry.bwd = reinterpret_cast<decltype(entry.bwd)>(p[2]);
  entry.bwd_bytes = reinterpret_cast<decltype(entry.bwd_bytes)>(p[3]);
  entry.step = reinterpret_cast<decltype(entry.step)>(p[4]);
  entry.bn_fwd = reinterpret_cast<decltype(entry.bn_fwd)>(p[5]);
  entry.bn_bwd = reinterpret_cast<decltype(entry.bn_bwd)>(p[6]);
  entry.bn_bytes = reinterpret_cast<decltype(entry.bn_bytes)>(p[7]);
  Py_INCREF(a[1]);
  Py_XSETREF(error_class, a[1]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),          FAST(lindecay_fwd),  FAST(lindecay_bwd), FAST(lindecay_decode_step),
                         FAST(blocknorm_fwd), FAST(blocknorm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
