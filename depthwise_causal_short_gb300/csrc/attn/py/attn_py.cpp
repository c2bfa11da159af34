// attn_py.cpp -- PyTorch binding of libcattn.so: argument checks, output allocation and the call,
// as a CPython extension.
//
// The C ABI sees pointers and sizes only, so every tensor's shape, dtype and layout is checked
// here first (TypeError / ValueError), then that all live on one CUDA device (ValueError); then the
// call runs with that device current, on its current stream unless one is given, and with tensors of
// its own from that stream's memory.  A nonzero status raises CConvError.  Nothing is computed here.  It is compiled because the smallest calls
// take 2 to 8 us on the device: the same checks in Python with ctypes cost 15 to 20 us a call.
//
// The functions take their arguments by position; attn.py holds the signatures that users see.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../../../include/cattn.h"

namespace {

PyObject* g_error = nullptr;  // CConvError

struct Raised {};  // a Python exception is set

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Raised{};
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

struct Arg {
  const char* name;
  const at::Tensor* t;  // NULL: None
  bool given() const { return t != nullptr; }
  const void* ptr() const { return t ? t->data_ptr() : nullptr; }
  void* out() const { return t ? t->data_ptr() : nullptr; }
};

Arg tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
  return Arg{name, &THPVariable_Unpack(o)};
}
const Arg none{"", nullptr};
Arg optional(PyObject* o, const char* name) {
  return o == Py_None ? Arg{name, nullptr} : tensor(o, name);
}

void check_type(const Arg& a, at::ScalarType type) {
  if (a.t->scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", a.name, c10::toString(type), c10::toString(a.t->scalar_type()));
}

// bf16 [rows, heads, channels], channel stride 1.
void check_rows(const Arg& a) {
  check_type(a, at::kBFloat16);
  if (a.t->dim() != 3)
    raise(PyExc_ValueError, "%s must have 3 dimensions, got shape %s", a.name, shape_of(a.t->sizes()).c_str());
  if (a.t->size(2) > 1 && a.t->stride(2) != 1)
    raise(PyExc_ValueError, "%s must have channel stride 1, got strides %s", a.name, shape_of(a.t->strides()).c_str());
}

// A tensor that is addressed densely.
void check_exact(const Arg& a, at::IntArrayRef shape, at::ScalarType type) {
  check_type(a, type);
  if (a.t->sizes() != shape)
    raise(PyExc_ValueError, "%s must have shape %s, got %s", a.name, shape_of(shape).c_str(),
          shape_of(a.t->sizes()).c_str());
  if (!a.t->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", a.name);
}

void check_same_shape(const Arg& a, const Arg& b) {
  if (a.t->sizes() != b.t->sizes())
    raise(PyExc_ValueError, "%s must have %s's shape %s, got %s", a.name, b.name, shape_of(b.t->sizes()).c_str(),
          shape_of(a.t->sizes()).c_str());
}

void check_status(const Arg& a) {
  if (a.t->scalar_type() != at::kInt || a.t->numel() < 2 || !a.t->is_contiguous())
    raise(PyExc_ValueError, "%s must be a contiguous int32 tensor of at least 2 elements", a.name);
}

void extent(const at::Tensor& t, uintptr_t* a, uintptr_t* b) {
  *a = *b = 0;
  if (t.numel() == 0) return;
  int64_t span = 1;
  for (int64_t i = 0; i < t.dim(); ++i) span += (t.size(i) - 1) * t.stride(i);
  *a = reinterpret_cast<uintptr_t>(t.data_ptr());
  *b = *a + static_cast<uintptr_t>(span) * t.element_size();
}

// What a call writes may overlap nothing that it reads, nor what else it writes.
void check_disjoint(std::initializer_list<const Arg*> outs, std::initializer_list<const Arg*> ins) {
  uintptr_t a0, a1, b0, b1;
  for (const Arg* const* out = outs.begin(); out != outs.end(); ++out) {
    if (!(*out)->given()) continue;
    extent(*(*out)->t, &a0, &a1);
    auto against = [&](const Arg* x) {
      if (!x->given()) return;
      extent(*x->t, &b0, &b1);
      if (a0 < b1 && b0 < a1) raise(PyExc_ValueError, "%s overlaps %s", (*out)->name, x->name);
    };
    for (const Arg* in : ins) against(in);
    for (const Arg* const* other = outs.begin(); other != out; ++other) against(*other);
  }
}

// Every given tensor on the first one's CUDA device; returns its index.
c10::DeviceIndex check_device(std::initializer_list<const Arg*> all) {
  int index = -1;
  for (const Arg* a : all) {
    if (!a->given()) continue;
    if (!a->t->is_cuda())
      raise(PyExc_ValueError, "%s must be a CUDA tensor, got device %s", a->name, a->t->device().str().c_str());
    const int d = a->t->device().index();
    if (index < 0) index = d;
    if (d != index)
      raise(PyExc_ValueError, "%s is on cuda:%d, but the call's tensors are on cuda:%d", a->name, d, index);
  }
  return static_cast<c10::DeviceIndex>(index);
}

// A torch stream, or a raw handle.
cudaStream_t stream_of(PyObject* o, c10::DeviceIndex dev) {
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (raw) {
    PyObject* index = PyObject_GetAttrString(o, "device_index");
    if (index) {
      const long d = PyLong_AsLong(index);
      Py_DECREF(index);
      if (d != dev && !PyErr_Occurred()) {
        Py_DECREF(raw);
        raise(PyExc_ValueError, "stream belongs to cuda:%ld, but the call's tensors are on cuda:%d", d, int(dev));
      }
    }
    PyErr_Clear();
  } else {
    PyErr_Clear();
    raw = PyNumber_Long(o);
    if (!raw) throw Raised{};
  }
  const unsigned long long v = PyLong_AsUnsignedLongLong(raw);
  Py_DECREF(raw);
  if (PyErr_Occurred()) throw Raised{};
  return reinterpret_cast<cudaStream_t>(v);
}

// The device and stream of a call, current while it runs: its own device's current stream where None
// is given.  What the call allocates comes from that stream's memory, so that a workspace, which is
// freed when the call returns, goes to nothing that does not wait for the kernels.  (From another
// stream's memory it could be handed out, and written, while they still use it.)
class Place {
 public:
  Place(PyObject* stream, c10::DeviceIndex dev)
      : dev_(dev), caller_(c10::cuda::getCurrentCUDAStream(dev)), stream_(caller_), device_(dev) {
    if (stream == Py_None) return;
    cudaStream_t raw = stream_of(stream, dev);
    if (raw == cudaStreamLegacy) raw = nullptr;  // the same stream; the allocator knows it by this
    stream_ = c10::cuda::getStreamFromExternal(raw, dev);
    aside_.reset_stream(stream_);
  }
  cconv_stream_t handle() const { return reinterpret_cast<cconv_stream_t>(stream_.stream()); }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(at::kCUDA, dev_)));
  }
  // The argument, or a new tensor in its place, for the caller to use and free on its own stream.
  void out_or_new(const Arg& a, at::Tensor& own, at::IntArrayRef shape, at::ScalarType type) const {
    if (a.given()) {
      own = *a.t;
      return;
    }
    own = make(shape, type);
    if (stream_.stream() != caller_.stream()) own.record_stream(caller_.unwrap());
  }

 private:
  c10::DeviceIndex dev_;
  c10::cuda::CUDAStream caller_, stream_;
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard aside_;
};

void check_rc(int rc, const char* call) {
  if (rc == CCONV_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", rc, call);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = t && t->defined() ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

#define ARGS(n)                                                             \
  if (count != (n)) raise(PyExc_TypeError, "%zd arguments, got %zd", Py_ssize_t(n), count)

// ---------------------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------------------
struct Norm {
  Arg q, k, wq, wk, cos, sin, pos;
  int64_t total, Hq, Hk, K, P = 0, R = 0;
  cconv_dtype wdt = CCONV_F32;
  cattn_norm mode;
  float eps;
  bool inter;
};

// q, k, wq, wk, cos, sin, positions, mode, eps, interleaved
Norm norm_args(PyObject* const* a) {
  Norm n{tensor(a[0], "q"), tensor(a[1], "k"), optional(a[2], "wq"), optional(a[3], "wk"),
         optional(a[4], "cos"), optional(a[5], "sin"), optional(a[6], "positions"), 0, 0, 0, 0};
  check_rows(n.q);
  check_rows(n.k);
  n.total = n.q.t->size(0), n.Hq = n.q.t->size(1), n.K = n.q.t->size(2), n.Hk = n.k.t->size(1);
  if (n.k.t->size(0) != n.total || n.k.t->size(2) != n.K)
    raise(PyExc_ValueError, "k must have q's rows and channels, got shape %s", shape_of(n.k.t->sizes()).c_str());
  for (const Arg* w : {&n.wq, &n.wk}) {
    if (!w->given()) continue;
    const auto type = w->t->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16)
      raise(PyExc_TypeError, "%s must be a float32 or bfloat16 tensor", w->name);
    check_exact(*w, {n.K}, type);
    n.wdt = type == at::kFloat ? CCONV_F32 : CCONV_BF16;
  }
  if (n.wq.given() && n.wk.given() && n.wq.t->scalar_type() != n.wk.t->scalar_type())
    raise(PyExc_TypeError, "wq and wk must have the same dtype");
  const char* mode = PyUnicode_Check(a[7]) ? PyUnicode_AsUTF8(a[7]) : "";
  if (!mode) throw Raised{};
  if (std::string(mode) == "rms")
    n.mode = CATTN_NORM_RMS;
  else if (std::string(mode) == "l2")
    n.mode = CATTN_NORM_L2;
  else
    raise(PyExc_ValueError, "mode must be 'rms' or 'l2', got %R", a[7]);
  n.eps = as_float(a[8]);
  n.inter = as_bool(a[9]);
  if (n.cos.given() != n.sin.given()) raise(PyExc_ValueError, "cos and sin come together");
  if (n.cos.given()) {
    if (n.cos.t->dim() != 2) raise(PyExc_ValueError, "cos must be a [P, R/2] tensor");
    n.P = n.cos.t->size(0), n.R = 2 * n.cos.t->size(1);
    check_exact(n.cos, {n.P, n.R / 2}, at::kFloat);
    check_exact(n.sin, {n.P, n.R / 2}, at::kFloat);
    if (n.pos.given())
      check_exact(n.pos, {n.total}, at::kInt);
    else if (n.P < n.total)
      raise(PyExc_ValueError, "without positions token t uses table row t: %lld rows for %lld tokens",
            (long long)n.P, (long long)n.total);
  } else if (n.pos.given()) {
    raise(PyExc_ValueError, "positions need the tables cos and sin");
  }
  return n;
}

// .., yq, yk, stream
PyObject* qknorm_fwd(PyObject* const* a, Py_ssize_t count) {
  ARGS(13);
  const Norm n = norm_args(a);
  const Arg yq = optional(a[10], "yq"), yk = optional(a[11], "yk");
  if (yq.given()) check_exact(yq, {n.total, n.Hq, n.K}, at::kBFloat16);
  if (yk.given()) check_exact(yk, {n.total, n.Hk, n.K}, at::kBFloat16);
  check_disjoint({&yq, &yk}, {&n.q, &n.k, &n.wq, &n.wk, &n.cos, &n.sin, &n.pos});
  const auto dev = check_device({&n.q, &n.k, &n.wq, &n.wk, &n.cos, &n.sin, &n.pos, &yq, &yk});
  const Place place(a[12], dev);
  at::Tensor oq, ok;
  place.out_or_new(yq, oq, {n.total, n.Hq, n.K}, at::kBFloat16);
  place.out_or_new(yk, ok, {n.total, n.Hk, n.K}, at::kBFloat16);
  const at::Tensor &q = *n.q.t, &k = *n.k.t;
  check_rc(cattn_qknorm_fwd(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1),
                            n.total, n.Hq, n.Hk, n.K, n.wq.ptr(), n.wk.ptr(), n.wdt, n.mode, n.eps,
                            static_cast<const float*>(n.cos.ptr()), static_cast<const float*>(n.sin.ptr()),
                            n.P, n.R, n.inter, static_cast<const int32_t*>(n.pos.ptr()), oq.data_ptr(),
                            ok.data_ptr(), place.handle()),
           "cattn_qknorm_fwd");
  return tuple({&oq, &ok});
}

// .., dyq, dyk, dq, dk, dwq, dwk, workspace, stream
PyObject* qknorm_bwd(PyObject* const* a, Py_ssize_t count) {
  ARGS(18);
  const Norm n = norm_args(a);
  const Arg dyq = tensor(a[10], "dyq"), dyk = tensor(a[11], "dyk"), dq = optional(a[12], "dq"),
            dk = optional(a[13], "dk"), dwq = optional(a[14], "dwq"), dwk = optional(a[15], "dwk"),
            ws = optional(a[16], "workspace");
  check_rows(dyq);
  check_rows(dyk);
  check_same_shape(dyq, n.q);
  check_same_shape(dyk, n.k);
  if (dq.given()) check_exact(dq, {n.total, n.Hq, n.K}, at::kBFloat16);
  if (dk.given()) check_exact(dk, {n.total, n.Hk, n.K}, at::kBFloat16);
  const Arg* sums[2][2] = {{&dwq, &n.wq}, {&dwk, &n.wk}};
  for (auto& s : sums) {
    if (!s[0]->given()) continue;
    if (!s[1]->given()) raise(PyExc_ValueError, "%s without its weight", s[0]->name);
    check_exact(*s[0], {n.K}, s[1]->t->scalar_type());
  }
  if (ws.given() && !ws.t->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  check_disjoint({&dq, &dk, &dwq, &dwk, &ws}, {&n.q, &n.k, &dyq, &dyk, &n.wq, &n.wk, &n.cos, &n.sin, &n.pos});
  const auto dev = check_device({&n.q, &n.k, &dyq, &dyk, &n.wq, &n.wk, &n.cos, &n.sin, &n.pos, &dq, &dk, &dwq,
                                 &dwk, &ws});
  const Place place(a[17], dev);
  at::Tensor oq, ok, wq, wk, work;
  place.out_or_new(dq, oq, {n.total, n.Hq, n.K}, at::kBFloat16);
  place.out_or_new(dk, ok, {n.total, n.Hk, n.K}, at::kBFloat16);
  if (n.wq.given()) place.out_or_new(dwq, wq, {n.K}, n.wq.t->scalar_type());
  if (n.wk.given()) place.out_or_new(dwk, wk, {n.K}, n.wk.t->scalar_type());
  if (ws.given()) {
    work = *ws.t;
  } else if (wq.defined() || wk.defined()) {
    size_t bytes = 0;
    check_rc(cattn_qknorm_bwd_workspace_bytes(n.total, n.Hq, n.Hk, n.K, &bytes), "cattn_qknorm_bwd_workspace_bytes");
    work = place.make({static_cast<int64_t>(bytes)}, at::kByte);
  }
  const at::Tensor &q = *n.q.t, &k = *n.k.t, &yq = *dyq.t, &yk = *dyk.t;
  check_rc(cattn_qknorm_bwd(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1),
                            yq.data_ptr(), yq.stride(0), yq.stride(1), yk.data_ptr(), yk.stride(0), yk.stride(1),
                            n.total, n.Hq, n.Hk, n.K, n.wq.ptr(), n.wk.ptr(), n.wdt, n.mode, n.eps,
                            static_cast<const float*>(n.cos.ptr()), static_cast<const float*>(n.sin.ptr()),
                            n.P, n.R, n.inter, static_cast<const int32_t*>(n.pos.ptr()), oq.data_ptr(),
                            ok.data_ptr(), wq.defined() ? wq.data_ptr() : nullptr,
                            wk.defined() ? wk.data_ptr() : nullptr, work.defined() ? work.data_ptr() : nullptr,
                            work.defined() ? work.nbytes() : 0, place.handle()),
           "cattn_qknorm_bwd");
  return tuple({&oq, &ok, &wq, &wk});
}

// ---------------------------------------------------------------------------------------
// linear attention
// ---------------------------------------------------------------------------------------
struct Linear {
  Arg q, k, v, g;
  int64_t rows, Hk, Hv, K, V;
  float scale;
};

// q, k, v, g, scale
Linear linear_args(PyObject* const* a) {
  Linear n{tensor(a[0], "q"), tensor(a[1], "k"), tensor(a[2], "v"), tensor(a[3], "g"), 0, 0, 0, 0, 0, 0.f};
  check_rows(n.q);
  check_rows(n.k);
  check_rows(n.v);
  check_same_shape(n.k, n.q);
  n.rows = n.q.t->size(0), n.Hk = n.q.t->size(1), n.K = n.q.t->size(2);
  n.Hv = n.v.t->size(1), n.V = n.v.t->size(2);
  if (n.v.t->size(0) != n.rows)
    raise(PyExc_ValueError, "v must have q's %lld rows, got %lld", (long long)n.rows, (long long)n.v.t->size(0));
  if (n.Hk < 1 || n.Hv < 1 || n.Hv % n.Hk)
    raise(PyExc_ValueError, "the value heads (%lld) must be a multiple of the key heads (%lld)", (long long)n.Hv,
          (long long)n.Hk);
  check_type(n.g, at::kFloat);
  if (n.g.t->dim() != 2 || n.g.t->size(0) != n.rows || n.g.t->size(1) != n.Hv)
    raise(PyExc_ValueError, "g must have shape (%lld, %lld), got %s", (long long)n.rows, (long long)n.Hv,
          shape_of(n.g.t->sizes()).c_str());
  n.scale = a[4] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(n.K))) : as_float(a[4]);
  return n;
}

int64_t check_states(const Arg& a, const Linear& n) {
  if (a.t->dim() != 4)
    raise(PyExc_ValueError, "%s must be a [S, %lld, %lld, %lld] tensor", a.name, (long long)n.Hv, (long long)n.K,
          (long long)n.V);
  check_exact(a, {a.t->size(0), n.Hv, n.K, n.V}, at::kFloat);
  return a.t->size(0);
}

int64_t check_cu(const Arg& a) {
  if (a.t->scalar_type() != at::kInt || a.t->dim() != 1)
    raise(PyExc_TypeError, "%s must be a 1-D int32 tensor", a.name);
  if (a.t->numel() < 2) raise(PyExc_ValueError, "%s must hold at least 2 entries (one sequence)", a.name);
  if (!a.t->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", a.name);
  return a.t->numel() - 1;
}

#define QKVG(n)                                                                                              \
  (n).q.t->data_ptr(), (n).q.t->stride(0), (n).q.t->stride(1), (n).k.t->data_ptr(), (n).k.t->stride(0),     \
      (n).k.t->stride(1), (n).v.t->data_ptr(), (n).v.t->stride(0), (n).v.t->stride(1),                      \
      static_cast<const float*>((n).g.t->data_ptr()), (n).g.t->stride(0), (n).g.t->stride(1)

at::Tensor workspace_of(const Arg& ws, int (*query)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, size_t*),
                        const char* call, const Linear& n, int64_t nseq, const Place& place) {
  if (ws.given()) return *ws.t;
  size_t bytes = 0;
  check_rc(query(n.rows, nseq, n.Hk, n.Hv, n.K, n.V, &bytes), call);
  return place.make({static_cast<int64_t>(bytes < 16 ? 16 : bytes)}, at::kByte);
}

// q, k, v, g, scale, cu_seqlens, initial_state, final_state (a tensor, True or None), state_indices,
// status, o, workspace, stream
PyObject* linear_fwd(PyObject* const* a, Py_ssize_t count) {
  ARGS(13);
  const Linear n = linear_args(a);
  const Arg cu = tensor(a[5], "cu_seqlens"), init = optional(a[6], "initial_state"),
            fin = a[7] == Py_True || a[7] == Py_False ? Arg{"final_state", nullptr} : optional(a[7], "final_state"),
            idx = optional(a[8], "state_indices"), status = idx.given() ? optional(a[9], "status") : Arg{"status", nullptr},
            o = optional(a[10], "o"), ws = optional(a[11], "workspace");
  const int64_t nseq = check_cu(cu);
  const bool want = a[7] == Py_True;
  int64_t S = nseq;
  bool pools = want;
  if (init.given()) S = check_states(init, n), pools = true;
  if (fin.given()) {
    const int64_t s = check_states(fin, n);
    S = init.given() && S < s ? S : s;
    pools = true;
  }
  if (want && S > nseq) S = nseq;
  if (idx.given()) {
    check_exact(idx, {nseq}, at::kInt);
    if (status.given()) check_status(status);
    // (a new array holds a slot for each sequence: the pool's other indices have no place in it)
    if (want && init.given() && init.t->size(0) > nseq)
      raise(PyExc_ValueError,
            "final_state=True makes %lld slots, but state_indices name slots of initial_state, which has %lld: pass a "
            "tensor for final_state (the pool itself updates it in place)",
            (long long)nseq, (long long)init.t->size(0));
  } else if (pools && S < nseq) {
    raise(PyExc_ValueError, "without state_indices sequence i uses slot i: state arrays need at least nseq=%lld slots",
          (long long)nseq);
  }
  if (o.given()) check_exact(o, {n.rows, n.Hv, n.V}, at::kBFloat16);
  if (ws.given() && !ws.t->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  check_disjoint({&o, &status, &ws, &fin}, {&n.q, &n.k, &n.v, &n.g, &cu, &idx});
  // the initial state may be the final state's array, but no other part of it
  const bool in_place = fin.given() && init.given() && fin.ptr() == init.ptr();
  check_disjoint({&o, &status, &ws, in_place ? &none : &fin}, {&init});
  const auto dev = check_device({&n.q, &n.k, &n.v, &n.g, &cu, &init, &fin, &idx, &status, &o, &ws});
  const Place place(a[12], dev);
  at::Tensor out, final_state, st;
  place.out_or_new(o, out, {n.rows, n.Hv, n.V}, at::kBFloat16);
  if (want || fin.given()) place.out_or_new(fin, final_state, {nseq, n.Hv, n.K, n.V}, at::kFloat);
  if (idx.given()) place.out_or_new(status, st, {2}, at::kInt);
  const at::Tensor work = workspace_of(ws, cattn_linear_fwd_workspace_bytes, "cattn_linear_fwd_workspace_bytes", n, nseq, place);
  check_rc(cattn_linear_fwd(QKVG(n), n.rows, n.Hk, n.Hv, n.K, n.V, static_cast<const int32_t*>(cu.ptr()), nseq,
                            n.scale, static_cast<const float*>(init.ptr()),
                            final_state.defined() ? static_cast<float*>(final_state.data_ptr()) : nullptr,
                            static_cast<const int32_t*>(idx.ptr()), S,
                            st.defined() ? static_cast<int32_t*>(st.data_ptr()) : nullptr, out.data_ptr(),
                            work.data_ptr(), work.nbytes(), place.handle()),
           "cattn_linear_fwd");
  return tuple({&out, &final_state, &st});
}

// q, k, v, g, scale, do, cu_seqlens, initial_state, state_indices, status, want_dinit (or None), dq, dk, dv,
// dg, d_initial_state, workspace, stream
PyObject* linear_bwd(PyObject* const* a, Py_ssize_t count) {
  ARGS(18);
  const Linear n = linear_args(a);
  const Arg dout = tensor(a[5], "do"), cu = tensor(a[6], "cu_seqlens"), init = optional(a[7], "initial_state"),
            idx = optional(a[8], "state_indices"), status = idx.given() ? optional(a[9], "status") : Arg{"status", nullptr},
            dq = optional(a[11], "dq"), dk = optional(a[12], "dk"), dv = optional(a[13], "dv"), dg = optional(a[14], "dg"),
            ws = optional(a[16], "workspace");
  Arg ds = optional(a[15], "d_initial_state");
  const int64_t nseq = check_cu(cu);
  check_rows(dout);
  check_same_shape(dout, n.v);
  int64_t S = nseq;
  if (init.given()) S = check_states(init, n);
  if (idx.given()) {
    check_exact(idx, {nseq}, at::kInt);
    if (!status.given())
      raise(PyExc_ValueError, "status (int32[2] on the device) is required with state_indices");
    check_status(status);
  } else if (S < nseq) {
    raise(PyExc_ValueError,
          "without state_indices sequence i uses slot i: initial_state needs at least nseq=%lld slots",
          (long long)nseq);
  }
  const bool want = a[10] == Py_None ? init.given() || ds.given() : as_bool(a[10]);
  if (!want) ds.t = nullptr;
  if (dq.given()) check_exact(dq, n.q.t->sizes(), at::kBFloat16);
  if (dk.given()) check_exact(dk, n.q.t->sizes(), at::kBFloat16);
  if (dv.given()) check_exact(dv, n.v.t->sizes(), at::kBFloat16);
  if (dg.given()) check_exact(dg, {n.rows, n.Hv}, at::kFloat);
  if (ds.given()) check_exact(ds, {nseq, n.Hv, n.K, n.V}, at::kFloat);
  if (ws.given() && !ws.t->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  check_disjoint({&dq, &dk, &dv, &dg, &ds, &status, &ws}, {&n.q, &n.k, &n.v, &n.g, &dout, &cu, &init, &idx});
  const auto dev = check_device({&n.q, &n.k, &n.v, &n.g, &dout, &cu, &init, &idx, &status, &dq, &dk, &dv, &dg, &ds, &ws});
  const Place place(a[17], dev);
  at::Tensor oq, ok, ov, og, os;
  place.out_or_new(dq, oq, n.q.t->sizes(), at::kBFloat16);
  place.out_or_new(dk, ok, n.q.t->sizes(), at::kBFloat16);
  place.out_or_new(dv, ov, n.v.t->sizes(), at::kBFloat16);
  place.out_or_new(dg, og, {n.rows, n.Hv}, at::kFloat);
  if (want) place.out_or_new(ds, os, {nseq, n.Hv, n.K, n.V}, at::kFloat);
  const at::Tensor work = workspace_of(ws, cattn_linear_bwd_workspace_bytes, "cattn_linear_bwd_workspace_bytes", n, nseq, place);
  const at::Tensor& d = *dout.t;
  check_rc(cattn_linear_bwd(QKVG(n), d.data_ptr(), d.stride(0), d.stride(1), n.rows, n.Hk, n.Hv, n.K, n.V,
                            static_cast<const int32_t*>(cu.ptr()), nseq, n.scale, static_cast<const float*>(init.ptr()),
                            static_cast<const int32_t*>(idx.ptr()), S, static_cast<int32_t*>(status.out()),
                            oq.data_ptr(), ok.data_ptr(), ov.data_ptr(), static_cast<float*>(og.data_ptr()),
                            os.defined() ? static_cast<float*>(os.data_ptr()) : nullptr, work.data_ptr(),
                            work.nbytes(), place.handle()),
           "cattn_linear_bwd");
  return tuple({&oq, &ok, &ov, &og, &os});
}

// q, k, v, g, scale, state, state_indices, pad_rows, o, status, stream
PyObject* linear_update(PyObject* const* a, Py_ssize_t count) {
  ARGS(11);
  const Linear n = linear_args(a);
  const Arg state = tensor(a[5], "state"), idx = optional(a[6], "state_indices"), o = optional(a[8], "o"),
            status = optional(a[9], "status");
  const int64_t S = check_states(state, n);
  if (idx.given())
    check_exact(idx, {n.rows}, at::kInt);
  else if (S < n.rows)
    raise(PyExc_ValueError, "without state_indices row i uses slot i: state needs S >= N=%lld", (long long)n.rows);
  if (o.given()) check_exact(o, n.v.t->sizes(), at::kBFloat16);
  if (status.given()) check_status(status);
  check_disjoint({&o, &state, &status}, {&n.q, &n.k, &n.v, &n.g, &idx});
  const auto dev = check_device({&n.q, &n.k, &n.v, &n.g, &state, &idx, &o, &status});
  const Place place(a[10], dev);
  at::Tensor out, st;
  place.out_or_new(o, out, n.v.t->sizes(), at::kBFloat16);
  place.out_or_new(status, st, {2}, at::kInt);
  check_rc(cattn_linear_update(QKVG(n), n.rows, n.Hk, n.Hv, n.K, n.V, n.scale, static_cast<float*>(state.out()), S,
                               static_cast<const int32_t*>(idx.ptr()), as_bool(a[7]), out.data_ptr(),
                               static_cast<int32_t*>(st.data_ptr()), place.handle()),
           "cattn_linear_update");
  return tuple({&out, &st});
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  try {
    return F(args, count);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(qknorm_fwd), METHOD(qknorm_bwd), METHOD(linear_fwd), METHOD(linear_bwd),
                         METHOD(linear_update), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cattn", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__cattn() { return PyModule_Create(&module); }
