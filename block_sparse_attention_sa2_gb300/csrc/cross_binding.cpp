// Python binding of the cross- and cache-attention calls (include/sa2.h): checks of the tensors,
// allocation of outputs and workspaces, and the C call, in one extension module.
//
// The rest of the library is called through ctypes (sa2.py).  These calls are not, because they are
// made with a few keys or a single token too, where the GPU needs 2 to 7 microseconds: packing the
// arguments and allocating two outputs from Python took 14 to 16 microseconds a call on a Grace core
// beside the 3 to 6 of the C call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "../../include/sa2.h"

namespace {

PyObject* g_error = nullptr;  // Sa2Error(function, code)

// A ValueError; thrown to the function's wrapper.
struct Refused {
  std::string what;
};
template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{s.str()};
}
struct Failed {  // a status of the library
  const char* fn;
  int code;
};
void check(const char* fn, sa2_status st) {
  if (st != SA2_OK) throw Failed{fn, (int)st};
}

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (none(o) || !THPVariable_Check(o)) refuse(name, " must be a tensor");
  return THPVariable_Unpack(o);
}

using Sizes = c10::IntArrayRef;

int dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return SA2_BF16;
  if (t == at::kHalf) return SA2_FP16;
  refuse("unsupported dtype ", t, ": torch.bfloat16 or torch.float16");
}

const at::Tensor& dims4(const at::Tensor& x, const char* name) {
  if (x.dim() != 4) refuse(name, ": token tensors are [B, H, N, d]");
  return x;
}

int32_t narrow(int64_t n, const char* what) {
  if (n < 0 || n > INT32_MAX) refuse(what, " = ", n, " is out of range");
  return (int32_t)n;
}

// The device of a call's tensors and the stream that it is issued on, both made the current ones: what is
// allocated here comes from that stream's memory, where work of the same stream alone can have gone before.
// (From the caller's current stream's memory a workspace could be one that an earlier call, still running
// there, has given back.)
struct Place {
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard stream_guard;
  std::optional<c10::cuda::CUDAStream> named, caller;  // a stream that the caller named; the one current then
  cudaStream_t stream = nullptr;

  Place(c10::Device d, PyObject* stream_handle) : device(d) {
    if (!d.is_cuda()) refuse("the tensors must be on a CUDA device, got ", d);
    guard.set_device(d);
    if (none(stream_handle)) {
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
    } else {
      stream = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(stream_handle));
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream must be a torch.cuda.Stream");
      }
      caller = c10::cuda::getCurrentCUDAStream(d.index());
      named = c10::cuda::getStreamFromExternal(stream, d.index());
      stream_guard.reset_stream(*named);
    }
  }
  // A tensor of the call, which may have been allocated on another stream: its memory is not given out
  // again before the named stream has got this far.
  const at::Tensor& use(const at::Tensor& x) const {
    if (named) x.record_stream(*named);
    return x;
  }
  // A tensor made here: the caller's stream may be the one that reads it.
  at::Tensor made(at::Tensor x) const {
    if (caller) x.record_stream(*caller);
    return x;
  }
  at::Tensor empty(Sizes shape, at::ScalarType t) const {
    return made(at::empty(shape, at::TensorOptions().dtype(t).device(device)));
  }
  at::Tensor empty_like(const at::Tensor& x) const { return made(at::empty_like(x)); }
  at::Tensor given_or_like(PyObject* o, const char* name, const at::Tensor& x) const {
    return none(o) ? empty_like(x) : tensor(o, name);
  }
};

// sa2_tensor of a token tensor of this shape, type and device.
sa2_tensor token(const at::Tensor& x, const char* name, Sizes shape, at::ScalarType dtype, const Place& at_) {
  if (x.sizes() != shape) refuse(name, " must be ", shape, ", got ", x.sizes());
  if (x.scalar_type() != dtype) refuse(name, " must be ", dtype, ", got ", x.scalar_type());
  if (x.device() != at_.device) refuse(name, " must be on ", at_.device, ", got ", x.device());
  const Sizes st = x.strides();
  if (st[3] != 1) refuse(name, ": the last dimension must be contiguous");
  return {at_.use(x).data_ptr(), st[0], st[1], st[2]};
}

const int32_t* int32s(PyObject* o, const char* name, int64_t B, const Place& at_) {
  if (none(o)) return nullptr;
  const at::Tensor& x = tensor(o, name);
  if (x.scalar_type() != at::kInt || x.dim() != 1 || x.size(0) != B || !x.is_contiguous() || x.device() != at_.device)
    refuse(name, " must be a contiguous int32 tensor of shape [", B, "] on ", at_.device);
  return static_cast<const int32_t*>(at_.use(x).data_ptr());
}

float* float32s(const at::Tensor& x, const char* name, Sizes shape, c10::Device device) {
  if (x.scalar_type() != at::kFloat || x.sizes() != shape || !x.is_contiguous() || x.device() != device)
    refuse(name, " must be a contiguous float32 tensor of shape ", shape, " on ", device);
  return static_cast<float*>(x.data_ptr());
}
float* float32s(const at::Tensor& x, const char* name, Sizes shape, const Place& at_) {
  float* p = float32s(x, name, shape, at_.device);
  at_.use(x);
  return p;
}

struct Workspace {
  at::Tensor hold;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* ws, size_t need, const Place& at_) {
    if (none(ws)) {
      if (need == 0) return;
      hold = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at_.device));
    } else {
      hold = tensor(ws, "ws");
      if (hold.device() != at_.device || hold.scalar_type() != at::kByte || !hold.is_contiguous())
        refuse("ws must be a contiguous uint8 tensor on ", at_.device);
      at_.use(hold);
    }
    p = hold.data_ptr();
    bytes = (size_t)hold.numel();
  }
};

sa2_cross_shape cross_shape(const at::Tensor& q, int64_t Hkv, int64_t M) {
  return {narrow(q.size(0), "B"), narrow(q.size(1), "H"), narrow(Hkv, "Hkv"), narrow(q.size(2), "N"),
          narrow(M, "M"),         narrow(q.size(3), "d"), dtype_code(q.scalar_type()), 0};
}

float scale_of(PyObject* o) {
  if (none(o)) return 0.f;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("scale must be a number");
  }
  return (float)x;
}

// A KvCache8's (sa2_cache8 as bytes, k, v, k_scale, v_scale).  The struct was made from the tensors when the cache
// was; one whose memory has been exchanged since (x.data = .., x.set_, x.resize_) is refused.
struct Cache {
  const sa2_cache8* c;
  const at::Tensor* t[4];
  const sa2_cache8* operator->() const { return c; }
  explicit Cache(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5 || !PyBytes_Check(PyTuple_GET_ITEM(o, 0)) ||
        PyBytes_GET_SIZE(PyTuple_GET_ITEM(o, 0)) != (Py_ssize_t)sizeof(sa2_cache8))
      refuse("cache must be a KvCache8");
    c = reinterpret_cast<const sa2_cache8*>(PyBytes_AS_STRING(PyTuple_GET_ITEM(o, 0)));
    const void* held[4] = {c->k, c->v, c->k_scale, c->v_scale};
    for (int i = 0; i < 4; ++i) {
      t[i] = &tensor(PyTuple_GET_ITEM(o, i + 1), "cache");
      if (t[i]->data_ptr() != held[i]) refuse("the cache's tensors have moved since the KvCache8 was made");
    }
  }
  void use(const Place& at_) const {
    for (const at::Tensor* x : t) at_.use(*x);
  }
};
c10::Device cuda(PyObject* index) {
  const long i = PyLong_AsLong(index);
  if (i < 0) {
    PyErr_Clear();
    refuse("the tensors must be on a CUDA device");
  }
  return c10::Device(c10::kCUDA, (c10::DeviceIndex)i);
}

template <typename... T>
PyObject* tuple_of(const T&... x) {
  PyObject* r = PyTuple_New(sizeof...(x));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(x)), ...);  // (steals the new references)
  return r;
}

// q, k, v, kv_len, scale, o, lse, ws, stream
PyObject* cross_fwd(PyObject* const* a) {
  const at::Tensor& q = dims4(tensor(a[0], "q"), "q");
  const at::Tensor& k = dims4(tensor(a[1], "k"), "k");
  const at::Tensor& v = tensor(a[2], "v");
  const sa2_cross_shape s = cross_shape(q, k.size(1), k.size(2));
  const Place at_(q.device(), a[8]);
  const int64_t kvs[4] = {q.size(0), k.size(1), k.size(2), q.size(3)}, ls[3] = {q.size(0), q.size(1), q.size(2)};
  const at::ScalarType t = q.scalar_type();
  const sa2_tensor qt = token(q, "q", q.sizes(), t, at_), kt = token(k, "k", kvs, t, at_),
                   vt = token(v, "v", kvs, t, at_);
  const int32_t* len = int32s(a[3], "kv_len", s.B, at_);
  const at::Tensor o = at_.given_or_like(a[5], "o", q);
  const at::Tensor lse = none(a[6]) ? at_.empty(ls, at::kFloat) : tensor(a[6], "lse");
  const sa2_tensor ot = token(o, "o", q.sizes(), t, at_);
  const Workspace ws(a[7], sa2_cross_fwd_workspace_size(&s), at_);
  check("sa2_cross_attn_fwd", sa2_cross_attn_fwd(&s, &qt, &kt, &vt, len, scale_of(a[4]), &ot,
                                                 float32s(lse, "lse", ls, at_), ws.p, ws.bytes, at_.stream));
  return tuple_of(o, lse);
}

// q, k, v, o, lse, do, kv_len, scale, dq, dk, dv, ws, stream
PyObject* cross_bwd(PyObject* const* a) {
  const at::Tensor& q = dims4(tensor(a[0], "q"), "q");
  const at::Tensor& k = dims4(tensor(a[1], "k"), "k");
  const at::Tensor& v = tensor(a[2], "v");
  const sa2_cross_shape s = cross_shape(q, k.size(1), k.size(2));
  const Place at_(q.device(), a[12]);
  const int64_t kvs[4] = {q.size(0), k.size(1), k.size(2), q.size(3)}, ls[3] = {q.size(0), q.size(1), q.size(2)};
  const at::ScalarType t = q.scalar_type();
  const sa2_tensor qt = token(q, "q", q.sizes(), t, at_), kt = token(k, "k", kvs, t, at_), vt = token(v, "v", kvs, t, at_),
                   ot = token(tensor(a[3], "o"), "o", q.sizes(), t, at_),
                   dot = token(tensor(a[5], "do"), "do", q.sizes(), t, at_);
  const float* lse = float32s(tensor(a[4], "lse"), "lse", ls, at_);
  const int32_t* len = int32s(a[6], "kv_len", s.B, at_);
  const at::Tensor dq = at_.given_or_like(a[8], "dq", q), dk = at_.given_or_like(a[9], "dk", k),
                   dv = at_.given_or_like(a[10], "dv", v);
  const sa2_tensor dqt = token(dq, "dq", q.sizes(), t, at_), dkt = token(dk, "dk", kvs, t, at_),
                   dvt = token(dv, "dv", kvs, t, at_);
  const Workspace ws(a[11], sa2_cross_bwd_workspace_size(&s), at_);
  check("sa2_cross_attn_bwd", sa2_cross_attn_bwd(&s, &qt, &kt, &vt, &ot, lse, &dot, len, scale_of(a[7]), &dqt, &dkt,
                                                 &dvt, ws.p, ws.bytes, at_.stream));
  return tuple_of(dq, dk, dv);
}

// k, v, k_scale, v_scale: checks a cache's tensors; its (shape, device index or -1, sa2_cache8 as bytes).
// (From Python the checks took 4 microseconds, half of a call with one token.)
PyObject* cache_pack(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.strides() != k.strides() || k.stride(3) != 1)
    refuse("the cache's k and v are [B, Hkv, C, d] with the same strides, d contiguous");
  auto held = [](const at::Tensor& x) { return x.scalar_type() == at::kFloat8_e4m3fn || x.scalar_type() == at::kByte; };
  if (!held(k) || !held(v) || v.device() != k.device())
    refuse("the cache's k and v are float8_e4m3fn (or uint8) on one device");
  const Sizes sz = k.sizes(), st = k.strides();
  const int64_t scales[3] = {sz[0], sz[1], (sz[2] + 63) / 64};
  sa2_cache8 c{k.data_ptr(), v.data_ptr(), float32s(tensor(a[2], "k_scale"), "k_scale", scales, k.device()),
               float32s(tensor(a[3], "v_scale"), "v_scale", scales, k.device()), st[0], st[1], st[2],
               narrow(sz[0], "B"), narrow(sz[1], "Hkv"), narrow(sz[2], "C"), narrow(sz[3], "d")};
  return Py_BuildValue("((LLLL)iy#)", (long long)sz[0], (long long)sz[1], (long long)sz[2], (long long)sz[3],
                       k.device().has_index() ? (int)k.device().index() : -1, reinterpret_cast<const char*>(&c),
                       (Py_ssize_t)sizeof(c));
}

// cache, device, k, v, pos, n_new, stream
PyObject* cache_append(PyObject* const* a) {
  const Cache c(a[0]);
  const Place at_(cuda(a[1]), a[6]);
  c.use(at_);
  const at::Tensor& k = dims4(tensor(a[2], "k"), "k");
  const at::ScalarType t = k.scalar_type();
  const int code = dtype_code(t);
  const int64_t shape[4] = {c->B, c->Hkv, k.size(2), c->d};
  if (none(a[4])) refuse("pos is required");
  const sa2_tensor kt = token(k, "k", shape, t, at_), vt = token(tensor(a[3], "v"), "v", shape, t, at_);
  const int32_t *pos = int32s(a[4], "pos", c->B, at_), *n_new = int32s(a[5], "n_new", c->B, at_);
  if (shape[2] > 0)
    check("sa2_cache8_append",
          sa2_cache8_append(c.c, narrow(shape[2], "n"), code, &kt, &vt, pos, n_new, at_.stream));
  Py_RETURN_NONE;
}

// cache, device, pos, n, fp16, k, v, stream
PyObject* cache_read(PyObject* const* a) {
  const Cache c(a[0]);
  const Place at_(cuda(a[1]), a[7]);
  c.use(at_);
  const long long n = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred() || n < 0) {
    PyErr_Clear();
    refuse("n must be a count of tokens");
  }
  const int64_t shape[4] = {c->B, c->Hkv, n, c->d};
  const at::ScalarType t = PyObject_IsTrue(a[4]) ? at::kHalf : at::kBFloat16;
  if (none(a[2])) refuse("pos is required");
  const int32_t* pos = int32s(a[2], "pos", c->B, at_);
  const at::Tensor k = none(a[5]) ? at_.empty(shape, t) : tensor(a[5], "k");
  const at::Tensor v = none(a[6]) ? at_.empty(shape, t) : tensor(a[6], "v");
  const sa2_tensor kt = token(k, "k", shape, t, at_), vt = token(v, "v", shape, t, at_);
  if (n > 0)
    check("sa2_cache8_read", sa2_cache8_read(c.c, narrow(n, "n"), dtype_code(t), &kt, &vt, pos, at_.stream));
  return tuple_of(k, v);
}

// q, cache, device, kv_len, scale, o, lse, ws, stream
PyObject* cache_attn(PyObject* const* a) {
  const at::Tensor& q = dims4(tensor(a[0], "q"), "q");
  const Cache c(a[1]);
  const sa2_cross_shape s = cross_shape(q, c->Hkv, c->C);
  if (s.B != c->B || s.d != c->d)
    refuse("the cache holds B = ", c->B, ", d = ", c->d, "; q has B = ", s.B, ", d = ", s.d);
  if (none(a[3])) refuse("kv_len is required");
  const Place at_(q.device(), a[8]);
  if (cuda(a[2]) != at_.device) refuse("the cache must be on ", at_.device, ", got ", cuda(a[2]));
  c.use(at_);
  const int64_t ls[3] = {q.size(0), q.size(1), q.size(2)};
  const at::ScalarType t = q.scalar_type();
  const sa2_tensor qt = token(q, "q", q.sizes(), t, at_);
  const int32_t* len = int32s(a[3], "kv_len", s.B, at_);
  const at::Tensor o = at_.given_or_like(a[5], "o", q);
  const at::Tensor lse = none(a[6]) ? at_.empty(ls, at::kFloat) : tensor(a[6], "lse");
  const sa2_tensor ot = token(o, "o", q.sizes(), t, at_);
  const Workspace ws(a[7], sa2_cross_fwd_workspace_size(&s), at_);
  check("sa2_cache8_attn", sa2_cache8_attn(&s, &qt, c.c, len, scale_of(a[4]), &ot, float32s(lse, "lse", ls, at_),
                                           ws.p, ws.bytes, at_.stream));
  return tuple_of(o, lse);
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) return PyErr_Format(PyExc_TypeError, "%zd arguments, %zd given", N, n);
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Failed& f) {
    if (PyObject* e = PyObject_CallFunction(g_error, "si", f.fn, f.code)) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FAST(name, f, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("cross_attn_fwd", cross_fwd, 9),   FAST("cross_attn_bwd", cross_bwd, 13),
                         FAST("cache8_append", cache_append, 7), FAST("cache8_read", cache_read, 8),
                         FAST("cache8_attn", cache_attn, 9),     FAST("cache8_pack", cache_pack, 4),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cross", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cross() { return PyModule_Create(&module); }
