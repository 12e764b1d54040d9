// kda_torch.cpp -- the Python module _fast: the common call of each layer.py
// entry point without Python between the tensors and the C ABI.  A call of one
// token is launch and argument checks (3.3 us and 4 to 7 us through Python), and
// the checks are what this saves.
//
// Every function takes all its arguments by position and returns what the entry
// point returns, or None for any call it does not take: tensors that are not
// dense or not on the current device, subclasses, a descriptor that the library
// refuses, an allocation that fails.  layer.py then makes the call itself, with
// its own checks and errors.  None always means that nothing was enqueued: the
// results are made ready before the library is called, and a launch that fails
// raises KdaError, since a second call would update states in place twice.
// Nothing is kept between calls.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <utility>

#include "kda_linear.h"
#include "kda_norm.h"

namespace {

// Lets other Python threads run: around allocations and the library's calls,
// both of which may wait for the device.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() { PyEval_RestoreThread(state); }
};

// A dense tensor argument of one device and type; `ok` turns false at the first
// argument that is none.
struct Args {
  bool ok = true;
  c10::DeviceIndex dev = -1;
  at::ScalarType dt = at::kFloat;

  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    // a plain tensor in memory: no lazy, functional or other wrapper
    ok = t.is_cuda() && t.layout() == at::kStrided && t.has_storage() && t.is_contiguous();
    return ok ? &t : nullptr;
  }
  // The tensor that sets device and type of the call.
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    dev = t->device().index();
    dt = t->scalar_type();
    ok = (dt == at::kFloat || dt == at::kBFloat16) && dev == c10::hip::current_device();
    return ok ? t : nullptr;
  }
  void* ptr(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    ok = t->scalar_type() == type && t->device().index() == dev && t->sizes() == shape;
    return ok ? t->data_ptr() : nullptr;
  }
  void* maybe(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : ptr(o, type, shape);
  }
  float number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)x;
  }
  // A scale: 0, the default's value, where there is none and for 0 alone.
  float scale(PyObject* o) {
    if (o == Py_None) return 0.f;
    const float x = number(o);
    if (x == 0.f && flag(o)) ok = false;
    return x;
  }
  bool flag(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
      PyErr_Clear();
      ok = false;
    }
    return x > 0;
  }
  int gate(PyObject* o) {
    if (o == Py_None) return KDA_NORM_GATE_LINEAR;
    if (PyUnicode_Check(o)) {
      if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return KDA_NORM_GATE_SIGMOID;
      if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return KDA_NORM_GATE_SILU;
      if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return KDA_NORM_GATE_LINEAR;
    }
    ok = false;
    return 0;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const NoGil no_gil;
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
  }
  // `o`'s tensor, or a new one where it is None; `made` then holds it.
  void* output(PyObject* o, at::ScalarType type, at::IntArrayRef shape, at::Tensor& made) {
    if (o != Py_None) return ptr(o, type, shape);
    if (!ok) return nullptr;
    made = empty(shape, type);
    return made.data_ptr();
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(dev).stream(); }
};

int type_of(at::ScalarType t) { return t == at::kBFloat16 ? KDA_DTYPE_BF16 : KDA_DTYPE_F32; }

// An owned reference, or none.
struct Ref {
  PyObject* p = nullptr;
  Ref() = default;
  explicit Ref(PyObject* owned) : p(owned) {}
  Ref(Ref&& o) noexcept : p(o.release()) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() { return std::exchange(p, nullptr); }
};

Ref wrap(PyObject* given, at::Tensor& made) {
  if (made.defined()) return Ref(THPVariable_Wrap(std::move(made)));
  Py_INCREF(given);
  return Ref(given);
}

Ref pair(const Ref& a, const Ref& b) { return Ref(a.p && b.p ? PyTuple_Pack(2, a.p, b.p) : nullptr); }

// `result` when the library took the call, None when its checks refused it, and
// KdaError when a launch failed, after which part of the call may run.
PyObject* answer(int status, const char* what, Ref& result) {
  if (status == KDA_OK) return result.release();
  if (status != KDA_ERR_HIP) Py_RETURN_NONE;
  const Ref module(PyImport_ImportModule("gated_delta_rule_55_amd._abi"));
  const Ref type(module.p ? PyObject_GetAttrString(module.p, "KdaError") : nullptr);
  const Ref error(type.p ? PyObject_CallFunction(type.p, "is", status, what) : nullptr);
  if (error.p) PyErr_SetObject(type.p, error.p);
  return nullptr;
}

template <typename F>
int unlocked(F call) {
  const NoGil no_gil;
  return call();
}

// Runs f, with None for everything it throws, which is before its call of the
// library.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// What prefill and decode share: q [R, Hk, dk], k, v [R, H, dv], g [R, H] or [H].
struct Rows {
  int64_t R = 0, Hk = 0, dk = 0, H = 0, dv = 0;
  void *q = nullptr, *k = nullptr, *v = nullptr, *g = nullptr;
  int decay = KDA_DECAY_TOKEN;

  bool read(Args& a, PyObject* qo, PyObject* ko, PyObject* vo, PyObject* go) {
    const at::Tensor* qt = a.first(qo);
    const at::Tensor* vt = a.tensor(vo);
    if (!qt || !vt || qt->dim() != 3 || vt->dim() != 3) return a.ok = false;
    R = qt->size(0), Hk = qt->size(1), dk = qt->size(2), H = vt->size(1), dv = vt->size(2);
    if (Hk < 1 || H > 65535 || dk > 1024 || dv > 1024 || R > INT32_MAX) return a.ok = false;
    q = qt->data_ptr();
    k = a.ptr(ko, a.dt, {R, Hk, dk});
    v = a.ptr(vo, a.dt, {R, H, dv});
    const at::Tensor* gt = a.tensor(go);
    if (!gt) return false;
    if (gt->dim() == 1) {
      decay = KDA_DECAY_HEAD;
      g = a.ptr(go, at::kFloat, {H});
    } else {
      g = a.ptr(go, at::kFloat, {R, H});
    }
    return a.ok;
  }
};

// (state, q, k, v, g, scale, out, state_indices)
PyObject* linear_decode(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    Rows r;
    if (n != 8 || !r.read(a, p[1], p[2], p[3], p[4])) Py_RETURN_NONE;
    kda_linear_decode_desc d{};
    const at::Tensor* st = a.tensor(p[0]);
    if (!st || st->dim() != 4 || (st->scalar_type() != at::kFloat && st->scalar_type() != at::kBFloat16))
      Py_RETURN_NONE;
    const int64_t S = p[7] == Py_None ? r.R : st->size(0);
    if (S > INT32_MAX) Py_RETURN_NONE;
    d.state = a.ptr(p[0], st->scalar_type(), {S, r.H, r.dk, r.dv});
    d.state_indices = static_cast<const int32_t*>(a.maybe(p[7], at::kInt, {r.R}));
    d.scale = a.scale(p[5]);
    at::Tensor made;
    d.o = a.output(p[6], a.dt, {r.R, r.H, r.dv}, made);
    if (!a.ok) Py_RETURN_NONE;
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.n_seqs = (int32_t)r.R;
    d.n_heads = (int32_t)r.H;
    d.n_k_heads = (int32_t)r.Hk;
    d.dk = (int32_t)r.dk;
    d.dv = (int32_t)r.dv;
    d.decay = r.decay;
    d.state_dtype = type_of(st->scalar_type());
    d.q = r.q;
    d.k = r.k;
    d.v = r.v;
    d.g = static_cast<const float*>(r.g);
    d.n_slots = d.state_indices ? (int32_t)S : 0;
    Ref result = wrap(p[6], made);
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_linear_decode(&d, stream); }), "kda_linear_decode", result);
  });
}

// (q, k, v, g, h0, cu_seqlens, scale, out, ht, workspace, output_final_state, state_indices,
// new states in bf16)
PyObject* linear_prefill(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    Rows r;
    if (n != 13 || !r.read(a, p[0], p[1], p[2], p[3])) Py_RETURN_NONE;
    kda_linear_prefill_desc d{};
    int64_t N = 1;
    if (p[5] != Py_None) {
      const at::Tensor* cu = a.tensor(p[5]);
      if (!cu || cu->dim() != 1 || cu->size(0) < 2) Py_RETURN_NONE;
      N = cu->size(0) - 1;
      d.cu_seqlens = static_cast<const int32_t*>(a.ptr(p[5], at::kInt, {N + 1}));
    }
    const bool keep = a.flag(p[10]);
    PyObject* pool = p[4] != Py_None ? p[4] : p[8];
    at::ScalarType sd = a.flag(p[12]) ? at::kBFloat16 : at::kFloat;
    int64_t S = N;
    if (pool != Py_None) {
      const at::Tensor* t = a.tensor(pool);
      if (!t || t->dim() != 4) Py_RETURN_NONE;
      sd = t->scalar_type();
      if (p[11] != Py_None) S = t->size(0);
    } else if (p[11] != Py_None) {
      Py_RETURN_NONE;
    }
    if (S > INT32_MAX || N > INT32_MAX || (sd != at::kFloat && sd != at::kBFloat16)) Py_RETURN_NONE;
    const int64_t shape[4] = {S, r.H, r.dk, r.dv};
    d.state_indices = static_cast<const int32_t*>(a.maybe(p[11], at::kInt, {N}));
    d.h0 = a.maybe(p[4], sd, shape);
    d.scale = a.scale(p[6]);
    at::Tensor out, ht;
    d.o = a.output(p[7], a.dt, {r.R, r.H, r.dv}, out);
    PyObject* hto = p[8] == Py_None && keep && p[11] != Py_None ? p[4] : p[8];
    if (hto != Py_None || keep) d.ht = a.output(hto, sd, shape, ht);
    if (!a.ok) Py_RETURN_NONE;
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.n_seqs = (int32_t)N;
    d.n_heads = (int32_t)r.H;
    d.n_k_heads = (int32_t)r.Hk;
    d.dk = (int32_t)r.dk;
    d.dv = (int32_t)r.dv;
    d.decay = r.decay;
    d.t_total = r.R;
    d.state_dtype = type_of(sd);
    d.q = r.q;
    d.k = r.k;
    d.v = r.v;
    d.g = static_cast<const float*>(r.g);
    d.n_slots = d.state_indices ? (int32_t)S : 0;
    at::Tensor made;
    void* ws = nullptr;
    size_t bytes = 0;
    if (p[9] != Py_None) {
      const at::Tensor* t = a.tensor(p[9]);
      if (!t || t->device().index() != a.dev) Py_RETURN_NONE;
      ws = t->data_ptr();
      bytes = (size_t)t->nbytes();
    } else {
      int status = KDA_OK;
      bytes = kda_linear_workspace_bytes(&d, &status);
      if (status != KDA_OK) Py_RETURN_NONE;
      if (bytes) {
        made = a.empty({(int64_t)bytes}, at::kByte);
        ws = made.data_ptr();
      }
    }
    Ref result = pair(wrap(p[7], out), wrap(hto, ht));
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_linear_prefill(&d, ws, bytes, stream); }), "kda_linear_prefill", result);
  });
}

// Rows of the norms: x [..., dim].
bool norm_rows(Args& a, PyObject* xo, const at::Tensor*& x, int64_t& dim, int64_t& rows) {
  x = a.first(xo);
  if (!x || x->dim() < 1) return a.ok = false;
  dim = x->size(-1);
  if (dim < 1 || dim > INT32_MAX) return a.ok = false;
  rows = x->numel() / dim;
  return true;
}

// (x, weight, gate, activation, gate_first, eps, out)
PyObject* gated_norm(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    const at::Tensor* x;
    int64_t dim, rows;
    if (n != 7 || !norm_rows(a, p[0], x, dim, rows)) Py_RETURN_NONE;
    kda_gated_norm_desc d{};
    d.weight = static_cast<const float*>(a.maybe(p[1], at::kFloat, {dim}));
    d.z = a.maybe(p[2], a.dt, x->sizes());
    d.gate = a.gate(p[3]);
    d.gate_first = a.flag(p[4]);
    d.eps = a.number(p[5]);
    at::Tensor made;
    d.y = a.output(p[6], a.dt, x->sizes(), made);
    if (!a.ok) Py_RETURN_NONE;
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.dim = (int32_t)dim;
    d.rows = rows;
    d.x = x->data_ptr();
    Ref result = wrap(p[6], made);
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_gated_norm(&d, stream); }), "kda_gated_norm", result);
  });
}

// (x, residual, weight_post, weight_pre, gate, activation, channel_scale, scale, eps,
// residual_out, out)
PyObject* block_norm(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    const at::Tensor* x;
    int64_t dim, rows;
    if (n != 11 || !norm_rows(a, p[0], x, dim, rows)) Py_RETURN_NONE;
    const at::Tensor* r = a.tensor(p[1]);
    if (!r || (r->scalar_type() != at::kFloat && r->scalar_type() != at::kBFloat16)) Py_RETURN_NONE;
    const at::ScalarType rt = r->scalar_type();
    kda_block_norm_desc d{};
    d.r = a.ptr(p[1], rt, x->sizes());
    d.w_post = static_cast<const float*>(a.maybe(p[2], at::kFloat, {dim}));
    d.w_pre = static_cast<const float*>(a.maybe(p[3], at::kFloat, {dim}));
    d.z = a.maybe(p[4], a.dt, x->sizes());
    d.gate = a.gate(p[5]);
    d.c = static_cast<const float*>(a.maybe(p[6], at::kFloat, {dim}));
    d.scale = a.number(p[7]);
    d.eps = a.number(p[8]);
    if (p[10] != Py_None && !d.w_pre) Py_RETURN_NONE;
    at::Tensor rout, out;
    d.r_out = a.output(p[9], rt, x->sizes(), rout);
    if (d.w_pre) d.y = a.output(p[10], a.dt, x->sizes(), out);
    if (!a.ok) Py_RETURN_NONE;
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.residual_dtype = type_of(rt);
    d.dim = (int32_t)dim;
    d.rows = rows;
    d.x = x->data_ptr();
    Ref result = pair(wrap(p[9], rout), wrap(p[10], out));
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_block_norm(&d, stream); }), "kda_block_norm", result);
  });
}

PyMethodDef kMethods[] = {
    {"linear_prefill", (PyCFunction)(void (*)(void))linear_prefill, METH_FASTCALL, nullptr},
    {"linear_decode", (PyCFunction)(void (*)(void))linear_decode, METH_FASTCALL, nullptr},
    {"gated_norm", (PyCFunction)(void (*)(void))gated_norm, METH_FASTCALL, nullptr},
    {"block_norm", (PyCFunction)(void (*)(void))block_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&kModule); }
