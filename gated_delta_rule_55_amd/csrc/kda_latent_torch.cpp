// kda_latent_torch.cpp -- the Python module _fast_latent: the common calls of latent.py
// without Python between the tensors and the C ABI, as kda_torch.cpp has them for
// layer.py (one after the other: 64 tokens' rotation 4.4 us and 9.3 through Python, their
// append 3.9 and 11.3).
//
// Every function takes all its arguments by position and returns what the entry point
// returns, or None for any call it does not take: latent.py then makes the call itself,
// with its own checks and errors.  None means that nothing was enqueued; a launch that
// fails raises KdaError.  Nothing is kept between calls.
#include "kda_torch.h"

#include "kda_latent.h"

namespace {

// A tensor [rows, heads, d] whose heads are dense, or [rows, d] (heads 1): the strides
// between rows and between heads.
struct View {
  void* p = nullptr;
  int64_t rows = 0, heads = 1, d = 0, row = 0, head = 0;

  bool read(Args& a, PyObject* o, int dims) {
    const at::Tensor* t = a.strided(o);
    if (!t || t->dim() != dims || t->scalar_type() != a.dt || t->device().index() != a.dev) return a.ok = false;
    rows = t->size(0), d = t->size(dims - 1);
    if (dims == 3) heads = t->size(1);
    if (rows > INT32_MAX || heads < 1 || heads > 65535 || d < 1 || d > 4096) return a.ok = false;
    head = heads > 1 ? t->stride(1) : d;
    row = rows > 1 ? t->stride(0) : heads * head;
    p = t->data_ptr();
    return a.ok = (t->stride(dims - 1) == 1 && head >= d && row >= (heads - 1) * head + d);
  }
  bool dense_heads() const { return heads == 1 || head == d; }
  bool is(int64_t r, int64_t h, int64_t w) const { return rows == r && heads == h && d == w; }
};

// Type and device of the call, from a tensor that need not be dense.
bool first(Args& a, PyObject* o) {
  const at::Tensor* t = a.strided(o);
  if (!t) return false;
  a.dev = t->device().index();
  a.dt = t->scalar_type();
  return a.ok = (a.dt == at::kFloat || a.dt == at::kBFloat16) && a.dev == c10::hip::current_device();
}

// The cache and the tables, into any of the two descriptors that have them.
template <typename Desc>
bool pages(Args& a, Desc& d, int64_t& W, PyObject* cache, PyObject* table, PyObject* lens, PyObject* cu, int64_t T) {
  const at::Tensor* c = a.strided(cache);
  const at::Tensor* t = a.tensor(table);
  if (!c || !t || c->dim() != 3 || t->dim() != 2 || c->scalar_type() != a.dt || c->device().index() != a.dev)
    return a.ok = false;
  const int64_t P = c->size(0), page = c->size(1), N = t->size(0), MP = t->size(1);
  W = c->size(2);
  if (P > INT32_MAX || page < 1 || page > INT32_MAX || N > INT32_MAX || MP > INT32_MAX || W > 4096 || T > INT32_MAX ||
      c->stride(2) != 1)
    return a.ok = false;
  d.row_stride = page > 1 ? c->stride(1) : W;
  d.page_stride = P > 1 ? c->stride(0) : 0;
  if (d.row_stride < W || (P > 1 && d.page_stride < (page - 1) * d.row_stride + W)) return a.ok = false;
  d.struct_size = sizeof(d);
  d.dtype = type_of(a.dt);
  d.n_seqs = (int32_t)N;
  d.page_size = (int32_t)page;
  d.max_pages = (int32_t)MP;
  d.n_pages = (int32_t)P;
  d.t_total = T;
  d.cache = c->data_ptr();
  d.block_table = static_cast<const int32_t*>(a.ptr(table, at::kInt, {N, MP}));
  d.seq_lens = static_cast<const int32_t*>(a.ptr(lens, at::kInt, {N}));
  d.cu_seqlens = static_cast<const int32_t*>(a.maybe(cu, at::kInt, {N + 1}));
  return a.ok = a.ok && (cu != Py_None || T == N);
}

// A call's workspace: the caller's tensor, or a new one of the bytes that need(&status) answers.
struct Workspace {
  void* p = nullptr;
  size_t bytes = 0;
  at::Tensor made;

  template <typename Need>
  bool take(Args& a, PyObject* given, Need need) {
    if (given != Py_None) {
      const at::Tensor* t = a.tensor(given);
      if (!t || t->device().index() != a.dev) return a.ok = false;
      p = t->data_ptr();
      bytes = (size_t)t->nbytes();
      return true;
    }
    int status = KDA_OK;
    bytes = need(&status);
    if (status != KDA_OK) return a.ok = false;
    if (bytes) {
      made = a.empty({(int64_t)bytes}, at::kByte);
      p = made.data_ptr();
    }
    return true;
  }
};

// (q, k, k_pe, v, cu_seqlens, cu_seqlens_k, scale, out, workspace)
PyObject* latent_prefill(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    View q, k, pe, v;
    if (n != 9 || !first(a, p[0]) || !q.read(a, p[0], 3) || !q.dense_heads() || !k.read(a, p[1], 3) ||
        !pe.read(a, p[2], 2) || !v.read(a, p[3], 3))
      Py_RETURN_NONE;
    const int64_t T = q.rows, K = k.rows, H = q.heads;
    if (!k.is(K, H, k.d) || !v.is(K, H, v.d) || !pe.is(K, 1, q.d - k.d)) Py_RETURN_NONE;
    kda_latent_prefill_desc d{};
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.n_seqs = 1;
    if (p[4] != Py_None) {
      const at::Tensor* cu = a.tensor(p[4]);
      if (!cu || cu->dim() != 1 || cu->size(0) < 1 || cu->size(0) > INT32_MAX) Py_RETURN_NONE;
      d.n_seqs = (int32_t)(cu->size(0) - 1);
      d.cu_seqlens = static_cast<const int32_t*>(a.ptr(p[4], at::kInt, {cu->size(0)}));
    }
    if (p[5] != Py_None) {
      if (p[4] == Py_None) Py_RETURN_NONE;
      d.cu_seqlens_k = static_cast<const int32_t*>(a.ptr(p[5], at::kInt, {(int64_t)d.n_seqs + 1}));
    } else if (K != T) {
      Py_RETURN_NONE;
    }
    if (p[6] != Py_None) {
      d.scale = a.number(p[6]);
      if (d.scale == 0.f) Py_RETURN_NONE;  // which stands for the default
    }
    d.n_heads = (int32_t)H;
    d.dn = (int32_t)k.d, d.dr = (int32_t)pe.d, d.dv = (int32_t)v.d;
    d.q_total = T, d.k_total = K;
    d.q = q.p, d.k = k.p, d.k_pe = pe.p, d.v = v.p;
    d.q_stride = q.row, d.k_stride = k.row, d.k_head_stride = k.head, d.k_pe_stride = pe.row;
    d.v_stride = v.row, d.v_head_stride = v.head;
    at::Tensor out;
    if (p[7] == Py_None) {
      d.o = a.output(p[7], a.dt, {T, H, v.d}, out);
    } else {
      View o;
      if (!o.read(a, p[7], 3) || !o.is(T, H, v.d) || !o.dense_heads()) Py_RETURN_NONE;
      d.o = o.p;
      d.o_stride = o.row;
    }
    if (!a.ok) Py_RETURN_NONE;
    Workspace ws;
    if (!ws.take(a, p[8], [&](int* status) { return kda_latent_prefill_workspace_bytes(&d, status); })) Py_RETURN_NONE;
    Ref result = wrap(p[7], out);
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_latent_prefill(&d, ws.p, ws.bytes, stream); }), "kda_latent_prefill", result);
  });
}

// (q, cache, block_table, seq_lens, cu_seqlens, latent_dim, scale, out, workspace)
PyObject* latent_attend(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    View q;
    kda_latent_attend_desc d{};
    int64_t W = 0;
    if (n != 9 || !first(a, p[0]) || !q.read(a, p[0], 3) || !q.dense_heads() ||
        !pages(a, d, W, p[1], p[2], p[3], p[4], q.rows) || q.d != W)
      Py_RETURN_NONE;
    const long dc = PyLong_Check(p[5]) ? PyLong_AsLong(p[5]) : -1;
    if (dc < 1 || dc >= W) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    d.n_heads = (int32_t)q.heads;
    d.dc = (int32_t)dc;
    d.dr = (int32_t)(W - dc);
    d.scale = a.number(p[6]);
    d.q = q.p;
    d.q_stride = q.row;
    at::Tensor out;
    if (p[7] == Py_None) {
      d.o = a.output(p[7], a.dt, {q.rows, q.heads, dc}, out);
    } else {
      View o;
      if (!o.read(a, p[7], 3) || !o.is(q.rows, q.heads, dc) || !o.dense_heads()) Py_RETURN_NONE;
      d.o = o.p;
      d.o_stride = o.row;
    }
    if (!a.ok) Py_RETURN_NONE;
    Workspace ws;
    if (!ws.take(a, p[8], [&](int* status) { return kda_latent_workspace_bytes(&d, status); })) Py_RETURN_NONE;
    Ref result = wrap(p[7], out);
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_latent_attend(&d, ws.p, ws.bytes, stream); }), "kda_latent_attend", result);
  });
}

// A factor that fp32 does not have as 0 (which stands for 1).
float magnitude(Args& a, PyObject* o) {
  const float m = a.number(o);
  if (m == 0.f) a.ok = false;
  return m;
}

// (cache, latent, k_pe, block_table, seq_lens, cu_seqlens, weight, eps, frequencies, interleaved,
// magnitude, rows_out)
PyObject* latent_append(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    View lat, pe;
    kda_latent_append_desc d{};
    int64_t W = 0;
    if (n != 12 || !first(a, p[1]) || !lat.read(a, p[1], 2) || !pe.read(a, p[2], 2) || pe.rows != lat.rows ||
        !pages(a, d, W, p[0], p[3], p[4], p[5], lat.rows) || lat.d + pe.d != W)
      Py_RETURN_NONE;
    d.dc = (int32_t)lat.d;
    d.dr = (int32_t)pe.d;
    d.latent = lat.p;
    d.latent_stride = lat.row;
    d.k_pe = pe.p;
    d.k_pe_stride = pe.row;
    d.weight = static_cast<const float*>(a.maybe(p[6], at::kFloat, {lat.d}));
    d.eps = a.number(p[7]);
    d.frequencies = static_cast<const double*>(a.maybe(p[8], at::kDouble, {pe.d / 2}));
    d.rotary = a.flag(p[9]) ? KDA_ROTARY_INTERLEAVED : KDA_ROTARY_HALF;
    d.magnitude = magnitude(a, p[10]);
    if (p[11] != Py_None) {
      View r;
      if (!r.read(a, p[11], 2) || !r.is(lat.rows, 1, W)) Py_RETURN_NONE;
      d.rows_out = r.p;
      d.rows_out_stride = r.row;
    }
    if (!a.ok) Py_RETURN_NONE;
    Py_INCREF(p[0]);
    Ref result(p[0]);
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_latent_append(&d, stream); }), "kda_latent_append", result);
  });
}

// (x, positions, frequencies, interleaved, magnitude, out)
PyObject* rotary(PyObject*, PyObject* const* p, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a;
    View x;
    if (n != 6 || !first(a, p[0]) || !x.read(a, p[0], 3)) Py_RETURN_NONE;
    kda_rotary_desc d{};
    d.struct_size = sizeof(d);
    d.dtype = type_of(a.dt);
    d.n_heads = (int32_t)x.heads;
    d.dim = (int32_t)x.d;
    d.t_total = x.rows;
    d.x = x.p;
    d.x_stride = x.row;
    d.x_head_stride = x.head;
    d.positions = static_cast<const int32_t*>(a.ptr(p[1], at::kInt, {x.rows}));
    d.frequencies = static_cast<const double*>(a.ptr(p[2], at::kDouble, {x.d / 2}));
    d.rotary = a.flag(p[3]) ? KDA_ROTARY_INTERLEAVED : KDA_ROTARY_HALF;
    d.magnitude = magnitude(a, p[4]);
    at::Tensor out;
    if (p[5] == Py_None) {
      d.y = a.output(p[5], a.dt, {x.rows, x.heads, x.d}, out);
    } else {
      View y;
      if (!y.read(a, p[5], 3) || !y.is(x.rows, x.heads, x.d)) Py_RETURN_NONE;
      d.y = y.p;
      d.y_stride = y.row;
      d.y_head_stride = y.head;
    }
    if (!a.ok) Py_RETURN_NONE;
    Ref result = wrap(p[5], out);
    if (!result.p) return nullptr;
    void* const stream = a.stream();
    return answer(unlocked([&] { return kda_rotary(&d, stream); }), "kda_rotary", result);
  });
}

PyMethodDef kMethods[] = {
    {"latent_prefill", (PyCFunction)(void (*)(void))latent_prefill, METH_FASTCALL, nullptr},
    {"latent_attend", (PyCFunction)(void (*)(void))latent_attend, METH_FASTCALL, nullptr},
    {"latent_append", (PyCFunction)(void (*)(void))latent_append, METH_FASTCALL, nullptr},
    {"rotary", (PyCFunction)(void (*)(void))rotary, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast_latent", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_latent(void) { return PyModule_Create(&kModule); }
