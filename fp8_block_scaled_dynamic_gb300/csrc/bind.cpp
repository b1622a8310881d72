// bind.cpp -- the Python binding of include/mxattn.h, as a CPython module.
//
// The small calls of a decode step run for 3-10 us on the GPU; marshalling ten
// tensors through ctypes took 17-27 us of host time a call, so these entry
// points read the tensors in C++ (3 us a call, attn_tree 7).  Like the rest of the binding
// it checks dtypes and shapes, allocates missing outputs with torch and calls
// the C entry point of the same name.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "mxattn.h"

namespace {

PyObject *g_error = nullptr;  // the package's MxgError

struct Raised {};  // a Python error is already set

[[noreturn]] void bad(const std::string &msg) { throw std::invalid_argument(msg); }
void need(bool ok, const char *msg) {
  if (!ok) bad(msg);
}
bool given(PyObject *o) { return o && o != Py_None; }

const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, int dim) {
  if (!o || !THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || t.dim() != dim)
    bad(std::string(name) + " must be a CUDA " + c10::toString(type) + " tensor of " + std::to_string(dim) +
        " dimension(s)");
  if (t.numel() > 0 && t.size(dim - 1) > 1 && t.stride(dim - 1) != 1)
    bad(std::string(name) + " must have a unit inner stride");
  if (t.get_device() != c10::cuda::current_device()) bad(std::string(name) + " is not on the current device");
  return t;
}

void *ptr(const at::Tensor &t) { return t.data_ptr(); }

mxg_heads heads(const at::Tensor &t) { return {ptr(t), t.stride(-3), t.stride(-2)}; }
const at::Tensor &heads_of(PyObject *o, const char *name) { return tensor(o, name, at::kBFloat16, 3); }

template <class T>
T *index(PyObject *o, const char *name, at::ScalarType type, int64_t n) {
  const at::Tensor &t = tensor(o, name, type, 1);
  if (n >= 0 && t.numel() != n) bad(std::string(name) + " must have " + std::to_string(n) + " entries");
  return static_cast<T *>(ptr(t));
}

int *status_word(PyObject *o) { return given(o) ? index<int>(o, "dev_status", at::kInt, -1) : nullptr; }

struct Table {
  int *p;
  int ld, cols;
};
Table table(PyObject *o, const char *name, int64_t rows) {
  const at::Tensor &t = tensor(o, name, at::kInt, 2);
  if (t.size(0) != rows) bad(std::string(name) + " must have a row for each sequence");
  const int64_t cols = t.size(1), ld = t.size(0) > 1 ? t.stride(0) : cols;
  if (ld > INT_MAX || cols > INT_MAX || ld < cols) bad(std::string(name) + " has overlapping or too long rows");
  return {static_cast<int *>(ptr(t)), (int)ld, (int)cols};
}

int as_int(int64_t n, const char *what) {
  if (n > INT_MAX) bad(std::string("too many ") + what);
  return (int)n;
}

// cache: a KVCache's k and v, (pages, page_size, Hkv, D) or with a leading
// layers dimension; one_layer: of a call that takes a single layer
mxg_kv_cache cache_of(PyObject *ko, PyObject *vo, int64_t Hkv, int64_t D, bool one_layer) {
  if (!ko || !THPVariable_Check(ko)) bad("a cache holds two tensors");
  const int dim = THPVariable_Unpack(ko).dim() == 5 ? 5 : 4;
  const at::Tensor &k = tensor(ko, "cache.k", at::kBFloat16, dim), &v = tensor(vo, "cache.v", at::kBFloat16, dim);
  need(k.sizes() == v.sizes() && k.strides() == v.strides(), "k and v of a cache differ in shape or strides");
  need(k.size(-2) == Hkv && k.size(-1) == D, "the cache does not fit k");
  need(!one_layer || dim == 4 || k.size(0) == 1, "the call takes one layer of the cache: cache.layer(i)");
  return {ptr(k),       ptr(v),
          dim == 5 ? k.stride(0) : 0,
          k.stride(-4), k.stride(-3), k.stride(-2),
          dim == 5 ? as_int(k.size(0), "layers") : 1,
          as_int(k.size(-4), "pages"),
          as_int(k.size(-3), "slots of a page")};
}

// The stream of a call, made torch's current one meanwhile, so that what is
// allocated here belongs to the stream that writes it.
struct Stream {
  std::optional<c10::cuda::CUDAStreamGuard> on;
  explicit Stream(PyObject *o) {
    if (!given(o)) return;
    PyObject *a = PyObject_GetAttrString(o, "cuda_stream");
    if (!a) throw Raised();
    void *x = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    if (!x && PyErr_Occurred()) throw Raised();
    on.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(x), c10::cuda::current_device()));
  }
  mxg_stream_t handle() const {
    return reinterpret_cast<mxg_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
  }
};

double number(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}
long integer(PyObject *o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  return x;
}

void check(const char *fn, mxg_status st) {
  if (st == MXG_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "si", fn, (int)st);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

template <class F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const Raised &) {
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want) { need(n == want, "wrong number of arguments"); }

// (q, k, pos, cos_sin, wq, wk, eps, interleaved, q_out, k_out, v, cache k, cache v, slots, dev_status, stream)
PyObject *py_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 16);
    const Stream stream(a[15]);
    const at::Tensor &q = heads_of(a[0], "q"), &k = heads_of(a[1], "k");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    need(k.size(0) == T && k.size(2) == D, "k must be (T, Hkv, D)");
    const at::Tensor qo = given(a[8]) ? heads_of(a[8], "q_out") : at::empty(q.sizes(), q.options());
    const at::Tensor ko = given(a[9]) ? heads_of(a[9], "k_out") : at::empty(k.sizes(), k.options());
    need(qo.sizes() == q.sizes() && ko.sizes() == k.sizes(), "q_out / k_out shape");
    const void *w[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i)
      if (given(a[4 + i])) w[i] = index<void>(a[4 + i], i ? "wk" : "wq", at::kBFloat16, D);
    const float *cs = nullptr;
    const int *pos = nullptr;
    int max_pos = 0, rot = 0;
    if (given(a[3])) {
      const at::Tensor &t = tensor(a[3], "cos_sin", at::kFloat, 2);
      need(t.is_contiguous(), "cos_sin must be contiguous");
      cs = static_cast<const float *>(ptr(t));
      max_pos = as_int(t.size(0), "positions");
      rot = as_int(t.size(1), "channels");
      need(given(a[2]), "a rotation needs pos");
      pos = index<int>(a[2], "pos", at::kInt, T);
    }
    const mxg_heads qh = heads(q), kh = heads(k), qoh = heads(qo), koh = heads(ko);
    mxg_heads vh;
    mxg_kv_cache c;
    const int64_t *slots = nullptr;
    const bool cached = given(a[11]);
    if (cached) {
      need(given(a[10]) && given(a[13]), "a cache needs v and slots");
      const at::Tensor &v = heads_of(a[10], "v");
      need(v.sizes() == k.sizes(), "v must have k's shape");
      vh = heads(v);
      c = cache_of(a[11], a[12], Hkv, D, true);
      slots = index<int64_t>(a[13], "slots", at::kLong, T);
    }
    check("qk_norm_rope",
          qk_norm_rope(&qh, &kh, as_int(T, "tokens"), as_int(Hq, "heads"), as_int(Hkv, "heads"), as_int(D, "channels"),
                       w[0], w[1], (float)number(a[6]), pos, cs, max_pos, rot, (int)integer(a[7]), &qoh, &koh,
                       cached ? &vh : nullptr, cached ? &c : nullptr, slots, status_word(a[14]), stream.handle()));
    PyObject *qp = THPVariable_Wrap(qo), *kp = THPVariable_Wrap(ko);
    return Py_BuildValue("NN", qp, kp);
  });
}

struct Attn {
  mxg_heads q, k, v, out;
  at::Tensor o;
  int64_t T, Hq, Hkv, D;
  float scale;
  mxg_attn_opts opts;
};

// scale and opts of both attention calls: (scale, out, dev_status, timeout_ms, debug_stall) at a[at ...]
Attn attn_of(PyObject *const *a, int at_) {
  Attn r;
  const at::Tensor &q = heads_of(a[0], "q"), &k = heads_of(a[1], "k"), &v = heads_of(a[2], "v");
  r.T = q.size(0), r.Hq = q.size(1), r.D = q.size(2), r.Hkv = k.size(1);
  need(k.size(0) == r.T && k.size(2) == r.D && v.sizes() == k.sizes(), "k and v must be (T, Hkv, D)");
  r.o = given(a[at_ + 1]) ? heads_of(a[at_ + 1], "out") : at::empty(q.sizes(), q.options());
  need(r.o.sizes() == q.sizes(), "out must have q's shape");
  r.q = heads(q), r.k = heads(k), r.v = heads(v), r.out = heads(r.o);
  r.scale = given(a[at_]) ? (float)number(a[at_]) : (float)(1.0 / std::sqrt((double)(r.D > 0 ? r.D : 1)));
  r.opts = {};
  r.opts.dev_status = status_word(a[at_ + 2]);
  const long ms = integer(a[at_ + 3]), stall = integer(a[at_ + 4]);
  need(ms >= 0 && ms <= (long)UINT32_MAX, "timeout_ms must be 0 (the default) or a number of milliseconds in 32 bits");
  need(stall == 0 || stall == 1, "debug_stall must be 0 or 1");
  r.opts.timeout_ms = (uint32_t)ms;
  r.opts.debug_stall = (int)stall;
  return r;
}

// (q, k, v, cu_seqlens, scale, out, dev_status, timeout_ms, debug_stall, stream)
PyObject *py_prompt(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 10);
    const Stream stream(a[9]);
    const Attn r = attn_of(a, 4);
    const at::Tensor &cu = tensor(a[3], "cu_seqlens", at::kInt, 1);
    check("attn_prompt", attn_prompt(&r.q, &r.k, &r.v, static_cast<int *>(ptr(cu)), as_int(cu.numel() - 1, "sequences"),
                                     as_int(r.T, "tokens"), as_int(r.Hq, "heads"), as_int(r.Hkv, "heads"),
                                     as_int(r.D, "channels"), r.scale, &r.out, &r.opts, stream.handle()));
    return THPVariable_Wrap(r.o);
  });
}

// (q, k, v, cu_nodes, mask, cache k, cache v, block_table, ctx_len, scale, out, dev_status, timeout_ms, debug_stall, ws, stream)
PyObject *py_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 16);
    const Stream stream(a[15]);
    Attn r = attn_of(a, 9);
    const at::Tensor &ctx = tensor(a[8], "ctx_len", at::kInt, 1);
    // (back with the allocator on return, for what follows in the stream)
    const at::Tensor ws = given(a[14]) ? tensor(a[14], "ws", at::kByte, 1)
                                       : at::empty({(int64_t)mxg_attn_tree_workspace_bytes((int)r.D)},
                                                   r.o.options().dtype(at::kByte));
    const int64_t B = ctx.numel();
    const int *cu = index<int>(a[3], "cu_nodes", at::kInt, B + 1);
    const uint64_t *mask = index<uint64_t>(a[4], "mask", at::kLong, r.T);
    const mxg_kv_cache c = cache_of(a[5], a[6], r.Hkv, r.D, true);
    const Table t = table(a[7], "block_table", B);
    r.opts.workspace = ptr(ws);
    r.opts.ws_bytes = (size_t)ws.numel();
    check("attn_tree",
          attn_tree(&r.q, &r.k, &r.v, cu, mask, as_int(B, "sequences"), as_int(r.T, "nodes"), &c, t.p, t.ld, t.cols,
                    static_cast<int *>(ptr(ctx)), as_int(r.Hq, "heads"), as_int(r.Hkv, "heads"),
                    as_int(r.D, "channels"), r.scale, &r.out, &r.opts, stream.handle()));
    return THPVariable_Wrap(r.o);
  });
}

// What attn_tree, attn_shared and attn_sparse take alike, at a[0 ... 8]: q, k, v, cu_nodes, mask, cache k, cache v,
// block_table, ctx_len; and at a[at ...] what attn_of takes there, then ws.
struct Paged {
  Attn r;
  const int *cu, *ctx;
  const uint64_t *mask;
  mxg_kv_cache c;
  Table t;
  int64_t B;
  at::Tensor ws;
};

template <class Bytes>
Paged paged_of(PyObject *const *a, int at_, Bytes bytes) {
  Paged p;
  p.r = attn_of(a, at_);
  const at::Tensor &ctx = tensor(a[8], "ctx_len", at::kInt, 1);
  p.B = ctx.numel();
  p.ctx = static_cast<int *>(ptr(ctx));
  p.cu = index<int>(a[3], "cu_nodes", at::kInt, p.B + 1);
  p.mask = index<uint64_t>(a[4], "mask", at::kLong, p.r.T);
  p.c = cache_of(a[5], a[6], p.r.Hkv, p.r.D, true);
  p.t = table(a[7], "block_table", p.B);
  as_int(p.r.T, "nodes"), as_int(p.r.Hq, "heads"), as_int(p.r.D, "channels");
  // (back with the allocator on return, for what follows in the stream)
  p.ws = given(a[at_ + 5]) ? tensor(a[at_ + 5], "ws", at::kByte, 1)
                           : at::empty({(int64_t)bytes(p.r)}, p.r.o.options().dtype(at::kByte));
  p.r.opts.workspace = ptr(p.ws);
  p.r.opts.ws_bytes = (size_t)p.ws.numel();
  return p;
}

// (q, k, v, cu_nodes, mask, cache k, cache v, block_table, ctx_len, cu_groups, prefix_len, scale, out, dev_status,
// timeout_ms, debug_stall, ws, stream)
PyObject *py_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 18);
    const Stream stream(a[17]);
    const Paged p = paged_of(
        a, 11, [](const Attn &r) { return mxg_attn_shared_workspace_bytes((int)r.T, (int)r.Hq, (int)r.D); });
    const at::Tensor &prefix = tensor(a[10], "prefix_len", at::kInt, 1);
    const int groups = as_int(prefix.numel(), "groups");
    const int *cg = index<int>(a[9], "cu_groups", at::kInt, (int64_t)groups + 1);
    check("attn_shared",
          attn_shared(&p.r.q, &p.r.k, &p.r.v, p.cu, p.mask, as_int(p.B, "sequences"), (int)p.r.T, &p.c, p.t.p, p.t.ld,
                      p.t.cols, p.ctx, cg, static_cast<int *>(ptr(prefix)), groups, (int)p.r.Hq, (int)p.r.Hkv,
                      (int)p.r.D, p.r.scale, &p.r.out, &p.r.opts, stream.handle()));
    return THPVariable_Wrap(p.r.o);
  });
}

// (q, k, v, cu_nodes, mask, cache k, cache v, block_table, ctx_len, sel, scale, out, dev_status, timeout_ms,
// debug_stall, ws, stream)
PyObject *py_sparse(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 17);
    const Stream stream(a[16]);
    const at::Tensor &sel = tensor(a[9], "sel", at::kInt, 3);
    const int n_sel = as_int(sel.size(2), "pages");
    const Paged p = paged_of(a, 10, [&](const Attn &r) {
      return mxg_attn_sparse_workspace_bytes((int)r.T, as_int(r.Hkv, "heads"), n_sel, (int)r.D);
    });
    need(sel.size(0) == p.r.T && sel.size(1) == p.r.Hkv && sel.is_contiguous(), "sel must be contiguous (N, Hkv, n_sel)");
    check("attn_sparse",
          attn_sparse(&p.r.q, &p.r.k, &p.r.v, p.cu, p.mask, as_int(p.B, "sequences"), (int)p.r.T, &p.c, p.t.p, p.t.ld,
                      p.t.cols, p.ctx, static_cast<int *>(ptr(sel)), n_sel, (int)p.r.Hq, (int)p.r.Hkv, (int)p.r.D,
                      p.r.scale, &p.r.out, &p.r.opts, stream.handle()));
    return THPVariable_Wrap(p.r.o);
  });
}

// a PageIndex's codes and exps, (pages, Hkv, 2, D) and (pages, Hkv), or with a leading layers dimension
mxg_page_index index_of(PyObject *co, PyObject *eo, int64_t Hkv, int64_t D, bool one_layer) {
  if (!co || !THPVariable_Check(co)) bad("an index holds two tensors");
  const int dim = THPVariable_Unpack(co).dim() == 5 ? 5 : 4;
  const at::Tensor &c = tensor(co, "index.codes", at::kChar, dim), &e = tensor(eo, "index.exps", at::kByte, dim - 2);
  need(c.size(-3) == Hkv && c.size(-2) == 2 && c.size(-1) == D, "the index does not fit the heads");
  need(c.stride(-2) == D, "the two rows of an index entry must follow one another");
  need(e.size(-1) == Hkv && e.size(-2) == c.size(-4) && (dim == 4 || e.size(0) == c.size(0)),
       "codes and exps of an index differ in shape");
  need(!one_layer || dim == 4 || c.size(0) == 1, "the call takes one layer of the index: index.layer(i)");
  return {static_cast<int8_t *>(ptr(c)),
          static_cast<uint8_t *>(ptr(e)),
          dim == 5 ? c.stride(0) : 0,
          c.stride(-4),
          c.stride(-3),
          dim == 5 ? e.stride(0) : 0,
          e.stride(-2),
          dim == 5 ? as_int(c.size(0), "layers") : 1,
          as_int(c.size(-4), "pages")};
}

// (cache k, cache v, codes, exps, page_size, block_table, ctx_old, ctx_new, dev_status, stream)
PyObject *py_index(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 10);
    const Stream stream(a[9]);
    if (!THPVariable_Check(a[0])) bad("a cache holds two tensors");
    const at::Tensor &kc = THPVariable_Unpack(a[0]);
    need(kc.dim() == 4 || kc.dim() == 5, "a cache is ([layers,] pages, page_size, Hkv, D)");
    const int64_t Hkv = kc.size(-2), D = kc.size(-1);
    const mxg_kv_cache c = cache_of(a[0], a[1], Hkv, D, false);
    const mxg_page_index x = index_of(a[2], a[3], Hkv, D, false);
    need(integer(a[4]) == c.page_size, "the index and the cache differ in page size");
    need(x.layers == c.layers, "the index and the cache differ in layers");
    const at::Tensor &now = tensor(a[7], "ctx_new", at::kInt, 1);
    const int64_t B = now.numel();
    const Table t = table(a[5], "block_table", B);
    const int *old = given(a[6]) ? index<int>(a[6], "ctx_old", at::kInt, B) : nullptr;
    check("kv_index", kv_index(&c, as_int(Hkv, "heads"), as_int(D, "channels"), &x, t.p, as_int(B, "sequences"), t.ld,
                               t.cols, old, static_cast<int *>(ptr(now)), status_word(a[8]), stream.handle()));
    Py_RETURN_NONE;
  });
}

// (q, cu_nodes, codes, exps, page_size, block_table, ctx_len, n_sel, first, last, out, dev_status, stream)
PyObject *py_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 13);
    const Stream stream(a[12]);
    const at::Tensor &q = heads_of(a[0], "q");
    if (!THPVariable_Check(a[2])) bad("an index holds two tensors");
    const at::Tensor &codes = THPVariable_Unpack(a[2]);
    need(codes.dim() == 4 || codes.dim() == 5, "index.codes is ([layers,] pages, Hkv, 2, D)");
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = codes.size(-3);
    const mxg_page_index x = index_of(a[2], a[3], Hkv, D, true);
    const at::Tensor &ctx = tensor(a[6], "ctx_len", at::kInt, 1);
    const int64_t B = ctx.numel();
    const int *cu = index<int>(a[1], "cu_nodes", at::kInt, B + 1);
    const Table t = table(a[5], "block_table", B);
    const long page = integer(a[4]), n_sel = integer(a[7]), first = integer(a[8]), last = integer(a[9]);
    for (const long i : {page, n_sel, first, last}) need(i >= 0 && i <= INT_MAX, "a number of pages is out of range");
    need(n_sel >= 1 && n_sel <= MXG_ATTN_MAX_SELECT, "n_sel must be 1 to 512");
    const at::Tensor sel = given(a[10]) ? tensor(a[10], "out", at::kInt, 3)
                                        : at::empty({N, Hkv, (int64_t)n_sel}, q.options().dtype(at::kInt));
    need(sel.size(0) == N && sel.size(1) == Hkv && sel.size(2) == n_sel && sel.is_contiguous(),
         "out must be contiguous (N, Hkv, n_sel)");
    const mxg_heads qh = heads(q);
    check("attn_select", attn_select(&qh, cu, as_int(B, "sequences"), as_int(N, "nodes"), &x, (int)page, t.p, t.ld, t.cols,
                                     static_cast<int *>(ptr(ctx)), as_int(Hq, "heads"), as_int(Hkv, "heads"),
                                     as_int(D, "channels"), (int)n_sel, (int)first, (int)last,
                                     static_cast<int *>(ptr(sel)), status_word(a[11]), stream.handle()));
    return THPVariable_Wrap(sel);
  });
}

// (k, v, cu_nodes, accept, cache k, cache v, block_table, ctx_len, ctx_out, dev_status, stream)
PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    count(n, 11);
    const Stream stream(a[10]);
    if (!THPVariable_Check(a[0])) bad("k must be a tensor");
    const int dim = THPVariable_Unpack(a[0]).dim() == 4 ? 4 : 3;
    const at::Tensor &k = tensor(a[0], "k", at::kBFloat16, dim), &v = tensor(a[1], "v", at::kBFloat16, dim);
    need(k.sizes() == v.sizes(), "k and v must be ([layers,] N, Hkv, D)");
    const int64_t N = k.size(-3), Hkv = k.size(-2), D = k.size(-1);
    const mxg_kv_cache c = cache_of(a[4], a[5], Hkv, D, false);
    need((dim == 4 ? k.size(0) : 1) == c.layers, "k and the cache differ in layers");
    const at::Tensor &ctx = tensor(a[7], "ctx_len", at::kInt, 1);
    const int64_t B = ctx.numel();
    const int *cu = index<int>(a[2], "cu_nodes", at::kInt, B + 1);
    const Table acc = table(a[3], "accept", B), t = table(a[6], "block_table", B);
    const at::Tensor out = given(a[8]) ? tensor(a[8], "ctx_out", at::kInt, 1) : at::empty_like(ctx);
    need(out.numel() == B, "ctx_out needs an entry a sequence");
    const mxg_heads kh = heads(k), vh = heads(v);
    check("kv_append",
          kv_append(&kh, dim == 4 ? k.stride(0) : 0, &vh, dim == 4 ? v.stride(0) : 0, cu, as_int(B, "sequences"),
                    as_int(N, "nodes"), acc.p, acc.ld, acc.cols, &c, t.p, t.ld, t.cols, static_cast<int *>(ptr(ctx)),
                    as_int(Hkv, "heads"), as_int(D, "channels"), static_cast<int *>(ptr(out)), status_word(a[9]),
                    stream.handle()));
    return THPVariable_Wrap(out);
  });
}

PyObject *py_set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {
    {"qk_norm_rope", fast<py_rope>(), METH_FASTCALL, nullptr},
    {"attn_prompt", fast<py_prompt>(), METH_FASTCALL, nullptr},
    {"attn_tree", fast<py_tree>(), METH_FASTCALL, nullptr},
    {"attn_shared", fast<py_shared>(), METH_FASTCALL, nullptr},
    {"attn_sparse", fast<py_sparse>(), METH_FASTCALL, nullptr},
    {"attn_select", fast<py_select>(), METH_FASTCALL, nullptr},
    {"kv_index", fast<py_index>(), METH_FASTCALL, nullptr},
    {"kv_append", fast<py_append>(), METH_FASTCALL, nullptr},
    {"set_error", py_set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_bind() { return PyModule_Create(&g_module); }
