// cache_binding.cpp -- Python binding of the 8-bit key/value cache
// (fa4fp4_cache_* of include/fa4fp4.h) as a native extension module.
//
// Marshalling only, like the ctypes binding of the other calls: it checks torch
// tensors, takes their pointers and the current stream, and calls the C ABI.
// These calls are made once per layer and generated token, where the checks, a
// ctypes call and the allocations of outputs cost more than the kernels of a
// small step: 15 us in Python and ctypes for an append whose kernel takes 5,
// 2.0 us here.
#include "binding.h"
#include "cross_binding.h"

namespace {

// ---------------------------------------------------------------- KVCache
// It keeps the tensors and their sizes, no addresses: a tensor may have been given
// other memory (resize_, set_) since.
struct Cache {
  PyObject_HEAD
  PyObject *k, *v, *ks, *vs, *kb;
  int index, num_pages, Hkv, page, d;
};

// The structure of a call, from tensors that have (still) the cache's sizes.
fa4fp4_cache structure(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, PyObject* kb, int index, int64_t n, int64_t H,
                       int64_t page, int64_t d) {
  fa4fp4_cache c;
  c.k_codes = expect(k, "k", index, at::kByte, {n, H, page, d}).data_ptr();
  c.v_codes = expect(v, "v", index, at::kByte, {n, H, page, d}).data_ptr();
  c.k_scales = expect(ks, "ks", index, at::kByte, {n, H}).data_ptr();
  c.v_scales = expect(vs, "vs", index, at::kByte, {n, H}).data_ptr();
  c.k_bounds = expect(kb, "kb", index, at::kByte, {n, H, 2, d}).data_ptr();
  c.num_pages = (int)n; c.Hkv = (int)H; c.page = (int)page; c.d = (int)d;
  return c;
}

int cache_init(PyObject* self, PyObject* args, PyObject* kwargs) {
  Cache* o = reinterpret_cast<Cache*>(self);
  static const char* names[] = {"k", "v", "ks", "vs", "kb", nullptr};
  PyObject *k, *v, *ks, *vs, *kb;
  if (!PyArg_ParseTupleAndKeywords(args, kwargs, "OOOOO", const_cast<char**>(names), &k, &v, &ks, &vs, &kb)) return -1;
  try {
    const at::Tensor& tk = as_tensor(k, "k");
    const int64_t n = dim(tk, "k", 4, 0), H = tk.size(1), page = tk.size(2), d = tk.size(3);
    if (!tk.is_cuda()) refuse("fa4fp4: a cache's tensors must be CUDA tensors");
    const int index = tk.get_device();
    if (n > INT_MAX || H > INT_MAX || page > INT_MAX || d > INT_MAX) refuse("k: too large");
    structure(k, v, ks, vs, kb, index, n, H, page, d);
    PyObject* had[] = {o->k, o->v, o->ks, o->vs, o->kb};
    Py_INCREF(k); Py_INCREF(v); Py_INCREF(ks); Py_INCREF(vs); Py_INCREF(kb);
    o->k = k; o->v = v; o->ks = ks; o->vs = vs; o->kb = kb;
    o->index = index;
    o->num_pages = (int)n; o->Hkv = (int)H; o->page = (int)page; o->d = (int)d;
    for (PyObject* x : had) Py_XDECREF(x);
    return 0;
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return -1;
}

void cache_dealloc(PyObject* self) {
  Cache* o = reinterpret_cast<Cache*>(self);
  Py_XDECREF(o->k); Py_XDECREF(o->v); Py_XDECREF(o->ks); Py_XDECREF(o->vs); Py_XDECREF(o->kb);
  Py_TYPE(self)->tp_free(self);
}

PyObject* cache_device(PyObject* self, void*) {
  PyObject* k = reinterpret_cast<Cache*>(self)->k;
  if (k) return PyObject_GetAttrString(k, "device");
  PyErr_SetString(PyExc_AttributeError, "device");
  return nullptr;
}

PyMemberDef cache_members[] = {
    {"k", T_OBJECT_EX, offsetof(Cache, k), READONLY, "K codes, uint8 [num_pages, Hkv, page, d]"},
    {"v", T_OBJECT_EX, offsetof(Cache, v), READONLY, "V codes, uint8 [num_pages, Hkv, page, d]"},
    {"ks", T_OBJECT_EX, offsetof(Cache, ks), READONLY, "K scales, uint8 [num_pages, Hkv]"},
    {"vs", T_OBJECT_EX, offsetof(Cache, vs), READONLY, "V scales, uint8 [num_pages, Hkv]"},
    {"kb", T_OBJECT_EX, offsetof(Cache, kb), READONLY, "K bounds, uint8 [num_pages, Hkv, 2, d]"},
    {"num_pages", T_INT, offsetof(Cache, num_pages), READONLY, "pages of the pool"},
    {"Hkv", T_INT, offsetof(Cache, Hkv), READONLY, "kv heads"},
    {"page", T_INT, offsetof(Cache, page), READONLY, "tokens of a page"},
    {"d", T_INT, offsetof(Cache, d), READONLY, "head dimension"},
    {nullptr}};
PyGetSetDef cache_getset[] = {{"device", cache_device, nullptr, "the tensors' device", nullptr}, {nullptr}};

PyTypeObject cache_type = {PyVarObject_HEAD_INIT(nullptr, 0)};

// ---------------------------------------------------------------- calls
// The sequences that every call is given.
struct Sequences {
  fa4fp4_cache c;
  int index, B, max_pages;
  const int *table, *lens, *counts;

  Sequences(PyObject* cache_, PyObject* table_, PyObject* lens_, PyObject* counts_, const char* counts_name) {
    if (Py_TYPE(cache_) != &cache_type || !reinterpret_cast<Cache*>(cache_)->k) refuse("cache: expected a KVCache");
    const Cache* o = reinterpret_cast<Cache*>(cache_);
    index = o->index;
    c = structure(o->k, o->v, o->ks, o->vs, o->kb, index, o->num_pages, o->Hkv, o->page, o->d);
    const at::Tensor& t = as_tensor(table_, "page_table");
    const int64_t b = dim(t, "page_table", 2, 0), m = t.size(1);
    if (b > INT_MAX || m > INT_MAX) refuse("page_table: too large");
    B = (int)b;
    max_pages = (int)m;
    table = ints(table_, "page_table", index, {b, m});
    if (!given(lens_)) refuse("lens: expected a tensor");
    lens = ints(lens_, "lens", index, {b});
    counts = ints(counts_, counts_name, index, {b});
  }
};

struct Queries {
  int Hq, T;
  const void* q;

  Queries(const Sequences& s, PyObject* q_) {
    const at::Tensor& t = as_tensor(q_, "q");
    const int64_t h = dim(t, "q", 4, 1), n = t.size(2);
    if (h > INT_MAX || n > INT_MAX) refuse("q: too large");
    q = expect(q_, "q", s.index, at::kBFloat16, {s.B, h, n, s.c.d}).data_ptr();
    Hq = (int)h;
    T = (int)n;
  }
};

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cache_append", 6, 5, {"cache", "k", "v", "page_table", "lens", "n_new"}};
    PyObject* a[6];
    parse(s, args, n, kw, a);
    const Sequences q(a[0], a[3], a[4], a[5], "n_new");
    const fa4fp4_cache* c = &q.c;
    const int64_t T = dim(as_tensor(a[1], "k"), "k", 4, 2);
    if (T > INT_MAX) refuse("k: too large");
    const void* k = expect(a[1], "k", q.index, at::kBFloat16, {q.B, c->Hkv, T, c->d}).data_ptr();
    const void* v = expect(a[2], "v", q.index, at::kBFloat16, {q.B, c->Hkv, T, c->d}).data_ptr();
    launch("fa4fp4_cache_append", q.index, [&](void* st) {
      return fa4fp4_cache_append(c, k, v, q.table, q.lens, q.counts, q.B, q.max_pages, (int)T, st);
    });
    Py_RETURN_NONE;
  });
}

PyObject* fwd(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cache_fwd", 13, 4,
                                {"q", "cache", "page_table", "lens", "q_lens", "causal", "softmax_scale", "out_dtype",
                                 "with_lse", "out", "lse", "pages", "workspace"}};
    PyObject* a[13];
    parse(s, args, n, kw, a);
    const Sequences q(a[1], a[2], a[3], a[4], "q_lens");
    const Queries r(q, a[0]);
    const fa4fp4_cache* c = &q.c;
    const bool causal = as_bool(a[5], true), with_lse = as_bool(a[8], true);
    const float scale = as_float(a[6]);
    const int out_dtype = a[7] ? as_int(a[7], "out_dtype") : FA4FP4_OUT_BF16;
    if (out_dtype != FA4FP4_OUT_F32 && out_dtype != FA4FP4_OUT_BF16) refuse("out_dtype must be OUT_F32 or OUT_BF16");
    const at::ScalarType type = out_dtype == FA4FP4_OUT_BF16 ? at::kBFloat16 : at::kFloat;
    // rows that the call does not write hold zeros, not what the allocator left
    const bool zero = q.counts != nullptr;
    const at::Tensor o = given(a[9]) ? expect(a[9], "out", q.index, type, {q.B, r.Hq, r.T, c->d})
                                     : fresh({q.B, r.Hq, r.T, c->d}, type, q.index, zero);
    at::Tensor l;
    if (with_lse)
      l = given(a[10]) ? expect(a[10], "lse", q.index, at::kFloat, {q.B, r.Hq, r.T})
                       : fresh({q.B, r.Hq, r.T}, at::kFloat, q.index, zero);
    const int* pages = nullptr;
    int n_sel = 0;
    if (given(a[11])) {
      const int64_t m = dim(as_tensor(a[11], "pages"), "pages", 4, 3);
      if (m > INT_MAX) refuse("pages: too large");
      pages = ints(a[11], "pages", q.index, {q.B, c->Hkv, r.T, m});
      n_sel = (int)m;
    }
    const size_t need = fa4fp4_cache_fwd_workspace_bytes(q.B, r.Hq, c->Hkv, r.T, c->d, c->page, q.max_pages, n_sel);
    const at::Tensor ws = workspace(a[12], q.index, need ? need : 16);
    launch("fa4fp4_cache_fwd", q.index, [&](void* st) {
      return fa4fp4_cache_fwd(c, r.q, q.table, q.lens, q.counts, pages, q.B, r.Hq, r.T, q.max_pages, n_sel, scale,
                              causal, o.data_ptr(), out_dtype, with_lse ? static_cast<float*>(l.data_ptr()) : nullptr,
                              ws.data_ptr(), (size_t)ws.numel(), st);
    });
    PyObject* po = given(a[9]) ? Py_NewRef(a[9]) : THPVariable_Wrap(o);
    PyObject* pl = !with_lse ? Py_NewRef(Py_None) : given(a[10]) ? Py_NewRef(a[10]) : THPVariable_Wrap(l);
    if (!po || !pl) {
      Py_XDECREF(po);
      Py_XDECREF(pl);
      return nullptr;
    }
    PyObject* both = PyTuple_Pack(2, po, pl);
    Py_DECREF(po);
    Py_DECREF(pl);
    return both;
  });
}

PyObject* select(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cache_select", 8, 5,
                                {"q", "cache", "page_table", "lens", "n_pages", "q_lens", "out", "workspace"}};
    PyObject* a[8];
    parse(s, args, n, kw, a);
    const Sequences q(a[1], a[2], a[3], a[5], "q_lens");
    const Queries r(q, a[0]);
    const fa4fp4_cache* c = &q.c;
    const int n_sel = as_int(a[4], "n_pages");
    if (n_sel < 1) refuse("n_pages must be at least 1");
    const at::Tensor out = given(a[6]) ? expect(a[6], "out", q.index, at::kInt, {q.B, c->Hkv, r.T, n_sel})
                                       : fresh({q.B, c->Hkv, r.T, n_sel}, at::kInt, q.index);
    const at::Tensor ws =
        workspace(a[7], q.index, fa4fp4_cache_select_workspace_bytes(q.B, c->Hkv, r.T, q.max_pages));
    launch("fa4fp4_cache_select", q.index, [&](void* st) {
      return fa4fp4_cache_select(c, r.q, q.table, q.lens, q.counts, q.B, r.Hq, r.T, q.max_pages, n_sel,
                                 static_cast<int*>(out.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                                 ws.defined() ? (size_t)ws.numel() : 0, st);
    });
    return given(a[6]) ? Py_NewRef(a[6]) : THPVariable_Wrap(out);
  });
}

PyObject* weigh(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cache_weigh", 11, 6,
                                {"q", "lse", "cache", "page_table", "lens", "weight", "q_lens", "causal",
                                 "softmax_scale", "out", "workspace"}};
    PyObject* a[11];
    parse(s, args, n, kw, a);
    const Sequences q(a[2], a[3], a[4], a[6], "q_lens");
    const Queries r(q, a[0]);
    const fa4fp4_cache* c = &q.c;
    const float* lse = static_cast<float*>(expect(a[1], "lse", q.index, at::kFloat, {q.B, r.Hq, r.T}).data_ptr());
    const int64_t L = (int64_t)q.max_pages * c->page;
    const float* w = static_cast<float*>(expect(a[5], "weight", q.index, at::kFloat, {q.B, c->Hkv, L}).data_ptr());
    PyObject* po = given(a[9]) ? a[9] : a[5];
    float* out = static_cast<float*>(expect(po, "out", q.index, at::kFloat, {q.B, c->Hkv, L}).data_ptr());
    const bool causal = as_bool(a[7], true);
    const float scale = as_float(a[8]);
    const at::Tensor ws =
        workspace(a[10], q.index, fa4fp4_cache_weigh_workspace_bytes(q.B, r.Hq, c->Hkv, r.T, c->d));
    launch("fa4fp4_cache_weigh", q.index, [&](void* st) {
      return fa4fp4_cache_weigh(c, r.q, lse, q.table, q.lens, q.counts, q.B, r.Hq, r.T, q.max_pages, scale, causal, w,
                                out, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, st);
    });
    return Py_NewRef(po);
  });
}

PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cache_evict", 7, 6,
                                {"cache", "page_table", "lens", "weight", "dst_table", "budget", "recent"}};
    PyObject* a[7];
    parse(s, args, n, kw, a);
    const Sequences q(a[0], a[1], a[2], nullptr, "");
    const fa4fp4_cache* c = &q.c;
    const int64_t L = (int64_t)q.max_pages * c->page;
    const float* w = static_cast<float*>(expect(a[3], "weight", q.index, at::kFloat, {q.B, c->Hkv, L}).data_ptr());
    const int64_t m = dim(as_tensor(a[4], "dst_table"), "dst_table", 2, 1);
    if (m > INT_MAX) refuse("dst_table: too large");
    const int* dst = ints(a[4], "dst_table", q.index, {q.B, m});
    if (!dst) refuse("dst_table: expected a tensor");
    const int budget = as_int(a[5], "budget"), recent = a[6] ? as_int(a[6], "recent") : 0;
    const at::Tensor lens = fresh({q.B}, at::kInt, q.index);
    const at::Tensor kept = fresh({q.B, c->Hkv, budget > 0 ? budget : 0}, at::kInt, q.index);
    const at::Tensor out = fresh({q.B, c->Hkv, m * c->page}, at::kFloat, q.index);
    launch("fa4fp4_cache_evict", q.index, [&](void* st) {
      return fa4fp4_cache_evict(c, q.table, q.lens, w, dst, q.B, q.max_pages, (int)m, budget, recent,
                                static_cast<int*>(lens.data_ptr()), static_cast<int*>(kept.data_ptr()),
                                static_cast<float*>(out.data_ptr()), st);
    });
    PyObject* parts[3] = {THPVariable_Wrap(lens), THPVariable_Wrap(kept), THPVariable_Wrap(out)};
    PyObject* all = parts[0] && parts[1] && parts[2] ? PyTuple_Pack(3, parts[0], parts[1], parts[2]) : nullptr;
    for (PyObject* x : parts) Py_XDECREF(x);
    return all;
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"cache_append", FA4_METHOD(append),
     "cache_append(cache, k, v, page_table, lens, n_new=None)\n\n"
     "Store new tokens k, v (bf16 [B, Hkv, T, d]) behind the lens[b] tokens of every sequence\n"
     "(fa4fp4_cache_append): n_new[b] of them, or all T.  lens is not changed."},
    {"cache_fwd", FA4_METHOD(fwd),
     "cache_fwd(q, cache, page_table, lens, q_lens=None, causal=True, softmax_scale=0.0, out_dtype=OUT_BF16,\n"
     "          with_lse=True, out=None, lse=None, pages=None, workspace=None) -> (o, lse or None)\n\n"
     "Attention of the T newest tokens of every sequence, q bf16 [B, Hq, T, d], over the cache\n"
     "(fa4fp4_cache_fwd); lens counts them in.  pages (from cache_select) restricts every token to its own\n"
     "pages.  Rows t >= q_lens[b] of out and lse are not written (zeros where the call allocates them)."},
    {"cache_select", FA4_METHOD(select),
     "cache_select(q, cache, page_table, lens, n_pages, q_lens=None, out=None, workspace=None) -> pages\n\n"
     "The n_pages pages whose keys could score highest for every query token and kv head\n"
     "(fa4fp4_cache_select): int32 [B, Hkv, T, n_pages], ascending indexes into the sequence's row of\n"
     "page_table, then -1."},
    {"cache_weigh", FA4_METHOD(weigh),
     "cache_weigh(q, lse, cache, page_table, lens, weight, q_lens=None, causal=True, softmax_scale=0.0,\n"
     "            out=None, workspace=None) -> out\n\n"
     "weight plus the attention weight that every cached token received from the queries\n"
     "(fa4fp4_cache_weigh), with the lse of cache_fwd: f32 [B, Hkv, max_pages * page], written to out\n"
     "(default: into weight itself), positions behind a sequence's end untouched."},
    {"cache_evict", FA4_METHOD(evict),
     "cache_evict(cache, page_table, lens, weight, dst_table, budget, recent=0) -> (lens, kept, weight)\n\n"
     "Cut every sequence back to its `recent` newest and otherwise heaviest tokens, `budget` in all per kv\n"
     "head, copied into the pages of dst_table (int32 [B, dst_pages], fresh pages of the same cache;\n"
     "fa4fp4_cache_evict).  Returns the new lens int32 [B], the kept positions int32 [B, Hkv, budget] with -1\n"
     "behind and their weights f32 [B, Hkv, dst_pages * page] with 0 behind."},
    FA4_CROSS_METHODS
    {"set_error", set_error, METH_O, "set_error(type): the exception raised for a status, called with (where, status)"},
    {nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_cache_binding", "The calls of the 8-bit key/value cache, of norm and rotation and of cross attention", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() {
  cache_type.tp_name = "precision_attention_fa4fp4_gb300.KVCache";
  cache_type.tp_basicsize = sizeof(Cache);
  cache_type.tp_flags = Py_TPFLAGS_DEFAULT;
  cache_type.tp_new = PyType_GenericNew;
  cache_type.tp_init = cache_init;
  cache_type.tp_dealloc = cache_dealloc;
  cache_type.tp_members = cache_members;
  cache_type.tp_getset = cache_getset;
  cache_type.tp_doc =
      "KVCache(k, v, ks, vs, kb)\n\n"
      "A paged pool of K and V as E4M3 codes with one E8M0 scale per page and head (fa4fp4_cache of\n"
      "include/fa4fp4.h): uint8 CUDA tensors k, v [num_pages, Hkv, page, d], ks, vs [num_pages, Hkv] and kb\n"
      "[num_pages, Hkv, 2, d] (K bounds).  cache_alloc makes an empty one.";
  if (PyType_Ready(&cache_type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module_def);
  if (!m) return nullptr;
  if (PyModule_AddObjectRef(m, "KVCache", reinterpret_cast<PyObject*>(&cache_type)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
