// cross_binding.h -- Python binding of the norm and rotation of queries and keys
// and of cross attention (fa4fp4_norm_rope*, fa4bf16_cross_* of
// include/fa4fp4.h).  Part of the native module of cache_binding.cpp, for the
// same reason: these are calls of every layer.
#pragma once
#include "binding.h"

namespace {

// A [B, H, N, d] tensor, strided but for its last dimension, on CUDA device
// `index`.
fa4fp4_heads heads(PyObject* x, const char* name, int index, at::ScalarType type, int64_t B, int64_t H, int64_t N,
                   int64_t d) {
  const at::Tensor& t = as_tensor(x, name);
  if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type || t.dim() != 4 || t.size(0) != B ||
      t.size(1) != H || t.size(2) != N || t.size(3) != d || t.stride(3) != 1)
    refuse("%s: expected a %s tensor of shape [%lld, %lld, %lld, %lld] with a dense last dimension on cuda:%d", name,
           at::toString(type), (long long)B, (long long)H, (long long)N, (long long)d, index);
  return fa4fp4_heads{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

fa4fp4_heads heads(const at::Tensor& t) {
  return fa4fp4_heads{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

// The sizes of a [B, H, N, d] tensor, each within an int.
void sizes(PyObject* x, const char* name, int64_t (&s)[4]) {
  const at::Tensor& t = as_tensor(x, name);
  if (t.dim() != 4) refuse("%s: expected 4 dimensions, got %d", name, (int)t.dim());
  for (int i = 0; i < 4; ++i)
    if ((s[i] = t.size(i)) > INT_MAX) refuse("%s: too large", name);
}

// The caller's output of a name, or a fresh dense one.
struct Output {
  at::Tensor t;
  PyObject* mine;
  fa4fp4_heads h;
  Output(PyObject* x, const char* name, int index, int64_t B, int64_t H, int64_t N, int64_t d) {
    mine = given(x) ? x : nullptr;
    if (mine) {
      h = heads(x, name, index, at::kBFloat16, B, H, N, d);
    } else {
      t = fresh({B, H, N, d}, at::kBFloat16, index);
      h = heads(t);
    }
  }
  PyObject* get() const { return mine ? Py_NewRef(mine) : THPVariable_Wrap(t); }
};

// A tuple of new references (any of them nullptr: an error is set).
template <size_t N>
PyObject* tuple(PyObject* (&parts)[N]) {
  bool ok = true;
  for (PyObject* x : parts) ok = ok && x;
  PyObject* all = ok ? PyTuple_New(N) : nullptr;
  for (size_t i = 0; i < N; ++i) {
    if (all) PyTuple_SET_ITEM(all, i, parts[i]);
    else Py_XDECREF(parts[i]);
  }
  return all;
}

// ---------------------------------------------------------------- norm and rotation
struct NormRotation {
  fa4fp4_norm norm;
  fa4fp4_rotation rotation;
  int sections[4];
  const fa4fp4_norm* n = nullptr;
  const fa4fp4_rotation* r = nullptr;
  bool has_wq = false, has_wk = false;

  static const void* weight(PyObject* x, const char* name, int index, int64_t d, int* type, bool first) {
    if (!given(x)) return nullptr;
    const at::Tensor& t = as_tensor(x, name);
    const bool bf16 = t.scalar_type() == at::kBFloat16;
    const int is = bf16 ? FA4FP4_OUT_BF16 : FA4FP4_OUT_F32;
    if (!first && is != *type) refuse("q_weight and k_weight must have the same type");
    *type = is;
    return expect(x, name, index, bf16 ? at::kBFloat16 : at::kFloat, {d}).data_ptr();
  }

  NormRotation(PyObject* positions, PyObject* freqs, PyObject* wq, PyObject* wk, PyObject* parts, PyObject* interleaved,
               PyObject* with_norm, PyObject* eps, int index, int64_t B, int64_t N, int64_t d) {
    if (as_bool(with_norm, true)) {
      norm.weight_dtype = FA4FP4_OUT_F32;
      norm.q_weight = weight(wq, "q_weight", index, d, &norm.weight_dtype, true);
      norm.k_weight = weight(wk, "k_weight", index, d, &norm.weight_dtype, !norm.q_weight);
      norm.eps = eps ? as_float(eps) : 1e-6f;
      has_wq = norm.q_weight;
      has_wk = norm.k_weight;
      n = &norm;
    } else if (given(wq) || given(wk)) {
      refuse("q_weight and k_weight need norm=True");
    }
    if (!given(positions)) {
      if (given(freqs)) refuse("freqs need positions");
      if (!n) refuse("neither a norm nor positions are given");
      return;
    }
    if (!given(freqs)) refuse("positions need freqs");
    const at::Tensor& f = as_tensor(freqs, "freqs");
    if (!f.is_cpu() || f.scalar_type() != at::kDouble || f.dim() != 1 || f.size(0) != d / 2 || !f.is_contiguous())
      refuse("freqs: expected a contiguous float64 CPU tensor of shape [%lld]", (long long)(d / 2));
    int axes = 1;
    sections[0] = (int)(d / 2);
    if (given(parts)) {
      PyObject* seq = PySequence_Fast(parts, "sections: expected a sequence");
      if (!seq) throw Refused();
      const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
      long long sum = 0;
      bool ok = count >= 1 && count <= 4;
      for (Py_ssize_t i = 0; ok && i < count; ++i) {
        const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        if (v == -1 && PyErr_Occurred()) {
          Py_DECREF(seq);
          throw Refused();
        }
        ok = v >= 0 && v <= d / 2;
        sections[i] = (int)v;
        sum += v;
      }
      Py_DECREF(seq);
      if (!ok || sum != d / 2) refuse("sections: expected 1 to 4 numbers of channel pairs, %lld in all", (long long)(d / 2));
      axes = (int)count;
    }
    const at::Tensor& t = as_tensor(positions, "positions");
    rotation.shared = t.dim() == 2;
    rotation.positions = rotation.shared ? ints(positions, "positions", index, {axes, N})
                                         : ints(positions, "positions", index, {B, axes, N});
    rotation.axes = axes;
    rotation.sections = sections;
    rotation.freqs = static_cast<const double*>(f.data_ptr());
    rotation.interleaved = as_bool(interleaved, false);
    r = &rotation;
  }
};

// q [B, Hq, N, d] and k [B, Hkv, N, d] or None.
struct QueriesKeys {
  int64_t s[4], Hkv = 0;
  int index;
  fa4fp4_heads q, k;
  bool has_k;

  QueriesKeys(PyObject* q_, PyObject* k_) {
    sizes(q_, "q", s);
    const at::Tensor& t = as_tensor(q_, "q");
    if (!t.is_cuda()) refuse("q: expected a CUDA tensor");
    index = t.get_device();
    q = heads(q_, "q", index, at::kBFloat16, s[0], s[1], s[2], s[3]);
    has_k = given(k_);
    if (has_k) {
      int64_t n[4];
      sizes(k_, "k", n);
      Hkv = n[1];
      k = heads(k_, "k", index, at::kBFloat16, s[0], Hkv, s[2], s[3]);
    }
  }
};

PyObject* norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"qk_norm_rope", 12, 2,
                                {"q", "k", "positions", "freqs", "q_weight", "k_weight", "sections", "interleaved",
                                 "norm", "eps", "q_out", "k_out"}};
    PyObject* a[12];
    parse(s, args, n, kw, a);
    const QueriesKeys x(a[0], a[1]);
    const int64_t B = x.s[0], Hq = x.s[1], N = x.s[2], d = x.s[3];
    const NormRotation how(a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], x.index, B, N, d);
    if (!x.has_k && (how.has_wk || given(a[11]))) refuse("k_weight and k_out need k");
    const Output qo(a[10], "q_out", x.index, B, Hq, N, d);
    const Output ko(x.has_k ? a[11] : nullptr, "k_out", x.index, x.has_k ? B : 0, x.Hkv, N, d);
    launch("fa4fp4_norm_rope", x.index, [&](void* st) {
      return fa4fp4_norm_rope(&x.q, x.has_k ? &x.k : nullptr, (int)B, (int)Hq, (int)x.Hkv, (int)N, (int)d, how.n, how.r,
                              &qo.h, x.has_k ? &ko.h : nullptr, st);
    });
    PyObject* parts[2] = {qo.get(), x.has_k ? ko.get() : Py_NewRef(Py_None)};
    return tuple(parts);
  });
}

PyObject* norm_rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"qk_norm_rope_bwd", 15, 4,
                                {"dq_out", "dk_out", "q", "k", "positions", "freqs", "q_weight", "k_weight", "sections",
                                 "interleaved", "norm", "eps", "dq", "dk", "workspace"}};
    PyObject* a[15];
    parse(s, args, n, kw, a);
    const QueriesKeys x(a[2], a[3]);
    const int64_t B = x.s[0], Hq = x.s[1], N = x.s[2], d = x.s[3];
    const NormRotation how(a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], x.index, B, N, d);
    if (!x.has_k && (how.has_wk || given(a[1]) || given(a[13]))) refuse("dk_out, k_weight and dk need k");
    const bool f32 = as_tensor(a[0], "dq_out").scalar_type() == at::kFloat;
    const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
    const fa4fp4_heads dyq = heads(a[0], "dq_out", x.index, type, B, Hq, N, d);
    fa4fp4_heads dyk{};
    if (x.has_k) dyk = heads(a[1], "dk_out", x.index, type, B, x.Hkv, N, d);
    const Output dq(a[12], "dq", x.index, B, Hq, N, d);
    const Output dk(x.has_k ? a[13] : nullptr, "dk", x.index, x.has_k ? B : 0, x.Hkv, N, d);
    at::Tensor wq, wk, ws;
    if (how.has_wq) wq = fresh({d}, at::kFloat, x.index);
    if (how.has_wk) wk = fresh({d}, at::kFloat, x.index);
    if (how.has_wq || how.has_wk)
      ws = workspace(a[14], x.index,
                     fa4fp4_norm_rope_bwd_workspace_bytes((int)B, (int)Hq, (int)x.Hkv, (int)N, (int)d));
    launch("fa4fp4_norm_rope_bwd", x.index, [&](void* st) {
      return fa4fp4_norm_rope_bwd(&dyq, x.has_k ? &dyk : nullptr, f32 ? FA4FP4_OUT_F32 : FA4FP4_OUT_BF16, &x.q,
                                  x.has_k ? &x.k : nullptr, (int)B, (int)Hq, (int)x.Hkv, (int)N, (int)d, how.n, how.r,
                                  &dq.h, x.has_k ? &dk.h : nullptr,
                                  how.has_wq ? static_cast<float*>(wq.data_ptr()) : nullptr,
                                  how.has_wk ? static_cast<float*>(wk.data_ptr()) : nullptr,
                                  ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, st);
    });
    PyObject* parts[4] = {dq.get(), x.has_k ? dk.get() : Py_NewRef(Py_None),
                          how.has_wq ? THPVariable_Wrap(wq) : Py_NewRef(Py_None),
                          how.has_wk ? THPVariable_Wrap(wk) : Py_NewRef(Py_None)};
    return tuple(parts);
  });
}

// ---------------------------------------------------------------- cross attention
struct CrossInputs {
  int64_t B, Hq, Hkv, Nq, Nk, d;
  int index;
  fa4fp4_heads q, k, v;
  const int* lens;

  CrossInputs(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* lens_) {
    int64_t s[4], t[4];
    sizes(q_, "q", s);
    sizes(k_, "k", t);
    const at::Tensor& x = as_tensor(q_, "q");
    if (!x.is_cuda()) refuse("q: expected a CUDA tensor");
    index = x.get_device();
    B = s[0]; Hq = s[1]; Nq = s[2]; d = s[3];
    Hkv = t[1]; Nk = t[2];
    q = heads(q_, "q", index, at::kBFloat16, B, Hq, Nq, d);
    k = heads(k_, "k", index, at::kBFloat16, B, Hkv, Nk, d);
    v = heads(v_, "v", index, at::kBFloat16, B, Hkv, Nk, d);
    lens = ints(lens_, "kv_lens", index, {B});
  }
};

PyObject* cross_fwd(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cross_fwd", 8, 3,
                                {"q", "k", "v", "kv_lens", "softmax_scale", "with_lse", "out", "lse"}};
    PyObject* a[8];
    parse(s, args, n, kw, a);
    const CrossInputs x(a[0], a[1], a[2], a[3]);
    const float scale = as_float(a[4]);
    const bool with_lse = as_bool(a[5], true);
    const Output o(a[6], "out", x.index, x.B, x.Hq, x.Nq, x.d);
    at::Tensor l;
    if (with_lse)
      l = given(a[7]) ? expect(a[7], "lse", x.index, at::kFloat, {x.B, x.Hq, x.Nq})
                      : fresh({x.B, x.Hq, x.Nq}, at::kFloat, x.index);
    launch("fa4bf16_cross_fwd", x.index, [&](void* st) {
      return fa4bf16_cross_fwd(&x.q, &x.k, &x.v, x.lens, (int)x.B, (int)x.Hq, (int)x.Hkv, (int)x.Nq, (int)x.Nk,
                               (int)x.d, scale, &o.h, with_lse ? static_cast<float*>(l.data_ptr()) : nullptr, st);
    });
    PyObject* parts[2] = {o.get(), !with_lse ? Py_NewRef(Py_None) : given(a[7]) ? Py_NewRef(a[7]) : THPVariable_Wrap(l)};
    return tuple(parts);
  });
}

PyObject* cross_bwd(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const Signature s = {"cross_bwd", 12, 6,
                                {"q", "k", "v", "o", "dout", "lse", "kv_lens", "softmax_scale", "dq", "dk", "dv",
                                 "workspace"}};
    PyObject* a[12];
    parse(s, args, n, kw, a);
    const CrossInputs x(a[0], a[1], a[2], a[6]);
    const fa4fp4_heads o = heads(a[3], "o", x.index, at::kBFloat16, x.B, x.Hq, x.Nq, x.d);
    const fa4fp4_heads g = heads(a[4], "dout", x.index, at::kBFloat16, x.B, x.Hq, x.Nq, x.d);
    const float* lse = static_cast<float*>(expect(a[5], "lse", x.index, at::kFloat, {x.B, x.Hq, x.Nq}).data_ptr());
    const float scale = as_float(a[7]);
    const Output dq(a[8], "dq", x.index, x.B, x.Hq, x.Nq, x.d);
    const Output dk(a[9], "dk", x.index, x.B, x.Hkv, x.Nk, x.d), dv(a[10], "dv", x.index, x.B, x.Hkv, x.Nk, x.d);
    const at::Tensor ws = workspace(a[11], x.index,
                                    fa4bf16_cross_bwd_workspace_bytes((int)x.B, (int)x.Hq, (int)x.Hkv, (int)x.Nq,
                                                                      (int)x.Nk, (int)x.d));
    launch("fa4bf16_cross_bwd", x.index, [&](void* st) {
      return fa4bf16_cross_bwd(&x.q, &x.k, &x.v, &o, &g, lse, x.lens, (int)x.B, (int)x.Hq, (int)x.Hkv, (int)x.Nq,
                               (int)x.Nk, (int)x.d, scale, &dq.h, &dk.h, &dv.h,
                               ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, st);
    });
    PyObject* parts[3] = {dq.get(), dk.get(), dv.get()};
    return tuple(parts);
  });
}

#define FA4_CROSS_METHODS                                                                                            \
  {"qk_norm_rope", FA4_METHOD(norm_rope),                                                                            \
   "qk_norm_rope(q, k, positions=None, freqs=None, q_weight=None, k_weight=None, sections=None,\n"                   \
   "             interleaved=False, norm=True, eps=1e-6, q_out=None, k_out=None) -> (q_out, k_out)\n\n"              \
   "RMS norm of every row of q (bf16 [B, Hq, N, d], strided views too) and k ([B, Hkv, N, d], or None)\n"            \
   "and its rotation by position, in one pass (fa4fp4_norm_rope).  positions: int32 [B, axes, N], or\n"              \
   "[axes, N] for all sequences; None: no rotation.  freqs: radians a position, float64 [d / 2] on the\n"            \
   "CPU (rope_freqs).  sections: channel pairs of each axis (default: one axis).  Pairs are (i, i + d/2),\n"         \
   "or (2i, 2i + 1) when interleaved.  Weights: f32 or bf16 [d]; None: ones.  q_out may be q, k_out k."},            \
  {"qk_norm_rope_bwd", FA4_METHOD(norm_rope_bwd),                                                                    \
   "qk_norm_rope_bwd(dq_out, dk_out, q, k, positions=None, freqs=None, q_weight=None, k_weight=None,\n"              \
   "                 sections=None, interleaved=False, norm=True, eps=1e-6, dq=None, dk=None, workspace=None)\n"     \
   "    -> (dq, dk, dq_weight, dk_weight)\n\n"                                                                       \
   "Gradients of qk_norm_rope (fa4fp4_norm_rope_bwd) from those of its outputs, f32 (as bwd gives them) or\n"        \
   "bf16, and its inputs: dq, dk bf16, the weights' in f32 (None where no weight was given)."},                      \
  {"cross_fwd", FA4_METHOD(cross_fwd),                                                                               \
   "cross_fwd(q, k, v, kv_lens=None, softmax_scale=0.0, with_lse=True, out=None, lse=None) -> (o, lse or None)\n\n"  \
   "BF16 attention of q [B, Hq, Nq, d] to k and v [B, Hkv, Nk, d] of another length, strided views too, no\n"        \
   "causal mask (fa4bf16_cross_fwd).  kv_lens: int32 [B], each sequence's number of keys (default: all);\n"          \
   "without a key o = 0 and lse = -inf."},                                                                           \
  {"cross_bwd", FA4_METHOD(cross_bwd),                                                                               \
   "cross_bwd(q, k, v, o, dout, lse, kv_lens=None, softmax_scale=0.0, dq=None, dk=None, dv=None,\n"                  \
   "          workspace=None) -> (dq, dk, dv)\n\n"                                                                   \
   "Gradients of cross_fwd from its inputs, its o and lse and o's gradient (fa4bf16_cross_bwd), in bf16."},

}  // namespace
