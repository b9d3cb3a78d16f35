// cross_api.cu -- the C ABI of the norm and rotation of queries and keys and of
// cross attention: argument checks and launches.
#include <cmath>
#include <cstring>
#include "../../include/fa4fp4.h"
#include "cross.h"
#include "internal.h"
#include "rope.h"

namespace fa4 {
unsigned* device_error_word();
}

using namespace fa4;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fa4fp4_status status_of(cudaError_t e) { return e == cudaSuccess ? FA4FP4_OK : FA4FP4_ERR_CUDA; }

// A [B][H][N][d] view of elements of `size` bytes; `out`: its rows may not overlap.
fa4fp4_status check_heads(const fa4fp4_heads* t, int B, int H, int N, int size, bool out) {
  if (!t || !t->ptr) return FA4FP4_ERR_INVALID_ARG;
  const int64_t strides[3] = {t->stride_b, t->stride_h, t->stride_n};
  const int dims[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (dims[i] <= 1) continue;
    if (strides[i] < 0 || strides[i] > ((1LL << 40) / size)) return FA4FP4_ERR_INVALID_ARG;
    if (out && strides[i] == 0) return FA4FP4_ERR_INVALID_ARG;
  }
  if (!aligned(t->ptr, 16)) return FA4FP4_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (dims[i] > 1 && strides[i] * size % 16 != 0) return FA4FP4_ERR_ALIGNMENT;
  return FA4FP4_OK;
}

// The strides of dimensions of one element are never used: 0.
Strided strided(const fa4fp4_heads* t, int B, int H, int N) {
  return Strided{t->ptr, B > 1 ? t->stride_b : 0, H > 1 ? t->stride_h : 0, N > 1 ? t->stride_n : 0};
}

fa4fp4_status check_dims(int B, int Hq, int Hkv, int N, int d) {
  if (B < 0 || Hq < 0 || Hkv < 0 || N < 0) return FA4FP4_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA4FP4_ERR_UNSUPPORTED;
  // (sums of) head counts and token counts stay within 32 bits
  if (Hq > (1 << 20) || Hkv > (1 << 20) || (long long)B * N > (1LL << 30)) return FA4FP4_ERR_UNSUPPORTED;
  if ((long long)B * N * (Hq + Hkv) > (1LL << 40)) return FA4FP4_ERR_UNSUPPORTED;
  return FA4FP4_OK;
}

// Of the norm and rotation: tasks of 128 rows and more, and one for each token, stay within 31 bits.
fa4fp4_status check_rows_in_all(int B, int Hq, int Hkv, int N, int d) {
  const fa4fp4_status s = check_dims(B, Hq, Hkv, N, d);
  if (s != FA4FP4_OK) return s;
  return (long long)B * N * (Hq + Hkv) > (1LL << 36) ? FA4FP4_ERR_UNSUPPORTED : FA4FP4_OK;
}

fa4fp4_status check_norm(const fa4fp4_norm* norm) {
  if (!norm) return FA4FP4_OK;
  if (norm->weight_dtype != FA4FP4_OUT_F32 && norm->weight_dtype != FA4FP4_OUT_BF16) return FA4FP4_ERR_INVALID_ARG;
  if (!(norm->eps >= 0.f) || std::isinf(norm->eps)) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16)) return FA4FP4_ERR_ALIGNMENT;
  return FA4FP4_OK;
}

fa4fp4_status check_rotation(const fa4fp4_rotation* r, int d) {
  if (!r) return FA4FP4_OK;
  if (!r->positions || !r->sections || !r->freqs || r->axes < 1 || r->axes > 4) return FA4FP4_ERR_INVALID_ARG;
  long long sum = 0;
  for (int i = 0; i < r->axes; ++i) {
    if (r->sections[i] < 0) return FA4FP4_ERR_INVALID_ARG;
    sum += r->sections[i];
  }
  if (sum != d / 2) return FA4FP4_ERR_INVALID_ARG;
  for (int i = 0; i < d / 2; ++i)
    if (!std::isfinite(r->freqs[i])) return FA4FP4_ERR_INVALID_ARG;
  return aligned(r->positions, 4) ? FA4FP4_OK : FA4FP4_ERR_ALIGNMENT;
}

// f / (2 pi) modulo 1, times 2^64.  One product of 53 bits would be off by 2^-54 of itself, times the position: so the
// product with 1 / (2 pi) in two parts, and what its own rounding leaves.
uint64_t turn_of(double f) {
  constexpr double HI = 0x1.45f306dc9c883p-3, LO = -0x1.6b01ec5417056p-57;   // 1 / (2 pi) to 2^-110
  // (this product too by fma: a compiler may make a plain one and the subtraction below one fma, which rounds elsewhere)
  const double hi = std::fma(f, HI, 0.0), lo = std::fma(f, LO, std::fma(f, HI, -hi));
  const auto turn = [](double x) { return (uint64_t)(int64_t)((x - std::rint(x)) * 9223372036854775808.0) * 2; };
  return turn(hi) + turn(lo);
}

void set_rotation(RopeParams* p, const fa4fp4_norm* norm, const fa4fp4_rotation* r) {
  if (norm) {
    p->norm = 1;
    p->t[0].w = norm->q_weight;
    p->t[1].w = norm->k_weight;
    p->w_bf16 = norm->weight_dtype == FA4FP4_OUT_BF16;
    p->eps = norm->eps;
  }
  if (!r) return;
  p->pos = r->positions;
  p->pos_b = r->shared ? 0 : (long long)r->axes * p->N;
  p->pairs = r->interleaved ? 1 : 0;
  for (int a = 0, i = 0; a < r->axes; ++a)
    for (int j = 0; j < r->sections[a]; ++j, ++i) {
      p->axis[i] = (uint8_t)a;
      p->turn[i] = turn_of(r->freqs[i]);
    }
}

// Cross attention reads rows by TMA boxes: they may not lie on each other.
fa4fp4_status check_rows(const Strided& t, int N, int d) {
  return N > 1 && t.n < d ? FA4FP4_ERR_UNSUPPORTED : FA4FP4_OK;
}

float softmax_scale_of(float s, int d) { return s > 0.f ? s : (float)(1.0 / std::sqrt((double)d)); }

fa4fp4_status check_cross(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  fa4fp4_status s = check_dims(B, Hq, Hkv, Nq, d);
  if (s == FA4FP4_OK) s = check_dims(B, Hq, Hkv, Nk, d);
  if (s != FA4FP4_OK) return s;
  if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0) return FA4FP4_ERR_UNSUPPORTED;
  // tiles and rows are counted, and key and query positions padded, in 32 bits
  if (Nq > (1 << 30) || Nk > (1 << 30) || (long long)B * Hq * Nq > (1LL << 31) - 1 ||
      (long long)B * Hkv * Nk > (1LL << 31) - 1 || (long long)B * Hq > (1LL << 24))
    return FA4FP4_ERR_UNSUPPORTED;
  if ((long long)B * Hq * ((Nq + 127) / 128) > (1LL << 36) / ((Nk + 127) / 128 + 1)) return FA4FP4_ERR_UNSUPPORTED;
  return FA4FP4_OK;
}

}  // namespace

extern "C" {

fa4fp4_status fa4fp4_norm_rope(const fa4fp4_heads* q, const fa4fp4_heads* k, int B, int Hq, int Hkv, int N, int d,
                               const fa4fp4_norm* norm, const fa4fp4_rotation* rotation, const fa4fp4_heads* q_out,
                               const fa4fp4_heads* k_out, void* stream) {
  fa4fp4_status s = check_rows_in_all(B, Hq, Hkv, N, d);
  if (s != FA4FP4_OK) return s;
  if ((!norm && !rotation) || (!k && Hkv != 0)) return FA4FP4_ERR_INVALID_ARG;
  if (B == 0 || N == 0 || Hq + Hkv == 0) return FA4FP4_OK;
  if ((s = check_norm(norm)) != FA4FP4_OK || (s = check_rotation(rotation, d)) != FA4FP4_OK) return s;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.B = B; p.N = N; p.d = d;
  const fa4fp4_heads *in[2] = {q, k}, *out[2] = {q_out, k_out};
  const int H[2] = {Hq, Hkv};
  for (int t = 0; t < 2; ++t) {
    if (H[t] == 0) continue;
    if ((s = check_heads(in[t], B, H[t], N, 2, false)) != FA4FP4_OK) return s;
    if ((s = check_heads(out[t], B, H[t], N, 2, true)) != FA4FP4_OK) return s;
    p.t[t].x = strided(in[t], B, H[t], N);
    p.t[t].out = strided(out[t], B, H[t], N);
    p.t[t].H = H[t];
  }
  set_rotation(&p, norm, rotation);
  return status_of(launch_norm_rope(p, static_cast<cudaStream_t>(stream)));
}

size_t fa4fp4_norm_rope_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_rows_in_all(B, Hq, Hkv, N, d) != FA4FP4_OK || B == 0 || N == 0 || Hq + Hkv == 0) return 0;
  int ctas[2];
  rope_bwd_ctas(B, Hq, Hkv, N, d, ctas);
  return (size_t)(ctas[0] + ctas[1]) * d * sizeof(float);
}

fa4fp4_status fa4fp4_norm_rope_bwd(const fa4fp4_heads* dq_out, const fa4fp4_heads* dk_out, int dout_dtype,
                                   const fa4fp4_heads* q, const fa4fp4_heads* k, int B, int Hq, int Hkv, int N, int d,
                                   const fa4fp4_norm* norm, const fa4fp4_rotation* rotation, const fa4fp4_heads* dq,
                                   const fa4fp4_heads* dk, float* dq_weight, float* dk_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  fa4fp4_status s = check_rows_in_all(B, Hq, Hkv, N, d);
  if (s != FA4FP4_OK) return s;
  if (dout_dtype != FA4FP4_OUT_F32 && dout_dtype != FA4FP4_OUT_BF16) return FA4FP4_ERR_INVALID_ARG;
  if ((!norm && !rotation) || (!k && Hkv != 0)) return FA4FP4_ERR_INVALID_ARG;
  if (!norm && (dq_weight || dk_weight)) return FA4FP4_ERR_INVALID_ARG;
  if ((s = check_norm(norm)) != FA4FP4_OK || (s = check_rotation(rotation, d)) != FA4FP4_OK) return s;
  if (!aligned(dq_weight, 16) || !aligned(dk_weight, 16)) return FA4FP4_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.B = B; p.N = N; p.d = d;
  p.dy_f32 = dout_dtype == FA4FP4_OUT_F32;
  const fa4fp4_heads *in[2] = {q, k}, *dy[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
  float* dw[2] = {dq_weight, dk_weight};
  const int H[2] = {Hq, Hkv};
  const bool empty = B == 0 || N == 0;
  for (int t = 0; t < 2; ++t) {
    p.t[t].dw = dw[t];
    p.t[t].H = H[t];
    if (H[t] == 0 || empty) continue;
    if ((s = check_heads(in[t], B, H[t], N, 2, false)) != FA4FP4_OK) return s;
    if ((s = check_heads(dy[t], B, H[t], N, p.dy_f32 ? 4 : 2, false)) != FA4FP4_OK) return s;
    if ((s = check_heads(out[t], B, H[t], N, 2, true)) != FA4FP4_OK) return s;
    p.t[t].x = strided(in[t], B, H[t], N);
    p.t[t].dy = strided(dy[t], B, H[t], N);
    p.t[t].out = strided(out[t], B, H[t], N);
  }
  // the weights' gradients of no rows are zeros
  for (int t = 0; t < 2; ++t)
    if (dw[t] && (empty || H[t] == 0)) {
      if (cudaMemsetAsync(dw[t], 0, d * sizeof(float), st) != cudaSuccess) return FA4FP4_ERR_CUDA;
      p.t[t].dw = nullptr;
    }
  if (empty || Hq + Hkv == 0) return FA4FP4_OK;
  rope_bwd_ctas(B, Hq, Hkv, N, d, p.ctas);
  if (p.t[0].dw || p.t[1].dw) {
    if (!workspace || workspace_bytes < (size_t)(p.ctas[0] + p.ctas[1]) * d * sizeof(float))
      return FA4FP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FA4FP4_ERR_ALIGNMENT;
    p.t[0].part = static_cast<float*>(workspace);
    p.t[1].part = p.t[0].part + (size_t)p.ctas[0] * d;
  }
  set_rotation(&p, norm, rotation);
  return status_of(launch_norm_rope_bwd(p, st));
}

fa4fp4_status fa4bf16_cross_fwd(const fa4fp4_heads* q, const fa4fp4_heads* k, const fa4fp4_heads* v,
                                const int* kv_lens, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                                float softmax_scale, const fa4fp4_heads* o, float* lse, void* stream) {
  fa4fp4_status s = check_cross(B, Hq, Hkv, Nq, Nk, d);
  if (s != FA4FP4_OK) return s;
  if (B == 0 || Hq == 0 || Nq == 0) return FA4FP4_OK;
  CrossParams p;
  memset(&p, 0, sizeof(p));
  if ((s = check_heads(q, B, Hq, Nq, 2, false)) != FA4FP4_OK) return s;
  if ((s = check_heads(o, B, Hq, Nq, 2, true)) != FA4FP4_OK) return s;
  if (Nk > 0) {
    if ((s = check_heads(k, B, Hkv, Nk, 2, false)) != FA4FP4_OK) return s;
    if ((s = check_heads(v, B, Hkv, Nk, 2, false)) != FA4FP4_OK) return s;
    p.k = strided(k, B, Hkv, Nk);
    p.v = strided(v, B, Hkv, Nk);
  }
  if (!aligned(kv_lens, 4) || !aligned(lse, 16)) return FA4FP4_ERR_ALIGNMENT;
  p.q = strided(q, B, Hq, Nq);
  p.o = strided(o, B, Hq, Nq);
  if ((s = check_rows(p.q, Nq, d)) != FA4FP4_OK || (s = check_rows(p.k, Nk, d)) != FA4FP4_OK ||
      (s = check_rows(p.v, Nk, d)) != FA4FP4_OK)
    return s;
  p.lse = lse;
  p.lens = kv_lens;
  p.err = device_error_word();
  if (!p.err) return FA4FP4_ERR_CUDA;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Nq = Nq; p.Nk = Nk; p.d = d;
  p.scale = softmax_scale_of(softmax_scale, d);
  p.c = (float)((double)p.scale * 1.4426950408889634);
  while ((1LL << p.keys_log2) < Nk) ++p.keys_log2;
  return status_of((cross_few_rows(p) ? launch_cross_token : launch_cross_fwd)(p, static_cast<cudaStream_t>(stream)));
}

size_t fa4bf16_cross_bwd_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (check_cross(B, Hq, Hkv, Nq, Nk, d) != FA4FP4_OK || B == 0 || Hq == 0) return 0;
  return cross_bwd_workspace(B, Hq, Hkv, Nq, Nk, d);
}

fa4fp4_status fa4bf16_cross_bwd(const fa4fp4_heads* q, const fa4fp4_heads* k, const fa4fp4_heads* v,
                                const fa4fp4_heads* o, const fa4fp4_heads* dout, const float* lse,
                                const int* kv_lens, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                                float softmax_scale, const fa4fp4_heads* dq, const fa4fp4_heads* dk,
                                const fa4fp4_heads* dv, void* workspace, size_t workspace_bytes, void* stream) {
  fa4fp4_status s = check_cross(B, Hq, Hkv, Nq, Nk, d);
  if (s != FA4FP4_OK) return s;
  if (Hq == 0) Nq = 0;                   // no queries: zeros for dk and dv
  if (B == 0 || (Nq == 0 && (Nk == 0 || Hkv == 0))) return FA4FP4_OK;
  CrossParams p;
  memset(&p, 0, sizeof(p));
  if (Nq > 0) {
    const fa4fp4_heads* in[] = {q, o, dout};
    Strided* to[] = {&p.q, &p.o, &p.dout};
    for (int i = 0; i < 3; ++i) {
      if ((s = check_heads(in[i], B, Hq, Nq, 2, false)) != FA4FP4_OK) return s;
      *to[i] = strided(in[i], B, Hq, Nq);
    }
    if ((s = check_heads(dq, B, Hq, Nq, 2, true)) != FA4FP4_OK) return s;
    p.dq = strided(dq, B, Hq, Nq);
    if (!lse) return FA4FP4_ERR_INVALID_ARG;
    if ((s = check_rows(p.q, Nq, d)) != FA4FP4_OK || (s = check_rows(p.dout, Nq, d)) != FA4FP4_OK ||
        (s = check_rows(p.o, Nq, d)) != FA4FP4_OK || (s = check_rows(p.dq, Nq, d)) != FA4FP4_OK)
      return s;
  }
  if (Nk > 0) {
    const fa4fp4_heads* in[] = {k, v, dk, dv};
    Strided* to[] = {&p.k, &p.v, &p.dk, &p.dv};
    for (int i = 0; i < 4; ++i) {
      if ((s = check_heads(in[i], B, Hkv, Nk, 2, i >= 2)) != FA4FP4_OK) return s;
      *to[i] = strided(in[i], B, Hkv, Nk);
    }
    for (const Strided* t : to)
      if ((s = check_rows(*t, Nk, d)) != FA4FP4_OK) return s;
  }
  if (!aligned(kv_lens, 4) || !aligned(lse, 16)) return FA4FP4_ERR_ALIGNMENT;
  const size_t need = cross_bwd_workspace(B, Hq, Hkv, Nq, Nk, d);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA4FP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FA4FP4_ERR_ALIGNMENT;
  p.work = static_cast<uint8_t*>(workspace);
  p.lse = const_cast<float*>(lse);
  p.lens = kv_lens;
  p.err = device_error_word();
  if (!p.err) return FA4FP4_ERR_CUDA;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Nq = Nq; p.Nk = Nk; p.d = d;
  p.scale = softmax_scale_of(softmax_scale, d);
  p.c = (float)((double)p.scale * 1.4426950408889634);
  return status_of(launch_cross_bwd(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
