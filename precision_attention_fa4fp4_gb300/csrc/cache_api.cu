// cache_api.cu -- the C ABI of the 8-bit key/value cache: argument checks and
// launches.
#include <cmath>
#include <cstring>
#include "../../include/fa4fp4.h"
#include "cache.h"

using namespace fa4;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fa4fp4_status status_of(cudaError_t e) { return e == cudaSuccess ? FA4FP4_OK : FA4FP4_ERR_CUDA; }

// Shape of the cache and of the call; `Hq` = Hkv where the call has no queries.
fa4fp4_status check_shape(int num_pages, int Hkv, int page, int d, int B, int Hq, int T, int max_pages) {
  if (B < 0 || Hq < 0 || Hkv < 0 || T < 0 || num_pages < 1 || max_pages < 1) return FA4FP4_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA4FP4_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FA4FP4_ERR_UNSUPPORTED;
  if (Hkv == 0 ? Hq != 0 : Hq % Hkv != 0) return FA4FP4_ERR_UNSUPPORTED;
  // positions and grid dimensions stay within 32 and 16 bits
  if ((long long)max_pages * page > (1LL << 30) || T > (1 << 30) || B > 65535 || Hkv > 32767)
    return FA4FP4_ERR_UNSUPPORTED;
  if ((long long)Hq * T > (1LL << 31) - 1 || (long long)Hq * T * (B > 0 ? B : 1) > (1LL << 31) - 1)
    return FA4FP4_ERR_UNSUPPORTED;
  return FA4FP4_OK;
}

uint64_t pool_rows(const fa4fp4_cache* c) { return (uint64_t)c->num_pages * c->Hkv * c->page; }

fa4fp4_status check_call(const fa4fp4_cache* c, int B, int Hq, int T, int max_pages) {
  if (!c) return FA4FP4_ERR_INVALID_ARG;
  const fa4fp4_status s = check_shape(c->num_pages, c->Hkv, c->page, c->d, B, Hq, T, max_pages);
  // a pool row (d codes of one token and head) is a 32-bit TMA coordinate
  return s == FA4FP4_OK && pool_rows(c) >= (1ull << 31) ? FA4FP4_ERR_UNSUPPORTED : s;
}

// Pointers of the cache and of the sequences.
fa4fp4_status check_cache(const fa4fp4_cache* c, const int* table, const int* lens, const int* counts) {
  const void* ptrs[] = {c->k_codes, c->v_codes, c->k_scales, c->v_scales, c->k_bounds};
  for (const void* p : ptrs)
    if (!p) return FA4FP4_ERR_INVALID_ARG;
  if (!table || !lens) return FA4FP4_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return FA4FP4_ERR_ALIGNMENT;
  if (!aligned(table, 4) || !aligned(lens, 4) || (counts && !aligned(counts, 4))) return FA4FP4_ERR_ALIGNMENT;
  return FA4FP4_OK;
}

bool view(CacheView* v, const fa4fp4_cache* c, const int* table, const int* lens, int B, int max_pages) {
  v->k = static_cast<uint8_t*>(c->k_codes);
  v->v = static_cast<uint8_t*>(c->v_codes);
  v->ks = static_cast<uint8_t*>(c->k_scales);
  v->vs = static_cast<uint8_t*>(c->v_scales);
  v->kb = static_cast<uint8_t*>(c->k_bounds);
  v->table = table;
  v->lens = lens;
  v->num_pages = c->num_pages; v->Hkv = c->Hkv; v->page = c->page; v->d = c->d;
  v->B = B; v->max_pages = max_pages;
  v->err = device_error_word();
  return v->err != nullptr;
}

float softmax_scale_of(float s, int d) { return s > 0.f ? s : (float)(1.0 / std::sqrt((double)d)); }
float log2_scale(float s) { return (float)((double)s * 1.4426950408889634); }

}  // namespace

extern "C" {

fa4fp4_status fa4fp4_cache_append(const fa4fp4_cache* cache, const void* k, const void* v, const int* page_table,
                                  const int* lens, const int* n_new, int B, int max_pages, int T, void* stream) {
  fa4fp4_status s = check_call(cache, B, cache ? cache->Hkv : 0, T, max_pages);
  if (s != FA4FP4_OK) return s;
  if (B == 0 || cache->Hkv == 0 || T == 0) return FA4FP4_OK;
  if ((s = check_cache(cache, page_table, lens, n_new)) != FA4FP4_OK) return s;
  if (!k || !v) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return FA4FP4_ERR_ALIGNMENT;
  CacheAppendParams p;
  memset(&p, 0, sizeof(p));
  if (!view(&p.c, cache, page_table, lens, B, max_pages)) return FA4FP4_ERR_CUDA;
  p.k = k; p.v = v; p.n_new = n_new; p.T = T;
  return status_of(launch_cache_append(p, static_cast<cudaStream_t>(stream)));
}

size_t fa4fp4_cache_fwd_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int page, int max_pages, int n_sel) {
  if (check_shape(1, Hkv, page, d, B, Hq, T, max_pages) != FA4FP4_OK || n_sel < 0) return 0;
  if ((long long)n_sel * page > (1LL << 30)) return 0;
  if (B == 0 || Hq == 0 || T == 0) return 0;
  return cache_fwd_workspace(B, Hq, Hkv, T, d, n_sel, page, max_pages);
}

fa4fp4_status fa4fp4_cache_fwd(const fa4fp4_cache* cache, const void* q, const int* page_table, const int* lens,
                               const int* q_lens, const int* pages, int B, int Hq, int T, int max_pages, int n_sel,
                               float softmax_scale, int causal, void* o, int out_dtype, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (out_dtype != FA4FP4_OUT_F32 && out_dtype != FA4FP4_OUT_BF16) return FA4FP4_ERR_INVALID_ARG;
  fa4fp4_status s = check_call(cache, B, Hq, T, max_pages);
  if (s != FA4FP4_OK) return s;
  if (pages ? n_sel < 1 : n_sel != 0) return FA4FP4_ERR_INVALID_ARG;
  if ((long long)n_sel * cache->page > (1LL << 30)) return FA4FP4_ERR_UNSUPPORTED;
  if (B == 0 || Hq == 0 || T == 0) return FA4FP4_OK;
  if ((s = check_cache(cache, page_table, lens, q_lens)) != FA4FP4_OK) return s;
  if (!q || !o) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || (lse && !aligned(lse, 16)) || (pages && !aligned(pages, 4)))
    return FA4FP4_ERR_ALIGNMENT;
  const size_t need = cache_fwd_workspace(B, Hq, cache->Hkv, T, cache->d, n_sel, cache->page, max_pages);
  if (need == 0) return FA4FP4_ERR_UNSUPPORTED;       // 2^31 units of 128 keys and a row block, or more
  if (!workspace || workspace_bytes < need) return FA4FP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FA4FP4_ERR_ALIGNMENT;
  CacheFwdParams p;
  memset(&p, 0, sizeof(p));
  if (!view(&p.c, cache, page_table, lens, B, max_pages)) return FA4FP4_ERR_CUDA;
  p.q = q; p.q_lens = q_lens; p.pages = pages; p.o = o; p.lse = lse;
  p.part = static_cast<uint8_t*>(workspace);
  if (!make_rows_map(&p.tm_k, cache->k_codes, cache->d, pool_rows(cache), cache_box(cache->page)) ||
      !make_rows_map(&p.tm_v, cache->v_codes, cache->d, pool_rows(cache), cache_box(cache->page)))
    return FA4FP4_ERR_CUDA;
  p.Hq = Hq; p.T = T; p.n_sel = n_sel; p.causal = causal ? 1 : 0;
  p.out_bf16 = out_dtype == FA4FP4_OUT_BF16;
  p.scale = softmax_scale_of(softmax_scale, cache->d);
  p.c2 = log2_scale(p.scale);
  return status_of(launch_cache_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t fa4fp4_cache_select_workspace_bytes(int B, int Hkv, int T, int max_pages) {
  if (B < 0 || Hkv < 0 || T < 0 || max_pages < 1) return 0;
  return cache_select_workspace(B, Hkv, T, max_pages);
}

fa4fp4_status fa4fp4_cache_select(const fa4fp4_cache* cache, const void* q, const int* page_table, const int* lens,
                                  const int* q_lens, int B, int Hq, int T, int max_pages, int n_sel, int* pages,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  fa4fp4_status s = check_call(cache, B, Hq, T, max_pages);
  if (s != FA4FP4_OK) return s;
  if (n_sel < 1) return FA4FP4_ERR_INVALID_ARG;
  if (max_pages > (1 << 18)) return FA4FP4_ERR_UNSUPPORTED;   // one bit per page in shared memory
  if (B == 0 || Hq == 0 || T == 0) return FA4FP4_OK;
  if ((s = check_cache(cache, page_table, lens, q_lens)) != FA4FP4_OK) return s;
  if (!q || !pages) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(pages, 4)) return FA4FP4_ERR_ALIGNMENT;
  const size_t need = cache_select_workspace(B, cache->Hkv, T, max_pages);
  if (need && (!workspace || workspace_bytes < need)) return FA4FP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return FA4FP4_ERR_ALIGNMENT;
  CacheSelectParams p;
  memset(&p, 0, sizeof(p));
  if (!view(&p.c, cache, page_table, lens, B, max_pages)) return FA4FP4_ERR_CUDA;
  p.q = q; p.q_lens = q_lens; p.Hq = Hq; p.T = T; p.n_sel = n_sel;
  p.score = static_cast<float2*>(workspace);
  p.out = pages;
  return status_of(launch_cache_select(p, static_cast<cudaStream_t>(stream)));
}

size_t fa4fp4_cache_weigh_workspace_bytes(int B, int Hq, int Hkv, int T, int d) {
  if (check_shape(1, Hkv, 16, d, B, Hq, T, 1) != FA4FP4_OK || B == 0 || Hq == 0 || T == 0) return 0;
  if ((long long)(Hq / Hkv) * T < WEIGH_MANY) return 0;
  size_t all;
  cache_weigh_rows_bytes(B, Hq, Hkv, T, d, &all);
  return all;
}

fa4fp4_status fa4fp4_cache_weigh(const fa4fp4_cache* cache, const void* q, const float* lse, const int* page_table,
                                 const int* lens, const int* q_lens, int B, int Hq, int T, int max_pages,
                                 float softmax_scale, int causal, const float* weight_in, float* weight_out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  fa4fp4_status s = check_call(cache, B, Hq, T, max_pages);
  if (s != FA4FP4_OK) return s;
  if (B == 0 || Hq == 0 || T == 0) return FA4FP4_OK;
  if ((s = check_cache(cache, page_table, lens, q_lens)) != FA4FP4_OK) return s;
  if (!cache_weigh_fits(B, cache->Hkv, cache->page, max_pages)) return FA4FP4_ERR_UNSUPPORTED;
  if (!q || !lse || !weight_in || !weight_out) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(weight_in, 4) || !aligned(weight_out, 4))
    return FA4FP4_ERR_ALIGNMENT;
  const size_t need = fa4fp4_cache_weigh_workspace_bytes(B, Hq, cache->Hkv, T, cache->d);
  if (need && (!workspace || workspace_bytes < need)) return FA4FP4_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return FA4FP4_ERR_ALIGNMENT;
  // a prepared row is a 32-bit TMA coordinate
  if (need / (2 * (size_t)cache->d) >= (1ull << 31)) return FA4FP4_ERR_UNSUPPORTED;
  CacheWeighParams p;
  memset(&p, 0, sizeof(p));
  if (!view(&p.c, cache, page_table, lens, B, max_pages)) return FA4FP4_ERR_CUDA;
  if (need) {
    size_t all;
    p.rows = static_cast<uint8_t*>(workspace);
    const size_t rows = cache_weigh_rows_bytes(B, Hq, cache->Hkv, T, cache->d, &all);
    p.metas = p.rows + rows;
    if (!make_f16_rows_map(&p.tm_q, p.rows, cache->d, rows / (2 * (size_t)cache->d))) return FA4FP4_ERR_CUDA;
  } else if (!make_rows_map(&p.tm_k, cache->k_codes, cache->d, pool_rows(cache), cache_box(cache->page))) {
    return FA4FP4_ERR_CUDA;
  }
  p.q = q; p.lse = lse; p.q_lens = q_lens; p.w_in = weight_in; p.w_out = weight_out;
  p.Hq = Hq; p.T = T; p.causal = causal ? 1 : 0;
  p.c2 = log2_scale(softmax_scale_of(softmax_scale, cache->d));
  return status_of(launch_cache_weigh(p, static_cast<cudaStream_t>(stream)));
}

fa4fp4_status fa4fp4_cache_evict(const fa4fp4_cache* cache, const int* page_table, const int* lens,
                                 const float* weight, const int* dst_table, int B, int max_pages, int dst_pages,
                                 int budget, int recent, int* new_lens, int* kept, float* weight_out, void* stream) {
  fa4fp4_status s = check_call(cache, B, cache ? cache->Hkv : 0, 1, max_pages);
  if (s != FA4FP4_OK) return s;
  if (dst_pages < 1 || budget < 1 || recent < 0 || recent > budget) return FA4FP4_ERR_INVALID_ARG;
  if ((long long)dst_pages * cache->page > (1LL << 30)) return FA4FP4_ERR_UNSUPPORTED;
  if (budget > (long long)dst_pages * cache->page) return FA4FP4_ERR_INVALID_ARG;
  if (B == 0 || cache->Hkv == 0) return FA4FP4_OK;
  if ((s = check_cache(cache, page_table, lens, nullptr)) != FA4FP4_OK) return s;
  if (!weight || !dst_table || !new_lens || !kept) return FA4FP4_ERR_INVALID_ARG;
  if (!aligned(weight, 4) || !aligned(dst_table, 4) || !aligned(new_lens, 4) || !aligned(kept, 4) ||
      (weight_out && !aligned(weight_out, 4)))
    return FA4FP4_ERR_ALIGNMENT;
  CacheEvictParams p;
  memset(&p, 0, sizeof(p));
  if (!view(&p.c, cache, page_table, lens, B, max_pages)) return FA4FP4_ERR_CUDA;
  p.w = weight; p.dst = dst_table; p.dst_pages = dst_pages; p.budget = budget; p.recent = recent;
  p.new_lens = new_lens; p.kept = kept; p.w_out = weight_out;
  return status_of(launch_cache_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
