// cache.h -- host-side declarations of the 8-bit key/value cache kernels.  Not
// part of the ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa4 {

// A paged pool and the sequences that live in it.  Page `p`, head `h`: codes
// [page][d] at ((p * Hkv + h) * page) * d, one E8M0 scale byte at p * Hkv + h,
// the K bounds [2][d] (elementwise least and greatest code) at
// (p * Hkv + h) * 2 * d.
struct CacheView {
  uint8_t *k, *v, *ks, *vs, *kb;
  const int* table;      // [B][max_pages]
  const int* lens;       // [B]
  int num_pages, Hkv, page, d, B, max_pages;
  unsigned* err;
};

struct CacheAppendParams {
  CacheView c;
  const void *k, *v;     // bf16 [B][Hkv][T][d]
  const int* n_new;      // [B] or nullptr (T)
  int T;
};
cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t st);

// Rows of a TMA box of codes: a warp's 32 keys, or a page of 16.
inline int cache_box(int page) { return page < 32 ? page : 32; }

struct CacheFwdParams {
  CUtensorMap tm_k, tm_v;  // codes as rows of d bytes, boxes of cache_box(page) rows
  CacheView c;
  const void* q;         // bf16 [B][Hq][T][d]
  const int* q_lens;     // [B] or nullptr (T)
  const int* pages;      // [B][Hkv][T][n_sel] selected pages, or nullptr (all pages)
  void* o;
  float* lse;
  uint8_t* part;         // workspace: counter words, then split partials
  int Hq, T, n_sel, causal, out_bf16;
  float scale, c2;       // softmax scale, fl32(scale * log2 e)
};
// Workspace of the split forward; 0: more work than one call takes.
size_t cache_fwd_workspace(int B, int Hq, int Hkv, int T, int d, int n_sel, int page, int max_pages);
cudaError_t launch_cache_fwd(const CacheFwdParams& p, cudaStream_t st);
// The same for many rows, all pages and bf16 output, with a workspace of its own
// size.
size_t cache_chunk_workspace(int B, int Hq, int Hkv, int T, int d, int page, int max_pages);
cudaError_t launch_cache_chunk(const CacheFwdParams& p, cudaStream_t st);

struct CacheSelectParams {
  CacheView c;
  const void* q;
  const int* q_lens;
  int Hq, T, n_sel;
  float2* score;         // workspace [B][Hkv][T][max_pages]: FP32 bound and its error
                         // (unused where max_pages fits shared memory)
  int* out;              // [B][Hkv][T][n_sel]
};
size_t cache_select_workspace(int B, int Hkv, int T, int max_pages);
cudaError_t launch_cache_select(const CacheSelectParams& p, cudaStream_t st);

struct CacheWeighParams {
  CUtensorMap tm_k, tm_q;    // codes; the prepared rows (many rows only)
  CacheView c;
  uint8_t *rows, *metas;     // workspace: prepared rows, their constants
  const void* q;
  const float* lse;      // [B][Hq][T]
  const int* q_lens;
  const float* w_in;     // [B][Hkv][max_pages * page]
  float* w_out;
  int Hq, T, causal;
  float c2;
};
bool cache_weigh_fits(int B, int Hkv, int page, int max_pages);
cudaError_t launch_cache_weigh(const CacheWeighParams& p, cudaStream_t st);
// The same for many rows (query heads of a kv head x T), with a workspace.
// Keys x sequences, heads of 128, 8 kv heads, us by mma.sync / by tcgen05:
//   2048 x 16:  32 rows 25 / 42,  64 rows 34 / 42,  96 rows 49 / 42,  256 rows 106 / 48
//   8192 x 1:   32 rows 8 / 14,   64 rows 11 / 14,  96 rows 14 / 14,  256 rows 29 / 16
// heads of 64, 4096 x 16: 64 rows 49 / 58, 96 rows 68 / 58.
constexpr int WEIGH_MANY = 80;
size_t cache_weigh_rows_bytes(int B, int Hq, int Hkv, int T, int d, size_t* all);
cudaError_t launch_cache_weigh_rows(const CacheWeighParams& p, cudaStream_t st);

struct CacheEvictParams {
  CacheView c;
  const float* w;        // [B][Hkv][max_pages * page]
  const int* dst;        // [B][dst_pages]
  int dst_pages, budget, recent;
  int* new_lens;         // [B]
  int* kept;             // [B][Hkv][budget]
  float* w_out;          // [B][Hkv][dst_pages * page]
};
cudaError_t launch_cache_evict(const CacheEvictParams& p, cudaStream_t st);

// Tensor map of `rows` rows of `row_bytes` (64 or 128) bytes for boxes of
// box_rows whole rows, swizzled over their whole width.
bool make_rows_map(CUtensorMap* m, const void* base, int row_bytes, uint64_t rows, uint32_t box_rows);
// ... of f16 rows of d values, for boxes of 64 values x 128 rows.
bool make_f16_rows_map(CUtensorMap* m, const void* base, int d, uint64_t rows);
// The library's device error word on the current device (nullptr on failure).
unsigned* device_error_word();

}  // namespace fa4
