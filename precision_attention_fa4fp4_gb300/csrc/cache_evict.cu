// cache_evict.cu -- a sequence cut back to its heaviest and its newest tokens.
//
// Per sequence and kv head the `recent` newest tokens stay, and of the others
// the heaviest, `budget` in all, ties to the lowest position.  Two kernels: the
// first finds the cut among the weights by radix selection (one CTA per
// sequence and head, four passes over the weights) and writes the kept
// positions in ascending order with their weights; the second copies the
// tokens into fresh pages, one CTA per (page, head, K or V).
//
// Tokens of pages with different scales meet in one page, so the codes are
// fitted anew under the append's rule: X = the least integer >= -127 with every
// kept value <= 448 2^X.  A code's magnitude fixes that integer by itself, so
// no value is formed: X = max(X_src + e(code)), e(code) = the least e with
// e4m3(code) <= 448 2^e.  The codes then move by 2^(X_src - X), exact but for
// codes that become subnormal.  Bound by HBM: d bytes read and written per kept
// token, head and tensor, 4 bytes of weight read per token.
#include "cache.cuh"

namespace fa4 {
namespace {

constexpr int NT1 = 1024;

// Unsigned keys in the order of the weights; NaN lowest, -0 as 0.
FA4_DEV uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(NT1) cache_keep_kernel(const __grid_constant__ CacheEvictParams p) {
  __shared__ unsigned s_hist[256];
  __shared__ unsigned s_bin, s_rank;
  __shared__ int s_warp[2][NT1 / 32];
  const CacheView& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = cache_len(c, b);
  const int keep = min(len, p.budget);
  const int recent = min(p.recent, keep);
  const int n = len - recent;                      // tokens to rank
  const int k = keep - recent;                     // of which to keep
  const float* w = p.w + ((long long)b * c.Hkv + h) * c.max_pages * c.page;
  int* kept = p.kept + ((long long)b * c.Hkv + h) * p.budget;
  float* w_out = p.w_out ? p.w_out + ((long long)b * c.Hkv + h) * p.dst_pages * c.page : nullptr;
  if (h == 0 && threadIdx.x == 0) p.new_lens[b] = keep;

  uint32_t cut = 0;                                // keys above it stay, and `ties` of those on it
  unsigned ties = 0;
  if (k > 0 && k < n) {
    unsigned rank = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += NT1) s_hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = threadIdx.x; i < n; i += NT1) {
        const uint32_t key = weight_key(__ldg(w + i));
        if ((key & mask) == cut) atomicAdd(&s_hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        unsigned v[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) { v[i] = s_hist[255 - (lane * 8 + i)]; sum += v[i]; }
        unsigned inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const unsigned u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        unsigned before = inc - sum;
        if (before < rank && rank <= inc) {
          unsigned r = rank - before;
          int i = 0;
          while (i < 7 && r > v[i]) { r -= v[i]; ++i; }
          s_bin = 255 - (lane * 8 + i);
          s_rank = r;
        }
      }
      __syncthreads();
      cut |= s_bin << shift;
      rank = s_rank;
    }
    ties = rank;
  }
  const bool all = k >= n, none = k == 0;
  // ordered copy of what stays: positions above the cut, and the first `ties` on it
  int done = 0;
  unsigned seen = 0;
  for (int base = 0; base < len; base += NT1) {
    const int i = base + threadIdx.x;
    bool above = false, on = false;
    float x = 0.f;
    if (i < len) {
      x = __ldg(w + i);
      const uint32_t key = weight_key(x);
      above = i >= n || all || (!none && key > cut);
      on = !above && !none && key == cut;
    }
    const unsigned bo = __ballot_sync(0xffffffffu, on);
    if (lane == 0) s_warp[0][warp] = __popc(bo);
    __syncthreads();
    unsigned before = seen, sum = 0;
#pragma unroll
    for (int j = 0; j < NT1 / 32; ++j) {
      if (j < warp) before += s_warp[0][j];
      sum += s_warp[0][j];
    }
    const bool take = above || (on && before + __popc(bo & ((1u << lane) - 1u)) < ties);
    seen += sum;
    const unsigned bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[1][warp] = __popc(bt);
    __syncthreads();
    int at = done, cnt = 0;
#pragma unroll
    for (int j = 0; j < NT1 / 32; ++j) {
      if (j < warp) at += s_warp[1][j];
      cnt += s_warp[1][j];
    }
    at += __popc(bt & ((1u << lane) - 1u));
    if (take && at < p.budget) {
      kept[at] = i;
      if (w_out) w_out[at] = x;
    }
    done += cnt;
  }
  for (int i = keep + threadIdx.x; i < p.budget; i += NT1) kept[i] = -1;
  if (w_out)
    for (int i = keep + threadIdx.x; i < p.dst_pages * c.page; i += NT1) w_out[i] = 0.f;
}

constexpr int NT2 = 128;

FA4_DEV float pow2_any(int x) {                    // 2^x for x in [-247, 127]
  return x >= -126 ? exp2i(x) : (x >= -149 ? __uint_as_float(1u << (x + 149)) : 0.f);
}

// The least e with e4m3(code) <= 448 * 2^e for a magnitude 1..0x7e (448 =
// 1.75 * 2^8): normal codes E - 15, plus one above a significand of 1.75;
// subnormal codes m * 2^-9.
FA4_DEV int code_exp(uint32_t mag) {
  const int E = mag >> 3, m = mag & 7;
  return E ? E - 15 + (m == 7) : (31 - __clz(m)) - 17;
}

template <int D, int P>
__global__ void __launch_bounds__(NT2) cache_copy_kernel(const __grid_constant__ CacheEvictParams p) {
  constexpr int PARTS = D / 8;
  constexpr int TOK = NT2 / PARTS;
  constexpr int N = (P + TOK - 1) / TOK;
  __shared__ int s_x[NT2 / 32];
  __shared__ float s_lo[NT2 / 32][D], s_hi[NT2 / 32][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheView& c = p.c;
  const int h = blockIdx.y >> 1, isv = blockIdx.y & 1, b = blockIdx.z;
  const int keep = min(cache_len(c, b), p.budget);
  const int first = blockIdx.x * P;
  if (first >= keep) return;
  const int dst = __ldg(p.dst + (long long)b * p.dst_pages + blockIdx.x);
  if (dst < 0 || dst >= c.num_pages) {
    if (threadIdx.x == 0) atomicOr(c.err, FA4_DEVERR_INDEX);
    return;
  }
  const uint8_t* pool = isv ? c.v : c.k;
  const uint8_t* scales = isv ? c.vs : c.ks;
  const int* kept = p.kept + ((long long)b * c.Hkv + h) * p.budget + first;
  const int part = threadIdx.x % PARTS, tok = threadIdx.x / PARTS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint2 w[N];
  int xs[N];
  long long at[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = tok + i * TOK;
    at[i] = -1;
    if (s < P && first + s < keep) {
      const int src = kept[s];
      const int pg = cache_page(c, c.table, b, src / P);
      if (pg >= 0) at[i] = ((long long)pg * c.Hkv + h) * P + src % P;
    }
  }
  int X = -127;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = make_uint2(0, 0);
    xs[i] = 0;
    if (at[i] >= 0) {
      w[i] = __ldg(reinterpret_cast<const uint2*>(pool + at[i] * D + part * 8));
      xs[i] = (int)__ldg(scales + at[i] / P) - 127;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t a = __vmaxu4(w[i].x & 0x7f7f7f7fu, w[i].y & 0x7f7f7f7fu);
    const uint32_t e = __vmaxu4(a, a >> 16);
    const uint32_t mag = max(e & 0xffu, (e >> 8) & 0xffu);
    if (mag) X = max(X, xs[i] + code_exp(mag));
  }
  X = __reduce_max_sync(0xffffffffu, X);
  if (lane == 0) s_x[warp] = X;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT2 / 32; ++i) X = max(X, s_x[i]);

  const long long ph = (long long)dst * c.Hkv + h;
  uint8_t* codes = (isv ? c.v : c.k) + ph * P * D;
  float lo[8], hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) { lo[j] = 448.f; hi[j] = -448.f; }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = tok + i * TOK;
    if (s < P && first + s < keep) {
      uint2 e = w[i];
      float f[8];
      const uint32_t u[2] = {e.x, e.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t a = e4m3x2_to_f16x2(u[j]), z = e4m3x2_hi_to_f16x2(u[j]);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&z));
        f[4 * j] = x.x; f[4 * j + 1] = x.y; f[4 * j + 2] = y.x; f[4 * j + 3] = y.y;
      }
      if (xs[i] != X) {
        // zero codes may come from any exponent: keep the factor finite
        const float mv = pow2_any(min(xs[i] - X, 127));
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] == 0.f ? f[j] : f[j] * mv;
        e = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
        if (!isv) {
          const uint32_t r[2] = {e.x, e.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a = e4m3x2_to_f16x2(r[j]), z = e4m3x2_hi_to_f16x2(r[j]);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&z));
            f[4 * j] = x.x; f[4 * j + 1] = x.y; f[4 * j + 2] = y.x; f[4 * j + 3] = y.y;
          }
        }
      }
      *reinterpret_cast<uint2*>(codes + (long long)s * D + part * 8) = e;
#pragma unroll
      for (int j = 0; j < 8; ++j) { lo[j] = fminf(lo[j], f[j]); hi[j] = fmaxf(hi[j], f[j]); }
    }
  }
  if (threadIdx.x == 0) ((isv ? c.vs : c.ks) + ph)[0] = (uint8_t)(X + 127);
  if (isv) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int o = PARTS; o < 32; o *= 2) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
    }
  if (lane < PARTS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) { s_lo[warp][part * 8 + j] = lo[j]; s_hi[warp][part * 8 + j] = hi[j]; }
  }
  __syncthreads();
  if (threadIdx.x < 2 * PARTS) {
    const bool up = threadIdx.x >= PARTS;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = up ? -448.f : 448.f;
#pragma unroll
      for (int i = 0; i < NT2 / 32; ++i)
        f[j] = up ? fmaxf(f[j], s_hi[i][part * 8 + j]) : fminf(f[j], s_lo[i][part * 8 + j]);
    }
    *reinterpret_cast<uint2*>(c.kb + ph * 2 * D + (up ? D : 0) + part * 8) =
        make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
  }
}

template <int D, int P>
cudaError_t launch(const CacheEvictParams& p, cudaStream_t st) {
  cache_keep_kernel<<<dim3((unsigned)p.c.Hkv, (unsigned)p.c.B), NT1, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.budget + P - 1) / P), (unsigned)(2 * p.c.Hkv), (unsigned)p.c.B);
  cache_copy_kernel<D, P><<<grid, NT2, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams& p, cudaStream_t st) {
#define FA4_CASE(D, P) \
  if (p.c.d == D && p.c.page == P) return launch<D, P>(p, st);
  FA4_CASE(64, 16) FA4_CASE(64, 32) FA4_CASE(64, 64) FA4_CASE(64, 128)
  FA4_CASE(128, 16) FA4_CASE(128, 32) FA4_CASE(128, 64) FA4_CASE(128, 128)
#undef FA4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa4
