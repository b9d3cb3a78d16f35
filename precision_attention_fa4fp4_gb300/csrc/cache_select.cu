// cache_select.cu -- the pages whose keys could score highest for each query
// token and kv head.
//
// A page's K bounds lo, hi (elementwise least and greatest key) give
//   sum over heads, dims of max(q lo, q hi) = sum_dim up hi + dn lo,
//   up = sum_heads max(q, 0),  dn = sum_heads min(q, 0),
// an upper bound of q.k for every key of the page, summed over the query heads
// of the kv head: 2 d products a page, whatever the number of heads.  The page
// of the query's last visible key is always taken; of the others the highest
// bounds, ties to the lowest page.
//
// The result is a set of whole numbers, so it has to be the right one.  One CTA
// per (sequence, kv head, token) sums in FP32 and keeps, per page, the sum and a
// bound of its rounding error (2 d + 1 bytes read a page); finds the cut among
// the lower and the upper ends of these intervals by radix selection; and
// evaluates only the pages that the intervals leave undecided in 64 bits:
// usually one or two.  The intervals stay in shared memory (in the workspace
// where there are more than 16384 pages), so one launch does it all: the same
// work as two kernels, a wide one for the sums and one CTA a row for the cut,
// took 22 us on 64 rows of 512 pages, against 9 us.
#include "cache.cuh"

namespace fa4 {
namespace {

constexpr int NT = 512;
constexpr int SMEM_PAGES = 16384;

// Unsigned keys in the order of the floats (NaN above everything).
FA4_DEV uint32_t key32(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
FA4_DEV unsigned long long key64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

// The ends of a page's interval as keys; what is not finite is undecided.
FA4_DEV void ends(const float2 v, uint32_t& lo, uint32_t& hi) {
  if (!(fabsf(v.x) <= 3.0e38f) || !(v.y <= 3.0e38f)) { lo = 0; hi = 0xffffffffu; return; }
  lo = key32(__fsub_rd(v.x, v.y));
  hi = key32(__fadd_ru(v.x, v.y));
}

constexpr int MAX_BORDER = 256;

// In the histogram's 256 bins, from the top: the bin that holds the rank-th
// largest value (1 = largest); rank becomes its rank inside the bin.  Warp 0.
FA4_DEV void find_bin(const unsigned* hist, unsigned& rank, unsigned& bin) {
  const int lane = threadIdx.x % 32;
  unsigned v[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) { v[i] = hist[255 - (lane * 8 + i)]; sum += v[i]; }
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const unsigned u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  unsigned before = inc - sum;
  const bool mine = before < rank && rank <= inc;
  const unsigned r0 = rank;
  unsigned my_bin = 0, my_rank = 0;
  if (mine) {
    unsigned r = r0 - before;
    int i = 0;
    while (i < 7 && r > v[i]) { r -= v[i]; ++i; }
    my_bin = 255 - (lane * 8 + i);
    my_rank = r;
  }
  const unsigned who = __ballot_sync(0xffffffffu, mine);
  const int src = who ? __ffs(who) - 1 : 0;
  bin = __shfl_sync(0xffffffffu, my_bin, src);
  rank = __shfl_sync(0xffffffffu, my_rank, src);
}

template <int D>
__global__ void __launch_bounds__(NT) cache_select_kernel(const __grid_constant__ CacheSelectParams p) {
  constexpr int LN = D / 8;                        // lanes of a page: 16 bounds each
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ unsigned s_hist[2][256];
  __shared__ unsigned s_pre[2], s_rank[2];
  __shared__ double s_up[D], s_dn[D], s_score[MAX_BORDER];
  __shared__ __align__(16) float s_w[2][D];        // dn against lo, up against hi
  __shared__ int s_page[MAX_BORDER];
  __shared__ int s_in, s_border, s_warp[NT / 32];
  const CacheView& c = p.c;
  const int h = blockIdx.x / p.T % c.Hkv, t = blockIdx.x % p.T, b = blockIdx.x / (p.T * c.Hkv);
  int* out = p.out + (long long)blockIdx.x * p.n_sel;
  const int len = cache_len(c, b), q_len = cache_count(p.q_lens, b, p.T, c.err);
  const int vis = t < q_len ? max(0, min(len, len - q_len + t + 1)) : 0;
  const int n = (vis + c.page - 1) / c.page;       // pages that the token sees keys of
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (n <= p.n_sel) {
    for (int i = threadIdx.x; i < p.n_sel; i += NT) out[i] = i < n ? i : -1;
    return;
  }
  const int m = n - 1;                             // pages to rank
  const unsigned k = p.n_sel - 1;                  // of which to take; k < m
  const int words = (n + 31) / 32;
  // [words] pages taken, then (in shared memory or the workspace) the intervals
  uint32_t* s_bits = s_dyn;
  const int bit_words = (c.max_pages + 31) / 32;
  float2* score = c.max_pages <= SMEM_PAGES ? reinterpret_cast<float2*>(s_dyn + (bit_words + 3) / 4 * 4)
                                            : p.score + (long long)blockIdx.x * c.max_pages;
  for (int i = threadIdx.x; i < words; i += NT) s_bits[i] = 0;
  if (threadIdx.x == 0) { s_in = 0; s_border = 0; s_pre[0] = s_pre[1] = 0; s_rank[0] = k; s_rank[1] = k + 1; }
  const int G = p.Hq / c.Hkv;
  if (threadIdx.x < D) {
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) +
                             (((long long)b * p.Hq + h * G) * p.T + t) * D + threadIdx.x;
    double up = 0., dn = 0.;
    float fu = 0.f, fd = 0.f;
#pragma unroll 4
    for (int gg = 0; gg < G; ++gg) {
      const float x = __bfloat162float(q[(long long)gg * p.T * D]);
      fu += fmaxf(x, 0.f);
      fd += fminf(x, 0.f);
      up += (double)fmaxf(x, 0.f);
      dn += (double)fminf(x, 0.f);
    }
    s_up[threadIdx.x] = up;
    s_dn[threadIdx.x] = dn;
    s_w[0][threadIdx.x] = fd;
    s_w[1][threadIdx.x] = fu;
  }
  __syncthreads();
  if (k > 0) {
    // lanes 0 .. LN / 2 - 1 of a page hold lo [D], the others hi [D]
    const int ln = threadIdx.x % LN;
    float w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(&s_w[ln / (LN / 2)][ln % (LN / 2) * 16 + 4 * j]);
      w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
    }
    // At most G - 1 roundings of a coefficient, 17 of the products and sums and
    // 4 across the lanes, each 2^-24 of the sum of magnitudes (doubled for the
    // second-order terms and the magnitudes' own rounding), and 2 D underflows.
    const float rel = (float)(G + 24) * 0x1p-23f;
    constexpr int PER = NT / LN;                   // pages at once
    constexpr int ITER = 8;
    for (int first = 0; first < m; first += PER * ITER) {
      uint4 x[ITER];
      uint32_t sc[ITER];
      int pg[ITER];
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int pi = first + threadIdx.x / LN + i * PER;
        pg[i] = pi < m ? cache_page(c, c.table, b, pi) : -1;
      }
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        sc[i] = 0;
        if (pg[i] >= 0) {
          const long long ph = (long long)pg[i] * c.Hkv + h;
          x[i] = __ldg(reinterpret_cast<const uint4*>(c.kb + ph * 2 * D + 16 * ln));
          sc[i] = __ldg(c.ks + ph);
        }
      }
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float s = 0.f, a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y[2] = {e4m3x2_to_f16x2(u[j]), e4m3x2_hi_to_f16x2(u[j])};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
            s = fmaf(v.x, w[4 * j + 2 * e], s);
            s = fmaf(v.y, w[4 * j + 2 * e + 1], s);
            a = fmaf(fabsf(v.x), fabsf(w[4 * j + 2 * e]), a);
            a = fmaf(fabsf(v.y), fabsf(w[4 * j + 2 * e + 1]), a);
          }
        }
#pragma unroll
        for (int o = 1; o < LN; o *= 2) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          a += __shfl_xor_sync(0xffffffffu, a, o);
        }
        const int pi = first + threadIdx.x / LN + i * PER;
        if (ln == 0 && pi < m) {
          const float f = e8m0_value(sc[i]);
          score[pi] = make_float2(s * f, __fmul_ru(__fmaf_ru(a, rel, 0x1p-140f), f));
        }
      }
    }
    __syncthreads();
    // the k-th largest lower end and the (k + 1)-th largest upper end
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 512; i += NT) (&s_hist[0][0])[i] = 0;
      __syncthreads();
      const unsigned p0 = s_pre[0], p1 = s_pre[1];
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = threadIdx.x; i < m; i += NT) {
        uint32_t lo, hi;
        ends(score[i], lo, hi);
        if ((lo & mask) == p0) atomicAdd(&s_hist[0][(lo >> shift) & 255u], 1u);
        if ((hi & mask) == p1) atomicAdd(&s_hist[1][(hi >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp < 2) {
        unsigned rank = s_rank[warp], bin;
        find_bin(s_hist[warp], rank, bin);
        if (lane == 0) { s_rank[warp] = rank; s_pre[warp] |= bin << shift; }
      }
      __syncthreads();
    }
    const uint32_t cut_lo = s_pre[0], cut_hi = s_pre[1];
    // certainly in: the lower end above the (k + 1)-th largest upper end;
    // certainly out: the upper end below the k-th largest lower end
    for (int i = threadIdx.x; i < m; i += NT) {
      uint32_t lo, hi;
      ends(score[i], lo, hi);
      if (lo > cut_hi) {
        atomicOr(&s_bits[i / 32], 1u << (i % 32));
        atomicAdd(&s_in, 1);
      } else if (hi >= cut_lo) {
        const int at = atomicAdd(&s_border, 1);
        if (at < MAX_BORDER) s_page[at] = i;
      }
    }
    __syncthreads();
    const int need = (int)k - s_in, nb = s_border;
    // a page's bound in 64 bits, by a whole warp
    auto exact = [&](int i) -> double {
      const int pg = cache_page(c, c.table, b, i);
      double s = 0.;
      if (pg >= 0) {
        const long long ph = (long long)pg * c.Hkv + h;
        const uint8_t* kb = c.kb + ph * 2 * D;
        for (int d = lane; d < D; d += 32)
          s += s_up[d] * (double)e4m3_value(kb[D + d]) + s_dn[d] * (double)e4m3_value(kb[d]);
#pragma unroll
        for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        s = ldexp(s, (int)c.ks[ph] - 127);
      }
      return s == 0. ? 0. : s;
    };
    if (nb == need) {
      for (int i = threadIdx.x; i < m; i += NT) {
        uint32_t lo, hi;
        ends(score[i], lo, hi);
        if (!(lo > cut_hi) && hi >= cut_lo) atomicOr(&s_bits[i / 32], 1u << (i % 32));
      }
    } else if (nb <= MAX_BORDER) {
      for (int j = warp; j < nb; j += NT / 32) {
        const double s = exact(s_page[j]);
        if (lane == 0) s_score[j] = s;
      }
      __syncthreads();
      for (int j = threadIdx.x; j < nb; j += NT) {
        const unsigned long long mine = key64(s_score[j]);
        int rank = 0;
        for (int i = 0; i < nb; ++i) {
          const unsigned long long o = key64(s_score[i]);
          rank += o > mine || (o == mine && s_page[i] < s_page[j]);
        }
        if (rank < need) atomicOr(&s_bits[s_page[j] / 32], 1u << (s_page[j] % 32));
      }
    } else {
      // many undecided pages (equal pages): their 64-bit bounds take the place
      // of the FP32 pairs, and the need-th largest is found byte by byte
      double* wide = reinterpret_cast<double*>(score);
      for (int i = warp; i < m; i += NT / 32) {
        uint32_t lo, hi;
        ends(score[i], lo, hi);
        const bool border = !(lo > cut_hi) && hi >= cut_lo;
        const double s = border ? exact(i) : 0.;
        __syncwarp();
        // what is decided already is kept apart by a NaN
        if (lane == 0) wide[i] = border && s == s ? s : __longlong_as_double(-1ll);
      }
      __syncthreads();
      if (threadIdx.x == 0) s_rank[0] = need;
      unsigned long long pre = 0;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += NT) s_hist[0][i] = 0;
        __syncthreads();
        const unsigned long long mask = shift == 56 ? 0ull : ~0ull << (shift + 8);
        for (int i = threadIdx.x; i < m; i += NT) {
          const double v = wide[i];
          const unsigned long long key = key64(v);
          if (v == v && (key & mask) == pre) atomicAdd(&s_hist[0][(unsigned)(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
          unsigned rank = s_rank[0], bin;
          find_bin(s_hist[0], rank, bin);
          if (lane == 0) { s_rank[0] = rank; s_pre[0] = bin; }
        }
        __syncthreads();
        pre |= (unsigned long long)s_pre[0] << shift;
      }
      // all above the cut, and of those on it the first s_rank[0]
      const int ties = (int)s_rank[0];
      for (int i = threadIdx.x; i < m; i += NT)
        if (wide[i] == wide[i] && key64(wide[i]) > pre) atomicOr(&s_bits[i / 32], 1u << (i % 32));
      __syncthreads();
      if (warp == 0) {
        int taken = 0;
        for (int base = 0; base < m && taken < ties; base += 32) {
          const int i = base + lane;
          const bool on = i < m && wide[i] == wide[i] && key64(wide[i]) == pre;
          const unsigned all = __ballot_sync(0xffffffffu, on);
          const int rank = taken + __popc(all & ((1u << lane) - 1u));
          const unsigned take = __ballot_sync(0xffffffffu, on && rank < ties);
          if (lane == 0) s_bits[base / 32] |= take;
          taken += __popc(all);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) s_bits[m / 32] |= 1u << (m % 32);   // the query's own page
  __syncthreads();
  // the taken pages in ascending order
  int done = 0;
  for (int base = 0; base < words; base += NT) {
    const int i = base + threadIdx.x;
    uint32_t bits = i < words ? s_bits[i] : 0u;
    const int cnt = __popc(bits);
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int at = done + inc - cnt;
    int all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) at += s_warp[w];
      all += s_warp[w];
    }
    while (bits) {
      if (at < p.n_sel) out[at] = 32 * i + __ffs(bits) - 1;
      ++at;
      bits &= bits - 1;
    }
    done += all;
    __syncthreads();
  }
  for (int i = done + threadIdx.x; i < p.n_sel; i += NT) out[i] = -1;
}

template <int D>
cudaError_t launch(const CacheSelectParams& p, cudaStream_t st) {
  const int bit_words = (p.c.max_pages + 31) / 32;
  size_t smem = (size_t)(bit_words + 3) / 4 * 16;
  if (p.c.max_pages <= SMEM_PAGES) smem += (size_t)p.c.max_pages * 8;
  if (smem > 32 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(cache_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cache_select_kernel<D><<<(unsigned)p.c.B * p.c.Hkv * p.T, NT, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t cache_select_workspace(int B, int Hkv, int T, int max_pages) {
  return max_pages <= SMEM_PAGES ? 0 : (size_t)B * Hkv * T * max_pages * sizeof(float2);
}

cudaError_t launch_cache_select(const CacheSelectParams& p, cudaStream_t st) {
  return p.c.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace fa4
