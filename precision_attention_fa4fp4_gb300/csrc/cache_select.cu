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
// per (sequence, kv head, token) first takes the bounds as FP32 sums and keeps,
// per page, the sum and a limit of its error (2 d + 1 bytes read a page); cuts
// the sums at the last one to take, by radix selection; and evaluates only the
// pages that the error leaves undecided in 64 bits: usually one or two.
//
// The sums are m16n8k16 products with 16 pages as rows, their codes as f16
// (exact) and the coefficients as two f16 columns, hi + 2^-11 lo: a tenth of the
// instructions of plain FP32 sums.  64 rows of 375 to 512 pages, heads of 128:
// 18.6 us alone (sums of plain FP32: 6.7 us more), bound by one CTA's chain:
// coefficients, bounds, the digits of the cut, the border.
//
// The intervals stay in shared memory (in the workspace where there are more
// than 16384 pages).
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NT = KTH_THREADS;
constexpr int SMEM_PAGES = 16384, MAX_PAGES = 1 << 18;    // (the call refuses more)

// Unsigned keys in the order of the floats (NaN above everything).
FA4_DEV uint32_t key32(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
FA4_DEV float key32_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
FA4_DEV unsigned long long key64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
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
  extern __shared__ __align__(16) uint32_t s_dyn[];
    __shared__ KthShared s_kth;
  __shared__ unsigned s_pre, s_rank, s_err;
  __shared__ double s_up[D], s_dn[D], s_score[MAX_BORDER];
  __shared__ __align__(16) float s_w[2 * D];       // dn against lo, up against hi
  __shared__ __align__(16) uint32_t s_b[2][D];
  __shared__ int s_page[MAX_BORDER];
  __shared__ int s_in, s_border;
  grid_start();
  grid_wait();
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
  // pages taken by words of 32, their prefix counts, then (here or in the
  // workspace) the sums with their errors
  uint32_t* s_bits = s_dyn;
  const int bit_words = (c.max_pages + 31) / 32;
  float2* score = c.max_pages <= SMEM_PAGES ? reinterpret_cast<float2*>(s_dyn + (bit_words + 1) / 2 * 4)
                                            : p.score + (long long)blockIdx.x * c.max_pages;
  for (int i = threadIdx.x; i < words; i += NT) s_bits[i] = 0;
  if (threadIdx.x == 0) { s_in = 0; s_border = 0; s_err = 0; }
  const int G = p.Hq / c.Hkv;
  // A warp sums up 16 pages at a time, lane (g, t4) reading 16-byte words of
  // pages g and g + 8; the first pages' bounds are on their way while the
  // coefficients are formed.
  const int g = lane / 4, t4 = lane % 4;
  int raw[2];
  uint4 x[2][D / 32];
  uint32_t sc[2];
  auto look = [&](int first) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int pi = first + g + 8 * r;
      raw[r] = pi < m ? c.table[(long long)b * c.max_pages + pi] : -1;
    }
  };
  auto load = [&](int first) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool in = raw[r] >= 0 && raw[r] < c.num_pages;
      if (!in && first + g + 8 * r < m) atomicOr(c.err, FA4_DEVERR_INDEX);
      const long long ph = in ? (long long)raw[r] * c.Hkv + h : 0;
      sc[r] = in ? c.ks[ph] : 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        x[r][i] = in ? *reinterpret_cast<const uint4*>(c.kb + ph * 2 * D + 64 * i + 16 * t4) : make_uint4(0, 0, 0, 0);
    }
  };
  if (k > 0) look(16 * warp);
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
    s_w[threadIdx.x] = fd;
    s_w[D + threadIdx.x] = fu;
  }
  if (k > 0) {
    load(16 * warp);
    __syncthreads();
    // the coefficients' largest magnitude and their sum of magnitudes
    uint32_t top = 0;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * D / 32; ++i) {
      const float x = fabsf(s_w[lane + 32 * i]);
      top = max(top, __float_as_uint(x));
      sum += x;
    }
    top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int E = (int)(top >> 23);
    const int e2 = (E == 0 || E == 255) ? 0 : max(-120, min(120, E - 134));
    // columns 0 and 1 of the B operand: hi and 2^11 lo, two coefficients a thread
    if (threadIdx.x < D) {
      const float2 w = *reinterpret_cast<const float2*>(&s_w[2 * threadIdx.x]);
      const float down = exp2i(-e2);
      const uint32_t hi = pack_f16x2(w.x * down, w.y * down);
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      s_b[0][threadIdx.x] = hi;
      s_b[1][threadIdx.x] = pack_f16x2((w.x * down - y.x) * 2048.f, (w.y * down - y.y) * 2048.f);
    }
    __syncthreads();
    // Error: a coefficient is off by G - 1 roundings and 2^-22 (and 2^-35 of the
    // largest, below 2^-36 of the sum per term); the products are exact and
    // 2 D of them are added with 2^-23 of the sum of magnitudes each, whatever
    // their order; doubled.  The sum of magnitudes is at most the largest code
    // times the coefficients'.
    const float rel = (float)(G + 2 * D + 16) * 0x1p-22f;
    for (int first = 16 * warp; first < m; first += 16 * (NT / 32)) {
      look(first + 16 * (NT / 32));
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
      MaxCode big[2];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t u[4] = {x[0][i].x, x[0][i].y, x[0][i].z, x[0][i].w};
        const uint32_t v[4] = {x[1][i].x, x[1][i].y, x[1][i].z, x[1][i].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // the sum runs in the order in which 16-byte words fall to the lanes
          uint2 wb = make_uint2(0, 0);
          if (g < 2) wb = *reinterpret_cast<const uint2*>(&s_b[g][32 * i + 8 * t4 + 2 * w]);
          mma_16816(w % 2 ? acc2 : acc, e4m3x2_to_f16x2(u[w]), e4m3x2_to_f16x2(v[w]), e4m3x2_hi_to_f16x2(u[w]),
                    e4m3x2_hi_to_f16x2(v[w]), wb.x, wb.y);
          big[0].add(u[w]);
          big[1].add(v[w]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t z = big[r].halves();
        z = max_u16x2(z, __shfl_xor_sync(0xffffffffu, z, 1));
        z = max_u16x2(z, __shfl_xor_sync(0xffffffffu, z, 2));
        z = MaxCode::of(z);
        const int pi = first + g + 8 * r;
        if (t4 == 0 && pi < m) {
          const float f = e8m0_value(sc[r]);
          const float err = __fmul_ru(__fmaf_ru(__fmul_ru(e4m3_value(z), sum), rel, 0x1p-120f), f);
          score[pi] = make_float2(
              fmaf(acc[2 * r + 1] + acc2[2 * r + 1], 0x1p-11f, acc[2 * r] + acc2[2 * r]) * exp2i(e2) * f, err);
          atomicMax(&s_err, __float_as_uint(err));
        }
      }
      if (first + 16 * (NT / 32) < m) load(first + 16 * (NT / 32));
    }
    __syncthreads();
    // the k-th largest sum, or a value that exactly k reach
    const Cut kth = kth_largest(s_kth, k, [&](auto f) {
      for (int i = threadIdx.x; i < m; i += NT) f(key32(score[i].x));
    });
    // With err the largest error: k pages have a bound of at least cut - err, so
    // a page is certainly out whose own is surely below; and at most k have one
    // above cut + err (the others' sums are at most cut), so a page is certainly
    // in whose own surely is.  Sums that are not finite decide nothing.
    const float cut = key32_value(kth.key), err = __uint_as_float(s_err);
    const float above = __fadd_ru(cut, err), below = __fsub_rd(cut, err);
    const bool sane = fabsf(above) <= 3.0e38f && fabsf(below) <= 3.0e38f;
    auto state = [&](int i) -> int {               // 1 in, -1 out, 0 undecided
      const float2 v = score[i];
      if (!sane || !(fabsf(v.x) <= 3.0e38f)) return 0;
      if (__fsub_rd(v.x, v.y) > above) return 1;
      return __fadd_ru(v.x, v.y) < below ? -1 : 0;
    };
    for (int i = threadIdx.x; i < m; i += NT) {
      const int z = state(i);
      if (z > 0) {
        atomicOr(&s_bits[i / 32], 1u << (i % 32));
        atomicAdd(&s_in, 1);
      } else if (z == 0) {
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
      for (int i = threadIdx.x; i < m; i += NT)
        if (state(i) == 0) atomicOr(&s_bits[i / 32], 1u << (i % 32));
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
        const bool border = state(i) == 0;
        const double s = border ? exact(i) : 0.;
        __syncwarp();
        // what is decided already is kept apart by a NaN
        if (lane == 0) wide[i] = border && s == s ? s : __longlong_as_double(-1ll);
      }
      __syncthreads();
      if (threadIdx.x == 0) s_rank = need;
      unsigned long long pre = 0;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += NT) s_kth.hist[i] = 0;
        __syncthreads();
        const unsigned long long mask = shift == 56 ? 0ull : ~0ull << (shift + 8);
        for (int i = threadIdx.x; i < m; i += NT) {
          const double v = wide[i];
          const unsigned long long key = key64(v);
          if (v == v && (key & mask) == pre) atomicAdd(&s_kth.hist[(unsigned)(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
          unsigned rank = s_rank, bin;
          find_bin(s_kth.hist, rank, bin);
          if (lane == 0) { s_rank = rank; s_pre = bin; }
        }
        __syncthreads();
        pre |= (unsigned long long)s_pre << shift;
      }
      // all above the cut, and of those on it the first s_rank
      const int ties = (int)s_rank;
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
  // the taken pages in ascending order: words' prefix, then a page a thread
  int* s_before = reinterpret_cast<int*>(s_bits + bit_words);
  if (warp == 0) {
    int done = 0;
    for (int base = 0; base < words; base += 32) {
      const int cnt = base + lane < words ? __popc(s_bits[base + lane]) : 0;
      int inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      if (base + lane < words) s_before[base + lane] = done + inc - cnt;
      done += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) s_in = done;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint32_t bits = s_bits[i / 32];
    const int at = s_before[i / 32] + __popc(bits & ((1u << (i % 32)) - 1u));
    if (((bits >> (i % 32)) & 1u) && at < p.n_sel) out[at] = i;
  }
  for (int i = s_in + threadIdx.x; i < p.n_sel; i += NT) out[i] = -1;
}

constexpr size_t smem_bytes(int max_pages) {
  const size_t bit_words = ((size_t)max_pages + 31) / 32;
  return (bit_words + 1) / 2 * 16 + (max_pages <= SMEM_PAGES ? (size_t)max_pages * 8 : 0);
}

template <int D>
cudaError_t launch(const CacheSelectParams& p, cudaStream_t st) {
  const size_t smem = smem_bytes(p.c.max_pages);
  if (smem > 32 * 1024) {
    // One limit for the kernel on a device, so every call sets the same (the most
    // that any needs): another thread's smaller one between here and the launch
    // would refuse it.
    constexpr size_t most = smem_bytes(SMEM_PAGES);
    static_assert(most >= smem_bytes(MAX_PAGES), "the limit covers the largest table");
    const cudaError_t e =
        cudaFuncSetAttribute(cache_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
  }
  return launch_next(cache_select_kernel<D>, dim3((unsigned)p.c.B * p.c.Hkv * p.T), NT, smem, st, p);
}

}  // namespace

size_t cache_select_workspace(int B, int Hkv, int T, int max_pages) {
  return max_pages <= SMEM_PAGES ? 0 : (size_t)B * Hkv * T * max_pages * sizeof(float2);
}

cudaError_t launch_cache_select(const CacheSelectParams& p, cudaStream_t st) {
  return p.c.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace fa4
