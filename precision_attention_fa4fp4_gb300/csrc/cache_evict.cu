// cache_evict.cu -- a sequence cut back to its heaviest and its newest tokens.
//
// Per sequence and kv head the `recent` newest tokens stay, and of the others
// the heaviest, `budget` in all, ties to the lowest position.  Two kernels: the
// first finds the cut among the weights (one CTA per sequence and head, the
// weights in registers while there are at most 32768) and writes the kept
// positions in ascending order with their weights; the second copies the tokens
// into fresh pages, one CTA per (page, head).
//
// Tokens of pages with different scales meet in one page, so the codes are
// fitted anew under the append's rule: X = the least integer >= -127 with every
// kept value <= 448 2^X.  A code's magnitude fixes that integer by itself, so
// no value is formed: X = max(X_src + e(code)), e(code) = the least e with
// e4m3(code) <= 448 2^e.  The codes then move by 2^(X_src - X), exact but for
// codes that become subnormal.
//
// HBM is the floor: d bytes read and written per kept token, head and tensor, 4
// bytes of weight read per token.  16 sequences of 4001..8192 tokens to 4096, 8
// heads of 128: 11 us of selection (its passes over the keys' bits, one after
// the other) and 51 us of copy, 5.3 TB/s: instructions, most of them for the
// exponents and the K bounds, keep it from more.  One of 4096 to 1000: 10.9 us.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NT1 = KTH_THREADS;

// Unsigned keys in the order of the weights; NaN lowest, -0 as 0.
FA4_DEV uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int WARPS1 = NT1 / 32;

// Exclusive prefix over the CTA, in the order (chunk, thread), of flags: chunk
// j's of this thread is bit j of `flags`; at(j) is what add() gets.  s_cnt has
// EPT * 32 entries, s_tot 32.  Returns the total.
template <int EPT, class F>
FA4_DEV int block_places(uint32_t flags, int* s_cnt, int* s_tot, F add) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const unsigned v = __ballot_sync(0xffffffffu, (flags >> j) & 1u);
    if (lane == 0) s_cnt[j * WARPS1 + warp] = __popc(v);
  }
  __syncthreads();
  if (warp < EPT) {                                // chunk `warp`: prefix over its warps
    const int v = s_cnt[warp * WARPS1 + lane];
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    s_cnt[warp * WARPS1 + lane] = inc - v;
    if (lane == 31) s_tot[warp] = inc;
  }
  __syncthreads();
  const int v = lane < EPT ? s_tot[lane] : 0;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  const int before = inc - v;
#pragma unroll
  for (int j = 0; j < EPT; ++j) {
    const int base = __shfl_sync(0xffffffffu, before, j) + s_cnt[j * WARPS1 + warp];
    const unsigned all = __ballot_sync(0xffffffffu, (flags >> j) & 1u);
    add(j, base + __popc(all & ((1u << lane) - 1u)));
  }
  return __shfl_sync(0xffffffffu, inc, 31);
}

// EPT chunks of NT1 weights at a time; all of them at once (and kept) if ONCE.
template <int EPT, bool ONCE>
__global__ void __launch_bounds__(NT1) cache_keep_kernel(const __grid_constant__ CacheEvictParams p) {
  __shared__ KthShared s_kth;
  __shared__ int s_cnt[EPT * WARPS1], s_tot[32];
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y;
  const int len = cache_len(c, b);
  const int keep = min(len, p.budget);
  const int recent = min(p.recent, keep);
  const int n = len - recent;                      // tokens to rank
  const int k = keep - recent;                     // of which to keep
  const float* w = p.w + ((long long)b * c.Hkv + h) * c.max_pages * c.page;
  int* kept = p.kept + ((long long)b * c.Hkv + h) * p.budget;
  float* w_out = p.w_out ? p.w_out + ((long long)b * c.Hkv + h) * p.dst_pages * c.page : nullptr;

  float x[EPT];
  auto load = [&](int base) {
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const int i = base + j * NT1 + threadIdx.x;
      x[j] = i < len ? *(w + i) : 0.f;
    }
  };
  if (ONCE) load(0);
  uint32_t cut = 0;                                // keys above it stay, and `ties` of those on it
  unsigned ties = 0;
  bool all_ties = true;                            // all of those on it
  if (k > 0 && k < n) {
    const Cut r = kth_largest(s_kth, (unsigned)k, [&](auto f) {
      for (int base = 0; base < n; base += EPT * NT1) {
        if (!ONCE) load(base);
#pragma unroll
        for (int j = 0; j < EPT; ++j)
          if (base + j * NT1 + (int)threadIdx.x < n) f(weight_key(x[j]));
      }
    });
    cut = r.key;
    ties = r.ties;
    all_ties = r.all;
  }
  const bool all = k >= n, none = k == 0;
  int done = 0, seen = 0;
  for (int base = 0; base < len; base += EPT * NT1) {
    if (!ONCE) load(base);
    uint32_t take = 0, on = 0;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const int i = base + j * NT1 + threadIdx.x;
      if (i < len) {
        const uint32_t key = weight_key(x[j]);
        if (i >= n || all || (!none && key > cut)) take |= 1u << j;
        else if (!none && key == cut) on |= 1u << j;
      }
    }
    if (all_ties) take |= on;
    else {
      uint32_t more = 0;
      seen += block_places<EPT>(on, s_cnt, s_tot, [&](int j, int place) {
        if (((on >> j) & 1u) && seen + place < (int)ties) more |= 1u << j;
      });
      take |= more;
    }
    done += block_places<EPT>(take, s_cnt, s_tot, [&](int j, int place) {
      if (((take >> j) & 1u) && done + place < p.budget) {
        kept[done + place] = base + j * NT1 + threadIdx.x;
        if (w_out) w_out[done + place] = x[j];
      }
    });
  }
  for (int i = keep + threadIdx.x; i < p.budget; i += NT1) kept[i] = -1;
  if (w_out)
    for (int i = keep + threadIdx.x; i < p.dst_pages * c.page; i += NT1) w_out[i] = 0.f;
}

constexpr int NT2 = 128;

// Four codes times a power of two, rounded to nearest even (0 stays 0 whatever
// the factor).
FA4_DEV uint32_t e4m3_times(uint32_t x, float f) {
  const uint32_t a = e4m3x2_to_f16x2(x), z = e4m3x2_hi_to_f16x2(x);
  const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&z));
  return pack_e4m3x4(u.x * f, u.y * f, v.x * f, v.y * f);
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
  constexpr int PARTS = D / 16;                    // 16-byte words of a token
  constexpr int TOK = NT2 / PARTS;                 // tokens at once
  constexpr int N = (P + TOK - 1) / TOK;
  __shared__ int s_x[2][NT2 / 32];
  __shared__ uint4 s_lo[NT2 / 32][PARTS], s_hi[NT2 / 32][PARTS];
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int keep = min(cache_len(c, b), p.budget);
  // here, where a length already cut back gives the same: new_lens may be lens, and
  // the first kernel's CTAs need the old ones
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.new_lens[b] = keep;
  const int first = blockIdx.x * P;
  if (first >= keep) return;
  const int dst = *(p.dst + (long long)b * p.dst_pages + blockIdx.x);
  if (dst < 0 || dst >= c.num_pages) {
    if (threadIdx.x == 0) atomicOr(c.err, FA4_DEVERR_INDEX);
    return;
  }
  const int* kept = p.kept + ((long long)b * c.Hkv + h) * p.budget + first;
  const int part = threadIdx.x % PARTS, tok = threadIdx.x / PARTS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int src[N], row[N];                              // position; pool row of it (-1: none)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = tok + i * TOK;
    src[i] = s < P && first + s < keep ? kept[s] : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    row[i] = -1;
    if (src[i] >= 0) {
      const int pg = cache_page(c, c.table, b, src[i] / P);
      if (pg >= 0) row[i] = (pg * c.Hkv + h) * P + src[i] % P;
    }
  }
  uint4 w[2][N];
  int xs[2][N];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[kv][i] = make_uint4(0, 0, 0, 0);
      xs[kv][i] = 0;
      if (row[i] >= 0) {
        w[kv][i] = *(reinterpret_cast<const uint4*>((kv ? c.v : c.k) + (long long)row[i] * D) + part);
        xs[kv][i] = (int)*((kv ? c.vs : c.ks) + row[i] / P) - 127;
      }
    }
  int X[2] = {-127, -127};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 x = w[kv][i];
      MaxCode most;
      most.add(x.x); most.add(x.y); most.add(x.z); most.add(x.w);
      const uint32_t mag = MaxCode::of(most.halves());
      if (mag) X[kv] = max(X[kv], xs[kv][i] + code_exp(mag));
    }
    X[kv] = __reduce_max_sync(0xffffffffu, X[kv]);
    if (lane == 0) s_x[kv][warp] = X[kv];
  }
  __syncthreads();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < NT2 / 32; ++i) X[kv] = max(X[kv], s_x[kv][i]);

  const long long ph = (long long)dst * c.Hkv + h;
  // odd bytes, then even ones in the odd place
  uint32_t lo2[2][4], hi2[2][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) { lo2[j / 4][j % 4] = 0xffffffffu; hi2[j / 4][j % 4] = 0u; }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint4* to = reinterpret_cast<uint4*>((kv ? c.v : c.k) + ph * P * D) + part;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (src[i] < 0) continue;
      uint4 x = w[kv][i];
      if (xs[kv][i] != X[kv]) {
        const float f = pow2_any(min(xs[kv][i] - X[kv], 127));
        x = make_uint4(e4m3_times(x.x, f), e4m3_times(x.y, f), e4m3_times(x.z, f), e4m3_times(x.w, f));
      }
      to[(tok + i * TOK) * PARTS] = x;
      if (kv == 0) {
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t o = e4m3_ordered(u[j]);
          lo2[0][j] = min_u16x2(lo2[0][j], o);
          hi2[0][j] = max_u16x2(hi2[0][j], o);
          lo2[1][j] = min_u16x2(lo2[1][j], o << 8);
          hi2[1][j] = max_u16x2(hi2[1][j], o << 8);
        }
      }
    }
  }
  if (threadIdx.x < 2) (threadIdx.x ? c.vs : c.ks)[ph] = (uint8_t)(X[threadIdx.x] + 127);
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = (lo2[0][j] & 0xff00ff00u) | ((lo2[1][j] >> 8) & 0x00ff00ffu);
    hi[j] = (hi2[0][j] & 0xff00ff00u) | ((hi2[1][j] >> 8) & 0x00ff00ffu);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int o = PARTS; o < 32; o *= 2) {
      lo[j] = __vminu4(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
      hi[j] = __vmaxu4(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
    }
  if (lane < PARTS) {
    s_lo[warp][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    s_hi[warp][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  __syncthreads();
  if (threadIdx.x < 2 * PARTS) {
    const bool up = threadIdx.x >= PARTS;
    uint4 r = up ? s_hi[0][part] : s_lo[0][part];
#pragma unroll
    for (int i = 1; i < NT2 / 32; ++i) {
      const uint4 y = up ? s_hi[i][part] : s_lo[i][part];
      r.x = up ? __vmaxu4(r.x, y.x) : __vminu4(r.x, y.x);
      r.y = up ? __vmaxu4(r.y, y.y) : __vminu4(r.y, y.y);
      r.z = up ? __vmaxu4(r.z, y.z) : __vminu4(r.z, y.z);
      r.w = up ? __vmaxu4(r.w, y.w) : __vminu4(r.w, y.w);
    }
    reinterpret_cast<uint4*>(c.kb + ph * 2 * D + (up ? D : 0))[part] =
        make_uint4(e4m3_unordered(r.x), e4m3_unordered(r.y), e4m3_unordered(r.z), e4m3_unordered(r.w));
  }
}

template <int D, int P>
cudaError_t launch(const CacheEvictParams& p, cudaStream_t st) {
  const long long cap = (long long)p.c.max_pages * p.c.page;
  const dim3 rows((unsigned)p.c.Hkv, (unsigned)p.c.B);
  auto keep = cap <= 8 * NT1 ? cache_keep_kernel<8, true>
              : cap <= 32 * NT1 ? cache_keep_kernel<32, true> : cache_keep_kernel<8, false>;
  const cudaError_t e = launch_next(keep, rows, NT1, 0, st, p);
  if (e != cudaSuccess) return e;
  const dim3 pages((unsigned)((p.budget + P - 1) / P), (unsigned)p.c.Hkv, (unsigned)p.c.B);
  return launch_next(cache_copy_kernel<D, P>, pages, NT2, 0, st, p);
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
