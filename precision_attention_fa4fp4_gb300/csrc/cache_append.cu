// cache_append.cu -- new K and V tokens into the paged 8-bit cache.
//
// One CTA per (sequence, touched page, head, K or V).  For the page's new
// tokens x of the head: X = the least integer >= -127 with max |x| <= 448 2^X,
// at least the page's exponent X_old when it already holds tokens; codes
// RNE(x 2^-X).  The rule saturates nothing (the OCP exponent would cut
// magnitudes in (448, 512) 2^X by up to 12.5 %: too much for a key that stays
// in the cache).  When X > X_old the older codes are moved to the new exponent,
// RNE(code 2^(X_old - X)): exact but for codes that become subnormal.
//
// The K bounds (elementwise least and greatest code of the page) need no look
// at the older codes: rounding to a coarser exponent is monotone, so the moved
// minimum is the minimum of the moved codes.  A token that joins a page thus
// reads its own 2 d bytes, a scale byte and 2 d bound bytes, and the older
// codes only in the rare step that raises the exponent.
//
// Bound by HBM for prompts (2 d bytes read, d written per token, head and
// tensor): 2 x 8192 tokens, 8 heads of 128, 19.7 us, 5.1 TB/s.  By latency for
// single tokens (launch; lens, table and scale one after the other; the token):
// 64 sequences, 8 heads of 128, 5.0 us.
#include "cache.cuh"

namespace fa4 {
namespace {

constexpr int NT = 128;

// Eight bf16 (one 16-byte word) to FP32.
FA4_DEV void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Eight E4M3 codes to FP32 values.
FA4_DEV void decode8(const uint2& w, float (&f)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = e4m3x2_to_f16x2(u[i]), hi = e4m3x2_hi_to_f16x2(u[i]);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[4 * i] = a.x; f[4 * i + 1] = a.y; f[4 * i + 2] = b.x; f[4 * i + 3] = b.y;
  }
}

FA4_DEV uint2 encode8(const float (&f)[8]) {
  return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// 2^x for x in [-254, 0]: the exact power, subnormal or zero where FP32 ends.
FA4_DEV float pow2_down(int x) {
  return x >= -126 ? exp2i(x) : (x >= -149 ? __uint_as_float(1u << (x + 149)) : 0.f);
}

template <int D, int P>
__global__ void __launch_bounds__(NT) cache_append_kernel(const __grid_constant__ CacheAppendParams p) {
  constexpr int PARTS = D / 8;                    // 16-byte words of a token
  constexpr int TOK = NT / PARTS;                 // tokens the CTA covers at once
  constexpr int N = (P + TOK - 1) / TOK;          // words a thread holds
  grid_start();
  grid_wait();
  const int h = blockIdx.y >> 1, isv = blockIdx.y & 1, b = blockIdx.z;
  const CacheView& c = p.c;
  const int len = cache_len(c, b);
  const int n = cache_count(p.n_new, b, p.T, c.err);
  const int lp = len / P + (int)blockIdx.x;       // the page, and what of it is new: [s0, s1)
  const long long first = (long long)lp * P;
  const int s0 = (int)max(0LL, (long long)len - first);
  const long long end = (long long)len + n - first;
  const int s1 = (int)min((long long)P, end);
  if (s1 <= s0) return;
  if (lp >= c.max_pages) {                        // no room in the table
    if (threadIdx.x == 0) atomicOr(c.err, FA4_DEVERR_INDEX);
    return;
  }
  const int page = cache_page(c, c.table, b, lp);
  if (page < 0) return;
  const long long ph = (long long)page * c.Hkv + h;
  uint8_t* codes = (isv ? c.v : c.k) + ph * P * D;
  uint8_t* scale = (isv ? c.vs : c.ks) + ph;
  const int part = threadIdx.x % PARTS, tok = threadIdx.x / PARTS;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(isv ? p.v : p.k) +
                             (((long long)b * c.Hkv + h) * p.T + (first - len)) * D + part * 8;

  const int X_old = s0 > 0 ? (int)*(scale) - 127 : -127;
  uint4 w[N];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = tok + i * TOK;
    w[i] = make_uint4(0, 0, 0, 0);
    if (s >= s0 && s < s1) w[i] = *(reinterpret_cast<const uint4*>(src + (long long)s * D));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
  }
  __shared__ uint32_t s_max[NT / 32];
  __shared__ float s_lo[NT / 32][D], s_hi[NT / 32][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) amax = max(amax, s_max[i]);
  if (amax >= 0x7f800000u) {
    // NaN or infinity among the new values: the cache holds finite codes only
    // (a code that a later query may not see must not reach it as 0 * NaN), so
    // NaN becomes 0, an infinity the largest finite code, neither counts for
    // the exponent, and the call is flagged.
    if (threadIdx.x == 0) atomicOr(c.err, FA4_DEVERR_NONFINITE);
    __syncthreads();
    amax = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t* u = reinterpret_cast<uint32_t*>(&w[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo = u[j] & 0xffffu, hi = u[j] >> 16;
        if ((lo & 0x7fffu) > 0x7f80u) lo = 0;
        if ((hi & 0x7fffu) > 0x7f80u) hi = 0;
        if ((lo & 0x7fffu) < 0x7f80u) amax = max(amax, (lo & 0x7fffu) << 16);
        if ((hi & 0x7fffu) < 0x7f80u) amax = max(amax, (hi & 0x7fffu) << 16);
        u[j] = lo | (hi << 16);
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) amax = max(amax, s_max[i]);
  }
  const int X = max(X_old, e4m3_p_block_exp(__uint_as_float(amax)));
  const float inv = exp2i(-X);                    // X in [-127, 120]
  const bool moved = s0 > 0 && X > X_old;

  float lo[8], hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) { lo[j] = 448.f; hi[j] = -448.f; }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = tok + i * TOK;
    if (s >= s0 && s < s1) {
      float f[8];
      unpack8(w[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= inv;
      const uint2 e = encode8(f);
      *reinterpret_cast<uint2*>(codes + (long long)s * D + part * 8) = e;
      if (!isv) {
        decode8(e, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) { lo[j] = fminf(lo[j], f[j]); hi[j] = fmaxf(hi[j], f[j]); }
      }
    }
  }
  const float mv = moved ? pow2_down(X_old - X) : 1.f;
  if (moved) {
#pragma unroll 1
    for (int s = tok; s < s0; s += TOK) {
      uint2* at = reinterpret_cast<uint2*>(codes + (long long)s * D + part * 8);
      float f[8];
      decode8(*at, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= mv;
      *at = encode8(f);
    }
  }
  if (threadIdx.x == 0) *scale = (uint8_t)(X + 127);
  if (isv) return;
  // bounds: lanes with the same part, then the warps, then the older tokens'
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
  uint8_t* kb = c.kb + ph * 2 * D;
  if (threadIdx.x < 2 * PARTS) {
    const bool up = threadIdx.x >= PARTS;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = up ? -448.f : 448.f;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i)
        f[j] = up ? fmaxf(f[j], s_hi[i][part * 8 + j]) : fminf(f[j], s_lo[i][part * 8 + j]);
    }
    uint2* at = reinterpret_cast<uint2*>(kb + (up ? D : 0) + part * 8);
    if (s0 > 0) {
      float o[8];
      decode8(*at, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= mv;
      const uint2 r = encode8(o);
      decode8(r, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = up ? fmaxf(f[j], o[j]) : fminf(f[j], o[j]);
    }
    *at = encode8(f);
  }
}

template <int D, int P>
cudaError_t launch(const CacheAppendParams& p, cudaStream_t st) {
  // T tokens behind any length touch at most (T + P - 2) / P + 1 pages
  const dim3 grid((unsigned)((p.T + P - 2) / P + 1), (unsigned)(2 * p.c.Hkv), (unsigned)p.c.B);
  return launch_next(cache_append_kernel<D, P>, grid, NT, 0, st, p);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t st) {
#define FA4_CASE(D, P) \
  if (p.c.d == D && p.c.page == P) return launch<D, P>(p, st);
  FA4_CASE(64, 16) FA4_CASE(64, 32) FA4_CASE(64, 64) FA4_CASE(64, 128)
  FA4_CASE(128, 16) FA4_CASE(128, 32) FA4_CASE(128, 64) FA4_CASE(128, 128)
#undef FA4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa4
