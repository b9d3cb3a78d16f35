// rope.cu -- RMS norm of every head's row of q and k and its rotation by
// position, in one pass, and the gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps), n = x r w, and channel pair i = (a, b) turns
//   by th = position[axis(i)] f_i:  y_a = n_a cos th - n_b sin th,
//                                   y_b = n_b cos th + n_a sin th.
// Backward, with g the outputs' gradient turned by -th and u = g w:
//   dx = r (u - x r mean(u x r)),  dw = sum over all rows of g x r.
//
// Both are bound by HBM: 2 bytes in and 2 out per element forward, 2 + 2 (or 4
// for f32 gradients) in and 2 out backward.
//
// A row of d channels is held by d / 16 lanes, 16 channels each as two 16-byte
// words: the 8 first and the 8 second channels of 8 pairs (pairs (i, i + d/2)),
// or 8 neighbouring pairs, so a pair never leaves its lane and the row's sums are
// three (two) shuffles.  A warp works on one token: its lanes' 8 sines and
// cosines are taken once and serve every head of the token.
//
// Angles: f_i / 2 pi is held as a fraction of a turn in 64 bits; position times
// it modulo 2^64 is the exact remainder, whose upper 32 bits give th in [-pi,
// pi) within 2^-30, at position 10^6 as at 1 (an FP32 product is off by 0.03
// there).  The native sine and cosine are off by 2^-21 there, against bf16's 2^-9.
#include <cuda_bf16.h>
#include "common.cuh"
#include <type_traits>
#include "rope.h"

namespace fa4 {
namespace {

constexpr int WARPS = 8;

// Two 16-byte words of bf16 -> first and second channels of 8 pairs.
template <bool PAIRS>
FA4_DEV void unpack(const uint4& u, const uint4& v, float (&a)[8], float (&b)[8]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
    if (PAIRS) {
      a[i] = lo; b[i] = hi;
    } else {
      (i < 4 ? a : b)[(2 * i) & 7] = lo;
      (i < 4 ? a : b)[(2 * i + 1) & 7] = hi;
    }
  }
}

FA4_DEV uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

template <bool PAIRS>
FA4_DEV void pack(const float (&a)[8], const float (&b)[8], uint4& u, uint4& v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (PAIRS) w[i] = pack2(a[i], b[i]);
    else w[i] = i < 4 ? pack2(a[2 * i], a[2 * i + 1]) : pack2(b[2 * i - 8], b[2 * i - 7]);
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}

// Where a lane's two words of a row start, in channels.
template <int D, bool PAIRS>
FA4_DEV int word0(int l) { return PAIRS ? 16 * l : 8 * l; }
template <int D, bool PAIRS>
FA4_DEV int word1(int l) { return PAIRS ? 16 * l + 8 : D / 2 + 8 * l; }

// Sines and cosines of a lane's 8 pairs at one token.
FA4_DEV void angles(const RopeParams& p, const uint64_t* turn, const uint8_t* axis, int b, int n, int l, float (&c)[8],
                    float (&s)[8]) {
  if (!p.pos) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
    return;
  }
  const int* at = p.pos + b * p.pos_b + n;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t where = __ldg(at + (long long)axis[8 * l + i] * p.N);
    const int rest = (int)(((uint64_t)where * turn[8 * l + i]) >> 32);   // of a turn, times 2^32
    const float th = (float)rest * 1.46291807926715968e-9f;              // 2 pi / 2^32
    c[i] = __cosf(th);
    s[i] = __sinf(th);
  }
}

template <int LANES>
FA4_DEV float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a CTA needs of the rotation and the weights, in shared memory.
template <int D>
struct Tables {
  uint64_t turn[D / 2];
  uint8_t axis[D / 2];
  __align__(16) float w[2][D];

  __device__ void load(const RopeParams& p) {
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) { turn[i] = p.turn[i]; axis[i] = p.axis[i]; }
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
      const void* src = p.t[i / D].w;
      w[i / D][i % D] = !src ? 1.f
                        : p.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(src)[i % D])
                                   : static_cast<const float*>(src)[i % D];
    }
    __syncthreads();
  }
};


// U rows of a lane group are on their way at a time.
template <int D, bool PAIRS, int U>
__global__ void __launch_bounds__(WARPS * 32) norm_rope_kernel(const __grid_constant__ RopeParams p, int chunk, int nq,
                                                               int nk) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES;
  __shared__ Tables<D> tab;
  tab.load(p);
  const int lane = threadIdx.x % 32, l = lane % LANES, sub = lane / LANES;
  const int c0 = word0<D, PAIRS>(l), c1 = word1<D, PAIRS>(l);
  const long long tokens = (long long)p.B * p.N;
  const long long tasks = tokens * (nq + nk);
  for (long long task = (long long)blockIdx.x * WARPS + threadIdx.x / 32; task < tasks;
       task += (long long)gridDim.x * WARPS) {
    const int part = (int)(task / tokens);
    const long long m = task % tokens;
    const int b = (int)(m / p.N), n = (int)(m % p.N);
    const int t = part >= nq;
    const RopeTensor& T = p.t[t];
    const int h0 = (t ? part - nq : part) * chunk, h1 = min(T.H, h0 + chunk);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(T.x.p) + b * T.x.b + n * T.x.n;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(T.out.p) + b * T.out.b + n * T.out.n;
    float c[8], s[8];
    bool first = true;
    for (int h = h0 + sub; h - sub < h1; h += ROWS * U) {
      uint4 u[U], v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (h + i * ROWS < h1) {
          const __nv_bfloat16* row = x + (h + i * ROWS) * T.x.h;
          u[i] = *reinterpret_cast<const uint4*>(row + c0);
          v[i] = *reinterpret_cast<const uint4*>(row + c1);
        }
      }
      if (first) angles(p, tab.turn, tab.axis, b, n, l, c, s);
      first = false;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float fa[8], fb[8];
        unpack<PAIRS>(u[i], v[i], fa, fb);
        float r = 1.f;
        if (p.norm) {
          float q = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) q = fmaf(fa[j], fa[j], fmaf(fb[j], fb[j], q));
          r = rsqrtf(row_sum<LANES>(q) * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float na = fa[j] * r * tab.w[t][PAIRS ? c0 + 2 * j : c0 + j];
          const float nb = fb[j] * r * tab.w[t][PAIRS ? c0 + 2 * j + 1 : c1 + j];
          fa[j] = na * c[j] - nb * s[j];
          fb[j] = nb * c[j] + na * s[j];
        }
        if (h + i * ROWS < h1) {
          pack<PAIRS>(fa, fb, u[i], v[i]);
          __nv_bfloat16* row = y + (h + i * ROWS) * T.out.h;
          *reinterpret_cast<uint4*>(row + c0) = u[i];
          *reinterpret_cast<uint4*>(row + c1) = v[i];
        }
      }
    }
  }
}

// Gradients.  The CTAs [0, ctas[0]) work on q, the others on k; every lane adds
// its 16 channels of the weight's gradient over its tasks, the CTA joins them in
// a fixed order and leaves one row of partials.
template <int D, bool PAIRS, bool F32>
__global__ void __launch_bounds__(WARPS * 32) norm_rope_bwd_kernel(const __grid_constant__ RopeParams p, int chunk,
                                                                   int nq, int nk) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES;
  __shared__ Tables<D> tab;
  __shared__ float join[WARPS][D];
  tab.load(p);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % LANES, sub = lane / LANES;
  const int c0 = word0<D, PAIRS>(l), c1 = word1<D, PAIRS>(l);
  const int t = (int)blockIdx.x >= p.ctas[0];
  const int cta = t ? (int)blockIdx.x - p.ctas[0] : (int)blockIdx.x;
  const RopeTensor& T = p.t[t];
  const long long tokens = (long long)p.B * p.N;
  const long long tasks = tokens * (t ? nk : nq);
  float da[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) da[j] = db[j] = 0.f;
  for (long long task = (long long)cta * WARPS + warp; task < tasks; task += (long long)p.ctas[t] * WARPS) {
    const long long m = task % tokens;
    const int b = (int)(m / p.N), n = (int)(m % p.N);
    const int h0 = (int)(task / tokens) * chunk, h1 = min(T.H, h0 + chunk);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(T.x.p) + b * T.x.b + n * T.x.n;
    const long long dy = b * T.dy.b + n * T.dy.n;
    __nv_bfloat16* dx = static_cast<__nv_bfloat16*>(T.out.p) + b * T.out.b + n * T.out.n;
    float c[8], s[8];
    angles(p, tab.turn, tab.axis, b, n, l, c, s);
    for (int h = h0 + sub; h - sub < h1; h += ROWS) {
      const bool on = h < h1;
      uint4 u = make_uint4(0, 0, 0, 0), v = u;
      float ga[8], gb[8], fa[8], fb[8];
      if (on) {
        const __nv_bfloat16* row = x + h * T.x.h;
        u = *reinterpret_cast<const uint4*>(row + c0);
        v = *reinterpret_cast<const uint4*>(row + c1);
      }
      if (F32) {
        float4 g[4] = {};
        if (on) {
          const float* row = static_cast<const float*>(T.dy.p) + dy + h * T.dy.h;
          g[0] = *reinterpret_cast<const float4*>(row + c0);
          g[1] = *reinterpret_cast<const float4*>(row + c0 + 4);
          g[2] = *reinterpret_cast<const float4*>(row + c1);
          g[3] = *reinterpret_cast<const float4*>(row + c1 + 4);
        }
        const float f[16] = {g[0].x, g[0].y, g[0].z, g[0].w, g[1].x, g[1].y, g[1].z, g[1].w,
                             g[2].x, g[2].y, g[2].z, g[2].w, g[3].x, g[3].y, g[3].z, g[3].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ga[j] = PAIRS ? f[2 * j] : f[j];
          gb[j] = PAIRS ? f[2 * j + 1] : f[8 + j];
        }
      } else {
        uint4 gu = make_uint4(0, 0, 0, 0), gv = gu;
        if (on) {
          const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(T.dy.p) + dy + h * T.dy.h;
          gu = *reinterpret_cast<const uint4*>(row + c0);
          gv = *reinterpret_cast<const uint4*>(row + c1);
        }
        unpack<PAIRS>(gu, gv, ga, gb);
      }
      unpack<PAIRS>(u, v, fa, fb);
      float xx = 0.f, ux = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = ga[j] * c[j] + gb[j] * s[j], e = gb[j] * c[j] - ga[j] * s[j];
        ga[j] = a;
        gb[j] = e;
      }
      if (p.norm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wa = tab.w[t][PAIRS ? c0 + 2 * j : c0 + j], wb = tab.w[t][PAIRS ? c0 + 2 * j + 1 : c1 + j];
          xx = fmaf(fa[j], fa[j], fmaf(fb[j], fb[j], xx));
          ux = fmaf(ga[j] * wa, fa[j], fmaf(gb[j] * wb, fb[j], ux));
        }
        xx = row_sum<LANES>(xx);
        ux = row_sum<LANES>(ux);
        // rows that are not there add nothing (with eps = 0 their r is infinite)
        const float r = on ? rsqrtf(xx * (1.f / D) + p.eps) : 0.f;
        const float k = r * r * ux * (1.f / D);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wa = tab.w[t][PAIRS ? c0 + 2 * j : c0 + j], wb = tab.w[t][PAIRS ? c0 + 2 * j + 1 : c1 + j];
          da[j] = fmaf(ga[j], fa[j] * r, da[j]);
          db[j] = fmaf(gb[j], fb[j] * r, db[j]);
          ga[j] = r * (ga[j] * wa - fa[j] * k);
          gb[j] = r * (gb[j] * wb - fb[j] * k);
        }
      }
      if (on) {
        pack<PAIRS>(ga, gb, u, v);
        __nv_bfloat16* row = dx + h * T.out.h;
        *reinterpret_cast<uint4*>(row + c0) = u;
        *reinterpret_cast<uint4*>(row + c1) = v;
      }
    }
  }
  if (!T.dw) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = LANES; o < 32; o *= 2) {
      da[j] += __shfl_xor_sync(0xffffffffu, da[j], o);
      db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
    }
    if (sub == 0) {
      join[warp][PAIRS ? c0 + 2 * j : c0 + j] = da[j];
      join[warp][PAIRS ? c0 + 2 * j + 1 : c1 + j] = db[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += WARPS * 32) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += join[w][i];
    T.part[(long long)cta * D + i] = sum;
  }
}

// dw = sum of the CTAs' partials: one CTA per tensor and 32 channels.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const __grid_constant__ RopeParams p) {
  const int per = p.d / 32, t = blockIdx.x / per, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = (blockIdx.x % per) * 32 + lane;
  const RopeTensor& T = p.t[t];
  if (!T.dw) return;
  __shared__ float join[8][32];
  float sum = 0.f;
  for (int c = warp; c < p.ctas[t]; c += 8) sum += T.part[(long long)c * p.d + i];
  join[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += join[w][lane];
    T.dw[i] = sum;
  }
}

int sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

// Heads of a warp's task: all of a tensor's where there are tokens enough to fill
// the GPU with one warp each, else as few as one round of its lanes.
int chunk_of(long long tokens, int H, int rows) {
  const long long want = (long long)sms() * 16;
  if (H <= rows || tokens >= want) return H > 0 ? H : 1;
  const long long parts = (want + tokens - 1) / tokens;
  const long long rounds = (H + rows - 1) / rows;
  const long long per = (rounds + parts - 1) / parts;
  return (int)(per * rows);
}

int parts_of(int H, int chunk) { return (H + chunk - 1) / chunk; }

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t st) {
  const int rows = 32 / (p.d / 16);
  const long long tokens = (long long)p.B * p.N;
  const int chunk = chunk_of(tokens, p.t[0].H > p.t[1].H ? p.t[0].H : p.t[1].H, rows);
  const int nq = parts_of(p.t[0].H, chunk), nk = parts_of(p.t[1].H, chunk);
  const long long tasks = tokens * (nq + nk);
  const long long need = (tasks + WARPS - 1) / WARPS;
  const int grid = (int)(need < (1 << 30) ? need : (1 << 30));
  auto k = p.d == 128 ? (p.pairs ? norm_rope_kernel<128, true, 4> : norm_rope_kernel<128, false, 4>)
                      : (p.pairs ? norm_rope_kernel<64, true, 4> : norm_rope_kernel<64, false, 4>);
  k<<<grid, WARPS * 32, 0, st>>>(p, chunk, nq, nk);
  return cudaGetLastError();
}

void rope_bwd_ctas(int B, int Hq, int Hkv, int N, int d, int* ctas) {
  const int rows = 32 / (d / 16);
  const long long tokens = (long long)B * N;
  const int chunk = chunk_of(tokens, Hq > Hkv ? Hq : Hkv, rows);
  const long long room = (long long)sms() * 4;
  const int H[2] = {Hq, Hkv};
  for (int t = 0; t < 2; ++t) {
    const long long need = (tokens * parts_of(H[t], chunk) + WARPS - 1) / WARPS;
    long long share = room * H[t] / (Hq + Hkv);
    if (share < 1) share = 1;
    ctas[t] = H[t] == 0 ? 0 : (int)(need < share ? need : share);
  }
}

cudaError_t launch_norm_rope_bwd(const RopeParams& p, cudaStream_t st) {
  const int rows = 32 / (p.d / 16);
  const int chunk = chunk_of((long long)p.B * p.N, p.t[0].H > p.t[1].H ? p.t[0].H : p.t[1].H, rows);
  const int nq = parts_of(p.t[0].H, chunk), nk = parts_of(p.t[1].H, chunk);
  auto pick = [&](auto f32) {
    constexpr bool F = decltype(f32)::value;
    return p.d == 128 ? (p.pairs ? norm_rope_bwd_kernel<128, true, F> : norm_rope_bwd_kernel<128, false, F>)
                      : (p.pairs ? norm_rope_bwd_kernel<64, true, F> : norm_rope_bwd_kernel<64, false, F>);
  };
  auto k = p.dy_f32 ? pick(std::true_type()) : pick(std::false_type());
  k<<<p.ctas[0] + p.ctas[1], WARPS * 32, 0, st>>>(p, chunk, nq, nk);
  if (p.t[0].dw || p.t[1].dw) norm_rope_dw_kernel<<<2 * (p.d / 32), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fa4
