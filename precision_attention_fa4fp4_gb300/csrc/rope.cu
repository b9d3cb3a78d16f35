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
// it modulo 2^64 is the remainder, whose upper 32 bits give th in [-pi, pi] within
// 2^-21 (two roundings to FP32 and a constant's, 3.0e-7), at position 2^31 as at 1
// (an FP32 product is off by 0.03 at 10^6).  The native sine and cosine are off by
// 2^-21 there, against bf16's 2^-8.
#include <cuda_bf16.h>
#include "common.cuh"
#include "divide.cuh"
#include <type_traits>
#include "rope.h"

namespace fa4 {
namespace {

constexpr int WARPS = 8;

// Two 16-byte words of bf16 -> first and second channels of 8 pairs, two pairs to
// a float2 (packed FP32 arithmetic: an instruction for two).
template <bool PAIRS>
FA4_DEV void unpack(const uint4& u, const uint4& v, float2 (&a)[4], float2 (&b)[4]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (PAIRS) {
      a[i] = make_float2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
      b[i] = make_float2(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
    } else {
      a[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      b[i] = make_float2(__uint_as_float(w[4 + i] << 16), __uint_as_float(w[4 + i] & 0xffff0000u));
    }
  }
}

FA4_DEV uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

template <bool PAIRS>
FA4_DEV void pack(const float2 (&a)[4], const float2 (&b)[4], uint4& u, uint4& v) {
  if (PAIRS) {
    u = make_uint4(pack2(a[0].x, b[0].x), pack2(a[0].y, b[0].y), pack2(a[1].x, b[1].x), pack2(a[1].y, b[1].y));
    v = make_uint4(pack2(a[2].x, b[2].x), pack2(a[2].y, b[2].y), pack2(a[3].x, b[3].x), pack2(a[3].y, b[3].y));
  } else {
    u = make_uint4(pack2(a[0].x, a[0].y), pack2(a[1].x, a[1].y), pack2(a[2].x, a[2].y), pack2(a[3].x, a[3].y));
    v = make_uint4(pack2(b[0].x, b[0].y), pack2(b[1].x, b[1].y), pack2(b[2].x, b[2].y), pack2(b[3].x, b[3].y));
  }
}

// 16 FP32 values of a lane's channels, laid out as a row's: the same.
template <bool PAIRS>
FA4_DEV void unpack(const float4 (&f)[4], float2 (&a)[4], float2 (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (PAIRS) {
      a[i] = make_float2(f[i].x, f[i].z);
      b[i] = make_float2(f[i].y, f[i].w);
    } else {
      a[i] = i % 2 ? make_float2(f[i / 2].z, f[i / 2].w) : make_float2(f[i / 2].x, f[i / 2].y);
      b[i] = i % 2 ? make_float2(f[2 + i / 2].z, f[2 + i / 2].w) : make_float2(f[2 + i / 2].x, f[2 + i / 2].y);
    }
  }
}

// Rows that are not there: their norm is no special case.
FA4_DEV uint4 ones() { return make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u); }

FA4_DEV float2 both(float x) { return make_float2(x, x); }
FA4_DEV float2 neg(float2 x) { return make_float2(-x.x, -x.y); }

// Where a lane's two words of a row start, in channels.
template <int D, bool PAIRS>
FA4_DEV int word0(int l) { return PAIRS ? 16 * l : 8 * l; }
template <int D, bool PAIRS>
FA4_DEV int word1(int l) { return PAIRS ? 16 * l + 8 : D / 2 + 8 * l; }

// Sines and cosines of a lane's 8 pairs at one token.
FA4_DEV void angles(const RopeParams& p, const uint64_t* turn, const uint8_t* axis, int b, int n, int l,
                    float2 (&c)[4], float2 (&s)[4]) {
  if (!p.pos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { c[i] = both(1.f); s[i] = both(0.f); }
    return;
  }
  const int* at = p.pos + b * p.pos_b + n;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t where = at[(long long)axis[8 * l + i] * p.N];   // (plainly: the launch before may have written it)
    const int rest = (int)(((uint64_t)where * turn[8 * l + i]) >> 32);   // of a turn, times 2^32
    const float th = (float)rest * 1.46291807926715968e-9f;              // 2 pi / 2^32
    (i % 2 ? c[i / 2].y : c[i / 2].x) = __cosf(th);
    (i % 2 ? s[i / 2].y : s[i / 2].x) = __sinf(th);
  }
}

template <int LANES>
FA4_DEV float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows whose squares come near an end of FP32's range (values from 2^50 on, or, with an eps that is smaller still,
// below 2^-50) are seldom: they are formed anew in units of 2^100 or 2^-100, and normalized before they go on.
FA4_DEV bool far(float ms) { return !(ms > 0x1p-100f && ms < 0x1p100f); }
struct Unit {
  float unit;
  FA4_DEV explicit Unit(float ms) : unit(ms < 1.f ? 0x1p100f : 0x1p-100f) {}
  FA4_DEV float squares(const float2 (&a)[4], const float2 (&b)[4]) const {
    float2 q = both(0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = fmul2(a[j], both(unit)), y = fmul2(b[j], both(unit));
      q = ffma2(y, y, ffma2(x, x, q));
    }
    return q.x + q.y;
  }
  // 1 / sqrt(mean(x^2) + eps) over the unit
  FA4_DEV float root(float sum, float per, float eps) const { return rsqrtf(fmaf(sum, per, eps * unit * unit)); }
  // x r (the root first: a channel far smaller than its row keeps its bits)
  FA4_DEV float2 apply(float2 x, float root) const { return fmul2(fmul2(x, both(root)), both(unit)); }
};

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
  // the weights of a lane's channels, which begin at c0 and c1
  template <bool PAIRS>
  FA4_DEV void weights(int t, int c0, int c1, float2 (&a)[4], float2 (&b)[4]) const {
    const float4 f[4] = {*reinterpret_cast<const float4*>(&w[t][c0]), *reinterpret_cast<const float4*>(&w[t][c0 + 4]),
                         *reinterpret_cast<const float4*>(&w[t][c1]), *reinterpret_cast<const float4*>(&w[t][c1 + 4])};
    unpack<PAIRS>(f, a, b);
  }
};


// U rows of a lane group are on their way at a time: 3, with 3 CTAs on a
// multiprocessor and as many in the grid (24 + 24 heads of 32760 tokens: 137 us, 0.88
// of measured HBM; 4 rows and 2 CTAs 144, 2 and 4 150; a CTA for every 8 tokens 145).
constexpr int FWD_CTAS = 3;
template <int D, bool PAIRS, int U>
__global__ void __launch_bounds__(WARPS * 32, FWD_CTAS)
    norm_rope_kernel(const __grid_constant__ RopeParams p, int chunk, int nq, int nk, Divisor by_tokens, Divisor by_n) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES;
  __shared__ Tables<D> tab;
  next_may_start();
  wait_for_previous();
  tab.load(p);
  const int lane = threadIdx.x % 32, l = lane % LANES, sub = lane / LANES;
  const int c0 = word0<D, PAIRS>(l), c1 = word1<D, PAIRS>(l);
  for (Tasks task{blockIdx.x * WARPS + threadIdx.x / 32, gridDim.x * WARPS, (uint32_t)by_tokens.d * (nq + nk)};
       task.more(); task.next()) {
    int part, m, b, n;
    divide((int)task.now, by_tokens, part, m);
    divide(m, by_n, b, n);
    const int t = part >= nq;
    const RopeTensor& T = p.t[t];
    const int h0 = (t ? part - nq : part) * chunk, h1 = min(T.H, h0 + chunk);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(T.x.p) + b * T.x.b + n * T.x.n;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(T.out.p) + b * T.out.b + n * T.out.n;
    float2 c[4], s[4], wa[4], wb[4];
    bool first = true;
    for (int h = h0 + sub; h - sub < h1; h += ROWS * U) {
      uint4 u[U], v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        u[i] = v[i] = ones();
        if (h + i * ROWS < h1) {
          const __nv_bfloat16* row = x + (h + i * ROWS) * T.x.h;
          u[i] = *reinterpret_cast<const uint4*>(row + c0);
          v[i] = *reinterpret_cast<const uint4*>(row + c1);
        }
      }
      if (first) {
        angles(p, tab.turn, tab.axis, b, n, l, c, s);
        tab.template weights<PAIRS>(t, c0, c1, wa, wb);
        first = false;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float2 fa[4], fb[4];
        unpack<PAIRS>(u[i], v[i], fa, fb);
        float r = 1.f;
        if (p.norm) {
          float2 q = fmul2(fa[0], fa[0]);
          q = ffma2(fb[0], fb[0], q);
#pragma unroll
          for (int j = 1; j < 4; ++j) q = ffma2(fb[j], fb[j], ffma2(fa[j], fa[j], q));
          const float ms = row_sum<LANES>(q.x + q.y) * (1.f / D) + p.eps;
          r = rsqrtf(ms);
          if (__builtin_expect(__any_sync(0xffffffffu, far(ms)), 0)) {
            const Unit by(ms);
            const float root = by.root(row_sum<LANES>(by.squares(fa, fb)), 1.f / D, p.eps);
            if (far(ms)) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                fa[j] = by.apply(fa[j], root);
                fb[j] = by.apply(fb[j], root);
              }
              r = 1.f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 na = fmul2(fmul2(fa[j], both(r)), wa[j]), nb = fmul2(fmul2(fb[j], both(r)), wb[j]);
          fa[j] = ffma2(neg(nb), s[j], fmul2(na, c[j]));
          fb[j] = ffma2(na, s[j], fmul2(nb, c[j]));
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

// What a lane holds of a row of x and of the output's gradient on their way.
template <bool F32>
struct RowPair {
  uint4 u, v;
  float4 g[F32 ? 4 : 2];

  // (a row that is not there: its gradient is 0)
  FA4_DEV void none() {
    u = v = ones();
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  FA4_DEV void fetch(const __nv_bfloat16* x, const void* dy, long long at, int c0, int c1) {
    u = *reinterpret_cast<const uint4*>(x + c0);
    v = *reinterpret_cast<const uint4*>(x + c1);
    if (F32) {
      const float* from = static_cast<const float*>(dy) + at;
      g[0] = *reinterpret_cast<const float4*>(from + c0);
      g[1] = *reinterpret_cast<const float4*>(from + c0 + 4);
      g[F32 ? 2 : 0] = *reinterpret_cast<const float4*>(from + c1);
      g[F32 ? 3 : 0] = *reinterpret_cast<const float4*>(from + c1 + 4);
    } else {
      const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(dy) + at;
      g[0] = *reinterpret_cast<const float4*>(from + c0);
      g[1] = *reinterpret_cast<const float4*>(from + c1);
    }
  }
  template <bool PAIRS>
  FA4_DEV void take(float2 (&fa)[4], float2 (&fb)[4], float2 (&ga)[4], float2 (&gb)[4]) const {
    unpack<PAIRS>(u, v, fa, fb);
    if constexpr (F32) unpack<PAIRS>(g, ga, gb);
    else unpack<PAIRS>(*reinterpret_cast<const uint4*>(&g[0]), *reinterpret_cast<const uint4*>(&g[1]), ga, gb);
  }
};

// A gradient turned back.
FA4_DEV void turn_back(float2 (&ga)[4], float2 (&gb)[4], const float2 (&c)[4], const float2 (&s)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 e = ga[j];
    ga[j] = ffma2(gb[j], s[j], fmul2(e, c[j]));
    gb[j] = ffma2(neg(e), s[j], fmul2(gb[j], c[j]));
  }
}

template <bool PAIRS>
FA4_DEV void put(__nv_bfloat16* row, int c0, int c1, const float2 (&a)[4], const float2 (&b)[4]) {
  uint4 u, v;
  pack<PAIRS>(a, b, u, v);
  *reinterpret_cast<uint4*>(row + c0) = u;
  *reinterpret_cast<uint4*>(row + c1) = v;
}

// A warp's sums of the weight's gradient, over its rows of lanes, by channels.
template <int D, bool PAIRS, class F>
FA4_DEV void by_channel(const float2 (&da)[4], const float2 (&db)[4], F to) {
  constexpr int LANES = D / 16;
  const int lane = threadIdx.x % 32, c0 = word0<D, PAIRS>(lane % LANES), c1 = word1<D, PAIRS>(lane % LANES);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float ya = j % 2 ? da[j / 2].y : da[j / 2].x, yb = j % 2 ? db[j / 2].y : db[j / 2].x;
#pragma unroll
    for (int o = LANES; o < 32; o *= 2) {
      ya += __shfl_xor_sync(0xffffffffu, ya, o);
      yb += __shfl_xor_sync(0xffffffffu, yb, o);
    }
    if (lane < LANES) {
      to(PAIRS ? c0 + 2 * j : c0 + j, ya);
      to(PAIRS ? c0 + 2 * j + 1 : c1 + j, yb);
    }
  }
}

// Gradients.  The CTAs [0, ctas[0]) work on q, the others on k; every lane adds
// its 16 channels of the weight's gradient over its tasks, the CTA joins them in
// a fixed order and leaves one row of partials.  A row's x and gradient are on their
// way while the row before is at work.  2 CTAs on a multiprocessor: a lane's sums,
// weights, sines and cosines and two rows take 128 registers (at 85, for 3 CTAs, they
// spill: 132 -> 210 us for 2 x 8192 tokens of 32 + 8 heads with f32 gradients; rows
// ahead by asynchronous copies to shared memory 157).
// Far rows are left out and told to shared memory; behind a task that had some the loop
// over the tasks is left for them.  (dx may lie in x's place: theirs is not written before.)
// Formed inside that loop they cost calls without such rows a tenth, in registers (126
// -> 138 us), as a call of their own 154.
constexpr int BWD_CTAS = 2;
template <int D, bool PAIRS, bool F32>
__global__ void __launch_bounds__(WARPS * 32, BWD_CTAS)
    norm_rope_bwd_kernel(const __grid_constant__ RopeParams p, int chunk, int nq, int nk, Divisor by_tokens,
                         Divisor by_n) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES;
  __shared__ Tables<D> tab;
  __shared__ float join[WARPS][D];
  __shared__ uint32_t left_out[WARPS][ROWS];   // rounds whose row is far
  next_may_start();
  wait_for_previous();
  tab.load(p);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % LANES, sub = lane / LANES;
  const int c0 = word0<D, PAIRS>(l), c1 = word1<D, PAIRS>(l);
  if (l == 0) left_out[warp][sub] = 0;
  __syncwarp();
  const int t = (int)blockIdx.x >= p.ctas[0];
  const int cta = t ? (int)blockIdx.x - p.ctas[0] : (int)blockIdx.x;
  const RopeTensor& T = p.t[t];
  float2 da[4], db[4], wa[4], wb[4];
  tab.template weights<PAIRS>(t, c0, c1, wa, wb);
#pragma unroll
  for (int j = 0; j < 4; ++j) da[j] = db[j] = both(0.f);
  // a task's heads and where its rows lie
  struct Place {
    int b, n, h0, h1;
    const __nv_bfloat16* x;
    __nv_bfloat16* dx;
    long long dy;
  };
  const auto place = [&](uint32_t task) {
    Place a;
    int part, m;
    divide((int)task, by_tokens, part, m);
    divide(m, by_n, a.b, a.n);
    a.h0 = part * chunk;
    a.h1 = min(T.H, a.h0 + chunk);
    a.x = static_cast<const __nv_bfloat16*>(T.x.p) + a.b * T.x.b + a.n * T.x.n;
    a.dx = static_cast<__nv_bfloat16*>(T.out.p) + a.b * T.out.b + a.n * T.out.n;
    a.dy = a.b * T.dy.b + a.n * T.dy.n;
    return a;
  };
  const auto fetch = [&](const Place& a, int h, RowPair<F32>& row) {
    row.none();
    if (h < a.h1) row.fetch(a.x + h * T.x.h, T.dy.p, a.dy + h * T.dy.h, c0, c1);
  };
  Tasks task{(uint32_t)(cta * WARPS + warp), (uint32_t)(p.ctas[t] * WARPS), (uint32_t)by_tokens.d * (t ? nk : nq)};
  while (task.more()) {
    uint32_t mine = 0, last = 0;
    for (; task.more(); task.next()) {
      const Place a = place(task.now);
      float2 c[4], s[4];
      RowPair<F32> next;
      fetch(a, a.h0 + sub, next);
      angles(p, tab.turn, tab.axis, a.b, a.n, l, c, s);
      for (int h = a.h0 + sub; h - sub < a.h1; h += ROWS) {
        bool on = h < a.h1;
        float2 ga[4], gb[4], fa[4], fb[4];
        next.template take<PAIRS>(fa, fb, ga, gb);
        fetch(a, h + ROWS, next);
        turn_back(ga, gb, c, s);
        if (p.norm) {
          float2 xx = both(0.f), ux = both(0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xx = ffma2(fa[j], fa[j], ffma2(fb[j], fb[j], xx));
            ux = ffma2(fmul2(ga[j], wa[j]), fa[j], ffma2(fmul2(gb[j], wb[j]), fb[j], ux));
          }
          const float sx = row_sum<LANES>(xx.x + xx.y), su = row_sum<LANES>(ux.x + ux.y);
          const float ms = sx * (1.f / D) + p.eps;
          const bool wait = far(ms);
          if (wait) {
            left_out[warp][sub] |= 1u << (h - a.h0) / ROWS;      // (the same by all lanes of the row)
            on = false;
          }
          // (rows that are left out add nothing)
          const float r = wait ? 0.f : rsqrtf(ms);
          const float k = r * r * su * (1.f / D);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            da[j] = ffma2(ga[j], fmul2(fa[j], both(r)), da[j]);
            db[j] = ffma2(gb[j], fmul2(fb[j], both(r)), db[j]);
            ga[j] = fmul2(ffma2(fa[j], both(-k), fmul2(ga[j], wa[j])), both(r));
            gb[j] = fmul2(ffma2(fb[j], both(-k), fmul2(gb[j], wb[j])), both(r));
          }
        }
        if (on) put<PAIRS>(a.dx + h * T.out.h, c0, c1, ga, gb);
      }
      __syncwarp();
      mine = left_out[warp][sub];
      if (__any_sync(0xffffffffu, mine)) {
        last = task.now;
        task.next();
        break;
      }
    }
    uint32_t all = __reduce_or_sync(0xffffffffu, mine);
    if (!all) break;
    // the far rows of the last task
    const Place a = place(last);
    float2 c[4], s[4];
    angles(p, tab.turn, tab.axis, a.b, a.n, l, c, s);
    for (; all; all &= all - 1) {
      const int round = __ffs(all) - 1, h = a.h0 + round * ROWS + sub;
      const bool on = (mine >> round & 1) && h < a.h1;
      RowPair<F32> row;
      fetch(a, on ? h : a.h1, row);
      float2 ga[4], gb[4], fa[4], fb[4];
      row.template take<PAIRS>(fa, fb, ga, gb);
      turn_back(ga, gb, c, s);
      float2 q = both(0.f), un = both(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) q = ffma2(fa[j], fa[j], ffma2(fb[j], fb[j], q));
      const Unit by(row_sum<LANES>(q.x + q.y) * (1.f / D) + p.eps);
      const float root = by.root(row_sum<LANES>(by.squares(fa, fb)), 1.f / D, p.eps);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fa[j] = by.apply(fa[j], root);
        fb[j] = by.apply(fb[j], root);
        un = ffma2(fmul2(ga[j], wa[j]), fa[j], ffma2(fmul2(gb[j], wb[j]), fb[j], un));
      }
      const float r = root * by.unit, k = row_sum<LANES>(un.x + un.y) * (1.f / D);
      if (!on) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        da[j] = ffma2(ga[j], fa[j], da[j]);
        db[j] = ffma2(gb[j], fb[j], db[j]);
        ga[j] = fmul2(ffma2(fa[j], both(-k), fmul2(ga[j], wa[j])), both(r));
        gb[j] = fmul2(ffma2(fb[j], both(-k), fmul2(gb[j], wb[j])), both(r));
      }
      put<PAIRS>(a.dx + h * T.out.h, c0, c1, ga, gb);
    }
    __syncwarp();
    left_out[warp][sub] = 0;
    __syncwarp();
  }
  if (!T.dw) return;
  by_channel<D, PAIRS>(da, db, [&](int i, float y) { join[warp][i] = y; });
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += WARPS * 32) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += join[w][i];
    T.part[(long long)cta * D + i] = sum;
  }
}

// dw = sum of the CTAs' partials: one CTA per tensor and 32 channels.
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(DW_WARPS * 32) norm_rope_dw_kernel(const __grid_constant__ RopeParams p) {
  const int per = p.d / 32, t = blockIdx.x / per, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = (blockIdx.x % per) * 32 + lane;
  const RopeTensor& T = p.t[t];
  wait_for_previous();
  if (!T.dw) return;
  __shared__ float join[DW_WARPS][32];
  float sum = 0.f;
#pragma unroll 4
  for (int c = warp; c < p.ctas[t]; c += DW_WARPS) sum += T.part[(long long)c * p.d + i];
  join[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < DW_WARPS; ++w) sum += join[w][lane];
    T.dw[i] = sum;
  }
}

// Heads of a warp's task: all of a tensor's where there are tokens enough to fill
// the GPU with one warp each, else as few as one round of its lanes.
// A task of the gradients has 32 rounds at most.
constexpr int BWD_ROUNDS = 32;
int chunk_of(long long tokens, int H, int rows) {
  const long long want = (long long)sm_count() * 16;
  if (H <= rows || tokens >= want) return H > 0 ? H : 1;
  const long long parts = (want + tokens - 1) / tokens;
  const long long rounds = (H + rows - 1) / rows;
  const long long per = (rounds + parts - 1) / parts;
  return (int)(per * rows);
}

int bwd_chunk_of(long long tokens, int H, int rows) {
  const int chunk = chunk_of(tokens, H, rows);
  return chunk < BWD_ROUNDS * rows ? chunk : BWD_ROUNDS * rows;
}

int parts_of(int H, int chunk) { return (H + chunk - 1) / chunk; }

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t st) {
  const int rows = 32 / (p.d / 16);
  const int tokens = p.B * p.N;
  const int chunk = chunk_of(tokens, p.t[0].H > p.t[1].H ? p.t[0].H : p.t[1].H, rows);
  const int nq = parts_of(p.t[0].H, chunk), nk = parts_of(p.t[1].H, chunk);
  const int need = (int)(((long long)tokens * (nq + nk) + WARPS - 1) / WARPS), room = FWD_CTAS * sm_count();
  auto k = p.d == 128 ? (p.pairs ? norm_rope_kernel<128, true, 3> : norm_rope_kernel<128, false, 3>)
                      : (p.pairs ? norm_rope_kernel<64, true, 3> : norm_rope_kernel<64, false, 3>);
  return launch(k, dim3(need < room ? need : room), WARPS * 32, 0, true, st, p, chunk, nq, nk, Divisor(tokens),
                Divisor(p.N));
}

void rope_bwd_ctas(int B, int Hq, int Hkv, int N, int d, int* ctas) {
  const int rows = 32 / (d / 16);
  const long long tokens = (long long)B * N;
  const int chunk = bwd_chunk_of(tokens, Hq > Hkv ? Hq : Hkv, rows);
  const long long room = (long long)sm_count() * BWD_CTAS;
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
  const int chunk = bwd_chunk_of((long long)p.B * p.N, p.t[0].H > p.t[1].H ? p.t[0].H : p.t[1].H, rows);
  const int nq = parts_of(p.t[0].H, chunk), nk = parts_of(p.t[1].H, chunk);
  const Divisor by_tokens(p.B * p.N), by_n(p.N);
  auto pick = [&](auto f32) {
    constexpr bool F = decltype(f32)::value;
    return p.d == 128 ? (p.pairs ? norm_rope_bwd_kernel<128, true, F> : norm_rope_bwd_kernel<128, false, F>)
                      : (p.pairs ? norm_rope_bwd_kernel<64, true, F> : norm_rope_bwd_kernel<64, false, F>);
  };
  auto k = p.dy_f32 ? pick(std::true_type()) : pick(std::false_type());
  const cudaError_t e =
      launch(k, dim3(p.ctas[0] + p.ctas[1]), WARPS * 32, 0, true, st, p, chunk, nq, nk, by_tokens, by_n);
  if (e != cudaSuccess || !(p.t[0].dw || p.t[1].dw)) return e;
  return launch(norm_rope_dw_kernel, dim3(2 * (p.d / 32)), DW_WARPS * 32, 0, true, st, p);
}

}  // namespace fa4
