// cross_bwd.cu -- gradients of cross attention.  A warp per query row takes D =
// rowsum(dO o) into the workspace and dQ; a warp per key takes dK and dV, over
// the queries of all heads that share the key.  32 partners at a time, a lane's
// score and dP each.
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"

namespace fa4 {
namespace {

constexpr int WARPS = 8;
constexpr float L2E = 1.4426950408889634f;

template <int D>
FA4_DEV void load_row(float* dst, const __nv_bfloat16* src, int lane) {
  for (int i = lane; i < D; i += 32) dst[i] = __bfloat162float(src[i]);
}

template <int D>
__global__ void __launch_bounds__(WARPS * 32) cross_dq_kernel(const __grid_constant__ CrossParams p) {
  constexpr int C = D / 32;
  __shared__ float qs[WARPS][D], gs[WARPS][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long row = (long long)blockIdx.x * WARPS + warp;
  if (row >= (long long)p.B * p.Hq * p.Nq) return;
  const int n = (int)(row % p.Nq), bh = (int)(row / p.Nq), h = bh % p.Hq, b = bh / p.Hq, hk = h / (p.Hq / p.Hkv);
  const int len = key_count(p, b);
  load_row<D>(qs[warp], at(p.q, b, h, n), lane);
  load_row<D>(gs[warp], at(p.dout, b, h, n), lane);
  __syncwarp();
  float del = 0.f;
  for (int i = lane; i < D; i += 32) del = fmaf(gs[warp][i], __bfloat162float(at(p.o, b, h, n)[i]), del);
  for (int x = 16; x > 0; x /= 2) del += __shfl_xor_sync(0xffffffffu, del, x);
  if (lane == 0) reinterpret_cast<float*>(p.work)[row] = del;
  const float lse = p.lse[row] * L2E;
  const bool use = p.lse[row] != -INFINITY;
  float g[C] = {};
  for (int j0 = 0; use && j0 < len; j0 += 32) {
    const int j = j0 + lane;
    float ds = 0.f;
    if (j < len) {
      const float e = exp2f(dot<D>(qs[warp], at(p.k, b, hk, j)) * p.c - lse);
      ds = e * (dot<D>(gs[warp], at(p.v, b, hk, j)) - del) * p.scale;
    }
    for (int x = 0; x < min(32, len - j0); ++x) {
      const float w = __shfl_sync(0xffffffffu, ds, x);
      const __nv_bfloat16* k = at(p.k, b, hk, j0 + x) + lane * C;
      for (int i = 0; i < C; ++i) g[i] = fmaf(w, __bfloat162float(k[i]), g[i]);
    }
  }
  __nv_bfloat16* out = at(p.dq, b, h, n) + lane * C;
  for (int i = 0; i < C; ++i) out[i] = __float2bfloat16(g[i]);
}

template <int D>
__global__ void __launch_bounds__(WARPS * 32) cross_dkv_kernel(const __grid_constant__ CrossParams p) {
  constexpr int C = D / 32;
  __shared__ float ks[WARPS][D], vs[WARPS][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, G = p.Hq / p.Hkv;
  const long long row = (long long)blockIdx.x * WARPS + warp;
  if (row >= (long long)p.B * p.Hkv * p.Nk) return;
  const int j = (int)(row % p.Nk), bh = (int)(row / p.Nk), hk = bh % p.Hkv, b = bh / p.Hkv;
  float dk[C] = {}, dv[C] = {};
  if (j < key_count(p, b)) {
    load_row<D>(ks[warp], at(p.k, b, hk, j), lane);
    load_row<D>(vs[warp], at(p.v, b, hk, j), lane);
    __syncwarp();
    for (int h = hk * G; h < (hk + 1) * G; ++h) {
      const long long r0 = ((long long)b * p.Hq + h) * p.Nq;
      for (int n0 = 0; n0 < p.Nq; n0 += 32) {
        const int n = n0 + lane;
        float e = 0.f, ds = 0.f;
        if (n < p.Nq && p.lse[r0 + n] != -INFINITY) {
          e = exp2f(dot<D>(ks[warp], at(p.q, b, h, n)) * p.c - p.lse[r0 + n] * L2E);
          ds = e * (dot<D>(vs[warp], at(p.dout, b, h, n)) - reinterpret_cast<const float*>(p.work)[r0 + n]) * p.scale;
        }
        for (int x = 0; x < min(32, p.Nq - n0); ++x) {
          const float we = __shfl_sync(0xffffffffu, e, x), ws = __shfl_sync(0xffffffffu, ds, x);
          const __nv_bfloat16 *g = at(p.dout, b, h, n0 + x) + lane * C, *q = at(p.q, b, h, n0 + x) + lane * C;
          for (int i = 0; i < C; ++i) {
            dv[i] = fmaf(we, __bfloat162float(g[i]), dv[i]);
            dk[i] = fmaf(ws, __bfloat162float(q[i]), dk[i]);
          }
        }
      }
    }
  }
  __nv_bfloat16 *ok = at(p.dk, b, hk, j) + lane * C, *ov = at(p.dv, b, hk, j) + lane * C;
  for (int i = 0; i < C; ++i) {
    ok[i] = __float2bfloat16(dk[i]);
    ov[i] = __float2bfloat16(dv[i]);
  }
}

}  // namespace

size_t cross_bwd_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  return ((size_t)B * Hq * Nq * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_cross_bwd(const CrossParams& p, cudaStream_t st) {
  auto grid = [](long long rows) { return (unsigned)((rows + WARPS - 1) / WARPS); };
  const unsigned gq = grid((long long)p.B * p.Hq * p.Nq), gk = grid((long long)p.B * p.Hkv * p.Nk);
  if (p.d == 128) {
    if (gq) cross_dq_kernel<128><<<gq, WARPS * 32, 0, st>>>(p);
    if (gk) cross_dkv_kernel<128><<<gk, WARPS * 32, 0, st>>>(p);
  } else {
    if (gq) cross_dq_kernel<64><<<gq, WARPS * 32, 0, st>>>(p);
    if (gk) cross_dkv_kernel<64><<<gk, WARPS * 32, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa4
