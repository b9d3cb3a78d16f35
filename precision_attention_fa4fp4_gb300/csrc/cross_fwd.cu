// cross_fwd.cu -- attention of queries to keys of another length, one warp per
// query row: 32 keys at a time, a lane's score each, an online softmax over the
// lanes, then the 32 rows of V with d / 32 channels a lane.
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"

namespace fa4 {
namespace {

constexpr int WARPS = 8;

template <int D>
__global__ void __launch_bounds__(WARPS * 32) cross_fwd_kernel(const __grid_constant__ CrossParams p) {
  constexpr int C = D / 32;
  __shared__ float qs[WARPS][D];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long row = (long long)blockIdx.x * WARPS + warp;
  if (row >= (long long)p.B * p.Hq * p.Nq) return;
  const int n = (int)(row % p.Nq), bh = (int)(row / p.Nq), h = bh % p.Hq, b = bh / p.Hq, hk = h / (p.Hq / p.Hkv);
  const int len = key_count(p, b);
  const __nv_bfloat16* q = at(p.q, b, h, n);
  for (int i = lane; i < D; i += 32) qs[warp][i] = __bfloat162float(q[i]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[C] = {};
  for (int j0 = 0; j0 < len; j0 += 32) {
    const int j = j0 + lane;
    const float s = j < len ? dot<D>(qs[warp], at(p.k, b, hk, j)) * p.c : -INFINITY;
    float top = s;
    for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float now = fmaxf(m, top);
    const float e = j < len ? exp2f(s - now) : 0.f;
    const float a = m == -INFINITY ? 0.f : exp2f(m - now);
    m = now;
    l = l * a + e;
    for (int i = 0; i < C; ++i) o[i] *= a;
    for (int x = 0; x < min(32, len - j0); ++x) {
      const float w = __shfl_sync(0xffffffffu, e, x);
      const __nv_bfloat16* v = at(p.v, b, hk, j0 + x) + lane * C;
      for (int i = 0; i < C; ++i) o[i] = fmaf(w, __bfloat162float(v[i]), o[i]);
    }
  }
  for (int x = 16; x > 0; x /= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
  __nv_bfloat16* out = at(p.o, b, h, n) + lane * C;
  for (int i = 0; i < C; ++i) out[i] = __float2bfloat16(len > 0 ? o[i] / l : 0.f);
  if (p.lse && lane == 0) p.lse[row] = len > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_cross_fwd(const CrossParams& p, cudaStream_t st) {
  const long long rows = (long long)p.B * p.Hq * p.Nq;
  const unsigned grid = (unsigned)((rows + WARPS - 1) / WARPS);
  if (p.d == 128) cross_fwd_kernel<128><<<grid, WARPS * 32, 0, st>>>(p);
  else cross_fwd_kernel<64><<<grid, WARPS * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fa4
