// cache_weigh.cu -- the attention weight that every cached token received from
// a call's queries:
//   out[j] = in[j] + sum over the query heads of the kv head and the tokens t
//            that see j of  e^(scale q.k_j - lse)
// with the log-sum-exp that the attention wrote.  Every (kv head, token) has
// one owner, so nothing is added in an order that changes.
//
// One query token: bound by HBM, d bytes of K and 8 bytes of weight per token
// and kv head.  Many query tokens: bound by the m16n8k16 products and one
// exponential per score; each warp converts its 32 keys once and keeps them as
// f16 operands while it walks over the query rows.
#include "cache.cuh"

namespace fa4 {
namespace {

constexpr int NW = 4;
constexpr int UNIT = 32 * NW;

template <int D>
__global__ void __launch_bounds__(32 * NW) cache_weigh_kernel(const __grid_constant__ CacheWeighParams p) {
  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t4 = lane % 4;
  const int h = blockIdx.y, b = blockIdx.z;
  const int len = cache_len(c, b);
  const int key0 = blockIdx.x * UNIT + 32 * warp;
  if (key0 >= len) return;
  const int q_len = cache_count(p.q_lens, b, p.T, c.err);
  const int G = p.Hq / c.Hkv;

  uint32_t ka[2][D / 16][4];
  float kx[2];
  int end[2];                                        // keys of each 16 that are there: below it
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = key0 + 16 * i;
    int pg = -1;
    if (k < len) pg = cache_page(c, c.table, b, k / c.page);
    const long long ph = (long long)max(pg, 0) * c.Hkv + h;
    const long long tok = ph * c.page + k % c.page;
    kx[i] = e8m0_value(__ldg(c.ks + ph));
    end[i] = pg < 0 ? 0 : len;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4 lo = __ldg(reinterpret_cast<const uint4*>(c.k + (tok + g) * D + 64 * j + 16 * t4));
      const uint4 hi = __ldg(reinterpret_cast<const uint4*>(c.k + (tok + g + 8) * D + 64 * j + 16 * t4));
      const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, e[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        ka[i][4 * j + w][0] = e4m3x2_to_f16x2(a[w]);
        ka[i][4 * j + w][1] = e4m3x2_to_f16x2(e[w]);
        ka[i][4 * j + w][2] = e4m3x2_hi_to_f16x2(a[w]);
        ka[i][4 * j + w][3] = e4m3x2_hi_to_f16x2(e[w]);
      }
    }
  }
  const int rows = q_len * G;
  // the first token that sees any key of the warp
  const int t_first = p.causal ? max(0, key0 - (len - q_len)) : 0;
  float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};          // keys g, g + 8 of each 16
  for (int r0 = t_first * G / 8 * 8; r0 < rows; r0 += 8) {
    const int rg = r0 + g;
    QFrag<D> q;
    const __nv_bfloat16* row = nullptr;
    if (rg < rows)
      row = reinterpret_cast<const __nv_bfloat16*>(p.q) +
            (((long long)b * p.Hq + h * G + rg % G) * p.T + rg / G) * D;
    QRaw<D> raw;
    raw.fetch(row, t4);
    const float e = raw.convert(q);
    float fx[2], hi[2], lo[2];
    int vis[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = r0 + 2 * t4 + j;
      fx[j] = p.c2 * __shfl_sync(0xffffffffu, e, (2 * t4 + j) * 4);
      vis[j] = 0;
      hi[j] = lo[j] = 0.f;
      if (r < rows) {
        const int t = r / G;
        // lse * log2 e as a sum of two floats
        const float z = __ldg(p.lse + ((long long)b * p.Hq + h * G + r % G) * p.T + t);
        hi[j] = z * 1.4426950216293335f;
        lo[j] = fmaf(z, 1.4426950216293335f, -hi[j]) + z * 1.9259629911266175e-8f;
        if (z != -INFINITY) vis[j] = p.causal ? max(0, min(len, len - q_len + t + 1)) : len;
      }
    }
    float s[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_16816(s[i], ka[i][k][0], ka[i][k][1], ka[i][k][2], ka[i][k][3], q.b[k][0], q.b[k][1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 16 * i + g + 8 * (j >> 1);
        const float x = s[i][j] * kx[i] * fx[j & 1];
        if (key < min(end[i], vis[j & 1])) w[i][j >> 1] += ex2_approx((x - hi[j & 1]) - lo[j & 1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      w[i][r] += __shfl_xor_sync(0xffffffffu, w[i][r], 1);
      w[i][r] += __shfl_xor_sync(0xffffffffu, w[i][r], 2);
      const int key = key0 + 16 * i + 8 * r + g;
      if (t4 == 0 && key < len) {
        const long long at = ((long long)b * c.Hkv + h) * c.max_pages * c.page + key;
        p.w_out[at] = p.w_in[at] + w[i][r];
      }
    }
}

}  // namespace

cudaError_t launch_cache_weigh(const CacheWeighParams& p, cudaStream_t st) {
  const long long cap = (long long)p.c.max_pages * p.c.page;
  const dim3 grid((unsigned)((cap + UNIT - 1) / UNIT), (unsigned)p.c.Hkv, (unsigned)p.c.B);
  if (p.c.d == 128) cache_weigh_kernel<128><<<grid, 32 * NW, 0, st>>>(p);
  else cache_weigh_kernel<64><<<grid, 32 * NW, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fa4
