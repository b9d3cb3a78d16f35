// cache_weigh.cu -- the attention weight that every cached token received from
// a call's queries:
//   out[j] = in[j] + sum over the query heads of the kv head and the tokens t
//            that see j of  e^(scale q.k_j - lse)
// with the log-sum-exp that the attention wrote.  Every (kv head, token) has
// one owner, so nothing is added in an order that changes.  The scores' products are
// summed over all of d by the tensor cores, which cut where they add: with the native
// exponential (0.4e-7 low by itself) a weight is about 1e-7 of itself off, plain FP32
// half of that.
//
// Up to 16 query rows per kv head: bound by HBM, d bytes of K and 8 of weights
// per token and kv head; K comes as in the attention, by TMA boxes into per-warp
// queues, and a fixed grid shares one line of (sequence, head, 128 keys): 16
// sequences of 4001..8192, 32 / 8 heads of 128, 23.2 us, 4.5 TB/s.
//
// Up to 79 rows: bound by the matrix products and one exponential per score.  A
// warp converts its 32 keys once and keeps them as f16 operands while it walks
// over the rows, which the CTA prepares 64 at a time: 32 rows of 8 heads of 128,
// 16 sequences of 2048, 25 us.  (The m16n8k32 E4M3 product would take the codes
// as they are, but is made of conversions and other products here: 631
// instructions a row tile, 175 us where this took 99.)
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NW = LINE_WARPS;

// ---------------------------------------------------------------- few rows
template <int D, int NT>
struct WQueue {
  static constexpr int S = D == 128 ? 3 : 4;
  static constexpr int BYTES = 32 * D;
  static constexpr int WARP = S * BYTES;
  static constexpr int OFF_BAR = NW * WARP;
  static constexpr int OFF_STEP = OFF_BAR + 8 * NW * S;
  static constexpr int OFF_MISC = OFF_STEP + 16 * NW * S;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
};

constexpr int weigh_ctas(int nt) { return nt == 1 ? 4 : 3; }

template <int D, int NT, bool SMALLP>
__global__ void __launch_bounds__(32 * NW, weigh_ctas(NT)) cache_weigh_kernel(const __grid_constant__ CacheWeighParams p) {
  using Q = WQueue<D, NT>;
  constexpr int S = Q::S;
  grid_start();
  constexpr int NP = SMALLP ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t4 = lane % 4;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Q::OFF_BAR) + warp * S;
  int4* steps = reinterpret_cast<int4*>(smem + Q::OFF_STEP) + warp * S;
  volatile int* abort_flag = reinterpret_cast<int*>(smem + Q::OFF_MISC);
  uint8_t* queue = smem + warp * Q::WARP;
  const int G = p.Hq / c.Hkv;

  const int log_p = 31 - __clz(c.page);
  unsigned phases = 0;
  if (lane == 0) {
    tma_prefetch_desc(&p.tm_k);
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();
  int ko[2][D / 64];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) ko[r][x] = boxed<D>(korder<D>(g) + 8 * r, 64 * x + 16 * t4);
  // of the eight sums of a quad's columns, the lane writes that of one key
  const int my_i = t4 >> 1, my_key = 16 * (t4 >> 1) + 8 * (t4 & 1) + korder<D>(g);

  auto seq = [&](int i) -> unsigned {
    const int n = cache_len(c, i);
    return n ? (unsigned)units_of(n) * c.Hkv : 0u;
  };
  grid_wait();
  const unsigned total = line_total(c.B, seq);
  if (total == 0) return;
  const unsigned ctas = workers(total, gridDim.x);
  if (blockIdx.x >= ctas) return;
  const Shares shares(total, ctas);
  const unsigned end = shares.begin(blockIdx.x + 1);
  unsigned at = shares.begin(blockIdx.x), seq0 = 0;
  int b = 0;
  if (!line_find(c.B, seq, at, b, seq0)) return;

  bool ok = true;
  int place = 0;
  while (ok && at < end) {
    while (at >= seq0 + seq(b)) seq0 += seq(b++);
    const int len = cache_len(c, b), units = units_of(len);
    const int q_len = cache_count(p.q_lens, b, p.T, c.err);
    const int h = (int)((at - seq0) / units), u0 = (int)((at - seq0) % units);
    const int u1 = (int)min((unsigned)units, u0 + (end - at));
    const int rows = G * q_len;                    // <= 8 NT: row r is token r / G, head r % G
    auto row_at = [&](int r) -> long long { return ((long long)b * p.Hq + h * G + r % G) * p.T + r / G; };
    QRaw<D> raw[NT];
    float lse[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
      raw[n].fetch(r < rows ? reinterpret_cast<const __nv_bfloat16*>(p.q) + row_at(r) * D : nullptr, t4);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rc = 8 * n + 2 * t4 + j;
        lse[n][j] = rc < rows ? *(p.lse + row_at(rc)) : 0.f;
      }
    }
    Window<NP> window;
    window.fill(c, b, h, len, nullptr, 0, u0, u1);
    auto issue = [&](int s, int u) {
      if (!window.has(u)) window.fill(c, b, h, len, nullptr, 0, u, u1);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int page = window.page(u, i), pos = window.pos(u, i);
        if (page >= 0 && lane == 0) {
          const int row = (int)(((long long)page * c.Hkv + h) << log_p) + (pos & (c.page - 1));
          mbar_expect_tx(&bars[s], (32 / NP) * D);
          tma_load_3d(queue + s * Q::BYTES + (SMALLP ? i * 16 * D : 0), &p.tm_k, &bars[s], 0, row, 0);
        }
      }
      if (lane == 0) mbar_arrive(&bars[s]);
    };
    auto note = [&](int s, int u) {
      int4 what = make_int4(window.pos(u, 0), window.scales(u, 0), NOWHERE, 0);
      if (NP == 2) { what.z = window.pos(u, NP - 1); what.w = window.scales(u, NP - 1); }
      if (lane == 0) steps[s] = what;
    };
    // the queue goes on where the last head left it
    for (int s = 0; s < S; ++s) issue((place + s) % S, u0 + s);
    for (int s = 0; s < S; ++s) note((place + s) % S, u0 + s);

    QFrag<D> q[NT];
    float fx[NT][2], ref[NT][2], fac[NT][2];
    int vis[NT][2], vis_min = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float e = raw[n].convert(q[n]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * t4 + j;
        const float f = __shfl_sync(0xffffffffu, e, (2 * t4 + j) * 4);
        reference(lse[n][j], r < rows, ref[n][j], fac[n][j]);
        fx[n][j] = fac[n][j] == 0.f ? 0.f : p.c2 * f;
        vis[n][j] = p.causal ? max(0, min(len, len - q_len + r / G + 1)) : len;
        if (r < rows) vis_min = min(vis_min, vis[n][j]);
      }
    }
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    const long long w_row = ((long long)b * c.Hkv + h) * c.max_pages * c.page;
    for (int u = u0; ok && u < u1; ++u) {
      if (!mbar_wait(&bars[place], (phases >> place) & 1, abort_flag, c.err)) { ok = false; break; }
      phases ^= 1u << place;
      __syncwarp();
      const uint8_t* from = queue + place * Q::BYTES;
      const int4 what = steps[place];
      int pos[NP];
      float kx[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        pos[i] = i ? what.z : what.x;
        kx[i] = e8m0_value((i ? what.w : what.y) & 0xff);
      }
      // the lane's key: its weight is read early (and written back as it was where
      // its page is not there)
      const int key = u * UNIT + 32 * warp + my_key;
      const bool there = (my_i ? pos[NP - 1] : pos[0]) != NOWHERE;
      const float had = key < len ? p.w_in[w_row + key] : 0.f;
      float s[NT][2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][i][j] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const uint4 ka = lds16(from + i * 16 * D + ko[0][k]);
          const uint4 kb = lds16(from + i * 16 * D + ko[1][k]);
          const uint32_t lo[4] = {ka.x, ka.y, ka.z, ka.w};
          const uint32_t hi[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(lo[w]), a2 = e4m3x2_hi_to_f16x2(lo[w]);
            const uint32_t a1 = e4m3x2_to_f16x2(hi[w]), a3 = e4m3x2_hi_to_f16x2(hi[w]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816(s[n][i], a0, a1, a2, a3, q[n].b[4 * k + w][0], q[n].b[4 * k + w][1]);
          }
        }
      __syncwarp();
      issue(place, u + S);
      note(place, u + S);
      place = place + 1 == S ? 0 : place + 1;

      bool full = true;
#pragma unroll
      for (int i = 0; i < NP; ++i) full = full && pos[i] + 32 / NP <= vis_min;
      float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};    // keys g, g + 8 of each 16
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (the factors first: K's times the sum alone may pass FP32's end)
            const float e = ex2_approx(fmaf(s[n][i][j], kx[i % NP] * fx[n][j & 1], -ref[n][j & 1]));
            // (a row that does not see the key must not reach it as 0 * NaN either)
            bool sees = true;
            if (!full) sees = pos[i % NP] + (SMALLP ? 0 : 16 * i) + korder<D>(g) + 8 * (j >> 1) < vis[n][j & 1];
            if (sees) w[i][j >> 1] = fmaf(e, fac[n][j & 1], w[i][j >> 1]);
          }
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          w[i][r] += __shfl_xor_sync(0xffffffffu, w[i][r], 1);
          w[i][r] += __shfl_xor_sync(0xffffffffu, w[i][r], 2);
          if (t4 == 2 * i + r) mine = w[i][r];
        }
      if (key < len) p.w_out[w_row + key] = had + (there ? mine : 0.f);
    }
    // the S steps behind the head's last unit have no boxes, only phases
    if (ok) {
      for (int s = 0; s < S; ++s) {
        const int st = (place + s) % S;
        ok = mbar_wait(&bars[st], (phases >> st) & 1, abort_flag, c.err) && ok;
        phases ^= 1u << st;
      }
    }
    at += u1 - u0;
  }
  if (!ok) {                                       // what is still in flight
    volatile int none = 0;
    for (int s = 0; s < S; ++s) mbar_wait(&bars[s], (phases >> s) & 1, &none, c.err);
  }
}

// ---------------------------------------------------------------- more rows
constexpr int BLOCK = 64;                          // rows prepared at once

template <int D>
__global__ void __launch_bounds__(32 * NW, 4) cache_weigh_block_kernel(const __grid_constant__ CacheWeighParams p) {
  constexpr int QW = D / 32;                       // 16-byte words of a lane's query operand
  __shared__ uint4 s_q[BLOCK / 8][QW][32];         // row tile, word, lane
  __shared__ float s_fx[BLOCK], s_ref[BLOCK], s_fac[BLOCK];
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t4 = lane % 4;
  // every gridDim.x-th of the line of (sequence, head, 128 keys that are there)
  int b = 0;
  unsigned seq0 = 0;
  auto units = [&](int i) { return (unsigned)((cache_len(c, i) + UNIT - 1) / UNIT) * (unsigned)c.Hkv; };
  for (unsigned u = blockIdx.x; line_find(c.B, units, u, b, seq0); u += gridDim.x) {
    const int len = cache_len(c, b);
    const unsigned per = (unsigned)(len + UNIT - 1) / UNIT;
    const int h = (int)((u - seq0) / per), cta0 = (int)((u - seq0) % per) * UNIT;
    const int key0 = cta0 + 32 * warp;
    const int q_len = cache_count(p.q_lens, b, p.T, c.err);
    const int G = p.Hq / c.Hkv;
    const int rows = G * q_len;
    auto row_at = [&](int r) -> long long { return ((long long)b * p.Hq + h * G + r % G) * p.T + r / G; };

    uint32_t ka[2][D / 16][4];
    float kx[2];
    int end[2];                                      // keys of each 16 that are there: below it
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = key0 + 16 * i;
      int pg = -1;
      if (key < len) pg = cache_page(c, c.table, b, key / c.page);
      end[i] = pg < 0 ? 0 : len;
      const long long ph = (long long)max(pg, 0) * c.Hkv + h;
      kx[i] = e8m0_value(*(c.ks + ph));
      const uint8_t* at = c.k + (ph * c.page + key % c.page + g) * D + 16 * t4;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint4 lo = *(reinterpret_cast<const uint4*>(at + 64 * x));
        const uint4 hi = *(reinterpret_cast<const uint4*>(at + 8 * D + 64 * x));
        const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, e[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          ka[i][4 * x + w][0] = e4m3x2_to_f16x2(a[w]);
          ka[i][4 * x + w][1] = e4m3x2_to_f16x2(e[w]);
          ka[i][4 * x + w][2] = e4m3x2_hi_to_f16x2(a[w]);
          ka[i][4 * x + w][3] = e4m3x2_hi_to_f16x2(e[w]);
        }
      }
    }
    float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};

    // tokens before these see none of the CTA's keys, of the warp's
    const int t_cta = p.causal ? max(0, cta0 - (len - q_len)) : 0;
    const int t_warp = p.causal ? max(0, key0 - (len - q_len)) : 0;
    const int first = (int)min((long long)rows, (long long)t_warp * G);
    for (int r0 = (int)min((long long)rows, (long long)t_cta * G) / BLOCK * BLOCK; r0 < rows; r0 += BLOCK) {
      QRaw<D> raw[BLOCK / 8 / NW];
      float lse[BLOCK / 8 / NW];
#pragma unroll
      for (int j = 0; j < BLOCK / 8 / NW; ++j) {
        const int r = r0 + 8 * (warp + j * NW) + g;
        raw[j].fetch(r < rows ? reinterpret_cast<const __nv_bfloat16*>(p.q) + row_at(r) * D : nullptr, t4);
        lse[j] = r < rows ? *(p.lse + row_at(r)) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < BLOCK / 8 / NW; ++j) {
        const int n = warp + j * NW;
        QFrag<D> q;
        const float e = raw[j].convert(q);
#pragma unroll
        for (int x = 0; x < QW; ++x)
          s_q[n][x][lane] = make_uint4(q.b[2 * x][0], q.b[2 * x][1], q.b[2 * x + 1][0], q.b[2 * x + 1][1]);
        if (t4 == 0) {
          float ref, fac;
          reference(lse[j], r0 + 8 * n + g < rows, ref, fac);
          s_ref[8 * n + g] = ref;
          s_fac[8 * n + g] = fac;
          s_fx[8 * n + g] = fac == 0.f ? 0.f : p.c2 * e;
        }
      }
      __syncthreads();
      if (key0 >= len) continue;                     // the sequence's last keys: this warp has none
      for (int n = max(0, (first - r0) / 8); n < BLOCK / 8 && r0 + 8 * n < rows; ++n) {
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
        for (int x = 0; x < QW; ++x) {
          const uint4 q = s_q[n][x][lane];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mma_16816(s[i], ka[i][2 * x][0], ka[i][2 * x][1], ka[i][2 * x][2], ka[i][2 * x][3], q.x, q.y);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mma_16816(s[i], ka[i][2 * x + 1][0], ka[i][2 * x + 1][1], ka[i][2 * x + 1][2], ka[i][2 * x + 1][3], q.z, q.w);
        }
        const float2 fx = *reinterpret_cast<const float2*>(&s_fx[8 * n + 2 * t4]);
        const float2 ref = *reinterpret_cast<const float2*>(&s_ref[8 * n + 2 * t4]);
        const float2 fac = *reinterpret_cast<const float2*>(&s_fac[8 * n + 2 * t4]);
        // the tile's first token sees the fewest keys
        const int r_min = r0 + 8 * n;
        const bool full = !p.causal || len - q_len + r_min / G + 1 >= key0 + 32;
        int vis[2] = {len, len};
        if (!full) {
#pragma unroll
          for (int j = 0; j < 2; ++j) vis[j] = len - q_len + (r_min + 2 * t4 + j) / G + 1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f0 = kx[i] * fx.x, f1 = kx[i] * fx.y;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = ex2_approx(fmaf(s[i][j], (j & 1) ? f1 : f0, (j & 1) ? -ref.y : -ref.x));
            if (full || key0 + 16 * i + g + 8 * (j >> 1) < vis[j & 1])
              w[i][j >> 1] = fmaf(e, (j & 1) ? fac.y : fac.x, w[i][j >> 1]);
          }
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
          p.w_out[at] = p.w_in[at] + (key < end[i] ? w[i][r] : 0.f);
        }
      }
  }
}

template <int D, int NT>
cudaError_t launch_few(const CacheWeighParams& p, cudaStream_t st) {
  constexpr int smem = WQueue<D, NT>::SMEM;
  auto k = p.c.page == 16 ? cache_weigh_kernel<D, NT, true> : cache_weigh_kernel<D, NT, false>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long all = (long long)units_of((long long)p.c.max_pages * p.c.page) * p.c.Hkv * p.c.B;
  const long long most = (long long)kSMs * weigh_ctas(NT);
  return launch_next(k, dim3((unsigned)(all < most ? all : most)), 32 * NW, smem, st, p);
}

}  // namespace

bool cache_weigh_fits(int B, int Hkv, int page, int max_pages) {
  return (long long)units_of((long long)max_pages * page) * Hkv * B < (1LL << 31);
}

cudaError_t launch_cache_weigh(const CacheWeighParams& p, cudaStream_t st) {
  const long long rows = (long long)(p.Hq / p.c.Hkv) * p.T;
  static_assert(WEIGH_MANY > 16, "below it the call makes the tensor map that the kernel for few rows reads");
  if (rows >= WEIGH_MANY) return launch_cache_weigh_rows(p, st);   // as the host decided on the tensor map
  if (rows <= 8) return p.c.d == 128 ? launch_few<128, 1>(p, st) : launch_few<64, 1>(p, st);
  if (rows <= 16) return p.c.d == 128 ? launch_few<128, 2>(p, st) : launch_few<64, 2>(p, st);
  const long long cap = (long long)p.c.max_pages * p.c.page;
  const long long all = (cap + UNIT - 1) / UNIT * p.c.Hkv * p.c.B, most = 4LL * kSMs;
  const dim3 grid((unsigned)(all < most ? all : most));
  return launch_next(p.c.d == 128 ? cache_weigh_block_kernel<128> : cache_weigh_block_kernel<64>, grid, 32 * NW, 0, st, p);
}

}  // namespace fa4
