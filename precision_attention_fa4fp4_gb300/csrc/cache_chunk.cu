// cache_chunk.cu -- attention of many query tokens per sequence (a chunk of a
// prompt) over the paged 8-bit cache, bf16 output.
//
//   s_j = scale q.k_j,  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the tensor cores (4 d flop per row and key): tcgen05.  The query
// heads of a kv head share its keys, so rows are (token, head of the group),
// token major; one CTA takes 256 rows of a kv head as two tiles A and B, which
// share every converted key tile.  16 warps:
//   0-3, 4-7  softmax of tile A, of tile B: one thread per row.  At the start it
//             brings its row of q to f16 under a power of two (a largest
//             magnitude in [2^7, 2^8): 2^-32 of it at most is lost); then exact
//             online softmax, P to f16 under a factor 2^15 into tensor memory
//             over the scores, o rescaled in tensor memory when the max grows.
//   8-11      conversion of the 128-key tiles: E4M3 -> f16 is exact, unscaled,
//             from the staged bytes into the swizzled layout that the products
//             read.
//   12        issues the products (kind::f16): S_X = Q_X K^T, O_X += P_X V.
//   13        looks the pages up and stages their bytes by bulk copies; writes
//             the tile's scales for the softmax.
// K's page scale multiplies the scores (folded into the exponent's FMA), V's
// goes into the exponent of P relative to the accumulator's own exponent, which
// is at most V_DOWN above the tile's largest: half of P's smallest f16 step is
// then 2^-36 of a tile's largest V.
// Tensor memory: S_A, S_B, O_A, O_B (512 columns at d = 128).  Two f16 stages of
// K and of V beside both query tiles leave room for one staged tile of bytes
// each: the copy of tile j + 1 runs while tile j is multiplied.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NTHREADS = 512;
constexpr int W_CONV = 8, W_MMA = 12, W_LOAD = 13;
// registers after setmaxnreg: 2 x 192 + 80 + 48 = 512 of 512 (x 128 threads)
constexpr int REG_SOFT = 192, REG_CONV = 80, REG_MISC = 48;
constexpr uint32_t TMEM_COLS = 512;
constexpr float P_BIAS = 15.f;
constexpr int V_DOWN = 4, V_LOWER = 80;      // as in the kernel for few rows
constexpr int METAS = 4;

// Scales of a 128-key tile, by groups of 16 keys.
struct alignas(16) Meta {
  float kx[8];
  int ev[8];                                 // V's exponents
  int ev_max;
  uint32_t absent;                           // groups without a page
};

template <int D>
struct SmemC {
  static constexpr int STAGES = 2;
  static constexpr int CH = F16_CHUNK;
  static constexpr int TILE = (D / 64) * CH;        // a tile of 128 f16 rows
  static constexpr int BYTES8 = 128 * D;            // a staged tile of codes
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  static constexpr int OFF_K8 = OFF_V + STAGES * TILE;
  static constexpr int OFF_V8 = OFF_K8 + BYTES8;
  static constexpr int OFF_META = OFF_V8 + BYTES8;
  static constexpr int OFF_BAR = (OFF_META + METAS * (int)sizeof(Meta) + 7) / 8 * 8;
  static constexpr int NBAR = 1 + 4 + 4 * STAGES + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;
  static constexpr uint32_t COL_O0 = 256;
  static_assert(COL_O0 + 2 * D <= TMEM_COLS, "tensor memory");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cache_chunk_kernel(const __grid_constant__ CacheFwdParams p) {
  using L = SmemC<D>;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t COL_O0 = L::COL_O0;
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int G = p.Hq / c.Hkv;
  const int len = cache_len(c, b);
  const int q_len = cache_count(p.q_lens, b, p.T, c.err);
  const int rows = G * q_len;
  const int r0 = (int)blockIdx.x * 2 * BM;
  if (r0 >= rows) return;
  // keys that the CTA's last token sees, in tiles
  const int t_last = (min(rows, r0 + 2 * BM) - 1) / G;
  const int see_last = p.causal ? max(0, min(len, len - q_len + t_last + 1)) : len;
  const int nt = (see_last + BN - 1) / BN;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k8_full = bars + 1;              // staged bytes
  uint64_t* k8_empty = bars + 2;
  uint64_t* v8_full = bars + 3;
  uint64_t* v8_empty = bars + 4;
  uint64_t* k_full = bars + 5;               // f16 tiles
  uint64_t* k_empty = k_full + STAGES;
  uint64_t* v_full = k_empty + STAGES;
  uint64_t* v_empty = v_full + STAGES;
  uint64_t* s_full = v_empty + STAGES;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* mma_done = o_done + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  Meta* metas = reinterpret_cast<Meta*>(smem + L::OFF_META);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    mbar_init(k8_full, 1); mbar_init(k8_empty, 4);
    mbar_init(v8_full, 1); mbar_init(v8_empty, 4);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&k_full[s], 4); mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4); mbar_init(&v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_done[x], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  if (warp >= W_MMA) {
    setmaxnreg_dec<REG_MISC>();
    if (warp == W_LOAD) {
      // ---------------------------------------------------------- pages
      const int log_p = 31 - __clz(c.page);
      int issued = 0;
      for (int j = 0; j < nt; ++j) {
        // lane i < 8: group i of 16 keys; the first lane of a page copies it
        const int key = j * BN + 16 * (lane & 7);
        const int lp = key >> log_p;
        int pg = -1;
        if (lane < 8 && key < len) pg = cache_page(c, c.table, b, lp);
        const long long ph = (long long)max(pg, 0) * c.Hkv + h;
        const float kx = e8m0_value(*(c.ks + ph));
        const int ev = (int)*(c.vs + ph) - 127;
        Meta& m = metas[j % METAS];
        if (j > 0 && !mbar_wait(k8_empty, (j - 1) & 1, abort_flag, c.err)) break;
        int top = pg >= 0 ? ev : -1000;
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        const uint32_t there = __ballot_sync(0xffffffffu, pg >= 0);
        if (lane < 8) {
          m.kx[lane] = kx;
          m.ev[lane] = ev;
          if (lane == 0) { m.ev_max = top; m.absent = ~there & 0xffu; }
        }
        __syncwarp();
        const bool copies = lane < 8 && pg >= 0 && ((16 * lane) & (c.page - 1)) == 0;
        const uint32_t bytes = (uint32_t)c.page * D;
        const uint32_t all = (uint32_t)__popc(__ballot_sync(0xffffffffu, copies)) * bytes;
        if (lane == 0) mbar_arrive_expect_tx(k8_full, all);
        __syncwarp();
        if (copies) bulk_load(smem + L::OFF_K8 + 16 * lane * D, c.k + (ph << log_p) * D, bytes, k8_full);
        if (j > 0 && !mbar_wait(v8_empty, (j - 1) & 1, abort_flag, c.err)) { issued = 2 * j + 1; break; }
        if (lane == 0) mbar_arrive_expect_tx(v8_full, all);
        __syncwarp();
        if (copies) bulk_load(smem + L::OFF_V8 + 16 * lane * D, c.v + (ph << log_p) * D, bytes, v8_full);
        issued = 2 * j + 2;
      }
      if (*abort_flag) {                     // what is still in flight lands first
        volatile int none = 0;
        const int nk = (issued + 1) / 2, nv = issued / 2;
        if (nk) mbar_wait(k8_full, (nk - 1) & 1, &none, c.err);
        if (nv) mbar_wait(v8_full, (nv - 1) & 1, &none, c.err);
      }
      __syncwarp();
    } else if (warp == W_MMA && nt > 0) {
      // ---------------------------------------------------------- products
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, false, false, false);
      const uint32_t idesc_o = idesc_f16(BM, D, false, false, true);   // A from TMEM, V MN-major
      const uint32_t sq = smem_u32(smem + L::OFF_Q);
      bool ok = mbar_wait(q_full, 0, abort_flag, c.err);
      tc_fence_after();
      auto issue_qk = [&](int x, int t) -> bool {
        const int st = t % STAGES;
        if (x == 0 && !mbar_wait(&k_full[st], (t / STAGES) & 1, abort_flag, c.err)) return false;
        tc_fence_after();
        const uint32_t sqx = sq + x * L::TILE;
        const uint32_t sk = smem_u32(smem + L::OFF_K + st * L::TILE);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * L::CH + (k % 4) * 32;
            mma_f16(tbase + 128 * x, make_sdesc(sqx + off, 16, 1024, SW_128B),
                    make_sdesc(sk + off, 16, 1024, SW_128B), idesc_s, k > 0);
          }
          mma_commit(&s_full[x]);
          if (x == 1) mma_commit(&k_empty[st]);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](int x, int t) -> bool {
        const int st = t % STAGES;
        if (x == 0 && !mbar_wait(&v_full[st], (t / STAGES) & 1, abort_flag, c.err)) return false;
        if (!mbar_wait(&p_full[x], t & 1, abort_flag, c.err)) return false;
        tc_fence_after();
        const uint32_t sv = smem_u32(smem + L::OFF_V + st * L::TILE);
        if (leader) {
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_f16_tmem_a(tbase + COL_O0 + D * x, tbase + 128 * x + 8 * k,
                           make_sdesc(sv + k * 16 * 128, L::CH, 1024, SW_128B), idesc_o, t > 0 || k > 0);
          mma_commit(&o_done[x]);
          if (x == 1) mma_commit(&v_empty[st]);
        }
        __syncwarp();
        return true;
      };
      // each tile's next Q K^T follows its own P V, so the pipe has read P_X
      // before it overwrites S_X
      if (ok) ok = issue_qk(0, 0) && issue_qk(1, 0);
      for (int j = 0; ok && j < nt; ++j) {
        if (!issue_pv(0, j)) { ok = false; break; }
        if (j + 1 < nt && !issue_qk(0, j + 1)) { ok = false; break; }
        if (!issue_pv(1, j)) { ok = false; break; }
        if (j + 1 < nt && !issue_qk(1, j + 1)) { ok = false; break; }
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int none = 0;
      mbar_wait(mma_done, 0, &none, c.err);
      __syncwarp();
    }
  } else if (warp >= W_CONV) {
    setmaxnreg_dec<REG_CONV>();
    // ------------------------------------------------------------ conversion
    constexpr int PARTS = D / 16;            // 16-byte words of a row
    constexpr int RSTEP = 128 / PARTS;       // rows at once
    const int tid = threadIdx.x - 32 * W_CONV;
    const int part = tid % PARTS, row0 = tid / PARTS;
    for (int j = 0; j < nt; ++j) {
      const int st = j % STAGES;
      const int left = len - j * BN;         // keys of the tile that are there
      const uint32_t parity = (j / STAGES - 1) & 1;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint64_t* full8 = kv ? v8_full : k8_full;
        uint64_t* empty8 = kv ? v8_empty : k8_empty;
        uint64_t* empty = kv ? &v_empty[st] : &k_empty[st];
        uint64_t* full = kv ? &v_full[st] : &k_full[st];
        if (!mbar_wait(full8, j & 1, abort_flag, c.err)) break;
        const uint8_t* from = smem + (kv ? L::OFF_V8 : L::OFF_K8) + row0 * D + part * 16;
        uint4 x[128 / RSTEP];
#pragma unroll
        for (int i = 0; i < 128 / RSTEP; ++i) x[i] = lds16(from + i * RSTEP * D);
        const uint32_t absent = metas[j % METAS].absent;
        // what is not there is zero: a score is masked by its place, but 0 * NaN
        // must not happen to P V
        if (left < BN || absent) {
#pragma unroll
          for (int i = 0; i < 128 / RSTEP; ++i) {
            const int row = row0 + i * RSTEP;
            if (row >= left || ((absent >> (row / 16)) & 1)) x[i] = make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty8);
        if (j >= STAGES && !mbar_wait(empty, parity, abort_flag, c.err)) break;
        uint8_t* tile = smem + (kv ? L::OFF_V : L::OFF_K) + st * L::TILE;
#pragma unroll
        for (int i = 0; i < 128 / RSTEP; ++i) store16<D>(tile, row0 + i * RSTEP, part, x[i]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      if (*abort_flag) break;
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int quad = warp & 3;
    const int rt = quad * 32 + lane;         // row within the tile
    const int r = r0 + x * BM + rt;
    const bool valid = r < rows;
    const int t = valid ? r / G : 0, gg = valid ? r % G : 0;
    const long long orow = ((long long)b * p.Hq + h * G + gg) * p.T + t;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_s = 128 * x, col_o = COL_O0 + D * x;
    const int vis = !valid ? 0 : p.causal ? max(0, min(len, len - q_len + t + 1)) : len;

    // the row of q: largest magnitude, then f16 under a power of two
    float f_row;
    {
      const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.q) + orow * D;
      f_row = p.c2 * exp2i(store_query_row<D, D / 8>(smem + L::OFF_Q + x * L::TILE, rt, valid ? src : nullptr));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }

    float m = -INFINITY, l = 0.f;
    int xo = -127;                           // o is in units of 2^xo
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      if (!mbar_wait(&s_full[x], j & 1, abort_flag, c.err)) { ok = false; break; }
      tc_fence_after();
      float s[4][32];
      {
        uint32_t v[4][32];
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_ld32(lane_base + col_s + 32 * g, v[g]);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          reg_fence32(v[g]);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[g][i] = __uint_as_float(v[g][i]);
        }
      }
      const Meta& meta = metas[j % METAS];
      const uint32_t absent = meta.absent;
      const int left = vis - j * BN;
      if (__any_sync(0xffffffffu, left < BN) || absent) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * g + i >= left || ((absent >> (2 * g + i / 16)) & 1)) s[g][i] = -INFINITY;
      }
      // exponent of V against the accumulator's
      const int ev_max = meta.ev_max;
      float back = 1.f;
      if (ev_max > -1000 && (ev_max > xo || ev_max < xo - V_DOWN)) {
        const int to = j == 0 ? ev_max : max(ev_max, xo - V_LOWER);
        back = pow2_any(xo - to);
        xo = to;
      }
      // max by groups of 16 keys, each with its K scale
      float F[8];
      {
        const float4 k0 = *reinterpret_cast<const float4*>(meta.kx), k1 = *reinterpret_cast<const float4*>(meta.kx + 4);
        F[0] = k0.x * f_row; F[1] = k0.y * f_row; F[2] = k0.z * f_row; F[3] = k0.w * f_row;
        F[4] = k1.x * f_row; F[5] = k1.y * f_row; F[6] = k1.z * f_row; F[7] = k1.w * f_row;
      }
      float m_new = m;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = s[g / 2][16 * (g % 2) + i];
        float top = fmax3(a[0], a[1], a[2]);
        float top2 = fmax3(a[3], a[4], a[5]);
        top = fmax3(top, a[6], a[7]);
        top2 = fmax3(top2, a[8], a[9]);
        top = fmax3(top, a[10], a[11]);
        top2 = fmax3(top2, a[12], a[13]);
        top = fmax3(top, a[14], a[15]);
        m_new = fmaxf(m_new, fmaxf(top, top2) * F[g]);
      }
      const float ref = (m_new == -INFINITY ? 0.f : m_new) - P_BIAS;
      float l_new = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t pk[16];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int gr = 2 * g + hf;
          const int d = min(0, max(meta.ev[gr] - xo, -100));
          const float Fg = F[gr], add = (float)d - ref;
          float2 ls = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = 16 * hf + 2 * i;
            const float2 e = ffma2(make_float2(s[g][k], s[g][k + 1]), make_float2(Fg, Fg), make_float2(add, add));
            const float2 pp = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            ls = fadd2(ls, pp);
            pk[8 * hf + i] = pack_f16x2(pp.x, pp.y);
          }
          l_new = fmaf(ls.x + ls.y, exp2i(-d), l_new);
        }
        tmem_st16(lane_base + col_s + 16 * g, pk);
      }
      const float alpha = (j == 0 || m_new == m) ? 1.f : ex2_approx(m - m_new);
      if (j > 0) {
        if (!mbar_wait(&o_done[x], (j - 1) & 1, abort_flag, c.err)) { ok = false; break; }
        tc_fence_after();
        const float by = alpha * back;
        if (__any_sync(0xffffffffu, by != 1.f)) {
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            uint32_t ov[32];
            tmem_ld32(lane_base + col_o + 32 * g, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 y = fmul2(make_float2(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])), make_float2(by, by));
              ov[i] = __float_as_uint(y.x);
              ov[i + 1] = __float_as_uint(y.y);
            }
            tmem_st32(lane_base + col_o + 32 * g, ov);
          }
        }
      }
      l = fmaf(alpha, l, l_new);
      m = m_new;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
    }
    if (ok && (nt == 0 || mbar_wait(&o_done[x], (nt - 1) & 1, abort_flag, c.err))) {
      tc_fence_after();
      // a row without keys: whatever the accumulator holds counts for nothing
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l, unit = pow2_any(xo);
#pragma unroll 1
      for (int g = 0; g < D / 32; ++g) {
        uint32_t v[32];
        tmem_ld32(lane_base + col_o + 32 * g, v);
        tmem_ld_wait();
        reg_fence32(v);
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + orow * D + 32 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = none ? 0.f : __uint_as_float(v[8 * i + 2 * e]) * unit * inv;
              const float z = none ? 0.f : __uint_as_float(v[8 * i + 2 * e + 1]) * unit * inv;
              const __nv_bfloat162 y = __floats2bfloat162_rn(a, z);
              w[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (valid && p.lse) p.lse[orow] = none ? -INFINITY : fmaf(m - P_BIAS, 0.69314718f, logf(l));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

template <int D>
cudaError_t launch(const CacheFwdParams& p, cudaStream_t st) {
  auto k = cache_chunk_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemC<D>::BYTES);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)(p.Hq / p.c.Hkv) * p.T;
  const dim3 grid((unsigned)((rows + 2 * BM - 1) / (2 * BM)), (unsigned)p.c.Hkv, (unsigned)p.c.B);
  return launch_next(k, grid, NTHREADS, SmemC<D>::BYTES, st, p);
}

}  // namespace

cudaError_t launch_cache_chunk(const CacheFwdParams& p, cudaStream_t st) {
  return p.c.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace fa4
