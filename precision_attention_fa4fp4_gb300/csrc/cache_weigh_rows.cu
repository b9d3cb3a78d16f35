// cache_weigh_rows.cu -- the attention weight that every cached token received,
// for many query rows (a chunk of a prompt):
//   out[j] = in[j] + sum over rows r that see j of  e^(scale q_r.k_j - lse_r)
//
// 2 d flop and one exponential per row and key: tcgen05 for the products, with
// the rows of q as rows of the accumulator (S = Q K^T).  A thread of the sums
// owns a row, whose constants stay in its registers, and keeps a sum for each of
// 32 keys while the rows go by; the rows' sums meet once, at the end of a key
// tile.  (With the keys as rows nothing has to meet, but every warp reads every
// row's constants from shared memory: 36 us where this takes 28.)
//
// A first kernel brings the rows to f16 under a power of two, in the order
// (token, head) and with what the sums need of each, into the workspace: every
// CTA of the second reads them all, and reading and converting bf16 rows there
// took 4.9 us per 128 rows (91 us for 2 x 256 tokens over 4096) against the 0.6
// us in which they are multiplied and summed.
//
// The second kernel: one CTA per SM goes through tiles of 128 keys of a kv head,
// converted to f16 once (exactly) while the tile before is at work, and walks
// over the rows 128 at a time.  23 warps:
//   0-15  sums: rows 32 (warp % 4).., keys 32 (warp / 4).. of a tile; four score
//         tiles in tensor memory, so that the products run ahead.
//   16-19 conversion of K.
//   20    issues the products.
//   21    loads the rows by TMA, and their constants by bulk copies.
//   22    looks the pages up and stages K's bytes by bulk copies (the conversion's
//         own loads, page after table after length, took 4 us a key tile).
// 2 x 256 tokens over 4096, 32 / 8 heads of 128: 28.5 us (5 of them the first
// kernel's), 0.59 PFLOP/s.  Latency bounds it: 512 key tiles are 3.4 an SM, so
// four rounds of eight row tiles, and of the 1500 clocks of a step 470 are sums.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NTHREADS = 736;
constexpr int W_CONV = 16, W_MMA = 20, W_LOAD = 21, W_PAGE = 22;
constexpr uint32_t TMEM_COLS = 512;
constexpr int QS = 3, KS = 2, SB = 4;        // tiles of rows, of keys, of scores
constexpr int KX = 16;                       // key tiles whose scales are kept: they are looked up at
                                             // most 2 KS + SB tiles ahead of the sums
constexpr int METAS = 8;                     // rows are loaded at most QS + SB tiles ahead of the sums

// What the sums need of 128 rows.
struct alignas(16) RowMeta {
  float fx[128], nref[128], fac[128];        // factor of a score; -reference; what its rounding makes up for
  int vis[128];                              // keys that it sees
};

template <int D>
struct SmemW {
  static constexpr int TILE = (D / 64) * F16_CHUNK;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = KS * TILE;
  static constexpr int OFF_META = OFF_Q + QS * TILE;
  static constexpr int OFF_K8 = OFF_META + METAS * (int)sizeof(RowMeta);   // staged codes
  static constexpr int OFF_KX = OFF_K8 + KS * 128 * D;       // [KX][8] scales of 16 keys; 0: no page
  static constexpr int OFF_SUM = OFF_KX + KX * 8 * 4;        // [2][4][128] sums of 32 rows
  static constexpr int OFF_BAR = OFF_SUM + 2 * 4 * 128 * 4;
  static constexpr int NBAR = 4 * KS + 2 * QS + 2 * SB + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// Workspace of one (sequence, kv head): its rows in tiles of 128, zeros behind
// the last, then the tiles' constants.
__host__ __device__ inline int row_tiles(int G, int T) { return (int)(((long long)G * T + 127) / 128); }

// D / 8 lanes a row; rows by grid x, (sequence, kv head) by y and z.
constexpr int NT_PREP = 256;
template <int D>
__global__ void __launch_bounds__(NT_PREP) cache_rows_kernel(const __grid_constant__ CacheWeighParams p) {
  constexpr int LANES = D / 8;
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int G = p.Hq / c.Hkv, tiles = row_tiles(G, p.T);
  const int part = threadIdx.x % LANES, r = blockIdx.x * (NT_PREP / LANES) + threadIdx.x / LANES;
  const int len = cache_len(c, b), q_len = cache_count(p.q_lens, b, p.T, c.err);
  const int t = r / G, gg = r % G;
  const bool valid = t < q_len;
  const long long at = ((long long)b * p.Hq + h * G + gg) * p.T + t;
  uint4 w = make_uint4(0, 0, 0, 0);
  float lse = -INFINITY;                             // a row that adds nothing
  if (valid) {
    w = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) + at * D)[part];
    lse = p.lse[at];
  }
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = max(amax, max((u[k] << 16) & 0x7fffffffu, u[k] & 0x7fff0000u));
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int E = (int)(amax >> 23);
  const int e = (E == 0 || E == 255) ? 0 : max(-120, min(120, E - 134));   // as in QRaw
  const float down = exp2i(-e);
  uint32_t z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    z[k] = pack_f16x2(__uint_as_float(u[k] << 16) * down, __uint_as_float(u[k] & 0xffff0000u) * down);
  const long long bh = (long long)b * c.Hkv + h;
  reinterpret_cast<uint4*>(p.rows + ((bh * tiles * 128 + r) * D) * 2)[part] = make_uint4(z[0], z[1], z[2], z[3]);
  if (part == 0) {
    RowMeta& m = reinterpret_cast<RowMeta*>(p.metas)[bh * tiles + r / 128];
    const int i = r % 128;
    float ref, fac;
    reference(lse, true, ref, fac);
    m.fx[i] = fac == 0.f ? 0.f : p.c2 * exp2i(e);
    m.nref[i] = -ref;
    m.fac[i] = fac;
    m.vis[i] = p.causal ? len - q_len + t + 1 : len;
  }
}

// A tile of 128 keys and the row tiles that see any of them.  The tiles that hold
// keys form a line of (sequence, kv head, tile); a CTA takes every gridDim.x-th.
struct KeyTile {
  int b = 0, h, key0, len = 0, q_len = 0, j0, nt;
  unsigned seq0 = 0, end = 0;                // the sequence's part of the line
  static FA4_DEV unsigned of(const CacheWeighParams& p, int b) {
    return (unsigned)((cache_len(p.c, b) + 127) / 128) * (unsigned)p.c.Hkv;
  }
  // goes on to tile `at` of the line, if there is one (whole warp)
  FA4_DEV bool go(const CacheWeighParams& p, int G, unsigned at) {
    if (at >= end) {
      if (!line_find(p.c.B, [&](int i) { return of(p, i); }, at, b, seq0)) return false;
      len = cache_len(p.c, b);
      q_len = cache_count(p.q_lens, b, p.T, p.c.err);
      end = seq0 + of(p, b);
    }
    const unsigned tiles = (unsigned)max((len + 127) / 128, 1);
    h = (int)((at - seq0) / tiles);
    key0 = (int)((at - seq0) - (unsigned)h * tiles) * 128;
    const int rows = G * q_len;
    // tokens before this one see none of the keys
    const int t_first = p.causal ? max(0, key0 - (len - q_len)) : 0;
    j0 = (int)min((long long)rows, (long long)t_first * G) / 128;
    nt = max(0, (rows + 127) / 128 - j0);
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cache_weigh_rows_kernel(const __grid_constant__ CacheWeighParams p) {
  using L = SmemW<D>;
  grid_start();
  const CacheView& c = p.c;
  const int G = p.Hq / c.Hkv;
  const int r_tiles = row_tiles(G, p.T);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_empty = k_full + KS;
  uint64_t* k8_full = k_empty + KS;
  uint64_t* k8_empty = k8_full + KS;
  uint64_t* q_full = k8_empty + KS;
  uint64_t* q_empty = q_full + QS;
  uint64_t* s_full = q_empty + QS;
  uint64_t* s_empty = s_full + SB;
  uint64_t* mma_done = s_empty + SB;
  float* s_kx = reinterpret_cast<float*>(smem + L::OFF_KX);
  RowMeta* metas = reinterpret_cast<RowMeta*>(smem + L::OFF_META);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 4); mbar_init(&k_empty[s], 1);
      mbar_init(&k8_full[s], 1); mbar_init(&k8_empty[s], 4);
    }
    for (int s = 0; s < QS; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < SB; ++s) { mbar_init(&s_full[s], 1); mbar_init(&s_empty[s], 16); }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  grid_wait();
  KeyTile k;                                 // (fewer than 2^31 of them: the call checks)

  if (warp == W_MMA) {
    // -------------------------------------------------------------- products
    const bool leader = elect_one();
    const uint32_t idesc = idesc_f16(128, 128, false, false, false);
    bool ok = true;
    int n = 0, t = 0;                        // key tiles and row tiles so far
    for (unsigned i = blockIdx.x; ok && k.go(p, G, i); i += gridDim.x) {
      if (k.nt == 0) continue;
      const uint32_t sk = smem_u32(smem + L::OFF_K + n % KS * L::TILE);
      ok = mbar_wait(&k_full[n % KS], (n / KS) & 1, abort_flag, c.err);
      for (int j = 0; ok && j < k.nt; ++j, ++t) {
        const int qs = t % QS, sb = t % SB;
        ok = mbar_wait(&q_full[qs], (t / QS) & 1, abort_flag, c.err) &&
             (t < SB || mbar_wait(&s_empty[sb], (t / SB - 1) & 1, abort_flag, c.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sq = smem_u32(smem + L::OFF_Q + qs * L::TILE);
        if (leader) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = (x / 4) * F16_CHUNK + (x % 4) * 32;
            mma_f16(tbase + 128 * sb, make_sdesc(sq + off, 16, 1024, SW_128B), make_sdesc(sk + off, 16, 1024, SW_128B),
                    idesc, x > 0);
          }
          mma_commit(&s_full[sb]);
          mma_commit(&q_empty[qs]);
          if (j + 1 == k.nt) mma_commit(&k_empty[n % KS]);
        }
        __syncwarp();
      }
      ++n;
    }
    if (leader) mma_commit(mma_done);
    __syncwarp();
    volatile int none = 0;
    mbar_wait(mma_done, 0, &none, c.err);
    __syncwarp();
  } else if (warp == W_LOAD) {
    // -------------------------------------------------------------- rows of q
    if (lane == 0) tma_prefetch_desc(&p.tm_q);
    bool ok = true;
    int t = 0;
    for (unsigned i = blockIdx.x; ok && k.go(p, G, i); i += gridDim.x) {
      const long long first = ((long long)k.b * c.Hkv + k.h) * r_tiles + k.j0;
      for (int j = 0; j < k.nt; ++j, ++t) {
        const int s = t % QS;
        ok = t < QS || mbar_wait(&q_empty[s], (t / QS - 1) & 1, abort_flag, c.err);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[s], L::TILE + (uint32_t)sizeof(RowMeta));
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(smem + L::OFF_Q + s * L::TILE + x * F16_CHUNK, &p.tm_q, &q_full[s], 64 * x,
                        (int)((first + j) * 128), 0);
          bulk_load(&metas[t % METAS], reinterpret_cast<const RowMeta*>(p.metas) + first + j, (uint32_t)sizeof(RowMeta),
                    &q_full[s]);
        }
        __syncwarp();
      }
    }
    if (*abort_flag) {                               // what is still in flight lands first
      volatile int none = 0;
      for (int j = max(0, t - QS); j < t; ++j) mbar_wait(&q_full[j % QS], (j / QS) & 1, &none, c.err);
    }
    __syncwarp();
  } else if (warp == W_PAGE) {
    // -------------------------------------------------------------- pages
    const int log_p = 31 - __clz(c.page);
    bool ok = true;
    int n = 0;
    for (unsigned i = blockIdx.x; k.go(p, G, i); i += gridDim.x) {
      if (k.nt == 0) continue;
      // lane i < 8: group i of 16 keys; the first lane of a page copies it
      const int key = k.key0 + 16 * (lane & 7);
      int pg = -1;
      if (lane < 8 && key < k.len) pg = cache_page(c, c.table, k.b, key >> log_p);
      const long long ph = (long long)max(pg, 0) * c.Hkv + k.h;
      const float kx = pg >= 0 ? e8m0_value(*(c.ks + ph)) : 0.f;
      ok = n < KS || mbar_wait(&k8_empty[n % KS], (n / KS - 1) & 1, abort_flag, c.err);
      if (!ok) break;
      if (lane < 8) s_kx[n % KX * 8 + lane] = kx;
      __syncwarp();
      const bool copies = lane < 8 && pg >= 0 && ((16 * lane) & (c.page - 1)) == 0;
      const uint32_t bytes = (uint32_t)c.page * D;
      const uint32_t all = (uint32_t)__popc(__ballot_sync(0xffffffffu, copies)) * bytes;
      if (lane == 0) mbar_arrive_expect_tx(&k8_full[n % KS], all);
      __syncwarp();
      if (copies)
        bulk_load(smem + L::OFF_K8 + n % KS * 128 * D + 16 * lane * D, c.k + (ph << log_p) * D, bytes, &k8_full[n % KS]);
      __syncwarp();
      ++n;
    }
    if (*abort_flag) {                               // what is still in flight lands first
      volatile int none = 0;
      for (int j = max(0, n - KS); j < n; ++j) mbar_wait(&k8_full[j % KS], (j / KS) & 1, &none, c.err);
    }
    __syncwarp();
  } else if (warp >= W_CONV) {
    // -------------------------------------------------------------- K
    constexpr int PARTS = D / 16, RSTEP = 128 / PARTS, N = 128 / RSTEP;
    const int tid = threadIdx.x - 32 * W_CONV;
    const int part = tid % PARTS, row0 = tid / PARTS;
    bool ok = true;
    int n = 0;
    for (unsigned i = blockIdx.x; ok && k.go(p, G, i); i += gridDim.x) {
      if (k.nt == 0) continue;
      ok = mbar_wait(&k8_full[n % KS], (n / KS) & 1, abort_flag, c.err);
      if (!ok) break;
      const uint8_t* from = smem + L::OFF_K8 + n % KS * 128 * D + row0 * D + part * 16;
      uint4 x[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int row = row0 + e * RSTEP;
        x[e] = lds16(from + e * RSTEP * D);
        // what is not there is zero
        if (k.key0 + row >= k.len || s_kx[n % KX * 8 + row / 16] == 0.f) x[e] = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&k8_empty[n % KS]);
      ok = n < KS || mbar_wait(&k_empty[n % KS], (n / KS - 1) & 1, abort_flag, c.err);
      if (!ok) break;
      uint8_t* tile = smem + L::OFF_K + n % KS * L::TILE;
#pragma unroll
      for (int e = 0; e < N; ++e) store16<D>(tile, row0 + e * RSTEP, part, x[e]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[n % KS]);
      ++n;
    }
  } else {
    // -------------------------------------------------------------- sums
    const int quad = warp & 3, part = warp >> 2;
    const int row = 32 * quad + lane;
    const uint32_t base = tbase + ((uint32_t)(32 * quad) << 16) + 32 * part;
    float* s_sum = reinterpret_cast<float*>(smem + L::OFF_SUM);
    // after a wait that ran out a warp computes no more, but comes to the barriers
    bool ok = true;
    int n = 0, t = 0, turn = 0;
    for (unsigned i = blockIdx.x; k.go(p, G, i); i += gridDim.x) {
      const long long bh = (long long)k.b * c.Hkv + k.h;
      const int my_key = k.key0 + 32 * part + lane;    // of the quadrant that writes the sums
      float before = 0.f;
      if (quad == 0 && my_key < k.len) before = p.w_in[bh * c.max_pages * c.page + my_key];
      float2 kx = make_float2(0.f, 0.f);
      float2 acc[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = make_float2(0.f, 0.f);
      if (k.nt > 0) {
        for (int j = 0; ok && j < k.nt; ++j, ++t) {
          const int sb = t % SB;
          ok = mbar_wait(&s_full[sb], (t / SB) & 1, abort_flag, c.err);
          if (!ok) break;
          tc_fence_after();
          if (j == 0) kx = *reinterpret_cast<const float2*>(s_kx + n % KX * 8 + 2 * part);
          const RowMeta& m = metas[t % METAS];
          const float fx = m.fx[row], nref = m.nref[row], fac = m.fac[row];
          const float2 nr = make_float2(nref, nref), fc = make_float2(fac, fac);
          const int left = m.vis[row] - k.key0 - 32 * part;      // keys of these that the row sees
          const bool all = __all_sync(0xffffffffu, left >= 32);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {                       // 16 keys, of one scale
            uint32_t v[16];
            tmem_ld16(base + 128 * sb + 16 * hf, v);
            const float F = fx * (hf ? kx.y : kx.x);
            const float2 f2 = make_float2(F, F);
            tmem_ld_wait();
            reg_fence16(v);
            if (hf) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_empty[sb]);
            }
            auto add = [&](bool full) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 y = ffma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), f2, nr);
                const float2 sum = ffma2(make_float2(ex2_approx(y.x), ex2_approx(y.y)), fc, acc[8 * hf + e]);
                // (a row that does not see the key must not reach it as 0 * NaN either)
                if (full || 16 * hf + 2 * e < left) acc[8 * hf + e].x = sum.x;
                if (full || 16 * hf + 2 * e + 1 < left) acc[8 * hf + e].y = sum.y;
              }
            };
            if (all) add(true);
            else add(false);
          }
        }
        ++n;
      }
      // the 32 rows' sums: lanes hand half of their keys over, five times; lane i
      // then has key i's
      float a[32];
#pragma unroll
      for (int e = 0; e < 16; ++e) { a[2 * e] = acc[e].x; a[2 * e + 1] = acc[e].y; }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int e = 0; e < o; ++e) {
          const float mine = up ? a[e + o] : a[e], theirs = up ? a[e] : a[e + o];
          a[e] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
        }
      }
      float* sums = s_sum + (turn++ & 1) * 512 + 32 * part + lane;
      sums[128 * quad] = a[0];
      named_bar(1 + part, 128);
      if (quad == 0 && my_key < k.len && !*abort_flag) {
        const float sum = (a[0] + sums[128]) + (sums[256] + sums[384]);
        // a page that is not there adds nothing
        p.w_out[bh * c.max_pages * c.page + my_key] = before + ((lane < 16 ? kx.x : kx.y) == 0.f ? 0.f : sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

template <int D>
cudaError_t launch(const CacheWeighParams& p, cudaStream_t st) {
  const int tiles = row_tiles(p.Hq / p.c.Hkv, p.T);
  const unsigned H = (unsigned)p.c.Hkv, B = (unsigned)p.c.B;
  cudaError_t e = launch_next(cache_rows_kernel<D>, dim3((unsigned)(tiles * 128 / (NT_PREP / (D / 8))), H, B), NT_PREP,
                              0, st, p);
  if (e != cudaSuccess) return e;
  auto k = cache_weigh_rows_kernel<D>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemW<D>::BYTES);
  if (e != cudaSuccess) return e;
  const long long items = ((long long)p.c.max_pages * p.c.page + 127) / 128 * H * B;
  return launch_next(k, dim3((unsigned)(items < kSMs ? items : kSMs)), NTHREADS, SmemW<D>::BYTES, st, p);
}

}  // namespace

// Bytes of the rows (the constants lie behind them) and of both.
size_t cache_weigh_rows_bytes(int B, int Hq, int Hkv, int T, int d, size_t* all) {
  const size_t tiles = (size_t)B * Hkv * row_tiles(Hq / Hkv, T);
  const size_t rows = tiles * 128 * d * 2;
  if (all) *all = rows + tiles * sizeof(RowMeta);
  return rows;
}

cudaError_t launch_cache_weigh_rows(const CacheWeighParams& p, cudaStream_t st) {
  return p.c.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace fa4
