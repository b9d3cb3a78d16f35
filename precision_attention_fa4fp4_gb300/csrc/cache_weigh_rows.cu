// cache_weigh_rows.cu -- the attention weight that every cached token received,
// for many query rows (a chunk of a prompt):
//   out[j] = in[j] + sum over rows r that see j of  e^(scale q_r.k_j - lse_r)
//
// 2 d flop and one exponential per row and key: tcgen05 for the products, with
// the keys as rows of the accumulator (S^T = K Q^T), so that a thread of the
// epilogue owns a key and its sum runs along its own tensor-memory lane: no
// exchange between threads until the end.
//
// A first kernel brings the rows to f16 under a power of two, in the order
// (token, head) and with what the epilogue needs of each, into the workspace:
// every CTA of the second reads them all, and reading and converting bf16 rows
// there took 4.9 us per 128 rows (91 us for 2 x 256 tokens over 4096) against
// the 0.6 us in which they are multiplied and summed.
//
// The second kernel: one CTA takes 128 keys of a kv head, converted to f16 once
// (exactly), and walks over the rows 128 at a time, two CTAs to an SM.  14 warps:
//   0-7   epilogue: lane quadrant warp % 4 (32 keys), columns 64 (warp / 4)..;
//         two score tiles in tensor memory, so the products of one run while the
//         other is summed.
//   8-11  conversion of K.
//   12    issues the products.
//   13    loads the rows by TMA, and their constants by bulk copies.
// 2 x 256 tokens over 4096, 32 / 8 heads of 128: 36 us (5 of them the first
// kernel's), 0.46 PFLOP/s.  The sums bound it: an exponential per score, and the
// rows' constants read from shared memory by every warp.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NTHREADS = 448;
constexpr int W_CONV = 8, W_MMA = 12, W_LOAD = 13;
constexpr uint32_t TMEM_COLS = 256;
constexpr int METAS = 6;                     // rows are loaded at most four tiles ahead of the sums

// What the epilogue needs of 128 rows; pairs of columns side by side.
struct alignas(16) RowMeta {
  float4 fx_ref[64];                         // fx, fx', -ref, -ref'
  float2 fac[64];
  int vis[128];
};

template <int D>
struct SmemW {
  static constexpr int TILE = (D / 64) * F16_CHUNK;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = TILE;
  static constexpr int OFF_META = OFF_Q + 2 * TILE;
  static constexpr int OFF_BAR = OFF_META + METAS * (int)sizeof(RowMeta);
  static constexpr int NBAR = 1 + 2 + 2 + 2 + 2;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_SUM = OFF_MISC + 24;
  static constexpr int BYTES = OFF_SUM + 128 * 4 + 1024;
  static_assert(2 * (BYTES + 1024) <= 228 * 1024, "two CTAs to an SM");
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
    float* fr = reinterpret_cast<float*>(&m.fx_ref[i / 2]) + i % 2;
    fr[0] = fac == 0.f ? 0.f : p.c2 * exp2i(e);
    fr[2] = -ref;
    reinterpret_cast<float*>(m.fac)[i] = fac;
    m.vis[i] = p.causal ? len - q_len + t + 1 : len;
  }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 2) cache_weigh_rows_kernel(const __grid_constant__ CacheWeighParams p) {
  using L = SmemW<D>;
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int len = cache_len(c, b);
  const int key0 = blockIdx.x * 128;
  if (key0 >= len) return;
  const int q_len = cache_count(p.q_lens, b, p.T, c.err);
  const int G = p.Hq / c.Hkv;
  const int rows = G * q_len;
  // tokens before this one see none of the CTA's keys
  const int t_first = p.causal ? max(0, key0 - (len - q_len)) : 0;
  const int j0 = (int)min((long long)rows, (long long)t_first * G) / 128;
  const int nt = max(0, (rows + 127) / 128 - j0);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = k_full + 1;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* s_empty = s_full + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  uint64_t* mma_done = reinterpret_cast<uint64_t*>(smem + L::OFF_MISC + 8);
  RowMeta* metas = reinterpret_cast<RowMeta*>(smem + L::OFF_META);
  float* s_sum = reinterpret_cast<float*>(smem + L::OFF_SUM);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(k_full, 4);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 8);
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

  float sum = 0.f, before = 0.f;             // of a key; what it had
  bool there = false;                        // its page
  if (warp == W_MMA) {
    // -------------------------------------------------------------- products
    if (nt > 0) {
      const bool leader = elect_one();
      const uint32_t idesc = idesc_f16(128, 128, false, false, false);
      const uint32_t sk = smem_u32(smem + L::OFF_K);
      bool ok = mbar_wait(k_full, 0, abort_flag, c.err);
      for (int j = 0; ok && j < nt; ++j) {
        const int s = j & 1;
        const uint32_t phase = (j >> 1) & 1;
        if (!mbar_wait(&q_full[s], phase, abort_flag, c.err)) break;
        if (j >= 2 && !mbar_wait(&s_empty[s], phase ^ 1, abort_flag, c.err)) break;
        tc_fence_after();
        const uint32_t sq = smem_u32(smem + L::OFF_Q + s * L::TILE);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * F16_CHUNK + (k % 4) * 32;
            mma_f16(tbase + 128 * s, make_sdesc(sk + off, 16, 1024, SW_128B), make_sdesc(sq + off, 16, 1024, SW_128B),
                    idesc, k > 0);
          }
          mma_commit(&s_full[s]);
          mma_commit(&q_empty[s]);
        }
        __syncwarp();
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int none = 0;
      mbar_wait(mma_done, 0, &none, c.err);
      __syncwarp();
    }
  } else if (warp == W_LOAD) {
    // -------------------------------------------------------------- rows of q
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_q);
      const long long bh = (long long)b * c.Hkv + h;
      const int tiles = row_tiles(G, p.T);
      int issued = 0;
      for (int j = 0; j < nt; ++j) {
        const int s = j & 1;
        if (j >= 2 && !mbar_wait(&q_empty[s], ((j >> 1) & 1) ^ 1, abort_flag, c.err)) break;
        mbar_arrive_expect_tx(&q_full[s], L::TILE + (uint32_t)sizeof(RowMeta));
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d(smem + L::OFF_Q + s * L::TILE + x * F16_CHUNK, &p.tm_q, &q_full[s], 64 * x,
                      (int)((bh * tiles + j0 + j) * 128), 0);
        bulk_load(&metas[j % METAS], reinterpret_cast<const RowMeta*>(p.metas) + bh * tiles + j0 + j,
                  (uint32_t)sizeof(RowMeta), &q_full[s]);
        issued = j + 1;
      }
      if (*abort_flag) {                             // what is still in flight lands first
        volatile int none = 0;
        for (int j = max(0, issued - 2); j < issued; ++j) mbar_wait(&q_full[j & 1], (j >> 1) & 1, &none, c.err);
      }
    }
    __syncwarp();
  } else if (warp >= W_CONV) {
    // -------------------------------------------------------------- K
    constexpr int PARTS = D / 16, RSTEP = 128 / PARTS;
    const int tid = threadIdx.x - 32 * W_CONV;
    const int part = tid % PARTS;
    constexpr int N = 128 / RSTEP;
    int pg[N];                               // all rows' loads in flight, one after the other's pages
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int key = key0 + tid / PARTS + i * RSTEP;
      pg[i] = key < len ? cache_page(c, c.table, b, key / c.page) : -1;
    }
    uint4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int key = key0 + tid / PARTS + i * RSTEP;
      x[i] = make_uint4(0, 0, 0, 0);         // what is not there is zero
      if (pg[i] >= 0)
        x[i] = reinterpret_cast<const uint4*>(c.k + (((long long)pg[i] * c.Hkv + h) * c.page + key % c.page) * D)[part];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) store16<D>(smem + L::OFF_K, tid / PARTS + i * RSTEP, part, x[i]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(k_full);
  } else {
    // -------------------------------------------------------------- sums
    const int quad = warp & 3, half = warp >> 2;
    const int key = key0 + 32 * quad + lane;
    float kx = 0.f;
    if (key < len) {
      const int pg = cache_page(c, c.table, b, key / c.page);
      there = pg >= 0;
      if (there) kx = e8m0_value(c.ks[(long long)pg * c.Hkv + h]);
      if (half == 0) before = p.w_in[((long long)b * c.Hkv + h) * c.max_pages * c.page + key];
    }
    const float2 kx2 = make_float2(kx, kx);
    const uint32_t base = tbase + ((uint32_t)(32 * quad) << 16) + 64 * half;
    float2 acc = make_float2(0.f, 0.f);
    for (int j = 0; j < nt; ++j) {
      const int s = j & 1;
      if (!mbar_wait(&s_full[s], (j >> 1) & 1, abort_flag, c.err)) break;
      tc_fence_after();
      const RowMeta& m = metas[j % METAS];
      const int r0 = (j0 + j) * 128;
      // the tile's first token sees the fewest keys
      const bool full = !p.causal || len - q_len + r0 / G + 1 >= key0 + 128;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t v[32];
        tmem_ld32(base + 128 * s + 32 * g, v);
        tmem_ld_wait();
        reg_fence32(v);
        if (g == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[s]);
        }
        const int c0 = 32 * half + 16 * g;           // pairs of columns
        if (full) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 fr = m.fx_ref[c0 + i];
            const float2 x = fmul2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), kx2);
            const float2 y = ffma2(x, make_float2(fr.x, fr.y), make_float2(fr.z, fr.w));
            acc = ffma2(make_float2(ex2_approx(y.x), ex2_approx(y.y)), m.fac[c0 + i], acc);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 fr = m.fx_ref[c0 + i];
            const float2 x = fmul2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), kx2);
            const float2 y = ffma2(x, make_float2(fr.x, fr.y), make_float2(fr.z, fr.w));
            const int2 vis = reinterpret_cast<const int2*>(m.vis)[c0 + i];
            acc = ffma2(make_float2(key < vis.x ? ex2_approx(y.x) : 0.f, key < vis.y ? ex2_approx(y.y) : 0.f),
                        m.fac[c0 + i], acc);
          }
        }
      }
    }
    sum = acc.x + acc.y;
    if (half == 1) s_sum[32 * quad + lane] = sum;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
  const int key = key0 + (int)threadIdx.x;
  if (warp < 4 && key < len) {
    const long long at = ((long long)b * c.Hkv + h) * c.max_pages * c.page + key;
    // a page that is not there adds nothing
    if (!*abort_flag) p.w_out[at] = before + (there ? sum + s_sum[threadIdx.x] : 0.f);
  }
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
  const long long cap = (long long)p.c.max_pages * p.c.page;
  return launch_next(k, dim3((unsigned)((cap + 127) / 128), H, B), NTHREADS, SmemW<D>::BYTES, st, p);
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
