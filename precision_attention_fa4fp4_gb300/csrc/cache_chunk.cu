// cache_chunk.cu -- attention of many query tokens per sequence (a chunk of a
// prompt) over the paged 8-bit cache, bf16 output.
//
//   s_j = scale q.k_j,  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the tensor cores (4 d flop per row and key): tcgen05.  The query
// heads of a kv head share its keys, so rows are (token, head of the group),
// token major; a block is 256 rows of a kv head as two tiles A and B, which share
// every converted key tile (B is left out where it has no rows).  All blocks'
// key tiles form a line that is cut into equal shares, one per SM; a block that
// is cut leaves partials in the workspace, and the last CTA to do so joins them
// (whole blocks instead of shares: 256 blocks on 152 SMs took two rounds, 270
// against 257 us).  16 warps:
//   0-3, 4-7  softmax of tile A, of tile B: one thread per row.  At the start it
//             brings its row of q to f16 under a power of two (a largest
//             magnitude in [2^7, 2^8): 2^-32 of it at most is lost); then exact
//             online softmax, P to f16 into tensor memory over the scores.  The
//             reference of a row's exponents follows its maximum only when that
//             has grown by 2^M_UP: o in tensor memory is rescaled in a few tiles
//             instead of most (10 us of 257).
//   8-11      conversion of the 128-key tiles: E4M3 -> f16 is exact, unscaled,
//             from the staged bytes into the swizzled layout that the products
//             read.
//   12        issues the products (kind::f16): S_X = Q_X K^T, O_X += P_X V, the
//             latter's first 96 keys while the last 32 are still in the making.
//   13        looks the pages up, stages their bytes by bulk copies, and works
//             the tile's factors out for the softmax.
// K's page scale multiplies the scores (folded into the exponent's FMA), V's
// goes into the exponent of P relative to that of the row's accumulator, which
// is at most V_DOWN above the tile's largest: half of P's smallest f16 step is
// then 2^-36 of a tile's largest V (or 2^-90 of what is in the accumulator already).
// Tensor memory: S_A, S_B, O_A, O_B (512 columns at d = 128).  Two f16 stages of
// K and of V beside both query tiles leave room for one staged tile of bytes
// each: the copy of tile j + 1 runs while tile j is multiplied.
//
// 2 x 1024 tokens over 8192, 32 / 8 heads of 128: 227 us, 1.14 PFLOP/s, 0.61 of
// the measured cuBLAS rate.  Four fifths of that are the tiles' loop, 3300 clocks
// for both tiles: a tile's own chain of softmax (2150) and products (1100), with
// the other tile's in between; the tensor cores are busy in 2050 of them and
// shared memory, from which they read, in 2500.  The rest are the starts and
// ends of a share's two or three blocks.  Two threads a row (24 warps) shorten
// the chain but add instructions: 294 us when one thread took 271.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NTHREADS = 512;
constexpr int W_CONV = 8, W_MMA = 12, W_LOAD = 13;
// registers after setmaxnreg: 2 x 192 + 80 + 48 = 512 of 512 (x 128 threads)
constexpr int REG_SOFT = 192, REG_CONV = 80, REG_MISC = 48;
constexpr uint32_t TMEM_COLS = 512;
// log2 of the factor on P, and how far a row's maximum may pass the reference of
// its exponents before the reference follows: P stays below 2^15.
constexpr float P_BIAS = 12.f, M_UP = 3.f;
// V_DOWN: f16's smallest step 2^-24 is then 2^-35 of a tile's largest V.  The loader
// gives a tile's exponent; a row whose accumulator would pass 2^O_MOST on the way
// there stops above it, and P takes the difference.  The bound of an accumulator is
// counted instead of read: a tile adds at most 2^O_TILE (2^15 * 448 * 128), and fewer
// than 2^23 of them are added.
constexpr int V_DOWN = 1;
constexpr float O_MOST = 100.f, O_TILE = 31.f;
// A factor of 2^-P_NONE leaves no f16 of P, and two of them leave FP32 the weights
// from 2^-40 on for the normalizer.
constexpr int P_NONE = 48;
constexpr int METAS = 4;
// Tiles of a share at least.  64 tokens over 8192, 32 / 8 heads: shares of 4
// tiles 55 us, of 8 43 us; over 1024 they are 26 and 23 us.
constexpr int MIN_SHARE = 8;

// Row blocks of 256 of a kv head's rows.
__host__ __device__ inline int row_blocks(int G, int T) { return (int)(((long long)G * T + 2 * BM - 1) / (2 * BM)); }

// Partial of a cut row block: o / l [d / 4][256][4], then m, l.
template <int D>
struct PartC {
  static constexpr int FLOATS = 2 * BM * (D + 2);
};

// Row block `i` of all (sequence, row block) pairs: what it is and the tiles of
// keys that its last token sees.
struct Block {
  int b, r0, rows, len, q_len, nt;
  FA4_DEV Block(const CacheFwdParams& p, int G, int RB, int i) {
    b = i / RB;
    r0 = (i - b * RB) * 2 * BM;
    len = cache_len(p.c, b);
    q_len = cache_count(p.q_lens, b, p.T, p.c.err);
    rows = G * q_len;
    const int t_last = (min(rows, r0 + 2 * BM) - 1) / G;
    const int see = p.causal ? max(0, min(len, len - q_len + t_last + 1)) : len;
    nt = r0 < rows ? (see + BN - 1) / BN : 0;
  }
  // units of the line: one where rows see no keys
  FA4_DEV int units() const { return r0 < rows ? max(nt, 1) : 0; }
};

// Factors of a 128-key tile, by groups of 16 keys.
struct alignas(16) Meta {
  float kx[8];                               // K's scales
  float vd[8], vu[8];                        // V's exponents against the tile's, and 2^-vd
  int xo;                                    // the tile's exponent
  int moved;                                 // the exponent of the tile before less it
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
  static constexpr int NBAR = 2 + 4 + 4 * STAGES + 2 + 4 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int OFF_SEG = (OFF_MISC + 16 + 15) / 16 * 16;    // 64 bytes a softmax warp
  static constexpr int BYTES = OFF_SEG + 8 * 64 + 1024;
  static constexpr uint32_t COL_O0 = 256;
  static_assert(COL_O0 + 2 * D <= TMEM_COLS, "tensor memory");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

FA4_DEV void store_bf16_32(__nv_bfloat16* dst, const float (&y)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 z = __floats2bfloat162_rn(y[8 * i + 2 * e], y[8 * i + 2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&z);
    }
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cache_chunk_kernel(const __grid_constant__ CacheFwdParams p) {
  using L = SmemC<D>;
  constexpr int STAGES = L::STAGES;
  constexpr uint32_t COL_O0 = L::COL_O0;
  grid_start();
  grid_wait();
  const CacheView& c = p.c;
  const int G = p.Hq / c.Hkv, RB = row_blocks(G, p.T), blocks = c.B * RB;
  // the line: (sequence, row block), kv head, tile
  auto units = [&](int i) -> unsigned { return (unsigned)(Block(p, G, RB, i).units() * c.Hkv); };
  const unsigned total = line_total(blocks, units);
  if (total == 0) return;
  const unsigned n_shares = workers(total, min((unsigned)gridDim.x, (total + MIN_SHARE - 1) / MIN_SHARE));
  if (blockIdx.x >= n_shares) return;
  const Shares shares(total, n_shares);
  const unsigned begin = shares.begin(blockIdx.x), end = shares.begin(blockIdx.x + 1);
  // the part of a row block of a kv head that starts at unit `at` (whole warp);
  // i, seq0: of the part before it
  struct Seg {
    int b, h, r0, rows, len, q_len, t0, tiles, nx;
    unsigned item, all;                      // the row block's first unit, its units
    unsigned next;                           // where the next part starts
  };
  auto segment = [&](unsigned at, int& i, unsigned& seq0) -> Seg {
    line_find(blocks, units, at, i, seq0);
    const Block k(p, G, RB, i);
    Seg g;
    g.b = k.b; g.r0 = k.r0; g.rows = k.rows; g.len = k.len; g.q_len = k.q_len;
    g.all = (unsigned)max(k.units(), 1);
    g.h = min((int)((at - seq0) / g.all), c.Hkv - 1);
    g.item = seq0 + (unsigned)g.h * g.all;
    g.t0 = (int)(at - g.item);
    g.next = min(end, g.item + g.all);
    g.tiles = k.nt == 0 ? 0 : (int)(g.next - at);
    g.nx = k.rows - k.r0 > BM ? 2 : 1;       // tile B may have no rows
    return g;
  };

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;                  // by tile
  uint64_t* k8_full = bars + 2;              // staged bytes
  uint64_t* k8_empty = bars + 3;
  uint64_t* v8_full = bars + 4;
  uint64_t* v8_empty = bars + 5;
  uint64_t* k_full = bars + 6;               // f16 tiles
  uint64_t* k_empty = k_full + STAGES;
  uint64_t* v_full = k_empty + STAGES;
  uint64_t* v_empty = v_full + STAGES;
  uint64_t* s_full = v_empty + STAGES;
  uint64_t* p_full = s_full + 2;            // by tile: 96 keys, 32
  uint64_t* o_done = p_full + 4;
  uint64_t* mma_done = o_done + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  volatile int* last_one = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 8);
  Meta* metas = reinterpret_cast<Meta*>(smem + L::OFF_META);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(k8_full, 1); mbar_init(k8_empty, 4);
    mbar_init(v8_full, 1); mbar_init(v8_empty, 4);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&k_full[s], 4); mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4); mbar_init(&v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4); mbar_init(&p_full[2 * x + 1], 4);
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
      int li = 0;
      unsigned lseq = 0;
      int issued = 0, n = 0;                 // n: tiles so far
      bool ok = true;
      for (unsigned at = begin; ok && at < end;) {
        const Seg sg = segment(at, li, lseq);
        at = sg.next;
        int xo = -127;
        for (int j = sg.t0; j < sg.t0 + sg.tiles; ++j, ++n) {
          // lane i < 8: group i of 16 keys; the first lane of a page copies it
          const int key = j * BN + 16 * (lane & 7);
          const int lp = key >> log_p;
          int pg = -1;
          if (lane < 8 && key < sg.len) pg = cache_page(c, c.table, sg.b, lp);
          const long long ph = (long long)max(pg, 0) * c.Hkv + sg.h;
          const float kx = pg >= 0 ? e8m0_value(*(c.ks + ph)) : 1.f;      // (what is absent is masked)
          const int ev = (int)*(c.vs + ph) - 127;
          Meta& m = metas[n % METAS];
          if (n > 0 && !mbar_wait(k8_empty, (n - 1) & 1, abort_flag, c.err)) { ok = false; break; }
          int top = pg >= 0 ? ev : -1000;
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = __shfl_sync(0xffffffffu, top, 0);
          // the exponent: at least the tile's largest, and not far above it
          const int had = xo;
          if (top > -1000 && (top > xo || top < xo - V_DOWN)) xo = top;
          const uint32_t there = __ballot_sync(0xffffffffu, pg >= 0);
          if (lane < 8) {
            const int d = min(0, max(ev - xo, -P_NONE));
            m.kx[lane] = kx;
            m.vd[lane] = (float)d;
            m.vu[lane] = exp2i(-d);
            if (lane == 0) { m.xo = xo; m.moved = had - xo; m.absent = ~there & 0xffu; }
          }
          __syncwarp();
          const bool copies = lane < 8 && pg >= 0 && ((16 * lane) & (c.page - 1)) == 0;
          const uint32_t bytes = (uint32_t)c.page * D;
          const uint32_t all = (uint32_t)__popc(__ballot_sync(0xffffffffu, copies)) * bytes;
          if (lane == 0) mbar_arrive_expect_tx(k8_full, all);
          __syncwarp();
          if (copies) bulk_load(smem + L::OFF_K8 + 16 * lane * D, c.k + (ph << log_p) * D, bytes, k8_full);
          issued = 2 * n + 1;
          if (n > 0 && !mbar_wait(v8_empty, (n - 1) & 1, abort_flag, c.err)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(v8_full, all);
          __syncwarp();
          if (copies) bulk_load(smem + L::OFF_V8 + 16 * lane * D, c.v + (ph << log_p) * D, bytes, v8_full);
          issued = 2 * n + 2;
        }
      }
      if (*abort_flag) {                     // what is still in flight lands first
        volatile int none = 0;
        const int nk = (issued + 1) / 2, nv = issued / 2;
        if (nk) mbar_wait(k8_full, (nk - 1) & 1, &none, c.err);
        if (nv) mbar_wait(v8_full, (nv - 1) & 1, &none, c.err);
      }
      __syncwarp();
    } else if (warp == W_MMA) {
      // ---------------------------------------------------------- products
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, false, false, false);
      const uint32_t idesc_o = idesc_f16(BM, D, false, false, true);   // A from TMEM, V MN-major
      const uint32_t sq = smem_u32(smem + L::OFF_Q);
      bool ok = true;
      // t: the CTA's tile, for the stages; u: the tile's (0: A, 1: B) own count
      auto issue_qk = [&](int x, int t, bool last) -> bool {
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
          if (last) mma_commit(&k_empty[st]);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](int x, int t, int u, bool first, bool last) -> bool {
        const int st = t % STAGES;
        if (x == 0 && !mbar_wait(&v_full[st], (t / STAGES) & 1, abort_flag, c.err)) return false;
        const uint32_t sv = smem_u32(smem + L::OFF_V + st * L::TILE);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait(&p_full[2 * x + half], u & 1, abort_flag, c.err)) return false;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int k = half ? 6 : 0; k < (half ? 8 : 6); ++k)
              mma_f16_tmem_a(tbase + COL_O0 + D * x, tbase + 128 * x + 8 * k,
                             make_sdesc(sv + k * 16 * 128, L::CH, 1024, SW_128B), idesc_o, !first || k > 0);
            if (half) {
              mma_commit(&o_done[x]);
              if (last) mma_commit(&v_empty[st]);
            }
          }
          __syncwarp();
        }
        return true;
      };
      // each tile's next Q K^T follows its own P V, so the pipe has read P_X
      // before it overwrites S_X
      int li = 0;
      unsigned lseq = 0;
      int n = 0, nb = 0, pa = 0, pb = 0;     // tiles and parts so far, those of B among them
      for (unsigned at = begin; ok && at < end;) {
        const Seg sg = segment(at, li, lseq);
        at = sg.next;
        if (sg.tiles == 0) continue;
        const bool two = sg.nx == 2;
        ok = mbar_wait(&q_full[0], pa++ & 1, abort_flag, c.err) && (!two || mbar_wait(&q_full[1], pb++ & 1, abort_flag, c.err));
        tc_fence_after();
        ok = ok && issue_qk(0, n, !two) && (!two || issue_qk(1, n, true));
        for (int j = 0; ok && j < sg.tiles; ++j) {
          const bool more = j + 1 < sg.tiles;
          ok = issue_pv(0, n + j, n + j, j == 0, !two) && (!more || issue_qk(0, n + j + 1, !two));
          if (two) ok = ok && issue_pv(1, n + j, nb + j, j == 0, true) && (!more || issue_qk(1, n + j + 1, true));
        }
        n += sg.tiles;
        if (two) nb += sg.tiles;
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
    int li = 0;
    unsigned lseq = 0;
    int n = 0;
    bool ok = true;
    for (unsigned at = begin; ok && at < end;) {
      const Seg sg = segment(at, li, lseq);
      at = sg.next;
      for (int j = sg.t0; ok && j < sg.t0 + sg.tiles; ++j, ++n) {
        const int st = n % STAGES;
        const int left = sg.len - j * BN;    // keys of the tile that are there
        const uint32_t parity = (n / STAGES - 1) & 1;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* full8 = kv ? v8_full : k8_full;
          uint64_t* empty8 = kv ? v8_empty : k8_empty;
          uint64_t* empty = kv ? &v_empty[st] : &k_empty[st];
          uint64_t* full = kv ? &v_full[st] : &k_full[st];
          ok = ok && mbar_wait(full8, n & 1, abort_flag, c.err);
          if (!ok) break;
          const uint8_t* from = smem + (kv ? L::OFF_V8 : L::OFF_K8) + row0 * D + part * 16;
          uint4 x[128 / RSTEP];
#pragma unroll
          for (int i = 0; i < 128 / RSTEP; ++i) x[i] = lds16(from + i * RSTEP * D);
          const uint32_t absent = metas[n % METAS].absent;
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
          if (n >= STAGES) ok = mbar_wait(empty, parity, abort_flag, c.err);
          if (!ok) break;
          uint8_t* tile = smem + (kv ? L::OFF_V : L::OFF_K) + st * L::TILE;
#pragma unroll
          for (int i = 0; i < 128 / RSTEP; ++i) store16<D>(tile, row0 + i * RSTEP, part, x[i]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
      }
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int quad = warp & 3;
    const int rt = quad * 32 + lane;         // row within the tile
    const int mate = BM * x + rt;            // row of the block
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_s = 128 * x, col_o = COL_O0 + D * x;
    // After a wait that ran out a warp computes no more, but comes to the
    // barriers of every join.
    bool ok = true;
    int n = 0, m0 = 0;                       // tiles so far of X, of the CTA
    // What is needed again after the tiles waits in shared memory: the tiles'
    // loop needs the registers.
    enum { E_B, E_H, E_R0, E_ROWS, E_NX, E_TILES, E_FIRST, E_C0, E_PARTS, E_ODD, E_NEXT, E_I, E_SEQ0 };
    volatile unsigned* rec = reinterpret_cast<volatile unsigned*>(smem + L::OFF_SEG + 64 * warp);
    if (lane == 0) { rec[E_I] = 0; rec[E_SEQ0] = 0; }
    __syncwarp();
    for (unsigned at = begin; at < end; at = rec[E_NEXT]) {
      int tiles, left0;                      // left0: keys that the row sees from the first tile on
      const __nv_bfloat16* src = nullptr;
      {
        int li = (int)rec[E_I];
        unsigned lseq = rec[E_SEQ0];
        const Seg sg = segment(at, li, lseq);
        tiles = x < sg.nx ? sg.tiles : 0;
        const int r = sg.r0 + mate;
        const bool valid = r < sg.rows;
        const int t = valid ? r / G : 0, gg = valid ? r - t * G : 0;
        const long long orow = ((long long)sg.b * p.Hq + sg.h * G + gg) * p.T + t;
        const int vis = !valid ? 0 : p.causal ? max(0, min(sg.len, sg.len - sg.q_len + t + 1)) : sg.len;
        left0 = vis - sg.t0 * BN;
        if (valid) src = reinterpret_cast<const __nv_bfloat16*>(p.q) + orow * D;
        const unsigned c0 = shares.of(sg.item), c1 = shares.of(sg.item + sg.all - 1);
        __syncwarp();
        if (lane == 0) {
          rec[E_B] = sg.b; rec[E_H] = sg.h; rec[E_R0] = sg.r0; rec[E_ROWS] = sg.rows; rec[E_NX] = sg.nx;
          rec[E_TILES] = sg.tiles; rec[E_FIRST] = at == begin; rec[E_C0] = c0; rec[E_PARTS] = c1 - c0 + 1;
          rec[E_ODD] = shares.begin(c0) != sg.item; rec[E_NEXT] = sg.next;
          rec[E_I] = li; rec[E_SEQ0] = lseq;
        }
        __syncwarp();
      }

      // the row of q: largest magnitude, then f16 under a power of two
      float f_row = 0.f;
      if (tiles > 0) {
        f_row = p.c2 * exp2i(store_query_rows<D>(smem + L::OFF_Q + x * L::TILE, 32 * quad, src));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[x]);
      }

      float m = -INFINITY, l = 0.f;
      // o is in units of 2^(xo + above), xo being the tile's exponent; `apart`: above
      // is not 0 in all rows of the warp.  With m_grown the row's maximum, o was below
      // 2^(grown + 23) when it last changed its unit.  What is rarely needed stays out
      // of the registers.
      int xo = -127;
      bool apart = false;
      enum { ABOVE, GROWN, M_GROWN, BY, UNDO };
      volatile float rare[5] = {0.f, O_TILE, -INFINITY, 1.f, 1.f};
      for (int j = 0; ok && j < tiles; ++j, ++n) {
        ok = mbar_wait(&s_full[x], n & 1, abort_flag, c.err);
        if (!ok) break;
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
        const Meta& meta = metas[(m0 + j) % METAS];
        const uint32_t absent = meta.absent;
        const int left = left0 - j * BN;
        if (__any_sync(0xffffffffu, left < BN) || absent) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * g + i >= left || ((absent >> (2 * g + i / 16)) & 1)) s[g][i] = -INFINITY;
        }
        // max by groups of 16 keys, each with its K scale
        float F[8], add[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          *reinterpret_cast<float4*>(F + 4 * g) = *reinterpret_cast<const float4*>(meta.kx + 4 * g);
          *reinterpret_cast<float4*>(add + 4 * g) = *reinterpret_cast<const float4*>(meta.vd + 4 * g);
        }
        const int moved = meta.moved;
        xo = meta.xo;
        const bool refit = j > 0 && (moved != 0 || apart);
        // (a masked score is -inf, which must not meet a factor of 0: 2^-126 more changes
        // a score of up to 2^24 units by 2^-102 at most)
#pragma unroll
        for (int g = 0; g < 8; ++g) F[g] = fmaf(F[g], f_row, 0x1p-126f);
        float top_all = -INFINITY;
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
          top_all = fmaxf(top_all, fmaxf(top, top2) * F[g]);
        }
        const float m_new = top_all > m + M_UP ? top_all : m;
        float ref = (m_new == -INFINITY ? 0.f : m_new) - P_BIAS;
        if (refit) {
          // what bounds the accumulator after this tile's alpha; before the row's first
          // key it holds zeros (and of a NaN fmaxf takes the other)
          const bool empty = m_new == -INFINITY;
          const float now = fmaxf(rare[GROWN] + (rare[M_GROWN] - m), O_TILE) + (m - m_new);
          const float x = (float)moved + rare[ABOVE];                // above the tile's exponent
          const float to = empty ? 0.f : fmaxf(0.f, x - floorf(fmaxf(O_MOST - now, 0.f)));
          rare[BY] = empty ? 1.f : ex2_approx((m_new == m ? 0.f : m - m_new) + (x - to));
          rare[GROWN] = fmaxf(O_TILE, now + (x - to));
          rare[M_GROWN] = m_new;
          rare[ABOVE] = to;
          const int n_above = (int)fminf(to, (float)P_NONE);
          ref += (float)n_above;
          rare[UNDO] = exp2i(n_above);
          apart = __any_sync(0xffffffffu, to != 0.f);
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) add[g] -= ref;
        const float alpha = (j == 0 || m_new == m) ? 1.f : ex2_approx(m - m_new);
        float l_new = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float2 undo = *reinterpret_cast<const float2*>(meta.vu + 2 * g);
          uint32_t pk[16];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int gr = 2 * g + hf;
            float2 ls = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 16 * hf + 2 * i;
              const float2 e = ffma2(make_float2(s[g][k], s[g][k + 1]), make_float2(F[gr], F[gr]), make_float2(add[gr], add[gr]));
              const float2 pp = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              ls = fadd2(ls, pp);
              pk[8 * hf + i] = pack_f16x2(pp.x, pp.y);
            }
            l_new = fmaf(ls.x + ls.y, hf ? undo.y : undo.x, l_new);
          }
          tmem_st16(lane_base + col_s + 16 * g, pk);
          if (g == 1 && j > 0) {
            ok = mbar_wait(&o_done[x], (n - 1) & 1, abort_flag, c.err);
            if (!ok) break;
            tc_fence_after();
            float by = alpha;
            if (refit) by = rare[BY];
            if (__any_sync(0xffffffffu, by != 1.f)) {
#pragma unroll
              for (int og = 0; og < D / 32; ++og) {
                uint32_t ov[32];
                tmem_ld32(lane_base + col_o + 32 * og, ov);
                tmem_ld_wait();
                reg_fence32(ov);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const float2 y = fmul2(make_float2(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])), make_float2(by, by));
                  ov[i] = __float_as_uint(y.x);
                  ov[i + 1] = __float_as_uint(y.y);
                }
                tmem_st32(lane_base + col_o + 32 * og, ov);
              }
            }
          }
          if (g >= 2) {                      // P V of 96 keys may go, of all
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * x + g - 2]);
          }
        }
        if (!ok) break;
        if (refit) l_new *= rare[UNDO];
        l = fmaf(alpha, l, l_new);
        m = m_new;
      }
      if (ok && tiles > 0) ok = mbar_wait(&o_done[x], (n - 1) & 1, abort_flag, c.err);
      tc_fence_after();
      // a row without keys: whatever the accumulator holds counts for nothing
      const bool none = l == 0.f;
      const int nx = (int)rec[E_NX], r0 = (int)rec[E_R0], rows = (int)rec[E_ROWS], sb = (int)rec[E_B], sh = (int)rec[E_H];
      const unsigned parts = rec[E_PARTS], c0 = rec[E_C0];
      const bool cut = parts > 1, valid = r0 + mate < rows;
      auto out_row = [&](int r) -> long long {
        return ((long long)sb * p.Hq + sh * G + r % G) * p.T + r / G;
      };
      const long long orow = valid ? out_row(r0 + mate) : 0;
      float4* part = reinterpret_cast<float4*>(p.part + (gridDim.x * 8 + 15) / 16 * 16);
      float4* slot = part + (size_t)(2 * blockIdx.x + (rec[E_FIRST] ? 0 : 1)) * (PartC<D>::FLOATS / 4);
      if (ok && x < nx) {
        const float inv = none ? 0.f : 1.f / l, unit = pow2_any(xo + (int)rare[ABOVE]);
#pragma unroll 1
        for (int g = 0; g < D / 32; ++g) {
          uint32_t v[32];
          tmem_ld32(lane_base + col_o + 32 * g, v);
          tmem_ld_wait();
          reg_fence32(v);
          if (!valid) continue;
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = none ? 0.f : __uint_as_float(v[i]) * inv * unit;    // in this order: it may be near FP32's end
          if (cut) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              slot[(8 * g + i) * 2 * BM + mate] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else {
            store_bf16_32(reinterpret_cast<__nv_bfloat16*>(p.o) + orow * D + 32 * g, y);
          }
        }
        if (valid && cut) {
          float* ml = reinterpret_cast<float*>(slot) + 2 * BM * D + mate;
          ml[0] = m;
          ml[2 * BM] = l;
        } else if (valid && p.lse) {
          p.lse[orow] = none ? -INFINITY : fmaf(m - P_BIAS, 0.69314718f, logf(l));
        }
      }
      if (cut) {
        // The block's parts meet: whoever is the last to have written one joins
        // them.  The barrier and the release order the CTA's part before its
        // arrival, the acquire the others' parts before the join.
        const unsigned odd = rec[E_ODD];
        named_bar(1, 2 * BM);
        if (threadIdx.x == 0) *last_one = !*abort_flag && marked_arrive(reinterpret_cast<unsigned long long*>(p.part) + c0, parts);
        named_bar(1, 2 * BM);
        // all eight warps: rows of two tiles, or the two halves of one tile's
        // dimensions; four parts' words in flight
        const int row = nx == 2 ? mate : rt, jr = r0 + row;
        if (*last_one && jr < rows) {
          auto slot_of = [&](unsigned i) { return part + (size_t)(2 * (c0 + i) + (i == 0 ? odd : 0)) * (PartC<D>::FLOATS / 4); };
          auto stat = [&](unsigned i, int which) {
            return __ldcg(reinterpret_cast<const float*>(slot_of(i)) + 2 * BM * (D + which) + row);
          };
          float mt = -INFINITY, lt = 0.f;
#pragma unroll 1
          for (unsigned i0 = 0; i0 < parts; i0 += 4) {
            float mi[4], li[4], mx = mt;
#pragma unroll
            for (unsigned k = 0; k < 4; ++k) {
              mi[k] = stat(min(i0 + k, parts - 1), 0);
              li[k] = i0 + k < parts ? stat(i0 + k, 1) : 0.f;
            }
#pragma unroll
            for (unsigned k = 0; k < 4; ++k) mx = fmaxf(mx, mi[k]);
            if (lt != 0.f) lt *= ex2_approx(mt - mx);
            mt = mx;
#pragma unroll
            for (unsigned k = 0; k < 4; ++k)
              if (li[k] != 0.f) lt = fmaf(li[k], ex2_approx(mi[k] - mt), lt);
          }
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
          const long long to = out_row(jr);
          const int from_g = nx == 2 ? 0 : x * (D / 64), to_g = nx == 2 ? D / 32 : from_g + D / 64;
#pragma unroll 1
          for (int g = from_g; g < to_g; ++g) {
            float y[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = 0.f;
#pragma unroll 1
            for (unsigned i0 = 0; i0 < parts; i0 += 4) {
              float4 z[4][8];
              float w[4];
#pragma unroll
              for (unsigned k = 0; k < 4; ++k) {
                const unsigned i = min(i0 + k, parts - 1);
                const float4* from = slot_of(i) + 16 * g * BM + row;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[k][e] = __ldcg(from + e * 2 * BM);
                const float li = stat(i, 1);
                w[k] = li == 0.f || i0 + k >= parts ? 0.f : li * inv * ex2_approx(stat(i, 0) - mt);
              }
#pragma unroll
              for (unsigned k = 0; k < 4; ++k) {
                if (w[k] == 0.f) continue;             // 0 * inf
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  y[4 * e] = fmaf(w[k], z[k][e].x, y[4 * e]);
                  y[4 * e + 1] = fmaf(w[k], z[k][e].y, y[4 * e + 1]);
                  y[4 * e + 2] = fmaf(w[k], z[k][e].z, y[4 * e + 2]);
                  y[4 * e + 3] = fmaf(w[k], z[k][e].w, y[4 * e + 3]);
                }
              }
            }
            store_bf16_32(reinterpret_cast<__nv_bfloat16*>(p.o) + to * D + 32 * g, y);
          }
          if (p.lse && from_g == 0) p.lse[to] = lt == 0.f ? -INFINITY : fmaf(mt - P_BIAS, 0.69314718f, logf(lt));
        }
      }
      m0 += (int)rec[E_TILES];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

// CTAs of the fixed grid: the GPU's, or fewer where the cache's capacity gives
// fewer tiles; 0: more than the line's 32 bits count.
int grid_of(int B, int Hq, int Hkv, int T, int page, int max_pages) {
  const long long blocks = (long long)row_blocks(Hq / Hkv, T) * B;
  const long long tiles = ((long long)max_pages * page + BN - 1) / BN;
  if (blocks * Hkv >= (1LL << 31) / (tiles < 1 ? 1 : tiles)) return 0;
  const long long all = blocks * Hkv * (tiles < 1 ? 1 : tiles);
  return (int)(all < kSMs ? all : kSMs);
}

template <int D>
cudaError_t launch(const CacheFwdParams& p, cudaStream_t st) {
  auto k = cache_chunk_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemC<D>::BYTES);
  if (e != cudaSuccess) return e;
  const int grid = grid_of(p.c.B, p.Hq, p.c.Hkv, p.T, p.c.page, p.c.max_pages);
  if (grid == 0) return cudaErrorInvalidValue;
  return launch_next(k, dim3((unsigned)grid), NTHREADS, SmemC<D>::BYTES, st, p);
}

}  // namespace

size_t cache_chunk_workspace(int B, int Hq, int Hkv, int T, int d, int page, int max_pages) {
  const size_t grid = (size_t)grid_of(B, Hq, Hkv, T, page, max_pages);
  return (grid * 8 + 15) / 16 * 16 + 2 * grid * 4 * (size_t)(d == 128 ? PartC<128>::FLOATS : PartC<64>::FLOATS);
}

cudaError_t launch_cache_chunk(const CacheFwdParams& p, cudaStream_t st) {
  return p.c.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace fa4
