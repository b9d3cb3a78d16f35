// cross_bwd.cu -- gradients of cross attention (tcgen05).
//
//   P = 2^(c s - lse log2 e), dP = dO V^T, D = rowsum(dO o), dS = P (dP - D)
//   dQ = scale dS K,  dV = sum P^T dO,  dK = scale sum dS^T Q
//
// Two kernels, so that every sum has one owner and one order: the first owns
// query rows and goes through their keys (3 products a tile: S, dP, dQ), the second
// owns keys and goes through the queries of all heads that share them (4: S^T,
// dP^T, dV, dK).  Seven products instead of the five of a kernel that adds its dQ
// into memory, but no FP32 dQ passes through memory several times, and nothing
// depends on the order of atomics.
//
// A query tile is 128 rows as in the forward (several heads where they have up to
// 64 rows); a key tile is 128 keys.
//
// Both kernels get equal ranges of steps (a key tile with a query tile) for as many
// CTAs as the GPU has multiprocessors: few queries with many keys, or many with few,
// keep it as busy as even shapes do.  A range that starts or ends inside an output
// tile's steps leaves FP32 partials in the workspace.
//
// cross_dq_kernel: a query tile's key tiles in turn.  Warps 0-15: a thread per
//   row and quarter of the keys: P from S, dS from P and dP, as bf16 into tensor memory
//   (the A operand of dQ).  Q is in tensor memory too (the A operand of S), so that its
//   place in shared memory takes the next item's Q, then this one's dQ on its way
//   out, and K has three places and V two.  S and dP of the next key tile run as soon
//   as these have been read.  D is summed by the same threads from the o and dO tiles,
//   and kept in the workspace.  Two warps issue the products: S; dP and dQ.  What bounds
//   it: with many key tiles what comes in (64 KB a step at 30 B a cycle, where the
//   products take 1536 of 2240 cycles), with one or two the item's own chain (Q to
//   tensor memory, D, dQ out), which is why there are sixteen warps: eight took 219
//   where these take 203 us (6 heads, 76,666 queries, 188 keys; 1024 queries over 4100
//   keys 323 with either).
// cross_dkv_kernel: a key tile's query tiles in turn.  Rows are keys: P^T and dS^T go
//   over S^T and dP^T as A operands of dV and dK, which are summed in tensor memory
//   (512 columns in all).  Two warps issue the products, S^T and dV the one, dP^T and
//   dK the other (one warp was the bound: a product takes 512 cycles, its waits,
//   instructions and commits 700).  Eight warps of threads with a key and half of the
//   queries each (sixteen: 175 -> 191 us of the 4100 keys).  What bounds it at d = 128:
//   shared memory, of which a step's products read 192 KB, TMA writes 64 KB and the
//   threads take 256 words of -lse and -D: 2304 cycles of 128 B, with the waits between
//   them 2800, where the products alone take 2048.
// cross_join_kernel: sums the partials in the ranges' order; zeros for keys behind
//   kv_lens.
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"
#include "internal.h"

namespace fa4 {
namespace {

constexpr int BM = 128, BN = 128;
// Warps of a kernel with N that do the element-wise work, behind them four that load and
// issue; registers are moved between the two.
template <int N>
struct Roles {
  static constexpr int SOFT = 32 * N, NTHREADS = SOFT + 128;
  static constexpr int W_PROD = N, W_MMA = N + 1, W_MMA_B = N + 2;
  // (of 168 and of 96 that a thread starts with: 2 x 208 + 88 = 3 x 168, 4 x 104 + 64 = 5 x 96)
  static constexpr int REG_SOFT = N == 8 ? 208 : 104, REG_MISC = N == 8 ? 88 : 64;
};
constexpr uint32_t TMEM_COLS = 512;
constexpr float L2E = 1.4426950408889634f;

struct Params {
  CrossParams p;
  HeadsMap q, dout, o, k, v;
  HeadsMap group_q, group_dout;                // second kernel, where heads share a tile
  HeadsMap dq, dk, dv;                         // boxes of 32 rows (dq: where heads share no tile)
  int tiles, heads, box;                       // query tiles of a kv head, as in the forward
  Divisor per_head, per_kv, hkv, nq;           // (per_kv: tiles)
  int key_tiles;                               // of Nk
  int items;                                   // query tiles in all
  int slots;                                   // CTAs at most, of either kernel
  int ctas;                                    // of the first kernel
  int joins, by_query_tile, by_key_tile;       // third kernel: x that join, and what an x is
  int parts_q, parts_k;                        // CTAs of a sum
  int side, ranges;                            // second kernel: key tiles side by side, ranges of steps (side CTAs each)
  int dq32, dk32, dv32;                        // rows begin on 32 bytes
  float* del;                                  // D [B][Hq][Nq]
  float *part, *part_q;                        // partial sums: [2 slots][dV, dK] and [2 slots] tiles of dQ
};

// Row r of a query tile: query head within the group (G: none) and position.
FA4_DEV void tile_row(const Params& a, int tile, int r, int G, int& g, int& n) {
  if (a.heads > 1) {
    divide(r, a.nq, g, n);
    g = r < a.heads * a.p.Nq ? min(G, tile * a.heads + g) : G;
  } else {
    divide(tile, a.per_head, g, n);
    n = n * BM + r;
    if (n >= a.p.Nq) g = G;
  }
}

FA4_DEV uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

// Columns 2 i and 2 i + 1 of a thread's row.
template <int N>
FA4_DEV float2 pair(const uint32_t (&v)[N], int i) {
  return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// N FP32 columns of a row, times f, to bf16 in global memory.
template <int N>
FA4_DEV void store_row(__nv_bfloat16* dst, const uint32_t (&v)[N], float f, bool wide) {
  uint32_t pk[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) pk[i] = pack2(pair(v, i).x * f, pair(v, i).y * f);
  if (wide) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i) st_global_v8(dst + 16 * i, pk + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
  }
}

// N columns of tensor memory (a thread's row).
template <int N>
FA4_DEV void load_columns(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N == 32) tmem_ld32(taddr, v);
  else tmem_ld16(taddr, v);
  tmem_ld_wait();
  if constexpr (N == 32) reg_fence32(v);
  else reg_fence16(v);
}

// ---------------------------------------------------------------------------
// steps
// ---------------------------------------------------------------------------
// Both kernels' work is cut into steps, a key tile that holds keys with a query
// tile each, and the CTAs get equal ranges of them: the first kernel's in the order
// (sequence, kv head, query tile, key tile), the second's in the order (sequence, kv
// head, key tile, query tile).  A line is the steps of one output tile.
//
// The second kernel reads each query tile once for each key tile.  Where `side` divides the
// key tiles, that many CTAs go through the same queries at the same time with a key tile
// each, so that one of them reads from memory and the others from L2: a step there
// is `side` key tiles with a query tile (24 heads, 32,760 queries, 512 keys: 570 -> 535 us; 816 -> 214 MB
// read with half of the queries).
struct Range {
  int b, hk, tile;             // sequence, kv head, the line's query (first kernel) or key tile
  int nt, len;                 // the sequence's key tiles and keys
  int t;                       // step within the line
  int left;                    // steps of the range from here on
  // the next line (the range has more), in the first kernel's order (rows) or the second's
  FA4_DEV void line(const Params& a, bool rows) {
    const int n = rows ? a.tiles : nt;
    t = 0;
    tile += rows ? 1 : a.side;
    if (tile < n) return;
    tile -= n;                 // (`side` divides n: back to the CTA's place among its neighbours)
    if (++hk < a.p.Hkv) return;
    hk = 0;
    do {
      ++b;
      len = key_count(a.p, b, false);
      nt = (len + BN - 1) / BN;
    } while (nt == 0);
  }
};

// a / b for 0 <= a, 0 < b: in 32 bits where they fit (64-bit divisions take some
// 500 cycles, and a kernel's start has several in a row).
FA4_DEV long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

FA4_DEV int tiles_of(const Params& a, int b, bool report = false) {
  return (key_count(a.p, b, report) + BN - 1) / BN;
}

// Steps of all sequences (one warp).
FA4_DEV long long all_steps(const Params& a, bool rows, int lane, bool report = false) {
  long long all = 0;
  if (!a.p.lens) {
    all = (long long)a.p.B * (rows ? a.key_tiles : a.key_tiles / a.side);
  } else {
    for (int x = lane; x < a.p.B; x += 32) all += tiles_of(a, x, report);
    for (int o = 16; o > 0; o /= 2) all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  return all * a.p.Hkv * a.tiles;
}

// The first step of range `i` of `ranges` over `total` steps.
FA4_DEV long long range_start(long long total, int i, int ranges) { return quotient(total * i, ranges); }

// The place of a step (one warp); rows: in the first kernel's order, else of the CTA
// with place `lane_tile` among the `side` that share its range.
FA4_DEV void find_step(const Params& a, long long step, bool rows, int lane_tile, int lane, Range& x) {
  const int side = rows ? 1 : a.side;            // (1 where sequences have lengths)
  x.b = 0;
  const long long per = (long long)a.p.Hkv * a.tiles;      // steps of a key tile of a sequence
  if (!a.p.lens) {
    x.b = (int)quotient(step, per * (a.key_tiles / side));
    step -= per * (a.key_tiles / side) * x.b;
  } else {
    // 32 sequences at a time
    for (int x0 = 0;; x0 += 32) {
      const long long n = x0 + lane < a.p.B ? tiles_of(a, x0 + lane) * per : 0;
      long long upto = n;
      for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto > step);
      if (past) {
        const int at = __ffs(past) - 1;
        x.b = x0 + at;
        step -= __shfl_sync(0xffffffffu, upto - n, at);
        break;
      }
      step -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  x.len = key_count(a.p, x.b, false);
  x.nt = (x.len + BN - 1) / BN;
  const int each = rows ? x.nt : a.tiles, lines = rows ? a.tiles : x.nt / side;
  const int line = (int)quotient(step, each);
  x.t = (int)(step - (long long)line * each);
  x.hk = line / lines;
  x.tile = (line - x.hk * lines) * side + lane_tile;
}

// This CTA's range (one warp).
FA4_DEV Range find_range(const Params& a, bool rows, int lane) {
  Range x;
  const long long total = all_steps(a, rows, lane, rows && blockIdx.x == 0);
  const int ranges = rows ? a.ctas : a.ranges, i = rows ? blockIdx.x : (int)blockIdx.x / a.side;
  const long long s0 = range_start(total, i, ranges), s1 = range_start(total, i + 1, ranges);
  x.b = x.hk = x.tile = x.nt = x.len = x.t = 0;
  x.left = (int)(s1 - s0);
  if (x.left > 0) find_step(a, s0, rows, rows ? 0 : (int)blockIdx.x % a.side, lane, x);
  return x;
}

// The place of an output tile's partial sums: [D / 4][128 rows][4] FP32, so that
// the threads of a warp, a row each, write lines.
FA4_DEV float* partial(float* part, int D, int which, int row, int column) {
  return part + (long long)which * 128 * D + (column / 4 * 128 + row) * 4;
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
template <int D>
struct SmemQ {
  static constexpr int TILE = (D / 64) * CH;
  // K is held from S to dQ, V for dP alone: rings of their own (o goes through V's)
  static constexpr int KS = D == 128 ? 3 : 5, VS = D == 128 ? 2 : 4;
  static constexpr int OFF_Q = 0, OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_DEL = OFF_V + VS * TILE;         // [4 quarters][128]: shares of D
  static constexpr int OFF_BAR = OFF_DEL + 2 * 1024;
  static constexpr int NBAR = 2 * KS + 2 * VS + 13;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 48;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

// The range's items: key tiles [j0, j1) of a query tile.
struct ItemQ {
  int b, hk, tile, len, j0, j1;
  bool whole;
};
struct WalkQ {
  Range x;
  FA4_DEV explicit WalkQ(const Range& r) : x(r) {}
  FA4_DEV bool get(ItemQ& it) const {
    if (x.left == 0) return false;
    it.b = x.b; it.hk = x.hk; it.tile = x.tile; it.len = x.len;
    it.j0 = x.t;
    it.j1 = min(x.nt, x.t + x.left);
    it.whole = it.j0 == 0 && it.j1 == x.nt;
    return true;
  }
  FA4_DEV void next(const Params& a) {
    x.left -= min(x.nt, x.t + x.left) - x.t;
    if (x.left > 0) x.line(a, true);
  }
};

template <int D>
__global__ void __launch_bounds__(Roles<16>::NTHREADS, 1) cross_dq_kernel(const __grid_constant__ Params a) {
  using L = SmemQ<D>;
  using R = Roles<16>;
  constexpr int KS = L::KS, VS = L::VS;
  constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DQ = 256, COL_DS = 384, COL_Q = 448;
  const CrossParams& p = a.p;
  // (no room to align it by hand: nothing else is in shared memory, so it begins on its alignment)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {
    atomicOr(p.err, FA4_DEVERR_TIMEOUT);
    return;
  }
  float* shares = reinterpret_cast<float*>(smem + L::OFF_DEL);
  uint8_t *q_tile = smem + L::OFF_Q, *do_tile = smem + L::OFF_DO;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + VS;
  uint64_t* q_full = v_empty + VS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* do_full = q_empty + 1;
  uint64_t* do_empty = do_full + 1;
  uint64_t* qt_full = do_empty + 1;      // Q is in tensor memory
  uint64_t* s_full = qt_full + 1;        // S is there
  uint64_t* s_free = s_full + 1;         // S has been read
  uint64_t* dp_full = s_free + 1;        // dP is there
  uint64_t* dp_free = dp_full + 1;       // dP has been read
  uint64_t* ds_full = dp_free + 1;       // dS is there
  uint64_t* ds_free = ds_full + 1;       // dS has gone into dQ
  uint64_t* dq_done = ds_free + 1;       // the item's dQ is there
  uint64_t* mma_done = dq_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  Range* range = reinterpret_cast<Range*>(smem + L::OFF_MISC + 8);
  static_assert(sizeof(Range) <= 40, "range's place");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int s = 0; s < VS; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); }
    mbar_init(q_full, 1);
    mbar_init(q_empty, R::W_PROD);
    mbar_init(do_full, 1);
    mbar_init(do_empty, R::W_PROD + 1);
    mbar_init(qt_full, R::W_PROD);
    mbar_init(s_full, 1);
    mbar_init(s_free, R::W_PROD);
    mbar_init(dp_full, 1);
    mbar_init(dp_free, R::W_PROD);
    mbar_init(ds_full, R::W_PROD);
    mbar_init(ds_free, 1);
    mbar_init(dq_done, 1);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == R::W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  // (in this order: the next kernel reads its inputs before it waits for this one)
  wait_for_previous();
  next_may_start();
  if (warp == R::W_PROD) {
    const Range x = find_range(a, true, lane);
    if (lane == 0) *range = x;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const int G = p.Hq / p.Hkv;
  WalkQ w(*range);
  ItemQ it{};

  if (warp >= R::W_PROD) {
    setmaxnreg_dec<R::REG_MISC>();
    if (warp == R::W_PROD) {
      if (lane == 0) {
        tma_prefetch_desc(&a.q.map);
        tma_prefetch_desc(&a.dout.map);
        tma_prefetch_desc(&a.o.map);
        tma_prefetch_desc(&a.k.map);
        tma_prefetch_desc(&a.v.map);
        int qn = 0, dn = 0, kn = 0, vn = 0;  // tiles issued
        auto load = [&](const HeadsMap& m, uint8_t* dst, uint64_t* full, int rows, int n, int h, int b) {
          mbar_arrive_expect_tx(full, rows * 2 * D);
          for (int c = 0; c < D / 64; ++c) tma_heads(dst + c * CH, m, full, 64 * c, n, h, b);
        };
        auto load_k = [&](int j) -> bool {
          const int st = kn % KS;
          if (kn >= KS && !mbar_wait(&k_empty[st], (kn / KS - 1) & 1, abort_flag, p.err)) return false;
          load(a.k, smem + L::OFF_K + st * L::TILE, &k_full[st], BN, j * BN, it.hk, it.b);
          ++kn;
          return true;
        };
        auto load_v = [&](const HeadsMap& m, int rows, int n, int h) -> bool {
          const int st = vn % VS;
          if (vn >= VS && !mbar_wait(&v_empty[st], (vn / VS - 1) & 1, abort_flag, p.err)) return false;
          load(m, smem + L::OFF_V + st * L::TILE, &v_full[st], rows, n, h, it.b);
          ++vn;
          return true;
        };
        for (bool ok = true; ok && w.get(it); w.next(a)) {
          int g, n;
          divide(it.tile, a.per_head, g, n);
          const int h = it.hk * G + g * a.heads;
          n *= BM;
          if (qn > 0 && !mbar_wait(q_empty, (qn - 1) & 1, abort_flag, p.err)) break;
          load(a.q, q_tile, q_full, a.box, n, h, it.b);
          ++qn;
          if (!load_k(it.j0) || !load_v(a.o, a.box, n, h)) break;
          if (dn > 0 && !mbar_wait(do_empty, (dn - 1) & 1, abort_flag, p.err)) break;
          load(a.dout, do_tile, do_full, a.box, n, h, it.b);
          ++dn;
          ok = load_v(a.v, BN, it.j0 * BN, it.hk);
          for (int j = it.j0 + 1; ok && j < it.j1; ++j) ok = load_k(j) && load_v(a.v, BN, j * BN, it.hk);
        }
        if (*abort_flag) {
          volatile int no_abort = 0;
          if (qn > 0) mbar_wait(q_full, (qn - 1) & 1, &no_abort, p.err);
          if (dn > 0) mbar_wait(do_full, (dn - 1) & 1, &no_abort, p.err);
          for (int i = max(0, kn - KS); i < kn; ++i) mbar_wait(&k_full[i % KS], (i / KS) & 1, &no_abort, p.err);
          for (int i = max(0, vn - VS); i < vn; ++i) mbar_wait(&v_full[i % VS], (i / VS) & 1, &no_abort, p.err);
        }
      }
      __syncwarp();
    } else if (warp == R::W_MMA) {
      // S of every step, once the one before has been read
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, true, false, false);
      int n = 0;
      bool ok = true;
      for (int i = 0; ok && w.get(it); w.next(a), ++i) {
        ok = mbar_wait(qt_full, i & 1, abort_flag, p.err);
        for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
          ok = mbar_wait(&k_full[n % KS], (n / KS) & 1, abort_flag, p.err) &&
               (n == 0 || mbar_wait(s_free, (n - 1) & 1, abort_flag, p.err));
          if (!ok) break;
          // rows of K behind the sequence's keys may be anything: dS is 0 there, and 0 x NaN is not
          uint8_t* k = smem + L::OFF_K + n % KS * L::TILE;
          if (it.len - j * BN < BN && it.len < p.Nk) clear_rows<D>(k, it.len - j * BN, lane);
          tc_fence_after();
          const uint32_t b = desc_rows(smem_u32(k));
          if (leader) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              mma_ts(tbase + COL_S, tbase + COL_Q + 8 * x, b + (((x / 4) * CH + (x % 4) * 32) >> 4), idesc_s, x > 0);
            mma_commit(s_full);
          }
          __syncwarp();
        }
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    } else if (warp == R::W_MMA_B) {
      // dP of every step, once the one before has been read; then dQ of that one
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, true, false, false);
      const uint32_t idesc_q = idesc_f16(BM, D, true, false, true);
      const uint32_t sdo = smem_u32(do_tile);
      int v = 0, n = 0;                    // ring position of V; steps whose dP is issued
      bool ok = true, add = false;
      // dQ += dS K of step m; last: of its item
      auto issue_dq = [&](int m, bool last) -> bool {
        if (!mbar_wait(ds_full, m & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        const uint32_t sk = smem_u32(smem + L::OFF_K + m % KS * L::TILE);
        if (leader) {
          product_cols(tbase + COL_DQ, tbase + COL_DS, sk, idesc_q, add);
          mma_commit(ds_free);
          mma_commit(&k_empty[m % KS]);
          if (last) mma_commit(dq_done);
        }
        __syncwarp();
        add = !last;
        return true;
      };
      for (int i = 0; ok && w.get(it); w.next(a), ++i) {
        for (int j = it.j0; ok && j < it.j1; ++j) {
          const bool first = j == it.j0;
          if (first) ++v;                  // (o)
          if (first && n > 0) ok = issue_dq(n - 1, true);
          if (n > 0) ok = ok && mbar_wait(dp_free, (n - 1) & 1, abort_flag, p.err);
          if (first) ok = ok && mbar_wait(do_full, i & 1, abort_flag, p.err);
          ok = ok && mbar_wait(&v_full[v % VS], (v / VS) & 1, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = smem_u32(smem + L::OFF_V + v % VS * L::TILE);
          if (leader) {
            product_rows<D>(tbase + COL_DP, sdo, sv, idesc_s);
            mma_commit(dp_full);
            mma_commit(&v_empty[v % VS]);
            if (j == it.j1 - 1) mma_commit(do_empty);
          }
          __syncwarp();
          if (!first) ok = issue_dq(n - 1, false);
          ++n;
          ++v;
        }
      }
      if (ok && n > 0) issue_dq(n - 1, true);
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<R::REG_SOFT>();
    const int part = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const float c = p.c;
    int n = 0, items = 0;                  // key tiles, items so far
    int o = 0;                             // ring position of the item's o
    bool ok = true, leaving = false;       // leaving: a dQ is on its way out of shared memory
    if (p.lens)                            // queries without a key
      for (int i = blockIdx.x; i < a.items; i += gridDim.x) {
        int bh, b, hk, tile, g, row;
        divide(i, a.per_kv, bh, tile);
        divide(bh, a.hkv, b, hk);
        tile_row(a, tile, r, G, g, row);
        if (g >= G || key_count(p, b, false) > 0) continue;
        uint4* dst = reinterpret_cast<uint4*>(at(p.dq, b, hk * G + g, row) + part * (D / 4));
        for (int x = 0; x < D / 32; ++x) dst[x] = make_uint4(0, 0, 0, 0);
      }
    // the item's row and its lse
    bool valid = false;
    int h = 0, row = 0;
    float lse = INFINITY;
    auto fetch = [&](const ItemQ& x) {
      int g;
      tile_row(a, x.tile, r, G, g, row);
      valid = g < G;
      h = x.hk * G + g;
      lse = valid ? p.lse[((long long)x.b * p.Hq + h) * p.Nq + row] : INFINITY;
    };
    // this quarter of the item's Q row into tensor memory
    auto take_q = [&](int i) -> bool {
      if (!mbar_wait(q_full, i & 1, abort_flag, p.err)) return false;
      uint32_t v[D / 8];
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 u = *tile_word(q_tile, r, part * (D / 32) + x);
        v[4 * x] = u.x; v[4 * x + 1] = u.y; v[4 * x + 2] = u.z; v[4 * x + 3] = u.w;
      }
      if constexpr (D == 128) tmem_st16(lane_base + COL_Q + 16 * part, v);
      else tmem_st8(lane_base + COL_Q + 8 * part, v);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qt_full);
      return true;
    };
    bool more = w.get(it);
    if (more) {
      fetch(it);
      ok = take_q(0);
      if (lane == 0) mbar_arrive(q_empty);
    }
    // (A warp whose wait ran out still meets the others at the barriers.)
    while (more) {
      // D: this quarter's share from the o and dO tiles, then all of them in their order
      float del = 0.f, z = INFINITY;       // (a row without keys: P = 2^-inf = 0)
      if (lse > -INFINITY) z = lse * L2E;
      ok = ok && mbar_wait(do_full, items & 1, abort_flag, p.err) &&
           mbar_wait(&v_full[o % VS], (o / VS) & 1, abort_flag, p.err);
      if (ok) {
        uint8_t* ot = smem + L::OFF_V + o % VS * L::TILE;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int x = part * (D / 32) + i;
          const uint4 u = *tile_word(ot, r, x), y = *tile_word(do_tile, r, x);
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            del = fmaf(__uint_as_float(uw[e] << 16), __uint_as_float(yw[e] << 16), del);
            del = fmaf(__uint_as_float(uw[e] & 0xffff0000u), __uint_as_float(yw[e] & 0xffff0000u), del);
          }
        }
      }
      shares[part * 128 + r] = del;
      named_bar(1, R::SOFT);
      del = (shares[r] + shares[128 + r]) + (shares[256 + r] + shares[384 + r]);
      if (lane == 0) {
        mbar_arrive(do_empty);
        if (leaving) {                     // the dQ before this one has left the place of Q
          bulk_wait_read0();
          mbar_arrive(q_empty);
        }
      }
      if (threadIdx.x == 0) mbar_arrive(&v_empty[o % VS]);
      if (ok && valid && part == 0) a.del[((long long)it.b * p.Hq + h) * p.Nq + row] = del;
      o += it.j1 - it.j0 + 1;
      for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
        if (!mbar_wait(s_full, n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        // (two elements an instruction)
        float2 e[16];
        {
          uint32_t v[32];
          load_columns(lane_base + COL_S + 32 * part, v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y = ffma2(pair(v, i), make_float2(c, c), make_float2(-z, -z));
            e[i] = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          }
        }
        if (!mbar_wait(dp_full, n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        const int keep = it.len - j * BN - 32 * part;
        uint32_t pk[16];
        {
          uint32_t v[32];
          load_columns(lane_base + COL_DP + 32 * part, v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_free);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            e[i] = fmul2(e[i], fadd2(pair(v, i), make_float2(-del, -del)));
            pk[i] = pack2(e[i].x, e[i].y);
          }
        }
        if (keep < 32) {
          // (what masked keys gave may be NaN: dS is 0 there)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (2 * i >= keep) pk[i] = 0;
            else if (2 * i + 1 >= keep) pk[i] &= 0xffffu;
          }
        }
        if (n >= 1 && !mbar_wait(ds_free, (n - 1) & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        tmem_st16(lane_base + COL_DS + 16 * part, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      // the next item's Q goes into tensor memory before this one's dQ is awaited, and dQ then into Q's place
      const ItemQ was = it;
      const bool here = valid;
      __nv_bfloat16* dst = here ? at(p.dq, it.b, h, row) + part * (D / 4) : nullptr;
      w.next(a);
      more = w.get(it);
      if (more) {
        fetch(it);
        ok = ok && take_q(items + 1);
      }
      named_bar(1, R::SOFT);
      ok = ok && mbar_wait(dq_done, items & 1, abort_flag, p.err);
      ++items;
      if (ok) {
        tc_fence_after();
        // (rows by themselves would be 32 places a store: they leave in boxes of 32 rows)
        uint32_t v[D / 4];
        load_columns(lane_base + COL_DQ + part * (D / 4), v);
        if (!was.whole) {
          // (the first item of the range in slot 0, its last one in slot 1)
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            *reinterpret_cast<uint4*>(partial(a.part_q, D, 2 * blockIdx.x + (items > 1), r, part * (D / 4) + 4 * e)) =
                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else if (a.heads > 1) {
          if (here) store_row(dst, v, p.scale, a.dq32);
        } else {
          const float f = p.scale;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pk[i] = pack2(pair(v, 4 * e + i).x * f, pair(v, 4 * e + i).y * f);
            *tile_word(q_tile, r, part * (D / 32) + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
      }
      __syncwarp();
      // (all quarters of a box of 64 channels)
      const int box = part * (D / 4) / 64;
      named_bar(2 + quad * (D / 64) + box, 8192 / D);
      if (lane == 0) {
        int g, m;
        divide(was.tile, a.per_head, g, m);
        m = m * BM + 32 * quad;
        if (ok && was.whole && a.heads == 1 && m < p.Nq && part * (D / 4) % 64 == 0) {
          tma_heads_store(a.dq, q_tile + box * CH + quad * 32 * 128, 64 * box, m, was.hk * G + g, was.b);
          bulk_commit();
        }
      }
      __syncwarp();
      leaving = true;
    }
    if (lane == 0) bulk_wait_read0();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == R::W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
// STAGED: dV and dK leave in boxes of 32 rows through shared memory (2 tiles of 64
// channels).  At d = 128 that takes a place of the ring of five, which costs long lines
// more than their ends gain: lines of up to STAGED_STEPS steps do so (24 heads of 2048
// keys: 1 step 36.7 against 38.6 us, 8 steps 101.9 and 103.9, 16 steps 159 and 161, 64
// steps 530 and 509).
constexpr int STAGED_STEPS = 24;
template <int D, bool STAGED>
struct SmemK {
  static constexpr int TILE = (D / 64) * CH;
  static constexpr int RS = D == 128 ? (STAGED ? 4 : 5) : 8; // ring: Q, dO, Q, dO, ...
  static constexpr int OFF_K = 0, OFF_V = TILE, OFF_R = 2 * TILE;
  static constexpr int OFF_OUT = OFF_R + RS * TILE;         // 64 channels of dV and of dK on their way out
  static constexpr int OFF_ST = OFF_OUT + (STAGED ? 2 * CH : 0);   // [2] x (-lse log2 e [128], -D [128])
  static constexpr int OFF_BAR = OFF_ST + 2 * 1024;
  static constexpr int NBAR = 4 + 2 * RS + 4 + 9;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 64;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

template <int D, bool STAGED>
__global__ void __launch_bounds__(Roles<8>::NTHREADS, 1) cross_dkv_kernel(const __grid_constant__ Params a) {
  using L = SmemK<D, STAGED>;
  using K = Roles<8>;
  constexpr int RS = L::RS;
  constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DV = 256, COL_DK = 256 + D;
  const CrossParams& p = a.p;
  // (no room to align it by hand: nothing else is in shared memory, so it begins on its alignment)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {
    atomicOr(p.err, FA4_DEVERR_TIMEOUT);
    return;
  }
  next_may_start();
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_empty = k_full + 1;
  uint64_t* v_full = k_empty + 1;
  uint64_t* v_empty = v_full + 1;
  uint64_t* r_full = v_empty + 1;
  uint64_t* r_empty = r_full + RS;
  uint64_t* st_full = r_empty + RS;      // [2]
  uint64_t* st_empty = st_full + 2;
  uint64_t* s_full = st_empty + 2;
  uint64_t* s_seen = s_full + 1;         // the step's threads have seen s_full
  uint64_t* p_full = s_seen + 1;         // [2] halves: P^T is there
  uint64_t* dp_full = p_full + 2;
  uint64_t* ds_full = dp_full + 1;       // [2] halves: dS^T is there
  uint64_t* acc_done = ds_full + 2;      // the line's dV and dK are there
  uint64_t* mma_done = acc_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  Range* range = reinterpret_cast<Range*>(smem + L::OFF_MISC + 8);
  static_assert(sizeof(Range) <= 56, "range's place");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1); mbar_init(k_empty, 1); mbar_init(v_full, 1); mbar_init(v_empty, 1);
    for (int s = 0; s < RS; ++s) { mbar_init(&r_full[s], 1); mbar_init(&r_empty[s], 2); }
    for (int s = 0; s < 2; ++s) { mbar_init(&st_full[s], 1); mbar_init(&st_empty[s], 8); }
    mbar_init(s_full, 1);
    mbar_init(s_seen, 1);
    mbar_init(dp_full, 1);
    for (int s = 0; s < 2; ++s) { mbar_init(&p_full[s], 8); mbar_init(&ds_full[s], 8); }
    mbar_init(acc_done, 2);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  // rows of a ring slot that no box brings are zeros, and so are those that it brings from behind the kv head's heads:
  // P and dS are 0 there, and 0 x NaN is not
  if (a.box < BM)
    for (int i = threadIdx.x; i < RS * L::TILE / 16; i += K::NTHREADS)
      reinterpret_cast<uint4*>(smem + L::OFF_R)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == K::W_PROD) {
    const Range x = find_range(a, false, lane);
    if (lane == 0) *range = x;
  }
  if (warp == K::W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const int G = p.Hq / p.Hkv;
  Range at_ = *range;

  if (warp >= K::W_PROD) {
    setmaxnreg_dec<K::REG_MISC>();
    if (warp == K::W_PROD) {
      if (lane == 0) {
        tma_prefetch_desc(&a.q.map);
        tma_prefetch_desc(&a.dout.map);
        tma_prefetch_desc(&a.k.map);
        tma_prefetch_desc(&a.v.map);
        int ln = 0, rn = 0, kn = 0, vn = 0;      // lines begun; tiles issued
        auto load_kv = [&](const HeadsMap& m, uint64_t* full, uint64_t* empty, int off, int& count) -> bool {
          if (ln > 0 && !mbar_wait(empty, (ln - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(full, L::TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + off + c * CH, m, full, 64 * c, at_.tile * BN, at_.hk, at_.b);
          ++count;
          return true;
        };
        auto load_r = [&](const HeadsMap& m, const HeadsMap& group) -> bool {
          const int st = rn % RS;
          if (rn >= RS && !mbar_wait(&r_empty[st], (rn / RS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&r_full[st], a.box * 2 * D);
          int g, n;
          divide(at_.t, a.per_head, g, n);
          n *= BM;
          for (int c = 0; c < D / 64; ++c) {
            uint8_t* dst = smem + L::OFF_R + st * L::TILE + c * CH;
            if (a.heads > 1) tma_group(dst, group, &r_full[st], 64 * c, n, g * a.heads, at_.hk, at_.b);
            else tma_heads(dst, m, &r_full[st], 64 * c, n, at_.hk * G + g, at_.b);
          }
          ++rn;
          return true;
        };
        bool ok = true, fresh = true;
        while (ok && at_.left > 0) {
          ok = load_r(a.q, a.group_q) && (!fresh || load_kv(a.k, k_full, k_empty, L::OFF_K, kn)) && load_r(a.dout, a.group_dout) &&
               (!fresh || load_kv(a.v, v_full, v_empty, L::OFF_V, vn));
          if (fresh) ++ln;
          fresh = false;
          --at_.left;
          if (++at_.t == a.tiles && at_.left > 0) {
            at_.line(a, false);
            fresh = true;
          }
        }
        if (*abort_flag) {
          volatile int no_abort = 0;
          for (int i = max(0, rn - RS); i < rn; ++i) mbar_wait(&r_full[i % RS], (i / RS) & 1, &no_abort, p.err);
          if (kn > 0) mbar_wait(k_full, (kn - 1) & 1, &no_abort, p.err);
          if (vn > 0) mbar_wait(v_full, (vn - 1) & 1, &no_abort, p.err);
        }
      }
      __syncwarp();
    } else if (warp == K::W_MMA_B + 1) {
      // (D is the first kernel's, which let this one start when the grids before it had ended; every CTA waits for it,
      // so that this kernel does not end before it)
      wait_for_previous();
      // -lse log2 e and -D of each step's queries (infinite lse where there is none: P = 0)
      float z[4], d4[4];
      auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int g, n;
          tile_row(a, at_.t, 4 * lane + i, G, g, n);
          z[i] = -INFINITY;
          d4[i] = 0.f;
          if (g < G) {
            const long long flat = ((long long)at_.b * p.Hq + at_.hk * G + g) * p.Nq + n;
            const float v = p.lse[flat];
            if (v > -INFINITY) z[i] = -v * L2E;
            d4[i] = -a.del[flat];
          }
        }
      };
      if (at_.left > 0) fetch();
      for (int n = 0; at_.left > 0; ++n) {
        const int st = n & 1;
        if (n >= 2 && !mbar_wait(&st_empty[st], (n / 2 - 1) & 1, abort_flag, p.err)) break;
        float* dst = reinterpret_cast<float*>(smem + L::OFF_ST + st * 1024);
        reinterpret_cast<float4*>(dst)[lane] = make_float4(z[0], z[1], z[2], z[3]);
        reinterpret_cast<float4*>(dst + 128)[lane] = make_float4(d4[0], d4[1], d4[2], d4[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[st]);
        --at_.left;
        if (at_.left == 0) break;
        if (++at_.t == a.tiles) at_.line(a, false);
        fetch();
      }
    } else if (warp == K::W_MMA || warp == K::W_MMA_B) {
      // the first warp issues S^T and dV, the second dP^T and dK.  Each overwrites, in its own order, what its own
      // product before has read: S^T the P^T, dP^T the dS^T.
      const int x = warp == K::W_MMA ? 0 : 1;
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, true, false, false);
      const uint32_t idesc_a = idesc_f16(BM, D, true, false, true);
      const uint32_t fixed = smem_u32(smem + (x ? L::OFF_V : L::OFF_K));
      const uint32_t col = tbase + (x ? COL_DP : COL_S), sum = tbase + (x ? COL_DK : COL_DV);
      uint64_t *full = x ? v_full : k_full, *empty = x ? v_empty : k_empty;
      uint64_t *there = x ? dp_full : s_full, *ready = x ? ds_full : p_full;
      const int steps = at_.left;
      int t = at_.t, lines = 0;              // the next step's place in its line; lines begun
      auto issue = [&](int n, bool first, bool last) -> bool {
        const int seq = 2 * n + x;           // Q for S^T, dO for dP^T
        if (first) {
          if (!mbar_wait(full, lines & 1, abort_flag, p.err)) return false;
          ++lines;
        }
        if (!mbar_wait(&r_full[seq % RS], (seq / RS) & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        const uint32_t b = smem_u32(smem + L::OFF_R + seq % RS * L::TILE);
        if (leader) {
          product_rows<D>(col, fixed, b, idesc_s);
          mma_commit(there);
          mma_commit(&r_empty[seq % RS]);
          if (last) mma_commit(empty);
        }
        __syncwarp();
        return true;
      };
      // of the step whose product is awaited: is it the first, the last here of its line?
      bool first = true, last = steps == 1 || t + 1 == a.tiles;
      bool ok = steps == 0 || issue(0, true, last);
      for (int n = 0; ok && n < steps; ++n) {
        t = t + 1 == a.tiles ? 0 : t + 1;
        const bool next_last = n + 2 == steps || t + 1 == a.tiles;
        const int seq = 2 * n + 1 - x;       // dO for dV, Q for dK (it has arrived: the step's scores are there)
        ok = mbar_wait(&r_full[seq % RS], (seq / RS) & 1, abort_flag, p.err) &&
             mbar_wait(ready, n & 1, abort_flag, p.err);
        // products of the two warps share the tensor cores, and the next S^T is what the key's threads wait for
        // first.  (They say that they have it: s_full itself may be a phase further by now.  At a line's end they are
        // waiting for its dK before they look at the next S^T.)
        if (x == 1 && !last) ok = ok && mbar_wait(s_seen, (n + 1) & 1, abort_flag, p.err);
        if (!ok) break;
        const uint32_t b = smem_u32(smem + L::OFF_R + seq % RS * L::TILE);
        tc_fence_after();
        if (leader) product_half(sum, col, col + 64, b, idesc_a, 0, !first);
        __syncwarp();
        if (!mbar_wait(&ready[1], n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        if (leader) {
          product_half(sum, col, col + 64, b, idesc_a, 1, true);
          mma_commit(&r_empty[seq % RS]);
          if (last) mma_commit(acc_done);
        }
        __syncwarp();
        if (n + 1 < steps) ok = issue(n + 1, last, next_last);
        first = last;
        last = next_last;
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<K::REG_SOFT>();
    const int half = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const float c = p.c;
    // half of the thread's P^T or dS^T: its product begins with it
    auto give = [&](uint32_t column, const uint32_t (&w)[16], uint64_t* bar) {
      tmem_st16(lane_base + column + 64 * half, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int n = 0, lines = 0;
    bool ok = true;
    while (ok && at_.left > 0) {
      const int s0 = at_.t, s1 = min(a.tiles, s0 + at_.left);
      for (; at_.t < s1; ++at_.t, ++n) {
        const int st = n & 1;
        const float* stat = reinterpret_cast<const float*>(smem + L::OFF_ST + st * 1024) + 64 * half;
        if (!mbar_wait(&st_full[st], (n / 2) & 1, abort_flag, p.err) || !mbar_wait(s_full, n & 1, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (threadIdx.x == 0) mbar_arrive(s_seen);
        tc_fence_after();
        float2 e[32];
        uint32_t pk[2][16];
        {
          uint32_t v[2][32];
          tmem_ld32(lane_base + COL_S + 64 * half, v[0]);
          tmem_ld32(lane_base + COL_S + 64 * half + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            if (i == 16) give(COL_S, pk[0], p_full);
            const float4 z = *reinterpret_cast<const float4*>(stat + 2 * i);
            const float2 x = ffma2(pair(v[i / 16], i % 16), make_float2(c, c), make_float2(z.x, z.y));
            const float2 y = ffma2(pair(v[i / 16], i % 16 + 1), make_float2(c, c), make_float2(z.z, z.w));
            e[i] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            e[i + 1] = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            pk[i / 16][i % 16] = pack2(e[i].x, e[i].y);
            pk[i / 16][i % 16 + 1] = pack2(e[i + 1].x, e[i + 1].y);
          }
        }
        give(COL_S + 16, pk[1], p_full + 1);
        if (!mbar_wait(dp_full, n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        {
          uint32_t v[2][32];
          tmem_ld32(lane_base + COL_DP + 64 * half, v[0]);
          tmem_ld32(lane_base + COL_DP + 64 * half + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            if (i == 16) give(COL_DP, pk[0], ds_full);
            const float4 z = *reinterpret_cast<const float4*>(stat + 128 + 2 * i);
            const float2 x = fmul2(e[i], fadd2(pair(v[i / 16], i % 16), make_float2(z.x, z.y)));
            const float2 y = fmul2(e[i + 1], fadd2(pair(v[i / 16], i % 16 + 1), make_float2(z.z, z.w)));
            pk[i / 16][i % 16] = pack2(x.x, x.y);
            pk[i / 16][i % 16 + 1] = pack2(y.x, y.y);
          }
        }
        give(COL_DP + 16, pk[1], ds_full + 1);
        if (lane == 0) mbar_arrive(&st_empty[st]);
      }
      if (!ok) break;
      // the line's sums: warps 0-3 dV, warps 4-7 dK, a key each
      if (!mbar_wait(acc_done, lines & 1, abort_flag, p.err)) { ok = false; break; }
      tc_fence_after();
      const bool whole = s0 == 0 && s1 == a.tiles;
      const int key = at_.tile * BN + r;
      const float f = half ? p.scale : 1.f;
      uint8_t* out = smem + L::OFF_OUT + half * CH;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t v[32];
        tmem_ld32(lane_base + (half ? COL_DK : COL_DV) + 32 * q, v);
        tmem_ld_wait();
        reg_fence32(v);
        // (what lies behind the sequence's keys may have come out as NaN)
        if (key >= at_.len) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (!whole) {
          // (the first line of the range in slot 0, its last one in slot 1)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(partial(a.part, D, (2 * blockIdx.x + (lines > 0)) * 2 + half, r, 32 * q + 4 * e)) =
                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          continue;
        }
        if (!STAGED) {
          if (key < p.Nk) store_row(at(half ? p.dk : p.dv, at_.b, at_.hk, key) + 32 * q, v, f, half ? a.dk32 : a.dv32);
          continue;
        }
        // rows by themselves would be 32 places a store: they leave in boxes of 32 rows and 64 channels
        if (q % 2 == 0) {
          if (lane == 0) bulk_wait_read0();
          __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pk[i] = pack2(__uint_as_float(v[8 * e + 2 * i]) * f, __uint_as_float(v[8 * e + 2 * i + 1]) * f);
          *tile_word(out, r, q % 2 * 4 + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (q % 2 == 1) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && at_.tile * BN + 32 * quad < p.Nk) {
            tma_heads_store(half ? a.dk : a.dv, out + quad * 32 * 128, q / 2 * 64, at_.tile * BN + 32 * quad, at_.hk,
                            at_.b);
            bulk_commit();
          }
        }
      }
      tc_fence_before();
      ++lines;
      at_.left -= s1 - s0;
      if (at_.left > 0) at_.line(a, false);
    }
    if (lane == 0) bulk_wait_read0();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == K::W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

// The sum of a tile's partials, EACH times 8 columns of a row for a thread; thin: the steps, where some ranges are
// empty.
template <int D, int EACH>
FA4_DEV void join(const Params& a, const Strided& out, const Range& place, int slot0, int c0, int c1, long long thin) {
  const CrossParams& p = a.p;
  const int which = blockIdx.y, G = p.Hq / p.Hkv;
  const bool rows = which == 2;
  const int side = rows ? 1 : a.side, ranges = rows ? a.ctas : a.ranges;
  const float f = which ? p.scale : 1.f;
  float* part = rows ? a.part_q : a.part;
  constexpr int STRIDE = 128 * (D / 8) / EACH;    // threads of all parts
  const int x0 = blockIdx.z * 256 + threadIdx.x;
  float v[EACH][8] = {};
  const auto add = [&](int c) {
    const int slot = 2 * (c * side + place.tile % side) + (c == c0 ? slot0 : 0);
    const int at = rows ? slot : 2 * slot + which;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int x = x0 + e * STRIDE;
      const float4 u = *reinterpret_cast<const float4*>(partial(part, D, at, x % 128, x / 128 * 8));
      const float4 w = *reinterpret_cast<const float4*>(partial(part, D, at, x % 128, x / 128 * 8 + 4));
      v[e][0] += u.x; v[e][1] += u.y; v[e][2] += u.z; v[e][3] += u.w;
      v[e][4] += w.x; v[e][5] += w.y; v[e][6] += w.z; v[e][7] += w.w;
    }
  };
  if (!thin) {
    constexpr int AHEAD = EACH == 1 ? 8 : 4;
#pragma unroll AHEAD
    for (int c = c0; c <= c1; ++c) add(c);
  } else {
    for (int c = c0; c <= c1; ++c)
      if (range_start(thin, c + 1, ranges) > range_start(thin, c, ranges)) add(c);
  }
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int x = x0 + e * STRIDE, r = x % 128, i = x / 128 * 8;
    int h = place.hk, row = place.tile * BN + r;
    bool valid = row < p.Nk;
    if (rows) {
      int g;
      tile_row(a, place.tile, r, G, g, row);
      valid = g < G;
      h = place.hk * G + g;
    }
    if (valid)
      *reinterpret_cast<uint4*>(fa4::at(out, place.b, h, row) + i) =
          make_uint4(pack2(v[e][0] * f, v[e][1] * f), pack2(v[e][2] * f, v[e][3] * f), pack2(v[e][4] * f, v[e][5] * f),
                     pack2(v[e][6] * f, v[e][7] * f));
  }
}

// dV (y = 0), dK (y = 1) and dQ (y = 2) of the output tiles whose steps lie in
// several ranges: a few CTAs (z) for each x below a.joins.  That is an output tile, where
// there are fewer of them than ranges, or else a range that ends inside a tile's steps
// and began at or before their first.  Then, where sequences have lengths, zeros for
// the key tiles behind them: an x for each sequence and kv head.
// Tiles of four ranges and more are shared by D / 16 CTAs, a row's 8 columns a thread, the
// others by two (6 heads, 76,666 queries, 188 keys 202 -> 167 us).  An x for every
// range and all parts for every sum were 3600 CTAs of which 50 found something (7
// heads, 241 queries, 1..1590 keys 38.0 -> 31.7 us; 6 heads, 5985 queries, 87 keys 40 -> 35).
// FEW: are there such tiles?  (Their sums take more registers.)
template <int D, bool FEW>
__global__ void __launch_bounds__(256, FEW ? 2 : 3) cross_join_kernel(const __grid_constant__ Params a) {
  const CrossParams& p = a.p;
  const int which = blockIdx.y;
  const Strided& out = which == 2 ? p.dq : which ? p.dk : p.dv;
  if ((int)blockIdx.x >= a.joins) {
    wait_for_previous();
    if (which == 2 || blockIdx.z > 0) return;
    int b, hk;
    divide((int)blockIdx.x - a.joins, a.hkv, b, hk);
    const int from = (key_count(p, b, false) + BN - 1) / BN * BN;
    for (long long x = threadIdx.x; x < (long long)(p.Nk - from) * (D / 8); x += 256)
      *reinterpret_cast<uint4*>(at(out, b, hk, from + (int)(x / (D / 8))) + x % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool rows = which == 2;
  const int parts = rows ? a.parts_q : a.parts_k;
  if ((int)blockIdx.z >= parts) return;
  const int side = rows ? 1 : a.side, ranges = rows ? a.ctas : a.ranges;
  __shared__ Range place;                         // (left: is there anything to join?)
  __shared__ int slot0, c0, c1, thin;
  __shared__ long long sum;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const long long total = all_steps(a, rows, lane);
    long long start = 0;                          // the tile's first step
    Range x;
    x.left = 0;
    if (rows ? a.by_query_tile : a.by_key_tile) {
      const int each = rows ? a.tiles : a.key_tiles, bh = blockIdx.x / each;
      x.tile = blockIdx.x - bh * each;
      divide(bh, a.hkv, x.b, x.hk);
      if (x.b < p.B) {
        x.nt = tiles_of(a, x.b);
        x.left = rows ? x.nt > 0 : x.tile < x.nt;
        start = (long long)x.b * a.key_tiles;     // key tiles of the sequences before
        if (p.lens) {
          start = 0;
          for (int b = lane; b < x.b; b += 32) start += tiles_of(a, b);
          for (int o = 16; o > 0; o /= 2) start += __shfl_xor_sync(0xffffffffu, start, o);
        }
        start = start / side * p.Hkv * a.tiles +
                (rows ? (long long)(x.hk * a.tiles + x.tile) * x.nt
                      : (long long)(x.hk * (x.nt / side) + x.tile / side) * a.tiles);
      }
    } else {
      const int c = blockIdx.x / side;            // (may be behind the last range)
      const long long begin = range_start(total, c, ranges), end = range_start(total, c + 1, ranges);
      if (end > begin && end < total) {
        find_step(a, end, rows, blockIdx.x % side, lane, x);
        start = end - x.t;
        x.left = x.t > 0 && begin <= start;
      }
    }
    if (x.left && lane == 0) {
      // the ranges of its first and last step
      c0 = (int)quotient((start + 1) * ranges - 1, total);
      c1 = (int)quotient((start + (rows ? x.nt : a.tiles)) * ranges - 1, total);
      slot0 = range_start(total, c0, ranges) < start;      // (slot 1 where the range began in a tile before)
      thin = total < ranges;                               // some ranges are empty: each has a step at most
      sum = total;
      x.left = c0 < c1;
    }
    if (lane == 0) place = x;
  }
  // (where the sums lie follows from the shapes and lengths: the partials are waited for after that, by every CTA,
  // so that this kernel does not end before the ones before it)
  wait_for_previous();
  __syncthreads();
  if (!place.left) return;
  if (!FEW || parts == 2) join<D, D / 32>(a, out, place, slot0, c0, c1, thin ? sum : 0);
  else join<D, 1>(a, out, place, slot0, c0, c1, thin ? sum : 0);
}

// Zeros where there is no partner at all.
__global__ void __launch_bounds__(256) cross_zero_kernel(Strided t, int H, int N, int d, long long words) {
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= words) return;
  const int per = d / 8, i = (int)(x % per) * 8;
  const long long row = x / per;
  const int n = (int)(row % N), bh = (int)(row / N);
  *reinterpret_cast<uint4*>(at(t, bh / H, bh % H, n) + i) = make_uint4(0, 0, 0, 0);
}

cudaError_t zero(const Strided& t, int B, int H, int N, int d, cudaStream_t st) {
  const long long words = (long long)B * H * N * (d / 8);
  if (words > 0) cross_zero_kernel<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(t, H, N, d, words);
  return cudaGetLastError();
}

// Query tiles as in the forward, and the kernels' ranges.
constexpr int SIDE_MAX = 8;
void plan(Params& a, int B, int Hq, int Hkv, int Nq, int Nk, bool share, bool lens) {
  const int G = Hq / Hkv;
  a.heads = share && Nq <= 64 ? (128 / Nq < G ? 128 / Nq : G) : 1;
  a.per_head = Divisor((Nq + BM - 1) / BM);
  a.tiles = a.heads > 1 ? (G + a.heads - 1) / a.heads : G * a.per_head.d;
  a.per_kv = Divisor(a.tiles);
  a.hkv = Divisor(Hkv);
  a.nq = Divisor(Nq);
  a.box = a.heads > 1 ? a.heads * Nq : BM;
  a.items = (int)((long long)B * Hkv * a.tiles);
  a.key_tiles = (Nk + BN - 1) / BN;
  const long long steps = (long long)B * Hkv * a.key_tiles * a.tiles;
  const int sms = sm_count();
  a.slots = (int)(steps < sms ? steps : sms);
  // as many key tiles side by side as divide them and leave no more than a fiftieth of the CTAs over
  a.side = 1;
  if (!lens)
    for (int n = 2; n <= SIDE_MAX; ++n)
      if (a.key_tiles % n == 0 && a.slots % n * 50 <= a.slots) a.side = n;
  // short ranges: no more of them than the longest needs, and fewer partials (182 steps are 91 ranges of two, not 152
  // of one or two: 7 heads, 241 queries, 1590 keys 34.1 -> 30.4 us; 24 heads, 5 queries, 6943 keys 31.4 -> 25.8;
  // ranges of 111 steps gain nothing: 324 -> 332).  With lengths the steps are fewer, nobody here knows how many.
  const auto ranges = [lens](long long n, int most) {
    const long long each = (n + most - 1) / most;
    return lens || each < 2 || each > 8 ? most : (int)((n + each - 1) / each);
  };
  a.ctas = ranges(steps, a.slots);
  a.ranges = ranges(steps / a.side, a.slots / a.side);
}

size_t del_bytes(int B, int Hq, int Nq) { return ((size_t)B * Hq * Nq * sizeof(float) + 127) / 128 * 128; }

bool on_words(const Strided& t) { return (reinterpret_cast<uintptr_t>(t.p) & 31) == 0 && ((t.b | t.h | t.n) & 15) == 0; }

cudaError_t start(void (*kernel)(const Params), dim3 grid, int threads, int smem, bool early, const Params& a, cudaStream_t st) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
  return e != cudaSuccess ? e : launch(kernel, grid, threads, smem, early, st, a);
}

}  // namespace

size_t cross_bwd_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (Nq == 0 || Nk == 0) return 0;
  // (heads that share no tile make more tiles, never fewer CTAs)
  Params a;
  plan(a, B, Hq, Hkv, Nq, Nk, false, true);
  return del_bytes(B, Hq, Nq) + (size_t)a.slots * 6 * 128 * d * sizeof(float);
}

cudaError_t launch_cross_bwd(const CrossParams& p, cudaStream_t st) {
  if (p.Nk == 0) return zero(p.dq, p.B, p.Hq, p.Nq, p.d, st);
  if (p.Nq == 0) {
    const cudaError_t e = zero(p.dk, p.B, p.Hkv, p.Nk, p.d, st);
    return e != cudaSuccess ? e : zero(p.dv, p.B, p.Hkv, p.Nk, p.d, st);
  }
  Params a;
  a.p = p;
  plan(a, p.B, p.Hq, p.Hkv, p.Nq, p.Nk, p.q.h != 0 && p.dout.h != 0 && p.o.h != 0,
       p.lens != nullptr);
  a.dq32 = on_words(p.dq); a.dk32 = on_words(p.dk); a.dv32 = on_words(p.dv);
  a.del = reinterpret_cast<float*>(p.work);
  a.part = reinterpret_cast<float*>(p.work + del_bytes(p.B, p.Hq, p.Nq));
  a.part_q = a.part + (size_t)a.slots * 4 * 128 * p.d;
  const int rows = a.heads > 1 ? p.Nq : BM, G = p.Hq / p.Hkv;
  if (a.heads > 1 && (!group_map(&a.group_q, p.q, p.B, p.Hkv, G, p.Nq, p.d, rows, a.heads) ||
                      !group_map(&a.group_dout, p.dout, p.B, p.Hkv, G, p.Nq, p.d, rows, a.heads)))
    return cudaErrorInvalidValue;
  if (!heads_map(&a.q, p.q, p.B, p.Hq, p.Nq, p.d, rows, a.heads) ||
      !heads_map(&a.dout, p.dout, p.B, p.Hq, p.Nq, p.d, rows, a.heads) ||
      !heads_map(&a.o, p.o, p.B, p.Hq, p.Nq, p.d, rows, a.heads) ||
      !heads_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, BN, 1) || !heads_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, BN, 1) ||
      !heads_map(&a.dq, p.dq, p.B, p.Hq, p.Nq, p.d, 32, 1) || !heads_map(&a.dk, p.dk, p.B, p.Hkv, p.Nk, p.d, 32, 1) ||
      !heads_map(&a.dv, p.dv, p.B, p.Hkv, p.Nk, p.d, 32, 1))
    return cudaErrorInvalidValue;
  const bool wide = p.d == 128;
  // does a range end inside an output tile's steps?
  const long long steps = (long long)p.B * p.Hkv * a.key_tiles * a.tiles;
  const auto apart = [](long long steps, int ranges, int line) {
    return line == 1 || (steps % ranges == 0 && steps / ranges % line == 0);
  };
  const bool join_q = p.lens ? a.key_tiles > 1 : !apart(steps, a.ctas, a.key_tiles);
  const bool join_k = p.lens ? a.tiles > 1 : !apart(steps / a.side, a.ranges, a.tiles);
  const long long query_tiles = a.items, key_tiles = (long long)p.B * p.Hkv * a.key_tiles;
  a.by_query_tile = query_tiles < a.slots;
  a.by_key_tile = key_tiles < a.slots;
  a.joins = max(join_q ? (int)min(query_tiles, (long long)a.slots) : 0,
                join_k ? (int)min(key_tiles, (long long)a.slots) : 0);
  a.parts_q = !join_q ? 0 : 4 * query_tiles <= a.slots ? p.d / 16 : 2;
  a.parts_k = !join_k ? 0 : 4 * key_tiles <= a.slots ? p.d / 16 : 2;
  const dim3 grid(a.ctas), gj(a.joins + (p.lens ? p.B * p.Hkv : 0), 3, max(max(a.parts_q, a.parts_k), 1));
  cudaError_t e = start(wide ? cross_dq_kernel<128> : cross_dq_kernel<64>, grid, Roles<16>::NTHREADS,
                        wide ? SmemQ<128>::BYTES : SmemQ<64>::BYTES, true, a, st);
  const bool staged = !wide || a.tiles <= STAGED_STEPS;
  if (e == cudaSuccess)
    e = start(!wide ? cross_dkv_kernel<64, true> : staged ? cross_dkv_kernel<128, true> : cross_dkv_kernel<128, false>,
              dim3(a.ranges * a.side), Roles<8>::NTHREADS,
              !wide ? SmemK<64, true>::BYTES : staged ? SmemK<128, true>::BYTES : SmemK<128, false>::BYTES, true, a, st);
  if (e == cudaSuccess && gj.x > 0)
    e = launch(gj.z > 2 ? wide ? cross_join_kernel<128, true> : cross_join_kernel<64, true>
                        : wide ? cross_join_kernel<128, false> : cross_join_kernel<64, false>,
               gj, 256, 0, true, st, a);
  return e;
}

}  // namespace fa4
