// cross_fwd.cu -- BF16 attention of many query rows to keys of another length
// (tcgen05), a persistent grid.
//
// A tile is 128 query rows of one kv head: 128 rows of a query head, or, where
// the heads have up to 64 rows, as many of its query heads as fit.  A work item is two
// neighbouring tiles A and B, which share K and V.  The CTAs take the items in turn
// (item i goes to CTA i mod grid), so that those at work at a time read the
// same K and V.  16 warps in four groups:
//   warps 0-3    softmax of tile A, warps 4-7 of tile B: a thread per row.  P =
//                2^(c s - c m - down) rounded to bf16 into tensor memory over S, in two
//                halves of the keys, so that P V sets out on the first while the second
//                is formed; the normalizer from P before the rounding.  The reference m
//                follows the running maximum only when that passes it by 2^8 (P keeps
//                bf16's relative precision), and only then O is rescaled.  2^down is
//                that 2^8 times the number of keys or more: no sum of P |v| passes the
//                largest |v|, and weights below 2^(down - 126) of the largest are lost.
//                (It costs no instruction; the exponent is rounded to 2^-20, of the
//                order of the native exponential's error.  Scaling the rounded P
//                instead: 177 -> 181 us.)
//   warp 8       producer: Q tiles through one ring, K and V tiles through another,
//                ahead of the item at work.
//   warp 9       issues the products: S = Q K^T, O += P V (P from tensor memory, V
//                MN-major).  The next S of a tile follows its P V, across items too.
//   warps 12-15  take O / l to the rows' places, tile A's and tile B's in turn, while
//                the softmax of the next item runs.
// Tensor memory: S_A, S_B, O_A, O_B (512 columns at d = 128).
//
// Measured: 24 heads of 128, 32,760 queries over 512 keys 177-183 us, 0.58-0.60 of the
// measured bf16 rate (0.69 with many keys).  What bounds that: an item of four key tiles
// has 5.3K cycles of products, while its first scores, its last sum and its O on its
// way out are waits, and a tile's softmax (500 cycles of exponentials, its maximum, P
// to tensor memory) is about as long as its share of the products.  4 x 16 heads of
// 4096 queries over 1..77 keys 33 us, 0.62 of the copy bandwidth: Q's way in and O's out
// of an item's one tile have little to hide behind.
#include <atomic>
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"
#include "internal.h"

namespace fa4 {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NTHREADS = 512;
constexpr int W_PROD = 8, W_MMA = 9, W_OUT = 12;
constexpr int REG_SOFT = 192, REG_MISC = 64;   // 2 x 192 + 2 x 64 = 512, the launch's
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_S0 = 0, COL_O0 = 256;
constexpr int TAU = 8;                         // log2 units

struct Params {
  CrossParams p;
  HeadsMap q, k, v;
  int tiles;        // per (sequence, kv head)
  int heads;        // query heads of a tile
  Divisor per_head; // tiles of a query head (1 where heads share a tile)
  Divisor pairs;    // items per (sequence, kv head)
  Divisor hkv, nq;
  int items;
  int box;          // rows that a Q box brings
  int o32;          // rows of O begin on 32 bytes
};

template <int D>
struct Smem {
  static constexpr int TILE = (D / 64) * CH;
  static constexpr int QS = D == 128 ? 3 : 5, KS = D == 128 ? 4 : 8;
  static constexpr int OFF_Q = 0, OFF_KV = OFF_Q + QS * TILE;
  static constexpr int OFF_SUM = OFF_KV + KS * TILE;         // float2 [2 tiles][128]: c m + down and l of the rows
  static constexpr int OFF_BAR = OFF_SUM + 2 * 1024;
  static constexpr int NBAR = 2 * QS + 2 * KS + 14 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

// Where an item lies.
struct Item {
  int b, hk, tile0, len, nt;
  bool two;
};

// The next item of this CTA from `i` on that has keys (skipping the others, which
// the softmax warps alone see to); `len` is kept from item to item.
struct Walk {
  int i, b = -1, len = 0;
  FA4_DEV Walk() : i(blockIdx.x) {}
  FA4_DEV bool at(const Params& a, Item& it, bool report) {
    if (i >= a.items) return false;
    int bh, pair;
    divide(i, a.pairs, bh, pair);
    divide(bh, a.hkv, it.b, it.hk);
    it.tile0 = 2 * pair;
    it.two = it.tile0 + 1 < a.tiles;
    if (it.b != b) {
      b = it.b;
      len = key_count(a.p, b, report);
    }
    it.len = len;
    it.nt = (len + BN - 1) / BN;
    return true;
  }
  FA4_DEV void next() { i += gridDim.x; }
  FA4_DEV bool with_keys(const Params& a, Item& it, bool report) {
    while (at(a, it, report)) {
      if (it.nt > 0) return true;
      next();
    }
    return false;
  }
};

FA4_DEV float rowmax128(const uint32_t (&s)[4][32]) {
  float a[32];
#pragma unroll
  for (int i = 0; i < 32; ++i)
    a[i] = fmax3(__uint_as_float(s[0][i]), __uint_as_float(s[1][i]),
                 fmaxf(__uint_as_float(s[2][i]), __uint_as_float(s[3][i])));
#pragma unroll
  for (int n = 32; n > 1; n /= 2)
#pragma unroll
    for (int i = 0; i < n / 2; ++i) a[i] = fmaxf(a[i], a[i + n / 2]);
  return a[0];
}
FA4_DEV float max32(const uint32_t (&s)[32]) {
  float a[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 16]));
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmax3(a[i], a[i + 4], fmaxf(a[i + 8], a[i + 12]));
  return fmax3(a[0], a[1], fmaxf(a[2], a[3]));
}

// Groups of 32 keys of key tile j that hold keys: the others are not scored, exponentiated or multiplied.
FA4_DEV int groups_of(int len, int j) { return (min(len - j * BN, BN) + 31) / 32; }

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cross_fwd_kernel(const __grid_constant__ Params a) {
  using L = Smem<D>;
  constexpr int QS = L::QS, KS = L::KS;
  const CrossParams& p = a.p;
  // (no room to align it by hand: nothing else is in shared memory, so it begins on its alignment)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {
    atomicOr(p.err, FA4_DEVERR_TIMEOUT);
    return;
  }
  float2* sums = reinterpret_cast<float2*>(smem + L::OFF_SUM);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_empty = q_full + QS;
  uint64_t* kv_full = q_empty + QS;
  uint64_t* kv_empty = kv_full + KS;
  uint64_t* s_full = kv_empty + KS;          // [X]: S_X is there
  uint64_t* p_full = s_full + 2;             // [X][half]: that half of P_X is there (the first: O_X rescaled)
  uint64_t* o_done = p_full + 4;             // [X]: the item's O_X is there
  uint64_t* o_free = o_done + 2;             // [X]: it has been read
  uint64_t* l_full = o_free + 2;             // [X]: the item's c m + down and l are there
  uint64_t* l_free = l_full + 2;             // [X]: they have been read
  uint64_t* mma_done = l_free + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < QS; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1); mbar_init(&p_full[2 * x], 4); mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&o_done[x], 1); mbar_init(&o_free[x], 4); mbar_init(&l_full[x], 4); mbar_init(&l_free[x], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  next_may_start();
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  if (warp >= W_PROD) {
    setmaxnreg_dec<REG_MISC>();
    if (warp == W_PROD) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        tma_prefetch_desc(&a.q.map);
        tma_prefetch_desc(&a.k.map);
        tma_prefetch_desc(&a.v.map);
        const int G = p.Hq / p.Hkv;
        int qn = 0, kn = 0;                  // tiles issued into each ring
        auto load_q = [&](const Item& it, int tile) -> bool {
          const int st = qn % QS;
          if (qn >= QS && !mbar_wait(&q_empty[st], (qn / QS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&q_full[st], a.box * 2 * D);
          int g, n;
          divide(tile, a.per_head, g, n);
          const int h = it.hk * G + g * a.heads;
          n *= BM;
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + L::OFF_Q + st * L::TILE + c * CH, a.q, &q_full[st], 64 * c, n, h, it.b);
          ++qn;
          return true;
        };
        auto load_kv = [&](const HeadsMap& m, const Item& it, int j) -> bool {
          const int st = kn % KS;
          if (kn >= KS && !mbar_wait(&kv_empty[st], (kn / KS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&kv_full[st], L::TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + L::OFF_KV + st * L::TILE + c * CH, m, &kv_full[st], 64 * c, j * BN, it.hk, it.b);
          ++kn;
          return true;
        };
        Walk w;
        Item it;
        bool ok = true;
        for (; ok && w.with_keys(a, it, true); w.next()) {
          ok = load_q(it, it.tile0) && load_kv(a.k, it, 0) && (!it.two || load_q(it, it.tile0 + 1)) &&
               load_kv(a.v, it, 0);
          for (int j = 1; ok && j < it.nt; ++j) ok = load_kv(a.k, it, j) && load_kv(a.v, it, j);
        }
        if (*abort_flag) {
          volatile int no_abort = 0;
          for (int i = max(0, qn - QS); i < qn; ++i) mbar_wait(&q_full[i % QS], (i / QS) & 1, &no_abort, p.err);
          for (int i = max(0, kn - KS); i < kn; ++i) mbar_wait(&kv_full[i % KS], (i / KS) & 1, &no_abort, p.err);
        }
      }
      __syncwarp();
    } else if (warp == W_MMA) {
      // ---------------------------------------------------------- products
      const bool leader = elect_one();
      const uint32_t idesc_o = idesc_f16(BM, D, true, false, true);
      // a key tile of an item, and where its operands are
      struct Step {
        Item it;
        int j, kv, q;                        // key tile; ring positions of its K, and of the item's Q tiles
      };
      Walk w;
      int qn = 0, kn = 0;
      auto first = [&](Step& s) -> bool {
        if (!w.with_keys(a, s.it, false)) return false;
        s.j = 0;
        s.kv = kn;
        s.q = qn;
        return true;
      };
      auto after = [&](const Step& s, Step& n) -> bool {
        kn = s.kv + 2;
        if (s.j + 1 < s.it.nt) {
          n = s;
          ++n.j;
          n.kv = kn;
          return true;
        }
        qn = s.q + (s.it.two ? 2 : 1);
        w.next();
        return first(n);
      };
      int pn[2] = {0, 0}, in[2] = {0, 0};    // of each tile: P V issued; items begun
      auto issue_s = [&](int x, const Step& s) -> bool {
        const int ks = s.kv % KS, q = s.q + x, qs = q % QS;
        if (s.j == 0 && !mbar_wait(&q_full[qs], (q / QS) & 1, abort_flag, p.err)) return false;
        if (x == 0 && !mbar_wait(&kv_full[ks], (s.kv / KS) & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        const uint32_t sq = smem_u32(smem + L::OFF_Q + qs * L::TILE), sk = smem_u32(smem + L::OFF_KV + ks * L::TILE);
        const uint32_t idesc_s = idesc_f16(BM, 32 * groups_of(s.it.len, s.j), true, false, false);
        if (leader) {
          product_rows<D>(tbase + COL_S0 + 128 * x, sq, sk, idesc_s);
          mma_commit(&s_full[x]);
          if (x == 1 || !s.it.two) mma_commit(&kv_empty[ks]);
          if (s.j == s.it.nt - 1) mma_commit(&q_empty[qs]);
        }
        __syncwarp();
        return true;
      };
      auto issue_pv = [&](int x, const Step& s) -> bool {
        const int seq = s.kv + 1, st = seq % KS;
        uint8_t* v = smem + L::OFF_KV + st * L::TILE;
        if (x == 0) {
          if (!mbar_wait(&kv_full[st], (seq / KS) & 1, abort_flag, p.err)) return false;
          // rows of V behind the sequence's keys may be anything: P is 0 there, and 0 x NaN is not
          const int keep = s.it.len - s.j * BN;
          if (keep < BN && s.it.len < p.Nk) clear_rows<D>(v, keep, lane);
        }
        if (s.j == 0) {                      // O_X of the item before has been read
          if (in[x] > 0 && !mbar_wait(&o_free[x], (in[x] - 1) & 1, abort_flag, p.err)) return false;
          ++in[x];
        }
        const uint32_t b = desc_cols(smem_u32(v)), acc = tbase + COL_O0 + D * x, pc = tbase + COL_S0 + 128 * x;
        const int steps = 2 * groups_of(s.it.len, s.j);            // of 16 keys
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait(&p_full[2 * x + half], pn[x] & 1, abort_flag, p.err)) return false;
          tc_fence_after();
          if (leader)
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
              if (k < steps) mma_ts(acc, pc + 8 * k, b + k * 128, idesc_o, s.j > 0 || k > 0);
          __syncwarp();
        }
        ++pn[x];
        if (leader) {
          if (x == 1 || !s.it.two) mma_commit(&kv_empty[st]);
          if (s.j == s.it.nt - 1) mma_commit(&o_done[x]);
        }
        __syncwarp();
        return true;
      };
      Step cur, nxt;
      bool more = first(cur);
      bool ok = !more || (issue_s(0, cur) && (!cur.it.two || issue_s(1, cur)));
      while (ok && more) {
        const bool then = after(cur, nxt);
        ok = issue_pv(0, cur) && (!then || issue_s(0, nxt)) && (!cur.it.two || issue_pv(1, cur)) &&
             (!then || !nxt.it.two || issue_s(1, nxt));
        more = then;
        cur = nxt;
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    } else if (warp >= W_OUT) {
      // ---------------------------------------------------------- O
      const int quad = warp & 3, r = quad * 32 + lane;
      const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
      const int G = p.Hq / p.Hkv;
      int in[2] = {0, 0};                    // items of each tile
      bool ok = true;
      Walk w;
      Item it;
      for (; ok && w.at(a, it, false); w.next()) {
        for (int x = 0; ok && x < (it.two ? 2 : 1); ++x) {
          const int tile = it.tile0 + x;
          int g, row;
          if (a.heads > 1) {
            divide(r, a.nq, g, row);
            g = r < a.heads * p.Nq ? tile * a.heads + g : G;
          } else {
            divide(tile, a.per_head, g, row);
            row = row * BM + r;
          }
          const bool valid = g < G && row < p.Nq;
          const int h = it.hk * G + g;
          float* lse = valid && p.lse ? p.lse + ((long long)it.b * p.Hq + h) * p.Nq + row : nullptr;
          __nv_bfloat16* dst = valid ? at(p.o, it.b, h, row) : nullptr;
          if (it.nt == 0) {
            if (lse) *lse = -INFINITY;
            if (valid)
              for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
            continue;
          }
          if (!mbar_wait(&l_full[x], in[x] & 1, abort_flag, p.err)) { ok = false; break; }
          const float2 ml = sums[128 * x + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_free[x]);
          if (lse) *lse = lse_of(ml.x, ml.y, p.keys_log2 + TAU);
          const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;      // (no score within FP32's range)
          if (!mbar_wait(&o_done[x], in[x] & 1, abort_flag, p.err)) { ok = false; break; }
          ++in[x];
          tc_fence_after();
          const uint32_t col = lane_base + COL_O0 + D * x;
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t v[32], pk[16];
            tmem_ld32(col + 32 * q, v);
            tmem_ld_wait();
            reg_fence32(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              __nv_bfloat162 t =
                  __floats2bfloat162_rn(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
              pk[i] = *reinterpret_cast<uint32_t*>(&t);
            }
            if (q == D / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&o_free[x]);
            }
            if (valid && a.o32) {
              st_global_v8(dst + 32 * q, pk);
              st_global_v8(dst + 32 * q + 16, pk + 8);
            } else if (valid) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4*>(dst + 32 * q)[i] =
                    make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            }
          }
        }
      }
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_s = COL_S0 + 128 * x, col_o = COL_O0 + D * x;
    const float c = p.c, down = (float)(p.keys_log2 + TAU);
    int n = 0, items = 0;                    // key tiles and items of this warp's tile so far
    bool ok = true;
    Walk w;
    Item it;
    for (; ok && w.with_keys(a, it, false); w.next()) {
      if (x == 1 && !it.two) continue;
      float m = -INFINITY, mc = 0.f, l = 0.f;
      for (int j = 0; j < it.nt; ++j, ++n) {
        if (!mbar_wait(&s_full[x], n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        const int keep = it.len - j * BN;
        float2 ls = make_float2(0.f, 0.f);
        // the reference: the first maximum (of tiles whose scores are all -inf there is none, and P is 0), then only
        // where a maximum passes it by far
        auto refer = [&](float top) {
          const bool lift = (top - m) * c > TAU;
          float f = 1.f;
          if (lift) {
            const float was = mc;
            const bool first = m == -INFINITY;
            m = top;
            mc = fmaf(m, c, down);
            if (!first) f = ex2_approx(was - mc);
          }
          if (j > 0 && __any_sync(0xffffffffu, lift)) {
            // (S of this tile came after P V of the one before: O is at rest)
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t ov[16];
              tmem_ld16(lane_base + col_o + 16 * q, ov);
              tmem_ld_wait();
              reg_fence16(ov);
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
              tmem_st16(lane_base + col_o + 16 * q, ov);
            }
            l *= f;
          }
        };
        // P of 32 keys, from their scores, over the place of keys that have been read
        auto weigh = [&](const uint32_t (&s)[32], int q) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y = ffma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                                   make_float2(c, c), make_float2(-mc, -mc));
            const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            ls = fadd2(ls, e);
            __nv_bfloat162 t = __floats2bfloat162_rn(e.x, e.y);
            pk[i] = *reinterpret_cast<uint32_t*>(&t);
          }
          tmem_st16(lane_base + col_s + 16 * q, pk);
        };
        auto ready = [&](int half) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
        };
        if (keep >= BN) {
          uint32_t s[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(lane_base + col_s + 32 * q, s[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) reg_fence32(s[q]);
          refer(rowmax128(s));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            weigh(s[q], q);
            if (q & 1) ready(q / 2);
          }
        } else {
          // a sequence's last tile, a group of 32 keys at a time, twice
          const int groups = groups_of(it.len, j);
          float top = -INFINITY;
          auto scores = [&](int q, uint32_t (&s)[32]) {
            tmem_ld32(lane_base + col_s + 32 * q, s);
            tmem_ld_wait();
            reg_fence32(s);
            if (keep < 32 * q + 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * q + i >= keep) s[i] = 0xff800000u;          // -inf
            }
          };
#pragma unroll 1
          for (int q = 0; q < groups; ++q) {
            uint32_t s[32];
            scores(q, s);
            top = fmaxf(top, max32(s));
          }
          refer(top);
#pragma unroll 1
          for (int q = 0; q < groups; ++q) {
            uint32_t s[32];
            scores(q, s);
            weigh(s, q);
            if (q == 1 && groups > 2) ready(0);
          }
          if (groups <= 2) ready(0);
          ready(1);
        }
        l += ls.x + ls.y;
      }
      if (!ok) break;
      if (items > 0 && !mbar_wait(&l_free[x], (items - 1) & 1, abort_flag, p.err)) { ok = false; break; }
      ++items;
      sums[128 * x + r] = make_float2(mc, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_full[x]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

}  // namespace

bool heads_map(HeadsMap* m, const Strided& t, int B, int H, int N, int d, int rows, int heads) {
  m->own_b = t.b != 0;
  m->own_h = t.h != 0;
  const uint64_t dims[3] = {(uint64_t)N, m->own_h ? (uint64_t)H : 1, m->own_b ? (uint64_t)B : 1};
  const int64_t strides[3] = {t.n, t.h, t.b};
  return make_heads_map(&m->map, t.p, d, 4, dims, strides, (uint32_t)rows, (uint32_t)heads);
}

bool group_map(HeadsMap* m, const Strided& t, int B, int Hkv, int G, int N, int d, int rows, int heads) {
  m->own_b = t.b != 0;
  m->own_h = 1;
  const uint64_t dims[4] = {(uint64_t)N, (uint64_t)G, (uint64_t)Hkv, m->own_b ? (uint64_t)B : 1};
  const int64_t strides[4] = {t.n, t.h, G * t.h, t.b};
  return make_heads_map(&m->map, t.p, d, 5, dims, strides, (uint32_t)rows, (uint32_t)heads);
}

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t allow_smem(const void* kernel, int bytes, bool clusters) {
  struct Known {
    std::atomic<const void*> kernel;
    std::atomic<uint64_t> devices;
  };
  static Known known[32];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  Known* at = nullptr;
  for (Known& k : known) {
    const void* none = nullptr;
    if (k.kernel.load(std::memory_order_acquire) == kernel ||
        k.kernel.compare_exchange_strong(none, kernel, std::memory_order_acq_rel) || none == kernel) {
      at = &k;
      break;
    }
  }
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (at && (at->devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && clusters) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && at) at->devices.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

cudaError_t launch_cross_fwd(const CrossParams& p, cudaStream_t st) {
  Params a;
  a.p = p;
  const int G = p.Hq / p.Hkv;
  a.heads = p.Nq <= 64 && p.q.h != 0 ? (128 / p.Nq < G ? 128 / p.Nq : G) : 1;
  a.per_head = Divisor((p.Nq + BM - 1) / BM);
  a.tiles = a.heads > 1 ? (G + a.heads - 1) / a.heads : G * a.per_head.d;
  a.pairs = Divisor((a.tiles + 1) / 2);
  a.hkv = Divisor(p.Hkv);
  a.nq = Divisor(p.Nq);
  const long long items = (long long)p.B * p.Hkv * a.pairs.d;
  a.items = (int)items;
  a.box = a.heads > 1 ? a.heads * p.Nq : BM;
  a.o32 = (reinterpret_cast<uintptr_t>(p.o.p) & 31) == 0 && ((p.o.b | p.o.h | p.o.n) & 15) == 0;
  if (!heads_map(&a.q, p.q, p.B, p.Hq, p.Nq, p.d, a.heads > 1 ? p.Nq : BM, a.heads)) return cudaErrorInvalidValue;
  if (p.Nk > 0) {
    if (!heads_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, BN, 1) || !heads_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, BN, 1))
      return cudaErrorInvalidValue;
  } else {
    a.k = a.v = a.q;       // never loaded from
  }
  const int sms = sm_count(), grid = a.items < sms ? a.items : sms;
  const int smem = p.d == 128 ? Smem<128>::BYTES : Smem<64>::BYTES;
  auto k = p.d == 128 ? cross_fwd_kernel<128> : cross_fwd_kernel<64>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem);
  return e != cudaSuccess ? e : launch(k, dim3(grid), NTHREADS, smem, true, st, a);
}

}  // namespace fa4
