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
// cross_dq_kernel: persistent, a query tile at a time.  Warps 0-7: a thread per
//   row and half of the keys: P from S while dP runs, dS as bf16 into tensor memory
//   (the A operand of dQ).  S of the next key tile runs as soon as S has been read.
//   D is summed by the same threads from dO and o, and kept in the workspace.
// cross_dkv_kernel: persistent over the steps (key tile, query tile), cut into
//   equal ranges.  Rows are keys: P^T and dS^T go over S^T and dP^T as A operands of
//   dV and dK, which are summed in tensor memory (512 columns in all).  The
//   products' order dV, next S^T, dK, next dP^T leaves each half of the element-wise
//   work two products to hide behind.  A range that starts or ends inside a key
//   tile leaves FP32 partials in the workspace.
// cross_join_kernel: sums those in the ranges' order; zeros for keys behind kv_lens.
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"
#include "internal.h"

namespace fa4 {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NTHREADS = 384;
constexpr int W_PROD = 8, W_MMA = 9, W_STAT = 10;
constexpr int REG_SOFT = 208, REG_MISC = 88;   // 2 x 208 + 88 = 504 of 512
constexpr uint32_t TMEM_COLS = 512;
constexpr float L2E = 1.4426950408889634f;
constexpr int CH = 128 * 128;                  // [128 rows][64 channels] of bf16

struct Params {
  CrossParams p;
  HeadsMap q, dout, k, v;
  int tiles, per_head, heads, box;             // query tiles of a kv head, as in the forward
  int key_tiles;                               // of Nk
  int items;                                   // query tiles in all
  int ctas;                                    // of the dK, dV kernel
  int dq32, dk32, dv32;                        // rows begin on 32 bytes
  float* del;                                  // D [B][Hq][Nq]
  float* part;                                 // [2 ctas][dV, dK][128][d]
};

// Row r of a query tile: query head within the group (G: none) and position.
FA4_DEV void tile_row(const Params& a, int tile, int r, int G, int& g, int& n) {
  if (a.heads > 1) {
    g = r < a.heads * a.p.Nq ? min(G, tile * a.heads + r / a.p.Nq) : G;
    n = r % a.p.Nq;
  } else {
    g = tile / a.per_head;
    n = tile % a.per_head * BM + r;
    if (n >= a.p.Nq) g = G;
  }
}

FA4_DEV uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

// 32 FP32 columns of a row, times f, to bf16 in global memory.
FA4_DEV void store32(__nv_bfloat16* dst, const uint32_t (&v)[32], float f, bool wide) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) pk[i] = pack2(__uint_as_float(v[2 * i]) * f, __uint_as_float(v[2 * i + 1]) * f);
  if (wide) {
    st_global_v8(dst, pk);
    st_global_v8(dst + 16, pk + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
  }
}

// A K-major product of 128 x 128 over D channels, both operands in shared memory.
template <int D>
FA4_DEV void product_kk(uint32_t acc, uint32_t sa, uint32_t sb, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = (k / 4) * CH + (k % 4) * 32;
    mma_f16(acc, make_sdesc(sa + off, 16, 1024, SW_128B), make_sdesc(sb + off, 16, 1024, SW_128B), idesc, k > 0);
  }
}
// ... over 128 rows of B (MN-major), A packed in tensor memory: the first 64
// of them in columns [a0, a0 + 32), the others in [a1, a1 + 32).
FA4_DEV void product_tmem(uint32_t acc, uint32_t a0, uint32_t a1, uint32_t sb, uint32_t idesc, bool add) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    mma_f16_tmem_a(acc, (k < 4 ? a0 : a1) + 8 * (k % 4), make_sdesc(sb + k * 16 * 128, CH, 1024, SW_128B), idesc,
                   add || k > 0);
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
template <int D>
struct SmemQ {
  static constexpr int TILE = (D / 64) * CH;
  static constexpr int QS = D == 128 ? 3 : 5, KS = D == 128 ? 4 : 8;
  static constexpr int OFF_Q = 0, OFF_KV = QS * TILE;
  static constexpr int OFF_DEL = OFF_KV + KS * TILE;        // float [2][128]
  static constexpr int OFF_BAR = OFF_DEL + 1024;
  static constexpr int NBAR = 2 * QS + 2 * KS + 6;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

struct ItemQ {
  int b, hk, tile, len, nt;
};
struct WalkQ {
  int i, b = -1, len = 0;
  FA4_DEV WalkQ() : i(blockIdx.x) {}
  FA4_DEV bool at(const Params& a, ItemQ& it, bool report) {
    if (i >= a.items) return false;
    const int bh = i / a.tiles;
    it.b = bh / a.p.Hkv;
    it.hk = bh % a.p.Hkv;
    it.tile = i % a.tiles;
    if (it.b != b) {
      b = it.b;
      len = key_count(a.p, b, report);
    }
    it.len = len;
    it.nt = (len + BN - 1) / BN;
    return true;
  }
  FA4_DEV void next() { i += gridDim.x; }
  FA4_DEV bool with_keys(const Params& a, ItemQ& it, bool report) {
    while (at(a, it, report)) {
      if (it.nt > 0) return true;
      next();
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cross_dq_kernel(const __grid_constant__ Params a) {
  using L = SmemQ<D>;
  constexpr int QS = L::QS, KS = L::KS;
  constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DQ = 256, COL_DS = 384;
  const CrossParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* del_half = reinterpret_cast<float*>(smem + L::OFF_DEL);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_empty = q_full + QS;
  uint64_t* kv_full = q_empty + QS;
  uint64_t* kv_empty = kv_full + KS;
  uint64_t* s_full = kv_empty + KS;      // S is there
  uint64_t* s_free = s_full + 1;         // S has been read
  uint64_t* dp_full = s_free + 1;        // dP is there
  uint64_t* ds_full = dp_full + 1;       // dS is there, dP has been read
  uint64_t* dq_done = ds_full + 1;       // the item's dQ is there
  uint64_t* mma_done = dq_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < QS; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    mbar_init(s_full, 1);
    mbar_init(s_free, 8);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(dq_done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const int G = p.Hq / p.Hkv;

  if (warp >= W_PROD) {
    setmaxnreg_dec<REG_MISC>();
    if (warp == W_PROD) {
      if (lane == 0) {
        tma_prefetch_desc(&a.q.map);
        tma_prefetch_desc(&a.dout.map);
        tma_prefetch_desc(&a.k.map);
        tma_prefetch_desc(&a.v.map);
        int qn = 0, kn = 0;
        auto load_q = [&](const HeadsMap& m, const ItemQ& it) -> bool {
          const int st = qn % QS;
          if (qn >= QS && !mbar_wait(&q_empty[st], (qn / QS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&q_full[st], a.box * 2 * D);
          const int h = it.hk * G + it.tile / a.per_head * a.heads, n = it.tile % a.per_head * BM;
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + L::OFF_Q + st * L::TILE + c * CH, m, &q_full[st], 64 * c, n, h, it.b);
          ++qn;
          return true;
        };
        auto load_kv = [&](const HeadsMap& m, const ItemQ& it, int j) -> bool {
          const int st = kn % KS;
          if (kn >= KS && !mbar_wait(&kv_empty[st], (kn / KS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&kv_full[st], L::TILE);
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + L::OFF_KV + st * L::TILE + c * CH, m, &kv_full[st], 64 * c, j * BN, it.hk, it.b);
          ++kn;
          return true;
        };
        WalkQ w;
        ItemQ it;
        bool ok = true;
        for (; ok && w.with_keys(a, it, true); w.next()) {
          ok = load_q(a.q, it) && load_kv(a.k, it, 0) && load_q(a.dout, it) && load_kv(a.v, it, 0);
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
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, true, false, false);
      const uint32_t idesc_q = idesc_f16(BM, D, true, false, true);
      struct Step {
        ItemQ it;
        int j, kv, q;                    // key tile; ring positions of its K, and of the item's Q
      };
      WalkQ w;
      int qn = 0, kn = 0, done = 0;      // done: steps whose dQ is issued
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
        qn = s.q + 2;
        w.next();
        return first(n);
      };
      auto tile_kv = [&](int seq) { return smem + L::OFF_KV + seq % KS * L::TILE; };
      auto issue_s = [&](const Step& s) -> bool {
        if (s.j == 0 && !mbar_wait(&q_full[s.q % QS], (s.q / QS) & 1, abort_flag, p.err)) return false;
        if (!mbar_wait(&kv_full[s.kv % KS], (s.kv / KS) & 1, abort_flag, p.err)) return false;
        // rows of K behind the sequence's keys may be anything: dS is 0 there, and 0 x NaN is not
        const int keep = s.it.len - s.j * BN;
        uint8_t* k = tile_kv(s.kv);
        if (keep < BN && s.it.len < p.Nk) {
          for (int c = 0; c < D / 64; ++c)
            for (int i = keep * 8 + lane; i < BN * 8; i += 32)
              reinterpret_cast<uint4*>(k + c * CH)[i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (leader) {
          product_kk<D>(tbase + COL_S, smem_u32(smem + L::OFF_Q + s.q % QS * L::TILE), smem_u32(k), idesc_s);
          mma_commit(s_full);
          if (s.j == s.it.nt - 1) mma_commit(&q_empty[s.q % QS]);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](const Step& s) -> bool {
        const int q = s.q + 1, v = s.kv + 1;
        if (s.j == 0 && !mbar_wait(&q_full[q % QS], (q / QS) & 1, abort_flag, p.err)) return false;
        if (!mbar_wait(&kv_full[v % KS], (v / KS) & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        if (leader) {
          product_kk<D>(tbase + COL_DP, smem_u32(smem + L::OFF_Q + q % QS * L::TILE), smem_u32(tile_kv(v)), idesc_s);
          mma_commit(dp_full);
          mma_commit(&kv_empty[v % KS]);
          if (s.j == s.it.nt - 1) mma_commit(&q_empty[q % QS]);
        }
        __syncwarp();
        return true;
      };
      auto issue_dq = [&](const Step& s) -> bool {
        if (!mbar_wait(ds_full, done & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        if (leader) {
          product_tmem(tbase + COL_DQ, tbase + COL_DS, tbase + COL_DS + 32, smem_u32(tile_kv(s.kv)), idesc_q, s.j > 0);
          mma_commit(&kv_empty[s.kv % KS]);
          if (s.j == s.it.nt - 1) mma_commit(dq_done);
        }
        __syncwarp();
        return true;
      };
      Step cur, nxt;
      bool more = first(cur);
      bool ok = !more || (issue_s(cur) && issue_dp(cur));
      while (ok && more) {
        const bool then = after(cur, nxt);
        if (then) ok = mbar_wait(s_free, done & 1, abort_flag, p.err) && issue_s(nxt);
        ok = ok && issue_dq(cur);
        ++done;
        if (then) ok = ok && issue_dp(nxt);
        more = then;
        cur = nxt;
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    const int half = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const float c = p.c;
    int n = 0, items = 0;
    bool ok = true;
    WalkQ w;
    ItemQ it;
    // (a warp whose wait ran out still meets the others at the barriers of later items)
    for (; w.at(a, it, false); w.next()) {
      int g, row;
      tile_row(a, it.tile, r, G, g, row);
      const bool valid = g < G;
      const int h = it.hk * G + (valid ? g : 0);
      const long long flat = ((long long)it.b * p.Hq + h) * p.Nq + row;
      // this half's share of D, both halves' sum
      float del = 0.f, lse = INFINITY;
      if (valid) {
        const __nv_bfloat16 *x = at(p.dout, it.b, h, row) + half * (D / 2), *y = at(p.o, it.b, h, row) + half * (D / 2);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 u = reinterpret_cast<const uint4*>(x)[i], v = reinterpret_cast<const uint4*>(y)[i];
          const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            del = fmaf(__uint_as_float(uw[e] << 16), __uint_as_float(vw[e] << 16), del);
            del = fmaf(__uint_as_float(uw[e] & 0xffff0000u), __uint_as_float(vw[e] & 0xffff0000u), del);
          }
        }
        const float z = p.lse[flat];
        if (z > -INFINITY) lse = z * L2E;          // a row without keys: P = 2^-inf = 0
      }
      del_half[half * 128 + r] = del;
      named_bar(1, 256);
      del += del_half[(half ^ 1) * 128 + r];
      named_bar(1, 256);
      if (!ok) continue;
      if (valid && half == 0) a.del[flat] = del;
      for (int j = 0; j < it.nt; ++j, ++n) {
        if (!mbar_wait(s_full, n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        float e[2][32];
        {
          uint32_t v[2][32];
          tmem_ld32(lane_base + COL_S + 64 * half, v[0]);
          tmem_ld32(lane_base + COL_S + 64 * half + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i) e[q][i] = ex2_approx(fmaf(__uint_as_float(v[q][i]), c, -lse));
        }
        if (!mbar_wait(dp_full, n & 1, abort_flag, p.err)) { ok = false; break; }
        tc_fence_after();
        const int keep = it.len - j * BN - 64 * half;
        uint32_t pk[32];
        {
          uint32_t v[2][32];
          tmem_ld32(lane_base + COL_DP + 64 * half, v[0]);
          tmem_ld32(lane_base + COL_DP + 64 * half + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i) e[q][i] *= __uint_as_float(v[q][i]) - del;
        }
        if (keep < 64) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * q + i >= keep) e[q][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = pack2(e[i / 16][2 * (i % 16)], e[i / 16][2 * (i % 16) + 1]);
        tmem_st32(lane_base + COL_DS + 32 * half, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) continue;
      __nv_bfloat16* dst = valid ? at(p.dq, it.b, h, row) + half * (D / 2) : nullptr;
      if (it.nt == 0) {
        if (valid)
          for (int i = 0; i < D / 16; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!mbar_wait(dq_done, items & 1, abort_flag, p.err)) { ok = false; continue; }
      ++items;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint32_t v[32];
        tmem_ld32(lane_base + COL_DQ + half * (D / 2) + 32 * q, v);
        tmem_ld_wait();
        reg_fence32(v);
        if (valid) store32(dst + 32 * q, v, p.scale, a.dq32);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
template <int D>
struct SmemK {
  static constexpr int TILE = (D / 64) * CH;
  static constexpr int RS = D == 128 ? 5 : 10;              // ring: Q, dO, Q, dO, ...
  static constexpr int OFF_K = 0, OFF_V = TILE, OFF_R = 2 * TILE;
  static constexpr int OFF_ST = OFF_R + RS * TILE;          // [2] x (lse log2 e [128], D [128])
  static constexpr int OFF_BAR = OFF_ST + 2 * 1024;
  static constexpr int NBAR = 4 + 2 * RS + 4 + 6;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int BYTES = OFF_MISC + 64;
  static_assert(BYTES <= 227 * 1024, "shared memory budget");
};

// Lines: the key tiles that hold keys, by sequence, kv head and position; a
// line's steps are the kv head's query tiles.  The CTAs get equal ranges of all
// steps.
struct Lines {
  int b, nt, i;                // sequence, its key tiles, line within it
  int t;                       // step within the line
  long long left;              // steps of the range from here on
  int len;
  FA4_DEV int hk() const { return i / nt; }
  FA4_DEV int tile() const { return i % nt; }
  // to the next line (the range has more)
  FA4_DEV void line(const Params& a) {
    t = 0;
    if (++i < a.p.Hkv * nt) return;
    i = 0;
    do {
      ++b;
      len = key_count(a.p, b, false);
      nt = (len + BN - 1) / BN;
    } while (nt == 0);
  }
};

FA4_DEV int tiles_of(const Params& a, int b) { return (key_count(a.p, b, false) + BN - 1) / BN; }

// Key tiles that hold keys, of the sequences before `b` and in all (one warp).
FA4_DEV void count_tiles(const Params& a, int b, int lane, long long& before, long long& all) {
  if (!a.p.lens) {
    before = (long long)b * a.key_tiles;
    all = (long long)a.p.B * a.key_tiles;
    return;
  }
  before = all = 0;
  for (int x = lane; x < a.p.B; x += 32) {
    const int n = tiles_of(a, x);
    all += n;
    if (x < b) before += n;
  }
  for (int o = 16; o > 0; o /= 2) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
}

// The first step of CTA `cta` of `total` steps.
FA4_DEV long long range_start(const Params& a, long long total, int cta) { return total * cta / a.ctas; }

// This CTA's range (one warp).
FA4_DEV Lines find_range(const Params& a, int lane) {
  Lines x;
  long long before, all;
  count_tiles(a, 0, lane, before, all);
  const long long total = all * a.p.Hkv * a.tiles;
  const long long s0 = range_start(a, total, blockIdx.x), s1 = range_start(a, total, blockIdx.x + 1);
  x.left = s1 - s0;
  x.b = x.nt = x.i = x.t = x.len = 0;
  if (x.left == 0) return x;
  long long line = s0 / a.tiles;
  x.t = (int)(s0 % a.tiles);
  if (!a.p.lens) {
    x.b = (int)(line / ((long long)a.p.Hkv * a.key_tiles));
    line -= (long long)x.b * a.p.Hkv * a.key_tiles;
  } else {
    // 32 sequences at a time
    for (int x0 = 0;; x0 += 32) {
      const long long n = x0 + lane < a.p.B ? (long long)tiles_of(a, x0 + lane) * a.p.Hkv : 0;
      long long upto = n;
      for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto > line);
      if (past) {
        const int at = __ffs(past) - 1;
        x.b = x0 + at;
        line -= __shfl_sync(0xffffffffu, upto - n, at);
        break;
      }
      line -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  x.i = (int)line;
  x.len = key_count(a.p, x.b, false);
  x.nt = (x.len + BN - 1) / BN;
  return x;
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) cross_dkv_kernel(const __grid_constant__ Params a) {
  using L = SmemK<D>;
  constexpr int RS = L::RS;
  constexpr uint32_t COL_S = 0, COL_DP = 128, COL_DV = 256, COL_DK = 256 + D;
  const CrossParams& p = a.p;
  // (no room to align it by hand: nothing else is in shared memory, so it begins on its alignment)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {
    atomicOr(p.err, FA4_DEVERR_TIMEOUT);
    return;
  }
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* k_empty = k_full + 1;
  uint64_t* v_full = k_empty + 1;
  uint64_t* v_empty = v_full + 1;
  uint64_t* r_full = v_empty + 1;
  uint64_t* r_empty = r_full + RS;
  uint64_t* st_full = r_empty + RS;      // [2]
  uint64_t* st_empty = st_full + 2;
  uint64_t* s_full = st_empty + 2;
  uint64_t* p_full = s_full + 1;         // P^T is there
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;       // dS^T is there
  uint64_t* acc_done = ds_full + 1;      // the line's dV and dK are there
  uint64_t* mma_done = acc_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  Lines* range = reinterpret_cast<Lines*>(smem + L::OFF_MISC + 8);
  static_assert(sizeof(Lines) <= 56, "range's place");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1); mbar_init(k_empty, 1); mbar_init(v_full, 1); mbar_init(v_empty, 1);
    for (int s = 0; s < RS; ++s) { mbar_init(&r_full[s], 1); mbar_init(&r_empty[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&st_full[s], 1); mbar_init(&st_empty[s], 8); }
    mbar_init(s_full, 1);
    mbar_init(p_full, 8);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(acc_done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  // rows of a ring slot that no box brings are zeros: P and dS are 0 there
  if (a.box < BM)
    for (int i = threadIdx.x; i < RS * L::TILE / 16; i += NTHREADS)
      reinterpret_cast<uint4*>(smem + L::OFF_R)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == W_PROD) {
    const Lines x = find_range(a, lane);
    if (lane == 0) *range = x;
  }
  if (warp == W_MMA) tmem_alloc(tmem_holder, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  const int G = p.Hq / p.Hkv;
  Lines at_ = *range;

  if (warp >= W_PROD) {
    setmaxnreg_dec<REG_MISC>();
    if (warp == W_PROD) {
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
            tma_heads(smem + off + c * CH, m, full, 64 * c, at_.tile() * BN, at_.hk(), at_.b);
          ++count;
          return true;
        };
        auto load_r = [&](const HeadsMap& m) -> bool {
          const int st = rn % RS;
          if (rn >= RS && !mbar_wait(&r_empty[st], (rn / RS - 1) & 1, abort_flag, p.err)) return false;
          mbar_arrive_expect_tx(&r_full[st], a.box * 2 * D);
          const int h = at_.hk() * G + at_.t / a.per_head * a.heads, n = at_.t % a.per_head * BM;
          for (int c = 0; c < D / 64; ++c)
            tma_heads(smem + L::OFF_R + st * L::TILE + c * CH, m, &r_full[st], 64 * c, n, h, at_.b);
          ++rn;
          return true;
        };
        bool ok = true, fresh = true;
        while (ok && at_.left > 0) {
          ok = load_r(a.q) && (!fresh || load_kv(a.k, k_full, k_empty, L::OFF_K, kn)) && load_r(a.dout) &&
               (!fresh || load_kv(a.v, v_full, v_empty, L::OFF_V, vn));
          if (fresh) ++ln;
          fresh = false;
          --at_.left;
          if (++at_.t == a.tiles && at_.left > 0) {
            at_.line(a);
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
    } else if (warp == W_STAT) {
      // lse log2 e and D of each step's queries (infinite lse where there is none: P = 0)
      float z[4], d4[4];
      auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int g, n;
          tile_row(a, at_.t, 4 * lane + i, G, g, n);
          z[i] = INFINITY;
          d4[i] = 0.f;
          if (g < G) {
            const long long flat = ((long long)at_.b * p.Hq + at_.hk() * G + g) * p.Nq + n;
            const float v = p.lse[flat];
            if (v > -INFINITY) z[i] = v * L2E;
            d4[i] = a.del[flat];
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
        if (++at_.t == a.tiles) at_.line(a);
        fetch();
      }
    } else if (warp == W_MMA) {
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16(BM, BN, true, false, false);
      const uint32_t idesc_a = idesc_f16(BM, D, true, false, true);
      const uint32_t sk = smem_u32(smem + L::OFF_K), sv = smem_u32(smem + L::OFF_V);
      auto ring = [&](int seq) { return smem_u32(smem + L::OFF_R + seq % RS * L::TILE); };
      auto arrived = [&](int seq) { return mbar_wait(&r_full[seq % RS], (seq / RS) & 1, abort_flag, p.err); };
      const long long steps = at_.left;
      // step n: the first or last of its line?  (t counts on from the range's start)
      auto first_of = [&](long long n) { return n == 0 || (at_.t + n) % a.tiles == 0; };
      auto last_of = [&](long long n) { return n == steps - 1 || (at_.t + n + 1) % a.tiles == 0; };
      int ls = 0, lp = 0;                  // lines begun by S^T, by dP^T
      auto issue_s = [&](int n) -> bool {
        if (first_of(n)) {
          if (!mbar_wait(k_full, ls & 1, abort_flag, p.err)) return false;
          ++ls;
        }
        if (!arrived(2 * n)) return false;
        tc_fence_after();
        if (leader) {
          product_kk<D>(tbase + COL_S, sk, ring(2 * n), idesc_s);
          mma_commit(s_full);
          if (last_of(n)) mma_commit(k_empty);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int n) -> bool {
        if (first_of(n)) {
          if (!mbar_wait(v_full, lp & 1, abort_flag, p.err)) return false;
          ++lp;
        }
        if (!arrived(2 * n + 1)) return false;
        tc_fence_after();
        if (leader) {
          product_kk<D>(tbase + COL_DP, sv, ring(2 * n + 1), idesc_s);
          mma_commit(dp_full);
          if (last_of(n)) mma_commit(v_empty);
        }
        __syncwarp();
        return true;
      };
      bool ok = steps == 0 || (issue_s(0) && issue_dp(0));
      for (int n = 0; ok && n < steps; ++n) {
        const bool add = !first_of(n);
        ok = mbar_wait(p_full, n & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          product_tmem(tbase + COL_DV, tbase + COL_S, tbase + COL_S + 64, ring(2 * n + 1), idesc_a, add);
          mma_commit(&r_empty[(2 * n + 1) % RS]);
        }
        __syncwarp();
        if (n + 1 < steps && !issue_s(n + 1)) { ok = false; break; }
        ok = mbar_wait(ds_full, n & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          product_tmem(tbase + COL_DK, tbase + COL_DP, tbase + COL_DP + 64, ring(2 * n), idesc_a, add);
          mma_commit(&r_empty[(2 * n) % RS]);
          if (last_of(n)) mma_commit(acc_done);
        }
        __syncwarp();
        if (n + 1 < steps && !issue_dp(n + 1)) { ok = false; break; }
      }
      if (leader) mma_commit(mma_done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(mma_done, 0, &no_abort, p.err);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    const int half = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quad * 32) << 16);
    const float c = p.c;
    int n = 0, lines = 0;
    bool ok = true;
    while (ok && at_.left > 0) {
      const int s0 = at_.t, s1 = (int)min((long long)a.tiles, s0 + at_.left);
      for (; at_.t < s1; ++at_.t, ++n) {
        const int st = n & 1;
        const float* stat = reinterpret_cast<const float*>(smem + L::OFF_ST + st * 1024) + 64 * half;
        if (!mbar_wait(&st_full[st], (n / 2) & 1, abort_flag, p.err) || !mbar_wait(s_full, n & 1, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float e[2][32];
        {
          uint32_t v[2][32];
          tmem_ld32(lane_base + COL_S + 64 * half, v[0]);
          tmem_ld32(lane_base + COL_S + 64 * half + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 z = *reinterpret_cast<const float4*>(stat + 32 * q + i);
              e[q][i] = ex2_approx(fmaf(__uint_as_float(v[q][i]), c, -z.x));
              e[q][i + 1] = ex2_approx(fmaf(__uint_as_float(v[q][i + 1]), c, -z.y));
              e[q][i + 2] = ex2_approx(fmaf(__uint_as_float(v[q][i + 2]), c, -z.z));
              e[q][i + 3] = ex2_approx(fmaf(__uint_as_float(v[q][i + 3]), c, -z.w));
            }
        }
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = pack2(e[i / 16][2 * (i % 16)], e[i / 16][2 * (i % 16) + 1]);
        tmem_st32(lane_base + COL_S + 64 * half, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
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
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 z = *reinterpret_cast<const float4*>(stat + 128 + 32 * q + i);
              e[q][i] *= __uint_as_float(v[q][i]) - z.x;
              e[q][i + 1] *= __uint_as_float(v[q][i + 1]) - z.y;
              e[q][i + 2] *= __uint_as_float(v[q][i + 2]) - z.z;
              e[q][i + 3] *= __uint_as_float(v[q][i + 3]) - z.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = pack2(e[i / 16][2 * (i % 16)], e[i / 16][2 * (i % 16) + 1]);
        tmem_st32(lane_base + COL_DP + 64 * half, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(&st_empty[st]);
        }
      }
      if (!ok) break;
      // the line's sums: warps 0-3 dV, warps 4-7 dK, a key each
      if (!mbar_wait(acc_done, lines & 1, abort_flag, p.err)) { ok = false; break; }
      tc_fence_after();
      const bool whole = s0 == 0 && s1 == a.tiles;
      const int key = at_.tile() * BN + r;
      const bool mine = key < p.Nk;
      const float f = key < at_.len ? (half ? p.scale : 1.f) : 0.f;
      __nv_bfloat16* dst = mine ? at(half ? p.dk : p.dv, at_.b, at_.hk(), key) : nullptr;
      // partials: slot 0 for the range's first line, 1 for its last
      float* part = a.part + ((((long long)blockIdx.x * 2 + (lines > 0)) * 2 + half) * BN + r) * D;
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
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(part + 32 * q + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else if (mine) {
          store32(dst + 32 * q, v, f, half ? a.dk32 : a.dv32);
        }
      }
      tc_fence_before();
      ++lines;
      at_.left -= s1 - s0;
      if (at_.left > 0) at_.line(a);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tbase, TMEM_COLS);
}

// A CTA per key tile of Nk, kv head and sequence (x), and dV or dK (y).
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ Params a) {
  const CrossParams& p = a.p;
  __shared__ long long counts[2];
  const int jt = blockIdx.x % a.key_tiles, bh = blockIdx.x / a.key_tiles, hk = bh % p.Hkv, b = bh / p.Hkv;
  const int which = blockIdx.y;
  const int len = key_count(p, b), nt = (len + BN - 1) / BN;
  const Strided& out = which ? p.dk : p.dv;
  const bool live = jt < nt;
  long long first = 0;
  int c0 = 0, c1 = 0;
  if (live) {
    if (threadIdx.x < 32) {
      long long before, all;
      count_tiles(a, b, threadIdx.x, before, all);
      if (threadIdx.x == 0) { counts[0] = before; counts[1] = all; }
    }
    __syncthreads();
    const long long line = counts[0] * p.Hkv + (long long)hk * nt + jt, total = counts[1] * p.Hkv * a.tiles;
    first = line * a.tiles;
    const long long end = first + a.tiles;
    // the CTAs whose ranges meet [first, end)
    auto owner = [&](long long s) {
      int c = (int)(s * a.ctas / total);
      while (c + 1 < a.ctas && range_start(a, total, c + 1) <= s) ++c;
      while (c > 0 && range_start(a, total, c) > s) --c;
      return c;
    };
    c0 = owner(first);
    c1 = owner(end - 1);
    if (c0 == c1) return;                       // written whole
    // of each range, slot 0 unless it began in a line before
    for (int x = threadIdx.x; x < BN * (D / 8); x += 256) {
      const int r = x / (D / 8), i = x % (D / 8) * 8, key = jt * BN + r;
      if (key >= p.Nk) break;
      float v[8] = {};
      for (int c = c0; c <= c1; ++c) {
        const long long s = range_start(a, total, c);
        if (range_start(a, total, c + 1) == s) continue;
        const float* from = a.part + ((((long long)c * 2 + (s < first)) * 2 + which) * BN + r) * D + i;
        const float4 u = *reinterpret_cast<const float4*>(from), w = *reinterpret_cast<const float4*>(from + 4);
        v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
        v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
      }
      const float f = which ? p.scale : 1.f;
      *reinterpret_cast<uint4*>(at(out, b, hk, key) + i) =
          make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f),
                     pack2(v[6] * f, v[7] * f));
    }
    return;
  }
  for (int x = threadIdx.x; x < BN * (D / 8); x += 256) {
    const int r = x / (D / 8), i = x % (D / 8) * 8, key = jt * BN + r;
    if (key >= p.Nk) break;
    *reinterpret_cast<uint4*>(at(out, b, hk, key) + i) = make_uint4(0, 0, 0, 0);
  }
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

// Query tiles as in the forward, and the grid of the second kernel.
void plan(Params& a, int B, int Hq, int Hkv, int Nq, int Nk, bool share) {
  const int G = Hq / Hkv;
  a.heads = share && Nq <= 64 ? (128 / Nq < G ? 128 / Nq : G) : 1;
  a.per_head = (Nq + BM - 1) / BM;
  a.tiles = a.heads > 1 ? (G + a.heads - 1) / a.heads : G * a.per_head;
  a.box = a.heads > 1 ? a.heads * Nq : BM;
  a.items = (int)((long long)B * Hkv * a.tiles);
  a.key_tiles = (Nk + BN - 1) / BN;
  const long long steps = (long long)B * Hkv * a.key_tiles * a.tiles;
  const int sms = sm_count();
  a.ctas = (int)(steps < sms ? steps : sms);
}

size_t del_bytes(int B, int Hq, int Nq) { return ((size_t)B * Hq * Nq * sizeof(float) + 127) / 128 * 128; }

bool wide(const Strided& t) { return (reinterpret_cast<uintptr_t>(t.p) & 31) == 0 && ((t.b | t.h | t.n) & 15) == 0; }

template <class K>
cudaError_t start(K kernel, dim3 grid, int smem, const Params& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, NTHREADS, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t cross_bwd_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (Nq == 0 || Nk == 0) return 0;
  // (heads that share no tile make more tiles, never fewer CTAs)
  Params a;
  plan(a, B, Hq, Hkv, Nq, Nk, false);
  return del_bytes(B, Hq, Nq) + (size_t)a.ctas * 4 * BN * d * sizeof(float);
}

cudaError_t launch_cross_bwd(const CrossParams& p, cudaStream_t st) {
  if (p.Nk == 0) return zero(p.dq, p.B, p.Hq, p.Nq, p.d, st);
  if (p.Nq == 0) {
    const cudaError_t e = zero(p.dk, p.B, p.Hkv, p.Nk, p.d, st);
    return e != cudaSuccess ? e : zero(p.dv, p.B, p.Hkv, p.Nk, p.d, st);
  }
  Params a;
  a.p = p;
  plan(a, p.B, p.Hq, p.Hkv, p.Nq, p.Nk, p.q.h != 0 && p.dout.h != 0);
  a.dq32 = wide(p.dq); a.dk32 = wide(p.dk); a.dv32 = wide(p.dv);
  a.del = reinterpret_cast<float*>(p.work);
  a.part = reinterpret_cast<float*>(p.work + del_bytes(p.B, p.Hq, p.Nq));
  const int rows = a.heads > 1 ? p.Nq : BM;
  if (!heads_map(&a.q, p.q, p.B, p.Hq, p.Nq, p.d, rows, a.heads) ||
      !heads_map(&a.dout, p.dout, p.B, p.Hq, p.Nq, p.d, rows, a.heads) ||
      !heads_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, BN, 1) || !heads_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, BN, 1))
    return cudaErrorInvalidValue;
  const int sms = sm_count();
  const dim3 gq(a.items < sms ? a.items : sms), gk(a.ctas), gj(p.B * p.Hkv * a.key_tiles, 2);
  cudaError_t e;
  if (p.d == 128) {
    e = start(cross_dq_kernel<128>, gq, SmemQ<128>::BYTES, a, st);
    if (e == cudaSuccess) e = start(cross_dkv_kernel<128>, gk, SmemK<128>::BYTES, a, st);
    if (e == cudaSuccess) cross_join_kernel<128><<<gj, 256, 0, st>>>(a);
  } else {
    e = start(cross_dq_kernel<64>, gq, SmemQ<64>::BYTES, a, st);
    if (e == cudaSuccess) e = start(cross_dkv_kernel<64>, gk, SmemK<64>::BYTES, a, st);
    if (e == cudaSuccess) cross_join_kernel<64><<<gj, 256, 0, st>>>(a);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fa4
