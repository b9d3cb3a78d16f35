// cross_token.cu -- cross attention of few query rows (the new tokens of a decoding
// step, all query heads of a kv head together; a CTA has up to 32 of them).
//
// Bound by reading K and V once.  A CTA (4 warps) works on one (sequence, kv head)
// or on a part of its keys: a cluster of up to 16 CTAs shares them where there are
// fewer heads than multiprocessors.  Blocks of keys go round the cluster's warps;
// each warp has a ring of its own in shared memory, filled by TMA boxes, so no warp
// waits for another.  The rows are the m16n8k16 products' A operand, held in
// registers (mma.sync: 16 rows have no use for a 128-row tensor memory tile, and the
// bytes of K and V, not the products, bound this kernel); a warp keeps its running
// maximum, sum and O.  The warps' results are joined in shared memory, the
// cluster's through distributed shared memory, each CTA taking a share of the
// outputs.
//
// Measured: 64 sequences of 16 heads of 64, a query over 1..1500 keys 37 us, 0.88 of
// the measured copy bandwidth.  One sequence of 8 kv heads of 128, 12 rows each over
// 16,383 keys 19.4 us, 0.52 (states that stay in L2: 18.7): of 128 CTAs with 0.5 MB of K
// and V each, by clock reads, the first block has come after 1.5 us, the blocks take
// 12 (5.5 TB/s in all; 11.6 from L2), the warps' results in shared memory and to the
// cluster 2.3, the wait for the cluster's last CTA 1.5, the outputs 0.6.  Eight warps a
// CTA there: 31 us when four took 23.
#include <cstring>
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.cuh"
#include "internal.h"

namespace fa4 {
namespace {

constexpr int WARPS = 4;
// Stages of a warp's ring: with two of them, 32 rows of d = 128 leave room for 2 CTAs
// on a multiprocessor.
template <int D, int MT>
constexpr int STAGES_OF = D == 128 && MT == 2 ? 2 : 3;

struct Params {
  CrossParams p;
  HeadsMap k, v;
  int splits;                    // CTAs of a cluster
  Divisor groups, hkv, nq;       // groups of 16 MT query rows of a (sequence, kv head)
};

// 8 KB of K and V a block: 16 keys at d = 128, 32 at d = 64.
template <int D>
constexpr int KEYS = 2048 / D;

FA4_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
FA4_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
FA4_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Two floats into the shared memory of CTA `rank` of the cluster, at this CTA's place `x`.
FA4_DEV void give(const float2* x, int rank, float a, float b) {
  asm volatile("{\n .reg .b32 r;\n mapa.shared::cluster.u32 r, %0, %1;\n st.shared::cluster.v2.f32 [r], {%2, %3};\n}\n" ::"r"(
                   smem_u32(x)),
               "r"(rank), "f"(a), "f"(b)
               : "memory");
}

FA4_DEV void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
FA4_DEV void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
FA4_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
FA4_DEV uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

template <int D, int MT>
struct Smem {
  static constexpr int CHUNK = KEYS<D> * 128;              // [keys][64 channels], 128-byte swizzle
  static constexpr int TILE = (D / 64) * CHUNK;            // 4 KB
  static constexpr int STAGE = 2 * TILE, STAGES = STAGES_OF<D, MT>;
  static constexpr int RING = WARPS * STAGES * STAGE;      // 24 KB a warp (16 with two stages)
  // after the loop the rings' place holds the warps' O, m and l
  static constexpr int ROWS = 16 * MT;
  static constexpr int WARP_F = ROWS * (D + 2);            // floats of one warp: O [ROWS][D], m, l
  static constexpr int JOIN = WARPS * WARP_F * 4;
  static constexpr int OFF_BAR = RING > JOIN ? RING : JOIN;
  // what the cluster's CTAs give this one: (m, l) of all rows, and their O of its share of the outputs
  static constexpr int OFF_ML = OFF_BAR + WARPS * STAGES * 8 + 32;
  static constexpr int OFF_O = OFF_ML + 16 * ROWS * 8;
  static constexpr int share(int splits) { return (ROWS * (D / 2) + splits - 1) / splits; }   // pairs of outputs
  static constexpr int bytes(int splits) { return (splits > 1 ? OFF_O + splits * share(splits) * 8 : OFF_ML) + 1024; }
};

template <int D, int MT>
__global__ void __launch_bounds__(WARPS * 32) cross_token_kernel(const __grid_constant__ Params a) {
  using L = Smem<D, MT>;
  constexpr int NK = KEYS<D>, STAGES = L::STAGES;
  const CrossParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + WARPS * STAGES);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = a.splits > 1 ? (int)cluster_rank() : 0;
  int bh, group, b, hk;
  divide((int)blockIdx.x / a.splits, a.groups, bh, group);
  divide(bh, a.hkv, b, hk);
  const int G = p.Hq / p.Hkv, r0 = group * L::ROWS, R = min(G * p.Nq - r0, L::ROWS);
  uint64_t* full = bars + warp * STAGES;
  uint8_t* ring = smem + warp * STAGES * L::STAGE;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
    if (warp == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (a.splits > 1) cluster_arrive();          // (this CTA is there to be given to)
  next_may_start();
  wait_for_previous();
  const int len = key_count(p, b, threadIdx.x == 0 && rank == 0);
  const int blocks = (len + NK - 1) / NK;
  // this warp's blocks: me, me + step, ...
  const int me = rank * WARPS + warp, step = a.splits * WARPS;
  const int mine = me < blocks ? (blocks - me + step - 1) / step : 0;
  auto load = [&](int i) {
    const int st = i % STAGES, key = (me + i * step) * NK;
    mbar_arrive_expect_tx(&full[st], L::STAGE);
    for (int c = 0; c < D / 64; ++c) {
      tma_heads(ring + st * L::STAGE + c * L::CHUNK, a.k, &full[st], 64 * c, key, hk, b);
      tma_heads(ring + st * L::STAGE + L::TILE + c * L::CHUNK, a.v, &full[st], 64 * c, key, hk, b);
    }
  };
  if (lane == 0)
    for (int i = 0; i < min(mine, STAGES); ++i) load(i);

  // the rows as A fragments: rows lane / 4 and + 8 of each 16, channels 2 (lane % 4) and + 8 of each 16
  uint32_t qf[MT][D / 16][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = 16 * t + lane / 4 + 8 * half;
      int g, n;
      divide(r0 + r, a.nq, g, n);
      const __nv_bfloat16* q = r < R ? at(p.q, b, hk * G + g, n) + 2 * (lane % 4) : nullptr;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[t][k][half] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
        qf[t][k][2 + half] = q ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
      }
    }
  // (m stands above the maximum by the number of keys: no sum of P |v| passes the largest |v|)
  const float down = (float)p.keys_log2;
  float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
  }
  // ldmatrix rows of this lane: K: matrices (keys 0-7, channels 0-7), (keys 0-7, 8-15), (keys 8-15, 0-7), (8-15, 8-15)
  const int krow = (lane & 7) + ((lane & 16) >> 1), kcol = (lane >> 3) & 1;
  // V, transposed: (keys 0-7, channels 0-7), (keys 8-15, 0-7), (keys 0-7, 8-15), (keys 8-15, 8-15)
  const int vrow = lane & 15, vcol = lane >> 4;

  for (int i = 0; i < mine; ++i) {
    const int st = i % STAGES;
    if (!mbar_wait(&full[st], (i / STAGES) & 1, abort_flag, p.err)) break;
    uint8_t* kt = ring + st * L::STAGE;
    uint8_t* vt = kt + L::TILE;
    const int keep = len - (me + i * step) * NK;
    if (keep < NK && len < p.Nk) {
      // rows of V behind the sequence's keys may be anything: P is 0 there, and 0 x NaN is not
      for (int x = keep * 8 + lane; x < NK * 8; x += 32)
        for (int c = 0; c < D / 64; ++c) reinterpret_cast<uint4*>(vt + c * L::CHUNK)[x] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    const uint32_t ks = smem_u32(kt), vs = smem_u32(vt);
    // two sums over every other 16 channels: chains of products half as long
    float s[MT][NK / 8][4], s2[MT][NK / 8][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][n][e] = s2[t][n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int n = 0; n < NK / 16; ++n) {
        const int row = 16 * n + krow;
        uint32_t kf[4];
        ldsm4(ks + (k / 4) * L::CHUNK + row * 128 + ((2 * (k % 4) + kcol) ^ (row & 7)) * 16, kf);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const bool second = MT == 1 && k % 2;      // (32 rows have chains enough, and no registers)
          mma_bf16(second ? s2[t][2 * n] : s[t][2 * n], qf[t][k], kf[0], kf[1]);
          mma_bf16(second ? s2[t][2 * n + 1] : s[t][2 * n + 1], qf[t][k], kf[2], kf[3]);
        }
      }
    uint32_t pf[MT][NK / 16][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int n = 0; n < NK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][n][e] += s2[t][n][e];
      if (keep < NK) {
#pragma unroll
        for (int n = 0; n < NK / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * n + 2 * (lane % 4) + (e & 1) >= keep) s[t][n][e] = -INFINITY;
      }
      // both rows of the lane side by side
      float now[2], ref[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        now[half] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NK / 8; ++n)
          now[half] = fmaxf(now[half], fmaxf(s[t][n][2 * half], s[t][n][2 * half + 1]));
      }
#pragma unroll
      for (int x = 1; x < 4; x *= 2)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          now[half] = fmaxf(now[half], __shfl_xor_sync(0xffffffffu, now[half], x));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        now[half] = fmaxf(m[t][half], fmaf(now[half], p.c, down));
        ref[half] = now[half] > -INFINITY ? now[half] : 0.f;
      }
      if (__any_sync(0xffffffffu, now[0] != m[t][0] || now[1] != m[t][1])) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float f = ex2_approx(m[t][half] - ref[half]);
          l[t][half] *= f;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[t][n][2 * half] *= f;
            o[t][n][2 * half + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        m[t][half] = now[half];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NK / 8; ++n) {
          const float e0 = ex2_approx(fmaf(s[t][n][2 * half], p.c, -ref[half]));
          const float e1 = ex2_approx(fmaf(s[t][n][2 * half + 1], p.c, -ref[half]));
          sum += e0 + e1;
          pf[t][n / 2][(n & 1) * 2 + half] = pack2(e0, e1);
        }
        l[t][half] += sum;
      }
    }
#pragma unroll
    for (int k = 0; k < NK / 16; ++k)
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        const int row = 16 * k + vrow;
        uint32_t vf[4];
        ldsm4_t(vs + (n / 4) * L::CHUNK + row * 128 + ((2 * (n % 4) + vcol) ^ (row & 7)) * 16, vf);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          mma_bf16(o[t][2 * n], pf[t][k], vf[0], vf[1]);
          mma_bf16(o[t][2 * n + 1], pf[t][k], vf[2], vf[3]);
        }
      }
    __syncwarp();
    if (i + STAGES < mine && lane == 0) load(i + STAGES);
  }
  if (*abort_flag) {                           // (a wait ran out: let the loads in flight land)
    volatile int no_abort = 0;
    for (int s = 0; s < min(mine, STAGES); ++s)
      for (int ph = 0; ph < 2; ++ph) mbar_wait_ns(&full[s], ph, &no_abort, p.err, 100000000ull);
  }

  // join: every warp leaves O [ROWS][D], m and l where the rings were
  __syncthreads();
  float* mem = reinterpret_cast<float*>(smem);
  float* my = mem + warp * L::WARP_F;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = 16 * t + lane / 4 + 8 * half;
      l[t][half] += __shfl_xor_sync(0xffffffffu, l[t][half], 1);
      l[t][half] += __shfl_xor_sync(0xffffffffu, l[t][half], 2);
      if (lane % 4 == 0) {
        my[L::ROWS * D + r] = m[t][half];
        my[L::ROWS * D + L::ROWS + r] = l[t][half];
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(my + r * D + 8 * n + 2 * (lane % 4)) =
            make_float2(o[t][n][2 * half], o[t][n][2 * half + 1]);
    }
  __syncthreads();
  auto store = [&](int r, int i, float v0, float v1, float top, float sum) {
    int g, n;
    divide(r0 + r, a.nq, g, n);
    const int h = hk * G + g;
    const bool none = sum == 0.f;        // (a sum that is NaN is no row without a key)
    const float inv = none ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(at(p.o, b, h, n) + i) = pack2(v0 * inv, v1 * inv);
    if (i == 0 && p.lse)
      p.lse[((long long)b * p.Hq + h) * p.Nq + n] = none ? -INFINITY : lse_of(top, sum, p.keys_log2);
  };
  // of a cluster, each CTA takes an equal share of the outputs, and is given the others' parts of it: stores to
  // another CTA's memory are not waited for, loads are (16 CTAs: 24.6 -> 18 us where they read)
  float2* ml = reinterpret_cast<float2*>(smem + L::OFF_ML);        // [splits][ROWS]
  float2* part = reinterpret_cast<float2*>(smem + L::OFF_O);       // [splits][share]
  const int share = L::share(a.splits);
  if (a.splits > 1) cluster_wait();
  for (int x = threadIdx.x; x < R * (D / 2); x += WARPS * 32) {
    const int r = x / (D / 2), i = x % (D / 2) * 2;
    float top = -INFINITY, sum = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, mem[w * L::WARP_F + L::ROWS * D + r]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float* from = mem + w * L::WARP_F;
      const float f = top > -INFINITY ? ex2_approx(from[L::ROWS * D + r] - top) : 0.f;
      const float2 v = *reinterpret_cast<const float2*>(from + r * D + i);
      sum = fmaf(from[L::ROWS * D + L::ROWS + r], f, sum);
      v0 = fmaf(v.x, f, v0);
      v1 = fmaf(v.y, f, v1);
    }
    if (a.splits == 1) {
      store(r, i, v0, v1, top, sum);
    } else {
      const int to = x / share;
      give(part + rank * share + (x - to * share), to, v0, v1);
      if (x % (D / 2) < a.splits) give(ml + rank * L::ROWS + r, x % (D / 2), top, sum);
    }
  }
  if (a.splits == 1) return;
  cluster_arrive();
  cluster_wait();
  for (int y = threadIdx.x; y < share; y += WARPS * 32) {
    const int x = rank * share + y;
    if (x >= R * (D / 2)) break;
    const int r = x / (D / 2), i = x % (D / 2) * 2;
    float top = -INFINITY, sum = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll 4
    for (int c = 0; c < a.splits; ++c) top = fmaxf(top, ml[c * L::ROWS + r].x);
#pragma unroll 4
    for (int c = 0; c < a.splits; ++c) {
      const float2 e = ml[c * L::ROWS + r], v = part[c * share + y];
      const float f = top > -INFINITY ? ex2_approx(e.x - top) : 0.f;
      sum = fmaf(e.y, f, sum);
      v0 = fmaf(v.x, f, v0);
      v1 = fmaf(v.y, f, v1);
    }
    store(r, i, v0, v1, top, sum);
  }
}

}  // namespace

namespace {

// CTAs that share a (sequence, kv head, row group)'s keys: a cluster, while there are
// more multiprocessors than CTAs (2 fit on one) and at least two blocks for each warp.
int splits_of(long long heads, int Nk, int d) {
  const int sms = sm_count(), nk = 2048 / d;
  int n = 1;
  while (n < 16 && heads * n * 2 <= 2LL * sms && Nk >= n * 2 * WARPS * 2 * nk) n *= 2;
  return n;
}

}  // namespace

// Which of the two kernels is quicker, by what 376 shapes (heads of 64 and 128, 1 to
// 128 of them, 8 to 256 rows, 50 to 8000 keys) took, in ns.  This kernel: a start,
// 0.6 us for a cluster's join, and a time for each block in a warp's turn, times the
// waves of CTAs (within 12% on average).  The kernel of 128-row tiles: a start, and for
// each wave of CTAs a start and a time per key tile (within 5%).  The quicker by this
// rule is the quicker one but for 0.6% on average and 21% at most; 32 rows as the border
// loses 19% on average.  One sequence of 8000 keys, 8 heads of 64: 12.8 us here for 32
// rows each and 27.4 for 256, 75 and 100 there; of 100 keys 6.6 here, 5.9 there.
bool cross_few_rows(const CrossParams& p) {
  const int G = p.Hq / p.Hkv, sms = sm_count(), d = p.d;
  const long long H = (long long)p.B * p.Hkv, rows = (long long)G * p.Nq;
  const bool two = rows > 16;
  const long long heads = H * (two ? (rows + 31) / 32 : 1);
  if (heads > (1 << 24)) return false;
  const int n = splits_of(heads, p.Nk, d), nk = 2048 / d;
  const long long blocks = ((p.Nk + nk - 1) / nk + WARPS * n - 1) / (WARPS * n);
  const double start = d == 128 ? (two ? 9000 : 4300) : (two ? 5000 : 3700);
  const double block = d == 128 ? (two ? 1350 : 1090) : (two ? 1440 : 860);
  const double waves = (double)heads * n / (2.0 * sms);
  const double here = start + (n > 1 ? 600 : 0) + block * blocks * (waves > 1 ? waves : 1);
  const int share = p.Nq <= 64 ? (128 / p.Nq < G ? 128 / p.Nq : G) : 1;
  const long long tiles = share > 1 ? (G + share - 1) / share : (long long)G * ((p.Nq + 127) / 128);
  const double turns = (double)((H * ((tiles + 1) / 2) + sms - 1) / sms);
  const double tile = d == 128 ? (tiles > 1 ? 1900 : 1250) : (tiles > 1 ? 1550 : 1120);
  const double there = 2300 + turns * (2300 + tile * ((p.Nk + 127) / 128));
  return here < there;
}

cudaError_t launch_cross_token(const CrossParams& p, cudaStream_t st) {
  Params a;
  a.p = p;
  const int nk = 2048 / p.d;
  if (p.Nk > 0) {
    if (!heads_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, nk, 1) || !heads_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, nk, 1))
      return cudaErrorInvalidValue;
  } else {
    memset(&a.k, 0, sizeof(a.k));          // never loaded from
    a.v = a.k;
  }
  const int rows = p.Hq / p.Hkv * p.Nq;
  const bool two = rows > 16, wide = p.d == 128;
  a.groups = Divisor((rows + 31) / 32);
  a.hkv = Divisor(p.Hkv);
  a.nq = Divisor(p.Nq);
  const long long heads = (long long)p.B * p.Hkv * a.groups.d;
  a.splits = splits_of(heads, p.Nk, p.d);
  const int n = a.splits;
  auto k = wide ? (two ? cross_token_kernel<128, 2> : cross_token_kernel<128, 1>)
                : (two ? cross_token_kernel<64, 2> : cross_token_kernel<64, 1>);
  const int smem = wide ? (two ? Smem<128, 2>::bytes(n) : Smem<128, 1>::bytes(n))
                        : (two ? Smem<64, 2>::bytes(n) : Smem<64, 1>::bytes(n));
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), 112 * 1024, true);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * a.splits));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace fa4
