// cache_line.cuh -- what the kernels that stream the cache share: the line of
// work units and its equal shares, the window of looked-up pages, and the
// layout of 8-bit rows as TMA's swizzle leaves them in shared memory.
#pragma once
#include "cache.cuh"

namespace fa4 {

constexpr int LINE_WARPS = 4;                // warps of a CTA
constexpr int UNIT = 32 * LINE_WARPS;        // keys of a unit; a warp's step is 32
constexpr int kSMs = 152;                    // GB300

// Units of a run of keys (at least one).
__host__ __device__ inline int units_of(long long keys) {
  const long long u = (keys + UNIT - 1) / UNIT;
  return u < 1 ? 1 : (int)u;
}

// CTAs that get a share.  No share is empty (a join reads every slot from the
// first to the last), and no CTA is there only to make some shares shorter
// than the longest: it would add a slot to the join and save nothing.
FA4_DEV unsigned workers(unsigned total, unsigned grid) {
  const unsigned longest = (total + grid - 1) / grid;
  return (total + longest - 1) / longest;
}

// The line cut into n shares, the first `rem` of them one unit longer.
struct Shares {
  unsigned per, rem;
  FA4_DEV Shares(unsigned total, unsigned n) : per(total / n), rem(total % n) {}
  FA4_DEV unsigned begin(unsigned i) const { return i * per + min(i, rem); }
  FA4_DEV unsigned of(unsigned u) const {          // the share that holds unit u
    const unsigned cut = rem * (per + 1);
    return u < cut ? u / (per + 1) : rem + (u - cut) / per;
  }
};

// Units of all sequences (whole warp); units(b) is a sequence's.
template <class F>
FA4_DEV unsigned line_total(int B, F units) {
  unsigned all = 0;
  for (int i = threadIdx.x % 32; i < B; i += 32) all += units(i);
  return __reduce_add_sync(0xffffffffu, all);
}

// The sequence b that holds unit `at` of the line and its first unit seq0
// (whole warp), looked for from the given b and seq0 on (0 and 0, or an earlier
// answer).  Returns false if the line ends before.
template <class F>
FA4_DEV bool line_find(int B, F units, unsigned at, int& b, unsigned& seq0) {
  const int lane = threadIdx.x % 32;
  for (int base = b; base < B; base += 32) {
    const unsigned mine = base + lane < B ? units(base + lane) : 0;
    unsigned inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, seq0 + inc > at);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = base + src;
      seq0 += __shfl_sync(0xffffffffu, inc - mine, src);
      return true;
    }
    seq0 += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// The mark of a counter word, in its high 48 bits (no number, no pointer and no
// pair of floats that a workspace could hold from other use).
constexpr unsigned long long MARK = 0xfa4c0de5eed5ull;
// One arrival at a counter word: whether it is the last of n, which leaves the
// word marked and at zero for the next call.  Release before, acquire after.
FA4_DEV bool marked_arrive(unsigned long long* word, unsigned n) {
  // one addition, unless the word holds anything but a marked count: then
  // whoever swaps that for the mark and a count of one has arrived, and the
  // others add again (a swap fails only when the word has changed, by another
  // arrival)
  unsigned long long had = atomic_add_acq_rel(word, 1ull);
  if ((had >> 16) != MARK) {
    ++had;
    for (;;) {
      __threadfence();
      const unsigned long long was = atomicCAS(word, had, MARK << 16 | 1u);
      if (was == had) { had = MARK << 16; break; }
      had = was;
      if ((had >> 16) == MARK) { had = atomic_add_acq_rel(word, 1ull); break; }
    }
  }
  const bool last = (unsigned)(had & 0xffffu) + 1 == n;
  if (last) {
    atomicExch(word, MARK << 16);
    __threadfence();
  }
  return last;
}

// A warp's keys of a unit lie in NP pages (one, or two of 16 keys).  The window
// holds, one entry a lane, what is to be known of the next 32 / NP units: pool
// page, position of the first key, scales.  Looking up 32 entries costs the
// three dependent loads (list, table, scale) once.
constexpr int NOWHERE = 0x40000000;          // a position that every query masks
struct Entry {
  int page, pos;                             // -1 and NOWHERE: no such keys
  uint32_t ks, vs;
};
template <int NP>
struct Window {
  int first;                                 // unit of the first entry
  Entry e;

  // Entries of units u.. < end for this warp of a CTA: sequence b of len tokens,
  // kv head h; sel: a list of n_sel pages to go through, or nullptr (all).
  FA4_DEV void fill(const CacheView& c, int b, int h, int len, const int* sel, int n_sel, int u, int end) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int log_p = 31 - __clz(c.page);
    first = u;
    const int unit = u + lane / NP;
    const int v = unit * UNIT + 32 * warp + 16 * (lane % NP);
    int lp = v >> log_p;
    e.page = -1;
    e.pos = NOWHERE;
    e.ks = e.vs = 0;
    if (unit < end) {
      if (sel) {
        lp = lp < n_sel ? *(sel + lp) : -1;
        if (lp >= c.max_pages || lp < -1) { atomicOr(c.err, FA4_DEVERR_INDEX); lp = -1; }
      }
      if (lp >= 0 && ((long long)lp << log_p) < len) {
        e.page = cache_page(c, c.table, b, lp);
        if (e.page >= 0) {
          const long long ph = (long long)e.page * c.Hkv + h;
          e.ks = *(c.ks + ph);
          e.vs = *(c.vs + ph);
          e.pos = (lp << log_p) + (v & (c.page - 1));
        }
      }
    }
    __syncwarp();
  }
  FA4_DEV bool has(int u) const { return u < first + 32 / NP; }
  FA4_DEV int page(int u, int i) const { return __shfl_sync(0xffffffffu, e.page, (u - first) * NP + i); }
  FA4_DEV int pos(int u, int i) const { return __shfl_sync(0xffffffffu, e.pos, (u - first) * NP + i); }
  // K's scale byte, and V's above it
  FA4_DEV int scales(int u, int i) const {
    return __shfl_sync(0xffffffffu, (int)(e.ks | e.vs << 8), (u - first) * NP + i);
  }
};

// Order of the eight keys of an operand (its row i is key korder(i)), and of
// the eight 16-byte words of a V row among the lanes: with the 128-byte swizzle
// both reads are then free of bank conflicts (D = 128).  The 64-byte rows of
// D = 64 are free of them for K in natural order, and two-way for V.
template <int D>
FA4_DEV constexpr int korder(int i) {
  return D == 128 ? ((i & 1) << 2) | (i & 2) | (i >> 2) : i;
}
// Byte of row `row` and byte column `x` in a box of D-byte rows as TMA's swizzle
// lays it out.
template <int D>
FA4_DEV int boxed(int row, int x) {
  return D == 128 ? row * 128 + (x ^ ((row & 7) << 4)) : row * 64 + (x ^ (((row >> 1) & 3) << 4));
}

// 2^x for x in [-382, 127]: the exact power, subnormal or zero where FP32 ends.
FA4_DEV float pow2_any(int x) {
  return x >= -126 ? exp2i(x) : (x >= -149 ? __uint_as_float(1u << (x + 149)) : 0.f);
}

// ----------------------------------------------------------------------------
// The rank-th largest (1 = largest) of a CTA's unsigned keys, 1024 threads.
// The keys' range is divided evenly into 2048 bins, which spreads values of any
// scale; the bin with the rank usually holds a few keys, which are ranked by
// counting, else it is divided again (three times at most).  Digits of the keys
// instead crowd them into few bins, and counting those costs 1.4 to 3 us a
// digit of 8192 weights; halving the range by comparisons 0.6 to 2 us a step.
constexpr int KTH_THREADS = 1024, KTH_BINS = 2048;
constexpr unsigned KTH_FEW = 256;
struct KthShared {
  unsigned hist[KTH_BINS];
  unsigned bin, rank, count, lo, hi, few, tot[32];
};
// `key`: fewer than `rank` keys are above it if not `all`, and of those equal to
// it `ties` belong to the rank-th largest; `all`: exactly `rank` keys reach it.
struct Cut {
  uint32_t key;
  unsigned ties;
  bool all;
};
// each(f) calls f(key) for every key of the thread; 0 < rank <= keys.
template <class EACH>
FA4_DEV Cut kth_largest(KthShared& s, unsigned rank, EACH each) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t lo = 0xffffffffu, hi = 0u;
  if (threadIdx.x == 0) { s.lo = 0xffffffffu; s.hi = 0u; s.few = 0u; }
  each([&](uint32_t key) { lo = min(lo, key); hi = max(hi, key); });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if (lane == 0) { atomicMin(&s.lo, lo); atomicMax(&s.hi, hi); }
  for (int turn = 0;; ++turn) {
    for (int i = threadIdx.x; i < KTH_BINS; i += KTH_THREADS) s.hist[i] = 0;
    __syncthreads();
    if (turn == 0) { lo = s.lo; hi = s.hi; }
    const int shift = max(0, 32 - __clz((int)(hi - lo)) - 11);     // 2048 bins cover lo .. hi
    each([&](uint32_t key) {
      if (key >= lo && key <= hi) atomicAdd(&s.hist[(key - lo) >> shift], 1u);
    });
    __syncthreads();
    // two bins a thread, from the top: where the rank falls
    const unsigned v0 = s.hist[KTH_BINS - 1 - 2 * threadIdx.x], v1 = s.hist[KTH_BINS - 2 - 2 * threadIdx.x];
    unsigned inc = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) s.tot[warp] = inc;
    __syncthreads();
    unsigned tot = s.tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned up = __shfl_up_sync(0xffffffffu, tot, o);
      if (lane >= o) tot += up;
    }
    const unsigned sum = __shfl_sync(0xffffffffu, tot, max(warp - 1, 0));
    const unsigned before = (warp ? sum : 0u) + inc - v0 - v1;
    if (before < rank && rank <= before + v0 + v1) {
      const bool first = rank <= before + v0;
      s.bin = KTH_BINS - 1 - 2 * threadIdx.x - (first ? 0 : 1);
      s.rank = rank - before - (first ? 0 : v0);
      s.count = first ? v0 : v1;
    }
    __syncthreads();
    lo += s.bin << shift;
    hi = lo + ((1u << shift) - 1u);
    rank = s.rank;
    const unsigned count = s.count;
    if (count == rank) return {lo, 0u, true};        // the whole bin
    if (shift == 0) return {lo, rank, false};        // the bin is one key
    if (count <= KTH_FEW) {                          // the bin's keys, ranked by counting
      each([&](uint32_t key) {
        if (key >= lo && key <= hi) s.hist[atomicAdd(&s.few, 1u)] = key;
      });
      __syncthreads();
      if (threadIdx.x < count) {
        const uint32_t mine = s.hist[threadIdx.x];
        unsigned more = 0, same = 0;
        for (unsigned i = 0; i < count; ++i) {
          const uint32_t o = s.hist[i];
          more += o > mine ? 1u : 0u;
          same += o == mine ? 1u : 0u;
        }
        if (more < rank && rank <= more + same) {
          s.lo = mine;
          s.rank = rank - more;
          s.count = same;
        }
      }
      __syncthreads();
      return {s.lo, s.rank, s.count == s.rank};
    }
    __syncthreads();                                 // all have read bin, rank, count
  }
}

// A contiguous copy into shared memory, counted on an mbarrier.
FA4_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// ----------------------------------------------------------------------------
// Tiles of f16 rows in shared memory as the products of tcgen05 read them: 128
// rows, 64 values (128 bytes, swizzled) a chunk.
constexpr int F16_CHUNK = 128 * 128;

// Sixteen codes to f16 into the two 16-byte units of a row that they fill.
// Lanes of the odd half store the units in the other order: eight lanes at a
// time then touch every bank once.
template <int D>
FA4_DEV void store16(uint8_t* tile, int row, int part, const uint4& x) {
  const uint4 lo = make_uint4(e4m3x2_to_f16x2(x.x), e4m3x2_hi_to_f16x2(x.x), e4m3x2_to_f16x2(x.y),
                              e4m3x2_hi_to_f16x2(x.y));
  const uint4 hi = make_uint4(e4m3x2_to_f16x2(x.z), e4m3x2_hi_to_f16x2(x.z), e4m3x2_to_f16x2(x.w),
                              e4m3x2_hi_to_f16x2(x.w));
  uint8_t* at = tile + part / 4 * F16_CHUNK + row * 128;
  const int u = 2 * (part % 4);
  const bool odd = part >= 4;
  *reinterpret_cast<uint4*>(at + (((u + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
  *reinterpret_cast<uint4*>(at + (((u + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
}

// Each lane's row of q (nullptr: zeros) as f16 under a power of two into rows
// row0..+31 of such a tile (whole warp): the largest magnitude comes into
// [2^7, 2^8), as in QRaw.  Returns the exponent that undoes it.  D / 8 lanes
// read a row, whole lines at a time.  A loop: the code runs once or twice in a
// kernel's life, and straight-line code waits for its own instructions then.
template <int D>
FA4_DEV int store_query_rows(uint8_t* tile, int row0, const __nv_bfloat16* mine) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, AT_ONCE = 32 / RPI;
  const int lane = threadIdx.x % 32, word = lane % LPR;
  int e_mine = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < 32; i0 += RPI * AT_ONCE) {
    uint4 w[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const unsigned long long src =
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), i0 + RPI * i + lane / LPR);
      w[i] = src ? reinterpret_cast<const uint4*>(src)[word] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int row = i0 + RPI * i + lane / LPR;
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = max(amax, max((u[k] << 16) & 0x7fffffffu, u[k] & 0x7fff0000u));
#pragma unroll
      for (int o = 1; o < LPR; o *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int E = (int)(amax >> 23);
      const int e = (E == 0 || E == 255) ? 0 : max(-120, min(120, E - 134));
      const float down = exp2i(-e);
      uint32_t z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        z[k] = pack_f16x2(__uint_as_float(u[k] << 16) * down, __uint_as_float(u[k] & 0xffff0000u) * down);
      *reinterpret_cast<uint4*>(tile + word / 8 * F16_CHUNK + (row0 + row) * 128 + ((word % 8 ^ (row & 7)) << 4)) =
          make_uint4(z[0], z[1], z[2], z[3]);
      const int theirs = __shfl_sync(0xffffffffu, e, lane % RPI * LPR);
      if (lane / RPI == i0 / RPI + i) e_mine = theirs;
    }
  }
  return e_mine;
}

// lse in log2 units as a float and the factor that makes up for its rounding;
// rows that add nothing (e^-inf for every key if lse is infinite) get (0, 0).
FA4_DEV void reference(float lse, bool in, float& ref, float& fac) {
  ref = 0.f;
  fac = 0.f;
  if (in && !isinf(lse)) {
    ref = lse * 1.4426950216293335f;
    const float rest = fmaf(lse, 1.4426950216293335f, -ref) + lse * 1.9259629911266175e-8f;
    fac = ex2_approx(-rest);
  }
}

}  // namespace fa4
