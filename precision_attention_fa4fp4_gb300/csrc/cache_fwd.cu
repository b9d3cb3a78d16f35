// cache_fwd.cu -- attention of a few queries per sequence over the paged 8-bit
// cache (all pages, or the pages selected for each query).
//
//   s_j = scale q.k_j,  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// The keys are the long axis and every key is read once per kv head, so the
// kernel is bound by HBM: d bytes of K and d of V per key and kv head, whatever
// the number of query heads that share them.  The query rows of a kv head
// (group x tokens) are taken 8 or 16 at a time.
//
// Work: the rows of one kv head over 128 keys are one unit; the units of all
// (sequence, head, row block) lie in one line, and CTA i of a fixed grid takes
// the i-th equal share of the line.  So a batch of very different lengths is as
// even as a batch of equal ones, and few rows over a long cache are split over
// the whole GPU.  A share that covers a row block completely writes its
// output; the others (at most two per CTA) leave (max, sum, unnormalized o) in
// the workspace, and the CTA that is the last to do so for a row block joins
// them, in a fixed order.  It knows that it is the last from a counter word in
// the workspace.  The words need no setting up: each carries a mark beside its
// count, the first arrival that finds none puts it there, and the last leaves
// the word marked and at zero for the next call.
//
// Inside a CTA four warps take 32 keys each of every unit and keep their own
// running max and sum; they meet once, at the end of a share.
//
// Products: m16n8k16 with the keys as rows, so that eight queries fill the
// instruction: S^T = K Q^T, O^T += V^T P.  A lane reads 16 bytes of an 8-bit row
// at a time and one conversion (E4M3 -> f16, exact) makes them A operands; for
// V^T the two keys of an operand pair are interleaved with a byte permute.
// Every warp has its own queue in shared memory, two or three steps of 32 keys
// deep, filled by TMA (a 4 KB box of K and of V a step) and drained by the warp
// alone: no barrier between warps in the loop, and far more in flight than
// loads through L1 allow (16-byte asynchronous copies of the same bytes, and
// loads into registers, both stopped at 4.8 TB/s).  The codes are used
// unscaled: K's page scale multiplies the scores, V's goes into the exponent of
// P, relative to that of the row's accumulator.
//
// 64 sequences of 1..8192 tokens, 32 / 8 heads of 128: 110 us, 5.1 TB/s; what
// is missing to a copy's 6.7 are the first 5 us of a launch and the ends of row
// blocks.  One of 1000: 9.2 us (start 2, lens and pages 1.5, first keys 2, join
// 2-3).  With 9 to 16 rows and FP32 output instructions bound it: 4 sequences of
// 16001..32760, 8 heads of 64, 42 us, 2.4 TB/s.
//
// Roundings: q to f16 under a power of two (2^-32 of the row's largest); P to
// f16 under a factor 2^15 and V's relative exponent (2^-11 of P, or 2^-36 of the
// largest V of the 32 keys or 2^-90 of the row's own sum if that is more), for FP32
// output as a sum of two f16 (2^-22, or the same).  The normalizer sums the FP32
// values of P.
#include "cache_line.cuh"

namespace fa4 {
namespace {

constexpr int NW = LINE_WARPS;
// log2 of the factor on P: the largest P is half of f16's largest power
constexpr float P_BIAS = 15.f;
// How far a step's greatest V exponent may lie below that of a row's accumulator
// before the latter is lowered: P's smallest f16 step, 2^-24 under its factor 2^15,
// is then at most 2^-35 of the step's largest V, its half 2^-36.  It is lowered only
// as far as leaves the row's sums below 2^O_MOST, beside which later terms (2^15 *
// 448, fewer than 2^20 of them a warp) are none: what a page far below loses then
// is 2^-90 of the row's own sum.  Rows have exponents of their own, as the sums of
// rows over the same keys may lie as far apart as V does.
constexpr int V_DOWN = 4, O_MOST = 100;
// A factor of 2^-P_NONE leaves no f16 of P.
constexpr float P_NONE = 48.f;
// 2^x for a whole number x in [-126, 127]: x + 127 is read off the significand.
FA4_DEV float exp2f_whole(float x) { return __uint_as_float(__float_as_uint(x + (12582912.f + 127.f)) << 23); }
// Rows of a kv head above which the kernel for many rows takes over.  It takes
// the same time for 1 to 128 of them, this one in proportion to blocks of 16.
// Keys x sequences, heads of 128, 8 kv heads, us here / there:
//   2048 x 16:  64 rows 63 / 60,  128 rows 114 / 52,  256 rows 208 / 64
//   8192 x 1:   64 rows 26 / 32,  128 rows 36 / 31,   256 rows 58 / 41
//   1024 x 1:   64 rows 16 / 22,  256 rows 19 / 23 (the price of one rule)
// heads of 64, 4096 x 16: 64 rows 69 / 72, 96 rows 98 / 72.
// FP32 output always comes here: 2048 x 16, 128 rows 142, 256 rows 265.
constexpr int MANY_ROWS = 64;

// Resident CTAs by registers, and the steps in flight that fill the shared
// memory they leave.
constexpr int ctas_per_sm(int d, int nt) { return d == 128 && nt == 2 ? 2 : 3; }
constexpr int stages(int d, int nt) { return d == 128 && nt == 1 ? 2 : d == 128 ? 3 : 4; }

// Row blocks and units of the line.
struct Line {
  int R;                // rows of a block
  int per_head;         // row blocks of one (sequence, head)
  int nb;               // row blocks of one sequence
  int G;                // query heads per kv head
  int QG;               // selected pages: row blocks of one token
};

__host__ __device__ inline Line make_line(int Hq, int Hkv, int T, bool sparse) {
  Line l;
  l.G = Hq / Hkv;
  const long long rows = sparse ? l.G : (long long)l.G * T;
  l.R = rows <= 8 ? 8 : 16;
  l.QG = sparse ? (l.G + l.R - 1) / l.R : 0;
  l.per_head = sparse ? T * l.QG : (int)((rows + l.R - 1) / l.R);
  l.nb = Hkv * l.per_head;
  return l;
}

// Units of one row block of sequence b (one, which writes the output, where the
// row has no keys).  A list of pages may name them in any order, with holes.
FA4_DEV int seq_units(const CacheFwdParams& p, int b) {
  const int len = cache_len(p.c, b), q_len = cache_count(p.q_lens, b, p.T, p.c.err);
  if (len == 0 || q_len == 0) return 1;
  return units_of(p.pages ? (long long)p.n_sel * p.c.page : len);
}

// Sums of V that leave the registers are in units of 2^HIGH where their exponent
// lies above FROM (the sum of many values near bf16's end would pass FP32's), and
// their sum of weights l is then negative.
constexpr float FROM = -40.f;
constexpr int HIGH = 48;             // |o| <= l * 2^128 with l < 2^15 * 2^30
constexpr float TO_HIGH = 0x1p-48f, FROM_HIGH = 0x1p48f;

template <int D, int NT>
struct Slot {
  static constexpr int R = 8 * NT;
  static constexpr int FLOATS = R * D + 2 * R;     // o, then m, then l
  // bytes of the counter words before the slots
  __host__ __device__ static constexpr size_t counters(unsigned grid) { return ((size_t)grid * 8 + 15) / 16 * 16; }
};

template <int D, int NT>
struct Queue {
  static constexpr int S = stages(D, NT);
  static constexpr int BYTES = 2 * 32 * D;                       // K and V of 32 keys
  static constexpr int WARP = S * BYTES;
  static constexpr int OS = D + 4;                               // row stride of the merge buffer
  static constexpr int MERGE = NW * 8 * NT * (OS + 2) * 4;       // lies over the queues
  static constexpr int OFF_BAR = NW * WARP > MERGE ? NW * WARP : MERGE;
  static constexpr int OFF_STEP = OFF_BAR + 8 * NW * S;          // 16 bytes a step: positions, scales
  static constexpr int OFF_MISC = OFF_STEP + 16 * NW * S;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;              // and the swizzle's alignment
};

template <int D, int NT, bool SPLIT, bool SMALLP>
__global__ void __launch_bounds__(32 * NW, ctas_per_sm(D, NT)) cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using Q = Queue<D, NT>;
  constexpr int R = 8 * NT;
  constexpr int S = Q::S;
  grid_start();
  constexpr int NP = SMALLP ? 2 : 1;               // pages of a warp's 32 keys
  constexpr int OS = Q::OS;
  constexpr int VW = D / 32;                       // 32-bit words of V a lane holds per key
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + smem_pad(smem_raw);
  float (*s_o)[R][OS] = reinterpret_cast<float (*)[R][OS]>(smem);
  float (*s_m)[R] = reinterpret_cast<float (*)[R]>(smem + NW * R * OS * 4);
  float (*s_l)[R] = s_m + NW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Q::OFF_BAR) + threadIdx.x / 32 * S;
  int4* steps = reinterpret_cast<int4*>(smem + Q::OFF_STEP) + threadIdx.x / 32 * S;
  int* s_misc = reinterpret_cast<int*>(smem + Q::OFF_MISC);
  volatile int* abort_flag = s_misc;

  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t4 = lane % 4;
  const Line ln = make_line(p.Hq, c.Hkv, p.T, p.pages != nullptr);
  const int G = ln.G;
  const int log_p = 31 - __clz(c.page);
  uint8_t* queue = smem + warp * Q::WARP;
  unsigned phases = 0;                             // parity of each step's barrier
  if (lane == 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();
  // byte offsets of the lane's words in a box of 16 keys
  int ko[2][D / 64], vo[4];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) ko[r][x] = boxed<D>(korder<D>(g) + 8 * r, 64 * x + 16 * t4);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    vo[r] = boxed<D>(korder<D>(2 * t4 + (r & 1)) + 8 * (r >> 1), (D / 8) * (D == 128 ? korder<D>(g) : g) & ~15) +
            (D == 64 ? 8 * (g & 1) : 0);
  const int v_dim = (D / 8) * (D == 128 ? korder<D>(g) : g);   // first head dimension of the lane's V bytes

  grid_wait();
  // Few row blocks: the shares are cut at their ends, into parts of at most `cut`
  // units, so that no CTA has to finish one row block and begin another.  The
  // shortest cut that leaves no more parts than CTAs is searched from below.
  // (lane i keeps the units of sequence i where there are no more than 32)
  const unsigned mine = lane < c.B ? (unsigned)seq_units(p, lane) : 0u;
  auto lane_units = [&](int i) -> unsigned { return i < 32 ? mine : (unsigned)seq_units(p, i); };   // i % 32 == lane
  const unsigned total = line_total(c.B, [&](int i) -> unsigned { return lane_units(i) * ln.nb; });
  unsigned cut = 0;
  if (2LL * ln.nb * c.B <= gridDim.x) {
    cut = (total + gridDim.x - 1) / gridDim.x;
    while (cut > 1 &&
           line_total(c.B, [&](int i) -> unsigned { return (lane_units(i) + cut - 1) / cut * ln.nb; }) > gridDim.x)
      cut += cut / 16 + 1;
  }
  // a sequence's stretch of the line: parts, or units
  auto stretch = [&](unsigned u) -> unsigned { return (cut > 1 ? (u + cut - 1) / cut : u) * ln.nb; };
  const Shares shares(total, workers(total, gridDim.x));
  unsigned at, end, seq0 = 0;
  if (cut) {
    at = blockIdx.x;
    end = at + 1;
  } else {
    if (blockIdx.x >= workers(total, gridDim.x)) return;
    at = shares.begin(blockIdx.x);
    end = shares.begin(blockIdx.x + 1);
  }
  const unsigned begin = at;
  int b = 0;
  if (!line_find(c.B, [&](int i) -> unsigned { return stretch(lane_units(i)); }, at, b, seq0))
    return;                                        // more CTAs than parts
  int units = seq_units(p, b);

  while (at < end) {
    while (at >= seq0 + stretch(units)) {
      seq0 += stretch(units);
      units = seq_units(p, ++b);
    }
    // row block, its units u0 .. u1, and where its slots lie: those of n CTAs
    // from c0, the first of them perhaps its second
    int rb, u0, u1, n, odd = 0;
    unsigned c0;
    if (cut) {
      n = (units + cut - 1) / cut;
      rb = (int)((at - seq0) / n);
      const unsigned part = (at - seq0) % n;
      u0 = (int)((unsigned long long)units * part / n);
      u1 = (int)((unsigned long long)units * (part + 1) / n);
      c0 = seq0 + (unsigned)rb * n;
    } else {
      rb = (int)((at - seq0) / units);
      u0 = (int)((at - seq0) % units);
      u1 = (int)min((unsigned)units, u0 + (end - at));
      const unsigned start = seq0 + (unsigned)rb * units;
      c0 = shares.of(start);
      n = (int)(shares.of(start + units - 1) - c0) + 1;
      odd = shares.begin(c0) >= start ? 0 : 1;
    }
    const int h = rb / ln.per_head, sub = rb % ln.per_head;
    const int len = cache_len(c, b);
    const int q_len = cache_count(p.q_lens, b, p.T, c.err);
    // query row of column col of this block
    auto row_of = [&](int col, int& t, int& gg) -> bool {
      if (p.pages) {
        t = sub / ln.QG;
        gg = (sub % ln.QG) * R + col;
      } else {
        const int r = sub * R + col;
        t = r / G;
        gg = r % G;
      }
      return gg < G && t < q_len;
    };
    const int* sel = p.pages ? p.pages + (((long long)b * c.Hkv + h) * p.T + sub / ln.QG) * p.n_sel : nullptr;

    QRaw<D> raw[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      int t, gg;
      const bool in = row_of(8 * n + g, t, gg);
      raw[n].fetch(in ? reinterpret_cast<const __nv_bfloat16*>(p.q) + (((long long)b * p.Hq + h * G + gg) * p.T + t) * D
                      : nullptr, t4);
    }
    Window<NP> window;
    window.fill(c, b, h, len, sel, p.n_sel, u0, u1);
    // A step's boxes; then, apart, what it needs besides them: the boxes are not
    // to wait for the scales' loads.
    auto issue = [&](int s, int u) {
      if (!window.has(u)) window.fill(c, b, h, len, sel, p.n_sel, u, u1);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int page = window.page(u, i), pos = window.pos(u, i);
        if (page >= 0 && lane == 0) {
          const int row = (int)(((long long)page * c.Hkv + h) << log_p) + (pos & (c.page - 1));
          uint8_t* to = queue + s * Q::BYTES + (SMALLP ? i * 16 * D : 0);
          // each box counts for itself: a step without a page has none
          mbar_expect_tx(&bars[s], 2 * (32 / NP) * D);
          tma_load_3d(to, &p.tm_k, &bars[s], 0, row, 0);
          tma_load_3d(to + 32 * D, &p.tm_v, &bars[s], 0, row, 0);
        }
      }
      if (lane == 0) mbar_arrive(&bars[s]);
    };
    auto note = [&](int s, int u) {
      int4 what = make_int4(window.pos(u, 0), window.scales(u, 0), NOWHERE, 0);
      if (NP == 2) { what.z = window.pos(u, NP - 1); what.w = window.scales(u, NP - 1); }
      if (lane == 0) steps[s] = what;
    };
    // (the first S units lie in the first window)
    for (int s = 0; s < S; ++s) issue(s, u0 + s);
    for (int s = 0; s < S; ++s) note(s, u0 + s);

    QFrag<D> q[NT];
    float fx[NT][2];                               // log2-unit factor of columns 2 t4, 2 t4 + 1
    int vis[NT][2];                                // keys they see
    int vis_min = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      int t, gg;
      const float e = raw[n].convert(q[n]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fx[n][j] = p.c2 * __shfl_sync(0xffffffffu, e, (2 * t4 + j) * 4);
        const bool in = row_of(8 * n + 2 * t4 + j, t, gg);
        const int see = p.causal ? len - q_len + t + 1 : len;
        vis[n][j] = in ? max(0, min(len, see)) : 0;
        if (in) vis_min = min(vis_min, vis[n][j]);
      }
    }
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
    // o is in units of 2^xo; the first step's to begin with
    float first = -127.f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (window.page(u0, i) >= 0) first = fmaxf(first, (float)((window.scales(u0, i) >> 8) - 127));
    float xo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xo[n][0] = xo[n][1] = first;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    auto body = [&](int st, int u) -> bool {
      if (!mbar_wait(&bars[st], (phases >> st) & 1, abort_flag, c.err)) return false;
      phases ^= 1u << st;
      __syncwarp();
      const uint8_t* from = queue + st * Q::BYTES;
      const int4 what = steps[st];
      int pos[NP];
      float kxc[NP];
      float ev[NP];                                // V's exponents
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        pos[i] = i ? what.z : what.x;
        const int sc = i ? what.w : what.y;
        kxc[i] = e8m0_value(sc & 0xff);
        ev[i] = pos[i] == NOWHERE ? -1000.f : (float)((sc >> 8) - 127);
      }
      // scores of 32 keys: rows g, g + 8 of each 16, columns 2 t4, 2 t4 + 1
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
          float half[SPLIT ? NT : 1][4];
          const uint4 ka = lds16(from + i * 16 * D + ko[0][k]);
          const uint4 kb = lds16(from + i * 16 * D + ko[1][k]);
          const uint32_t lo[4] = {ka.x, ka.y, ka.z, ka.w};
          const uint32_t hi[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(lo[w]), a2 = e4m3x2_hi_to_f16x2(lo[w]);
            const uint32_t a1 = e4m3x2_to_f16x2(hi[w]), a3 = e4m3x2_hi_to_f16x2(hi[w]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (SPLIT) {
                if (w % 2 == 0) half[n][0] = half[n][1] = half[n][2] = half[n][3] = 0.f;
                mma_16816(half[n], a0, a1, a2, a3, q[n].b[4 * k + w][0], q[n].b[4 * k + w][1]);
                if (w % 2)
#pragma unroll
                  for (int e = 0; e < 4; ++e) s[n][i][e] += half[n][e];
              } else {
                mma_16816(s[n][i], a0, a1, a2, a3, q[n].b[4 * k + w][0], q[n].b[4 * k + w][1]);
              }
            }
          }
        }
      bool full = true;
#pragma unroll
      for (int i = 0; i < NP; ++i) full = full && pos[i] + 32 / NP <= vis_min;

      float ev_max = ev[0];
#pragma unroll
      for (int i = 1; i < NP; ++i) ev_max = fmaxf(ev_max, ev[i]);

      uint32_t ph[NT][2][2], pl[NT][2][2];         // P^T as the B operand: [16 keys][k half]
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mx[2] = {m[n][0], m[n][1]};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (the factors first: K's times the sum alone may pass FP32's end)
            float x = s[n][i][j] * (kxc[i % NP] * fx[n][j & 1]);
            if (!full) {
              const int key = pos[i % NP] + (SMALLP ? 0 : 16 * i) + korder<D>(g) + 8 * (j >> 1);
              if (key >= vis[n][j & 1]) x = -INFINITY;
            }
            s[n][i][j] = x;
            mx[j & 1] = fmaxf(mx[j & 1], x);
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
        }
        if (__any_sync(0xffffffffu, mx[0] != m[n][0] || mx[1] != m[n][1])) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float a = mx[j] == m[n][j] ? 1.f : ex2_approx(m[n][j] - mx[j]);
            m[n][j] = mx[j];
            l[n][j] *= a;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[n][i][j] *= a;
              o[n][i][2 + j] *= a;
            }
          }
        }
        // V's exponents relative to the accumulators' go into P.  A page above an
        // accumulator raises it, a step far below lowers it
        auto off = [&](float x) { return ev_max > x || ev_max < x - V_DOWN; };
        if (ev_max > -1000.f && __any_sync(0xffffffffu, off(xo[n][0]) || off(xo[n][1]))) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t most = 0;                     // of the row's sums, over the lanes that hold it
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              most = max(most, max(__float_as_uint(o[n][i][j]) & 0x7fffffffu, __float_as_uint(o[n][i][2 + j]) & 0x7fffffffu));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 4));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 8));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
            const int x = (int)xo[n][j], e = (int)ev_max;
            const int room = max(0, O_MOST + 126 - (int)(most >> 23));      // up to 226
            const int to = !off(xo[n][j]) ? x : most == 0 ? e : max(e, x - room);
            const int up = most == 0 ? 0 : x - to;
            const float by = pow2_any(min(up, 100)), more = exp2i(max(up - 100, 0));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[n][i][j] = o[n][i][j] * by * more;
              o[n][i][2 + j] = o[n][i][2 + j] * by * more;
            }
            xo[n][j] = (float)to;
          }
        }
        float vd[2][NP], up[2][NP];                // exponent on P, its whole factor
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            vd[j][i] = fmaxf(ev[i] - xo[n][j], -P_NONE);
            up[j][i] = exp2f_whole(P_BIAS + vd[j][i]);
          }
        // nothing seen yet: any finite reference will do, the masked scores
        // stay -inf
        const float r0 = (m[n][0] == -INFINITY ? 0.f : m[n][0]) - (SPLIT ? 0.f : P_BIAS);
        const float r1 = (m[n][1] == -INFINITY ? 0.f : m[n][1]) - (SPLIT ? 0.f : P_BIAS);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // FP32 output: the factor on P comes after the exponential, whose
            // argument (and so its rounding) is then small for large weights
            if constexpr (SPLIT) e[j] = ex2_approx(s[n][i][j] - ((j & 1) ? r1 : r0)) * up[j & 1][i % NP];
            else e[j] = ex2_approx(s[n][i][j] - (((j & 1) ? r1 : r0) - vd[j & 1][i % NP]));
          }
          l[n][0] = fmaf(e[0] + e[2], exp2f_whole(-vd[0][i % NP]), l[n][0]);
          l[n][1] = fmaf(e[1] + e[3], exp2f_whole(-vd[1][i % NP]), l[n][1]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = pack_f16x2(e[2 * r], e[2 * r + 1]);
            ph[n][i][r] = movmatrix_trans(x);
            if constexpr (SPLIT) {
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
              pl[n][i][r] = movmatrix_trans(pack_f16x2(e[2 * r] - y.x, e[2 * r + 1] - y.y));
            }
          }
        }
      }
      uint32_t vr[2][4][VW];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (VW == 4) {
            const uint4 x = lds16(from + (32 + 16 * i) * D + vo[r]);
            vr[i][r][0] = x.x; vr[i][r][1] = x.y; vr[i][r][2] = x.z; vr[i][r][3] = x.w;
          } else {
            const uint2 x = lds8(from + (32 + 16 * i) * D + vo[r]);
            vr[i][r][0] = x.x; vr[i][r][1] = x.y;
          }
        }
      // keys past the sequence's end hold anything: 0 * NaN must not happen
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = pos[i % NP] + (SMALLP ? 0 : 16 * i) + korder<D>(2 * t4 + (k & 1)) + 8 * (k >> 1);
            if (key >= len)
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[i][k][w] = 0;
          }
      }
      // O^T += V^T P: lane rows (D / 8) g + 2 mt and + 1 of the head dimension.
      // The products' accumulators are cut, not rounded: for FP32 output a step's
      // sum is taken by itself and added with rounding, as the scores' are by 32
      // dimensions.  All in all 3 us of 42 (4 x 16001..32760 keys), and on six
      // sequences of 4205..15496 an output off by 3.3e-7 of its norm (4.9e-7 in
      // plain FP32) that was off by more than 1e-6.
      float part[SPLIT ? NT : 1][4];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const int mt = j / 2, i = j % 2, w = mt / 2, pick = mt % 2 ? 0x7362 : 0x5140;
        const uint32_t x = __byte_perm(vr[i][0][w], vr[i][1][w], pick);
        const uint32_t y = __byte_perm(vr[i][2][w], vr[i][3][w], pick);
        const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_hi_to_f16x2(x);
        const uint32_t a2 = e4m3x2_to_f16x2(y), a3 = e4m3x2_hi_to_f16x2(y);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (SPLIT) {
            if (i == 0) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
            mma_16816(part[n], a0, a1, a2, a3, pl[n][i][0], pl[n][i][1]);
            mma_16816(part[n], a0, a1, a2, a3, ph[n][i][0], ph[n][i][1]);
            if (i == 1)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[n][mt][k] += part[n][k];
          } else {
            mma_16816(o[n][mt], a0, a1, a2, a3, ph[n][i][0], ph[n][i][1]);
          }
        }
      }
      // the step's bytes are in registers: its place takes unit u + S
      __syncwarp();
      issue(st, u + S);
      note(st, u + S);
      return true;
    };
    bool ok = true;
    int place = 0;                                 // in the queue
    for (int u = u0; ok && u < u1; ++u) {
      ok = body(place, u);
      place = place + 1 == S ? 0 : place + 1;
    }
    // the steps behind the last unit, empty but for their barriers' phases;
    // after a wait that ran out, what is still in flight
    if (!ok) {
      volatile int none = 0;
#pragma unroll
      for (int s = 0; s < S; ++s) mbar_wait(&bars[s], (phases >> s) & 1, &none, c.err);
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        mbar_wait(&bars[s], (phases >> s) & 1, abort_flag, c.err);
        phases ^= 1u << s;
      }
    }
    __syncthreads();
    if (*abort_flag) return;                       // the error word says why

    // the four warps' shares of the keys
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
        const int col = 8 * n + 2 * t4 + j;
        const bool high = xo[n][j] > FROM;
        if (g == 0) { s_m[warp][col] = m[n][j]; s_l[warp][col] = high ? -l[n][j] : l[n][j]; }
        const float unit = pow2_any((int)xo[n][j] - (high ? HIGH : 0));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(&s_o[warp][col][v_dim + 2 * i]) = make_float2(o[n][i][j] * unit, o[n][i][2 + j] * unit);
      }
    }
    __syncthreads();
    auto write = [&](int col, int x, const float4& a, bool high, float mt, float lt) {
      int t, gg;
      if (!row_of(col, t, gg)) return;
      const long long row = ((long long)b * p.Hq + h * G + gg) * p.T + t;
      const float inv = lt == 0.f ? 0.f : (high ? FROM_HIGH : 1.f) / lt;
      if (p.out_bf16) {
        __nv_bfloat162 z[2] = {__floats2bfloat162_rn(a.x * inv, a.y * inv), __floats2bfloat162_rn(a.z * inv, a.w * inv)};
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + x) = *reinterpret_cast<uint2*>(z);
      } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + row * D + x) =
            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      }
      if (x == 0 && p.lse) p.lse[row] = lt == 0.f ? -INFINITY : fmaf(mt - P_BIAS, 0.69314718f, logf(lt));
    };
    const bool whole = u0 == 0 && u1 == units;
    float* part = reinterpret_cast<float*>(p.part + Slot<D, NT>::counters(gridDim.x));
    float* slot = part + (size_t)(blockIdx.x * 2 + (at == begin ? 0 : 1)) * Slot<D, NT>::FLOATS;
    for (int i = threadIdx.x; i < R * (D / 4); i += 32 * NW) {
      const int col = i / (D / 4), x = i % (D / 4) * 4;
      float mt = s_m[0][col];
#pragma unroll
      for (int w = 1; w < NW; ++w) mt = fmaxf(mt, s_m[w][col]);
      float lt = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      bool high = false;
#pragma unroll
      for (int w = 0; w < NW; ++w) high = high || s_l[w][col] < 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        float f = s_m[w][col] == mt ? 1.f : ex2_approx(s_m[w][col] - mt);
        const float4 y = *reinterpret_cast<const float4*>(&s_o[w][col][x]);
        const float lw = s_l[w][col];
        lt = fmaf(f, fabsf(lw), lt);
        if (high && !(lw < 0.f)) f *= TO_HIGH;
        a.x = fmaf(f, y.x, a.x); a.y = fmaf(f, y.y, a.y); a.z = fmaf(f, y.z, a.z); a.w = fmaf(f, y.w, a.w);
      }
      if (whole) {
        write(col, x, a, high, mt, lt);
      } else {
        *reinterpret_cast<float4*>(slot + col * D + x) = a;
        if (x == 0) { slot[R * D + col] = mt; slot[R * D + R + col] = high ? -lt : lt; }
      }
    }
    __syncthreads();
    if (!whole) {
      if (threadIdx.x == 0) {
        // the barrier above and the release here order the CTA's slot before
        // its arrival, the acquire the others' slots before the join
        unsigned long long* word = reinterpret_cast<unsigned long long*>(p.part) + c0;
        s_misc[1] = marked_arrive(word, (unsigned)n);
      }
      __syncthreads();
      if (s_misc[1]) {
        auto slot_of = [&](int i) -> const float* {
          return part + (size_t)((c0 + i) * 2 + (i == 0 ? odd : 0)) * Slot<D, NT>::FLOATS;
        };
        // 128 threads: D / 4 of them a row, four dimensions each, sixteen slots
        // with their maxima and sums in flight at once
        for (int j = threadIdx.x; j < R * (D / 4); j += 32 * NW) {
          const int col = j / (D / 4), x = j % (D / 4) * 4;
          int t, gg;
          if (!row_of(col, t, gg)) continue;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          float mt = -INFINITY, lt = 0.f;
          bool high = false;
          for (int i0 = 0; i0 < n; i0 += 16) {
            float4 y[16];
            float mi[16], li[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              mi[i] = -INFINITY;
              li[i] = 0.f;
              if (i0 + i < n) {
                const float* from = slot_of(i0 + i);
                y[i] = __ldcg(reinterpret_cast<const float4*>(from + col * D + x));
                mi[i] = __ldcg(from + R * D + col);
                li[i] = __ldcg(from + R * D + R + col);
              }
            }
            float mx = mt;
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, mi[i]);
            float back = mx == mt ? 1.f : ex2_approx(mt - mx);
            mt = mx;
            lt *= back;
            const bool was = high;
#pragma unroll
            for (int i = 0; i < 16; ++i) high = high || li[i] < 0.f;
            if (high && !was) back *= TO_HIGH;
            a.x *= back; a.y *= back; a.z *= back; a.w *= back;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float f = mi[i] == mx ? 1.f : ex2_approx(mi[i] - mx);
              lt = fmaf(f, fabsf(li[i]), lt);
              if (high && !(li[i] < 0.f)) f *= TO_HIGH;
              a.x = fmaf(f, y[i].x, a.x); a.y = fmaf(f, y[i].y, a.y);
              a.z = fmaf(f, y[i].z, a.z); a.w = fmaf(f, y[i].w, a.w);
            }
          }
          write(col, x, a, high, mt, lt);
        }
      }
    }
    // the merge buffer makes room for the next row block's boxes
    fence_proxy_async_smem();
    __syncthreads();
    at += cut ? 1 : u1 - u0;
  }
}

// CTAs of the fixed grid: the GPU's, or fewer where the cache's capacity gives
// fewer units.
int grid_of(const Line& ln, int B, int d, int n_sel, int page, int max_pages) {
  const long long all = (long long)units_of((long long)(n_sel > 0 ? n_sel : max_pages) * page) * ln.nb * B;
  if (all >= (1LL << 31)) return 0;                // more than the line's 32 bits count
  const long long most = (long long)kSMs * ctas_per_sm(d, ln.R / 8);
  return (int)(all < most ? all : most);
}

template <int D, int NT, bool SPLIT>
cudaError_t launch(const CacheFwdParams& p, int grid, cudaStream_t st) {
  constexpr int smem = Queue<D, NT>::SMEM;
  auto k = p.c.page == 16 ? cache_fwd_kernel<D, NT, SPLIT, true> : cache_fwd_kernel<D, NT, SPLIT, false>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_next(k, dim3((unsigned)grid), 32 * NW, smem, st, p);
}

}  // namespace

static bool many_rows(int Hq, int Hkv, int T) {
  return (long long)(Hq / Hkv) * T > MANY_ROWS;
}

size_t cache_fwd_workspace(int B, int Hq, int Hkv, int T, int d, int n_sel, int page, int max_pages) {
  const Line ln = make_line(Hq, Hkv, T, n_sel > 0);
  const size_t slot = (size_t)ln.R * (d + 2) * 4;
  const size_t grid = (size_t)grid_of(ln, B, d, n_sel, page, max_pages);
  if (!grid) return 0;
  const size_t few = Slot<64, 1>::counters((unsigned)grid) + 2 * slot * grid;
  // either, as the output's type decides
  const size_t many = n_sel == 0 && many_rows(Hq, Hkv, T) ? cache_chunk_workspace(B, Hq, Hkv, T, d, page, max_pages) : 0;
  return many > few ? many : few;
}

cudaError_t launch_cache_fwd(const CacheFwdParams& p, cudaStream_t st) {
  if (!p.pages && p.out_bf16 && many_rows(p.Hq, p.c.Hkv, p.T)) return launch_cache_chunk(p, st);
  const Line ln = make_line(p.Hq, p.c.Hkv, p.T, p.pages != nullptr);
  const int grid = grid_of(ln, p.c.B, p.c.d, p.pages ? p.n_sel : 0, p.c.page, p.c.max_pages);
  if (grid == 0) return cudaErrorInvalidValue;
  const bool split = !p.out_bf16;
#define FA4_CASE(D, NT, S) \
  if (p.c.d == D && ln.R == 8 * NT && split == S) return launch<D, NT, S>(p, grid, st);
  FA4_CASE(64, 1, false) FA4_CASE(64, 1, true) FA4_CASE(64, 2, false) FA4_CASE(64, 2, true)
  FA4_CASE(128, 1, false) FA4_CASE(128, 1, true) FA4_CASE(128, 2, false) FA4_CASE(128, 2, true)
#undef FA4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa4
