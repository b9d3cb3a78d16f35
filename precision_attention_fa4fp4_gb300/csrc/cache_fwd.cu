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
// the workspace for the second kernel, which joins them in a fixed order.
//
// Inside a CTA four warps take 32 keys each of every unit and keep their own
// running max and sum; they meet once, at the end of a share.
//
// Products: m16n8k16 with the keys as rows, so that eight queries fill the
// instruction: S^T = K Q^T, O^T += V^T P.  The 8-bit rows go from global
// memory into registers and are the A operand after one conversion (E4M3 ->
// f16 is exact): no shared memory, no barrier in the loop.  For V^T the two
// keys of an operand pair are interleaved with a byte permute.  The codes are
// used unscaled: K's page scale multiplies the scores, V's page scale
// multiplies the FP32 sum of the page's products.
//
// Roundings: q to f16 under a power of two (2^-32 of the row's largest), P to
// f16 under a factor 2^15 (half a step is 2^-12, and values keep it down to
// 2^-29), or for FP32 output P as a sum of two f16 (2^-23).  The normalizer
// sums the FP32 values of P.
#include "cache.cuh"

namespace fa4 {
namespace {

constexpr int NW = 4;                 // warps of a CTA
constexpr int UNIT = 32 * NW;         // keys of a unit
constexpr int kSMs = 152;             // GB300
constexpr float P_BIAS = 15.f;        // log2 of the factor on P

constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

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

// Units of one row block of a sequence of n tokens (at least one, which writes
// the output of a row without keys).
FA4_DEV int units_of(int n, int q_len, int n_sel, int page) {
  long long keys = q_len > 0 ? n : 0;
  // a list may name its pages in any order, with holes
  if (n_sel > 0 && keys > 0) keys = (long long)n_sel * page;
  return max(1, (int)((keys + UNIT - 1) / UNIT));
}

FA4_DEV int seq_units(const CacheFwdParams& p, int b) {
  return units_of(cache_len(p.c, b), cache_count(p.q_lens, b, p.T, p.c.err), p.pages ? p.n_sel : 0, p.c.page);
}

// Units of the sequences before `b` and of all sequences (whole warp).
FA4_DEV void scan_units(const CacheFwdParams& p, int b, long long& before, long long& total) {
  long long lo = 0, all = 0;
  for (int i = threadIdx.x % 32; i < p.c.B; i += 32) {
    const int u = seq_units(p, i);
    all += u;
    if (i < b) lo += u;
  }
#pragma unroll
  for (int o = 16; o; o /= 2) {
    lo += __shfl_xor_sync(0xffffffffu, lo, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  before = lo;
  total = all;
}

// CTAs that get a share: no more than there are units, so that no share is
// empty (the join reads every slot from the first to the last).
FA4_DEV int workers(long long total, int grid) { return (int)min((long long)grid, total); }
// First unit of CTA i's share.
FA4_DEV long long share_begin(long long total, int i, int n) { return total * i / n; }
// CTA whose share holds unit u.
FA4_DEV int share_of(long long u, long long total, int n) {
  return (int)min((long long)n - 1, ((u + 1) * n - 1) / total);
}

template <int D, int NT>
struct Slot {
  static constexpr int R = 8 * NT;
  static constexpr int FLOATS = R * D + 2 * R;     // o, then m, then l
};

template <int D, int NT, bool SPLIT, bool SMALLP>
__global__ void __launch_bounds__(32 * NW, ctas_per_sm(NT)) cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  constexpr int R = 8 * NT;
  constexpr int NP = SMALLP ? 2 : 1;               // pages of a warp's 32 keys
  constexpr int OS = D + 4;                        // row stride of the merge buffer
  constexpr int VW = D / 32;                       // 32-bit words of V a lane holds per key
  __shared__ float s_o[NW][R][OS];
  __shared__ float s_m[NW][R], s_l[NW][R];
  asm volatile("griddepcontrol.launch_dependents;");

  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t4 = lane % 4;
  const Line ln = make_line(p.Hq, c.Hkv, p.T, p.pages != nullptr);
  const int G = ln.G;
  long long before, total;
  scan_units(p, 0, before, total);
  total *= ln.nb;
  const int ctas = workers(total, gridDim.x);
  if (blockIdx.x >= ctas) return;
  long long at = share_begin(total, blockIdx.x, ctas);
  const long long begin = at, end = share_begin(total, blockIdx.x + 1, ctas);
  // the sequence that holds unit `at`
  int b = 0, units = 1;
  long long seq0 = 0;                              // its first unit
  for (int base = 0;; base += 32) {
    const int i = base + lane;
    const long long mine = i < c.B ? (long long)seq_units(p, i) * ln.nb : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, seq0 + inc > at);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = base + src;
      seq0 += __shfl_sync(0xffffffffu, inc - mine, src);
      break;
    }
    seq0 += __shfl_sync(0xffffffffu, inc, 31);
    if (base + 32 >= c.B) return;                  // cannot happen: at < total
  }
  units = seq_units(p, b);

  while (at < end) {
    while (at >= seq0 + (long long)units * ln.nb) {
      seq0 += (long long)units * ln.nb;
      units = seq_units(p, ++b);
    }
    const int rb = (int)((at - seq0) / units);     // row block of the sequence
    const int u0 = (int)((at - seq0) % units);
    const int u1 = (int)min((long long)units, u0 + (end - at));
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

    QFrag<D> q[NT];
    float fx[NT][2];                               // log2-unit factor of columns 2 t4, 2 t4 + 1
    int vis[NT][2];                                // keys they see
    int vis_min = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      int t, gg;
      const bool ok = row_of(8 * n + g, t, gg);
      const __nv_bfloat16* row = ok ? reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                          (((long long)b * p.Hq + h * G + gg) * p.T + t) * D
                                    : nullptr;
      const float e = load_qfrag<D>(q[n], row, t4);
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
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    // Pool offset (in tokens) and first key position of the warp's keys of a
    // unit; keys that are not there get a position that every query masks.
    auto lookup = [&](int u, long long (&tok)[NP], int (&pos)[NP]) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int v = u * UNIT + 32 * warp + 16 * i;
        const int j = v / c.page, off = v % c.page;
        int lp = j;
        if (sel) {
          lp = j < p.n_sel ? __ldg(sel + j) : -1;
          if (lp >= c.max_pages || lp < -1) { atomicOr(c.err, FA4_DEVERR_INDEX); lp = -1; }
        }
        int pg = -1;
        if (u < u1 && lp >= 0 && (long long)lp * c.page < len) pg = cache_page(c, c.table, b, lp);
        pos[i] = pg >= 0 ? lp * c.page + off : 0x40000000;
        tok[i] = ((long long)max(pg, 0) * c.Hkv + h) * c.page + off;
      }
    };
    uint4 kr[2][2][D / 64];
    uint32_t vr[2][4][VW];
    float kx[NP], vx[NP];
    auto load_k = [&](const long long (&tok)[NP]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const long long t = SMALLP ? tok[i % NP] : tok[0] + 16 * i;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            kr[i][r][k] = __ldg(reinterpret_cast<const uint4*>(c.k + (t + g + 8 * r) * D + 64 * k + 16 * t4));
      }
    };
    auto load_v = [&](const long long (&tok)[NP]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const long long t = SMALLP ? tok[i % NP] : tok[0] + 16 * i;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* a = c.v + (t + 2 * t4 + (k & 1) + 8 * (k >> 1)) * D + (D / 8) * g;
          if constexpr (VW == 4) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(a));
            vr[i][k][0] = x.x; vr[i][k][1] = x.y; vr[i][k][2] = x.z; vr[i][k][3] = x.w;
          } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(a));
            vr[i][k][0] = x.x; vr[i][k][1] = x.y;
          }
        }
      }
    };
    auto load_x = [&](const long long (&tok)[NP]) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const long long ph = tok[i] / c.page;
        kx[i] = e8m0_value(__ldg(c.ks + ph));
        vx[i] = e8m0_value(__ldg(c.vs + ph));
      }
    };

    long long tok[NP], tok_n[NP];
    int pos[NP], pos_n[NP];
    lookup(u0, tok, pos);
    load_k(tok);
    load_x(tok);
    load_v(tok);
    lookup(u0 + 1, tok_n, pos_n);
    for (int u = u0; u < u1; ++u) {
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
          const uint32_t lo[4] = {kr[i][0][k].x, kr[i][0][k].y, kr[i][0][k].z, kr[i][0][k].w};
          const uint32_t hi[4] = {kr[i][1][k].x, kr[i][1][k].y, kr[i][1][k].z, kr[i][1][k].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = e4m3x2_to_f16x2(lo[w]), a2 = e4m3x2_hi_to_f16x2(lo[w]);
            const uint32_t a1 = e4m3x2_to_f16x2(hi[w]), a3 = e4m3x2_hi_to_f16x2(hi[w]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816(s[n][i], a0, a1, a2, a3, q[n].b[4 * k + w][0], q[n].b[4 * k + w][1]);
          }
        }
      float kxc[NP], vxc[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) { kxc[i] = kx[i]; vxc[i] = vx[i]; }
      const bool more = u + 1 < u1;
      if (more) {
        load_k(tok_n);
        load_x(tok_n);
      }
      bool full = true;
#pragma unroll
      for (int i = 0; i < NP; ++i) full = full && pos[i] + 32 / NP <= vis_min;

      uint32_t ph[NT][2][2], pl[NT][2][2];         // P^T as the B operand: [16 keys][k half]
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mx[2] = {m[n][0], m[n][1]};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = s[n][i][j] * kxc[i % NP] * fx[n][j & 1];
            if (!full) {
              const int key = pos[i % NP] + (SMALLP ? 0 : 16 * i) + g + 8 * (j >> 1);
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
        // nothing seen yet: any finite reference will do, the masked scores
        // stay -inf
        const float r0 = (m[n][0] == -INFINITY ? 0.f : m[n][0]) - P_BIAS;
        const float r1 = (m[n][1] == -INFINITY ? 0.f : m[n][1]) - P_BIAS;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = ex2_approx(s[n][i][j] - ((j & 1) ? r1 : r0));
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
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
      // keys past the sequence's end hold anything: 0 * NaN must not happen
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = pos[i % NP] + (SMALLP ? 0 : 16 * i) + 2 * t4 + (k & 1) + 8 * (k >> 1);
            if (key >= len)
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[i][k][w] = 0;
          }
      }
      // O^T += V^T P: lane rows (D / 8) g + 2 mt and + 1 of the head dimension
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int mt = 2 * w + half;
          float acc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = __byte_perm(vr[i][0][w], vr[i][1][w], half ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(vr[i][2][w], vr[i][3][w], half ? 0x7362 : 0x5140);
            const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_hi_to_f16x2(x);
            const uint32_t a2 = e4m3x2_to_f16x2(y), a3 = e4m3x2_hi_to_f16x2(y);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_16816(acc[n], a0, a1, a2, a3, ph[n][i][0], ph[n][i][1]);
              if constexpr (SPLIT) mma_16816(acc[n], a0, a1, a2, a3, pl[n][i][0], pl[n][i][1]);
            }
            if (SMALLP || i == 1) {
              const float x2 = vxc[i % NP];
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  o[n][mt][j] = fmaf(acc[n][j], x2, o[n][mt][j]);
                  acc[n][j] = 0.f;
                }
            }
          }
        }
      if (more) {
        load_v(tok_n);
#pragma unroll
        for (int i = 0; i < NP; ++i) { tok[i] = tok_n[i]; pos[i] = pos_n[i]; }
        lookup(u + 2, tok_n, pos_n);
      }
    }

    // the four warps' shares of the keys
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
        const int col = 8 * n + 2 * t4 + j;
        if (g == 0) { s_m[warp][col] = m[n][j]; s_l[warp][col] = l[n][j]; }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(&s_o[warp][col][(D / 8) * g + 2 * i]) = make_float2(o[n][i][j], o[n][i][2 + j]);
      }
    }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;
    float* slot = p.part + ((long long)blockIdx.x * 2 + (at == begin ? 0 : 1)) * Slot<D, NT>::FLOATS;
    for (int i = threadIdx.x; i < R * (D / 4); i += 32 * NW) {
      const int col = i / (D / 4), x = i % (D / 4) * 4;
      float mt = s_m[0][col];
#pragma unroll
      for (int w = 1; w < NW; ++w) mt = fmaxf(mt, s_m[w][col]);
      float lt = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = s_m[w][col] == mt ? 1.f : ex2_approx(s_m[w][col] - mt);
        const float4 y = *reinterpret_cast<const float4*>(&s_o[w][col][x]);
        lt = fmaf(f, s_l[w][col], lt);
        a.x = fmaf(f, y.x, a.x); a.y = fmaf(f, y.y, a.y); a.z = fmaf(f, y.z, a.z); a.w = fmaf(f, y.w, a.w);
      }
      if (!whole) {
        *reinterpret_cast<float4*>(slot + col * D + x) = a;
        if (x == 0) { slot[R * D + col] = mt; slot[R * D + R + col] = lt; }
        continue;
      }
      int t, gg;
      if (!row_of(col, t, gg)) continue;
      const long long row = ((long long)b * p.Hq + h * G + gg) * p.T + t;
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      if (p.out_bf16) {
        __nv_bfloat162 z[2] = {__floats2bfloat162_rn(a.x * inv, a.y * inv), __floats2bfloat162_rn(a.z * inv, a.w * inv)};
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + x) = *reinterpret_cast<uint2*>(z);
      } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + row * D + x) =
            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      }
      if (x == 0 && p.lse) p.lse[row] = lt == 0.f ? -INFINITY : fmaf(mt - P_BIAS, 0.69314718f, logf(lt));
    }
    __syncthreads();
    at += u1 - u0;
  }
}

// Joins the partials of every row block that more than one CTA worked on: one
// CTA per row block, one warp per row, a lane holding D / 32 dimensions.
template <int D, int NT>
__global__ void __launch_bounds__(32 * 8 * NT) cache_join_kernel(const __grid_constant__ CacheFwdParams p, int grid) {
  constexpr int R = 8 * NT;
  constexpr int E = D / 32;
  const CacheView& c = p.c;
  const Line ln = make_line(p.Hq, c.Hkv, p.T, p.pages != nullptr);
  const int b = blockIdx.x / ln.nb, rb = blockIdx.x % ln.nb;
  const int lane = threadIdx.x % 32, col = threadIdx.x / 32;
  long long before, total;
  scan_units(p, b, before, total);
  total *= ln.nb;
  const int ctas = workers(total, grid);
  const int units = seq_units(p, b);
  const long long start = before * ln.nb + (long long)rb * units;
  const int c0 = share_of(start, total, ctas), c1 = share_of(start + units - 1, total, ctas);
  if (c0 == c1) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = rb / ln.per_head, sub = rb % ln.per_head;
  const int q_len = cache_count(p.q_lens, b, p.T, c.err);
  int t, gg;
  if (p.pages) { t = sub / ln.QG; gg = (sub % ln.QG) * R + col; }
  else { const int r = sub * R + col; t = r / ln.G; gg = r % ln.G; }
  if (gg >= ln.G || t >= q_len) return;
  const int n = c1 - c0 + 1;
  auto slot = [&](int i) -> const float* {
    const int cta = c0 + i;
    return p.part + ((long long)cta * 2 + (share_begin(total, cta, ctas) >= start ? 0 : 1)) * Slot<D, NT>::FLOATS;
  };
  float mt = -INFINITY;
  for (int i = lane; i < n; i += 32) mt = fmaxf(mt, slot(i)[R * D + col]);
#pragma unroll
  for (int o = 16; o; o /= 2) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
  float lt = 0.f, a[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* s = slot(i);
    const float mi = s[R * D + col];
    const float f = mi == mt ? 1.f : ex2_approx(mi - mt);
    lt = fmaf(f, s[R * D + R + col], lt);
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = fmaf(f, s[col * D + lane * E + e], a[e]);
  }
  const long long row = ((long long)b * p.Hq + h * ln.G + gg) * p.T + t;
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const long long i = row * D + lane * E + e;
    if (p.out_bf16)
      *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(p.o) + i) =
          __floats2bfloat162_rn(a[e] * inv, a[e + 1] * inv);
    else
      *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.o) + i) = make_float2(a[e] * inv, a[e + 1] * inv);
  }
  if (lane == 0 && p.lse) p.lse[row] = lt == 0.f ? -INFINITY : fmaf(mt - P_BIAS, 0.69314718f, logf(lt));
}

// CTAs of the fixed grid: the GPU's, or fewer where the cache's capacity gives
// fewer units.
int grid_of(const Line& ln, int B, int n_sel, int page, int max_pages) {
  const long long keys = (long long)(n_sel > 0 ? n_sel : max_pages) * page;
  long long units = (keys + UNIT - 1) / UNIT;
  if (units < 1) units = 1;
  const long long all = units * ln.nb * B;
  const long long most = (long long)kSMs * ctas_per_sm(ln.R / 8);
  return (int)(all < most ? all : most);
}

template <int D, int NT, bool SPLIT>
cudaError_t launch(const CacheFwdParams& p, const Line& ln, int grid, cudaStream_t st) {
  if (p.c.page == 16) cache_fwd_kernel<D, NT, SPLIT, true><<<grid, 32 * NW, 0, st>>>(p);
  else cache_fwd_kernel<D, NT, SPLIT, false><<<grid, 32 * NW, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ln.nb * p.c.B));
  cfg.blockDim = dim3(32 * 8 * NT);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, NT>, p, grid);
}

}  // namespace

size_t cache_fwd_workspace(int B, int Hq, int Hkv, int T, int d, int n_sel, int page, int max_pages) {
  const Line ln = make_line(Hq, Hkv, T, n_sel > 0);
  const size_t slot = (size_t)ln.R * (d + 2) * 4;
  return 2 * slot * (size_t)grid_of(ln, B, n_sel, page, max_pages);
}

cudaError_t launch_cache_fwd(const CacheFwdParams& p, cudaStream_t st) {
  const Line ln = make_line(p.Hq, p.c.Hkv, p.T, p.pages != nullptr);
  const int grid = grid_of(ln, p.c.B, p.pages ? p.n_sel : 0, p.c.page, p.c.max_pages);
  const bool split = !p.out_bf16;
#define FA4_CASE(D, NT, S) \
  if (p.c.d == D && ln.R == 8 * NT && split == S) return launch<D, NT, S>(p, ln, grid, st);
  FA4_CASE(64, 1, false) FA4_CASE(64, 1, true) FA4_CASE(64, 2, false) FA4_CASE(64, 2, true)
  FA4_CASE(128, 1, false) FA4_CASE(128, 1, true) FA4_CASE(128, 2, false) FA4_CASE(128, 2, true)
#undef FA4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fa4
