// cache.cuh -- device routines shared by the 8-bit cache kernels: bounds-checked
// page lookups, E4M3 <-> f16 conversion and the register layouts in which the
// m16n8k16 products read 8-bit rows straight from global memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "cache.h"
#include "common.cuh"

namespace fa4 {

// Every kernel of the cache may be launched while the one before it in the
// stream still runs (launch_next below).  It lets its own successor start right
// away, and waits here, in every thread and before it touches global memory, for
// everything before it; so the order of the stream holds however many calls
// follow each other.  What other calls write is read by plain loads: a
// non-coherent load would need it unchanged from the kernel's start.
FA4_DEV void grid_start() { asm volatile("griddepcontrol.launch_dependents;"); }
FA4_DEV void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Length of sequence b: a value outside [0, capacity] is flagged and clamped.
FA4_DEV int cache_len(const CacheView& c, int b) {
  const int n = *(c.lens + b);
  const long long cap = (long long)c.max_pages * c.page;
  if (n < 0 || n > cap) {
    atomicOr(c.err, FA4_DEVERR_INDEX);
    return n < 0 ? 0 : (int)cap;
  }
  return n;
}

// A per-sequence count in [0, most] (nullptr: most), flagged and clamped.
FA4_DEV int cache_count(const int* n, int b, int most, unsigned* err) {
  if (!n) return most;
  const int x = *(n + b);
  if (x < 0 || x > most) {
    atomicOr(err, FA4_DEVERR_INDEX);
    return x < 0 ? 0 : most;
  }
  return x;
}

// Pool page of a sequence's page lp in [0, max_pages): -1 (flagged) where the
// table's entry is no page of the pool.
FA4_DEV int cache_page(const CacheView& c, const int* table, int b, int lp) {
  const int p = *(table + (long long)b * c.max_pages + lp);
  if (p < 0 || p >= c.num_pages) {
    atomicOr(c.err, FA4_DEVERR_INDEX);
    return -1;
  }
  return p;
}

// 2^(byte - 127) of an E8M0 scale byte; byte 0 is the subnormal 2^-127.
FA4_DEV float e8m0_value(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x400000u); }

// Two E4M3 codes (low 16 bits) to two f16 values, exactly.
FA4_DEV uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n mov.b32 {t, _}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
// ... the high 16 bits
FA4_DEV uint32_t e4m3x2_hi_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n mov.b32 {_, t}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
  return r;
}

// Value of one E4M3 code.
FA4_DEV float e4m3_value(uint32_t code) {
  return __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(code) & 0xffffu)));
}

// D(16x8) += A(16x16, row) B(16x8, col), f16 operands, FP32 accumulators.
// Lane (g = lane / 4, t = lane % 4): A rows g, g + 8 at k = 2t.. and 2t + 8..;
// B column g at the same k; D rows g, g + 8 at columns 2t, 2t + 1.
FA4_DEV void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Raises the bytes that the current phase of an mbarrier waits for, before the
// arrival that lets the phase end.
FA4_DEV void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Bytes from p to the next multiple of 1024 (the swizzle's period).  Added to the
// array itself, so that the compiler still sees shared memory: through an
// address rounded as an integer every access became a generic one, with the
// latency of a global load.
FA4_DEV uint32_t smem_pad(const void* p) { return (0u - smem_u32(p)) & 1023u; }
FA4_DEV uint4 lds16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
FA4_DEV uint2 lds8(const void* p) { return *reinterpret_cast<const uint2*>(p); }

// Transpose of an 8x8 matrix of 16-bit values held two to a lane.
FA4_DEV uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

FA4_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ----------------------------------------------------------------------------
// Queries as the B operand.  The sum over the head dimension may run in any
// order, so its order is chosen to suit K: with K rows read as 16-byte words,
// lane t of a quad holds bytes 64 c + 16 t + (0..15) of a row for c < d / 64,
// and word w (four bytes) of it feeds step 4 c + w: k = 2t, 2t + 1 are the
// word's bytes 0, 1 and k = 2t + 8, 2t + 9 its bytes 2, 3.  The query fragment
// of step 4 c + w therefore holds dims 64 c + 16 t + 4 w + (0..3).
//
// Each query row is scaled by a power of two to a largest magnitude in
// [2^7, 2^8) before it is rounded to f16: bf16's 8 bits fit f16's 11 except
// below 2^-14, i.e. 2^-21 of the row's largest, where the rounding is at most
// 2^-25 absolute: 2^-32 of the largest.  `f` gets the power of two that undoes
// it.  An all-zero row keeps 1.
template <int D>
struct QFrag {
  uint32_t b[D / 16][2];
};

// The bf16 words of the query that a lane's column g = lane / 4 stands for, read
// ahead of their use; nullptr: a row of zeros.
template <int D>
struct QRaw {
  uint2 w[D / 16];

  FA4_DEV void fetch(const __nv_bfloat16* row, int t) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row) x = reinterpret_cast<const uint4*>(row + 64 * c + 16 * t)[i];
        w[4 * c + 2 * i] = make_uint2(x.x, x.y);
        w[4 * c + 2 * i + 1] = make_uint2(x.z, x.w);
      }
  }
  // Exponent e of the row's scale, the same in every lane of the quad.
  FA4_DEV int exponent() const {
    uint32_t amax = 0;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      amax = max(amax, max((w[s].x << 16) & 0x7fffffffu, w[s].x & 0x7fff0000u));
      amax = max(amax, max((w[s].y << 16) & 0x7fffffffu, w[s].y & 0x7fff0000u));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // E - 127 - 7 for the largest's exponent field E, within what a normal FP32
    // power of two can undo; zeros, infinities and NaN keep 0
    const int E = (int)(amax >> 23);
    return (E == 0 || E == 255) ? 0 : max(-120, min(120, E - 134));
  }
  // f16 operands of the scaled row; returns 2^e.
  FA4_DEV float convert(QFrag<D>& q) const {
    const int e = exponent();
    const float down = exp2i(-e);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      q.b[s][0] = pack_f16x2(__uint_as_float(w[s].x << 16) * down, __uint_as_float(w[s].x & 0xffff0000u) * down);
      q.b[s][1] = pack_f16x2(__uint_as_float(w[s].y << 16) * down, __uint_as_float(w[s].y & 0xffff0000u) * down);
    }
    return exp2i(e);
  }
};

FA4_DEV unsigned long long atomic_add_acq_rel(unsigned long long* p, unsigned long long x) {
  unsigned long long had;
  asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(had) : "l"(p), "l"(x) : "memory");
  return had;
}

// E4M3 codes, four to a word, as unsigned bytes in the order of their values
// (-0 just below 0), and back.
FA4_DEV uint32_t e4m3_ordered(uint32_t x) {
  const uint32_t neg = (x >> 7) & 0x01010101u;
  return x ^ (neg * 0x7fu | 0x80808080u);
}
FA4_DEV uint32_t e4m3_unordered(uint32_t x) {
  const uint32_t neg = (~x >> 7) & 0x01010101u;
  return x ^ (neg * 0x7fu | 0x80808080u);
}

// Least and greatest by 16-bit halves (one instruction each; by bytes they are
// made of several).  A half's high byte is then right whatever the low one is.
FA4_DEV uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
FA4_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The largest magnitude among codes, in two words whose high bytes hold it.
struct MaxCode {
  uint32_t odd = 0, even = 0;
  FA4_DEV void add(uint32_t x) {
    const uint32_t m = x & 0x7f7f7f7fu;
    odd = max_u16x2(odd, m);
    even = max_u16x2(even, m << 8);
  }
  FA4_DEV uint32_t halves() const { return max_u16x2(odd, even); }
  static FA4_DEV uint32_t of(uint32_t halves) { return max(halves >> 24, (halves >> 8) & 0xffu); }
};

// Launches a kernel that begins with grid_start and grid_wait.
template <class P>
cudaError_t launch_next(void (*kernel)(const P), dim3 grid, int threads, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace fa4
