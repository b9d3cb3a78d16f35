// cross.cuh -- device routines that the cross attention kernels share.
#pragma once
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.h"

namespace fa4 {

// Row (b, h, n) of a strided tensor.
FA4_DEV __nv_bfloat16* at(const Strided& t, int b, int h, int n) {
  return static_cast<__nv_bfloat16*>(t.p) + b * t.b + h * t.h + n * t.n;
}

// Keys of sequence b; a length outside 0 .. Nk is reported and taken as the nearer
// end.
FA4_DEV int key_count(const CrossParams& p, int b, bool report = true) {
  if (!p.lens) return p.Nk;
  const int len = p.lens[b];
  if (len >= 0 && len <= p.Nk) return len;
  if (report) atomicOr(p.err, FA4_DEVERR_INDEX);
  return len < 0 ? 0 : p.Nk;
}

// A box at channel c, row n, head h, sequence b.
FA4_DEV void tma_heads(void* dst, const HeadsMap& m, uint64_t* bar, int c, int n, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(smem_u32(bar)), "r"(c), "r"(n), "r"(h * m.own_h), "r"(b * m.own_b)
      : "memory");
}

// x . row, x in shared memory.
template <int D>
FA4_DEV float dot(const float* x, const __nv_bfloat16* row) {
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < D; i += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(x[i + 2 * e], __uint_as_float(w[e] << 16), s);
      s = fmaf(x[i + 2 * e + 1], __uint_as_float(w[e] & 0xffff0000u), s);
    }
  }
  return s;
}

}  // namespace fa4
