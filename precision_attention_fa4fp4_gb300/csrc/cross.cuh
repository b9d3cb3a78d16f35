// cross.cuh -- device routines that the cross attention kernels share.
#pragma once
#include <cuda_bf16.h>
#include "common.cuh"
#include "cross.h"
#include "divide.cuh"

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

// lse of a row whose weights 2^(c s - ref) add up to l; ref holds `down` (0 to 126), which is taken out of both before
// the logarithm: what little l differs from 2^-down by is not rounded away beside it.
FA4_DEV float lse_of(float ref, float l, int down) {
  return ((ref - (float)down) + log2f(l * __uint_as_float((uint32_t)(127 + down) << 23))) * 0.69314718055994531f;
}

// A box at channel c, row n, head h, sequence b.
FA4_DEV void tma_heads(void* dst, const HeadsMap& m, uint64_t* bar, int c, int n, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(smem_u32(bar)), "r"(c), "r"(n), "r"(h * m.own_h), "r"(b * m.own_b)
      : "memory");
}

// A box of a group_map at channel c, row n, head g of kv head hk, sequence b.
FA4_DEV void tma_group(void* dst, const HeadsMap& m, uint64_t* bar, int c, int n, int g, int hk, int b) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(smem_u32(bar)), "r"(c), "r"(n), "r"(g), "r"(hk), "r"(b * m.own_b)
      : "memory");
}

// A box from shared memory, by one lane; rows behind the tensor's are left out.
FA4_DEV void tma_heads_store(const HeadsMap& m, const void* src, int c, int n, int h, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(&m.map)),
               "r"(smem_u32(src)), "r"(c), "r"(n), "r"(h * m.own_h), "r"(b * m.own_b)
               : "memory");
}

// 16-byte word x (of D / 8) of a row of a tile.
FA4_DEV uint4* tile_word(uint8_t* tile, int r, int x) {
  return reinterpret_cast<uint4*>(tile + x / 8 * (128 * 128) + r * 128 + ((x % 8) ^ (r & 7)) * 16);
}

// ---------------------------------------------------------------- products
// Tiles are [128 rows][64 channels] of bf16 with the 128-byte swizzle, D / 64 of
// them.  Their descriptors differ in the low word alone (address, leading
// offset): one add for each instruction, which costs the issuing lane 33 cycles
// instead of 42 with descriptors formed in full.
constexpr int CH = 128 * 128;                // bytes of 64 channels of 128 rows
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | ((uint32_t)SW_128B << 29);
FA4_DEV uint32_t desc_rows(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }              // rows x channels
FA4_DEV uint32_t desc_cols(uint32_t saddr) { return (saddr >> 4) | ((uint32_t)(CH >> 4) << 16); }   // channels x rows

FA4_DEV void mma_ss(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n"
      " mov.b64 db, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(acc),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(DESC_HI)
      : "memory");
}
FA4_DEV void mma_ts(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(acc),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(DESC_HI)
      : "memory");
}
// acc = A B^T over D channels, both tiles in shared memory.
template <int D>
FA4_DEV void product_rows(uint32_t acc, uint32_t sa, uint32_t sb, uint32_t idesc) {
  const uint32_t a = desc_rows(sa), b = desc_rows(sb);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = ((k / 4) * CH + (k % 4) * 32) >> 4;
    mma_ss(acc, a + off, b + off, idesc, k > 0);
  }
}
// acc (+)= A B over B's 128 rows, A packed in tensor memory.
FA4_DEV void product_cols(uint32_t acc, uint32_t a, uint32_t sb, uint32_t idesc, bool add) {
  const uint32_t b = desc_cols(sb);
#pragma unroll
  for (int k = 0; k < 8; ++k) mma_ts(acc, a + 8 * k, b + k * 128, idesc, add || k > 0);
}
// Half of that product: the first or the last 32 of A's columns from a0 and from a1
// (64 columns, packed, each).
FA4_DEV void product_half(uint32_t acc, uint32_t a0, uint32_t a1, uint32_t sb, uint32_t idesc, int part, bool add) {
  const uint32_t b = desc_cols(sb);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 2 * part + i % 2;
    mma_ts(acc, (i < 2 ? a0 : a1) + 8 * k, b + (i / 2 * 4 + k) * 128, idesc, add || i > 0);
  }
}

// Rows [keep, 128) of a tile to zeros (one warp).
template <int D>
FA4_DEV void clear_rows(uint8_t* tile, int keep, int lane) {
  for (int c = 0; c < D / 64; ++c)
    for (int i = keep * 8 + lane; i < 128 * 8; i += 32)
      reinterpret_cast<uint4*>(tile + c * CH)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace fa4
