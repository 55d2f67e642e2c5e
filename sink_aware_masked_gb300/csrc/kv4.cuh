// The 4-bit paged key/value cache: layout, addressing and conversions shared
// by its kernels (include/sinkattn.h describes the format).
//
// A block holds 16 tokens of one head, 1152 bytes, in the order in which the
// lanes of a warp use it as m16n8k16 matrix fragments (lane = 4 g + t,
// g = 0..7, t = 0..3), so that every access of a whole block is one
// contiguous 512-byte (codes) or 64-byte (scales) access of the warp:
//   keys    lane: tokens g and g + 8, dims 16 t .. 16 t + 15 (one scale each)
//   values  lane: tokens 2t, 2t+1, 2t+8, 2t+9, dims 8 g .. 8 g + 7
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace kv4 {

constexpr int kBlockTokens = 16;
constexpr int kBlockBytes = 1152;
constexpr int kVCodes = 512, kKScales = 1024, kVScales = 1088;
constexpr uint8_t kNaNScale = 0x7f;

SA_DEV int lane_g() { return (threadIdx.x & 31) >> 2; }
SA_DEV int lane_t() { return threadIdx.x & 3; }

// Length of a slot; 0 for a slot number outside the cache (an idle entry).
SA_DEV int slot_len(const Kv4Cache& c, int slot) {
  if (slot < 0 || slot >= c.num_slots) return 0;
  return max(c.seqlens[slot], 0);
}

// Page that holds block `blk` of a slot, or -1 where the table has none.
SA_DEV int page_of(const Kv4Cache& c, int slot, int blk) {
  const int col = blk >> c.blocks_log2;
  if (col >= c.max_pages) return -1;
  const int p = c.page_table[static_cast<int64_t>(slot) * c.max_pages + col];
  return (p >= 0 && p < c.num_pages) ? p : -1;
}

SA_DEV uint8_t* block_ptr(const Kv4Cache& c, int page, int head, int blk) {
  const int in_page = blk & ((1 << c.blocks_log2) - 1);
  return c.pages + ((((static_cast<int64_t>(page) * c.num_heads_kv + head) << c.blocks_log2) + in_page) * kBlockBytes);
}

// Two e2m1 codes (low nibble first) in each byte of w -> four f16 pairs, exactly.
SA_DEV void e2m1x8(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}

// Two e4m3 scales -> a pair of f16, exactly (NaN stays NaN).
SA_DEV uint32_t e4m3x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

SA_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Whether a byte of four e4m3 scales is NaN.
SA_DEV bool any_nan_scale(uint32_t four) { return (((four & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

SA_DEV float2 f16x2_to_f32(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Words of two tokens (8 dims each, one nibble per dim) -> bytes that hold the
// two tokens' codes of one dim: `even` the dims 0, 2, 4, 6, `odd` the others.
SA_DEV void pair_tokens(uint32_t a, uint32_t b, uint32_t& even, uint32_t& odd) {
  even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
  odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}

}  // namespace kv4
}  // namespace sa
