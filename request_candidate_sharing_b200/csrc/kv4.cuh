// The 4-bit history cache's storage format (rocs_kv4_desc), shared by its kernels.
//
// A page holds page_size tokens of every head.  For each (page, head) there is one contiguous
// record of page_size * d_h * 9 / 8 bytes:
//   key codes    page_size rows of d_h / 2 bytes: element 2i in the low nibble of byte i, 2i + 1 in
//                the high one; code n stands for the whole number n - 8, in [-7, 7]
//   key scales   page_size rows of d_h / 32 bf16, one per 32 elements
//   value codes, value scales: the same
// An element is (n - 8) * scale.  A scale has four significant bits, so its product with a whole
// number up to 7 is a bf16 value: dequantising rounds nothing, and the tensor cores get the cache's
// values themselves.  Rounding the scale up to four bits makes a group's steps at most 1/8 wider
// (6% on average) than an exact seventh of its largest magnitude would.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace rocs {

constexpr int KV4_GROUP = 32;   // elements per scale

__host__ __device__ constexpr int kv4_codes_bytes(int tokens, int d) { return tokens * d / 2; }
__host__ __device__ constexpr int kv4_scales_bytes(int tokens, int d) { return tokens * d / KV4_GROUP * 2; }
__host__ __device__ constexpr int kv4_half_bytes(int tokens, int d) {
  return kv4_codes_bytes(tokens, d) + kv4_scales_bytes(tokens, d);
}
__host__ __device__ constexpr int kv4_record_bytes(int tokens, int d) { return 2 * kv4_half_bytes(tokens, d); }

// (128 + n) as a bf16 pair for the nibbles at bits 0..3 and 16..19 of w: 0x4300 is 128 in bf16 with
// unit spacing, so the nibble is the low mantissa bits.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x43004300u));   // (w & a) | b
  return r;
}

// x * s + c on bf16 pairs, one rounding (none here: every result is representable).
__device__ __forceinline__ uint32_t kv4_fma2(uint32_t x, uint32_t s, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(s), "r"(c));
  return r;
}

// -136 s for a pair of scales, the constant that turns (128 + n) * s into (n - 8) * s.  Exact: 136 is
// 17 * 8, and 17 times a four-bit number is at most 255; scales are at most 2^120, so it is finite.
__device__ __forceinline__ uint32_t kv4_offset(uint32_t s2) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(s2), "r"(0xC308C308u));   // bf16(-136) = 0xC308
  return r;
}

}  // namespace rocs
