// Layout of the 8-bit paged KV cache, shared by the kernels that write, read, attend
// over and evict from it.
//
// One block per (page, kv head): 64 tokens of head_dim values for K and for V, as four
// sub-blocks of 16 tokens, each 32 hd + 16 bytes:
//   [0, 16 hd)       K codes, token-major, in 16-byte chunks of 16 dims
//   [16 hd, 32 hd)   V codes
//   [32 hd, +16)     exponent of K, exponent of V (signed bytes), 14 bytes of zeros
// A code is an e4m3 number c and stands for c * 2^e, -15 <= e <= 8: 2^8 * 448 is past
// fp16's largest number, and 2^-15 * 2^-9 is its least.  A power of two, because raising
// it (a later token of the sub-block that is larger) then moves codes by whole
// exponents: what was held stays as it was, but for codes that become subnormal.
//
// The codes lie as the tensor cores' A operand (mma m16n8k16, tokens x dims for the
// scores, dims x tokens for the values) wants them after one cvt of two codes to two
// fp16 numbers.  K: lane (g, c) takes chunks c and c + 4 of tokens g and g + 8; the
// halves of odd tokens' rows are exchanged (head_dim 128), so that the eight lanes of a
// shared-memory phase hit all banks.  V: lane (g, c) takes dims g hd/8 .. of tokens 2c,
// 2c + 1, 2c + 8 and 2c + 9; a word is one dim of the four, a chunk four dims, and the 32
// lanes' chunks are adjacent.
#pragma once

#include "common.cuh"

namespace spec {

constexpr int kSub = 16;  // tokens of a sub-block

__host__ __device__ constexpr int kv8_sub_bytes(int hd) { return 2 * kSub * hd + 16; }
__host__ __device__ constexpr int kv8_block_bytes(int hd) { return kPage / kSub * kv8_sub_bytes(hd); }

// Byte offset in a sub-block of dims 16 j .. 16 j + 15 of K of token t.
template <int HD>
SPEC_DEVICE_INLINE int kv8_k_chunk(int t, int j) {
  return t * HD + ((HD == 128 ? j ^ ((t & 1) << 2) : j) << 4);
}
// Byte offset of V's chunk j (dims 4 j .. of the lane's) for lane (g, c) = g * 4 + c.
template <int HD>
SPEC_DEVICE_INLINE int kv8_v_chunk(int j, int lane) {
  return kSub * HD + j * 512 + lane * 16;
}

constexpr int kKv8MinExp = -15, kKv8MaxExp = 8;

// Exponent of K (side 0) or V (1) from a sub-block's parameter word.  Clamped: the bytes of
// a sub-block that was never written may be anything.
SPEC_DEVICE_INLINE int kv8_exp(uint32_t word, int side) {
  const int e = (int)(int8_t)(word >> (8 * side));
  return max(kKv8MinExp, min(e, kKv8MaxExp));
}
SPEC_DEVICE_INLINE uint32_t kv8_param_word(int ek, int ev) { return (uint32_t)(ek & 255) | (uint32_t)(ev & 255) << 8; }

// 2^e as fp32, -126 <= e <= 127.
SPEC_DEVICE_INLINE float kv8_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Least exponent in range with a <= 448 * 2^e (448 = 1.75 * 2^8), for a >= 0.
SPEC_DEVICE_INLINE int kv8_needed_exp(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kKv8MinExp, min(e, kKv8MaxExp));
}

// The two codes in the low (high) half of w, as fp16; exact.
SPEC_DEVICE_INLINE uint32_t kv8_lo(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
SPEC_DEVICE_INLINE uint32_t kv8_hi(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
// Four fp16 numbers (two words) to four codes, ties to even.
SPEC_DEVICE_INLINE uint32_t kv8_codes(uint32_t lo, uint32_t hi) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(y)
      : "r"(lo), "r"(hi));
  return y;
}

SPEC_DEVICE_INLINE uint32_t kv8_mul2(uint32_t a, __half2 s) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Codes of exponent `from` as codes of exponent `to` (2^(from - to) as a half2 factor):
// what no longer fits the grid is rounded to even.  (A product that is subnormal in
// fp16 is less than 2^-14, and rounds to the code 0 whatever its last bits.)
SPEC_DEVICE_INLINE uint32_t kv8_requant(uint32_t w, __half2 f) {
  return kv8_codes(kv8_mul2(kv8_lo(w), f), kv8_mul2(kv8_hi(w), f));
}

}  // namespace spec
