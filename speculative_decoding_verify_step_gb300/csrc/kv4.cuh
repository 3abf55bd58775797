// Layout of the 4-bit paged KV cache, shared by the kernels that write, read and
// attend over it.
//
// One block per (page, kv head): 64 tokens of head_dim values for K and for V.
//   [0, 32 hd)          K codes, token-major: byte i of a token holds dims 2i (low
//                       nibble) and 2i + 1
//   [32 hd, 64 hd)      V codes (v_piece below)
//   [64 hd, +256)       K parameters, one word per token: offset m (low half) and
//                       scale s (high half), both fp16
//   [64 hd + 256, +256) V parameters
// A code c of a token stands for s * c + m.  The 64 hd + 512 bytes of a block are
// 4 + 32 / hd bits per value and a multiple of 16, so a block is
// one bulk copy.
//
// V's codes feed the transposed operand of the PV product (rows are dims, the
// contraction runs over tokens): a register of that operand holds one dim of two
// neighbouring tokens.  Four consecutive dims of a token are one 16-bit piece, the
// pieces of tokens 2n and 2n + 1 are adjacent, and one AND of such a word yields one
// dim of both tokens.  A lane's pieces of one 16-token step are a 16-byte chunk;
// eight chunks (dims in order) make a 128-byte row whose chunks are XOR-ed with the
// lane's token group, which spreads the eight lanes of a shared-memory phase over
// all banks.  A token still owns whole 16-bit pieces, so writing one token never
// reads or rewrites another's bytes.
#pragma once

#include "common.cuh"

namespace spec {

__host__ __device__ constexpr int kv4_block_bytes(int hd) { return kPage * hd + 2 * kPage * 4; }

// Byte offset, from the V codes of a block, of the piece with dims d .. d + 3 (d a
// multiple of 4) of token t.
template <int HD>
SPEC_DEVICE_INLINE int kv4_v_piece(int t, int d) {
  constexpr int kPer = HD / 8;  // dims of a chunk
  const int g = d / kPer, piece = (d % kPer) / 4;
  if (HD == 128) {
    const int blk = t >> 1;  // token pair; chunk = 4 pieces x 2 tokens
    return blk * 128 + ((g ^ (2 * (blk & 3))) << 4) + piece * 4 + (t & 1) * 2;
  }
  const int blk = (t >> 4) * 4 + ((t & 7) >> 1);  // chunk = tokens {2n, 2n+1}, {2n+8, 2n+9} x 2 pieces
  return blk * 128 + ((g ^ (2 * (blk & 3))) << 4) + ((t >> 3) & 1) * 8 + piece * 4 + (t & 1) * 2;
}

// Copy one token's cell from block `src`, token ts, to block `dst`, token td.
template <int HD>
SPEC_DEVICE_INLINE void kv4_move_token(const uint8_t* src, int ts, uint8_t* dst, int td) {
#pragma unroll
  for (int i = 0; i < HD / 32; ++i)
    reinterpret_cast<uint4*>(dst + td * (HD / 2))[i] = reinterpret_cast<const uint4*>(src + ts * (HD / 2))[i];
  const uint8_t* vs = src + kPage * HD / 2;
  uint8_t* vd = dst + kPage * HD / 2;
#pragma unroll 8
  for (int d = 0; d < HD; d += 4)
    *reinterpret_cast<uint16_t*>(vd + kv4_v_piece<HD>(td, d)) =
        *reinterpret_cast<const uint16_t*>(vs + kv4_v_piece<HD>(ts, d));
  const uint32_t* ps = reinterpret_cast<const uint32_t*>(src + kPage * HD);
  uint32_t* pd = reinterpret_cast<uint32_t*>(dst + kPage * HD);
  pd[td] = ps[ts];
  pd[kPage + td] = ps[kPage + ts];
}

// fp32 in fp16's range to fp16, towards -infinity / +infinity.
SPEC_DEVICE_INLINE __half kv4_half_down(float x) { return __float2half_rd(x); }
SPEC_DEVICE_INLINE __half kv4_half_up(float x) { return __float2half_ru(x); }

// Two elements of the caller's type as fp32, and back.
template <bool BF16>
SPEC_DEVICE_INLINE float2 kv4_unpack2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
SPEC_DEVICE_INLINE uint32_t kv4_pack2(float lo, float hi) {
  if (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  return pack_f16x2(lo, hi);
}

// The library's fp16 saturation (to_act): finite values beyond +-65504 and
// infinities clamp, NaN becomes -65504.
SPEC_DEVICE_INLINE float kv4_sat(float x) { return fminf(fmaxf(x, -65504.f), 65504.f); }

}  // namespace spec
