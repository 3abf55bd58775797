// Writing K/V into the 4-bit paged cache and reading it back.
//
// Per (token, kv head), for K and for V alike, a vector x of head_dim values becomes
//   x' = clamp(x, -65504, 65504)                         (NaN: -65504)
//   m  = fp16, rounded down, of min x'
//   s  = fp16, rounded up, of (max x' - m) / 15
//   c  = floor((x' - m) / s + 1/2), 0 where s = 0        (a half goes up)
// and stands for s * c + m, which a read rounds once to the caller's type.  Rounding
// s up and m down keeps every quotient inside [0, 15], so no code needs a clamp.
#include <type_traits>

#include "kv4.cuh"
#include "kv4.h"
#include "kvstate.cuh"
#include "launch.cuh"

namespace spec {

namespace {

// Physical slot of flat row r; -1: no slot given, position past the page table, or a
// page outside the pool; -2: a row of no sequence.
SPEC_DEVICE_INLINE int kv4_slot(const Kv4Rows& a, int r) {
  if (a.row_slot) {
    const int s = a.row_slot[r];
    return s >= 0 && s < a.num_pages * kPage ? s : -1;
  }
  int b, j;
  if (a.row_off) {
    int lo = 0, hi = a.B;  // last b with row_off[b] <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.row_off[mid] <= r) lo = mid;
      else hi = mid;
    }
    b = lo;
    j = r - a.row_off[b];
    if (j < 0 || r >= a.row_off[b + 1]) return -2;
  } else {
    b = r / a.rows_per_seq;
    j = r - b * a.rows_per_seq;
  }
  const long long t = (long long)a.start[b] + j;
  if (t < 0 || t >= (long long)a.max_pages * kPage) return -1;
  const int pg = a.page_table[(long long)b * a.max_pages + (int)(t / kPage)];
  return pg >= 0 && pg < a.num_pages ? pg * kPage + (int)(t % kPage) : -1;
}

// Offset m, scale s and the factor of the quotients of a vector with the given extremes.
// With d = x - m, the sum d inv + 1.5 * 2^23 rounds to the nearest whole number in the
// float's last bits.  inv is 1/s raised by 2^-22 of itself, more than the roundings of inv and
// of the product (2^-23), so an exact half (about one value in a thousand: x, m and s have
// 11 bits) goes up and no code is too small; one is too large only if 2 d lies less than
// 2^-16.5 s below an odd multiple of s (q < 14.5, at most 1.5 * 2^-22 of it).  That difference
// is a multiple of s's last bit (2^-11 s at least) or of twice x's or m's, so x or m is below
// 2^-6.5 s then.  The quotient of such an x lies that near to zero's, -m/s: `near` tells of
// rows whose -m/s is within 0.0115 of a half, or whose m is below 0.0115 s (two or three rows
// of a hundred).  All others need no second look.
SPEC_DEVICE_INLINE uint32_t kv4_params(float lo, float hi, float& m, float& inv, bool& near) {
  const __half mh = kv4_half_down(lo);
  m = __half2float(mh);
  const __half sh = kv4_half_up(__fdiv_rn(__fsub_rn(hi, m), 15.f));
  const float s = __half2float(sh);
  inv = s > 0.f ? __fmul_rn(__frcp_rn(s), 1.f + 2.384185791015625e-7f) : 0.f;
  const float zero = -m * inv;
  near = fabsf(zero - floorf(zero) - 0.5f) < 0.0115f || fabsf(m) < 0.0115f * s;
  return ((uint32_t)__half_as_ushort(sh) << 16) | __half_as_ushort(mh);
}

// Codes of eight values, value i in nibble i.  The sums' bits are 0x4b400000 + c; they are
// added up shifted and the constants' sum taken off once.  Two values to an instruction, each
// rounded as by itself.
SPEC_DEVICE_INLINE uint32_t kv4_codes(const float (&x)[8], float m, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    float lo, hi;
    asm("{\n\t.reg .b64 d, f, t;\n\t"
        "mov.b64 d, {%2, %3};\n\tmov.b64 t, {%4, %4};\n\tadd.rn.f32x2 d, d, t;\n\t"
        "mov.b64 t, {%5, %5};\n\tmov.b64 f, {%6, %6};\n\tfma.rn.f32x2 f, d, t, f;\n\tmov.b64 {%0, %1}, f;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "f"(x[i]), "f"(x[i + 1]), "f"(-m), "f"(inv), "f"(12582912.f));
    w = (w << 4) + __float_as_uint(hi);
    w = (w << 4) + __float_as_uint(lo);
  }
  return w - 0x4b400000u * 0x11111111u;
}
// The same for rows that are near: a code c is too large where d < (c - 1/2) s.  c - 1/2 is
// exact, and an fma's sign is that of the exact d - (c - 1/2) s.  (d - s c itself need not fit
// a float: for c = 1 and d the last number below s/2 it rounds to -s/2.)
SPEC_DEVICE_INLINE uint32_t kv4_codes_near(const float (&x)[8], float m, float s, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float d = __fsub_rn(x[i], m), f = __fmaf_rn(d, inv, 12582912.f);
    w = (w << 4) + __float_as_uint(f) - (__fmaf_rn(__fsub_rn(f, 12582912.f) - 0.5f, -s, d) < 0.f ? 1u : 0u);
  }
  return w - 0x4b400000u * 0x11111111u;
}

// Eight of the caller's values: saturated in their own type (fp16 at once; bf16 to +-65536,
// its next numbers beyond, so NaN and infinities are gone) ...
template <bool BF16>
SPEC_DEVICE_INLINE void kv4_clamp(uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&w[i]);
      v = __hmin2(__hmax2(v, __float2bfloat162_rn(-65536.f)), __float2bfloat162_rn(65536.f));
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    } else {
      __half2 v = *reinterpret_cast<__half2*>(&w[i]);
      v = __hmin2(__hmax2(v, __float2half2_rn(-65504.f)), __float2half2_rn(65504.f));
      w[i] = *reinterpret_cast<uint32_t*>(&v);
    }
  }
}
// ... their minimum (low half) and negated maximum (high half) over LANES neighbouring
// lanes, NaN if there is one ...
template <bool BF16>
SPEC_DEVICE_INLINE uint32_t kv4_min2(uint32_t a, uint32_t b) {
  if (BF16) {
    __nv_bfloat162 v = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __half2 v = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&v);
}
// Whether such a pair is within +-65504 (then so is every value, and saturating changes none).
template <bool BF16>
SPEC_DEVICE_INLINE bool kv4_in_range(uint32_t e) {
  const float2 f = kv4_unpack2<BF16>(e);
  return f.x >= -65504.f && f.y >= -65504.f;
}
template <bool BF16, int LANES>
SPEC_DEVICE_INLINE uint32_t kv4_extremes(const uint32_t (&w)[4]) {
  uint32_t lo = kv4_min2<BF16>(kv4_min2<BF16>(w[0], w[1]), kv4_min2<BF16>(w[2], w[3]));
  uint32_t hi = kv4_min2<BF16>(kv4_min2<BF16>(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                               kv4_min2<BF16>(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
  uint32_t r = kv4_min2<BF16>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) r = kv4_min2<BF16>(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}
// ... and as fp32.
template <bool BF16>
SPEC_DEVICE_INLINE void kv4_floats(const uint32_t (&w)[4], bool in_range, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = kv4_unpack2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  if (BF16 && !in_range)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kv4_sat(x[i]);
}

// Both kernels: grid (chunks of 8 RPW rows, kv heads); a warp takes RPW <= 16 consecutive
// rows of one head, 32 / (hd / 8) of them at a time with eight dims per lane.  Lane (kv,
// row) -- the upper half of the warp for V -- looks after one row's slot and parameters,
// so a row's address chain and its division are paid once and in parallel for all 16.  A V
// piece is two bytes, next to the same dims of the neighbouring token: where a pair of rows
// fills a pair of cells, the lanes of the two rows exchange halves and move whole words.
//
// What bounds them: HBM for many rows.  262144 rows of 8 heads (head_dim 128) are read in
// 207 us (either type), 0.97 of the measured copy rate over 1.36 GB; a write of 65536 rows and their
// reading back take 125 us, 0.80 of it, of which the write is 75: its instructions.  (One
// row per half-warp, with every address and division computed by all of its lanes and
// int-to-float conversions, took 282 and 188: the special-function and integer pipes were
// the limit.  The second look at every row took 138 in place of 125, at near rows after the
// others 132; scalar differences and quotients 128; saturating every value 132.)  For few rows it is the latency of
// one warp's chain, so a warp then takes one step of rows only.
template <int HD, bool BF16, int RPW>
__global__ void __launch_bounds__(256, RPW == 16 ? 3 : 1) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
  constexpr int L = HD / 8;                 // lanes of a row
  constexpr int T = 32 / L;                 // rows at a time
  constexpr int IT = RPW / T;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, h = blockIdx.y, j8 = lane % L;
  const int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW;
  const int n = p.rows.total_rows - r0;     // rows from r0 on
  if (n <= 0) return;
  uint32_t w[2][IT][4];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int tok = it * T + lane / L;
    const int r = r0 + min(tok, n - 1);
    const long long at = (long long)(r / p.row_blk) * p.blk_stride + (long long)h * p.head_stride + j8 * 8;
    const int rr = r % p.row_blk;
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + at + rr * p.k_row_stride));
    const uint4 b = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + at + rr * p.v_row_stride));
    w[0][it][0] = a.x, w[0][it][1] = a.y, w[0][it][2] = a.z, w[0][it][3] = a.w;
    w[1][it][0] = b.x, w[1][it][1] = b.y, w[1][it][2] = b.z, w[1][it][3] = b.w;
  }
  const int my_row = lane & 15, my_kv = lane >> 4;
  const int my_slot = my_row < min(n, RPW) ? kv4_slot(p.rows, r0 + my_row) : -1;
  uint32_t mine = 0;                        // extremes of this lane's row
  bool in_range = true;                     // all of the warp's values
  // Saturating costs eight instructions of eight values: it is done only where the extremes
  // show a value that needs it, for all of the warp's rows, and they are taken again.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (pass == 1) kv4_clamp<BF16>(w[kv][it]);
        const uint32_t e = __shfl_sync(0xffffffffu, kv4_extremes<BF16, L>(w[kv][it]), my_row % T * L);
        if (my_row / T == it && my_kv == kv) mine = e;
      }
    }
    if (pass == 1 || __all_sync(0xffffffffu, kv4_in_range<BF16>(mine))) break;
    in_range = false;
  }
  const float2 ext = kv4_unpack2<BF16>(mine);
  float m, inv;
  bool my_near;
  const uint32_t par = kv4_params(kv4_sat(ext.x), kv4_sat(-ext.y), m, inv, my_near);
  const uint32_t near = __ballot_sync(0xffffffffu, my_near);
  constexpr int kBlock = kv4_block_bytes(HD);
  if (my_slot >= 0)
    reinterpret_cast<uint32_t*>(p.pool + ((long long)(my_slot / kPage) * p.Hkv + h) * kBlock + kPage * HD)[
        my_kv * kPage + my_slot % kPage] = par;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int tok = it * T + lane / L;
    const int slot = __shfl_sync(0xffffffffu, my_slot, tok), other_slot = __shfl_sync(0xffffffffu, my_slot, tok ^ 1);
    uint32_t code[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float tm = __shfl_sync(0xffffffffu, m, kv * 16 + tok), ti = __shfl_sync(0xffffffffu, inv, kv * 16 + tok);
      float x[8];
      kv4_floats<BF16>(w[kv][it], in_range, x);
      if (near >> (kv * 16 + it * T) & ((1u << T) - 1u)) {
        const uint32_t s = __shfl_sync(0xffffffffu, par, kv * 16 + tok) >> 16;
        code[kv] = kv4_codes_near(x, tm, __half2float(__ushort_as_half((unsigned short)s)), ti);
      } else {
        code[kv] = kv4_codes(x, tm, ti);
      }
    }
    const uint32_t other = __shfl_xor_sync(0xffffffffu, code[1], L);
    if (slot < 0) continue;
    uint8_t* block = p.pool + ((long long)(slot / kPage) * p.Hkv + h) * kBlock;
    const int t = slot % kPage;
    reinterpret_cast<uint32_t*>(block + t * (HD / 2))[j8] = code[0];
    uint8_t* v = block + kPage * HD / 2;
    if (other_slot == (slot ^ 1) && (tok & 1) == (slot & 1)) {
      // the even row stores dims 0..3 of both, the odd one dims 4..7
      const int odd = tok & 1;
      *reinterpret_cast<uint32_t*>(v + kv4_v_piece<HD>(t & ~1, j8 * 8 + 4 * odd)) =
          odd ? __byte_perm(other, code[1], 0x7632) : __byte_perm(code[1], other, 0x5410);
    } else {
      *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8)) = (uint16_t)code[1];
      *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8 + 4)) = (uint16_t)(code[1] >> 16);
    }
  }
}

// s * c + m, or the odd one of the two floats around it: an inexact sum is then never a tie of
// bf16's, so rounding it to bf16 next is one rounding in all.
SPEC_DEVICE_INLINE float kv4_value_odd(uint32_t c, float s, float m) {
  const float lo = __fmaf_rd((float)c, s, m), hi = __fmaf_ru((float)c, s, m);
  return __float_as_uint(lo) & 1u ? lo : hi;
}

// s * c + m of eight codes, rounded once to the caller's type.  fp16: a nibble OR-ed under
// 0x6400 (or 0x5400, one nibble up) is the number 1024 + c (64 + c), so a subtraction gives
// c exactly and one fused multiply-add the result.  bf16: the sum is rounded to fp32 on the way,
// which most parameters leave exact: s c + m is a multiple of the smaller one's last bit (2^-11
// of it at least) and below 2 max(15 s, |m|).  CARE, where kv4_care says so of a row of
// the warp: the results are held to 65504 (fp16), the sums are kept odd (bf16; for all rows it
// cost a fifth of a large read: 262144 rows of 8 heads 250 against 207 us).
template <bool BF16>
SPEC_DEVICE_INLINE bool kv4_care(uint32_t par) {
  const float2 ms = __half22float2(*reinterpret_cast<const __half2*>(&par));
  const float m = fabsf(ms.x), s = ms.y;
  if (BF16) return m > 0.f && s > 0.f && fmaxf(m, 15.f * s) > 4096.f * fminf(m, s);
  return fmaf(15.f, s, ms.x) > 65504.f;  // by at most 16: s is rounded up
}
template <bool BF16, bool CARE>
SPEC_DEVICE_INLINE uint4 kv4_expand8(uint32_t code, uint32_t par) {
  uint32_t o[4];
  if (BF16) {
    const float2 ms = __half22float2(*reinterpret_cast<const __half2*>(&par));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c0 = (code >> (8 * i)) & 15u, c1 = (code >> (8 * i + 4)) & 15u;
      o[i] = CARE ? kv4_pack2<true>(kv4_value_odd(c0, ms.y, ms.x), kv4_value_odd(c1, ms.y, ms.x))
                  : kv4_pack2<true>(__fmaf_rn((float)c0, ms.y, ms.x), __fmaf_rn((float)c1, ms.y, ms.x));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  const uint32_t m2 = __byte_perm(par, par, 0x1010), s2 = __byte_perm(par, par, 0x3232);
  const uint32_t hi = code >> 8;
  const uint32_t raw[4] = {(code & 0x000f000fu) | 0x64006400u, (code & 0x00f000f0u) | 0x54005400u,
                           (hi & 0x000f000fu) | 0x64006400u, (hi & 0x00f000f0u) | 0x54005400u};
  uint32_t v[4];                            // (0, 4) (1, 5) (2, 6) (3, 7)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&raw[i]), __float2half2_rn(i & 1 ? 64.f : 1024.f));
    __half2 r = __hfma2(c, *reinterpret_cast<const __half2*>(&s2), *reinterpret_cast<const __half2*>(&m2));
    if (CARE) r = __hmin2(r, __float2half2_rn(65504.f));
    v[i] = *reinterpret_cast<uint32_t*>(&r);
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                    __byte_perm(v[2], v[3], 0x7632));
}

template <int HD, bool BF16, int RPW>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  constexpr int L = HD / 8;
  constexpr int T = 32 / L;
  constexpr int IT = RPW / T;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, h = blockIdx.y, j8 = lane % L;
  const int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW;
  const int n = p.rows.total_rows - r0;
  if (n <= 0) return;
  const int my_row = lane & 15, my_kv = lane >> 4;
  const int my_slot = my_row < min(n, RPW) ? kv4_slot(p.rows, r0 + my_row) : -2;
  constexpr int kBlock = kv4_block_bytes(HD);
  uint32_t par = 0;                         // a position without a page reads as zeros
  if (my_slot >= 0)
    par = reinterpret_cast<const uint32_t*>(p.pool + ((long long)(my_slot / kPage) * p.Hkv + h) * kBlock + kPage * HD)[
        my_kv * kPage + my_slot % kPage];
  uint32_t kc[IT], vc[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int tok = it * T + lane / L, odd = tok & 1;
    const int slot = __shfl_sync(0xffffffffu, my_slot, tok), other_slot = __shfl_sync(0xffffffffu, my_slot, tok ^ 1);
    kc[it] = vc[it] = 0;
    if (slot < 0) continue;
    const uint8_t* block = p.pool + ((long long)(slot / kPage) * p.Hkv + h) * kBlock;
    const int t = slot % kPage;
    kc[it] = reinterpret_cast<const uint32_t*>(block + t * (HD / 2))[j8];
    const uint8_t* v = block + kPage * HD / 2;
    if (other_slot == (slot ^ 1) && odd == (slot & 1))
      vc[it] = *reinterpret_cast<const uint32_t*>(v + kv4_v_piece<HD>(t & ~1, j8 * 8 + 4 * odd));  // both rows' dims
    else
      vc[it] = *reinterpret_cast<const uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8)) |
               ((uint32_t)*reinterpret_cast<const uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8 + 4)) << 16);
  }
  const auto expand = [&](auto care) {
    constexpr bool kCare = decltype(care)::value;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int tok = it * T + lane / L, odd = tok & 1;
      const int slot = __shfl_sync(0xffffffffu, my_slot, tok), other_slot = __shfl_sync(0xffffffffu, my_slot, tok ^ 1);
      const uint32_t kp = __shfl_sync(0xffffffffu, par, tok), vp = __shfl_sync(0xffffffffu, par, 16 + tok);
      const uint32_t other = __shfl_xor_sync(0xffffffffu, vc[it], L);
      uint32_t v = vc[it];
      if (slot >= 0 && other_slot == (slot ^ 1) && odd == (slot & 1))
        v = odd ? __byte_perm(other, v, 0x7632) : __byte_perm(v, other, 0x5410);
      if (slot == -2) continue;             // past the last row, or a row of no sequence
      const long long at = ((long long)(r0 + tok) * p.Hkv + h) * L + j8;
      __stcs(reinterpret_cast<uint4*>(p.k) + at, kv4_expand8<BF16, kCare>(kc[it], kp));
      __stcs(reinterpret_cast<uint4*>(p.v) + at, kv4_expand8<BF16, kCare>(v, vp));
    }
  };
  if (__any_sync(0xffffffffu, kv4_care<BF16>(par))) expand(std::true_type{});
  else expand(std::false_type{});
}

// Pseudo-random cells.  grid (pages, n_layers, n); each block fills one page of one layer.
template <int HD>
__global__ void kv4_fill_kernel(uint8_t* pool, long long layer_bytes, const int32_t* page_table,
                                const int32_t* seq_npages, int max_pages, const int32_t* seq_ids, int num_pages, int Hkv,
                                uint64_t seed, float scale) {
  constexpr int kLanes = HD / 8;
  pdl_wait();
  pdl_launch_dependents();
  const int s = seq_ids[blockIdx.z];
  const int layer = blockIdx.y, pi = blockIdx.x;
  if (pi >= seq_npages[s]) return;
  const int pg = page_table[(long long)s * max_pages + pi];
  if (pg < 0) return;
  const int j8 = threadIdx.x % kLanes;
  for (int e = threadIdx.x / kLanes; e < Hkv * kPage; e += blockDim.x / kLanes) {
    const int h = e / kPage, t = e % kPage;
    const long long base = ((((long long)layer * num_pages + pg) * Hkv + h) * kPage + t) * HD + j8 * 8;
    uint8_t* block = pool + layer * layer_bytes + ((long long)pg * Hkv + h) * kv4_block_bytes(HD);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t w = splitmix64(seed ^ (uint64_t)(base + i) * 0x2545F4914F6CDD1Dull) >> (32 * kv);
        x[i] = ((float)(uint32_t)(w & 0xffffffu) * (1.0f / 16777216.0f) * 2.f - 1.f) * scale;
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 v = __halves2half2(to_act(x[2 * i]), to_act(x[2 * i + 1]));
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      const float2 ext = kv4_unpack2<false>(kv4_extremes<false, kLanes>(w));
      kv4_floats<false>(w, true, x);
      float m, inv;
      bool near;
      const uint32_t par = kv4_params(ext.x, -ext.y, m, inv, near);
      const uint32_t code = kv4_codes_near(x, m, __half2float(__ushort_as_half((unsigned short)(par >> 16))), inv);
      if (j8 == 0) reinterpret_cast<uint32_t*>(block + kPage * HD)[kv * kPage + t] = par;
      if (kv == 0) {
        reinterpret_cast<uint32_t*>(block + t * (HD / 2))[j8] = code;
      } else {
        uint8_t* v = block + kPage * HD / 2;
        *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8)) = (uint16_t)code;
        *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8 + 4)) = (uint16_t)(code >> 16);
      }
    }
  }
}

template <typename P, typename K>
cudaError_t launch_rows(K kernel, int rows_per_warp, const P& p, cudaStream_t st) {
  const unsigned chunks = (unsigned)(((long long)p.rows.total_rows + 8 * rows_per_warp - 1) / (8 * rows_per_warp));
  return launch_k(kernel, dim3(chunks, p.Hkv), dim3(256), 0, st, p);
}

// One step of rows per warp while all warps are resident at once (64 on each of 152 SMs): measured
// (8 heads of 128, a write and its reading back) 80 rows 4.5 against 9.0 us.
bool few_rows(const Kv4Rows& r, int Hkv, int hd) { return (long long)r.total_rows * Hkv <= 152ll * 64 * (256 / hd); }

template <int HD, bool BF16>
cudaError_t launch_write(const Kv4WriteParams& p, cudaStream_t st) {
  constexpr int kStep = 256 / HD;
  return few_rows(p.rows, p.Hkv, HD) ? launch_rows(kv4_write_kernel<HD, BF16, kStep>, kStep, p, st)
                                     : launch_rows(kv4_write_kernel<HD, BF16, 16>, 16, p, st);
}
template <int HD, bool BF16>
cudaError_t launch_read(const Kv4ReadParams& p, cudaStream_t st) {
  constexpr int kStep = 256 / HD;
  return few_rows(p.rows, p.Hkv, HD) ? launch_rows(kv4_read_kernel<HD, BF16, kStep>, kStep, p, st)
                                     : launch_rows(kv4_read_kernel<HD, BF16, 16>, 16, p, st);
}

}  // namespace

cudaError_t launch_kv4_fill_pages(uint8_t* pool, long long layer_bytes, const int32_t* page_table,
                                  const int32_t* seq_npages, int max_pages, const int32_t* seq_ids, int n, int n_layers,
                                  int num_pages, int Hkv, int hd, uint64_t seed, float scale, cudaStream_t st) {
  return launch_k(hd == 128 ? kv4_fill_kernel<128> : kv4_fill_kernel<64>, dim3(max_pages, n_layers, n), dim3(256), 0, st,
                  pool, layer_bytes, page_table, seq_npages, max_pages, seq_ids, num_pages, Hkv, seed, scale);
}

cudaError_t launch_kv4_write(const Kv4WriteParams& p, cudaStream_t st) {
  if (p.rows.total_rows == 0) return cudaSuccess;
  if (p.hd == 128) return p.bf16 ? launch_write<128, true>(p, st) : launch_write<128, false>(p, st);
  return p.bf16 ? launch_write<64, true>(p, st) : launch_write<64, false>(p, st);
}

cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t st) {
  if (p.rows.total_rows == 0) return cudaSuccess;
  if (p.hd == 128) return p.bf16 ? launch_read<128, true>(p, st) : launch_read<128, false>(p, st);
  return p.bf16 ? launch_read<64, true>(p, st) : launch_read<64, false>(p, st);
}

}  // namespace spec
