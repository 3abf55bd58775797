// Writing K/V into the 8-bit paged cache and reading it back.
//
// Per (16-token sub-block, kv head), for K and for V alike, the values x of the call's
// rows become
//   x' = clamp(x, -65504, 65504)                        (NaN: -65504)
//   e  = least exponent in -15..8 with max |x'| <= 448 * 2^e
//   c  = e4m3 number nearest to x' / 2^e, ties to even
// and stand for c * 2^e, which a read rounds once to the caller's type.  A row at the
// sub-block's first token starts it anew; otherwise e is at least what it was, and where
// it rises, the codes of the tokens that the call does not write are brought to it.
//
// A warp takes one sub-block of one head, all its tokens: the exponent is a warp's
// maximum, and the codes of V, four tokens to a word, are put together in registers.
// Neighbouring warps take neighbouring heads, whose rows are adjacent in memory.
//
// Both are bound by their bytes: 65536 rows of 8 heads of 128 in 62 us each, 0.95 of the copy rate;
// 80 rows in 3 us, a launch's latency.
#include "kv4.cuh"
#include "kv8.cuh"
#include "kv8.h"
#include "launch.cuh"

namespace spec {

namespace {

constexpr int kIoWarps = 4;

// The part of a sub-block that a call's rows touch: tokens [t0, t1), the first of them flat
// row `row`; `at` is its place in the pool (page * 4 + sub-block), or -1: no cell.
struct SubRows {
  long long row;
  int t0, t1;
  long long at;
};

// Work item x of a call.  The n_b rows of sequence b touch at most n_b / 16 + 2 sub-blocks,
// so its items are those from row_off[b] / 16 + 2 b on (a rising sequence whose gaps are
// wide enough); with rows_per_seq each, (n + 30) / 16 per sequence.
SPEC_DEVICE_INLINE bool item_rows(const Kv4Rows& a, long long x, SubRows& s) {
  const int lane = threadIdx.x & 31;
  int b, i, n;
  long long r0;
  if (a.row_off) {
    // the last b whose first item is at most x, 32 candidates at a time
    const auto first = [&](int j) { return ((long long)min(max(a.row_off[j], 0), a.total_rows) >> 4) + 2ll * j; };
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int j = lo + lane * step;
      const unsigned le = __ballot_sync(0xffffffffu, j < hi && (lane == 0 || first(j) <= x));
      lo += (31 - __clz(le)) * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    r0 = min(max(a.row_off[b], 0), a.total_rows);
    n = (int)max(0ll, min((long long)a.row_off[b + 1], (long long)a.total_rows) - r0);
    const long long d = x - ((r0 >> 4) + 2ll * b);
    if (d < 0 || d > (1ll << 30)) return false;
    i = (int)d;
  } else {
    const int per = (a.rows_per_seq + 30) / kSub;
    b = (int)(x / per);
    i = (int)(x - (long long)b * per);
    n = a.rows_per_seq;
    r0 = (long long)b * n;
  }
  if (b >= a.B || n <= 0) return false;
  const long long p0 = a.start[b], sub = (p0 >> 4) + i, base = sub * kSub;
  if (base >= p0 + n) return false;
  s.t0 = (int)max(0ll, p0 - base);
  s.t1 = (int)min((long long)kSub, p0 + n - base);
  s.row = r0 + (base + s.t0 - p0);
  s.at = -1;
  if (sub >= 0 && sub < (long long)a.max_pages * (kPage / kSub)) {
    const int pg = a.page_table[(long long)b * a.max_pages + (sub >> 2)];
    if (pg >= 0 && pg < a.num_pages) s.at = (long long)pg * (kPage / kSub) + (sub & 3);
  }
  return true;
}

long long item_count(const Kv4Rows& a) {
  return a.row_off ? (a.total_rows >> 4) + 2ll * a.B : (long long)a.B * ((a.rows_per_seq + 30) / kSub);
}

// Saturated in the caller's type: fp16 at once; bf16 to +-65536, its next numbers past
// +-65504, which give the same exponent and the same code.
template <bool BF16>
SPEC_DEVICE_INLINE uint4 sat8(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&w[i]);
      h = __hmin2(__hmax2(h, __float2bfloat162_rn(-65536.f)), __float2bfloat162_rn(65536.f));
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    } else {
      __half2 h = *reinterpret_cast<__half2*>(&w[i]);
      h = __hmin2(__hmax2(h, __float2half2_rn(-65504.f)), __float2half2_rn(65504.f));
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitudes, pairwise: with the sign bits off, the bit patterns of either type
// order like the numbers.
SPEC_DEVICE_INLINE uint32_t absmax8(uint32_t m, uint4 v) {
  m = __vmaxu2(m, v.x & 0x7fff7fffu);
  m = __vmaxu2(m, v.y & 0x7fff7fffu);
  m = __vmaxu2(m, v.z & 0x7fff7fffu);
  return __vmaxu2(m, v.w & 0x7fff7fffu);
}
template <bool BF16>
SPEC_DEVICE_INLINE float absmax_value(uint32_t m) {
  uint32_t a = max(m & 0xffffu, m >> 16);
  a = __reduce_max_sync(0xffffffffu, a);
  if (BF16) return __uint_as_float(a << 16);
  return __half2float(__ushort_as_half((unsigned short)a));
}

// Two values over 2^e as fp16.  (The quotient is at most 448; one below fp16's normal
// range is below 2^-14 and becomes the code 0.)
template <bool BF16>
SPEC_DEVICE_INLINE uint32_t scaled2(uint32_t w, float inv, __half2 inv2) {
  if (!BF16) return kv8_mul2(w, inv2);
  const float2 f = kv4_unpack2<true>(w);
  return pack_f16x2(f.x * inv, f.y * inv);
}

SPEC_DEVICE_INLINE __half2 half2_pow2(int e) { return __float2half2_rn(kv8_pow2(e)); }

template <int HD, bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32) kv8_write_kernel(const __grid_constant__ Kv8WriteParams p,
                                                                  long long total) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  constexpr int SUB = kv8_sub_bytes(HD);
  for (long long x = (long long)blockIdx.x * kIoWarps + (threadIdx.x >> 5); x < total;
       x += (long long)gridDim.x * kIoWarps) {
    SubRows s;
    const int h = (int)(x % p.Hkv);
    if (!item_rows(p.rows, x / p.Hkv, s) || s.at < 0) continue;
    uint8_t* const sub = p.pool + ((s.at >> 2) * p.Hkv + h) * kv8_block_bytes(HD) + (s.at & 3) * SUB;
    const bool keep = s.t0 > 0;                 // tokens held already
    uint32_t* const par = reinterpret_cast<uint32_t*>(sub + 2 * kSub * HD);
    const uint32_t old_par = keep ? *par : 0u;
    const auto in = [&](int t) { return t >= s.t0 && t < s.t1; };
    int e[2];
    {
      constexpr int N = HD / 32, CH = HD / 16;  // chunks of a lane, of a token
      const uint16_t* src = static_cast<const uint16_t*>(p.k) + (s.row - s.t0) * p.k_row_stride + (long long)h * HD;
      uint4 v[N][2];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i, t = id / CH, j = id % CH;
        v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (in(t)) {
          const uint4* a = reinterpret_cast<const uint4*>(src + t * p.k_row_stride + j * 16);
          v[i][0] = a[0];
          v[i][1] = a[1];
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          v[i][u] = sat8<BF16>(v[i][u]);
          m = absmax8(m, v[i][u]);
        }
      e[0] = kv8_needed_exp(absmax_value<BF16>(m));
      const int was = keep ? kv8_exp(old_par, 0) : e[0];
      e[0] = max(e[0], was);
      const float inv = kv8_pow2(-e[0]);
      const __half2 inv2 = half2_pow2(-e[0]), f = half2_pow2(was - e[0]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i, t = id / CH, j = id % CH;
        uint4* dst = reinterpret_cast<uint4*>(sub + kv8_k_chunk<HD>(t, j));
        if (in(t)) {
          uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = scaled2<BF16>(w[k], inv, inv2);
          *dst = make_uint4(kv8_codes(w[0], w[1]), kv8_codes(w[2], w[3]), kv8_codes(w[4], w[5]), kv8_codes(w[6], w[7]));
        } else if (e[0] != was) {
          const uint4 o = *dst;
          *dst = make_uint4(kv8_requant(o.x, f), kv8_requant(o.y, f), kv8_requant(o.z, f), kv8_requant(o.w, f));
        }
      }
    }
    {
      constexpr int N = HD / 32, L = HD / 64;   // chunks of a lane, 16-byte loads of a token
      const uint16_t* src =
          static_cast<const uint16_t*>(p.v) + (s.row - s.t0) * p.v_row_stride + (long long)h * HD + g * (HD / 8);
      uint4 v[4][L];                            // tokens 2c, 2c + 1, 2c + 8, 2c + 9
      uint32_t m = 0, mine = 0;                 // mine: the bytes of a word that the call writes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 2 * c + (i & 1) + (i >> 1) * 8;
#pragma unroll
        for (int u = 0; u < L; ++u) v[i][u] = make_uint4(0u, 0u, 0u, 0u);
        if (in(t)) {
          mine |= 0xffu << (8 * i);
#pragma unroll
          for (int u = 0; u < L; ++u) v[i][u] = reinterpret_cast<const uint4*>(src + t * p.v_row_stride)[u];
        }
      }
      uint4 old[N];
      if (mine != 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < N; ++j) old[j] = *reinterpret_cast<const uint4*>(sub + kv8_v_chunk<HD>(j, lane));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < L; ++u) {
          v[i][u] = sat8<BF16>(v[i][u]);
          m = absmax8(m, v[i][u]);
        }
      e[1] = kv8_needed_exp(absmax_value<BF16>(m));
      const int was = keep ? kv8_exp(old_par, 1) : e[1];
      e[1] = max(e[1], was);
      const float inv = kv8_pow2(-e[1]);
      const __half2 inv2 = half2_pow2(-e[1]), f = half2_pow2(was - e[1]);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {           // dims 4 j + 2 k, 4 j + 2 k + 1
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 q = v[i][j / 2];
            y[i] = scaled2<BF16>((j & 1) ? (k ? q.w : q.z) : (k ? q.y : q.x), inv, inv2);
          }
          w[2 * k] = kv8_codes(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410));
          w[2 * k + 1] = kv8_codes(__byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
        }
        if (mine != 0xffffffffu) {
          uint32_t o[4] = {old[j].x, old[j].y, old[j].z, old[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (e[1] != was) o[k] = kv8_requant(o[k], f);
            w[k] = (w[k] & mine) | (o[k] & ~mine);
          }
        }
        *reinterpret_cast<uint4*>(sub + kv8_v_chunk<HD>(j, lane)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();  // every lane has read the old exponents
    if (lane == 0) *reinterpret_cast<uint4*>(par) = make_uint4(kv8_param_word(e[0], e[1]), 0u, 0u, 0u);
  }
}

// Two held values in the caller's type (fp16: at most 65504).
template <bool BF16>
SPEC_DEVICE_INLINE uint32_t held2(uint32_t y, float s, __half2 s2) {
  if (BF16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y));
    return kv4_pack2<true>(f.x * s, f.y * s);
  }
  const uint32_t w = kv8_mul2(y, s2);
  __half2 v = *reinterpret_cast<const __half2*>(&w);
  v = __hmin2(__hmax2(v, __float2half2_rn(-65504.f)), __float2half2_rn(65504.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 bytes of a lane at `mine` and those of its partner (lane ^ D, alike but for the address
// `theirs`), stored so that two lanes fill a 32-byte sector at once: with two stores of its own per lane,
// each half a sector, 65536 rows were read in 73 us, and so in 62.
template <int D>
SPEC_DEVICE_INLINE void store_pair(bool on, uint16_t* mine, uint16_t* theirs, const uint32_t (&y)[8]) {
  const bool odd = (threadIdx.x & D) != 0;
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = __shfl_xor_sync(0xffffffffu, odd ? y[k] : y[4 + k], D);
  if (!on) return;
  // even: its first half, then the partner's first; odd: the partner's second, then its second
  uint4* const a = reinterpret_cast<uint4*>(odd ? theirs + 8 : mine);
  uint4* const b = reinterpret_cast<uint4*>(odd ? mine + 8 : theirs);
  *a = odd ? make_uint4(r[0], r[1], r[2], r[3]) : make_uint4(y[0], y[1], y[2], y[3]);
  *b = odd ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(r[0], r[1], r[2], r[3]);
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32) kv8_read_kernel(const __grid_constant__ Kv8ReadParams p,
                                                                 long long total) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  constexpr int SUB = kv8_sub_bytes(HD), N = HD / 32, CH = HD / 16;
  for (long long x = (long long)blockIdx.x * kIoWarps + (threadIdx.x >> 5); x < total;
       x += (long long)gridDim.x * kIoWarps) {
    SubRows s;
    const int h = (int)(x % p.Hkv);
    if (!item_rows(p.rows, x / p.Hkv, s)) continue;
    const auto in = [&](int t) { return t >= s.t0 && t < s.t1; };
    const auto at = [&](void* out, int t) { return static_cast<uint16_t*>(out) + ((s.row + t - s.t0) * p.Hkv + h) * HD; };
    uint4 kc[N], vc[N];
    uint32_t par = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) kc[i] = vc[i] = make_uint4(0u, 0u, 0u, 0u);
    if (s.at >= 0) {
      const uint8_t* sub = p.pool + ((s.at >> 2) * p.Hkv + h) * kv8_block_bytes(HD) + (s.at & 3) * SUB;
      par = *reinterpret_cast<const uint32_t*>(sub + 2 * kSub * HD);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i;
        if (in(id / CH)) kc[i] = *reinterpret_cast<const uint4*>(sub + kv8_k_chunk<HD>(id / CH, id % CH));
        vc[i] = *reinterpret_cast<const uint4*>(sub + kv8_v_chunk<HD>(i, lane));
      }
    }
    {
      const float f = kv8_pow2(kv8_exp(par, 0));
      const __half2 f2 = half2_pow2(kv8_exp(par, 0));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i, t = id / CH, j = id % CH;
        const uint32_t w[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[2 * k] = held2<BF16>(kv8_lo(w[k]), f, f2);
          y[2 * k + 1] = held2<BF16>(kv8_hi(w[k]), f, f2);
        }
        uint16_t* const dst = at(p.k, t);
        store_pair<1>(in(t), dst + j * 16, dst + (j ^ 1) * 16, y);
      }
    }
    {
      const float f = kv8_pow2(kv8_exp(par, 1));
      const __half2 f2 = half2_pow2(kv8_exp(par, 1));
      uint32_t y[4][HD / 16];                   // tokens 2c, 2c + 1, 2c + 8, 2c + 9: HD / 8 dims
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t w[4] = {vc[j].x, vc[j].y, vc[j].z, vc[j].w};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a = held2<BF16>(kv8_lo(w[2 * k]), f, f2), b = held2<BF16>(kv8_lo(w[2 * k + 1]), f, f2);
          const uint32_t d = held2<BF16>(kv8_hi(w[2 * k]), f, f2), q = held2<BF16>(kv8_hi(w[2 * k + 1]), f, f2);
          y[0][2 * j + k] = __byte_perm(a, b, 0x5410);
          y[1][2 * j + k] = __byte_perm(a, b, 0x7632);
          y[2][2 * j + k] = __byte_perm(d, q, 0x5410);
          y[3][2 * j + k] = __byte_perm(d, q, 0x7632);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 2 * c + (i & 1) + (i >> 1) * 8;
        uint16_t* const dst = at(p.v, t);
        if constexpr (HD == 128)
          store_pair<4>(in(t), dst + g * 16, dst + (g ^ 1) * 16, y[i]);
        else if (in(t))
          *reinterpret_cast<uint4*>(dst + g * 8) = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
      }
    }
  }
}

template <typename P>
cudaError_t launch_io(void (*f16_64)(P, long long), void (*f16_128)(P, long long), void (*b16_64)(P, long long),
                      void (*b16_128)(P, long long), const P& p, cudaStream_t st) {
  const long long total = item_count(p.rows) * p.Hkv;
  if (total <= 0) return cudaSuccess;
  const long long ctas = (total + kIoWarps - 1) / kIoWarps;
  const unsigned grid = (unsigned)(ctas < (1ll << 30) ? ctas : 1ll << 30);
  auto* k = p.bf16 ? (p.hd == 128 ? b16_128 : b16_64) : (p.hd == 128 ? f16_128 : f16_64);
  return launch_k(k, dim3(grid), dim3(kIoWarps * 32), 0, st, p, total);
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteParams& p, cudaStream_t st) {
  return launch_io<Kv8WriteParams>(kv8_write_kernel<64, false>, kv8_write_kernel<128, false>, kv8_write_kernel<64, true>,
                                   kv8_write_kernel<128, true>, p, st);
}
cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t st) {
  return launch_io<Kv8ReadParams>(kv8_read_kernel<64, false>, kv8_read_kernel<128, false>, kv8_read_kernel<64, true>,
                                  kv8_read_kernel<128, true>, p, st);
}

}  // namespace spec
