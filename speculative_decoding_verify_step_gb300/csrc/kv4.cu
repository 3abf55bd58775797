// Writing K/V into the 4-bit paged cache and reading it back.
//
// Per (token, kv head), for K and for V alike, a vector x of head_dim values becomes
//   x' = clamp(x, -65504, 65504)                         (NaN: -65504)
//   m  = fp16, rounded down, of min x'
//   s  = fp16, rounded up, of (max x' - m) / 15
//   c  = floor((x' - m) / s + 1/2), 0 where s = 0        (a half goes up)
// and stands for s * c + m, which a read rounds once to the caller's type.  Rounding
// s up and m down keeps every quotient inside [0, 15], so no code needs a clamp.
#include "kv4.cuh"
#include "kv4.h"
#include "kvstate.cuh"
#include "launch.cuh"

namespace spec {

namespace {

// Physical slot of flat row r; -1: no slot given, position past the page table, or a
// page outside the pool; -2: a row of no sequence.
SPEC_DEVICE_INLINE long long kv4_slot(const Kv4Rows& a, int r) {
  if (a.row_slot) {
    const int s = a.row_slot[r];
    return s >= 0 && s < (long long)a.num_pages * kPage ? s : -1;
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
  if (pg < 0 || pg >= a.num_pages) return -1;
  return (long long)pg * kPage + (int)(t % kPage);
}

// Codes of the 8 values of this thread; LANES neighbouring threads hold the token's
// vector.  Returns the 8 codes as one word (value i in nibble i) and the parameters.
template <int LANES>
SPEC_DEVICE_INLINE uint32_t kv4_quantise(const float (&x)[8], uint32_t& par) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const __half mh = kv4_half_down(lo);
  const float m = __half2float(mh);
  const __half sh = kv4_half_up(__fdiv_rn(__fsub_rn(hi, m), 15.f));
  const float s = __half2float(sh);
  // (x - m) / s + 1/2, floored: the sum (x - m) * inv + 1.5 * 2^23 rounds to the
  // nearest whole number in the float's last bits.  inv is 1/s raised by 2^-20 of
  // itself, so an exact half (about one value in a thousand: x, m and s have 11
  // bits) always goes up, whichever way 1/s was rounded.
  const float inv = s > 0.f ? __fmul_rn(__frcp_rn(s), 1.f + 9.5367431640625e-7f) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fmaf_rn(__fsub_rn(x[i], m), inv, 12582912.f);
    w |= (__float_as_uint(t) & 15u) << (4 * i);
  }
  par = ((uint32_t)__half_as_ushort(sh) << 16) | __half_as_ushort(mh);
  return w;
}

// Store a thread's codes and its token's parameters in the token's cell.
template <int HD>
SPEC_DEVICE_INLINE void kv4_store(uint8_t* block, int t, int j8, const uint32_t (&code)[2], const uint32_t (&par)[2]) {
  reinterpret_cast<uint32_t*>(block + t * (HD / 2))[j8] = code[0];
  uint8_t* v = block + kPage * HD / 2;
  *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8)) = (uint16_t)code[1];
  *reinterpret_cast<uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8 + 4)) = (uint16_t)(code[1] >> 16);
  if (j8 < 2) reinterpret_cast<uint32_t*>(block + kPage * HD)[j8 * kPage + t] = j8 ? par[1] : par[0];
}

// One token and kv head per hd / 8 threads, eight dims of K and of V each.  The
// warp's tokens are neighbouring rows of one head, so a token pair's V pieces meet
// in one 128-byte row of the block.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
  constexpr int kLanes = HD / 8;
  constexpr int kTok = 32 / kLanes;  // tokens of a warp
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long wid = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int h = (int)(wid % p.Hkv);
  const long long r = wid / p.Hkv * kTok + lane / kLanes;
  const int j8 = lane % kLanes;
  const bool in = r < p.rows.total_rows;
  const long long slot = in ? kv4_slot(p.rows, (int)r) : -1;
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
  if (slot >= 0) {
    const long long blk = r / p.row_blk, rr = r % p.row_blk;
    const long long at = blk * p.blk_stride + h * p.head_stride + j8 * 8;
    kw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + at + rr * p.k_row_stride);
    vw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + at + rr * p.v_row_stride);
  }
  uint32_t code[2], par[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = i ? vw : kw;
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = kv4_unpack2<BF16>(ws[e]);
      x[2 * e] = kv4_sat(f.x);
      x[2 * e + 1] = kv4_sat(f.y);
    }
    code[i] = kv4_quantise<kLanes>(x, par[i]);
  }
  if (slot < 0) return;
  uint8_t* block = p.pool + ((slot / kPage) * p.Hkv + h) * (long long)kv4_block_bytes(HD);
  const int t = (int)(slot % kPage);
  kv4_store<HD>(block, t, j8, code, par);
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
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t w = splitmix64(seed ^ (uint64_t)(base + i) * 0x2545F4914F6CDD1Dull);
      x[0][i] = ((float)(uint32_t)(w & 0xffffffu) * (1.0f / 16777216.0f) * 2.f - 1.f) * scale;
      x[1][i] = ((float)(uint32_t)((w >> 32) & 0xffffffu) * (1.0f / 16777216.0f) * 2.f - 1.f) * scale;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) x[kv][i] = __half2float(to_act(x[kv][i]));
    }
    uint32_t code[2], par[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) code[kv] = kv4_quantise<kLanes>(x[kv], par[kv]);
    kv4_store<HD>(pool + layer * layer_bytes + ((long long)pg * Hkv + h) * kv4_block_bytes(HD), t, j8, code, par);
  }
}

// Two fp32 to fp16, finite: s is rounded up, so 15 s + m can pass 65504 by 16.
SPEC_DEVICE_INLINE uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// s * c + m of eight codes, rounded once to the caller's type.
template <bool BF16>
SPEC_DEVICE_INLINE uint4 kv4_expand8(uint32_t code, uint32_t par) {
  const float m = __half2float(__ushort_as_half((unsigned short)(par & 0xffffu)));
  const float s = __half2float(__ushort_as_half((unsigned short)(par >> 16)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __fmaf_rn((float)((code >> (8 * i)) & 15u), s, m);
    const float hi = __fmaf_rn((float)((code >> (8 * i + 4)) & 15u), s, m);
    w[i] = BF16 ? kv4_pack2<true>(lo, hi) : pack_f16x2_sat(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  constexpr int kLanes = HD / 8;
  constexpr int kTok = 32 / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long wid = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int h = (int)(wid % p.Hkv);
  const long long r = wid / p.Hkv * kTok + lane / kLanes;
  const int j8 = lane % kLanes;
  if (r >= p.rows.total_rows) return;
  const long long slot = kv4_slot(p.rows, (int)r);
  if (slot == -2) return;
  uint32_t kc = 0, vc = 0, kp = 0, vp = 0;  // a position without a page reads as zeros
  if (slot >= 0) {
    const uint8_t* block = p.pool + ((slot / kPage) * p.Hkv + h) * (long long)kv4_block_bytes(HD);
    const int t = (int)(slot % kPage);
    kc = reinterpret_cast<const uint32_t*>(block + t * (HD / 2))[j8];
    const uint8_t* v = block + kPage * HD / 2;
    vc = *reinterpret_cast<const uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8)) |
         ((uint32_t)*reinterpret_cast<const uint16_t*>(v + kv4_v_piece<HD>(t, j8 * 8 + 4)) << 16);
    const uint32_t* par = reinterpret_cast<const uint32_t*>(block + kPage * HD);
    kp = par[t];
    vp = par[kPage + t];
  }
  const long long at = (r * p.Hkv + h) * kLanes + j8;
  reinterpret_cast<uint4*>(p.k)[at] = kv4_expand8<BF16>(kc, kp);
  reinterpret_cast<uint4*>(p.v)[at] = kv4_expand8<BF16>(vc, vp);
}

// Blocks of 8 warps; a warp takes 256 / hd rows of one head.
template <typename P, typename K>
cudaError_t launch_rows(K kernel, const P& p, cudaStream_t st) {
  const long long per = 256 / p.hd;
  const long long warps = (p.rows.total_rows + per - 1) / per * p.Hkv;
  if (warps == 0) return cudaSuccess;
  const long long blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_k(kernel, dim3((unsigned)blocks), dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_kv4_fill_pages(uint8_t* pool, long long layer_bytes, const int32_t* page_table,
                                  const int32_t* seq_npages, int max_pages, const int32_t* seq_ids, int n, int n_layers,
                                  int num_pages, int Hkv, int hd, uint64_t seed, float scale, cudaStream_t st) {
  return launch_k(hd == 128 ? kv4_fill_kernel<128> : kv4_fill_kernel<64>, dim3(max_pages, n_layers, n), dim3(256), 0, st,
                  pool, layer_bytes, page_table, seq_npages, max_pages, seq_ids, num_pages, Hkv, seed, scale);
}

cudaError_t launch_kv4_write(const Kv4WriteParams& p, cudaStream_t st) {
  if (p.hd == 128)
    return p.bf16 ? launch_rows(kv4_write_kernel<128, true>, p, st) : launch_rows(kv4_write_kernel<128, false>, p, st);
  return p.bf16 ? launch_rows(kv4_write_kernel<64, true>, p, st) : launch_rows(kv4_write_kernel<64, false>, p, st);
}

cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t st) {
  if (p.hd == 128)
    return p.bf16 ? launch_rows(kv4_read_kernel<128, true>, p, st) : launch_rows(kv4_read_kernel<128, false>, p, st);
  return p.bf16 ? launch_rows(kv4_read_kernel<64, true>, p, st) : launch_rows(kv4_read_kernel<64, false>, p, st);
}

}  // namespace spec
