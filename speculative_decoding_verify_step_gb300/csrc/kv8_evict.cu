// Eviction from the 8-bit paged cache by accumulated attention weight.
//
// Of the n tokens of a sequence and kv head, m = min(keep, n) stay: the last `recent`, and
// of the others those of the largest weight, the earlier of equal ones.  They move, in
// order, to cells 0..m-1 of the destination table's pages; a destination sub-block gets the
// least exponents that hold its tokens, as if the held values were written there.
//
// Two kernels.  The first takes a CTA or two per (sequence, kv head): its weights, as integers
// that order like them, come into shared memory once (up to 48 K tokens; of longer ones
// they are read from L2 again) and a radix select of 11, 11 and 10 bits finds the
// threshold, the last two digits among the few tokens that share the first.  11 bits, because
// weights spread over exponents: with 8 most lanes of a warp would add to the same counter.
// Warps own runs of neighbouring tokens, four to a lane, so the tokens that stay come out in
// order from a scan of the warps' counts.  It is bound by one SM's integer pipe and shared-memory
// atomics: 19 us for 64 heads of 32768 tokens.  (Passes of one token to a lane and step over all
// tokens took 35, and clusters of four CTAs, whose barriers cost about 1 us each, 32.)
//
// The second kernel takes one warp per destination sub-block and head.  A token's K is one run of
// bytes; its V one byte of each word of a quarter of its sub-block (four tokens share a word), in 16-byte
// pieces, so where neighbours do not stay together, V is mostly read whole: 8 x 32768 tokens to 2048, 8
// heads of 128, move in 40 us, the selection before it takes 19.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "kv4.cuh"
#include "kv8.cuh"
#include "kv8.h"
#include "launch.cuh"

namespace spec {

namespace {

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickKeys = 48 * 1024;  // weights held in shared memory; whole steps of 128
constexpr int kPickList = 2048;

// Orders like the weight; NaN lowest, -0 as 0.
SPEC_DEVICE_INLINE uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

SPEC_DEVICE_INLINE float key_weight(uint32_t k) {
  return k == 0u ? NAN : __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

SPEC_DEVICE_INLINE int seq_tokens(const Kv8EvictParams& p, int b) {
  const long long cap = min((long long)p.max_pages * kPage, p.weight_len);
  return (int)max(0ll, min((long long)p.kv_len[b], cap));
}

// grid (Hkv, B, shares): CTAs of a head find the same threshold, and each writes a share of what comes out.
__global__ void __launch_bounds__(kPickThreads) kv8_pick_kernel(const __grid_constant__ Kv8EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(8) unsigned int hist[2048];
  __shared__ int list[kPickList];       // tokens that share the threshold's first digit
  __shared__ unsigned int wsum[kPickWarps], weq[kPickWarps];
  __shared__ unsigned int s_bin, s_above, s_list;
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long group = (long long)b * p.Hkv + h;
  const float* w = p.weight + group * p.weight_len;
  int32_t* kept = p.kept + group * p.keep;
  float* wout = p.weight_out + group * p.weight_out_len;
  const int n = seq_tokens(p, b), m = min(n, p.keep);
  const int share = blockIdx.z, shares = gridDim.z, me = share * kPickThreads + tid, step = shares * kPickThreads;
  if (h == 0 && me == 0) p.new_len[b] = m;
  for (int i = m + me; i < p.keep; i += step) kept[i] = -1;
  const auto zeros = [&] {  // of 16 bytes where they can be
    const long long a = m + ((16 - (reinterpret_cast<uintptr_t>(wout + m) & 15)) & 15) / 4, e = p.weight_out_len;
    for (long long i = a + 4 * me; i + 4 <= e; i += 4 * step) *reinterpret_cast<float4*>(wout + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m + me < min(a, e)) wout[m + me] = 0.f;
    const long long z = e - 1 - me;  // behind the last 16 bytes
    if (me < 3 && z >= a + (e - a) / 4 * 4) wout[z] = 0.f;
  };
  if (n == m) {
    for (int i = me; i < m; i += step) {
      kept[i] = i;
      wout[i] = w[i];
    }
    zeros();
    return;
  }
  const int last = n - min(p.recent, m);   // tokens [last, n) stay anyway
  const unsigned need = (unsigned)(m - (n - last));
  const bool held = n <= kPickKeys;
  const auto key_at = [&](int i) { return held ? keys[i] : weight_key(w[i]); };
  // keys of tokens i .. i + 3 (i a multiple of 4; anything behind the last)
  const auto keys4 = [&](int i) {
    if (held) return *reinterpret_cast<const uint4*>(&keys[i]);
    return make_uint4(weight_key(w[min(i, n - 1)]), weight_key(w[min(i + 1, n - 1)]), weight_key(w[min(i + 2, n - 1)]),
                      weight_key(w[min(i + 3, n - 1)]));
  };
  uint32_t t = 0xffffffffu;                // threshold: keys above it stay, and `eq` of the `ties` equal to it
  unsigned eq = 0, ties = 0;
  if (need > 0) {
    for (int i = tid; i < 2048; i += kPickThreads) hist[i] = 0;
    if (tid == 0) s_list = 0;
    __syncthreads();
#pragma unroll 16
    for (int i = tid; i < n; i += kPickThreads) {
      const uint32_t k = weight_key(w[i]);
      if (held) keys[i] = k;
      if (i < last) atomicAdd(&hist[k >> 21], 1u);
    }
    uint32_t prefix = 0;
    unsigned left = need;
    int M = -1;                            // tokens of the list; -1: all
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u, mask = pass == 2 ? ~1023u : ~0u << 21;
      if (pass > 0) {
        const auto count = [&](uint32_t k) {
          if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
        };
        if (M >= 0)
          for (int i = tid; i < M; i += kPickThreads) count(key_at(list[i]));
        else
          for (int i = 4 * tid; i < last; i += 4 * kPickThreads) {
            const uint4 k = keys4(i);
            count(k.x);
            if (i + 1 < last) count(k.y);
            if (i + 2 < last) count(k.z);
            if (i + 3 < last) count(k.w);
          }
      }
      __syncthreads();
      // bins from the top: thread i has bins 2047 - 2 i and 2046 - 2 i
      const uint2 c = *reinterpret_cast<const uint2*>(&hist[2046 - 2 * tid]);
      unsigned inc = c.x + c.y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u) + inc - c.x - c.y;
      *reinterpret_cast<uint2*>(&hist[2 * tid]) = make_uint2(0u, 0u);  // for the next pass: all have read theirs
      if (before < left && left <= before + c.y) {
        s_bin = 2047 - 2 * tid, s_above = before, ties = c.y;
        weq[0] = c.y;
      } else if (before + c.y < left && left <= before + c.y + c.x) {
        s_bin = 2046 - 2 * tid, s_above = before + c.y;
        weq[0] = c.x;
      }
      __syncthreads();
      prefix |= s_bin << shift;
      left -= s_above;
      ties = weq[0];
      if (pass == 0 && ties <= kPickList) {  // line them up
        const auto put = [&](uint32_t k, int i) {
          if ((k >> 21) == s_bin && i < last) list[atomicAdd(&s_list, 1u)] = i;
        };
#pragma unroll 2
        for (int i = 4 * tid; i < last; i += 4 * kPickThreads) {
          const uint4 k = keys4(i);
          put(k.x, i), put(k.y, i + 1), put(k.z, i + 2), put(k.w, i + 3);
        }
        M = (int)ties;
      }
      __syncthreads();
    }
    t = prefix;
    eq = left;
  }
  zeros();
  // A warp's run of neighbouring tokens, 128 a step: counts, then places.
  const int run = ((n + kPickWarps - 1) / kPickWarps + 127) & ~127;
  const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
  const bool cut = eq < ties;              // not all of the ties stay: the first ones
  const uint32_t from = cut ? t + 1u : t;  // keys from here on stay
  // which of tokens i .. i + 3 stay anyway, a bit each, and which are the cut ties
  const auto staying = [&](uint4 k, int i) {
    unsigned f = (k.x >= from) | (k.y >= from) << 1 | (k.z >= from) << 2 | (k.w >= from) << 3;
    if (need == 0) f = 0;                  // (the keys were not read)
    if (i + 4 > last) f = ((i < last ? f & ((1u << (last - i)) - 1u) : 0u) | 15u << max(last - i, 0)) & ((1u << min(max(n - i, 0), 4)) - 1u);
    return f;
  };
  const auto tied = [&](uint4 k, int i) {
    const unsigned f = (k.x == t) | (k.y == t) << 1 | (k.z == t) << 2 | (k.w == t) << 3;
    return i < last ? f & ((1u << min(last - i, 4)) - 1u) : 0u;
  };
  // this CTA's steps: tokens [a0, a1) of the run
  const int part = ((r1 - r0 + shares - 1) / shares + 127) & ~127, a0 = min(r1, r0 + share * part), a1 = min(r1, a0 + part);
  unsigned gt = 0, tie = 0, gt0 = 0, tie0 = 0;
#pragma unroll 2
  for (int i = r0 + 4 * lane; i < r1; i += 128) {
    const uint4 k = keys4(i);
    const unsigned c = __popc(staying(k, i)), e = cut ? __popc(tied(k, i)) : 0u;
    gt += c, tie += e;
    if (i < a0) gt0 += c, tie0 += e;
  }
  gt = __reduce_add_sync(0xffffffffu, gt), tie = __reduce_add_sync(0xffffffffu, tie);
  if (lane == 0) wsum[warp] = gt, weq[warp] = tie;
  __syncthreads();
  unsigned at0 = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u);
  unsigned eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? weq[lane] : 0u);
  at0 += __reduce_add_sync(0xffffffffu, gt0), eq0 += __reduce_add_sync(0xffffffffu, tie0);
  at0 += min(eq0, eq);
  // Sum over the lanes before this one of counts up to 4, and (added to `all`) over all lanes.
  const unsigned below = (1u << lane) - 1u;
  const auto ahead = [&](unsigned c, unsigned& all) {
    unsigned sum = all;
#pragma unroll
    for (int b = 0; b < 3; ++b) {
      const unsigned f = __ballot_sync(0xffffffffu, (c >> b) & 1u);
      sum += __popc(f & below) << b, all += __popc(f) << b;
    }
    return sum;
  };
  for (int i0 = a0; i0 < a1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint4 k4 = keys4(i);
    unsigned f = staying(k4, i);
    if (cut) {  // the first of the ties, by their ranks
      unsigned e = tied(k4, i);
      for (unsigned before = ahead(__popc(e), eq0); e && before < eq; e &= e - 1u, ++before) f |= e & -e;
    }
    for (unsigned at = ahead(__popc(f), at0); f; f &= f - 1u, ++at) {
      const int j = __ffs(f) - 1;
      kept[at] = i + j;
      wout[at] = held && need > 0 ? key_weight(keys[i + j]) : w[i + j];
    }
  }
}

// c * 2^d as two exact factors that fp16 has, for |d| <= 23.
struct Shift2 {
  __half2 a, b;
  SPEC_DEVICE_INLINE explicit Shift2(int d)
      : a(__float2half2_rn(kv8_pow2(d / 2))), b(__float2half2_rn(kv8_pow2(d - d / 2))) {}
  SPEC_DEVICE_INLINE uint32_t operator()(uint32_t x) const { return kv8_mul2(kv8_mul2(x, a), b); }
};

// Largest magnitude (a code) of four words.
SPEC_DEVICE_INLINE uint32_t max_code(uint4 v) {
  uint32_t m = __vmaxu4(__vmaxu4(v.x & 0x7f7f7f7fu, v.y & 0x7f7f7f7fu), __vmaxu4(v.z & 0x7f7f7f7fu, v.w & 0x7f7f7f7fu));
  m = __vmaxu4(m, m >> 16);
  return max(m & 0xffu, (m >> 8) & 0xffu);
}
SPEC_DEVICE_INLINE float code_value(uint32_t code) {
  const uint32_t y = kv8_lo(code);
  return __half2float(__ushort_as_half((unsigned short)y));
}

constexpr int kMoveWarps = 4;

// One warp per (sequence, destination sub-block, kv head), heads fastest.
template <int HD>
__global__ void __launch_bounds__(kMoveWarps * 32) kv8_move_kernel(const __grid_constant__ Kv8EvictParams p,
                                                                   long long total) {
  constexpr int SUB = kv8_sub_bytes(HD), BLOCK = kv8_block_bytes(HD), N = HD / 32, CH = HD / 16;
  const int lane = threadIdx.x & 31, c = lane & 3;
  const int subs = (p.keep + kSub - 1) / kSub;
  pdl_wait();
  pdl_launch_dependents();
  for (long long x = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5); x < total;
       x += (long long)gridDim.x * kMoveWarps) {
    const int h = (int)(x % p.Hkv);
    const long long y = x / p.Hkv;
    const int s = (int)(y % subs), b = (int)(y / subs);
    const int m = min(seq_tokens(p, b), p.keep);
    if (s * kSub >= m) continue;
    const int dpage = s / 4 < p.dst_pages ? p.dst_table[(long long)b * p.dst_pages + s / 4] : -1;
    if (dpage < 0 || dpage >= p.num_pages) continue;
    uint8_t* const dst = p.pool + ((long long)dpage * p.Hkv + h) * BLOCK + (s & 3) * SUB;
    // lane t < 16: token t of the sub-block: its cell (page * 64 + token of the page), or -1
    long long cell = -1;
    uint32_t par = 0;
    if (lane < kSub && s * kSub + lane < m) {
      const int i = p.kept[((long long)b * p.Hkv + h) * p.keep + s * kSub + lane];
      const int pg = p.page_table[(long long)b * p.max_pages + i / kPage];
      if (pg >= 0 && pg < p.num_pages) {
        cell = (long long)pg * kPage + i % kPage;
        par = *reinterpret_cast<const uint32_t*>(p.pool + ((long long)pg * p.Hkv + h) * BLOCK + (i % kPage / kSub) * SUB +
                                                 2 * kSub * HD);
      }
    }
    const auto source = [&](long long cl) { return p.pool + ((cl >> 6) * p.Hkv + h) * BLOCK + ((cl & 63) >> 4) * SUB; };
    int e[2];
    {  // K: chunk id % CH of token id / CH
      uint4 v[N];
      int es[N];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i, t = id / CH, j = id % CH;
        const long long cl = __shfl_sync(0xffffffffu, cell, t);
        es[i] = kv8_exp(__shfl_sync(0xffffffffu, par, t), 0);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (cl >= 0) v[i] = *reinterpret_cast<const uint4*>(source(cl) + kv8_k_chunk<HD>((int)(cl & 15), j));
      }
#pragma unroll
      for (int i = 0; i < N; ++i) a = fmaxf(a, code_value(max_code(v[i])) * kv8_pow2(es[i]));
      e[0] = kv8_needed_exp(warp_max(a));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = lane + 32 * i, t = id / CH, j = id % CH;
        const Shift2 f(es[i] - e[0]);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = kv8_codes(f(kv8_lo(w[k])), f(kv8_hi(w[k])));
        *reinterpret_cast<uint4*>(dst + kv8_k_chunk<HD>(t, j)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    {  // V: this lane's dims of tokens 2c, 2c + 1, 2c + 8, 2c + 9
      uint4 v[4][N];
      int es[4], sel[4];
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 2 * c + (i & 1) + (i >> 1) * 8;
        const long long cl = __shfl_sync(0xffffffffu, cell, t);
        es[i] = kv8_exp(__shfl_sync(0xffffffffu, par, t), 1);
        const int ts = (int)(cl & 15), from = (lane & ~3) | ((ts & 7) >> 1);
        sel[i] = (ts >> 3) * 2 + (ts & 1);           // the token's byte of a word
#pragma unroll
        for (int j = 0; j < N; ++j) {
          v[i][j] = make_uint4(0u, 0u, 0u, 0u);
          if (cl >= 0) v[i][j] = *reinterpret_cast<const uint4*>(source(cl) + kv8_v_chunk<HD>(j, from));
        }
      }
      uint32_t b4[4][N];                             // that byte of each of a chunk's words
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pr = sel[i] | (sel[i] + 4) << 4;
        uint32_t mc = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t lo = __byte_perm(v[i][j].x, v[i][j].y, pr), hi = __byte_perm(v[i][j].z, v[i][j].w, pr);
          b4[i][j] = __byte_perm(lo, hi, 0x5410);
          mc = __vmaxu4(mc, b4[i][j] & 0x7f7f7f7fu);
        }
        a = fmaxf(a, code_value(max_code(make_uint4(mc, 0u, 0u, 0u))) * kv8_pow2(es[i]));
      }
      e[1] = kv8_needed_exp(warp_max(a));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Shift2 f(es[i] - e[1]);
#pragma unroll
        for (int j = 0; j < N; ++j) b4[i][j] = kv8_codes(f(kv8_lo(b4[i][j])), f(kv8_hi(b4[i][j])));
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                // dim 4 j + k of the four tokens
          const uint32_t pr = k | (k + 4) << 4;
          o[k] = __byte_perm(__byte_perm(b4[0][j], b4[1][j], pr), __byte_perm(b4[2][j], b4[3][j], pr), 0x5410);
        }
        *reinterpret_cast<uint4*>(dst + kv8_v_chunk<HD>(j, lane)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (lane == 0) *reinterpret_cast<uint4*>(dst + 2 * kSub * HD) = make_uint4(kv8_param_word(e[0], e[1]), 0u, 0u, 0u);
  }
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8EvictParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1ull)) {
    e = cudaFuncSetAttribute(kv8_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPickKeys * 4);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  const long long most = std::min((long long)p.max_pages * kPage, p.weight_len);
  // whole steps of 128 tokens: a warp's last step reads past the last one
  const size_t smem = (size_t)std::min<long long>((most + 127) & ~127ll, kPickKeys) * 4;
  int sms = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // two CTAs to a head of many tokens where that leaves none waiting (64 heads of 32768 tokens to 2048
  // take 2.4 us less than with one each; nothing is won where few tokens come out)
  const int shares = most > 8192 && (long long)p.Hkv * p.B * 2 <= sms ? 2 : 1;
  e = launch_k(kv8_pick_kernel, dim3(p.Hkv, p.B, shares), dim3(kPickThreads), smem, st, p);
  if (e != cudaSuccess) return e;
  const long long total = (long long)p.B * p.Hkv * ((p.keep + kSub - 1) / kSub);
  const long long ctas = (total + kMoveWarps - 1) / kMoveWarps;
  const unsigned grid = (unsigned)std::min<long long>(ctas, 1ll << 30);
  return p.hd == 128 ? launch_k(kv8_move_kernel<128>, dim3(grid), dim3(kMoveWarps * 32), 0, st, p, total)
                     : launch_k(kv8_move_kernel<64>, dim3(grid), dim3(kMoveWarps * 32), 0, st, p, total);
}

}  // namespace spec
