// Sampling of one token per logits row, and the distribution it was drawn from.
//
// With the row's largest logit m and x_v = (l_v - m) / T, a token's mass is the whole number
//   R_v = floor(2^40 e^x_v),
// sums of masses are exact, and every decision after it is integer arithmetic, which
// does not depend on the order of the sums: as in the acceptance kernels, a draw takes
// the first token whose running kept sum exceeds floor(floor(2^24 u) Z / 2^24).  Ranked
// by logit (equal ones: the lower index first) the kept tokens are the shortest of three
// prefixes: the first top_k; those whose masses reach top_p of the top-k's sum; those
// with R_v >= min_p 2^40.  q_v = R_v / Z.
//
// The mass has 40 bits behind the point, where fp32's e^x has 24: a draw from a row of
// 128256 tokens compares u Z with running sums whose neighbours lie as near as the tails'
// masses, and masses good to 2^-24 move one draw in some ten thousand to another token.
// l - m, its product with log2(e) / T, 2^(-i/256) (a table) and what is left of the
// exponential are pairs of floats, good to about 2^-42, and the mass is taken from the last
// pair in two parts of 20 bits: 70 issue cycles per warp, nearly all fp32, which runs at twice
// the integer pipe's rate here.  (With a table in whole numbers and 64-bit shifts the same took
// 150; fp64 runs at 1/64 of fp32's rate.)
//
// A row is one thread-block cluster, its slices in shared memory, read from HBM once.  What
// can be kept is often a few hundred tokens, and is found without a mass per token:
//   top_k   the k-th largest of the threads' own maxima is a lower bound of the k-th logit;
//           a histogram of those maxima, in bins 1/16 wide in x, gives its bin
//   min_p   x >= log(min_p)
//   top_p   (alone) the histogram of all masses, in the same bins
// The tokens down to that bin, the candidates, go to one CTA, which ranks them and takes
// every decision on its own, exactly.  Where there are more than 1024 of them (or top_k is
// above 512) only the threshold's bin goes to that CTA, which sends back the threshold, and
// all CTAs sum up what is kept; a bin of more than 1024 tokens is first cut finer, by
// histograms over its logits (as ordered integers).  Bins go through distributed shared
// memory, each CTA adding up its share of them.
//
// A small top_k needs no more than each CTA's own maxima: its tokens down to the bin of its own
// k-th largest go to the first CTA at once, after one barrier.
//
// Up to 128 candidates are ranked by comparing each with each; more are sorted, or first cut down
// by a histogram of the candidates alone.
//
// What bounds it: chains of short steps (cluster barriers of 0.8 us, instructions fetched once per
// row), not bytes.  GPU us against the bytes at the copy rate: 1 x 128256 fp32 with top_p 22.6 (0.08),
// 64 x 128256 fp32 with top_k, top_p and q 28.2 (9.7), 256 x 50257 bf16, settings per row, 73 (3.8): there
// the 51 rows without top_k, a mass and four shared atomics per token on two CTAs each, which run on when
// the others have ended (the 51 alone take 45, the 205 others alone 38; with the 51 first the batch takes
// 61).  Decisions by histograms of all CTAs alone, without
// candidates, took 41, 111 and 340; sorting every list of candidates 27.6, 33.7 and 88.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "launch.cuh"
#include "sample.h"

namespace cg = cooperative_groups;

namespace spec {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;          // a thread per bin
constexpr int kMaxCluster = 16;          // of few rows; 8 else (portable)
constexpr int kMaxSlice = 48 * 1024;     // logits of a CTA (shared memory)
constexpr float kBinsPerUnit = 16.f;     // bins of x in the first histogram
constexpr int kBatch = 4;                // tokens of a thread under way at once
constexpr int kCand = 1024;              // candidates that one CTA sorts
constexpr int kCandK = kCand / 2;        // largest top_k that is tried so
constexpr int kFew = kThreads / 4;       // candidates that are ranked by comparing each with each

// Temperatures for which log2(e) / T is a pair of normal floats, and T's steps are fp32's.
constexpr float kMinTemp = 1e-6f, kMaxTemp = 1e30f;

// 2^(-i/256) as a pair of floats, by the exponential series.
struct Pow2Table {
  float2 v[256];
};
constexpr Pow2Table make_pow2_table() {
  Pow2Table t{};
  for (int i = 0; i < 256; ++i) {
    const double x = -0.69314718055994530942 * i / 256.0;
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 30; ++k) {
      term *= x / k;
      sum += term;
    }
    t.v[i].x = (float)sum;
    t.v[i].y = (float)(sum - (double)t.v[i].x);
  }
  return t;
}
__device__ const Pow2Table kPow2 = make_pow2_table();

struct Bins {
  unsigned int cnt[kBins], m0[kBins], m1[kBins], m2[kBins];  // this CTA's histogram; a mass in three parts
  unsigned int gc[kBins];                                    // the cluster's
  unsigned long long gm[kBins];
};
struct Shared {
  float2 pow2[256];
  Bins h;
  unsigned long long key[kCand];                             // candidates (the first CTA's)
  unsigned long long part[8][kMaxCluster];                   // exchanges: one value of each CTA
  unsigned long long warp[kWarps], warp2[kWarps];
  unsigned long long found, tau, upto;
  int pick;
  unsigned int cand[2];                                      // candidates in the first CTA, of this and the next time
  unsigned int picked, place;                                // candidates of this CTA, and their place there
};

// A mass <= 2^40, as a 2^20 + b, in parts of 14, 13 and 14 bits: over a slice's at most 48 * 1024
// tokens each part's sum stays below 2^30.
struct Parts {
  unsigned lo, mid, hi;
  SPEC_DEVICE_INLINE Parts(int a, int b) {
    const unsigned v = (unsigned)((b >> 14) + (a << 6));
    lo = (unsigned)b & 0x3fffu, mid = v & 0x1fffu, hi = v >> 13;
  }
};
SPEC_DEVICE_INLINE unsigned long long joined(unsigned a, unsigned b, unsigned c) {
  return (unsigned long long)a + ((unsigned long long)b << 14) + ((unsigned long long)c << 27);
}
SPEC_DEVICE_INLINE unsigned long long whole(long long a, long long b) { return (unsigned long long)((a << 20) + b); }

SPEC_DEVICE_INLINE uint32_t order_key(float l) {  // orders like l, -0 as 0
  const uint32_t b = __float_as_uint(l + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
SPEC_DEVICE_INLINE float key_logit(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

struct Row {
  float mx;          // largest logit, finite
  float ch, cl;      // log2(e) / T
  float bin;         // kBinsPerUnit / T
  const float2* pow2;

  // Bin of x: never falls as l falls.
  SPEC_DEVICE_INLINE int bin_of(float l) const {
    return __float_as_int(__fadd_rd(fminf((mx - l) * bin, (float)(kBins - 1)), 8388608.f)) - 0x4b000000;
  }

  // R = a 2^20 + b, |b| <= 2^19.  Without a branch, so that several can be under way.
  SPEC_DEVICE_INLINE void mass_parts(float l, int& a, int& b) const {
    const float dh = mx - l;
    const float yh = dh * ch;
    const float bb = dh - mx;
    const float dl = (mx - (dh - bb)) - (l + bb);           // what dh lost
    const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
    const float t = fmaf(yh, 256.f, 12582912.f);
    const int k = __float_as_int(t) - 0x4b400000;           // 256 y, rounded
    const float fh = fmaf(t - 12582912.f, -0.00390625f, yh);
    // r = -(fh + yl) ln 2 as a pair, e^r - 1 = r + r^2 (1/2 + r/6 + r^2/24), |r| < 2^-9
    const float rh = fh * -0.693147182464599609375f;
    const float rl = fmaf(fh, -0.693147182464599609375f, -rh) +
                     fmaf(yl, -0.693147182464599609375f, fh * 1.90465429995776804525e-9f);
    const float q = fmaf(rh * rh, fmaf(rh, fmaf(rh, 0.0416666667f, 0.16666667f), 0.5f), rl);
    // 2^(-i/256) (1 + rh + q) as a pair, times 2^-n
    const float2 p = pow2[k & 255];
    const float z = p.x * rh;
    const float lo = fmaf(p.x, q, fmaf(p.x, rh, -z) + fmaf(p.y, rh, p.y));
    const float s = __int_as_float(0x3f800000 - (k & ~255) * 32768);
    const float wh = (p.x + z) * s, wl = ((z - ((p.x + z) - p.x)) + lo) * s;
    const float ta = fmaf(wh, 1048576.f, 8388608.f);        // 2^20 w, rounded
    const bool some = yh < 41.f;                            // 2^-41 and less: no mass
    a = some ? __float_as_int(ta) - 0x4b000000 : 0;
    b = some ? __float_as_int(__fadd_rd((fmaf(ta - 8388608.f, -9.5367431640625e-7f, wh) + wl) * 1099511627776.f, 12582912.f)) - 0x4b400000 : 0;
  }
  SPEC_DEVICE_INLINE unsigned long long mass(float l) const {
    int a, b;
    mass_parts(l, a, b);
    return whole(a, b);
  }
};

// Most of the kernel runs once per row, so its time is much that of fetching its instructions: what
// is used in several places is a function, and loops without parallel work are not unrolled.

SPEC_DEVICE_INLINE unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __noinline__ unsigned long long block_sum64(unsigned long long v, unsigned long long* w) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum64((threadIdx.x & 31) < kWarps ? w[threadIdx.x & 31] : 0ull);
}

// Sum over the CTA's threads before this one.
__device__ __noinline__ unsigned long long block_before64(unsigned long long v, unsigned long long* w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) w[warp] = inc;
  __syncthreads();
  return warp_sum64(lane < warp ? w[lane] : 0ull) + inc - v;
}

// M <= kCand keys sorted, the largest first: thread i gets those at 2 i and 2 i + 1 (0 behind the
// last).  Bitonic: partners up to 32 apart are in one warp and are exchanged in registers.
struct Two {
  unsigned long long x0, x1;
};
__device__ __noinline__ Two sorted_keys(unsigned long long* key, int M) {
  int P = 64;
  while (P < M) P *= 2;
  const int e = 2 * threadIdx.x;
  unsigned long long x0 = e < M ? key[e] : 0ull, x1 = e + 1 < M ? key[e + 1] : 0ull;
  const bool on = P > 64 || threadIdx.x < 32;  // the first warp holds all, if they are few
  __syncthreads();
#pragma unroll 1
  for (int k = 2; k <= P; k *= 2) {
    const bool down = (e & k) == 0;
    int j = k / 2;
#pragma unroll 1
    for (; j >= 64; j /= 2) {
      key[e] = x0, key[e + 1] = x1;
      __syncthreads();
      const unsigned long long y0 = key[e ^ j], y1 = key[(e + 1) ^ j];
      const bool most = ((e & j) == 0) == down;
      x0 = (x0 > y0) == most ? x0 : y0;
      x1 = (x1 > y1) == most ? x1 : y1;
      __syncthreads();
    }
    if (on) {
#pragma unroll 1
      for (; j >= 2; j /= 2) {
        const unsigned long long y0 = __shfl_xor_sync(0xffffffffu, x0, j / 2), y1 = __shfl_xor_sync(0xffffffffu, x1, j / 2);
        const bool most = ((e & j) == 0) == down;
        x0 = (x0 > y0) == most ? x0 : y0;
        x1 = (x1 > y1) == most ? x1 : y1;
      }
      const unsigned long long y0 = x0;
      x0 = (x0 > x1) == down ? x0 : x1;
      x1 = (y0 > x1) == down ? x1 : y0;
    }
  }
  return Two{x0, x1};
}

// Among M <= kFew keys with measures m, four threads to one key x: how many are larger, their
// measures' sum, and that of all.  (Sorting 64 keys takes 2.5 K cycles, this 0.5 K.)
struct Ranked {
  unsigned long long before, total;
  int above;
};
__device__ __noinline__ Ranked ranked(const unsigned long long* key, const unsigned long long* m, int M, unsigned long long x) {
  Ranked r{0ull, 0ull, 0};
#pragma unroll 4
  for (int j = threadIdx.x & 3; j < M; j += 4) {
    const unsigned long long v = m[j];
    const bool more = key[j] > x;
    r.total += v;
    r.before += more ? v : 0ull;
    r.above += more;
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    r.total += __shfl_xor_sync(0xffffffffu, r.total, o);
    r.before += __shfl_xor_sync(0xffffffffu, r.before, o);
    r.above += __shfl_xor_sync(0xffffffffu, r.above, o);
  }
  return r;
}

// What is kept: logits above the threshold, and of those equal to it the tokens up to cut.
struct Kept {
  float t;
  int cut;
  SPEC_DEVICE_INLINE bool has(float l, int v) const { return l > t || (l == t && v <= cut); }
};

template <typename T>
SPEC_DEVICE_INLINE float to_f32(T x);
template <>
SPEC_DEVICE_INLINE float to_f32<float>(float x) { return x; }
template <>
SPEC_DEVICE_INLINE float to_f32<__half>(__half x) { return __half2float(x); }
template <>
SPEC_DEVICE_INLINE float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
SPEC_DEVICE_INLINE T from_f32(float x);
template <>
SPEC_DEVICE_INLINE float from_f32<float>(float x) { return x; }
template <>
SPEC_DEVICE_INLINE __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
SPEC_DEVICE_INLINE __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / cs;
  const int V = p.V, set = (int)(row / p.rows_per_setting);
  const int slice = (V + cs - 1) / cs, s0 = min(V, rank * slice), n = min(V, s0 + slice) - s0;

  if (tid < 256) sh.pow2[tid] = kPow2.v[tid];
  if (tid < 2) sh.cand[tid] = 0;
  cluster_arrive();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_launch_dependents();

  const float temp = p.temperature ? p.temperature[set] : p.temperature_all;
  const int K = p.top_k ? p.top_k[set] : 0;
  const float TP = p.top_p ? p.top_p[set] : 1.f, MP = p.min_p ? p.min_p[set] : 0.f;
  const float u = temp == 0.f ? 0.f : p.u[row];
  const bool bad = !(temp == 0.f || (temp >= kMinTemp && temp <= kMaxTemp)) || K < 0 || !(TP > 0.f && TP <= 1.f) ||
                   !(MP >= 0.f && MP <= 1.f) || !(u >= 0.f && u < 1.f);

  // The slice, as it is, in 16-byte copies (its place in shared memory is as far off a 16-byte
  // boundary as its address), and the thread's largest logit.
  constexpr int PER = 16 / sizeof(T);
  const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + s0;
  const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  const int head = min(n, ((16 - off) & 15) / (int)sizeof(T));
  T* const val = reinterpret_cast<T*>(smem + off);
  const auto logit = [&](int i) { return fmaxf(to_f32(val[i]), -INFINITY); };  // NaN counts as -infinity
  const int vecs = (n - head) / PER, tail0 = head + vecs * PER;
  float own = -INFINITY;
  auto put = [&](int i) {
    val[i] = src[i];
    own = fmaxf(own, to_f32(val[i]));  // fmaxf passes over NaN
  };
  if (tid < head) put(tid);
  if (tid < n - tail0) put(tail0 + tid);
  constexpr int UN = 4;  // pieces at once
  for (int j0 = tid; j0 < vecs; j0 += UN * kThreads) {
    uint4 w[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (j0 + k * kThreads < vecs) w[k] = __ldcs(reinterpret_cast<const uint4*>(src + head) + j0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (j0 + k * kThreads < vecs) {
        reinterpret_cast<uint4*>(val + head)[j0 + k * kThreads] = w[k];
        const T* e = reinterpret_cast<const T*>(&w[k]);
#pragma unroll
        for (int i = 0; i < PER; ++i) own = fmaxf(own, to_f32(e[i]));
      }
  }

  // f(i, logit of i) for the slice's tokens from least_l to most_l, read in 16-byte pieces.
  const auto each_in = [&](float least_l, float most_l, auto f) {
    const auto is = [&](T e) {
      const float l = fmaxf(to_f32(e), -INFINITY);
      return l >= least_l && l <= most_l;
    };
    // tokens of the pieces j, j + kThreads, ..: a bit each
    const auto each = [&](int j, unsigned hits) {
#pragma unroll 1
      for (; hits; hits &= hits - 1) {
        const int b = __ffs(hits) - 1, at = head + (j + b / PER * kThreads) * PER + b % PER;
        f(at, logit(at));
      }
    };
#pragma unroll 1
    for (int j = tid; j < vecs; j += UN * kThreads) {
      unsigned m = 0;
#pragma unroll
      for (int k = 0; k < UN; ++k)
        if (j + k * kThreads < vecs) {
          const uint4 w = reinterpret_cast<const uint4*>(val + head)[j + k * kThreads];
          const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
          for (int i = 0; i < PER; ++i) m |= is(e[i]) ? 1u << (k * PER + i) : 0u;
        }
      each(j, m);
    }
    // what lies around the pieces: the first threads before, the last ones behind them
    const int i = tid < kThreads / 2 ? tid : tail0 + (kThreads - 1 - tid);
    if ((tid < head || (tid >= kThreads / 2 && i < n)) && is(val[i])) f(i, logit(i));
  };

  // Exchange number xchg: one 64-bit value of every CTA, read after a cluster barrier.  A
  // number comes up again only after at least six barriers.
  int xchg = 0;
  auto give = [&](unsigned long long v) {
    if (tid < cs) *cluster.map_shared_rank(&sh.part[xchg][rank], tid) = v;
  };
  float mx = warp_max(own);  // this CTA's, for now
  if (lane == 0) sh.warp[warp] = __float_as_uint(mx);
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, __uint_as_float((uint32_t)sh.warp[i]));
  cluster_wait();

  float* const probs = p.probs ? p.probs + row * V + s0 : nullptr;
  auto fill = [&](auto q) {
    if (probs)
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) probs[i] = q(i);
  };

  auto zero_probs = [&] {
    if (!probs) return;
    const int h = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(probs) & 15)) & 15) / 4), vec = (n - h) / 4;
    if (tid < h) probs[tid] = 0.f;
    for (int i = tid; i < vec; i += kThreads) reinterpret_cast<float4*>(probs + h)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tid < n - h - vec * 4) probs[h + vec * 4 + tid] = 0.f;
  };

  Row R;
  R.mx = mx;
  R.ch = __fdiv_rn(1.44269502162933349609375f, temp);   // log2(e) is this + 1.92596299e-8
  R.cl = __fdiv_rn(fmaf(-R.ch, temp, 1.44269502162933349609375f) + 1.92596299112661746887e-8f, temp);
  R.bin = kBinsPerUnit / temp;
  R.pow2 = sh.pow2;

  // The cluster's bins, from every CTA's (cnt alone, summed in 64 bits, or with masses), into gc
  // and gm of all; each CTA adds up its share.
  enum { kCounts, kMasses };
  auto reduce_bins = [&](int what) {
    cluster.sync();
    // a thread for each bin of this CTA's share and each CTA: neighbours add up
    const int r = tid % cs, bin = rank * (kBins / cs) + tid / cs;
    Shared* const o = cluster.map_shared_rank(&sh, r);
    unsigned long long gc = o->h.cnt[bin], gm = 0;
    if (what == kMasses) gm = joined(o->h.m0[bin], o->h.m1[bin], o->h.m2[bin]);
    for (int k = cs / 2; k > 0; k /= 2) {
      gc += __shfl_xor_sync(0xffffffffu, gc, k);
      gm += __shfl_xor_sync(0xffffffffu, gm, k);
    }
    o->h.gc[bin] = (unsigned)gc;
    o->h.gm[bin] = what == kMasses ? gm : gc;
    cluster.sync();
  };
  auto sum_given = [&] {
    unsigned long long s = 0;
    for (int r = 0; r < cs; ++r) s += sh.part[xchg][r];
    xchg = xchg == 7 ? 1 : xchg + 1;
    return s;
  };
  // One histogram pass over the slice's tokens that `cls` gives a bin >= 0, with their masses
  // a 2^20 + b; the cluster's bins end up in gc and gm, and the sum of all masses in `total`.
  auto histogram = [&](bool masses, unsigned long long& total, auto cls) {
    sh.h.cnt[tid] = sh.h.m0[tid] = sh.h.m1[tid] = sh.h.m2[tid] = 0;
    __syncthreads();
    long long sum_a = 0, sum_b = 0;
    for (int i0 = tid; i0 < n; i0 += kBatch * kThreads) {
      int a[kBatch], m[kBatch], bin[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = min(i0 + k * kThreads, n - 1);
        a[k] = m[k] = 0;
        bin[k] = cls(i, logit(i), a[k], m[k]);
        if (i0 + k * kThreads >= n) a[k] = m[k] = 0, bin[k] = -1;
      }
      int ta = 0, tb = 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ta += a[k], tb += m[k];
        if (bin[k] >= 0) {
          atomicAdd(&sh.h.cnt[bin[k]], 1u);
          if (masses) {
            const Parts q(a[k], m[k]);
            atomicAdd(&sh.h.m0[bin[k]], q.lo);
            atomicAdd(&sh.h.m1[bin[k]], q.mid);
            atomicAdd(&sh.h.m2[bin[k]], q.hi);
          }
        }
      }
      sum_a += ta, sum_b += tb;
    }
    const unsigned long long sum = whole(sum_a, sum_b);
    if (masses) give(block_sum64(sum, sh.warp));
    reduce_bins(masses ? kMasses : kCounts);
    if (masses) total = sum_given();
  };

  // The first bin where the running measure (counts, or masses), `base` so far, reaches
  // `target`; -1: none does.
  struct Found {
    int bin;
    unsigned int count;
    unsigned long long size, above;  // the bin's measure; base and what lies above the bin
    unsigned int upto;               // tokens of the histogram down to the bin
  };
  auto find = [&](bool by_mass, unsigned long long base, unsigned long long target) {
    const unsigned long long mine = by_mass ? sh.h.gm[tid] : (unsigned long long)sh.h.gc[tid];
    if (tid == 0) sh.pick = -1;
    const unsigned long long before = base + block_before64(mine, sh.warp);
    if (before < target && target <= before + mine) {
      sh.pick = tid;
      sh.found = before;
    }
    const unsigned long long upto = sh.h.gc[tid] + block_before64(sh.h.gc[tid], sh.warp);
    if (tid == sh.pick) sh.upto = upto;
    __syncthreads();
    Found f;
    f.upto = (unsigned)sh.upto;
    f.bin = sh.pick;
    f.count = sh.h.gc[max(f.bin, 0)];
    f.size = by_mass ? sh.h.gm[max(f.bin, 0)] : f.count;
    f.above = sh.found;
    __syncthreads();
    return f;
  };

  // The least key in a bin of the first histogram up to b: 32 tries at a time.
  auto first_key = [&](int b) {
    uint32_t a = order_key(-INFINITY), z = order_key(R.mx);  // z is in bin 0
    while (a < z) {
      const uint32_t step = (z - a) / 32 + 1;
      const unsigned long long m = (unsigned long long)a + (unsigned long long)lane * step;
      const unsigned in = __ballot_sync(0xffffffffu, m >= z || R.bin_of(key_logit((uint32_t)m)) <= b);
      const int l = in ? __ffs(in) - 1 : 32;
      const unsigned long long hi = (unsigned long long)a + (unsigned long long)l * step;
      if (l > 0) a = a + (uint32_t)(l - 1) * step + 1u;
      if (hi < z) z = (uint32_t)hi;
    }
    return z;
  };
  auto bin_bounds = [&](int b, uint32_t& lo, uint32_t& hi) {
    lo = first_key(b);
    hi = b > 0 ? first_key(b - 1) - 1u : order_key(R.mx);
  };

  // Below every logit of the bins up to b, and above every one of the bins from b on: the bins'
  // bounds, by more than bin_of's roundings.
  auto bin_floor = [&](int b) {
    const float d = (float)(b + 1) / R.bin;
    return b < kBins - 1 ? R.mx - d - (fabsf(R.mx) + d) * 0x1p-20f : -INFINITY;
  };
  auto bin_ceil = [&](int b) {
    const float d = (float)b / R.bin;
    return R.mx - d + (fabsf(R.mx) + d) * 0x1p-20f;
  };

  Shared* const first = cluster.map_shared_rank(&sh, 0);
  // The keys of this CTA's tokens from least_l to most_l that `is` picks (order of the logit, then the
  // lower index first) into the first CTA's list, in any order, as far as it and this CTA's own list, in the
  // bins' place, go; how many there were.
  unsigned long long* const local = reinterpret_cast<unsigned long long*>(&sh.h);
  static_assert(sizeof(Bins) >= kCand * sizeof(unsigned long long), "lists in the bins' place");
  int sent = 0;
  auto send = [&](float least_l, float most_l, auto is) {
    __syncthreads();  // the bins have been read
    if (tid == 0) sh.picked = 0, sh.cand[(sent + 1) & 1] = 0;
    __syncthreads();
    each_in(least_l, most_l, [&](int i, float x) {
      if (is(i, x)) {
        const unsigned at = atomicAdd(&sh.picked, 1u);
        if (at < kCand) local[at] = (unsigned long long)order_key(x) << 32 | (0xffffffffu - (unsigned)(s0 + i));
      }
    });
    __syncthreads();
    const unsigned mine = sh.picked;
    if (mine > 0 && mine <= kCand) {
      if (tid == 0) sh.place = atomicAdd(&first->cand[sent & 1], mine);
      __syncthreads();
      const unsigned at = sh.place;
      for (int i = tid; i < mine && at + i < kCand; i += kThreads) first->key[at + i] = local[i];
    }
    ++sent;
    return mine;
  };
  // All CTAs' such tokens: how many there were, and, if at most kCand, all their keys.
  auto gather = [&](float least_l, float most_l, auto is) {
    give(send(least_l, most_l, is));
    cluster.sync();
    return sum_given();
  };
  unsigned long long* const mass = reinterpret_cast<unsigned long long*>(&sh.h);  // the first CTA's, in the bins' place
  static_assert(sizeof(Bins) >= (kCand + 2 * kFew) * sizeof(unsigned long long), "masses of candidates");
  // The candidate (its key) among the M in the first CTA whose measure, `before` lying ahead of them all,
  // completes target; to all CTAs' sh.found.
  auto last_kept = [&](bool by_mass, unsigned long long target, unsigned long long before, int M) {
    const auto measure = [&](unsigned long long key) {
      return key == 0ull ? 0ull : by_mass ? R.mass(key_logit((uint32_t)(key >> 32))) : 1ull;
    };
    const auto tell = [&](unsigned long long key, unsigned long long b, unsigned long long m) {
      if (b < target && target <= b + m)
        for (int r = 0; r < cs; ++r) cluster.map_shared_rank(&sh, r)->found = key;
    };
    if (M > kFew) {  // only those of a finer bin
      const unsigned long long k[2] = {tid < M ? sh.key[tid] : 0ull, tid + kThreads < M ? sh.key[tid + kThreads] : 0ull};
      const unsigned h0 = (unsigned)(k[0] >> 32), h1 = (unsigned)(k[1] >> 32);
      const unsigned most = __reduce_max_sync(0xffffffffu, max(h0, h1));
      const unsigned fell = __reduce_max_sync(0xffffffffu, max(k[0] ? ~h0 : 0u, k[1] ? ~h1 : 0u));
      if (lane == 0) sh.warp[warp] = (unsigned long long)most << 32 | fell;
      sh.h.cnt[tid] = sh.h.m0[tid] = sh.h.m1[tid] = sh.h.m2[tid] = 0;
      if (tid == 0) sh.picked = 0;
      __syncthreads();
      const unsigned long long w = lane < kWarps ? sh.warp[lane] : 0ull;
      const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(w >> 32)), lo = ~__reduce_max_sync(0xffffffffu, (unsigned)w);
      const int sft = max(0, 32 - __clz(hi - lo) - 9);
      int bin[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        bin[i] = k[i] ? (int)((hi - (i ? h1 : h0)) >> sft) : -1;
        if (!k[i]) continue;
        if (by_mass) {
          int a, b;
          R.mass_parts(key_logit(i ? h1 : h0), a, b);
          const Parts q(a, b);
          atomicAdd(&sh.h.m0[bin[i]], q.lo);
          atomicAdd(&sh.h.m1[bin[i]], q.mid);
          atomicAdd(&sh.h.m2[bin[i]], q.hi);
        } else {
          atomicAdd(&sh.h.m0[bin[i]], 1u);
        }
      }
      __syncthreads();
      const unsigned long long here = joined(sh.h.m0[tid], sh.h.m1[tid], sh.h.m2[tid]);
      const unsigned long long ahead = before + block_before64(here, sh.warp);
      if (ahead < target && target <= ahead + here) sh.pick = tid, sh.found = ahead;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (bin[i] == sh.pick) sh.key[atomicAdd(&sh.picked, 1u)] = k[i];
      before = sh.found;
      __syncthreads();
      M = (int)sh.picked;
    }
    if (M <= kFew) {
      const unsigned long long x = tid / 4 < M ? sh.key[tid / 4] : 0ull, m = measure(x);
      if (tid % 4 == 0 && x) mass[tid / 4] = m;
      __syncthreads();
      const Ranked r = ranked(sh.key, mass, M, x);
      if (tid % 4 == 0) tell(x, before + r.before, m);
      return;
    }
    const Two k = sorted_keys(sh.key, M);
    const unsigned long long m0 = measure(k.x0), m1 = measure(k.x1);
    before += block_before64(m0 + m1, sh.warp);
    tell(k.x0, before, m0);
    tell(k.x1, before + m0, m1);
  };
  // The shortest prefix (by rank) of the tokens of `in` whose measure reaches target, from the
  // bin of their first histogram that holds its end.
  auto select = [&](bool by_mass, unsigned long long target, const Kept& in, Found f) -> Kept {
    const int coarse = f.bin;
    uint32_t lo = 0, hi = 0;  // the bin's keys, once they are needed
    bool known = false;
    const auto bounds = [&] {
      if (!known) bin_bounds(coarse, lo, hi);
      known = true;
    };
    while (true) {
      if (f.above + f.size == target) {  // all of the bin
        bounds();
        return key_logit(lo) > in.t ? Kept{key_logit(lo), V} : in;
      }
      const bool exact = known;
      const uint32_t l = lo, h = hi;
      // by keys: as floats, 0 would lie in a range that ends at -0
      const auto inside = [&](int i, float x) {
        const uint32_t key = order_key(x);
        return (exact ? key >= l && key <= h : R.bin_of(x) == coarse) && in.has(x, s0 + i);
      };
      if (f.count <= kCand) {
        // (top_p's bins leave out tokens of no mass, which lie inside too)
        const unsigned long long M =
            gather(exact ? key_logit(l) : bin_floor(coarse), exact ? key_logit(h) : bin_ceil(coarse), inside);
        if (M <= kCand) {
          if (rank == 0) last_kept(by_mass, target, f.above, (int)M);
          cluster.sync();
          const unsigned long long end = sh.found;
          __syncthreads();
          return Kept{key_logit((uint32_t)(end >> 32)), (int)(0xffffffffu - (uint32_t)end)};
        }
      }
      if (!exact) {
        bounds();
        continue;
      }
      if (l == h) break;
      const int sft = max(0, 32 - __clz(h - l) - 9);  // (h - l) >> sft < 512
      unsigned long long sum;
      histogram(by_mass, sum, [&](int i, float x, int& a, int& b) {
        if (!inside(i, x)) return -1;
        if (by_mass) R.mass_parts(x, a, b);
        return (int)((h - order_key(x)) >> sft);
      });
      f = find(by_mass, f.above, target);
      hi = h - ((uint32_t)f.bin << sft);
      lo = hi - l < (1u << sft) ? l : hi - ((1u << sft) - 1u);
    }
    // many equal logits: as many of the first as are needed
    unsigned long long need = target - f.above;
    if (by_mass) {
      const unsigned long long m = R.mass(key_logit(lo));
      need = (need + m - 1) / m;
    }
    const float tie = key_logit(lo);
    const auto tied = [&](int i) { return logit(i) == tie && in.has(tie, s0 + i) ? 1ull : 0ull; };
    // the slice in runs of neighbouring tokens, one per thread
    const int run = (n + kThreads - 1) / kThreads, i0 = min(n, tid * run), i1 = min(n, i0 + run);
    unsigned long long k = 0;
    for (int i = i0; i < i1; ++i) k += tied(i);
    unsigned long long b = block_before64(k, sh.warp);
    unsigned long long mine = 0;
    for (int i = 0; i < kWarps; ++i) mine += sh.warp[i];
    give(mine);
    cluster.sync();
    for (int r = 0; r < rank; ++r) b += sh.part[xchg][r];
    xchg = xchg == 7 ? 1 : xchg + 1;
    if (b < need && need <= b + k)
      for (int i = i0; i < i1; ++i)
        if (tied(i) && ++b == need)
          for (int r = 0; r < cs; ++r) cluster.map_shared_rank(&sh, r)->pick = s0 + i;
    cluster.sync();
    const int cut = sh.pick;
    __syncthreads();
    return Kept{tie, cut};
  };

  const bool k_on = K >= 1 && K < V, p_on = TP < 1.f;
  const unsigned long long least = __float2ull_ru(MP * 1099511627776.f);
  auto kept_share = [](unsigned long long m, float inv) {
    // 24 bits of m are enough: from 2^32 on its last nine are less than 2^-23 of it
    return (m >> 32 ? (float)(uint32_t)(m >> 9) * 512.f : (float)(uint32_t)m) * inv;
  };
  // t = floor(floor(2^24 u) Z / 2^24)
  auto draw_target = [&](unsigned long long Z) {
    const unsigned long long m24 = (unsigned long long)(u * 16777216.f);
    return (__umul64hi(m24, Z) << 40) | ((m24 * Z) >> 24);
  };

  // tau = ceil(top_p * sum) into sh.tau, of top_p = m 2^-e, 2^23 <= m < 2^24 (fp64 is slow here).
  auto set_tau = [&](unsigned long long sum) {
    if (tid == 0) {
      const unsigned b = __float_as_uint(TP), m = (b & 0x7fffffu) | 0x800000u;
      const int e = 150 - (int)(b >> 23);  // 24 or more
      const unsigned long long lo = m * sum, hi = __umul64hi(m, sum);
      unsigned long long q = 0, rest = 1;  // (a top_p below 2^-39: the largest mass alone reaches it)
      if (e < 64) q = hi << (64 - e) | lo >> e, rest = lo << (64 - e);
      sh.tau = q + (rest != 0);
    }
    __syncthreads();
  };
  // In the first CTA: M <= kCand candidates, all that can be kept, of which top_k leaves the
  // first nk, to the token and the row's distribution.  counted: sh.tau is top_p's target
  // already.
  auto finish = [&](int M, int nk, bool counted) {
    if (M == 0) {  // no logit above -infinity
      if (tid == 0) p.tokens[row] = -1;
      return;
    }
    {
      const unsigned long long k[2] = {tid < M ? sh.key[tid] : 0ull, tid + kThreads < M ? sh.key[tid + kThreads] : 0ull};
      const unsigned most = __reduce_max_sync(0xffffffffu, max((unsigned)(k[0] >> 32), (unsigned)(k[1] >> 32)));
      if (lane == 0) sh.warp[warp] = most;
      sh.h.cnt[tid] = 0;
      if (tid == 0) sh.picked = 0;
      __syncthreads();
      R.mx = key_logit(__reduce_max_sync(0xffffffffu, lane < kWarps ? (unsigned)sh.warp[lane] : 0u));
      if (nk < M && M > kFew) {
        // every CTA's first top_k are there: down to the bin of the row's k-th first, which leaves
        // fewer to rank (64 rows of 128256 tokens, top_k 50: 38.0 us without, 33.9 with)
        int bin[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bin[i] = k[i] ? R.bin_of(key_logit((uint32_t)(k[i] >> 32))) : kBins;
          if (k[i]) atomicAdd(&sh.h.cnt[bin[i]], 1u);
        }
        __syncthreads();
        const unsigned here = sh.h.cnt[tid];
        const unsigned long long above = block_before64(here, sh.warp);
        if (above < (unsigned long long)nk && (unsigned long long)nk <= above + here) sh.pick = tid;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (bin[i] <= sh.pick) sh.key[atomicAdd(&sh.picked, 1u)] = k[i];
        __syncthreads();
        M = (int)sh.picked;
      }
      __syncthreads();
    }
    // top_p's target, from the sum of the first nk
    const auto target = [&](bool last, unsigned long long sum) {
      if (p_on && !counted) {
        if (last) sh.found = sum;
        __syncthreads();
        set_tau(sh.found);
      }
      return p_on ? sh.tau : ~0ull;
    };
    if (M <= kFew) {
      const int i = tid / 4;
      const bool lead = tid % 4 == 0;
      const unsigned long long x = i < M ? sh.key[i] : 0ull, m = x ? R.mass(key_logit((uint32_t)(x >> 32))) : 0ull;
      if (lead && x) mass[i] = m;
      __syncthreads();
      const Ranked r = ranked(sh.key, mass, M, x);
      const unsigned long long tau = target(lead && x && r.above == nk - 1, r.before + m);
      const bool keep = x && r.above < nk && r.before < tau && m >= least;
      // now by index (the low halves of the keys fall as it rises)
      const unsigned long long y = keep ? x << 32 | 1u : 0ull;
      unsigned long long* const by = mass + kCand;
      if (lead) by[i] = y, by[kFew + i] = keep ? m : 0ull;
      __syncthreads();
      const Ranked q = ranked(by, by + kFew, M, y);
      const unsigned long long t = draw_target(q.total);
      const int v = (int)(0xffffffffu - (uint32_t)x);
      if (lead && keep) {
        if (q.before <= t && t < q.before + m) p.tokens[row] = v;
        if (p.probs) p.probs[row * V + v] = kept_share(m, 1.f / (float)q.total);
      }
      return;
    }
    const Two k = sorted_keys(sh.key, M);
    unsigned long long x0 = k.x0, x1 = k.x1;
    const int i0 = 2 * tid, i1 = 2 * tid + 1;
    const unsigned long long m0 = x0 ? R.mass(key_logit((uint32_t)(x0 >> 32))) : 0ull;
    const unsigned long long m1 = x1 ? R.mass(key_logit((uint32_t)(x1 >> 32))) : 0ull;
    const unsigned long long b0 = block_before64(m0 + m1, sh.warp), b1 = b0 + m0;
    const unsigned long long tau = target(i0 == nk - 1 || i1 == nk - 1, i0 == nk - 1 ? b0 + m0 : b1 + m1);
    // a rank is kept if it is among the top_k, what lies before it falls short of tau, and its mass suffices
    const bool keep0 = i0 < nk && b0 < tau && m0 >= least, keep1 = i1 < nk && b1 < tau && m1 >= least;
    const int kept_n = __syncthreads_count(keep0) + __syncthreads_count(keep1);
    if (i0 == kept_n - 1) sh.found = b0 + m0;
    if (i1 == kept_n - 1) sh.found = b1 + m1;
    // now by index (the low halves of the keys fall as it rises), with the rank to find the mass by
    if (i0 < kCand) {
      sh.key[i0] = keep0 ? x0 << 32 | (unsigned)i0 : 0ull, sh.key[i1] = keep1 ? x1 << 32 | (unsigned)i1 : 0ull;
      mass[i0] = m0, mass[i1] = m1;
    }
    __syncthreads();
    const unsigned long long Z = sh.found, t = draw_target(Z);
    if (p.probs) {
      const float inv = 1.f / (float)Z;
      if (keep0) p.probs[row * V + (0xffffffffu - (uint32_t)x0)] = kept_share(m0, inv);
      if (keep1) p.probs[row * V + (0xffffffffu - (uint32_t)x1)] = kept_share(m1, inv);
    }
    if (kept_n <= kFew) {
      const unsigned long long y = tid / 4 < kept_n ? sh.key[tid / 4] : 0ull;
      const Ranked q = ranked(sh.key, mass, kept_n, y);
      if (tid % 4 == 0 && y && q.before <= t && t < q.before + mass[tid / 4]) p.tokens[row] = (int)(0xffffffffu - (uint32_t)(y >> 32));
      return;
    }
    const Two by_index = sorted_keys(sh.key, kept_n);
    x0 = by_index.x0, x1 = by_index.x1;
    const unsigned long long y0 = x0 ? mass[(uint32_t)x0] : 0ull, y1 = x1 ? mass[(uint32_t)x1] : 0ull;
    const unsigned long long c0 = block_before64(y0 + y1, sh.warp), c1 = c0 + y0;
    if (c0 <= t && t < c0 + y0) p.tokens[row] = (int)(0xffffffffu - (uint32_t)(x0 >> 32));
    if (c1 <= t && t < c1 + y1) p.tokens[row] = (int)(0xffffffffu - (uint32_t)(x1 >> 32));
  };

  // A small top_k: every CTA's tokens down to the bin of its own threads' k-th largest maximum
  // hold its k first, so all CTAs' such tokens hold the row's, and nothing else has to be known
  // before they are sent.  (Tokens at -infinity have no mass and are left out; a row with
  // +infinity goes the long way.)
  if (!bad && temp > 0.f && k_on && 2 * K <= kThreads && K * cs <= kCand * 5 / 8) {
    zero_probs();  // now, so that the barrier below does not wait for them
    sh.h.cnt[tid] = 0;
    __syncthreads();
    atomicAdd(&sh.h.cnt[R.bin_of(own)], 1u);
    __syncthreads();
    const unsigned here = sh.h.cnt[tid];
    const unsigned long long above = block_before64(here, sh.warp);
    if (above < (unsigned long long)K && (unsigned long long)K <= above + here) sh.pick = tid;
    __syncthreads();
    const int bin = sh.pick;
    const float least_l = mx == INFINITY ? INFINITY : fmaxf(bin_floor(bin), -3.402823466e38f);
    const unsigned mine =  // by all CTAs: they take turns with cand[]
        send(least_l, INFINITY, [&](int, float x) { return R.bin_of(x) <= bin; });
    give(mx == INFINITY ? kCand + 1 : mine);
    cluster.sync();
    const unsigned long long M = sum_given();
    if (M <= kCand) {
      if (rank == 0) finish((int)M, min(K, (int)M), false);
      return;
    }
  }

  // The row's largest logit.
  give(__float_as_uint(mx));
  cluster.sync();
  for (int r = 0; r < cs; ++r) mx = fmaxf(mx, __uint_as_float((uint32_t)sh.part[xchg][r]));
  ++xchg;
  if (bad || mx == -INFINITY) {  // nothing to draw from
    if (rank == 0 && tid == 0) p.tokens[row] = -1;
    zero_probs();
    cluster.sync();
    return;
  }
  if (temp == 0.f) {  // the first of the largest logits
    int first = V;
    for (int i = tid; i < n; i += kThreads)
      if (logit(i) == mx) {
        first = s0 + i;
        break;
      }
    first = (int)__reduce_min_sync(0xffffffffu, (unsigned)first);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = first;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) first = min(first, (int)sh.warp[i]);
    give(first);
    cluster.sync();
    for (int r = 0; r < cs; ++r) first = min(first, (int)sh.part[xchg][r]);
    if (rank == 0 && tid == 0) p.tokens[row] = first;
    fill([&](int i) { return s0 + i == first ? 1.f : 0.f; });
    cluster.sync();
    return;
  }

  if (mx == INFINITY) {  // such tokens share all mass: 0 for them, and nothing for the others
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) val[i] = from_f32<T>(logit(i) == INFINITY ? 0.f : -INFINITY);
    own = own == INFINITY ? 0.f : -INFINITY;
    mx = 0.f;
    __syncthreads();
  }
  R.mx = mx;

  Kept kept{-INFINITY, V};   // what no limit has cut yet
  int last_bin = kBins;      // the last bin of the first histogram that kept tokens can fall into; kBins: any
  bool k_done = !k_on;       // top_k is in `kept`
  bool counted = false;      // all masses of `kept` were summed up: sh.tau is set,
  Found f{};                 // and this is where they reach it
  const auto count_tokens = [&] {
    unsigned long long none;
    histogram(false, none, [&](int, float x, int&, int&) { return R.bin_of(x); });
    return find(false, 0ull, (unsigned long long)K);
  };
  const auto count_masses = [&] {
    const Kept in = kept;
    // Without top_k, tokens with x below log((1 - top_p) / V) - 1 hold less than 1 - top_p of
    // the mass together, so the prefix ends above them: they are summed up, but have no bin.
    const int far = k_on ? kBins : (int)fminf((logf((float)V / (1.f - TP)) + 1.f) * kBinsPerUnit, (float)kBins);
    unsigned long long S;
    histogram(true, S, [&](int i, float x, int& a, int& b) {
      R.mass_parts(x, a, b);
      const int bin = R.bin_of(x);
      const bool is = in.has(x, s0 + i);
      a = is ? a : 0, b = is ? b : 0;
      return bin <= far && (a | b) != 0 ? bin : -1;
    });
    set_tau(S);
    f = find(true, 0ull, sh.tau);
    counted = true;
  };
  if (k_on) {
    if (K <= kCandK && 2 * K <= cs * kThreads) {
      sh.h.cnt[tid] = 0;
      __syncthreads();
      atomicAdd(&sh.h.cnt[R.bin_of(own)], 1u);
      reduce_bins(kCounts);
      last_bin = find(false, 0ull, (unsigned long long)K).bin;
    } else {
      const Found at = count_tokens();
      if (at.upto <= kCand) last_bin = at.bin;
      else kept = select(false, (unsigned long long)K, kept, at), k_done = true;
    }
  }
  if (p_on && last_bin == kBins) {
    count_masses();
    if (f.upto <= kCand) last_bin = f.bin;
  }
  if (least > 0 && (k_done || !p_on))  // (top_p counts all of the top_k)
    last_bin = min(last_bin, (int)fminf(-logf(MP) * kBinsPerUnit + 1.f, (float)(kBins - 1)));
  if (last_bin < kBins) {
    const Kept in = kept;
    const unsigned long long M = gather(bin_floor(last_bin), INFINITY, [&](int i, float x) {
      return R.bin_of(x) <= last_bin && in.has(x, s0 + i);
    });
    if (M <= kCand) {
      zero_probs();
      cluster.sync();  // the zeros lie before the kept tokens' shares
      if (rank == 0) finish((int)M, k_done ? (int)M : min(K, (int)M), counted);
      return;
    }
    if (!k_done) kept = select(false, (unsigned long long)K, kept, count_tokens());
    if (p_on && !counted) count_masses();
  }
  if (p_on) kept = select(true, sh.tau, kept, f);

  // The kept masses: a warp's sum over its run of neighbouring tokens, then the cluster's.
  const int run = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const bool limit = least > 0;
  const auto parts_at = [&](int i, int& a, int& b) {
    const float x = logit(i);
    R.mass_parts(x, a, b);
    const bool is = kept.has(x, s0 + i) && (!limit || whole(a, b) >= least);
    a = is ? a : 0, b = is ? b : 0;
  };
  const auto mass_at = [&](int i) {
    int a, b;
    parts_at(i, a, b);
    return whole(a, b);
  };
  const int w0 = min(n, warp * run), w1 = min(n, w0 + run);
  long long sum_a = 0, sum_b = 0;
  const auto add = [&](int i, bool on) {
    int a, b;
    parts_at(i, a, b);
    sum_a += on ? a : 0, sum_b += on ? b : 0;
  };
  if (kept.t == -INFINITY) {
    for (int i0 = w0 + lane; i0 < w1; i0 += 32 * kBatch)
#pragma unroll
      for (int k = 0; k < kBatch; ++k) add(min(i0 + 32 * k, n - 1), i0 + 32 * k < w1);
  } else {
    // kept tokens are lined up first, so that no lane works out a mass that is not wanted
    static_assert(kCand * 2 / kWarps >= 63 + 64, "queues in the candidates' place");
    int* const queue = reinterpret_cast<int*>(sh.key) + warp * (kCand * 2 / kWarps);
    int waiting = 0;
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32 * 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + 32 * k + lane;
        const bool is = i < w1 && kept.has(logit(min(i, n - 1)), s0 + i);
        const unsigned m = __ballot_sync(0xffffffffu, is);
        if (is) queue[waiting + __popc(m & ((1u << lane) - 1u))] = i;
        waiting += __popc(m);
      }
      if (waiting >= 64) {
        __syncwarp();
        waiting -= 64;
        add(queue[waiting + lane], true), add(queue[waiting + 32 + lane], true);
        __syncwarp();
      }
    }
    __syncwarp();
    for (int k = lane; k < waiting; k += 32) add(queue[k], true);
  }
  unsigned long long sum = whole(sum_a, sum_b);
  sum = warp_sum64(sum);
  __syncthreads();
  if (lane == 0) sh.warp2[warp] = sum;
  __syncthreads();
  unsigned long long mine = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) mine += sh.warp2[i];
  give(mine);
  cluster.sync();
  unsigned long long Z = 0, before = 0;
  for (int r = 0; r < cs; ++r) {
    const unsigned long long v = sh.part[xchg][r];
    if (r < rank) before += v;
    Z += v;
  }
  const unsigned long long t = draw_target(Z);
  if (before <= t && t < before + mine) {
    int w = 0;
    unsigned long long at = before;
    while (w < kWarps - 1 && at + sh.warp2[w] <= t) at += sh.warp2[w++];
    const int b0 = min(n, w * run), b1 = min(n, b0 + run);
    const int each = (b1 - b0 + kThreads - 1) / kThreads, i0 = min(b1, b0 + tid * each), i1 = min(b1, i0 + each);
    unsigned long long k = 0;
    for (int i = i0; i < i1; ++i) k += mass_at(i);
    unsigned long long b = at + block_before64(k, sh.warp);
    if (b <= t && t < b + k)
      for (int i = i0; i < i1; ++i) {
        b += mass_at(i);
        if (b > t) {
          p.tokens[row] = s0 + i;
          break;
        }
      }
  }
  if (probs) {
    const float inv = 1.f / (float)Z;
    fill([&](int i) { return kept_share(mass_at(i), inv); });
  }
  cluster.sync();  // no CTA leaves while another may still write to it
}

template <typename T>
cudaError_t launch_t(const SampleParams& p, int cs, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1ull)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * (int)sizeof(T) + 32);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  const size_t smem = (size_t)((p.V + cs - 1) / cs) * sizeof(T) + 32;
  return launch_k_cluster(sample_kernel<T>, dim3((unsigned)(p.rows * cs)), dim3(kThreads), smem, st, dim3(cs, 1, 1), p);
}

// CTAs of a row: as many as keep two per SM busy, with 4096 tokens or more each and their logits
// in half an SM's shared memory; twice the portable size for a few rows.
int cluster_size(int rows, int V, int elem, int sm_count) {
  int cs = 1;
  while (cs < 8 && V > 4096 * cs && ((long long)rows * cs < 2 * sm_count || (V + cs - 1) / cs * elem > 84 * 1024)) cs *= 2;
  return cs == 8 && rows <= 8 && V > 8 * 4096 ? 16 : cs;
}

}  // namespace

bool sample_temperature_ok(float t) { return t == 0.f || (t >= kMinTemp && t <= kMaxTemp); }
int sample_max_vocab() { return 8 * kMaxSlice; }

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  const int cs = cluster_size(p.rows, p.V, p.dtype == 2 ? 4 : 2, p.sm_count);
  switch (p.dtype) {
    case 0: return launch_t<__half>(p, cs, st);
    case 1: return launch_t<__nv_bfloat16>(p, cs, st);
    default: return launch_t<float>(p, cs, st);
  }
}

}  // namespace spec
