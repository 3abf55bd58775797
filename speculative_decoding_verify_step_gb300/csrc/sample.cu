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
// l - m and its product with log2(e) / T are pairs of floats, a table holds 2^(-i/1024) to
// 62 bits, and the rest, below 2^-11, is three terms of a series in whole numbers of
// 2^-42: about 2^-42 of the mass, for 40 instructions and no fp64 (which runs at 1/64 of
// fp32's rate here).
//
// A row is one thread-block cluster, its slices in shared memory, read from HBM once.
// top_k needs no masses: a histogram of counts over bins 1/16 wide in x finds the bin of
// the k-th token, a histogram over that bin's logits (as ordered integers) the logit; few
// rows need a third.  top_p does the same with masses, over what top_k left.  Bins go
// through distributed shared memory, each CTA adding up its share of them.
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
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 48 * 1024;     // logits of a CTA (shared memory)
constexpr float kBinsPerUnit = 16.f;     // bins of x in the first histogram

// 2^(-i/1024) in units of 2^-62, by the exponential series.
struct Pow2Table {
  unsigned long long v[1024];
};
constexpr Pow2Table make_pow2_table() {
  Pow2Table t{};
  for (int i = 0; i < 1024; ++i) {
    const double x = -0.69314718055994530942 * i / 1024.0;
    double term = 1.0, sum = 0.0;
    for (int k = 1; k < 30; ++k) {
      term *= x / k;
      sum += term;
    }
    // 1 + sum in whole numbers: the one is exact, and i = 0 gives 2^62
    t.v[i] = (1ull << 62) - (unsigned long long)(-sum * 4611686018427387904.0);
  }
  return t;
}
__device__ const Pow2Table kPow2 = make_pow2_table();

struct Shared {
  unsigned long long pow2[1024];
  unsigned int cnt[kBins], m0[kBins], m1[kBins], m2[kBins];  // this CTA's histogram; a mass in three parts
  unsigned int gc[kBins];                                    // the cluster's
  unsigned long long gm[kBins];
  unsigned long long part[8][kMaxCluster];                   // exchanges: one value of each CTA
  unsigned long long warp[kWarps], warp2[kWarps];
  unsigned long long found, tau;
  int pick;
};

// A mass <= 2^40 in parts of 14, 13 and 14 bits: over a slice's at most 48 * 1024 tokens
// each part's sum stays below 2^30.
SPEC_DEVICE_INLINE unsigned long long joined(unsigned a, unsigned b, unsigned c) {
  return (unsigned long long)a + ((unsigned long long)b << 14) + ((unsigned long long)c << 27);
}

SPEC_DEVICE_INLINE uint32_t order_key(float l) {  // orders like l
  const uint32_t b = __float_as_uint(l);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
SPEC_DEVICE_INLINE float key_logit(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

struct Row {
  float mx;          // largest logit; 0 where that is +infinity
  bool inf;          // the largest logit is +infinity: such tokens share all mass
  float ch, cl;      // log2(e) / T
  float bin;         // kBinsPerUnit / T
  const unsigned long long* pow2;

  SPEC_DEVICE_INLINE float dist(float l) const { return inf ? (l == INFINITY ? 0.f : INFINITY) : mx - l; }
  // Bin of x: never falls as l falls.
  SPEC_DEVICE_INLINE int bin_of(float l) const { return (int)fminf(dist(l) * bin, (float)(kBins - 1)); }

  SPEC_DEVICE_INLINE unsigned long long mass(float l) const {
    const float dh = dist(l);
    const float yh = dh * ch;
    if (!(yh < 41.f)) return 0ull;  // 2^-41 and less: no mass
    float dl = 0.f;
    if (!inf) {  // what dh lost
      const float bb = dh - mx;
      dl = (mx - (dh - bb)) - (l + bb);
    }
    const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
    const float t = fmaf(yh, 1024.f, 12582912.f);
    const int k = __float_as_int(t) - 0x4b400000;          // 1024 y, rounded
    const float fh = fmaf(t - 12582912.f, -0.0009765625f, yh);
    // r = -(fh + yl) ln 2 as a pair, e^r - 1 = r + r^2 (1/2 + r/6)
    const float rh = fh * -0.693147182464599609375f;
    const float rl = fmaf(fh, -0.693147182464599609375f, -rh) +
                     fmaf(yl, -0.693147182464599609375f, fh * 1.90465429995776804525e-9f);
    const float q = rh * rh * fmaf(rh, 0.16666667f, 0.5f) + rl;
    const int s = __float2int_rn(rh * 4398046511104.f) +
                  (__float_as_int(fmaf(q, 4398046511104.f, 12582912.f)) - 0x4b400000);
    const unsigned long long p = pow2[k & 1023];
    const unsigned long long w = p + (((long long)(int)((p >> 32) + ((p >> 31) & 1ull)) * s) >> 10);
    return w >> (22 + (k >> 10));
  }
};

SPEC_DEVICE_INLINE unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

SPEC_DEVICE_INLINE unsigned long long block_sum64(unsigned long long v, unsigned long long* w) {
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long s = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) s += w[i];
  return s;
}

// Sum over the CTA's threads before this one.
SPEC_DEVICE_INLINE unsigned long long block_before64(unsigned long long v, unsigned long long* w) {
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
  unsigned long long s = inc - v;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) s += i < warp ? w[i] : 0ull;
  return s;
}

// What is kept: logits above the threshold key, and of those equal to it the tokens up to cut.
struct Kept {
  uint32_t t;
  int cut;
  SPEC_DEVICE_INLINE bool has(uint32_t key, int v) const { return key > t || (key == t && v <= cut); }
};

template <typename T>
SPEC_DEVICE_INLINE float to_f32(T x);
template <>
SPEC_DEVICE_INLINE float to_f32<float>(float x) { return x; }
template <>
SPEC_DEVICE_INLINE float to_f32<__half>(__half x) { return __half2float(x); }
template <>
SPEC_DEVICE_INLINE float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// A stored logit: NaN counts as -infinity, and -0 as 0.
SPEC_DEVICE_INLINE float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / cs;
  const int V = p.V, set = (int)(row / p.rows_per_setting);
  const int slice = (V + cs - 1) / cs, s0 = min(V, rank * slice), n = min(V, s0 + slice) - s0;

  for (int i = tid; i < 1024; i += kThreads) sh.pow2[i] = kPow2.v[i];
  pdl_wait();
  pdl_launch_dependents();

  const float temp = p.temperature ? p.temperature[set] : p.temperature_all;
  const int K = p.top_k ? p.top_k[set] : 0;
  const float TP = p.top_p ? p.top_p[set] : 1.f, MP = p.min_p ? p.min_p[set] : 0.f;
  const float u = temp == 0.f ? 0.f : p.u[row];
  const bool bad = !(temp == 0.f || (temp >= 1e-6f && temp < INFINITY)) || K < 0 || !(TP > 0.f && TP <= 1.f) ||
                   !(MP >= 0.f && MP <= 1.f) || !(u >= 0.f && u < 1.f);

  // The slice, in 16-byte loads where the row's address lets them; local index i lies at
  // val[i], val chosen so that those loads are stored aligned.
  constexpr int PER = 16 / sizeof(T);
  const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + s0;
  const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / (int)sizeof(T));
  float* const val = smem + ((4 - (head & 3)) & 3);
  const int vecs = (n - head) / PER, tail0 = head + vecs * PER;
  float mx = -INFINITY;
  auto put = [&](int i, float x) {
    x = clean(x);
    val[i] = x;
    mx = fmaxf(mx, x);
  };
  if (tid < head) put(tid, to_f32(src[tid]));
  if (tid < n - tail0) put(tail0 + tid, to_f32(src[tail0 + tid]));
  constexpr int UN = 4;  // loads in flight
  for (int j0 = tid; j0 < vecs; j0 += UN * kThreads) {
    uint4 w[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (j0 + k * kThreads < vecs) w[k] = __ldcs(reinterpret_cast<const uint4*>(src + head) + j0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (j0 + k * kThreads < vecs) {
        const T* e = reinterpret_cast<const T*>(&w[k]);
        float4* dst = reinterpret_cast<float4*>(val + head + (j0 + k * kThreads) * PER);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const float4 f = make_float4(clean(to_f32(e[4 * i])), clean(to_f32(e[4 * i + 1])), clean(to_f32(e[4 * i + 2])),
                                       clean(to_f32(e[4 * i + 3])));
          dst[i] = f;
          mx = fmaxf(fmaxf(fmaxf(mx, f.x), fmaxf(f.y, f.z)), f.w);
        }
      }
  }

  // Exchange number xchg: one 64-bit value of every CTA, read after a cluster barrier.  A
  // number comes up again only after at least six barriers.
  int xchg = 0;
  auto give = [&](unsigned long long v) {
    if (tid < cs) *cluster.map_shared_rank(&sh.part[xchg][rank], tid) = v;
  };
  mx = warp_max(mx);
  if (lane == 0) sh.warp[warp] = __float_as_uint(mx);
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, __uint_as_float((uint32_t)sh.warp[i]));
  cluster.sync();  // every CTA of the cluster runs: its shared memory may be written
  give(__float_as_uint(mx));
  cluster.sync();
  for (int r = 0; r < cs; ++r) mx = fmaxf(mx, __uint_as_float((uint32_t)sh.part[0][r]));
  ++xchg;

  float* const probs = p.probs ? p.probs + row * V + s0 : nullptr;
  auto fill = [&](auto q) {
    if (probs)
      for (int i = tid; i < n; i += kThreads) probs[i] = q(i);
  };

  if (bad || mx == -INFINITY) {  // nothing to draw from
    if (rank == 0 && tid == 0) p.tokens[row] = -1;
    fill([](int) { return 0.f; });
    cluster.sync();
    return;
  }
  if (temp == 0.f) {  // the first of the largest logits
    int first = V;
    for (int i = tid; i < n; i += kThreads)
      if (val[i] == mx) {
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

  Row R;
  R.inf = mx == INFINITY;
  R.mx = R.inf ? 0.f : mx;
  R.ch = __fdiv_rn(1.44269502162933349609375f, temp);   // log2(e) is this + 1.92596299e-8
  R.cl = __fdiv_rn(fmaf(-R.ch, temp, 1.44269502162933349609375f) + 1.92596299112661746887e-8f, temp);
  R.bin = kBinsPerUnit / temp;
  R.pow2 = sh.pow2;

  // One histogram pass over the slice's tokens that `cls` gives a bin >= 0; the cluster's
  // bins end up in gc and gm, and the sum of all masses that cls found in `total`.
  auto histogram = [&](bool masses, unsigned long long& total, auto cls) {
    sh.cnt[tid] = sh.m0[tid] = sh.m1[tid] = sh.m2[tid] = 0;
    __syncthreads();
    unsigned long long sum = 0;
    for (int i = tid; i < n; i += kThreads) {
      unsigned long long m = 0;
      const int b = cls(i, val[i], m);
      sum += m;
      if (b >= 0) {
        atomicAdd(&sh.cnt[b], 1u);
        if (masses) {
          atomicAdd(&sh.m0[b], (unsigned)m & 0x3fffu);
          atomicAdd(&sh.m1[b], (unsigned)(m >> 14) & 0x1fffu);
          atomicAdd(&sh.m2[b], (unsigned)(m >> 27));
        }
      }
    }
    if (masses) {
      sum = block_sum64(sum, sh.warp);
      give(sum);
    } else {
      __syncthreads();
    }
    cluster.sync();
    // this CTA's share of the bins, added up and sent to all
    const int share = kBins / cs, b = rank * share + tid;
    if (tid < share) {
      unsigned int gc = 0;
      unsigned long long gm = 0;
      for (int r = 0; r < cs; ++r) {
        const Shared* o = cluster.map_shared_rank(&sh, r);
        gc += o->cnt[b];
        if (masses) gm += joined(o->m0[b], o->m1[b], o->m2[b]);
      }
      for (int r = 0; r < cs; ++r) {
        Shared* o = cluster.map_shared_rank(&sh, r);
        o->gc[b] = gc;
        o->gm[b] = gm;
      }
    }
    cluster.sync();
    if (masses) {
      total = 0;
      for (int r = 0; r < cs; ++r) total += sh.part[xchg][r];
      xchg = xchg == 7 ? 1 : xchg + 1;
    }
  };

  // The first bin where the running measure (counts, or masses), `base` so far, reaches
  // `target`.
  struct Found {
    int bin;
    unsigned int count;
    unsigned long long size, above;  // the bin's measure; base and what lies above the bin
  };
  auto find = [&](bool by_mass, unsigned long long base, unsigned long long target) {
    const unsigned long long mine = by_mass ? sh.gm[tid] : (unsigned long long)sh.gc[tid];
    const unsigned long long before = base + block_before64(mine, sh.warp);
    if (before < target && target <= before + mine) {
      sh.pick = tid;
      sh.found = before;
    }
    __syncthreads();
    Found f;
    f.bin = sh.pick;
    f.count = sh.gc[f.bin];
    f.size = by_mass ? sh.gm[f.bin] : f.count;
    f.above = sh.found;
    __syncthreads();
    return f;
  };

  // The least and the largest key whose distance falls into bin b of the first histogram.
  auto bin_bounds = [&](int b, uint32_t& lo, uint32_t& hi) {
    const uint32_t highest = order_key(R.inf ? INFINITY : R.mx), lowest = order_key(-INFINITY);
    uint32_t a = lowest, z = highest;
    while (a < z) {
      const uint32_t m = a + (z - a) / 2;
      if (R.bin_of(key_logit(m)) <= b) z = m;
      else a = m + 1;
    }
    lo = a;
    z = highest;
    while (a < z) {
      const uint32_t m = a + (z - a + 1) / 2;
      if (R.bin_of(key_logit(m)) >= b) a = m;
      else z = m - 1;
    }
    hi = a;
  };

  // The shortest prefix (by rank) of the tokens of `in` whose measure reaches target; their
  // first histogram has been taken.
  auto select = [&](bool by_mass, unsigned long long target, const Kept& in) -> Kept {
    Found f = find(by_mass, 0ull, target);
    uint32_t lo, hi;
    bin_bounds(f.bin, lo, hi);
    while (true) {
      if (f.count == 1 || f.above + f.size == target) return lo > in.t ? Kept{lo, V} : in;  // all of the bin
      if (lo == hi) break;
      const uint32_t span = hi - lo, l = lo, h = hi;
      const int sft = max(0, 32 - __clz(span) - 9);  // span >> sft < 512
      unsigned long long sum;
      histogram(by_mass, sum, [&](int i, float x, unsigned long long& m) {
        const uint32_t key = order_key(x);
        if (key < l || key > h || !in.has(key, s0 + i)) return -1;
        if (by_mass) m = R.mass(x);
        return (int)((h - key) >> sft);
      });
      f = find(by_mass, f.above, target);
      hi = h - ((uint32_t)f.bin << sft);
      lo = hi - l < (1u << sft) ? l : hi - ((1u << sft) - 1u);
    }
    // equal logits: as many of the first as are needed
    unsigned long long need = target - f.above;
    if (by_mass) {
      const unsigned long long m = R.mass(key_logit(lo));
      need = (need + m - 1) / m;
    }
    const auto tied = [&](int i) { return order_key(val[i]) == lo && in.has(lo, s0 + i) ? 1ull : 0ull; };
    // the slice in runs of neighbouring tokens, one per thread
    const int run = (n + kThreads - 1) / kThreads, i0 = min(n, tid * run), i1 = min(n, i0 + run);
    unsigned long long k = 0;
    for (int i = i0; i < i1; ++i) k += tied(i);
    unsigned long long b = block_before64(k, sh.warp);
    unsigned long long mine = 0;
    for (int i = 0; i < kWarps; ++i) mine += sh.warp[i];
    give(mine);
    if (tid == 0) sh.pick = V;
    cluster.sync();
    for (int r = 0; r < rank; ++r) b += sh.part[xchg][r];
    xchg = xchg == 7 ? 1 : xchg + 1;
    if (b < need && need <= b + k)
      for (int i = i0; i < i1; ++i)
        if (tied(i) && ++b == need)
          for (int r = 0; r < cs; ++r) *cluster.map_shared_rank(&sh.pick, r) = s0 + i;
    cluster.sync();
    const int cut = sh.pick;
    __syncthreads();
    return Kept{lo, cut};
  };

  const Kept everything{0u, V};
  Kept kept = everything;
  const bool k_on = K >= 1 && K < V, p_on = TP < 1.f;
  unsigned long long S = 0;
  if (k_on) {
    histogram(false, S, [&](int, float x, unsigned long long&) { return R.bin_of(x); });
    kept = select(false, (unsigned long long)K, everything);
  }
  if (p_on) {
    const Kept in = kept;
    // Without top_k, tokens with x below log((1 - top_p) / V) - 1 hold less than 1 - top_p of
    // the mass together, so the prefix ends above them: they are summed up, but have no bin.
    const int far = k_on ? kBins : (int)fminf((logf((float)V / (1.f - TP)) + 1.f) * kBinsPerUnit, (float)kBins);
    histogram(true, S, [&](int i, float x, unsigned long long& m) {
      if (!in.has(order_key(x), s0 + i)) return -1;
      m = R.mass(x);
      const int b = R.bin_of(x);
      return b <= far && m > 0ull ? b : -1;
    });
    if (tid == 0) sh.tau = max(1ull, (unsigned long long)ceil(__dmul_rn((double)TP, (double)S)));  // fp64: one warp's
    __syncthreads();
    kept = select(true, sh.tau, in);
  }
  const unsigned long long least = __float2ull_ru(MP * 1099511627776.f);

  // The kept masses: a warp's sum over its run of neighbouring tokens, then the cluster's.
  const int run = ((n + kWarps - 1) / kWarps + 31) & ~31;
  auto mass_at = [&](int i) -> unsigned long long {
    const float x = val[i];
    if (!kept.has(order_key(x), s0 + i)) return 0ull;
    const unsigned long long m = R.mass(x);
    return m >= least ? m : 0ull;
  };
  const int w0 = min(n, warp * run), w1 = min(n, w0 + run);
  unsigned long long sum = 0;
  for (int i = w0 + lane; i < w1; i += 32) sum += mass_at(i);
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
  // t = floor(floor(2^24 u) Z / 2^24)
  const unsigned long long m24 = (unsigned long long)(u * 16777216.f);
  const unsigned long long hi64 = __umul64hi(m24, Z), lo64 = m24 * Z;
  const unsigned long long t = (hi64 << 40) | (lo64 >> 24);
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
    fill([&](int i) {
      const unsigned long long m = mass_at(i);
      // 24 bits of m are enough: from 2^32 on its last nine are less than 2^-23 of it
      return (m >> 32 ? (float)(uint32_t)(m >> 9) * 512.f : (float)(uint32_t)m) * inv;
    });
  }
  cluster.sync();  // no CTA leaves while another may still write to it
}

template <typename T>
cudaError_t launch_t(const SampleParams& p, int cs, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1ull)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4 + 16);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  }
  return launch_k_cluster(sample_kernel<T>, dim3((unsigned)(p.rows * cs)), dim3(kThreads), smem, st, dim3(cs, 1, 1), p);
}

}  // namespace

int sample_max_vocab() { return kMaxCluster * kMaxSlice; }

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  // the narrowest cluster whose CTAs have at most 4096 tokens, or the widest
  int cs = 1;
  while (cs < kMaxCluster && (p.V + cs - 1) / cs > 4096) cs *= 2;
  const size_t smem = (size_t)((p.V + cs - 1) / cs) * 4 + 16;
  switch (p.dtype) {
    case 0: return launch_t<__half>(p, cs, smem, st);
    case 1: return launch_t<__nv_bfloat16>(p, cs, smem, st);
    default: return launch_t<float>(p, cs, smem, st);
  }
}

}  // namespace spec
