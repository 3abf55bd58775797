// Attention of the verify window over the 8-bit paged cache, and each token's share of it.
//
// For query row r (a window row and one of the query heads that share the kv head) and
// cached token k of a sub-block with exponents a (K) and b (V), with codes c:
//   S[r, k] = 2^a (q_r . c_k) scale,   O[r] = sum_k P[r, k] 2^b c_k / sum_k P[r, k]
// one pass over the pages with a running maximum and sum per row.  A code is expanded to
// fp16, exactly, by one cvt for two of them (2 cycles per SM quarter, measured; shifts and
// masks for the same take 5), and both products run on mma.sync m16n8k16 with fp32
// accumulators.  Tokens (scores) and dims (values) are the M side, so the work goes up in
// steps of 8 query rows: S comes out as [token, row], and one movmatrix per 8 x 8 tile
// turns the weights into the B operand of the second product.
//
// Rounding.  q is scaled per row by a power of two into fp16's range (bf16 queries keep
// all their bits); the weights times 2^b are rounded to fp16.  Everything else is fp32.  The
// running maximum of a row is that of score + b over the tokens it sees, so the largest
// weight times 2^b is near one whatever the exponents of tokens that the row does not see
// or hardly weighs; the sum takes the weights without 2^b.  They are rounded as multiples
// of 2^-11, which takes the largest next to the end of fp16's range: a weight times 2^b is off
// by 2^-11 of itself down to 2^-25 of the largest, and below by 2^-36 of the largest at most.
// So 2^20 light tokens beside a heavy one keep their share to 2^-16, and dims where a
// sub-block of large exponent has zeros keep the others' values, as long as those weigh that much.  Score and maximum
// are numbers of one float grid (the product with the scale is rounded before the difference
// is taken), so scores past 2^24 keep all weight on the largest.
//
// Work split.  A group is a sequence and a kv head, a unit 32 of its tokens.  Groups longer
// than a common target are cut into pieces of at most that many units; a CTA of four warps
// takes one piece, a warp every fourth unit of it, with a ring of its own in shared memory
// (bulk copies of 32 tokens: K, V and exponents are one run of bytes) and accumulators of
// its own, so the loop has no CTA barrier.  The warps' results are merged at the end, those
// of a cut group by a second kernel.  Short caches need neither the common target nor the
// second kernel: the CTAs of a group are one thread-block cluster, and each finishes a share
// of the rows from all partials, through distributed shared memory.
//
// What bounds it (8 kv heads of 128 with 4 query heads).  Two tiles of query rows: the cache's bytes,
// 8 x 32768 tokens at width 4 in 92.5 us, 0.86 of the copy rate (a decode step of the same 87, 0.91).  Three
// and four: latencies, since 243 registers leave two warps per SM quarter: 64 x 512..2048 at
// width 5 in 63 us, 0.41.  Short caches: one chain of latencies, 1 x 1024 tokens in 6.5 us.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "kv4.cuh"
#include "kv8.cuh"
#include "kv8.h"
#include "launch.cuh"

namespace spec {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;             // tokens of a unit
constexpr int kMinUnits = 4;          // of a piece: one for each warp
constexpr int kMaxCtas = 3;           // per SM, of any variant
constexpr int kMaxCluster = 8;
constexpr int kClusterUnits = 40;     // of a cluster's CTA, at most
constexpr float kNoMax = -1e30f;      // running maximum of a row that has seen no token
// How far score + b may pass the running maximum: 64 x 512..2048 tokens at width 5 take 65.0 us with
// 2, 63.3 with 4 and 62.5 with 6, but the weights' unit rises with it.
constexpr float kSlack = 4.f;
// Unit of the weights times 2^b as fp16: they are at most 2^kSlack, or, where maxima are 2^25 or
// more (float steps of 4 or more, to which score + b is rounded down), 2^8.
constexpr float kLift = 2048.f, kLiftHuge = 128.f, kHuge = 33554432.f;

SPEC_DEVICE_INLINE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D(16x8 fp32) += A(16x16 f16, row) * B(16x8 f16, col); not volatile, so that independent
// products can be moved between dependent ones.
SPEC_DEVICE_INLINE void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across the warp.
SPEC_DEVICE_INLINE uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

SPEC_DEVICE_INLINE void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Window geometry of sequence b.
struct Seq {
  int row0, Wb, L, n_keys, units;
};
SPEC_DEVICE_INLINE Seq seq_of(const Kv8AttnParams& p, int b) {
  Seq s;
  s.row0 = p.row_off ? p.row_off[b] : b * p.W;
  s.Wb = p.row_off ? p.row_off[b + 1] - s.row0 : p.W;
  s.row0 = max(0, min(s.row0, p.total_rows));
  s.Wb = max(0, min(min(s.Wb, p.W), p.total_rows - s.row0));
  const int cap = p.max_pages * kPage;
  s.L = max(-kMaxWidth, min(p.kv_len[b], cap));  // below 0: the window's first rows have no cell
  s.n_keys = s.Wb > 0 ? max(0, min(s.L + s.Wb, cap)) : 0;
  s.units = (s.n_keys + kUnit - 1) / kUnit;
  return s;
}
// Sequence `lane` of the first 32: most batches need no other.
SPEC_DEVICE_INLINE Seq first_seqs(const Kv8AttnParams& p) {
  const int lane = threadIdx.x & 31;
  Seq s{};
  if (lane < p.B) s = seq_of(p, lane);
  return s;
}
SPEC_DEVICE_INLINE Seq seq_at(const Kv8AttnParams& p, const Seq& mine, int b) {
  if (b >= 32) return seq_of(p, b);
  Seq s;
  s.row0 = __shfl_sync(0xffffffffu, mine.row0, b);
  s.Wb = __shfl_sync(0xffffffffu, mine.Wb, b);
  s.L = __shfl_sync(0xffffffffu, mine.L, b);
  s.n_keys = __shfl_sync(0xffffffffu, mine.n_keys, b);
  s.units = __shfl_sync(0xffffffffu, mine.units, b);
  return s;
}

SPEC_DEVICE_INLINE int pieces_of(int units, int target) { return (units + target - 1) / target; }

// Units of a piece, at most.  Pieces number at most groups + units / target: with few groups
// as many as there are slots (CTAs that the GPU holds at once), with many up to half again
// as many.  With 1.5 times the slots always, 37 x 64..8000 tokens at width 4 took 66 us instead of 69,
// but 8 x 32768 104 instead of 92 and 64 x 512..2048 at width 5 67 instead of 63.  (Equal runs of units
// over group bounds, a CTA taking several groups one behind another: 118, 98 and 75.)
SPEC_DEVICE_INLINE int target_of(const Kv8AttnParams& p, const Seq& mine) {
  const int lane = threadIdx.x & 31;
  unsigned n = mine.units;
  for (int b = lane + 32; b < p.B; b += 32) n += seq_of(p, b).units;
  const long long total = (long long)__reduce_add_sync(0xffffffffu, n) * p.Hkv;  // at most 2^31 units
  const long long groups = (long long)p.B * p.Hkv;
  const long long share = max((long long)p.slots - groups, (long long)p.slots / 2);
  return (int)max((long long)kMinUnits, (total + share - 1) / share);
}
// The sequence that holds piece x (per sequence all pieces of head 0, then head 1, ...), B if
// there is none, and the pieces before it: of all sequences, and of those cut in two or more.
SPEC_DEVICE_INLINE int find_piece(const Kv8AttnParams& p, const Seq& mine, int target, int x, int& before,
                                  int& before_cut) {
  const int lane = threadIdx.x & 31;
  int base = 0, base_cut = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int units = b0 == 0 ? mine.units : b0 + lane < p.B ? seq_of(p, b0 + lane).units : 0;
    const int n = pieces_of(units, target) * p.Hkv, nc = n > p.Hkv ? n : 0;
    int incl = n, incl_cut = nc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, incl_cut, o);
      if (lane >= o) incl += u, incl_cut += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      before = base + __shfl_sync(0xffffffffu, incl - n, l);
      before_cut = base_cut + __shfl_sync(0xffffffffu, incl_cut - nc, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    base_cut += __shfl_sync(0xffffffffu, incl_cut, 31);
  }
  before = base, before_cut = base_cut;
  return p.B;
}

// Partial i of the workspace (pieces of cut groups, in order): rows x hd of O, then the rows'
// maxima and sums.
SPEC_DEVICE_INLINE float* partial(float* ws, long long i, int rows, int hd) { return ws + i * rows * (hd + 2); }

// Four output values of a row: o / l in the caller's type; a row that sees no token is zeros.
SPEC_DEVICE_INLINE void store_row4(const Kv8AttnParams& p, long long row, int head, int hd, int d4, float4 o, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint2 w;
  if (p.bf16) {
    w.x = kv4_pack2<true>(o.x * inv, o.y * inv);
    w.y = kv4_pack2<true>(o.z * inv, o.w * inv);
  } else {
    const __half2 most = __float2half2_rn(65504.f);
    const __half2 a = __hmin2_nan(__hmax2_nan(__floats2half2_rn(o.x * inv, o.y * inv), __hneg2(most)), most);
    const __half2 b = __hmin2_nan(__hmax2_nan(__floats2half2_rn(o.z * inv, o.w * inv), __hneg2(most)), most);
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row * p.Hq + head) * hd + d4 * 4) = w;
}
// What turns a row's scores into weights, 2^(score - m) / l: m and 1 / l apart, since from m = 2^24 on
// m + log2(l) would lose l.  A row that sees no token gives nobody any.
SPEC_DEVICE_INLINE void store_norm(const Kv8AttnParams& p, long long row, int head, float m, float l) {
  if (p.norm) p.norm[row * p.Hq + head] = l > 0.f ? make_float2(m, 1.f / l) : l == l ? make_float2(INFINITY, 0.f) : make_float2(NAN, NAN);
}

// Rows [r0, r0 + 8 NT) of a group's query rows (`rows` in all; window at flat row row0, kv head
// kvh) as B fragments: piece [8 rows][HD / 32][lane (g, c)] holds dims 16 (c + 4 (i / 2)) +
// 8 (i % 2) .. + 7 of row g.  f gets the rows' factors from products to log2 units.  A row is
// scaled by a power of two that takes its largest element to [2^14, 2^15).
template <int HD, int NT, int THREADS>
SPEC_DEVICE_INLINE void load_queries(const Kv8AttnParams& p, int row0, int kvh, int r0, int rows, uint8_t* qfrag,
                                     float* f) {
  constexpr int LPR = HD / 8;                       // lanes of a row, eight dims each
  const int grp = p.Hq / p.Hkv, lane = threadIdx.x & 31;
  const int m = lane % LPR, chunk = m / 2;
  const int piece = HD == 128 ? (chunk / 4) * 2 + (m & 1) : m & 1, c = chunk % 4;
  constexpr int PER = THREADS / LPR, N = (NT * 8 + PER - 1) / PER;
  uint4 raw[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int r = threadIdx.x / LPR + k * PER, w = (r0 + r) / grp, hh = (r0 + r) % grp;
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    if (r < NT * 8 && r0 + r < rows)
      raw[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (long long)(row0 + w) * p.q_row_stride +
                                               (long long)(kvh * grp + hh) * HD + m * 8);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int r = threadIdx.x / LPR + k * PER;
    const uint32_t in[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    float x[8], mx = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = p.bf16 ? kv4_unpack2<true>(in[i]) : kv4_unpack2<false>(in[i]);
      x[2 * i] = kv4_sat(v.x);
      x[2 * i + 1] = kv4_sat(v.y);
      mx = fmaxf(mx, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^sh with 2^14 <= mx 2^sh < 2^15; rows below 2^-112 count as zeros (|scale| <= 2^40)
    const int sh = mx > 1.9259299e-34f ? 14 - (int)((__float_as_uint(mx) >> 23) - 127u) : 0;
    const float up = kv8_pow2(sh);
    if (r < NT * 8) {
      if (m == 0) f[r] = p.scale * 1.44269504f * kv8_pow2(-sh);
      *reinterpret_cast<uint4*>(qfrag + (((r >> 3) * (HD / 32) + piece) * 32 + (r & 7) * 4 + c) * 16) =
          make_uint4(pack_f16x2(x[0] * up, x[1] * up), pack_f16x2(x[2] * up, x[3] * up), pack_f16x2(x[4] * up, x[5] * up),
                     pack_f16x2(x[6] * up, x[7] * up));
    }
  }
}

// Products of 16 tokens (`load` gives 16 bytes of K codes: token g or g + 8, chunk c + 4 jj) with
// the rows' fragments: s[nt] = tokens g, g + 8 x rows 2c, 2c + 1.
template <int HD, int NT, typename F>
SPEC_DEVICE_INLINE void qk_sub(F load, const uint8_t* qfrag, float (&s)[NT][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
  for (int jj = 0; jj < HD / 64; ++jj) {
    const uint4 k0 = load(0, jj), k1 = load(1, jj);
    const uint32_t a[4] = {k0.x, k0.y, k0.z, k0.w}, b[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x0 = kv8_lo(a[2 * h]), x2 = kv8_hi(a[2 * h]), x1 = kv8_lo(b[2 * h]), x3 = kv8_hi(b[2 * h]);
      const uint32_t y0 = kv8_lo(a[2 * h + 1]), y2 = kv8_hi(a[2 * h + 1]);
      const uint32_t y1 = kv8_lo(b[2 * h + 1]), y3 = kv8_hi(b[2 * h + 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 q = *reinterpret_cast<const uint4*>(qfrag + ((nt * (HD / 32) + jj * 2 + h) * 32 + lane) * 16);
        mma(s[nt], x0, x1, x2, x3, q.x, q.y);
        mma(s[nt], y0, y1, y2, y3, q.z, q.w);
      }
    }
  }
}

// Whether a window row with ancestors anc sees the key that is w behind the cached tokens.
SPEC_DEVICE_INLINE bool sees(uint32_t anc, int w) { return w < 0 || (w < 16 && ((anc >> w) & 1u)); }

// HD: head_dim; NT: tiles of 8 query rows.
template <int HD, int NT>
struct Cfg {
  static constexpr int kStage = kUnit / kSub * kv8_sub_bytes(HD);
  // CTAs per SM, by registers.  Two tiles in 168 registers instead of 186: 32 x 512..8192 tokens at
  // width 4 64.5 us instead of 73.5; three tiles spill then (64 x 512..2048 at width 5 70 instead of 63).
  static constexpr int kCtas = NT <= 2 ? 3 : 2;
  static constexpr int kQ = NT * (HD / 32) * 512;             // query fragments
  static constexpr int kStatic = NT * 8 * 4 * (1 + 2 * kWarps) + 1024;
  static constexpr int kStages0 = (233472 / kCtas - 1024 - kStatic - kQ) / (kWarps * kStage);
  static constexpr int kStages = kStages0 < 6 ? kStages0 : 6; // of a warp
  static constexpr int kSmem = kQ + kWarps * kStages * kStage;
  static_assert(kStages >= 2 && kCtas <= kMaxCtas, "ring");
  static constexpr int kRec = HD + 4;                         // floats of a row's partial for the cluster: O, maximum, sum
  static_assert(NT * (8 * HD + 2 * kRec) * 4 <= kStages * kStage, "a warp's partial, and two rows of each tile of the CTA's, reuse its ring");
};

// grid (pieces, row blocks): rows [y NT 8, (y + 1) NT 8) of the group's.  CL: the p.cluster CTAs
// of a group are one cluster, its pieces.
template <int HD, int NT, bool CL>
__global__ void __launch_bounds__(kThreads, (Cfg<HD, NT>::kCtas))
    kv8_attention_kernel(const __grid_constant__ Kv8AttnParams p) {
  using C = Cfg<HD, NT>;
  constexpr int ROWS = NT * 8, D = C::kStages, SUB = kv8_sub_bytes(HD), MT = HD / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const qfrag = smem;
  __shared__ uint64_t full[kWarps][D];
  __shared__ __align__(8) float s_f[ROWS];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ uint32_t s_anc[16];
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int grp = p.Hq / p.Hkv;
  uint8_t* const ring = smem + C::kQ + warp * D * C::kStage;

  pdl_wait();
  // The merge kernel reads the call's tables before its own wait: they are complete now.  Clusters
  // let the next kernel in only as they end: its first CTAs would take places that its other
  // clusters, if it has any, then lack.
  if (!CL) pdl_launch_dependents();
  int b, kvh, piece, pieces, slot = 0;
  Seq seq;
  if constexpr (CL) {
    pieces = p.cluster;
    piece = blockIdx.x % pieces;
    kvh = blockIdx.x / pieces % p.Hkv;
    b = blockIdx.x / pieces / p.Hkv;
    seq = seq_of(p, b);
  } else {
    const Seq mine = first_seqs(p);
    const int target = target_of(p, mine);
    int before, before_cut;
    b = find_piece(p, mine, target, blockIdx.x, before, before_cut);
    if (b >= p.B) return;
    seq = seq_at(p, mine, b);
    pieces = pieces_of(seq.units, target);
    kvh = (blockIdx.x - before) / pieces, piece = (blockIdx.x - before) % pieces;
    slot = before_cut + (blockIdx.x - before);
  }
  const int r0 = blockIdx.y * ROWS, rows = min(seq.Wb * grp - r0, ROWS);  // of this CTA
  if (rows <= 0) return;  // (all CTAs of a cluster alike)
  const int u0 = (int)((long long)seq.units * piece / pieces);
  const int u1 = (int)((long long)seq.units * (piece + 1) / pieces);
  const int L = seq.L, n_keys = seq.n_keys;

  if (lane == 0) {
    for (int s = 0; s < D; ++s) mbar_init(&full[warp][s], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) s_fail = 0;
  if (threadIdx.x < 16) s_anc[threadIdx.x] = p.anc[threadIdx.x];
  __syncwarp();

  const int32_t* table = p.page_table + (long long)b * p.max_pages;
  // The page of unit u, or -1: past the piece, or no page of the pool.
  const auto page_of = [&](int u) {
    const int pg = u < u1 ? table[u >> 1] : -1;
    return pg < p.num_pages ? pg : -1;
  };
  uint32_t there = 0, phase = 0;  // stages with a copy, parity of their next phase
  const auto issue = [&](int u, int s, int pg) {
    there &= ~(1u << s);
    if (pg < 0) return;
    there |= 1u << s;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp][s], C::kStage);
      bulk_load(ring + s * C::kStage, p.pool + ((long long)pg * p.Hkv + kvh) * kv8_block_bytes(HD) + (u & 1) * C::kStage,
                C::kStage, &full[warp][s]);
    }
  };
  {
    int pg[D];
#pragma unroll
    for (int s = 0; s < D; ++s) pg[s] = page_of(u0 + warp + s * kWarps);
#pragma unroll
    for (int s = 0; s < D; ++s) issue(u0 + warp + s * kWarps, s, pg[s]);
  }
  int next_pg = page_of(u0 + warp + D * kWarps);  // of the unit that is issued next
  load_queries<HD, NT, kThreads>(p, seq.row0, kvh, r0, r0 + rows, qfrag, s_f);
  __syncthreads();

  float acc[NT][MT][4];   // dims (row of the tile: g, g + 8) x query rows 2c, 2c + 1
  float top[NT][2], sum[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[nt][t][0] = acc[nt][t][1] = acc[nt][t][2] = acc[nt][t][3] = 0.f;
    top[nt][0] = top[nt][1] = kNoMax;
    sum[nt][0] = sum[nt][1] = 0.f;
  }

  int s = 0;
  float lift = kLift;
  bool failed = false;
  for (int u = u0 + warp; u < u1; u += kWarps) {
    if ((there >> s) & 1u) {
      if (!mbar_wait(&full[warp][s], (phase >> s) & 1u, p.status)) {
        failed = true;  // the rows come out as NaN
        break;
      }
      phase ^= 1u << s;
      const uint8_t* st = ring + s * C::kStage;
      float sc[2][NT][4];
      int ev[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        qk_sub<HD, NT>([&](int half, int jj) {
          return *reinterpret_cast<const uint4*>(st + k * SUB + kv8_k_chunk<HD>(g + 8 * half, c + 4 * jj));
        }, qfrag, sc[k]);
      const int key0 = u * kUnit;
      const bool masked = key0 + kUnit > L;
      bool over = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t par = *reinterpret_cast<const uint32_t*>(st + k * SUB + 2 * kSub * HD);
        const float ka = kv8_pow2(kv8_exp(par, 0));
        ev[k] = kv8_exp(par, 1);
        const float room = kSlack - (float)ev[k];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2*>(&s_f[nt * 8 + 2 * c]);
          const float f0 = f.x * ka, f1 = f.y * ka;
          float* x = sc[k][nt];
          // rounded here, so that the difference with the maximum is exact near it
          x[0] = __fmul_rn(x[0], f0), x[1] = __fmul_rn(x[1], f1);
          x[2] = __fmul_rn(x[2], f0), x[3] = __fmul_rn(x[3], f1);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = nt * 8 + 2 * c + e;
              const uint32_t anc = r < rows ? s_anc[(r0 + r) / grp] & ((1u << seq.Wb) - 1u) : 0u;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = key0 + k * kSub + g + 8 * h;
                if (key >= n_keys || !sees(anc, key - L)) x[2 * h + e] = -INFINITY;
              }
            }
          }
          if (NT == 1 && p.scores) {  // for the tokens' weights
            float* to = p.scores + (((long long)b * p.Hkv + kvh) * p.max_pages * 2 + u) * (p.W * grp * kUnit) + k * kSub + g;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (2 * c + e < rows) __stcs(to + (2 * c + e) * kUnit, x[e]), __stcs(to + (2 * c + e) * kUnit + 8, x[2 + e]);
          }
          over |= fmaxf(x[0], x[2]) - top[nt][0] > room || fmaxf(x[1], x[3]) - top[nt][1] > room;
        }
      }
      if (__any_sync(0xffffffffu, over)) {  // raise the maxima and rescale what is summed up
        bool huge = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float y = fmaxf(sc[k][nt][e], sc[k][nt][2 + e]);
              // towards the score: a maximum of the scores' grid
              m = fmaxf(m, ev[k] < 0 ? __fadd_ru(y, (float)ev[k]) : __fadd_rd(y, (float)ev[k]));
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, top[nt][e]);
            huge |= m > kNoMax && fabsf(m) >= kHuge;
            const float a = ex2(top[nt][e] - m);
            top[nt][e] = m;
            sum[nt][e] *= a;
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[nt][t][e] *= a, acc[nt][t][2 + e] *= a;
          }
        if (lift != kLiftHuge && __any_sync(0xffffffffu, huge)) {
          lift = kLiftHuge;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[nt][t][i] *= kLiftHuge / kLift;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float vb = kv8_pow2(ev[k]) * lift;
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float* x = sc[k][nt];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float w0 = ex2(x[2 * h] - top[nt][0]), w1 = ex2(x[2 * h + 1] - top[nt][1]);
            sum[nt][0] += w0;
            sum[nt][1] += w1;
            pb[nt][h] = movmatrix_trans(pack_f16x2(w0 * vb, w1 * vb));
          }
        }
        // tokens behind the last have weight zero, but their bytes may be anything, NaN among them
        uint32_t real = 0xffffffffu;
        if (masked) {
          const int t = key0 + k * kSub + 2 * c;
          real = (t < n_keys ? 0xffu : 0u) | (t + 1 < n_keys ? 0xff00u : 0u) | (t + 8 < n_keys ? 0xff0000u : 0u) |
                 (t + 9 < n_keys ? 0xff000000u : 0u);
        }
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
          uint4 v = *reinterpret_cast<const uint4*>(st + k * SUB + kv8_v_chunk<HD>(j, lane));
          if (masked) v.x &= real, v.y &= real, v.z &= real, v.w &= real;
          const uint32_t a0 = kv8_lo(v.x), a2 = kv8_hi(v.x), a1 = kv8_lo(v.y), a3 = kv8_hi(v.y);
          const uint32_t b0 = kv8_lo(v.z), b2 = kv8_hi(v.z), b1 = kv8_lo(v.w), b3 = kv8_hi(v.w);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(acc[nt][2 * j], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            mma(acc[nt][2 * j + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();
      fence_proxy_async();  // the stage was read through the generic proxy
    }
    issue(u + D * kWarps, s, next_pg);
    next_pg = page_of(u + (D + 1) * kWarps);
    s = s + 1 == D ? 0 : s + 1;
  }
  if (failed) {
    s_fail = 1;
    // give copies still in flight the same time to land before the shared memory is given up
    for (int i = 0; i < D; ++i)
      if ((there >> i) & 1u) (void)mbar_wait(&full[warp][i], (phase >> i) & 1u, nullptr);
  }
  __syncwarp();

  // The warp's partial in its ring's place: [ROWS][HD].
  const float unit = 1.f / lift;
  float* const part = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = sum[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const int r = nt * 8 + 2 * c + e;
      if (g == 0) s_m[warp][r] = top[nt][e], s_l[warp][r] = l;
      // tile t: rows g and g + 8 are the lane's dims 2 t and 2 t + 1
#pragma unroll
      for (int t = 0; t < MT; t += 2)
        *reinterpret_cast<float4*>(part + r * HD + g * (HD / 8) + 2 * t) =
            make_float4(acc[nt][t][e] * unit, acc[nt][t][2 + e] * unit, acc[nt][t + 1][e] * unit, acc[nt][t + 1][2 + e] * unit);
    }
  __syncthreads();
  constexpr int V4 = HD / 4;
  const bool whole = !CL && pieces == 1;
  float* const ws = CL ? nullptr : partial(p.workspace, (long long)slot * gridDim.y + blockIdx.y, ROWS, HD);
  // row r of the CTA's partial, for the cluster: behind warp r % 4's own
  const auto record = [&](int r) {
    return reinterpret_cast<float*>(smem + C::kQ + (r & 3) * D * C::kStage) + ROWS * HD + (r >> 2) * C::kRec;
  };
  for (int it = threadIdx.x; it < rows * V4; it += kThreads) {
    const int r = it / V4, d4 = it % V4;
    float M = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2(s_m[w][r] - M);
      const float4 x = *reinterpret_cast<const float4*>(smem + C::kQ + w * D * C::kStage + (r * HD + d4 * 4) * 4);
      o.x = fmaf(a, x.x, o.x);
      o.y = fmaf(a, x.y, o.y);
      o.z = fmaf(a, x.z, o.z);
      o.w = fmaf(a, x.w, o.w);
      l = fmaf(a, s_l[w][r], l);
    }
    if (s_fail) o = make_float4(NAN, NAN, NAN, NAN), l = NAN;  // a wait ran out
    if (whole) {
      const int row = seq.row0 + (r0 + r) / grp, head = kvh * grp + (r0 + r) % grp;
      store_row4(p, row, head, HD, d4, o, s_fail ? 1.f : l);
      if (d4 == 0) store_norm(p, row, head, M, l);
    } else {
      float* const rec = CL ? record(r) : ws + r * HD;
      *reinterpret_cast<float4*>(rec + d4 * 4) = o;
      if (d4 == 0) {
        (CL ? rec + HD : ws + ROWS * HD + r)[0] = M;
        (CL ? rec + HD + 1 : ws + ROWS * HD + ROWS + r)[0] = l;
      }
    }
  }
  if constexpr (CL) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // rows piece, piece + pieces, ...: sum_i 2^(m_i - M) o_i over the cluster
    const int own = (rows - piece + pieces - 1) / pieces;
    for (int it = threadIdx.x; it < own * V4; it += kThreads) {
      const int r = piece + it / V4 * pieces, d4 = it % V4;
      const uint32_t at = smem_u32(record(r));
      float m[kMaxCluster], s1[kMaxCluster], M = kNoMax, l = 0.f;
      float4 x[kMaxCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < pieces) {
          const uint32_t a = mapa_u32(at, i);
          x[i] = ld_dsmem_f4(a + d4 * 16);
          m[i] = ld_dsmem_f32(a + HD * 4);
          s1[i] = ld_dsmem_f32(a + HD * 4 + 4);
        }
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < pieces) M = fmaxf(M, m[i]);
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < pieces) {
          const float a = ex2(m[i] - M);
          l = fmaf(a, s1[i], l);
          o.x = fmaf(a, x[i].x, o.x);
          o.y = fmaf(a, x[i].y, o.y);
          o.z = fmaf(a, x[i].z, o.z);
          o.w = fmaf(a, x[i].w, o.w);
        }
      const int row = seq.row0 + (r0 + r) / grp, head = kvh * grp + (r0 + r) % grp;
      store_row4(p, row, head, HD, d4, l == l ? o : make_float4(NAN, NAN, NAN, NAN), l == l ? l : 1.f);
      if (d4 == 0) store_norm(p, row, head, M, l);
    }
    __syncwarp();
    cluster_arrive_relaxed();  // its reads are done: no CTA leaves before all have
    cluster_wait();
  }
}

// Merge the partials of cut groups: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.  grid
// (shares of a group's rows, Hkv, B).  hd / 4 lanes take a row, and up to all warps share its
// partials, eight loads in flight each.
constexpr int kMergeWarps = 8;
__host__ __device__ constexpr int merge_split(int n) {  // warps of a row, a power of two
  int split = 1;
  while (split < kMergeWarps && split * 4 < n) split *= 2;
  return split;
}
template <int HD>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv8_merge_kernel(const __grid_constant__ Kv8AttnParams p, int ws_rows, int row_blocks) {
  constexpr int V4 = HD / 4, RPW = 32 / V4;
  __shared__ float4 s_o[kMergeWarps][32];
  __shared__ float2 s_ml[kMergeWarps][32];
  const int b = blockIdx.z, kvh = blockIdx.y, grp = p.Hq / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq mine = first_seqs(p);
  const Seq seq = seq_at(p, mine, b);
  const int target = target_of(p, mine);
  const int n = pieces_of(seq.units, target);
  if (n < 2) {  // one CTA finished the group, or it has no token
    const int rows = n == 0 ? seq.Wb * grp : 0;
    pdl_wait();
    pdl_launch_dependents();
    for (int it = blockIdx.x * kMergeWarps * 32 + threadIdx.x; it < rows * V4; it += gridDim.x * kMergeWarps * 32) {
      const int r = it / V4;
      store_row4(p, seq.row0 + r / grp, kvh * grp + r % grp, HD, it % V4, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
      if (it % V4 == 0) store_norm(p, seq.row0 + r / grp, kvh * grp + r % grp, 0.f, 0.f);
    }
    return;
  }
  int cut = 0;  // partials of the sequences before this one
  for (int i = lane; i < b; i += 32) {
    const int k = pieces_of(i < 32 ? mine.units : seq_of(p, i).units, target);
    if (k > 1) cut += k;
  }
  const int i0 = (int)__reduce_add_sync(0xffffffffu, (unsigned)cut) * p.Hkv + kvh * n;
  pdl_wait();
  pdl_launch_dependents();
  const int split = merge_split(n);
  const int part = warp & (split - 1), at_once = kMergeWarps / split * RPW;
  const int d4 = lane % V4, rows = seq.Wb * grp;
  for (int rb = blockIdx.x * at_once; rb < rows; rb += gridDim.x * at_once) {
    const int r = rb + warp / split * RPW + lane / V4;
    const int rr = min(r, rows - 1), blk = rr / ws_rows, rw = rr % ws_rows;
    float M = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int NB = 8;  // partials whose loads are in flight together
    for (int k0 = part; k0 < n; k0 += NB * split) {
      float ms[NB], ls[NB];
      float4 os[NB];
      float mb = M;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float* ws = partial(p.workspace, (long long)(i0 + min(k0 + k * split, n - 1)) * row_blocks + blk, ws_rows, HD);
        os[k] = *reinterpret_cast<const float4*>(ws + rw * HD + d4 * 4);
        ms[k] = ws[ws_rows * HD + rw];
        ls[k] = ws[ws_rows * HD + ws_rows + rw];
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) mb = fmaxf(mb, ms[k]);
      const float a = ex2(M - mb);
      M = mb;
      l *= a;
      o.x *= a, o.y *= a, o.z *= a, o.w *= a;
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (k0 + k * split < n) {
          const float w = ex2(ms[k] - M);
          l = fmaf(w, ls[k], l);
          o.x = fmaf(w, os[k].x, o.x);
          o.y = fmaf(w, os[k].y, o.y);
          o.z = fmaf(w, os[k].z, o.z);
          o.w = fmaf(w, os[k].w, o.w);
        }
    }
    if (split > 1) {
      s_o[warp][lane] = o;
      s_ml[warp][lane] = make_float2(M, l);
      __syncthreads();
      if (part == 0) {
        float m2 = M;
        for (int k = 1; k < split; ++k) m2 = fmaxf(m2, s_ml[warp + k][lane].x);
        const float a = ex2(M - m2);
        M = m2;
        l *= a;
        o.x *= a, o.y *= a, o.z *= a, o.w *= a;
        for (int k = 1; k < split; ++k) {
          const float2 ml = s_ml[warp + k][lane];
          const float4 x = s_o[warp + k][lane];
          const float w = ex2(ml.x - M);
          l = fmaf(w, ml.y, l);
          o.x = fmaf(w, x.x, o.x);
          o.y = fmaf(w, x.y, o.y);
          o.z = fmaf(w, x.z, o.z);
          o.w = fmaf(w, x.w, o.w);
        }
      }
      __syncthreads();
    }
    if (part == 0 && r < rows) {
      const int row = seq.row0 + r / grp, head = kvh * grp + r % grp;
      store_row4(p, row, head, HD, d4, l == l ? o : make_float4(NAN, NAN, NAN, NAN), l == l ? l : 1.f);
      if (d4 == 0) store_norm(p, row, head, M, l);
    }
  }
}

// weight[b, h, t] += sum over the group's rows of 2^(score - m) / l: the scores once more, from K
// alone.  grid (CTAs of a group, Hkv, B); a unit of 32 tokens is one warp's, which alone touches
// their weights.
constexpr int kWeightWarps = 8;
template <int HD, int NT>
__global__ void __launch_bounds__(kWeightWarps * 32) kv8_weight_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr int ROWS = NT * 8, SUB = kv8_sub_bytes(HD);
  __shared__ __align__(16) uint8_t qfrag[NT * (HD / 32) * 512];
  __shared__ float s_f[ROWS];
  __shared__ float2 s_norm[ROWS];
  __shared__ uint32_t s_anc[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, kvh = blockIdx.y, grp = p.Hq / p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  const Seq seq = seq_of(p, b);
  const int rows = seq.Wb * grp;
  const int units = (int)min((long long)seq.units, (p.weight_len + kUnit - 1) / kUnit);
  if ((int)blockIdx.x * kWeightWarps >= units) return;
  load_queries<HD, NT, kWeightWarps * 32>(p, seq.row0, kvh, 0, rows, qfrag, s_f);
  if (threadIdx.x < 16) s_anc[threadIdx.x] = p.anc[threadIdx.x];
  for (int r = threadIdx.x; r < ROWS; r += kWeightWarps * 32)
    s_norm[r] = r < rows ? p.norm[(long long)(seq.row0 + r / grp) * p.Hq + kvh * grp + r % grp] : make_float2(INFINITY, 0.f);
  __syncthreads();
  float* const weight = p.weight + ((long long)b * p.Hkv + kvh) * p.weight_len;
  for (int u = blockIdx.x * kWeightWarps + warp; u < units; u += gridDim.x * kWeightWarps) {
    const int pg = p.page_table[(long long)b * p.max_pages + (u >> 1)];
    if (pg < 0 || pg >= p.num_pages) continue;
    const uint8_t* st = p.pool + ((long long)pg * p.Hkv + kvh) * kv8_block_bytes(HD) + (u & 1) * 2 * SUB;
    const int t = u * kUnit + (c >> 1) * kSub + (c & 1) * 8 + g;  // the token whose weight this lane adds to
    const bool mine = t < seq.n_keys && t < p.weight_len;
    const float was = mine ? weight[t] : 0.f;
    float add[4];  // tokens g, g + 8 of either sub-block
    const bool masked = (u + 1) * kUnit > seq.L;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* sub = st + k * SUB;
      float sc[NT][4];
      const uint32_t par = *reinterpret_cast<const uint32_t*>(sub + 2 * kSub * HD);
      qk_sub<HD, NT>([&](int half, int jj) {
        return __ldcs(reinterpret_cast<const uint4*>(sub + kv8_k_chunk<HD>(g + 8 * half, c + 4 * jj)));
      }, qfrag, sc);
      const float ka = kv8_pow2(kv8_exp(par, 0));
      add[2 * k] = add[2 * k + 1] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * c + e;
          const float f = s_f[r] * ka;
          const float2 norm = s_norm[r];
          uint32_t anc = 0xffffffffu;
          if (masked) anc = r < rows ? s_anc[r / grp] & ((1u << seq.Wb) - 1u) : 0u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float w = ex2(__fmul_rn(sc[nt][2 * h + e], f) - norm.x);
            const int key = u * kUnit + k * kSub + g + 8 * h;
            if (!masked || (key < seq.n_keys && sees(anc, key - seq.L))) add[2 * k + h] = fmaf(w, norm.y, add[2 * k + h]);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      add[i] += __shfl_xor_sync(0xffffffffu, add[i], 1);
      add[i] += __shfl_xor_sync(0xffffffffu, add[i], 2);
    }
    const float w = c == 0 ? add[0] : c == 1 ? add[1] : c == 2 ? add[2] : add[3];
    if (mine) weight[t] = was + w;
  }
}

// The same from the scores that the attention left (few rows): a lane per token, eight CTAs per SM.
__global__ void __launch_bounds__(kWeightWarps * 32, 8) kv8_weight_scores_kernel(const __grid_constant__ Kv8AttnParams p) {
  __shared__ float2 s_norm[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, kvh = blockIdx.y, grp = p.Hq / p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  const Seq seq = seq_of(p, b);
  const int rows = seq.Wb * grp;
  const int units = (int)min((long long)seq.units, (p.weight_len + kUnit - 1) / kUnit);
  if ((int)blockIdx.x * kWeightWarps >= units) return;
  if (threadIdx.x < 8)
    s_norm[threadIdx.x] = threadIdx.x < rows ? p.norm[(long long)(seq.row0 + threadIdx.x / grp) * p.Hq + kvh * grp + threadIdx.x % grp]
                                             : make_float2(INFINITY, 0.f);
  __syncthreads();
  float* const weight = p.weight + ((long long)b * p.Hkv + kvh) * p.weight_len;
  const float* const scores = p.scores + ((long long)b * p.Hkv + kvh) * p.max_pages * 2 * (p.W * grp * kUnit);
#pragma unroll 1
  for (int u = blockIdx.x * kWeightWarps + warp; u < units; u += gridDim.x * kWeightWarps) {
    const int pg = p.page_table[(long long)b * p.max_pages + (u >> 1)];
    const int t = u * kUnit + lane;
    if (pg < 0 || pg >= p.num_pages || t >= seq.n_keys || t >= p.weight_len) continue;
    const float* x = scores + (long long)u * (p.W * grp * kUnit) + lane;
    float s[8], w = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s[r] = r < rows ? __ldcs(x + r * kUnit) : 0.f;
    const float was = weight[t];
#pragma unroll
    for (int r = 0; r < 8; ++r) w = fmaf(ex2(s[r] - s_norm[r].x), s_norm[r].y, w);
    weight[t] = was + w;
  }
}

// Function attributes are per device: one bit per device once they are set there.
template <typename K>
cudaError_t configure(K kernel, int smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done.load(std::memory_order_acquire) >> (dev & 63) & 1ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  return e;
}

// Row blocks of a group (CTAs with the same pages), and 8-row tiles of each: up to four tiles
// fit a warp's registers.
constexpr int row_blocks(int rows) { return rows > 32 ? 2 : 1; }
constexpr int row_tiles(int rows) { return ((rows + 7) / 8 + row_blocks(rows) - 1) / row_blocks(rows); }

// CTAs of a group where they are one cluster: short caches, by the hint.  0: not short.  A CTA gets
// at most 40 units where the clusters fill the SMs, 20 where they leave some idle.  Clusters
// against pieces, in us (8 kv heads of 128 with 4 query heads; units of a CTA in brackets): decode,
// 1 x 4096 tokens 8.9, 9.2 (16), 1 x 8192 11.7, 9.9 (32); 4 x 4096 10.0, 12.1 (32), 8 x 2048 9.8, 11.4
// (32); width 5, 4 x 4096 17.1, 18.1 (32), 16 x 1024 17.9, 19.5 (32); 16 x 5003, 4 heads of 64,
// width 4 12.0, 12.6 (40), and 16 x 0..5003 at widths 1 to 7 11.7, 12.7 (40).
int cluster_size(int B, int Hkv, int rows, int len_hint, int sm_count) {
  const long long groups = (long long)B * Hkv * row_blocks(rows), units = (len_hint + kUnit - 1) / kUnit;
  int cs = 1;
  while (cs < kMaxCluster && cs * kMinUnits < units && groups * cs * 2 <= 2 * sm_count) cs *= 2;
  return units <= (groups * cs > sm_count ? kClusterUnits : kClusterUnits / 2) * cs && groups <= (1 << 27) ? cs : 0;
}

template <int HD, int NT>
cudaError_t launch_nt(Kv8AttnParams p, cudaStream_t st) {
  using C = Cfg<HD, NT>;
  static std::atomic<uint64_t> done{0}, done_cl{0};
  const int rows = p.W * (p.Hq / p.Hkv), blocks = row_blocks(rows);
  if (const int cs = cluster_size(p.B, p.Hkv, rows, p.kv_len_hint, p.sm_count)) {
    cudaError_t e = configure(kv8_attention_kernel<HD, NT, true>, C::kSmem, done_cl);
    if (e != cudaSuccess) return e;
    p.cluster = cs;
    return launch_k_cluster(kv8_attention_kernel<HD, NT, true>, dim3((unsigned)(p.B * p.Hkv * cs), blocks), dim3(kThreads),
                            C::kSmem, st, dim3(cs, 1, 1), p);
  }
  cudaError_t e = configure(kv8_attention_kernel<HD, NT, false>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  p.slots = std::max(2, C::kCtas * p.sm_count / blocks);
  // as many CTAs as any lengths can make of it; pieces number groups + units / target at most
  const long long groups = (long long)p.B * p.Hkv;
  const long long ctas = groups + std::max<long long>(p.slots - groups, p.slots / 2);
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  e = launch_k(kv8_attention_kernel<HD, NT, false>, dim3((unsigned)ctas, blocks), dim3(kThreads), C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  const int n = (int)std::max<long long>(1, p.slots / groups);
  const int at_once = kMergeWarps / merge_split(n) * (128 / HD);
  return launch_k(kv8_merge_kernel<HD>, dim3((rows + at_once - 1) / at_once, p.Hkv, p.B), dim3(kMergeWarps * 32), 0, st,
                  p, NT * 8, blocks);
}

// CTAs of the weights' kernels: `ctas` per SM where there is that much work.
dim3 weight_grid(const Kv8AttnParams& p, int ctas) {
  const long long groups = (long long)p.B * p.Hkv, units = (p.kv_len_hint + kUnit - 1) / kUnit;
  const long long per = std::max<long long>(1, (long long)ctas * p.sm_count / groups);  // CTAs of a group
  return dim3((unsigned)std::max<long long>(1, std::min(per, (units + kWeightWarps - 1) / kWeightWarps)), p.Hkv, p.B);
}
template <int HD, int NT>
cudaError_t launch_weight(const Kv8AttnParams& p, cudaStream_t st) {
  return launch_k(kv8_weight_kernel<HD, NT>, weight_grid(p, 4), dim3(kWeightWarps * 32), 0, st, p);
}

template <int HD>
cudaError_t launch_hd(const Kv8AttnParams& p, cudaStream_t st) {
  const int rows = p.W * (p.Hq / p.Hkv);
  cudaError_t e = cudaErrorInvalidValue;
  switch (row_tiles(rows)) {
    case 1: e = launch_nt<HD, 1>(p, st); break;
    case 2: e = launch_nt<HD, 2>(p, st); break;
    case 3: e = launch_nt<HD, 3>(p, st); break;
    case 4: e = launch_nt<HD, 4>(p, st); break;
  }
  if (e != cudaSuccess || !p.weight) return e;
  if (p.scores) return launch_k(kv8_weight_scores_kernel, weight_grid(p, 8), dim3(kWeightWarps * 32), 0, st, p);
  const int tiles = (rows + 7) / 8;
  return tiles == 1 ? launch_weight<HD, 1>(p, st) : tiles == 2 ? launch_weight<HD, 2>(p, st)
       : tiles <= 4 ? launch_weight<HD, 4>(p, st) : launch_weight<HD, 8>(p, st);
}

// Floats of the partials: pieces of cut groups, at most two per slot.
long long partial_floats(const Kv8AttnParams& p) {
  const int rows = p.W * (p.Hq / p.Hkv);
  if (cluster_size(p.B, p.Hkv, rows, p.kv_len_hint, p.sm_count)) return 0;
  return 2ll * (kMaxCtas * p.sm_count) * row_tiles(rows) * 8 * row_blocks(rows) * (p.hd + 2);
}

// Floats of the scores that are kept for the tokens' weights, or 0: they are worked out again.  Up
// to 8 rows they are a quarter of K's bytes; writing and reading them takes 62 us where K once more
// takes 85 (8 x 16384 tokens, 8 kv heads of 128, one row of 4 query heads).  Room for every page
// of the table: up to 256 MB.
long long score_floats(const Kv8AttnParams& p) {
  const long long rows = p.W * (p.Hq / p.Hkv), n = (long long)p.B * p.Hkv * p.max_pages * kPage * rows;
  return rows <= 8 && n <= (64ll << 20) ? n : 0;
}

}  // namespace

long long kv8_attention_workspace(const Kv8AttnParams& p, bool weight) {
  return 4 * (partial_floats(p) + (weight ? 2ll * p.total_rows * p.Hq + score_floats(p) : 0));
}

bool kv8_attention_needs_workspace(const Kv8AttnParams& p, bool weight) {
  return weight || (p.kv_len_hint + kUnit - 1) / kUnit > kMaxCluster * kClusterUnits;
}

cudaError_t launch_kv8_attention(const Kv8AttnParams& params, cudaStream_t st) {
  Kv8AttnParams p = params;
  if (p.weight) {
    float* const norm = p.workspace + partial_floats(p);  // (a whole number of row pairs)
    p.norm = reinterpret_cast<float2*>(norm);
    if (score_floats(p) > 0) p.scores = norm + 2ll * p.total_rows * p.Hq;
  }
  return p.hd == 128 ? launch_hd<128>(p, st) : launch_hd<64>(p, st);
}

}  // namespace spec
