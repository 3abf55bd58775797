// Attention of the verify window over the 4-bit paged cache.
//
// For query row r (a window row and one of the query heads that share the kv head)
// and cached token k, with codes c, scale s, offset m:
//   S[r, k] = q_r . (s_k c_k + m_k) = s_k (q_r . c_k) + m_k sum(q_r)
//   O[r]    = sum_k P (s_k c_k + m_k) = sum_k (P s_k) c_k + sum_k P m_k
// so the tensor cores multiply the bare codes, and the two parameters of a token are
// applied to its score and its weight, in fp32.  Softmax is taken in one pass over
// the pages with a running maximum (of P s, below) and sum per row.
//
// Codes as fp16.  A nibble left in place, x & 0x000f000f, is a pair of fp16
// subnormals c * 2^-24 (x & 0x00f000f0: c * 2^-20), which the tensor cores multiply
// exactly: eight codes become four operand registers with four ANDs and a shift.
// The 2^-20 columns meet queries stored 1/16 as large; in the PV product they are
// separate output rows, scaled at the end.
//
// Tokens are the M side of both products (mma.sync m16n8k16, A = codes, B = queries
// or weights), so the work goes up in steps of 8 query rows, not 16: one decode or
// narrow window costs half.  S comes out as [token, row]; one movmatrix per 8 x 8
// tile turns the weights into the B operand of the PV product.
//
// Rounding.  P s_k is rounded to fp16: by 2^-11 of itself, or 2^-25 of the row's largest P s_k
// where it is subnormal (see the running maximum below).  c lies in 0..15, so that
// rounding would weigh on c's mean of 7.5 as well; the kernel sums the rounded
// weights R with one more MMA per step (A = ones) and forms
//   O = sum (P s)_fp16 c - 7.5 R + sum P (m + 7.5 s),
// which leaves only the rounding of the weights of c - 7.5.  Everything else is fp32.
//
// Work split.  A group is a sequence and a kv head.  Groups longer than a common target are
// cut into pieces of at most that many pages; a CTA takes one piece.  With few groups the target
// gives about as many pieces as the GPU holds CTAs.  The more groups there are, up to that number,
// the fewer cuts are left for the long ones (kv4_plan), and a batch of one long sequence
// among short ones is unbalanced there: width 4, 36 x 1024 + 1 x 32768 tokens 184 us, with 37 x 1024,
// where the rule for more groups than CTAs begins, 50; decode, 55 x 1024 + 1 x 65520 279, with 56 47.
// A group of one piece is finished by its CTA; the others leave partials (unnormalised O, running
// maximum and sum per row) in the workspace, and a second kernel merges them.  Short
// caches need neither: the CTAs of a group are one thread-block cluster and merge
// through distributed shared memory.  (One list of all pages cut into exactly equal
// shares was slower: a share that crosses from one group into the next pays the
// prologue and the epilogue twice.)  In a cluster every CTA sends each row's partial to the
// CTA that finishes the row, in one bulk copy per CTA, into memory kept for it: reading the
// others' partials instead took 3 to 8 thousand cycles more, a remote load at a time.
//
// A page of one kv head is one block (8704 bytes at head_dim 128) and one bulk copy
// into the CTA's ring.  A team of TW warps works on a page: with TW = 1 each of the
// four warps has pages of its own, with TW = 4 each takes 16 of the page's 64 tokens
// for S and the softmax and a quarter of the dims for the PV product, the weights
// passing through shared memory.  Either way every code is unpacked once per CTA.  A
// team of four keeps a warp's accumulators small (8 registers per 8 rows, against 32),
// so wide windows fit, and has a page's result sooner; one warp needs no barriers.
// Measured when the rule was made (head_dim 128, 8 kv heads; one warp, four): one row tile, 2 x
// 65520 tokens 32, 37 us; two, 8 x 32768 tokens 76, 83; three, 64 x 512-2048 tokens 63, 58 (8 x
// 32768 tokens 109, 111).  Teams of two warps have no figure: with the ring they had, a wait ran
// out.  In a team the scores of the next page are computed before the barrier that
// releases this page's weights: one barrier per page.
//
// What bounds it.  mma.sync runs at 8 cycles per m16n8k16 and SM quarter here and shares
// its pipe with the fp32 instructions; AND and shift take 2 cycles, exp2 and movmatrix 4
// (measured).  Per page and 16 query rows that is 272 + 75 cycles of the first pipe, 209
// of the integer pipe and 48 of the special functions; HBM delivers a page per SM in
// 365 at the 1.87 GHz of these runs.  Registers allow two CTAs per SM at two row tiles (222 a
// thread) and three at one (150), so two and three warps per SM quarter, and the pipes overlap
// little: 8 x 32768 tokens at 16 rows take at most 566 cycles a page where an SM has two CTAs,
// with 42% of the issue slots used, and 2 x 65520 tokens at 8 rows 460, prologue
// included, with 46%.  (At one and two tiles more CTAs per SM, for which the loop spilled, half pages,
// and packed fp32 pairs -- 3 cycles each -- were all slower.  Three and five tiles of 128 dims
// spill a few words at their bound of four and three CTAs.)  The wide windows were also built on tcgen05, codes unpacked into shared
// memory, S and O in tensor memory: with a token per thread a score costs twice the
// instructions, and the phases between its two barriers per tile do not overlap; 24 rows
// of 8 x 32768 tokens took 246 against 116 us, 60 rows 364 against 306.
//
// The running maximum of a row is that of t = score + floor(log2 s), s being V's scale, over the
// tokens the row sees: a token that it does not see, or hardly weighs, may have any scale.
// (One exponent for all rows, of the largest s alone, left the other weights few bits beside
// one such token.)  The weights are 2^(score - maximum), so their products with s lie
// below 2^9 and the largest is at least 1; the weights themselves and their sums, in fp32, may
// pass 2^32 where s is tiny.  The maximum of a row moves only when a t passes it by more than 8:
// the barrier (or vote) carries that question, asked of the largest score and the largest s of a
// thread's tokens, and the exact maxima, their exchange and the rescaling of the accumulators
// are a rare branch.  What a row does not see leaves no trace in its result.
//
// Large scores.  Queries and keys of +-65504, or a large `scale`, take scores past 2^24, where a
// float's last bit is a whole power of two of weight or more: score and maximum have to be numbers
// of one grid, or the largest weight is off by any power.  So the mantissa of scale * log2(e) goes
// into the products with s and m, and what is left of it for a row, with the row's own power of
// two, only shifts the score: a product and a difference without rounding.  floor(log2 s) is added
// to the score with a rounding towards the score, so the largest P s stays between
// min(1, s) and max(2, s).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "kv4.cuh"
#include "kv4.h"
#include "launch.cuh"

namespace spec {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxStages = 24;        // pages of a CTA's ring
constexpr float kNoMax = -1e30f;      // running maximum of a row that has seen no token
constexpr float kSlack = 8.f;         // how far t may pass the running maximum

SPEC_DEVICE_INLINE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D(16x8 fp32) += A(16x16 f16, row) * B(16x8 f16, col).  Not volatile: the compiler may
// order independent products, whose latency (21 cycles, 8 cycles apart) would
// otherwise show between two into one accumulator.
SPEC_DEVICE_INLINE void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with D = A * B.
SPEC_DEVICE_INLINE void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// floor(log2 s) of a parameter word; -24, the least scale's, where s is 0.
SPEC_DEVICE_INLINE float log2_scale(uint32_t w) {
  const uint32_t e = __float_as_uint(__half2float(__ushort_as_half((unsigned short)(w >> 16)))) >> 23;
  return fmaxf(__uint_as_float(0x4b000000u | e) - 8388735.f, -24.f);
}

// score + lg, rounded towards the score.
SPEC_DEVICE_INLINE float plus_log2(float score, float lg) {
  return lg < 0.f ? __fadd_ru(score, lg) : __fadd_rd(score, lg);
}

// 8 x 8 transpose of 16-bit elements across the warp.
SPEC_DEVICE_INLINE uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Barrier of a team (one warp or the CTA), and the same with an OR.
template <int TW>
SPEC_DEVICE_INLINE void team_sync() {
  if (TW == 1) __syncwarp();
  else __syncthreads();
}
template <int TW>
SPEC_DEVICE_INLINE bool team_any(bool x) {
  return TW == 1 ? __any_sync(0xffffffffu, x) : __syncthreads_or(x);
}

SPEC_DEVICE_INLINE void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Bytes of this CTA's shared memory to another CTA of the cluster (shared::cluster addresses).
SPEC_DEVICE_INLINE void bulk_push(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// Window geometry of sequence b, from the call's tables.
struct Kv4Seq {
  int sid, row0, Wb, L, n_keys, pages;
};
SPEC_DEVICE_INLINE Kv4Seq kv4_seq(const Kv4AttnParams& p, int b) {
  Kv4Seq s;
  s.sid = p.seq_ids ? p.seq_ids[b] : b;
  s.row0 = p.row_begin ? p.row_begin[b] : b * p.W;
  s.Wb = p.row_count ? p.row_count[b] : p.row_begin ? p.row_begin[b + 1] - s.row0 : p.W;
  s.row0 = max(0, min(s.row0, p.total_rows));
  s.Wb = max(0, min(min(s.Wb, p.W), p.total_rows - s.row0));
  const int cap = p.max_pages * kPage;
  s.L = max(-kMaxWidth, min(p.kv_len[b], cap));  // below 0: the window's first rows have no cell
  s.n_keys = s.sid >= 0 && s.sid < p.table_rows && s.Wb > 0 ? max(0, min(s.L + s.Wb, cap)) : 0;
  s.pages = (s.n_keys + kPage - 1) / kPage;
  return s;
}

// How the groups are cut into pieces, one CTA each.  All pieces of a call have about
// `target` pages; a group of that many or fewer is one piece.
struct Kv4Plan {
  int target, total;  // total: pieces of all groups
};
SPEC_DEVICE_INLINE int kv4_pieces(int pages, int target) { return (pages + target - 1) / target; }

// Sequence `lane` of the first 32 (every warp starts with it: most batches need no other).
SPEC_DEVICE_INLINE Kv4Seq kv4_first_seqs(const Kv4AttnParams& p) {
  const int lane = threadIdx.x & 31;
  Kv4Seq s{};
  if (lane < p.B) s = kv4_seq(p, lane);
  return s;
}
SPEC_DEVICE_INLINE Kv4Seq kv4_seq_at(const Kv4AttnParams& p, const Kv4Seq& mine, int b) {
  if (b >= 32) return kv4_seq(p, b);
  Kv4Seq s;
  s.sid = __shfl_sync(0xffffffffu, mine.sid, b);
  s.row0 = __shfl_sync(0xffffffffu, mine.row0, b);
  s.Wb = __shfl_sync(0xffffffffu, mine.Wb, b);
  s.L = __shfl_sync(0xffffffffu, mine.L, b);
  s.n_keys = __shfl_sync(0xffffffffu, mine.n_keys, b);
  s.pages = __shfl_sync(0xffffffffu, mine.pages, b);
  return s;
}
// With fewer groups than slots (CTAs the GPU holds at once) the pieces fit the slots: every
// group has at most pages / target + 1.  With more, a group is cut only if it is longer
// than a slot's share of all pages.
SPEC_DEVICE_INLINE Kv4Plan kv4_plan(const Kv4AttnParams& p, const Kv4Seq& mine) {
  const int lane = threadIdx.x & 31;
  int n = mine.pages;
  for (int b = lane + 32; b < p.B; b += 32) n += kv4_seq(p, b).pages;
  n = (int)__reduce_add_sync(0xffffffffu, (unsigned)n) * p.Hkv;
  const int groups = p.B * p.Hkv;
  const int share = groups < p.slots ? p.slots - groups : p.slots;
  Kv4Plan r;
  r.target = max(1, (n + share - 1) / share);
  int k = kv4_pieces(mine.pages, r.target);
  for (int b = lane + 32; b < p.B; b += 32) k += kv4_pieces(kv4_seq(p, b).pages, r.target);
  r.total = (int)__reduce_add_sync(0xffffffffu, (unsigned)k) * p.Hkv;
  return r;
}
// The sequence that holds piece x (below the total; per sequence all pieces of head 0, then
// head 1, ...), and the pieces before it: of all sequences, and of those cut in two or more.
SPEC_DEVICE_INLINE int kv4_find_piece(const Kv4AttnParams& p, const Kv4Seq& mine, int target, int x, int& before,
                                      int& before_cut) {
  const int lane = threadIdx.x & 31;
  int base = 0, base_cut = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int pages = b0 == 0 ? mine.pages : b0 + lane < p.B ? kv4_seq(p, b0 + lane).pages : 0;
    const int n = kv4_pieces(pages, target) * p.Hkv, nc = n > p.Hkv ? n : 0;
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
SPEC_DEVICE_INLINE float* kv4_partial(float* ws, int i, int rows, int hd) {
  return ws + (long long)i * rows * (hd + 2);
}

// Two output values as fp16, saturated; what is no number stays none.
SPEC_DEVICE_INLINE uint32_t out_f16x2(float a, float b) {
  const __half2 most = __float2half2_rn(65504.f);
  const __half2 v = __hmin2_nan(__hmax2_nan(__floats2half2_rn(a, b), __hneg2(most)), most);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four output values of a row: o / l in the caller's type; a row that sees no token is zeros.
SPEC_DEVICE_INLINE void store_row4(const Kv4AttnParams& p, int row, int head, int hd, int d4, float4 o, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint2 w;
  if (p.bf16) {
    w.x = kv4_pack2<true>(o.x * inv, o.y * inv);
    w.y = kv4_pack2<true>(o.z * inv, o.w * inv);
  } else {
    w.x = out_f16x2(o.x * inv, o.y * inv);
    w.y = out_f16x2(o.z * inv, o.w * inv);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + ((long long)row * p.Hq + head) * hd + d4 * 4) = w;
}

// V words of 16-token step t for a lane whose chunk starts at v: NPIECE pieces of tokens
// {2c, 2c+1} (x0) and {2c+8, 2c+9} (x1).
template <int HD, int NPIECE>
SPEC_DEVICE_INLINE void kv4_v_words(const uint8_t* v, int t, uint32_t (&x0)[NPIECE], uint32_t (&x1)[NPIECE]) {
  const uint8_t* a = v + t * (HD == 128 ? 1024 : 512);
  const uint8_t* d = a + (HD == 128 ? 512 : 8);
  if constexpr (HD == 64 && NPIECE == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(a);
    x0[0] = w.x, x0[1] = w.y, x1[0] = w.z, x1[1] = w.w;
  } else if constexpr (NPIECE == 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(d);
    x0[0] = w.x, x0[1] = w.y, x0[2] = w.z, x0[3] = w.w;
    x1[0] = y.x, x1[1] = y.y, x1[2] = y.z, x1[3] = y.w;
  } else if constexpr (NPIECE == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(d);
    x0[0] = w.x, x0[1] = w.y;
    x1[0] = y.x, x1[1] = y.y;
  } else {
    x0[0] = *reinterpret_cast<const uint32_t*>(a);
    x1[0] = *reinterpret_cast<const uint32_t*>(d);
  }
}

// HD: head_dim; NT: tiles of 8 query rows; TW: warps of a team.
template <int HD, int NT, int TW>
struct Cfg {
  static constexpr int kPieces = HD / 32 >= TW ? HD / 32 / TW : 1;  // V words of a token pair per warp
  static constexpr int kTeams = kWarps / TW;
  static constexpr int kBlock = kPage * HD + 2 * kPage * 4;    // bytes of a page of one kv head: a stage
  // CTAs per SM by the registers of a warp
  static constexpr int kRegs = NT * (HD / 4 / TW + 8 + 16 / TW) + (TW == 1 ? 90 : 68);
  static constexpr int kCtas = kRegs <= 128 ? 4 : kRegs <= 168 ? 3 : 2;
  static constexpr int kQ = NT * (HD / 32) * 512;              // query fragments
  static constexpr int kP = TW == 1 ? 0 : 2 * NT * 1024;       // weights of two pages
  static constexpr int kFixed = kQ + kP;
  static constexpr int kStatic = NT * 8 * 4 * (5 + 2 * kWarps + kTeams) + 512;  // static shared memory, at most
  static constexpr int kRec = HD + 4;                          // floats of a row's partial: O, maximum, sum
  // A cluster's partials of this CTA's rows: cs ceil(rows / cs) records at most, cs up to 16.
  static constexpr int kRecv = (NT + 1) / 2 * 16 * kRec * 4;
  // Ring depth with `ctas` CTAs on an SM: 228 KB, 1 KB of system use per CTA.  A multiple
  // of the teams, so that the pages of one stage are one team's, in order: a team that
  // waited for a stage's next page while another team's was still in flight would take
  // the phase before for its own.
  static constexpr int stages(int ctas, int other = 0) {
    const int n = (233472 / ctas - 1024 - kStatic - kFixed - other) / kBlock;
    return (n < kMaxStages ? n : kMaxStages) / kTeams * kTeams;
  }
  static_assert(kCtas <= (NT <= 3 ? 4 : 3), "workspace");
  // a team refills a stage two of its pages late and computes scores one page ahead
  static_assert(TW == 1 || TW == kWarps, "a team is one warp or the CTA");
  static_assert(stages(kCtas) >= (TW == 1 ? 2 : 4) * kTeams, "ring");
  static_assert(kTeams * NT * 8 * HD * 4 <= stages(kCtas) * kBlock, "the teams' partials reuse the ring");
  static_assert(TW == 1 || (stages(2, kRecv) >= 4 && NT * 8 * kRec * 4 <= stages(2, kRecv) * kBlock), "clusters");
};

// Query row r of the CTA is window row r / grp, head r % grp of the group.
// CL: a group's pieces are the CTAs of one thread-block cluster (gridDim.x / (B Hkv) of them,
// possibly one), merged through distributed shared memory.
template <int HD, int NT, int TW, bool CL>
__global__ void __launch_bounds__(kThreads, (Cfg<HD, NT, TW>::kCtas))
    kv4_attention_kernel(const __grid_constant__ Kv4AttnParams p) {
  using C = Cfg<HD, NT, TW>;
  constexpr int WORDS = HD / 32;     // 32-bit words of K codes per lane and token
  constexpr int MT = 4 / TW;         // 16-token steps of a page per warp (S and softmax)
  constexpr int PW = WORDS * 2 / TW; // 16-row tiles of the PV product per warp
  constexpr int TEAMS = C::kTeams;
  constexpr int ROWS = NT * 8;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const ring = smem;
  const int S = p.stages;            // ring depth
  uint8_t* const qfrag = smem + S * C::kBlock;
  __shared__ uint64_t full[kMaxStages];
  __shared__ float4 s_row[ROWS / 2];          // rows 2i, 2i + 1: sums of q, factors to exp2 units
  __shared__ float2 s_max[TEAMS][ROWS / 2];   // running maxima of t
  __shared__ float s_red[kWarps][ROWS], s_red2[kWarps][ROWS];
  __shared__ uint64_t received;               // partials of the cluster's CTAs
  __shared__ uint32_t s_anc[16];
  __shared__ int s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / TW, tw = warp % TW;
  const int g = lane >> 2, c = lane & 3;
  const int grp = p.Hq / p.Hkv;
  uint8_t* const pfrag = qfrag + C::kQ;

  // the merge kernel reads the call's tables before its own wait, so it may only start
  // once they are complete
  if (!p.early) pdl_wait();
  // Clusters let the next kernel in only as they end: its first CTAs would take places that
  // its other clusters, if it has any, then lack (back to back, 32 clusters of 8 CTAs took 24
  // against 17 us; let in after the loop, 22).
  if (!CL) pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    if (CL) mbar_init(&received, 1);
    s_fail = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 16) s_anc[threadIdx.x] = p.anc[threadIdx.x];

  if (threadIdx.x < ROWS / 2)
#pragma unroll
    for (int i = 0; i < TEAMS; ++i) s_max[i][threadIdx.x] = make_float2(kNoMax, kNoMax);

  // this CTA's share of the next projections' weights
  auto prefetch_next = [&] {
    if (threadIdx.x == kThreads - 1) {
      l2_prefetch_share(p.l2_next[0], p.l2_next_bytes[0]);
      l2_prefetch_share(p.l2_next[1], p.l2_next_bytes[1]);
    }
  };

  int kvh, piece, pieces, slot = 0;
  Kv4Seq seq;
  if constexpr (CL) {
    pieces = p.cluster;
    piece = blockIdx.x % pieces;
    const int group = blockIdx.x / pieces;
    kvh = group % p.Hkv;
    seq = kv4_seq(p, group / p.Hkv);
  } else {
    const Kv4Seq mine = kv4_first_seqs(p);
    const Kv4Plan plan = kv4_plan(p, mine);
    if ((int)blockIdx.x >= plan.total) {
      if (p.early) pdl_wait();  // the grid's end stands for the predecessor's, too
      prefetch_next();
      return;
    }
    int before, before_cut;
    const int b = kv4_find_piece(p, mine, plan.target, blockIdx.x, before, before_cut);
    seq = kv4_seq_at(p, mine, b);
    pieces = kv4_pieces(seq.pages, plan.target);
    kvh = (blockIdx.x - before) / pieces;
    piece = (blockIdx.x - before) % pieces;
    slot = before_cut + (blockIdx.x - before);
  }
  const int pg0 = (int)((long long)seq.pages * piece / pieces);
  const int npg = (int)((long long)seq.pages * (piece + 1) / pieces) - pg0;
  const int L = seq.L, n_keys = seq.n_keys, Wb = seq.Wb, row0 = seq.row0, rows = seq.Wb * grp;
  const int key_base = pg0 * kPage;
  bool failed = false;
  // a cluster's CTA finishes rows [own0, own0 + own)
  const int share = CL ? (rows + pieces - 1) / pieces : 0;
  const int own0 = share * piece, own = max(0, min(rows - own0, share));
  __syncthreads();
  if (CL && pieces > 1) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&received, pieces * own * C::kRec * 4);
    __syncwarp();
    cluster_arrive();  // its barrier is ready to receive
  }

  // Page numbers of the piece's pages [base, base + 32) and the 32 after them, one per
  // lane, and which of the first 32 are there.
  const int32_t* table = p.page_table + (long long)seq.sid * p.max_pages + pg0;
  auto page_at = [&](int j) {
    const int pg = j < npg ? table[j] : -1;
    return pg < p.num_pages ? pg : -1;
  };
  int pid0 = page_at(lane), pid1 = page_at(32 + lane);
  uint32_t there = __ballot_sync(0xffffffffu, pid0 >= 0);
  int base = 0;
  // Start the copy of page j into stage s (an absent page completes its phase empty); j is
  // in [base, base + 64), a whole warp calls it.
  auto issue = [&](int j, int s) {
    const int pg = __shfl_sync(0xffffffffu, j - base < 32 ? pid0 : pid1, j & 31);
    if (lane == 0) {
      if (pg >= 0) {
        mbar_arrive_expect_tx(&full[s], C::kBlock);
        bulk_load(ring + s * C::kBlock, p.pool + ((long long)pg * p.Hkv + kvh) * C::kBlock, C::kBlock, &full[s]);
      } else {
        mbar_arrive(&full[s]);
      }
    }
  };
  int issued = 0;
  if (p.early) {
    // before pdl_wait only pages without window slots may be read
    if (warp == 0)
      for (; issued < min(S, npg) && key_base + (issued + 1) * kPage <= L; ++issued) issue(issued, issued);
    pdl_wait();
  }
  // Queries: a lane takes eight dims of a row, two rows (head_dim 64: four) at a time per
  // warp, all loads before the pages' (which they would queue behind).  Each row is scaled
  // by a power of two (largest element in [2^14, 2^15)), so the factor 1/16 of the odd
  // columns costs no precision; the sum of the scaled row and the factor (a power of two) back to
  // exp2 units are kept per row.
  constexpr int RPP = HD == 128 ? 2 : 4;                       // rows of a warp at a time
  constexpr int QP = (ROWS + kWarps * RPP - 1) / (kWarps * RPP);
  const int q_cc = lane & 3, q_w = lane / (4 * RPP);           // dims (q_cc WORDS + q_w) 8 ..
  const int q_r = warp * RPP + ((lane >> 2) & (RPP - 1));      // rows q_r, q_r + kWarps RPP, ..
  uint4 raw[QP];
#pragma unroll
  for (int k = 0; k < QP; ++k) {
    const int r = q_r + k * kWarps * RPP;
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows)
      raw[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (row0 + r / grp) * p.q_row_stride +
                                               (long long)(kvh * grp + r % grp) * HD + (q_cc * WORDS + q_w) * 8);
  }
  if (warp == 0)
    for (; issued < min(S, npg); ++issued) issue(issued, issued);
  prefetch_next();
#pragma unroll
  for (int k = 0; k < QP; ++k) {
    const uint32_t in[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    float x[8], mx = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = p.bf16 ? kv4_unpack2<true>(in[i]) : kv4_unpack2<false>(in[i]);
      x[2 * i] = kv4_sat(f.x);
      x[2 * i + 1] = kv4_sat(f.y);
      mx = fmaxf(mx, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o < 4 || o >= 4 * RPP) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^sh with 2^14 <= mx 2^sh < 2^15; rows below 2^-112 count as zeros (|scale| <= 2^40)
    const int sh = mx > 1.9259299e-34f ? 14 - (int)((__float_as_uint(mx) >> 23) - 127u) : 0;
    const float up = __uint_as_float(((uint32_t)(127 + sh) << 23) | (p.scale < 0.f ? 0x80000000u : 0u));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= up;
      sum += x[i];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (o < 4 || o >= 4 * RPP) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int r = q_r + k * kWarps * RPP;
    if (r < ROWS) {
      if (q_cc == 0 && q_w == 0) {
        float* row = reinterpret_cast<float*>(&s_row[r >> 1]) + (r & 1);
        row[0] = sum * (p.scale_m * 5.9604644775390625e-8f);  // in the units of the code products (2^-24)
        row[2] = fmaxf(p.scale_2 * 16777216.f * __uint_as_float((uint32_t)(127 - sh) << 23), 0x1p-100f);
      }
      // fragment of lane (r % 8, q_cc), word q_w: halves (d0, d4) (d1, d5)/16 (d2, d6) (d3, d7)/16
      *reinterpret_cast<uint4*>(qfrag + (((r >> 3) * WORDS + q_w) * 32 + (r & 7) * 4 + q_cc) * 16) =
          make_uint4(pack_f16x2(x[0], x[4]), pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f), pack_f16x2(x[2], x[6]),
                     pack_f16x2(x[3] * 0.0625f, x[7] * 0.0625f));
    }
  }
  __syncthreads();

  float acc[NT][PW][4], accr[NT][4];        // codes^T . weights, and the weights' sums
  float lrow[NT][2], zrow[NT][2];           // rows 2c, 2c + 1
  float sc[NT][MT][4];                      // scores / factor: tokens g, g + 8 of a step; rows 2c, 2c + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < PW; ++t) acc[nt][t][0] = acc[nt][t][1] = acc[nt][t][2] = acc[nt][t][3] = 0.f;
    accr[nt][0] = accr[nt][1] = accr[nt][2] = accr[nt][3] = 0.f;
    lrow[nt][0] = lrow[nt][1] = zrow[nt][0] = zrow[nt][1] = 0.f;
  }
  uint32_t vw[2 * MT];                      // V parameter words of the lane's tokens

  const int kk = tw * MT * 16 + g;          // this lane's first token in a page
  // Scores of page j (in stage s, phase parity par) into sc; returns whether a t may pass its
  // row's maximum by more than the slack.
  auto scores = [&](int j, int s, uint32_t par) -> bool {
    if (j - base >= 32) {
      base += 32;
      pid0 = pid1;
      there = __ballot_sync(0xffffffffu, pid0 >= 0);
      pid1 = page_at(base + 32 + lane);
    }
    // a wait that runs out is the warp's last: it goes on without data, so that the
    // CTA's barriers stay whole, and its rows come out as NaN
    if (!failed && !mbar_wait(&full[s], par, p.status)) {
      failed = true;
      s_fail = 1;
    }
    const uint8_t* st = ring + s * C::kBlock;
    const uint32_t* kpar = reinterpret_cast<const uint32_t*>(st + kPage * HD) + kk;
    uint32_t kw[2 * MT];
#pragma unroll
    for (int t = 0; t < 2 * MT; ++t) {
      kw[t] = kpar[8 * t];
      vw[t] = kpar[kPage + 8 * t];
    }
    // two steps at a time: enough independent products to cover their latency
    constexpr int HB = MT < 2 ? 1 : 2;
#pragma unroll
    for (int h = 0; h < MT; h += HB) {
      uint32_t kc[2 * HB][WORDS];
#pragma unroll
      for (int t = 0; t < 2 * HB; ++t) {
        const uint8_t* a = st + (kk + 16 * h + 8 * t) * (HD / 2) + c * (HD / 8);
        if constexpr (WORDS == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(a);
          kc[t][0] = v.x, kc[t][1] = v.y, kc[t][2] = v.z, kc[t][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(a);
          kc[t][0] = v.x, kc[t][1] = v.y;
        }
      }
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        uint4 q[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          q[nt] = *reinterpret_cast<const uint4*>(qfrag + ((nt * WORDS + w) * 32 + lane) * 16);
#pragma unroll
        for (int t = 0; t < HB; ++t) {
          const uint32_t x0 = kc[2 * t][w], x1 = kc[2 * t + 1][w];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (w == 0)
              mma0(sc[nt][h + t], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, q[nt].x,
                   q[nt].y);
            else
              mma(sc[nt][h + t], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, q[nt].x,
                  q[nt].y);
          }
        }
#pragma unroll
        for (int t = 0; t < HB; ++t) {
          const uint32_t y0 = kc[2 * t][w] >> 8, y1 = kc[2 * t + 1][w] >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(sc[nt][h + t], y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, q[nt].z,
                q[nt].w);
        }
      }
    }
    const int key0 = key_base + j * kPage;
    const bool here = (there >> (j & 31)) & 1u;
    const bool masked = key0 + kPage > L || !here;
    if (masked) {
      const int end = here ? n_keys : 0;
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t)
        if (key0 + kk + 8 * t >= end) kw[t] = vw[t] = 0;  // never written: may hold anything
    }
    float km[2 * MT], ks[2 * MT];
    uint32_t smax = 0;
#pragma unroll
    for (int t = 0; t < 2 * MT; ++t) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&kw[t]));
      km[t] = f.x;
      ks[t] = f.y * p.scale_m;
      smax = max(smax, vw[t]);
    }
    const float lim = kSlack - log2_scale(smax);
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 row = s_row[nt * 4 + c];
      const float2 top = s_max[team][nt * 4 + c];
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        float* x = &sc[nt][t >> 1][(t & 1) * 2];
        x[0] = fmaf(ks[t], x[0], km[t] * row.x);
        x[1] = fmaf(ks[t], x[1], km[t] * row.y);
      }
      if (masked) {
        // window slots are seen by their descendants only; slots past the window by nobody
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * c + e;
          const uint32_t anc = r < rows && here ? s_anc[r / grp] & ((1u << Wb) - 1u) : 0u;
#pragma unroll
          for (int t = 0; t < 2 * MT; ++t) {
            const int w = key0 + kk + 8 * t - L;
            const bool vis = w < 0 ? here : w < 16 && ((anc >> w) & 1u) && w + L < n_keys;
            if (!vis) sc[nt][t >> 1][(t & 1) * 2 + e] = -INFINITY;
          }
        }
      }
      float m0 = sc[nt][0][0], m1 = sc[nt][0][1];
#pragma unroll
      for (int t = 1; t < 2 * MT; ++t) {
        m0 = fmaxf(m0, sc[nt][t >> 1][(t & 1) * 2]);
        m1 = fmaxf(m1, sc[nt][t >> 1][(t & 1) * 2 + 1]);
      }
      over |= fmaf(m0, row.z, -top.x) > lim || fmaf(m1, row.w, -top.y) > lim;
    }
    return over;
  };

  // Move the running maxima that a t of this page passes by more than the slack, and rescale the
  // accumulators.
  auto raise_max = [&] {
    float lg[2 * MT];
#pragma unroll
    for (int t = 0; t < 2 * MT; ++t) lg[t] = log2_scale(vw[t]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 row = s_row[nt * 4 + c];
      float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        m0 = fmaxf(m0, plus_log2(sc[nt][t >> 1][(t & 1) * 2] * row.z, lg[t]));
        m1 = fmaxf(m1, plus_log2(sc[nt][t >> 1][(t & 1) * 2 + 1] * row.w, lg[t]));
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      }
      if (g == 0) {
        s_red[warp][nt * 8 + 2 * c] = m0;
        s_red[warp][nt * 8 + 2 * c + 1] = m1;
      }
    }
    team_sync<TW>();
    // the maximum of row r, `old` until now
    const auto raised = [&](float old, int r) {
      float m = s_red[team * TW][r];
#pragma unroll
      for (int w = 1; w < TW; ++w) m = fmaxf(m, s_red[team * TW + w][r]);
      return m - old >= kSlack ? m : old;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 old = s_max[team][nt * 4 + c];
      const float a0 = ex2(old.x - raised(old.x, nt * 8 + 2 * c)), a1 = ex2(old.y - raised(old.y, nt * 8 + 2 * c + 1));
#pragma unroll
      for (int t = 0; t < PW; ++t) {
        acc[nt][t][0] *= a0;
        acc[nt][t][1] *= a1;
        acc[nt][t][2] *= a0;
        acc[nt][t][3] *= a1;
      }
      accr[nt][0] *= a0;
      accr[nt][1] *= a1;
      lrow[nt][0] *= a0;
      lrow[nt][1] *= a1;
      zrow[nt][0] *= a0;
      zrow[nt][1] *= a1;
    }
    team_sync<TW>();
    for (int r = tw * 32 + lane; r < ROWS; r += TW * 32) {
      float* top = reinterpret_cast<float*>(s_max[team]) + r;
      *top = raised(*top, r);
    }
    team_sync<TW>();
  };

  // Weights of 16-token step t of the page whose scores are in sc, as B fragments pb.
  uint32_t pb[NT][2 * MT];
  auto weights = [&](int t) {
    float vs[2], vz[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&vw[2 * t + u]));
      vs[u] = f.y;
      vz[u] = fmaf(7.5f, f.y, f.x);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 row = s_row[nt * 4 + c];
      const float2 top = s_max[team][nt * 4 + c];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float* x = &sc[nt][t][u * 2];
        const float w0 = ex2(fmaf(x[0], row.z, -top.x)), w1 = ex2(fmaf(x[1], row.w, -top.y));
        lrow[nt][0] += w0;
        lrow[nt][1] += w1;
        zrow[nt][0] = fmaf(w0, vz[u], zrow[nt][0]);
        zrow[nt][1] = fmaf(w1, vz[u], zrow[nt][1]);
        pb[nt][2 * t + u] = movmatrix_trans(pack_f16x2(w0 * vs[u], w1 * vs[u]));
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      mma(accr[nt], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pb[nt][2 * t], pb[nt][2 * t + 1]);
  };

  // Pieces (words of a token pair) of this lane: which of a chunk's words it takes varies
  // with g, so that the 32 lanes of a narrow load hit all banks (any dim may be any row
  // of the product).
  constexpr int NPIECE = C::kPieces;
  int piece0 = 0;  // first of them
  if (TW == kWarps) piece0 = HD == 128 ? tw ^ (g >> 1) : (tw >> 1) ^ ((g >> 1) & 1);
  const int v_off = kPage * HD / 2 + c * 128 + ((g ^ (2 * c)) << 4) + piece0 * 4;
  // PV product of the 16-token step t of the page whose V codes (of this lane) start at v.
  auto pv_step = [&](const uint8_t* v, int t, const uint32_t (&b)[NT][2]) {
    uint32_t x0[NPIECE], x1[NPIECE];  // tokens {2c, 2c+1} and {2c+8, 2c+9}
    kv4_v_words<HD, NPIECE>(v, t, x0, x1);
    if (PW == 1 && (tw & 1)) x0[0] >>= 8, x1[0] >>= 8;  // head_dim 64, team of four: half of a piece's dims
#pragma unroll
    for (int w = 0; w < NPIECE; ++w) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma(acc[nt][(2 * w) % PW], x0[w] & 0x000f000fu, x0[w] & 0x00f000f0u, x1[w] & 0x000f000fu, x1[w] & 0x00f000f0u,
            b[nt][0], b[nt][1]);
      if (PW > 1) {
        const uint32_t y0 = x0[w] >> 8, y1 = x1[w] >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma(acc[nt][(2 * w + 1) % PW], y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu, y1 & 0x00f000f0u,
              b[nt][0], b[nt][1]);
      }
    }
  };

  // The team's pages: team, team + TEAMS, ...; page j is in stage j % S.
  int s = team, ps = 0;   // stages of the team's current page and of the one before
  uint32_t par = 0;
  auto advance = [&] {
    ps = s;
    s += TEAMS;
    if (s >= S) {
      s -= S;
      par ^= 1u;
    }
  };
  if constexpr (TW == 1) {
    for (int j = team; j < npg; j += TEAMS) {
      if (team_any<1>(scores(j, s, par))) raise_max();
      // the weights of a step are computed beside the products of the step before: the
      // exp2 and transposes then run under the tensor cores
      const uint8_t* v = ring + s * C::kBlock + v_off;
      weights(0);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (t + 1 < MT) weights(t + 1);
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt][0] = pb[nt][2 * t], b[nt][1] = pb[nt][2 * t + 1];
        pv_step(v, t, b);
      }
      __syncwarp();
      fence_proxy_async();  // the stage was read through the generic proxy
      if (j + S < npg) issue(j + S, s);
      advance();
    }
  } else {
    bool over = npg > 0 && scores(0, s, par);
    uint8_t* pf0 = pfrag + lane * 16;  // weights: [page parity][nt][step / 2][lane][step % 2], 8 bytes each
    for (int j = 0;; ++j) {
      // after this barrier the weights of page j - 1 are stored, and every warp has left
      // the PV product of page j - 2
      const bool any = team_any<TW>(over);
      if (j > 0) {
        if (warp == 0 && j > 1 && j - 2 + S < npg) {
          fence_proxy_async();  // the stage was read through the generic proxy
          issue(j - 2 + S, ps == 0 ? S - 1 : ps - 1);
        }
        const uint8_t* v = ring + ps * C::kBlock + v_off;
        const uint8_t* pf = pf0 + ((j - 1) & 1) * (NT * 1024);
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          uint4 pw[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) pw[nt] = *reinterpret_cast<const uint4*>(pf + (nt * 2 + t2) * 512);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t b[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) b[nt][0] = u ? pw[nt].z : pw[nt].x, b[nt][1] = u ? pw[nt].w : pw[nt].y;
            pv_step(v, t2 * 2 + u, b);
          }
        }
      }
      if (j >= npg) break;
      if (any) raise_max();
      weights(0);
      uint8_t* pf = pf0 + (j & 1) * (NT * 1024) + (tw >> 1) * 512 + (tw & 1) * 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) *reinterpret_cast<uint2*>(pf + nt * 1024) = make_uint2(pb[nt][0], pb[nt][1]);
      advance();
      over = j + 1 < npg && scores(j + 1, s, par);
    }
  }
  if (failed) {
    // give copies still in flight the same time to land before the
    // CTA's shared memory is given up
    (void)mbar_wait(&full[lane % S], 0, nullptr);
    (void)mbar_wait(&full[lane % S], 1, nullptr);
  }
  __syncthreads();
  // The teams' partials: sums over the team's tokens, then O, in the ring's place.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float2 l = make_float2(lrow[nt][0], lrow[nt][1]), z = make_float2(zrow[nt][0], zrow[nt][1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l.x += __shfl_xor_sync(0xffffffffu, l.x, o);
      l.y += __shfl_xor_sync(0xffffffffu, l.y, o);
      z.x += __shfl_xor_sync(0xffffffffu, z.x, o);
      z.y += __shfl_xor_sync(0xffffffffu, z.y, o);
    }
    if (g == 0) {
      s_red[warp][nt * 8 + 2 * c] = l.x;
      s_red[warp][nt * 8 + 2 * c + 1] = l.y;
      s_red2[warp][nt * 8 + 2 * c] = z.x - 7.5f * accr[nt][0];
      s_red2[warp][nt * 8 + 2 * c + 1] = z.y - 7.5f * accr[nt][1];
    }
  }
  team_sync<TW>();
  constexpr int REC = CL ? C::kRec : HD;  // floats of a row
  float* const part = reinterpret_cast<float*>(ring);  // [TEAMS][ROWS][REC]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * c + e;
      float bias = 0.f;
#pragma unroll
      for (int w = 0; w < TW; ++w) bias += s_red2[team * TW + w][r];
      constexpr float u0 = 16777216.f, u1 = 1048576.f;  // a nibble left in place is c 2^-24 or 2^-20
      float* o = part + (team * ROWS + r) * REC + g * (HD / 8) + piece0 * 4;
      if constexpr (PW == 1)
        *reinterpret_cast<float2*>(o + (tw & 1) * 2) =
            make_float2(fmaf(acc[nt][0][e], u0, bias), fmaf(acc[nt][0][2 + e], u1, bias));
      else
#pragma unroll
        for (int w = 0; w < PW / 2; ++w)
          *reinterpret_cast<float4*>(o + w * 4) =
              make_float4(fmaf(acc[nt][2 * w][e], u0, bias), fmaf(acc[nt][2 * w][2 + e], u1, bias),
                          fmaf(acc[nt][(2 * w + 1) % PW][e], u0, bias), fmaf(acc[nt][(2 * w + 1) % PW][2 + e], u1, bias));
    }
  constexpr int V4 = HD / 4;
  if constexpr (CL) {
    if (pieces > 1) {
      // Every CTA sends each row's partial to the CTA that finishes the row, one bulk copy per
      // CTA, and merges what it receives: sum_i 2^(m_i - M) o_i over the cluster.
      if (threadIdx.x < ROWS) {
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < TW; ++k) l += s_red[k][threadIdx.x];
        const float m = reinterpret_cast<const float*>(s_max[0])[threadIdx.x];
        // a wait that ran out: a maximum that is NaN makes the row NaN
        *reinterpret_cast<float2*>(part + threadIdx.x * REC + HD) = make_float2(s_fail ? NAN : m, l);
      }
      fence_proxy_async();
      __syncthreads();
      cluster_wait();  // every CTA's barrier is ready
      float* const recv = reinterpret_cast<float*>(qfrag + C::kFixed);  // [pieces][own][REC]
      if (threadIdx.x < pieces) {
        const int n = max(0, min(rows - share * (int)threadIdx.x, share));
        if (n > 0)
          bulk_push(mapa_u32(smem_u32(recv + piece * n * REC), threadIdx.x), part + threadIdx.x * share * REC, n * REC * 4,
                    mapa_u32(smem_u32(&received), threadIdx.x));
      }
      __syncwarp();
      cluster_arrive_relaxed();  // this CTA's copies are issued (with the release a round of 32 layers took 10 us more)
      const bool ok = mbar_wait(&received, 0, p.status);
      __syncwarp();
      cluster_wait();
      // all copies are issued, also those of a CTA that this one did not wait out: they land now
      if (!ok) (void)mbar_wait(&received, 0, nullptr);
      __syncwarp();
      cluster_arrive();  // all copies to this CTA have landed: when all have, no source is needed
      for (int it = threadIdx.x; it < own * V4; it += kThreads) {
        const int r = it / V4, d4 = it % V4;
        float M = kNoMax, l = 0.f, m[16];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < pieces) {
            m[i] = recv[(i * own + r) * REC + HD];
            M = fmaxf(M, m[i]);
          }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < pieces) {
            const float4 x = *reinterpret_cast<const float4*>(recv + (i * own + r) * REC + d4 * 4);
            const float w = ex2(m[i] - M);
            l = fmaf(w, recv[(i * own + r) * REC + HD + 1], l);
            o.x = fmaf(w, x.x, o.x);
            o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z);
            o.w = fmaf(w, x.w, o.w);
          }
        if (!ok) o = make_float4(NAN, NAN, NAN, NAN), l = 1.f;
        const int row = own0 + r;
        store_row4(p, row0 + row / grp, kvh * grp + row % grp, HD, d4, o, l);
      }
      __syncwarp();
      cluster_wait();
      return;
    }
  }
  __syncthreads();
  // the CTA's: sum_i 2^(m_i - M) o_i over the teams; normalised and rounded where the
  // group is whole, else left in the workspace
  {
    const bool whole = pieces == 1;
    float* const ws = CL ? nullptr : kv4_partial(p.workspace, slot, ROWS, HD);
    for (int it = threadIdx.x; it < rows * V4; it += kThreads) {
      const int r = it / V4, d4 = it % V4;
      float m[TEAMS], M = kNoMax, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < TEAMS; ++i) {
        m[i] = reinterpret_cast<const float*>(s_max[i])[r];
        M = fmaxf(M, m[i]);
      }
#pragma unroll
      for (int i = 0; i < TEAMS; ++i) {
        const float w = TEAMS == 1 ? 1.f : ex2(m[i] - M);
        const float4 x = *reinterpret_cast<const float4*>(part + (i * ROWS + r) * REC + d4 * 4);
        o.x = fmaf(w, x.x, o.x);
        o.y = fmaf(w, x.y, o.y);
        o.z = fmaf(w, x.z, o.z);
        o.w = fmaf(w, x.w, o.w);
#pragma unroll
        for (int k = 0; k < TW; ++k) l = fmaf(w, s_red[i * TW + k][r], l);
      }
      if (s_fail) o = make_float4(NAN, NAN, NAN, NAN), l = 1.f;  // a wait ran out
      if (CL || whole) {
        store_row4(p, row0 + r / grp, kvh * grp + r % grp, HD, d4, o, l);
      } else {
        *reinterpret_cast<float4*>(ws + r * HD + d4 * 4) = o;
        if (d4 == 0) {
          ws[ROWS * HD + r] = M;
          ws[ROWS * HD + ROWS + r] = l;
        }
      }
    }
  }
}

// Merge the partials of one cut group: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// grid (shares of a group's rows, Hkv, B).  A group of few has many partials, and reading them
// one after the other is what a merge costs: hd / 4 lanes take a row, and up to all warps
// share its partials, eight loads in flight each.
__host__ __device__ constexpr int merge_split(int n, int warps) {  // warps of a row, a power of two
  int split = 1;
  while (split < warps && split * (warps == 16 ? 4 : 8) < n) split *= 2;
  return split;
}
template <int HD, int kMergeWarps>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv4_merge_kernel(const __grid_constant__ Kv4AttnParams p, int ws_rows) {
  constexpr int V4 = HD / 4;
  constexpr int RPW = 32 / V4;  // rows of a warp
  __shared__ float4 s_o[kMergeWarps][32];
  __shared__ float2 s_ml[kMergeWarps][32];
  const int b = blockIdx.z, kvh = blockIdx.y, grp = p.Hq / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Kv4Seq mine = kv4_first_seqs(p);
  const Kv4Seq seq = kv4_seq_at(p, mine, b);
  const Kv4Plan plan = kv4_plan(p, mine);
  const int n = kv4_pieces(seq.pages, plan.target);
  if (n < 2) {  // one CTA finished the group
    pdl_wait();
    return;
  }
  int before_cut = 0;  // partials of the sequences before this one
  for (int i = lane; i < b; i += 32) {
    const int k = kv4_pieces(i < 32 ? mine.pages : kv4_seq(p, i).pages, plan.target);
    if (k > 1) before_cut += k;
  }
  const int i0 = (int)__reduce_add_sync(0xffffffffu, (unsigned)before_cut) * p.Hkv + kvh * n;
  pdl_wait();
  pdl_launch_dependents();
  const int split = merge_split(n, kMergeWarps);
  const int part = warp & (split - 1), at_once = kMergeWarps / split * RPW;
  const int d4 = lane % V4, rows = seq.Wb * grp;
  for (int r0 = blockIdx.x * at_once; r0 < rows; r0 += gridDim.x * at_once) {
    const int r = r0 + warp / split * RPW + lane / V4;
    const int rr = min(r, rows - 1);
    float M = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int NB = 8;  // partials whose loads are in flight together
    for (int k0 = part; k0 < n; k0 += NB * split) {
      float ms[NB], ls[NB];
      float4 os[NB];
      float mb = M;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float* ws = kv4_partial(p.workspace, i0 + min(k0 + k * split, n - 1), ws_rows, HD);
        os[k] = *reinterpret_cast<const float4*>(ws + rr * HD + d4 * 4);
        ms[k] = ws[ws_rows * HD + rr];
        ls[k] = ws[ws_rows * HD + ws_rows + rr];
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
        float top = M;
        for (int k = 1; k < split; ++k) top = fmaxf(top, s_ml[warp + k][lane].x);
        const float a = ex2(M - top);
        l *= a;
        o.x *= a, o.y *= a, o.z *= a, o.w *= a;
#pragma unroll 4
        for (int k = 1; k < split; ++k) {
          const float2 ml = s_ml[warp + k][lane];
          const float4 x = s_o[warp + k][lane];
          const float w = ex2(ml.x - top);
          l = fmaf(w, ml.y, l);
          o.x = fmaf(w, x.x, o.x);
          o.y = fmaf(w, x.y, o.y);
          o.z = fmaf(w, x.z, o.z);
          o.w = fmaf(w, x.w, o.w);
        }
      }
      __syncthreads();
    }
    if (part == 0 && r < rows) store_row4(p, seq.row0 + r / grp, kvh * grp + r % grp, HD, d4, o, l);
  }
}

// Function attributes are per device: one bit per device once they are set there.
template <typename K>
cudaError_t configure(K kernel, int smem, bool cluster, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done.load(std::memory_order_acquire) >> (dev & 63) & 1ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  return e;
}

// Pages of a group, at most.
int hint_pages(const Kv4AttnParams& p) { return (p.kv_len_hint + kPage - 1) / kPage; }

// Short caches: the CTAs of a group as one cluster, where all clusters fit the GPU at once (14 of
// 16 CTAs, 36 of 8, 74 of 4 and 152 of 2 do with two CTAs per SM) and a CTA gets few pages: nine
// at most where the clusters fill the SMs, six where they leave some idle.  No workspace and no
// second launch.  0: not short.  Clusters against pieces, in us (8 kv heads of 128; 1, 5 and 15
// rows of 4 query heads each):
//   sequences x tokens   1 x 4096    1 x 8192   4 x 4096    8 x 2048    16 x 1024
//   pages of a CTA       4           8          8           8           8
//   1 row                 8.4,  9.7  11.0,  9.9 11.3, 11.2  11.5, 11.4  11.5, 11.3
//   5 rows               12.4, 13.5  16.7, 15.3 17.3, 20.9  17.7, 18.6  18.1, 20.0
//   15 rows              20.9, 25.7  28.2, 30.9 32.3, 36.2  33.4, 38.5
// and at 16 pages for each CTA (8 x 4096 tokens, 1 and 5 rows) 16.9, 14.5 and 26.1, 25.2.
int cluster_size(int B, int Hkv, int pages, int sm_count) {
  const long long groups = (long long)B * Hkv;
  if (pages <= 4 && groups <= (1 << 30)) return 1;
  const struct { int cs, fit; } sizes[] = {{2, 152}, {4, 74}, {8, 36}, {16, 14}};
  int cs = 0;  // the widest that fits: fewer pages for each CTA
  for (const auto& s : sizes)
    if (groups <= s.fit && pages >= s.cs) cs = s.cs;
  return pages <= (groups * cs > sm_count ? 9 : 6) * cs ? cs : 0;
}

template <int HD, int NT>
cudaError_t launch_cluster(Kv4AttnParams p, int cs, cudaStream_t st) {
  using C = Cfg<HD, NT, kWarps>;
  static std::atomic<uint64_t> done{0};
  p.stages = C::stages(2, C::kRecv);
  const int smem = C::kFixed + C::kRecv + p.stages * C::kBlock;
  cudaError_t e = configure(kv4_attention_kernel<HD, NT, kWarps, true>, smem, true, done);
  if (e != cudaSuccess) return e;
  p.cluster = cs;
  return launch_k_cluster(kv4_attention_kernel<HD, NT, kWarps, true>, dim3(p.B * p.Hkv * cs), dim3(kThreads), smem, st,
                          dim3(cs, 1, 1), p);
}

template <int HD, int NT, int TW>
cudaError_t launch_pieces(Kv4AttnParams p, cudaStream_t st) {
  using C = Cfg<HD, NT, TW>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = configure(kv4_attention_kernel<HD, NT, TW, false>, C::kFixed + C::stages(1) * C::kBlock, false, done);
  if (e != cudaSuccess) return e;
  const int pages = hint_pages(p);
  const long long groups = (long long)p.B * p.Hkv;
  const long long most = std::min<long long>(groups * pages, (long long)C::kCtas * p.sm_count);
  const int occ = (int)std::min<long long>(C::kCtas, (std::max(most, groups) + p.sm_count - 1) / p.sm_count);
  p.slots = occ * p.sm_count;
  p.stages = C::stages(occ);
  // as many CTAs as the plan can make of any lengths: the hint sets the speed, not the result
  const long long ctas = groups < p.slots ? p.slots : groups + p.slots;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  e = launch_k(kv4_attention_kernel<HD, NT, TW, false>, dim3((unsigned)ctas), dim3(kThreads),
               C::kFixed + p.stages * C::kBlock, st, p);
  if (e != cudaSuccess) return e;
  // four warps, or sixteen for groups that may have sixteen partials or more
  const int n = (int)std::max<long long>(1, p.slots / groups), rows = p.W * (p.Hq / p.Hkv);
  const auto merge = [&](auto kernel, int warps) {
    const int at_once = warps / merge_split(n, warps) * (128 / HD);
    return launch_k(kernel, dim3((rows + at_once - 1) / at_once, p.Hkv, p.B), dim3(warps * 32), 0, st, p, NT * 8);
  };
  return n >= 16 ? merge(kv4_merge_kernel<HD, 16>, 16) : merge(kv4_merge_kernel<HD, 4>, 4);
}

template <int HD, int NT>
cudaError_t launch_nt(const Kv4AttnParams& p, cudaStream_t st) {
  if (const int cs = cluster_size(p.B, p.Hkv, hint_pages(p), p.sm_count)) return launch_cluster<HD, NT>(p, cs, st);
  return launch_pieces<HD, NT, (NT <= 2 ? 1 : kWarps)>(p, st);
}

template <int HD>
cudaError_t launch_hd(const Kv4AttnParams& p, cudaStream_t st) {
  switch ((p.W * (p.Hq / p.Hkv) + 7) / 8) {
    case 1: return launch_nt<HD, 1>(p, st);
    case 2: return launch_nt<HD, 2>(p, st);
    case 3: return launch_nt<HD, 3>(p, st);
    case 4: return launch_nt<HD, 4>(p, st);
    case 5: return launch_nt<HD, 5>(p, st);
    case 6: return launch_nt<HD, 6>(p, st);
    case 7: return launch_nt<HD, 7>(p, st);
    case 8: return launch_nt<HD, 8>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// The partials of cut groups: at most two for each slot of the largest grid (4 CTAs per SM, 3
// from four row tiles on).
long long kv4_attention_workspace(int B, int Hkv, int rows, int hd, int kv_len_hint, int sm_count) {
  if (cluster_size(B, Hkv, (kv_len_hint + kPage - 1) / kPage, sm_count)) return 0;
  const int nt = (rows + 7) / 8;
  return 2ll * (nt <= 3 ? 4 : 3) * sm_count * nt * 8 * (hd + 2) * 4;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& params, cudaStream_t st) {
  Kv4AttnParams p = params;
  int e = 0;
  p.scale_m = 2.f * std::frexp(std::fabs(p.scale) * 1.4426950408889634f, &e);
  p.scale_2 = std::ldexp(1.f, std::max(e - 1, -126));
  return p.hd == 128 ? launch_hd<128>(p, st) : launch_hd<64>(p, st);
}

}  // namespace spec
