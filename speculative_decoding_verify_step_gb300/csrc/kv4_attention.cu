// Attention of the verify window over the 4-bit paged cache.
//
// For query row r (a window row and one of the query heads that share the kv head)
// and cached token k, with codes c, scale s, offset m:
//   S[r, k] = q_r . (s_k c_k + m_k) = s_k (q_r . c_k) + m_k sum(q_r)
//   O[r]    = sum_k P (s_k c_k + m_k) = sum_k (P s_k) c_k + sum_k P m_k
// so the tensor cores multiply the bare codes, and the two parameters of a token are
// applied to its score and its weight, in fp32.  Softmax is taken in one pass over
// the pages with a running maximum and sum per row.
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
// Rounding.  P s_k is rounded to fp16 (scaled by a power of two that follows the
// largest s seen, so small scales stay normal numbers).  c lies in 0..15, so that
// rounding would weigh on c's mean of 7.5 as well; the kernel sums the rounded
// weights R with one more MMA per step (A = ones) and forms
//   O = sum (P s)_fp16 c - 7.5 R + sum P (m + 7.5 s),
// which leaves only the rounding of the weights of c - 7.5.  Everything else is fp32.
//
// One CTA of four warps per (sequence, kv head, split of its pages); the splits of a
// sequence are a thread-block cluster that merges its partials through distributed
// shared memory.  A page of one kv head is one block (8704 bytes at head_dim 128)
// and one bulk copy into the ring of its warp team; a team is 1, 2 or 4 warps that
// take different 16-token steps of a page (short caches) or different query rows
// (wide windows).
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "kv4.cuh"
#include "kv4.h"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace spec {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxStages = 12;  // pages in flight per CTA

SPEC_DEVICE_INLINE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 x 8 transpose of 16-bit elements across the warp.
SPEC_DEVICE_INLINE uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

SPEC_DEVICE_INLINE void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int HD>
struct Cfg {
  static constexpr int kBlock = kPage * HD + 2 * kPage * 4;
  static constexpr int kQTile = (HD / 32) * 512;  // query fragments of 8 rows
  static constexpr int kMaxTiles = 8;             // 64 query rows
  // two CTAs per SM: 228 KB less 1 KB of system use and this kernel's static arrays each
  static constexpr int kSmemBudget = 112 * 1024;
  static constexpr int stages(int tiles) {
    const int n = (kSmemBudget - tiles * kQTile) / kBlock;
    return n < kMaxStages ? n : kMaxStages;
  }
};

// Query row r of the CTA is window row r / grp, head r % grp of the group.
// HD: head_dim; NT: tiles of 8 query rows per warp; KG: warps that share a page's keys.
template <int HD, int NT, int KG>
__global__ void __launch_bounds__(kThreads, 2) kv4_attention_kernel(const __grid_constant__ Kv4AttnParams p) {
  using C = Cfg<HD>;
  constexpr int MT = 4 / KG;        // 16-token steps of a page per warp
  constexpr int WORDS = HD / 32;    // 32-bit words of K codes per lane and token
  constexpr int DM = HD / 16;       // 16-row tiles of the PV product
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ float s_sumq[64], s_f[64];
  __shared__ uint32_t s_anc[16];
  __shared__ float s_m[64], s_l[64];
  __shared__ float part_m[kWarps * 32], part_l[kWarps * 32];
  __shared__ int s_fail;
  cg::cluster_group cluster = cg::this_cluster();

  const int rank = blockIdx.x, CS = gridDim.x, kvh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int NG = p.row_tiles / NT;          // row groups (row_tiles is a multiple of NT)
  const int TW = KG * NG;                   // warps of a team
  const int teams = kWarps / TW;
  const int team = warp / TW, kg = warp % KG, ng = (warp % TW) / KG;
  const int S = p.stages;                   // ring depth of a team
  const int grp = p.Hq / p.Hkv;

  pdl_launch_dependents();
  if (!p.early) pdl_wait();
  const int b = p.seq_order ? p.seq_order[blockIdx.z] : blockIdx.z;
  const int sid = p.seq_ids ? p.seq_ids[b] : b;
  int row0 = p.row_begin ? p.row_begin[b] : b * p.W;
  int Wb = p.row_count ? p.row_count[b] : p.row_begin ? p.row_begin[b + 1] - row0 : p.W;
  row0 = max(0, min(row0, p.total_rows));
  Wb = max(0, min(min(Wb, p.W), p.total_rows - row0));
  const bool sid_ok = sid >= 0 && sid < p.table_rows;
  const int cap = p.max_pages * kPage;
  const int L = max(0, min(p.kv_len[b], cap));
  const int n_keys = sid_ok && Wb > 0 ? min(L + Wb, cap) : 0;
  const int rows = Wb * grp;
  const int n_pages = (n_keys + kPage - 1) / kPage;
  const int pps = (n_pages + CS - 1) / CS;
  const int pg0 = min(rank * pps, n_pages);
  const int npg = min(pg0 + pps, n_pages) - pg0;
  const int n_it = npg > team ? (npg - team + teams - 1) / teams : 0;  // pages of this team

  uint8_t* const ring = smem + team * S * C::kBlock;
  uint64_t* const fullb = full + team * S;
  uint64_t* const emptyb = empty + team * S;
  uint8_t* const qfrag = smem + kWarps / TW * S * C::kBlock;
  if (threadIdx.x == 0) {
    for (int s = 0; s < teams * S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], TW);
    }
    s_fail = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 16) s_anc[threadIdx.x] = p.anc[threadIdx.x];
  __syncthreads();

  // Page numbers of iterations [i0, i0 + 32) and the 32 after them, one per lane.
  const int32_t* table = p.page_table + (long long)(sid_ok ? sid : 0) * p.max_pages;
  auto page_at = [&](int i) {
    const int pg = i < n_it ? table[pg0 + i * teams + team] : -1;
    return pg < p.num_pages ? pg : -1;
  };
  int pid0 = page_at(lane), pid1 = page_at(32 + lane);
  int base = 0;
  auto pid = [&](int i) {  // base <= i < base + 64, the same in all lanes
    const int a = __shfl_sync(0xffffffffu, pid0, i & 31), d = __shfl_sync(0xffffffffu, pid1, i & 31);
    return i - base < 32 ? a : d;
  };
  // Start the copy of iteration i's block (an absent page completes its phase empty).
  auto issue = [&](int i, int s) {
    const int pg = pid(i);
    if (lane == 0) {
      if (pg >= 0) {
        mbar_arrive_expect_tx(&fullb[s], C::kBlock);
        bulk_load(ring + s * C::kBlock, p.pool + ((long long)pg * p.Hkv + kvh) * C::kBlock, C::kBlock, &fullb[s]);
      } else {
        mbar_arrive(&fullb[s]);
      }
    }
  };
  const bool leader = warp % TW == 0;
  // Before pdl_wait only pages without window slots may be read.
  int issued = 0;
  if (leader) {
    for (; issued < min(S, n_it); ++issued) {
      if (p.early && (pg0 + issued * teams + team + 1) * kPage > L) break;
      issue(issued, issued);
    }
  }
  if (p.early) pdl_wait();
  if (leader)
    for (; issued < min(S, n_it); ++issued) issue(issued, issued);

  // Queries: each row is scaled by a power of two (largest element in [2^14, 2^15)),
  // so the factor 1/16 of the odd columns costs no precision; the sum of the scaled
  // row and the factor back to exp2 units are kept per row.  One warp per row.
  {
    constexpr int PER = HD / 32;  // elements of a lane
    for (int r = warp; r < p.row_tiles * 8; r += kWarps) {
      float x[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] = 0.f;
      if (r < rows) {
        const uint16_t* qr = static_cast<const uint16_t*>(p.q) + (row0 + r / grp) * p.q_row_stride +
                             (long long)(kvh * grp + r % grp) * HD + lane * PER;
        const uint32_t* q2 = reinterpret_cast<const uint32_t*>(qr);
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
          const float2 f = p.bf16 ? kv4_unpack2<true>(q2[i]) : kv4_unpack2<false>(q2[i]);
          x[2 * i] = kv4_sat(f.x);
          x[2 * i + 1] = kv4_sat(f.y);
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) mx = fmaxf(mx, fabsf(x[i]));
      mx = warp_max(mx);
      // 2^sh with 2^14 <= mx 2^sh < 2^15; rows below 2^-40 count as zeros
      const int sh = mx > 9.1e-13f ? 14 - (int)((__float_as_uint(mx) >> 23) - 127u) : 0;
      const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        x[i] *= p.scale < 0.f ? -up : up;
        sum += x[i];
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        s_sumq[r] = sum * 5.9604644775390625e-8f;  // in the units of the code products (2^-24)
        s_f[r] = fmaxf(fabsf(p.scale) * 1.4426950408889634f * 16777216.f * __uint_as_float((uint32_t)(127 - sh) << 23),
                       1e-30f);
      }
      // fragment of lane (r % 8, cc), word w: halves (d0, d4) (d1, d5)/16 (d2, d6) (d3, d7)/16
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int d = lane * PER + i;
        const int cc = d / (HD / 4), w = (d % (HD / 4)) / 8, n = d % 8;
        __half* dst = reinterpret_cast<__half*>(qfrag + (r >> 3) * C::kQTile + (w * 32 + (r & 7) * 4 + cc) * 16);
        dst[(n & 3) * 2 + (n >> 2)] = __float2half_rn((n & 1) ? x[i] * 0.0625f : x[i]);
      }
    }
  }
  __syncthreads();

  float acc[NT][DM][4], accr[NT][4];
  float mrow[NT][2], lrow[NT][2], zrow[NT][2], sq[NT][2], fr[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < DM; ++t) acc[nt][t][0] = acc[nt][t][1] = acc[nt][t][2] = acc[nt][t][3] = 0.f;
    accr[nt][0] = accr[nt][1] = accr[nt][2] = accr[nt][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = (ng * NT + nt) * 8 + 2 * c + e;
      mrow[nt][e] = -INFINITY;
      lrow[nt][e] = zrow[nt][e] = 0.f;
      sq[nt][e] = s_sumq[r];
      fr[nt][e] = s_f[r];
    }
  }
  uint32_t smax = 0;      // largest V scale so far (its word), and 2^-exponent of it
  float inv_e = 1.f;

  int s = 0;
  uint32_t par = 0;
  for (int i = 0; i < n_it; ++i) {
    if (i - base == 32) {
      base = i;
      pid0 = pid1;
      pid1 = page_at(base + 32 + lane);
    }
    const int pg = pid(i);
    if (!mbar_wait(&fullb[s], par, p.status)) {
      s_fail = 1;
      break;
    }
    if (pg >= 0) {
      const uint8_t* st = ring + s * C::kBlock;
      const int key0 = (pg0 + i * teams + team) * kPage;
      const bool masked = key0 + kPage > L;

      // parameter words of this lane's tokens: 16-token step t, tokens g and g + 8
      uint32_t kw[2 * MT], vw[2 * MT];
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(st + kPage * HD);
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        const int k = (kg * MT + (t >> 1)) * 16 + (t & 1) * 8 + g;
        kw[t] = kpar[k];
        vw[t] = kpar[kPage + k];
        if (masked && key0 + k >= n_keys) kw[t] = vw[t] = 0;  // never written: may hold anything
      }
      // K codes
      uint32_t kc[2 * MT][WORDS];
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        const int k = (kg * MT + (t >> 1)) * 16 + (t & 1) * 8 + g;
        const uint8_t* a = st + k * (HD / 2) + c * (HD / 8);
        if constexpr (WORDS == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(a);
          kc[t][0] = v.x, kc[t][1] = v.y, kc[t][2] = v.z, kc[t][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(a);
          kc[t][0] = v.x, kc[t][1] = v.y;
        }
      }
      // S = codes . q, then s (.) + m sum(q)
      float sc[NT][MT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int t = 0; t < MT; ++t) sc[nt][t][0] = sc[nt][t][1] = sc[nt][t][2] = sc[nt][t][3] = 0.f;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        uint4 qf[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          qf[nt] = *reinterpret_cast<const uint4*>(qfrag + (ng * NT + nt) * C::kQTile + (w * 32 + lane) * 16);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint32_t x0 = kc[2 * t][w], x1 = kc[2 * t + 1][w];
          const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(sc[nt][t], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qf[nt].x,
                          qf[nt].y);
            mma_f16_16816(sc[nt][t], y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qf[nt].z,
                          qf[nt].w);
          }
        }
      }
      // largest V scale: 2^-E keeps P s below 2 and, for the larger scales, normal
      float rescale_e = 1.f;
      {
        uint32_t mx = 0;
#pragma unroll
        for (int t = 0; t < 2 * MT; ++t) mx = max(mx, vw[t]);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if ((mx >> 16) > smax) {
          smax = mx >> 16;
          const uint32_t e = __float_as_uint(__half2float(__ushort_as_half((unsigned short)smax))) >> 23;
          const float now = __uint_as_float((254u - e) << 23);
          rescale_e = now / inv_e;
          inv_e = now;
        }
      }
      float vs[2 * MT], vz[2 * MT];
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        const float2 kmv = __half22float2(*reinterpret_cast<const __half2*>(&kw[t]));
        const float2 vmv = __half22float2(*reinterpret_cast<const __half2*>(&vw[t]));
        vs[t] = vmv.y * inv_e;
        vz[t] = fmaf(7.5f, vmv.y, vmv.x);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[nt][t >> 1][(t & 1) * 2 + e];
            x = fmaf(kmv.y, x, kmv.x * sq[nt][e]);
          }
      }
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = (ng * NT + nt) * 8 + 2 * c + e;
            const uint32_t anc = r < rows ? s_anc[r / grp] & ((1u << Wb) - 1u) : 0u;
#pragma unroll
            for (int t = 0; t < 2 * MT; ++t) {
              const int w = key0 + (kg * MT + (t >> 1)) * 16 + (t & 1) * 8 + g - L;
              const bool vis = w < 0 || (w < 16 && ((anc >> w) & 1u) && w + L < n_keys);
              if (!vis) sc[nt][t >> 1][(t & 1) * 2 + e] = -INFINITY;
            }
          }
      }
      // running maximum and sum; weights into fp16 B fragments
      uint32_t pb[NT][2 * MT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = sc[nt][0][e];
#pragma unroll
          for (int t = 1; t < 2 * MT; ++t) mx = fmaxf(mx, sc[nt][t >> 1][(t & 1) * 2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float now = fmaxf(mrow[nt][e], mx * fr[nt][e]);
          alpha[e] = mrow[nt][e] == now ? 1.f : ex2(mrow[nt][e] - now);
          mrow[nt][e] = now;
        }
        const float off0 = mrow[nt][0] == -INFINITY ? 0.f : mrow[nt][0];
        const float off1 = mrow[nt][1] == -INFINITY ? 0.f : mrow[nt][1];
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f) || rescale_e != 1.f) {
          const float a0 = alpha[0] * rescale_e, a1 = alpha[1] * rescale_e;
#pragma unroll
          for (int t = 0; t < DM; ++t) {
            acc[nt][t][0] *= a0;
            acc[nt][t][1] *= a1;
            acc[nt][t][2] *= a0;
            acc[nt][t][3] *= a1;
          }
          accr[nt][0] *= a0;
          accr[nt][1] *= a1;
          lrow[nt][0] *= alpha[0];
          lrow[nt][1] *= alpha[1];
          zrow[nt][0] *= alpha[0];
          zrow[nt][1] *= alpha[1];
        }
#pragma unroll
        for (int t = 0; t < 2 * MT; ++t) {
          const float p0 = ex2(fmaf(sc[nt][t >> 1][(t & 1) * 2], fr[nt][0], -off0));
          const float p1 = ex2(fmaf(sc[nt][t >> 1][(t & 1) * 2 + 1], fr[nt][1], -off1));
          lrow[nt][0] += p0;
          lrow[nt][1] += p1;
          zrow[nt][0] = fmaf(p0, vz[t], zrow[nt][0]);
          zrow[nt][1] = fmaf(p1, vz[t], zrow[nt][1]);
          pb[nt][t] = movmatrix_trans(pack_f16x2(p0 * vs[t], p1 * vs[t]));
        }
      }
      // O^T += codes^T . weights
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int step = kg * MT + t;
        const uint8_t* vbase = st + kPage * HD / 2 + ((g ^ (2 * c)) << 4);
        uint32_t lo[HD / 32], hi[HD / 32];  // pieces of tokens {2c, 2c+1} and {2c+8, 2c+9}
        if constexpr (HD == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(vbase + (step * 8 + c) * 128);
          const uint4 d = *reinterpret_cast<const uint4*>(vbase + (step * 8 + 4 + c) * 128);
          lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w;
          hi[0] = d.x, hi[1] = d.y, hi[2] = d.z, hi[3] = d.w;
        } else {
          const uint4 a = *reinterpret_cast<const uint4*>(vbase + (step * 4 + c) * 128);
          lo[0] = a.x, lo[1] = a.y;
          hi[0] = a.z, hi[1] = a.w;
        }
#pragma unroll
        for (int w = 0; w < HD / 32; ++w) {
          const uint32_t x0 = lo[w], x1 = hi[w], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(acc[nt][2 * w], x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu, x1 & 0x00f000f0u,
                          pb[nt][2 * t], pb[nt][2 * t + 1]);
            mma_f16_16816(acc[nt][2 * w + 1], y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu, y1 & 0x00f000f0u,
                          pb[nt][2 * t], pb[nt][2 * t + 1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16_16816(accr[nt], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pb[nt][2 * t], pb[nt][2 * t + 1]);
      }
    }
    // The stage is refilled through the async proxy: order this warp's reads before it.
    fence_proxy_async();
    __syncwarp();
    if (TW == 1) {
      if (i + S < n_it) issue(i + S, s);
    } else {
      if (lane == 0) mbar_arrive(&emptyb[s]);
      // the team's first warp refills the stage of the page before, which the others
      // have usually left by now
      if (leader && i > 0 && i - 1 + S < n_it) {
        const int ps = s == 0 ? S - 1 : s - 1;
        const uint32_t pp = s == 0 ? par ^ 1u : par;
        if (!mbar_wait(&emptyb[ps], pp, p.status)) {
          s_fail = 1;
          break;
        }
        issue(i - 1 + S, ps);
      }
    }
    if (++s == S) {
      s = 0;
      par ^= 1u;
    }
  }
  __syncthreads();
  if (s_fail && threadIdx.x < teams * S) {
    // a wait ran out: give copies still in flight the same time to land before the
    // CTA's shared memory is given up
    (void)mbar_wait(&full[threadIdx.x], 0, nullptr);
    (void)mbar_wait(&full[threadIdx.x], 1, nullptr);
  }

  // Partials of every warp (the ring is drained): out-of-loop order is
  // [key partial][row][HD], with NP = kWarps / NG partials per row.
  const int NP = kWarps / NG;
  const int n_rows8 = p.row_tiles * 8;
  float* part_o = reinterpret_cast<float*>(smem);
  {
    const int np = team * KG + kg;
    const float e_up = 1.f / inv_e;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[nt][e], z = zrow[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, o);
          z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        const int r = (ng * NT + nt) * 8 + 2 * c + e;
        const float bias = z - 7.5f * e_up * accr[nt][e];
        float* o = part_o + ((long long)np * n_rows8 + r) * HD + g * (HD / 8);
#pragma unroll
        for (int t = 0; t < DM; t += 2)
          *reinterpret_cast<float4*>(o + 2 * t) =
              make_float4(fmaf(acc[nt][t][e], e_up * 16777216.f, bias), fmaf(acc[nt][t][2 + e], e_up * 1048576.f, bias),
                          fmaf(acc[nt][t + 1][e], e_up * 16777216.f, bias),
                          fmaf(acc[nt][t + 1][2 + e], e_up * 1048576.f, bias));
        if (g == 0) {
          part_m[np * n_rows8 + r] = mrow[nt][e];
          part_l[np * n_rows8 + r] = l;
        }
      }
    }
  }
  __syncthreads();
  // merge the CTA's partials into the first; out = sum_i 2^(m_i - M) o_i, the same for l
  constexpr int V4 = HD / 4;
  for (int it = threadIdx.x; it < rows * V4; it += kThreads) {
    const int r = it / V4, d4 = it % V4;
    float M = -INFINITY;
    for (int i = 0; i < NP; ++i) M = fmaxf(M, part_m[i * n_rows8 + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int i = 0; i < NP; ++i) {
      const float m = part_m[i * n_rows8 + r];
      const float w = m == -INFINITY ? 0.f : ex2(m - M);
      const float4 x = *reinterpret_cast<const float4*>(part_o + ((long long)i * n_rows8 + r) * HD + d4 * 4);
      if (w != 0.f) {
        o.x = fmaf(w, x.x, o.x);
        o.y = fmaf(w, x.y, o.y);
        o.z = fmaf(w, x.z, o.z);
        o.w = fmaf(w, x.w, o.w);
        l = fmaf(w, part_l[i * n_rows8 + r], l);
      }
    }
    *reinterpret_cast<float4*>(part_o + (long long)r * HD + d4 * 4) = o;
    if (d4 == 0) {
      s_m[r] = M;
      s_l[r] = l;
    }
  }
  if (CS > 1) cluster.sync();
  else __syncthreads();
  // the cluster's CTAs share the rows
  if (!s_fail) {
    const uint32_t o_base = smem_u32(part_o), m_base = smem_u32(s_m), l_base = smem_u32(s_l);
    const int n_my = rows > rank ? (rows - rank + CS - 1) / CS : 0;
    for (int it = threadIdx.x; it < n_my * V4; it += kThreads) {
      const int r = rank + it / V4 * CS, d4 = it % V4;
      float M = -INFINITY;
      float ms[16], ls[16];
      float4 os[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < CS) {
          ms[i] = ld_dsmem_f32(mapa_u32(m_base + r * 4, i));
          ls[i] = ld_dsmem_f32(mapa_u32(l_base + r * 4, i));
          os[i] = ld_dsmem_f4(mapa_u32(o_base + (r * HD + d4 * 4) * 4, i));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < CS) M = fmaxf(M, ms[i]);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < CS && ms[i] != -INFINITY) {
          const float w = ex2(ms[i] - M);
          l = fmaf(w, ls[i], l);
          o.x = fmaf(w, os[i].x, o.x);
          o.y = fmaf(w, os[i].y, o.y);
          o.z = fmaf(w, os[i].z, o.z);
          o.w = fmaf(w, os[i].w, o.w);
        }
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;  // a row that sees no token is zeros
      uint2 w2;
      if (p.bf16) {
        w2.x = kv4_pack2<true>(o.x * inv, o.y * inv);
        w2.y = kv4_pack2<true>(o.z * inv, o.w * inv);
      } else {
        w2 = pack_act4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      }
      uint16_t* dst = static_cast<uint16_t*>(p.out) +
                      ((long long)(row0 + r / grp) * p.Hq + kvh * grp + r % grp) * HD + d4 * 4;
      *reinterpret_cast<uint2*>(dst) = w2;
    }
  }
  if (CS > 1) cluster.sync();  // keep this CTA's shared memory until every CTA has read it
}

// Function attributes are per device: one bit per device once they are set there.
template <typename K>
cudaError_t configure(K kernel, int smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done.load(std::memory_order_acquire) >> (dev & 63) & 1ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_release);
  return e;
}

template <int HD, int NT, int KG>
cudaError_t launch_kg(Kv4AttnParams p, int ng, int cs, cudaStream_t st) {
  using C = Cfg<HD>;
  const int teams = kWarps / (KG * ng);
  p.row_tiles = NT * ng;
  p.stages = C::stages(p.row_tiles) / teams;
  const int smem = teams * p.stages * C::kBlock + p.row_tiles * C::kQTile;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = configure(kv4_attention_kernel<HD, NT, KG>, C::kSmemBudget, done);
  if (e != cudaSuccess) return e;
  return launch_k_cluster(kv4_attention_kernel<HD, NT, KG>, dim3(cs, p.Hkv, p.B), dim3(kThreads),
                          smem, st, dim3(cs, 1, 1), p);
}

template <int HD>
cudaError_t launch_hd(const Kv4AttnParams& p, cudaStream_t st) {
  const int tiles = (p.W * (p.Hq / p.Hkv) + 7) / 8;
  if (tiles < 1 || tiles > Cfg<HD>::kMaxTiles) return cudaErrorInvalidValue;
  // The widest cluster whose grid fits two CTAs per SM.
  int cs = 16;
  while (cs > 1 && p.B * p.Hkv * cs > 2 * p.sm_count) cs >>= 1;
  const int pages = (p.kv_len_hint + kPage - 1) / kPage;
  const int per_cta = (pages + cs - 1) / cs;
  const bool few = per_cta < 8;  // too few pages for four independent teams
  switch (tiles) {
    case 1: return few ? launch_kg<HD, 1, 4>(p, 1, cs, st) : launch_kg<HD, 1, 1>(p, 1, cs, st);
    case 2: return few ? launch_kg<HD, 2, 4>(p, 1, cs, st) : launch_kg<HD, 2, 1>(p, 1, cs, st);
    case 3: return few ? launch_kg<HD, 3, 4>(p, 1, cs, st) : launch_kg<HD, 3, 1>(p, 1, cs, st);
    case 4: return few ? launch_kg<HD, 2, 2>(p, 2, cs, st) : launch_kg<HD, 2, 1>(p, 2, cs, st);
    case 5:
    case 6: return few ? launch_kg<HD, 3, 2>(p, 2, cs, st) : launch_kg<HD, 3, 1>(p, 2, cs, st);
    default: return launch_kg<HD, 2, 1>(p, 4, cs, st);
  }
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, cudaStream_t st) {
  return p.hd == 128 ? launch_hd<128>(p, st) : launch_hd<64>(p, st);
}

}  // namespace spec
